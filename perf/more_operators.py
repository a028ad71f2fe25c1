"""The operators of the INT8 expert path and of routing in training, as they are
measured: cases, inputs, the plain forms in elementary torch operations and the
library's calls.

  quantize   int8_quantize: bf16 rows to int8 with one fp32 scale per row
             (tokens, or a weight's output channels)
  linear     int8_linear: the product of int8 rows with scales for each token
             and channel, with bias, activation and residual in its epilogue
  experts    gmm_int8: the same product over rows sorted by expert, each with
             its expert's weights, plain or with SwiGLU
  permute    moe_permute: token rows sorted by expert
  unpermute  moe_unpermute and moe_unpermute_backward: expert rows back to
             their tokens with the routing weights, and the gradients of both
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8}


def listed():
    return [
        # one token of a decode step, before its projection
        {"name": "quantize 1 token", "op": "quantize", "rows": 1, "K": 4096},
        # prefill activations before a product (or an expert's weights at load time)
        {"name": "quantize 16K tokens", "op": "quantize", "rows": 16384, "K": 2048},
        # one token through a projection with a bias, unquantised input
        {"name": "linear 1 token", "op": "linear", "T": 1, "K": 2048, "N": 4096, "x": "bf16", "bias": "fp32",
         "act": "none", "residual": False},
        # a short prompt, a width that no tile divides and a reduction that no stage divides
        {"name": "linear ragged", "op": "linear", "T": 203, "K": 2096, "N": 4099, "x": "int8", "bias": "bf16",
         "act": "gelu", "residual": True},
        # prefill through an output projection that adds to the residual stream
        {"name": "linear 16K tokens", "op": "linear", "T": 16384, "K": 4096, "N": 4096, "x": "int8", "bias": "none",
         "act": "none", "residual": True},
        # decode: 32 tokens, 8 of 128 experts each, gate and up projections
        {"name": "experts 32 tokens", "op": "experts", "T": 32, "k": 8, "E": 128, "K": 2048, "N": 768,
         "swiglu": True, "spread": "even"},
        # prefill, gate and up projections
        {"name": "experts 16K tokens", "op": "experts", "T": 16384, "k": 8, "E": 128, "K": 2048, "N": 768,
         "swiglu": True, "spread": "even"},
        # decode: int8 rows and their scales to the experts
        {"name": "permute 32 tokens", "op": "permute", "T": 32, "K": 2048, "k": 8, "E": 128, "x": "int8",
         "spread": "even", "padded": False},
        # a training batch
        {"name": "permute 16K tokens", "op": "permute", "T": 16384, "K": 2048, "k": 8, "E": 128, "x": "bf16",
         "spread": "even", "padded": False},
        # an odd width, a few crowded experts, some assignments dropped
        {"name": "unpermute 2049 tokens", "op": "unpermute", "T": 2049, "K": 1001, "k": 8, "E": 64, "y": "fp16",
         "weighted": True, "spread": "zipf", "dropped": 0.02, "gradient": False},
        # the backward pass of a small batch
        {"name": "unpermute 64 tokens gradient", "op": "unpermute", "T": 64, "K": 4096, "k": 2, "E": 8, "y": "bf16",
         "weighted": True, "spread": "even", "dropped": 0.0, "gradient": True},
        # the backward pass of a training batch
        {"name": "unpermute 16K tokens gradient", "op": "unpermute", "T": 16384, "K": 2048, "k": 8, "E": 128,
         "y": "bf16", "weighted": True, "spread": "even", "dropped": 0.0, "gradient": True},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "experts", "experts", "permute", "unpermute", "unpermute"])
    if op == "quantize":
        K = _spread(rng, 64, 16384)
        K -= K % rng.choice([1, 8, 16])
        return {"op": op, "rows": _spread(rng, 1, min(16384, 16384 * 2048 // K)), "K": K}
    if op == "linear":
        K = 16 * _spread(rng, 8, 512)
        K -= K % rng.choice([16, 128, 128])
        N = _spread(rng, 64, 8192)
        N = max(64, N - N % rng.choice([1, 8, 32, 256]))
        T = _spread(rng, 1, min(16384, 16384 * 4096 * 4096 // (K * N), 16384 * 4096 // N))
        return {"op": op, "T": T, "K": K, "N": N, "x": rng.choice(["bf16", "int8", "int8"]),
                "bias": rng.choice(["none", "bf16", "fp32"]),
                "act": rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]),
                "residual": rng.random() < 0.5}
    E = rng.choice([8, 16, 60, 64, 128])
    k = rng.randint(1, 8)
    spread = rng.choice(["even", "even", "zipf"])
    if op == "experts":
        swiglu = rng.random() < 0.5
        K = 16 * _spread(rng, 8, 256)
        K -= K % rng.choice([16, 128, 128])
        most = 128 * 1536 * 2048 // (E * K)            # output features that the largest listed weights have
        N = _spread(rng, 32, min(4096, most) // (1 + swiglu))
        N = max(32, N - N % rng.choice([1, 8, 32, 64]))
        cost = K * N * (1 + swiglu) * k
        T = _spread(rng, 1, min(16384 if spread == "even" else 2048, 16384 * 8 * 2048 * 1536 // cost))
        return {"op": op, "T": T, "k": k, "E": E, "K": K, "N": N, "swiglu": swiglu, "spread": spread}
    K = _spread(rng, 64, 8192)
    K -= K % rng.choice([1, 8, 32, 32])
    if op == "permute":
        x = rng.choice(["bf16", "bf16", "fp16", "fp32", "int8"])
        T = _spread(rng, 1, min(16384, 16384 * 8 * 2048 // (2 * K * k)))
        return {"op": op, "T": T, "K": K, "k": k, "E": E, "x": x, "spread": spread, "padded": rng.random() < 0.3}
    gradient = rng.random() < 0.6
    T = _spread(rng, 1, min(16384, 16384 * 8 * 2048 // (2 * K * k)))
    return {"op": op, "T": T, "K": K, "k": k, "E": E, "y": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
            "weighted": rng.random() < 0.7, "spread": spread, "dropped": rng.choice([0.0, 0.0, 0.05]),
            "gradient": gradient}


# ---- inputs -------------------------------------------------------------------------

def _activations(shape, gen):
    """N(0, 1) with 1 % of the channels twenty times as large, bf16."""
    x = torch.randn(shape, generator=gen, device="cuda")
    hot = torch.randperm(shape[1], generator=gen, device="cuda")[: -(-shape[1] // 100)]
    x[:, hot] *= 20
    return x.bfloat16()


def _routes(case, gen):
    """Each token's k experts, [T, k] int32."""
    T, k, E = case["T"], case["k"], case["E"]
    logits = torch.randn((T, E), generator=gen, device="cuda")
    if case["spread"] == "zipf":
        logits -= 1.1 * torch.log(torch.arange(1, E + 1, device="cuda"))[torch.randperm(E, generator=gen, device="cuda")]
    return torch.topk(logits, k, dim=1).indices.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, scale=1.0, shift=0.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale + shift

    def buffer(shape, dtype):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    st = dict(case)
    op = case["op"]
    if op == "quantize":
        st["x"] = _activations((case["rows"], case["K"]), gen)
        st["to"] = buffer((case["rows"], case["K"]), torch.int8), buffer(case["rows"], torch.float32)
        return st
    T, K = case["T"], case["K"]
    if op == "linear":
        N = case["N"]
        x = _activations((T, K), gen)
        st["x"], st["xs"] = (x, None) if case["x"] == "bf16" else _int8_quantise(x)
        st["w"], st["ws"] = _int8_quantise(normal((N, K), 0.02).bfloat16())
        b = normal((N,), 0.5)
        st["b"] = {"none": None, "bf16": b.bfloat16(), "fp32": b}[case["bias"]]
        st["r"] = normal((T, N), 2.0).bfloat16() if case["residual"] else None
        st["to"] = buffer((T, N), torch.bfloat16)
        return st
    E, k = case["E"], case["k"]
    M = T * k
    ids = _routes(case, gen)
    if op == "experts":
        rows = case["N"] * (2 if case["swiglu"] else 1)
        st["count"] = torch.bincount(ids.reshape(-1), minlength=E)
        st["most"] = int(st["count"].max())
        st["x"], st["xs"] = _int8_quantise(_activations((M, K), gen))
        w, ws = _int8_quantise(normal((E * rows, K), 0.02).bfloat16())
        st["w"], st["ws"] = w.view(E, rows, K), ws.view(E, rows)
        st["to"] = buffer((M, case["N"]), torch.bfloat16)
    elif op == "permute":
        x = _activations((T, K), gen)
        st["x"], st["xs"] = _int8_quantise(x) if case["x"] == "int8" else (x.to(DTYPES[case["x"]]), None)
        if case["padded"]:   # the batch's last eighth holds no tokens
            ids[T - T // 8:] = -1
        st["ids"] = ids
        st["to"] = (buffer((M, K), DTYPES[case["x"]]), buffer(M, torch.float32) if case["x"] == "int8" else None,
                    buffer(M, torch.int32), buffer(M, torch.int32), buffer(E, torch.int64))
    else:
        place = torch.empty(M, dtype=torch.int32, device="cuda")
        place[torch.argsort(ids.reshape(-1), stable=True)] = torch.arange(M, dtype=torch.int32, device="cuda")
        place[torch.rand(M, generator=gen, device="cuda") < case["dropped"]] = -1
        st["place"] = place
        dtype = DTYPES[case["y"]]
        st["y"] = normal((M, K), 0.5).to(dtype)
        st["w"] = torch.softmax(normal((T, k)), dim=1) if case["weighted"] else None
        if case["gradient"]:
            st["d"] = normal((T, K)).to(dtype)
            st["to"] = buffer((M, K), dtype), buffer((T, k), torch.float32) if case["weighted"] else None
        else:
            st["to"] = buffer((T, K), dtype)
    return st


# ---- the plain forms ----------------------------------------------------------------

def _int8_quantise(x):
    """[R, K] -> int8 [R, K] and fp32 scales [R]: largest magnitude / 127 (2^-126 at least)."""
    v = x.float()
    s = (v.abs().amax(dim=1) * (1 / 127)).clamp(min=2.0 ** -126)
    r = torch.ones_like(s) / s
    return torch.round(v * r[:, None]).to(torch.int8), s


def _activate(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_quantize(st):
    return _int8_quantise(st["x"])


def _plain_linear(st):
    x, xs = (st["x"], st["xs"]) if st["xs"] is not None else _int8_quantise(st["x"])
    z = x.float() @ st["w"].float().T * xs[:, None] * st["ws"]
    if st["b"] is not None:
        z = z + st["b"].float()
    z = _activate(z, st["act"])
    if st["r"] is not None:
        z = z + st["r"].float()
    return z.bfloat16()


def _plain_experts(st):
    # each expert's rows padded to the largest expert's count, one batched product, the padding left out
    M, E, N = st["x"].shape[0], st["E"], st["N"]
    end = st["count"].cumsum(0)
    first = end - st["count"]
    place = (first[:, None] + torch.arange(st["most"], device="cuda")).clamp(max=M - 1)
    z = torch.bmm(st["w"].float(), st["x"].float()[place].transpose(1, 2).contiguous())   # [E, rows, most]
    row = torch.arange(M, device="cuda")
    expert = torch.searchsorted(end, row, right=True)
    z = z.transpose(1, 2)[expert, row - first[expert]]
    z = z * st["xs"][:, None] * st["ws"][expert]
    if st["swiglu"]:
        g, u = z[:, :N], z[:, N:]
        z = g / (1 + torch.exp(-g)) * u
    return z.bfloat16()


def _plain_permute(st):
    ids = st["ids"].reshape(-1)
    M, E = ids.numel(), st["E"]
    order = torch.argsort(torch.where(ids < 0, E, ids), stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(M, device="cuda")
    count = (ids[:, None] == torch.arange(E, device="cuda")).sum(dim=0)
    real = torch.arange(M, device="cuda") < count.sum()   # the rows behind the last expert's stay as they were
    token = order // st["k"]
    rows = torch.where(real[:, None], st["x"][token], 0)
    scales = None if st["xs"] is None else torch.where(real, st["xs"][token], 0)
    return rows, scales, torch.where(real, order, 0).int(), torch.where(ids < 0, -1, place).int(), count


def _plain_unpermute(st):
    T, k = st["T"], st["k"]
    kept = st["place"] >= 0
    at = st["place"].clamp(min=0)
    if not st["gradient"]:
        rows = torch.where(kept[:, None], st["y"][at].float(), 0.0).view(T, k, -1)
        if st["w"] is not None:
            rows = rows * st["w"][:, :, None]
        return rows.sum(dim=1).to(st["y"].dtype)
    d = st["d"].float().repeat_interleave(k, dim=0)
    dw = None
    if st["w"] is not None:
        dw = torch.where(kept, (d * st["y"][at].float()).sum(dim=1), 0.0).view(T, k)
        d = d * st["w"].view(-1, 1)
    M = st["y"].shape[0]
    dy = torch.zeros((M + 1, d.shape[1]), device="cuda")
    dy[torch.where(kept, at, M)] = d
    return dy[:M].to(st["y"].dtype), dw


def run(st):
    op = st["op"]
    if own:
        import mxfp8_block_scaled_topk_amd as mx
        if op == "quantize":
            got = mx.int8_quantize(st["x"], out=st["to"])
        elif op == "linear":
            got = mx.int8_linear(st["x"], st["w"], st["ws"], x_s=st["xs"], bias=st["b"], act=st["act"],
                                 residual=st["r"], out=st["to"])
        elif op == "experts":
            got = mx.gmm_int8(st["x"], st["xs"], st["w"], st["ws"], st["count"], swiglu=st["swiglu"], out=st["to"])
        elif op == "permute":
            got = mx.moe_permute(st["x"], st["ids"], st["E"], x_s=st["xs"], out=st["to"])
        elif st["gradient"]:
            got = mx.moe_unpermute_backward(st["d"], st["place"], st["k"], topk_w=st["w"],
                                            y=st["y"] if st["w"] is not None else None, out=st["to"])
        else:
            got = mx.moe_unpermute(st["y"], st["place"], st["k"], topk_w=st["w"], out=st["to"])
    else:
        got = {"quantize": _plain_quantize, "linear": _plain_linear, "experts": _plain_experts,
               "permute": _plain_permute, "unpermute": _plain_unpermute}[op](st)
    return _named(st, got)


def _named(st, got):
    op = st["op"]
    if op in ("linear", "experts") or (op == "unpermute" and not st["gradient"]):
        return {"y": got}
    names = {"quantize": ("q", "s"), "permute": ("rows", "scales", "sorted_row", "expanded_row_idx", "group_list"),
             "unpermute": ("dy", "dw")}[op]
    return dict(zip(names, got))


# ---- the definitions in 64 bits -----------------------------------------------------

def _exact_quantize(st):
    """The scale and its reciprocal are fp32 by definition; everything between their roundings in 64 bits."""
    x = st["x"].double()
    s = (x.abs().max(dim=1).values * torch.tensor(1 / 127, dtype=torch.float32).double()).float().double()
    s = torch.maximum(s, torch.tensor(2.0 ** -126, dtype=torch.float64, device="cuda"))
    r = s.reciprocal().float().double()
    return (x * r[:, None]).float().double().round().to(torch.int8), s


def _exact_linear(st):
    x, xs = (st["x"], st["xs"].double()) if st["xs"] is not None else _exact_quantize(st)
    z = torch.mm(x.double(), st["w"].double().T.contiguous())
    z *= xs[:, None] * st["ws"].double()[None, :]
    if st["b"] is not None:
        z += st["b"].double()
    act = st["act"]
    if act == "relu":
        z = torch.where(z > 0, z, 0.0)
    elif act == "silu":
        z = z * torch.sigmoid(z)
    elif act == "gelu":
        z = z * torch.special.ndtr(z)
    elif act == "gelu_tanh":
        z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3)))
    return z + st["r"].double() if st["r"] is not None else z


def _exact_experts(st):
    N = st["N"]
    y = torch.empty((st["x"].shape[0], N), dtype=torch.float64, device="cuda")
    at = 0
    for e, n in enumerate(st["count"].tolist()):
        if n == 0:
            continue
        z = torch.mm(st["x"][at:at + n].double(), st["w"][e].double().T.contiguous())
        z *= st["xs"][at:at + n].double()[:, None] * st["ws"][e].double()
        y[at:at + n] = z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:] if st["swiglu"] else z
        at += n
    return y


def _exact_permute(st):
    # each assignment's place: its expert's first row, then its rank among the expert's assignments
    E, k = st["E"], st["k"]
    ids = st["ids"].reshape(-1).long()
    M = ids.numel()
    mine = torch.nn.functional.one_hot(ids + 1, E + 1)[:, 1:]
    count = mine.sum(dim=0)
    at = (count.cumsum(0) - count) + mine.cumsum(0) - 1
    place = torch.where(ids >= 0, at.gather(1, ids.clamp(min=0)[:, None])[:, 0], -1)
    source = torch.full((M + 1,), -1, device="cuda").scatter_(0, torch.where(place < 0, M, place),
                                                               torch.arange(M, device="cuda"))[:M]
    rows = st["x"].double()[source.clamp(min=0) // k] * (source >= 0)[:, None]
    if st["xs"] is None:
        scales = None
    else:
        rows = rows.to(torch.int8)
        scales = st["xs"].double()[source.clamp(min=0) // k] * (source >= 0)
    return rows, scales, source.clamp(min=0).int(), place.int(), count


def _exact_unpermute(st):
    T, k, K = st["T"], st["k"], st["K"]
    place = st["place"].view(T, k).long()
    w = torch.ones((T, k), dtype=torch.float64, device="cuda") if st["w"] is None else st["w"].double()
    if not st["gradient"]:
        out = torch.zeros((T, K), dtype=torch.float64, device="cuda")
        for j in range(k):
            t = (place[:, j] >= 0).nonzero()[:, 0]
            out[t] += w[t, j, None] * st["y"][place[t, j]].double()
        return out
    d = st["d"].double()
    dy = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        t = (place[:, j] >= 0).nonzero()[:, 0]
        dy[place[t, j]] = w[t, j, None] * d[t]
        dw[t, j] = torch.linalg.vecdot(d[t], st["y"][place[t, j]].double())
    return dy, dw if st["w"] is not None else None


def exact(case, seed):
    st = prepare(case, seed)
    return _named(st, {"quantize": _exact_quantize, "linear": _exact_linear, "experts": _exact_experts,
                       "permute": _exact_permute, "unpermute": _exact_unpermute}[case["op"]](st))


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    op, K = case["op"], case["K"]
    if op == "quantize":
        rows = case["rows"]
        return {"bytes": rows * (3 * K + 4), "flops": 3 * rows * K}
    T = case["T"]
    if op == "linear":
        N = case["N"]
        n = T * (2 * K if case["x"] == "bf16" else K + 4) + N * (K + 4) + 2 * T * N * (1 + case["residual"])
        n += N * {"none": 0, "bf16": 2, "fp32": 4}[case["bias"]]
        return {"bytes": n, "flops": 2 * T * K * N}
    k, E = case["k"], case["E"]
    M = T * k
    if op == "experts":
        rows = case["N"] * (2 if case["swiglu"] else 1)
        used = E * (1 - (1 - k / E) ** T)   # experts that get a row, where all are as likely
        return {"bytes": int(M * (K + 4) + used * rows * (K + 4) + 2 * M * case["N"] + 8 * E), "flops": 2 * M * K * rows}
    if op == "permute":
        size = DTYPES[case["x"]].itemsize
        real = (T - T // 8) * k if case["padded"] else M
        row = K * size + (4 if case["x"] == "int8" else 0)
        return {"bytes": (real // k + real) * row + 12 * M + 8 * E, "flops": 0}
    size = DTYPES[case["y"]].itemsize
    real = M * (1 - case["dropped"])
    n = (T + real) * K * size + 4 * M + (4 * M if case["weighted"] else 0)
    flops = 2 * real * K
    if case["gradient"] and case["weighted"]:
        n += real * K * size + 4 * M
        flops += real * K
    return {"bytes": int(n), "flops": int(flops)}
