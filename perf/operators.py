"""The operators around the expert layer, as they are measured: cases, inputs,
the plain forms in elementary torch operations and the library's calls.

  norm    mx_add_rmsnorm: residual addition, root-mean-square norm, MXFP8 (and
          bf16) output
  linear  mx_linear_fused: MXFP8 matrix product with bias, activation and
          residual in its epilogue, bf16 or MXFP8 output
  route   moe_route_mx: rows that are already MXFP8 sent to their experts

MXFP8 is returned as the values it is made of: payloads as float8_e4m3fn,
block scales as float8_e8m0fnu (views of the bytes, nothing is converted).
"""

import math

import torch

own = False

EPS = 1e-6
BLOCK = 32   # elements per MX scale


def listed():
    return [
        # one token of a decode step, before the router and the experts
        {"name": "norm 1 token", "op": "norm", "T": 1, "K": 2048, "residual": True, "weight": "bf16", "y": True},
        # a decode batch before a dense projection: only MXFP8 is wanted
        {"name": "norm 32 tokens", "op": "norm", "T": 32, "K": 4096, "residual": True, "weight": "f32", "y": False},
        # a row that no block size divides (K = 4304 of a checkpoint whose scale rows are padded), first norm of a
        # stack (nothing to add)
        {"name": "norm ragged rows", "op": "norm", "T": 1031, "K": 4304, "residual": False, "weight": "bf16", "y": True},
        # prefill, before the router and the experts
        {"name": "norm 16K tokens", "op": "norm", "T": 16384, "K": 2048, "residual": True, "weight": "bf16", "y": True},
        # one token through a projection with bias and activation, unquantised input
        {"name": "linear 1 token", "op": "linear", "T": 1, "K": 2048, "N": 2048, "x": "bf16", "bias": "f32",
         "act": "silu", "residual": False, "out": "bf16"},
        # a decode batch through an output projection that adds to the residual stream
        {"name": "linear 32 tokens", "op": "linear", "T": 32, "K": 4096, "N": 4096, "x": "mx", "bias": "none",
         "act": "none", "residual": True, "out": "bf16"},
        # a short prompt, an output width that no tile divides
        {"name": "linear ragged", "op": "linear", "T": 203, "K": 2080, "N": 4099, "x": "mx", "bias": "bf16",
         "act": "gelu", "residual": True, "out": "bf16"},
        # the first half of a two-layer block whose second half reads MXFP8
        {"name": "linear 2K tokens to MX", "op": "linear", "T": 2048, "K": 2048, "N": 4096, "x": "mx", "bias": "bf16",
         "act": "gelu_tanh", "residual": False, "out": "mx"},
        # prefill through an output projection
        {"name": "linear 16K tokens", "op": "linear", "T": 16384, "K": 4096, "N": 4096, "x": "mx", "bias": "bf16",
         "act": "none", "residual": True, "out": "bf16"},
        # decode, 32 tokens to 8 of 128 experts each
        {"name": "route 32 tokens", "op": "route", "T": 32, "K": 2048, "k": 8, "E": 128, "spread": "even"},
        # a few crowded experts, a token count that no chunk divides
        {"name": "route 2049 tokens", "op": "route", "T": 2049, "K": 4096, "k": 8, "E": 64, "spread": "zipf"},
        # prefill
        {"name": "route 16K tokens", "op": "route", "T": 16384, "K": 2048, "k": 8, "E": 128, "spread": "even"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "route"])
    if op == "norm":
        K = _spread(rng, 64, 16384)
        K -= K % rng.choice([1, 8, 32, 32])
        T = _spread(rng, 1, min(16384, 16384 * 2048 // K))
        return {"op": op, "T": T, "K": K, "residual": rng.random() < 0.7, "weight": rng.choice(["bf16", "f32"]),
                "y": rng.random() < 0.5}
    if op == "linear":
        K = _spread(rng, 128, 8192)
        K -= K % rng.choice([32, 128, 128])
        N = _spread(rng, 64, 8192)
        N -= N % rng.choice([1, 8, 32, 256])
        N = max(N, 64)
        T = _spread(rng, 1, min(16384, 16384 * 4096 * 4096 // (K * N), 16384 * 4096 // N))
        return {"op": op, "T": T, "K": K, "N": N, "x": rng.choice(["bf16", "mx", "mx"]),
                "bias": rng.choice(["none", "bf16", "f32"]),
                "act": rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]),
                "residual": rng.random() < 0.5, "out": rng.choice(["bf16", "bf16", "mx"])}
    K = 32 * _spread(rng, 4, 256)
    E = rng.choice([8, 16, 60, 64, 128, 256])
    k = rng.randint(1, 8)
    T = _spread(rng, 1, min(16384, 16384 * 8 * 2048 // (K * k)))
    return {"op": op, "T": T, "K": K, "k": k, "E": E, "spread": rng.choice(["even", "zipf"])}


# ---- inputs -------------------------------------------------------------------------

def _activations(shape, gen):
    """N(0, 1) with 1 % of the channels twenty times as large, bf16."""
    x = torch.randn(shape, generator=gen, device="cuda")
    hot = torch.randperm(shape[1], generator=gen, device="cuda")[: -(-shape[1] // 100)]
    x[:, hot] *= 20
    return x.bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, K = case["T"], case["K"]

    def normal(shape, scale=1.0, shift=0.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale + shift

    def u8(*shape):
        return torch.empty(shape, dtype=torch.uint8, device="cuda")

    def bf16(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda")

    st = dict(case)
    if case["op"] == "norm":
        st["x"] = _activations((T, K), gen)
        st["r"] = normal((T, K), 2.0).bfloat16() if case["residual"] else None
        w = normal((K,), 0.2, 1.0)
        st["w"] = w if case["weight"] == "f32" else w.bfloat16()
        # the buffers that a serving loop keeps for its results
        st["to"] = (u8(T, K), u8(T, -(-K // 64), 2), bf16(T, K) if case["residual"] else None,
                    bf16(T, K) if case["y"] else None)
    elif case["op"] == "linear":
        N = case["N"]
        x = _activations((T, K), gen)
        st["x"], st["xs"] = (x, None) if case["x"] == "bf16" else _mx_quantise(x.float())
        st["w"], st["ws"] = _mx_quantise(normal((N, K), 0.02).bfloat16().float())
        b = normal((N,), 0.5)
        st["b"] = {"none": None, "bf16": b.bfloat16(), "f32": b}[case["bias"]]
        st["r"] = normal((T, N), 2.0).bfloat16() if case["residual"] else None
        st["to"] = bf16(T, N) if case["out"] == "bf16" else (u8(T, N), u8(T, -(-N // 64), 2))
    else:
        E, k = case["E"], case["k"]
        st["x"], st["xs"] = _mx_quantise(_activations((T, K), gen).float())
        logits = normal((T, E))
        if case["spread"] == "zipf":
            logits -= 1.1 * torch.log(torch.arange(1, E + 1, device="cuda"))[torch.randperm(E, generator=gen, device="cuda")]
        st["ids"] = torch.topk(logits, k, dim=1).indices.int()
        M = T * k
        st["to"] = (u8(M, K), u8(M, -(-K // 64), 2), torch.empty(M, dtype=torch.int32, device="cuda"),
                    torch.empty(M, dtype=torch.int32, device="cuda"), torch.empty(E, dtype=torch.int64, device="cuda"))
    return st


# ---- the plain forms ----------------------------------------------------------------

def _mx_quantise(v):
    """fp32 [R, K] -> e4m3 bytes [R, K] and e8m0 bytes [R, ceil(K/64), 2]."""
    R, K = v.shape
    nb = -(-K // BLOCK)
    blocks = torch.nn.functional.pad(v, (0, nb * BLOCK - K)).view(R, nb, BLOCK)
    amax = blocks.abs().amax(dim=2)
    # floor(log2 amax) - 8 in [-127, 127], as a byte
    byte = torch.where(amax > 0, torch.frexp(amax)[1].int() + 118, 0).clamp(0, 254)
    inverse = ((254 - byte) << 23).view(torch.float32)   # 2^(127 - byte)
    q = (blocks * inverse[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.zeros((R, -(-K // 64) * 2), dtype=torch.uint8, device=v.device)
    s[:, :nb] = byte
    return q.view(torch.uint8).view(R, -1)[:, :K].contiguous(), s.view(R, -1, 2)


def _mx_values(q, s):
    """What MXFP8 stands for, fp32 [R, K]."""
    K = q.shape[1]
    byte = s.reshape(s.shape[0], -1)[:, : -(-K // BLOCK)].int()
    scale = torch.where(byte > 0, (byte << 23).view(torch.float32), 2.0 ** -127)
    return q.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(BLOCK, dim=1)[:, :K]


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


def _plain_norm(st):
    h = st["x"].float()
    if st["r"] is not None:
        h = h + st["r"].float()
    n = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * st["w"].float()
    q, s = _mx_quantise(n)
    return q, s, h.bfloat16() if st["r"] is not None else None, n.bfloat16() if st["y"] else None


def _plain_linear(st):
    x, xs = (st["x"], st["xs"]) if st["xs"] is not None else _mx_quantise(st["x"].float())
    z = _mx_values(x, xs) @ _mx_values(st["w"], st["ws"]).T
    if st["b"] is not None:
        z = z + st["b"].float()
    z = _activate(z, st["act"])
    if st["r"] is not None:
        z = z + st["r"].float()
    return z.bfloat16() if st["out"] == "bf16" else _mx_quantise(z)


def _plain_route(st):
    ids = st["ids"].reshape(-1)
    order = torch.argsort(ids, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    count = (ids[:, None] == torch.arange(st["E"], device=ids.device)).sum(dim=0)
    token = order // st["k"]
    return st["x"][token], st["xs"][token], order.int(), place.int(), count


def run(st):
    if own:
        import mxfp8_block_scaled_topk_amd as mx
        if st["op"] == "norm":
            got = mx.mx_add_rmsnorm(st["x"], st["w"], st["r"], eps=EPS, out=st["to"])
        elif st["op"] == "linear":
            got = mx.mx_linear_fused(st["x"], st["w"], st["ws"], x_s=st["xs"], bias=st["b"], act=st["act"],
                                     residual=st["r"], out=st["to"])
        else:
            got = mx.moe_route_mx(st["x"], st["xs"], st["ids"], st["E"], out=st["to"])
    else:
        got = {"norm": _plain_norm, "linear": _plain_linear, "route": _plain_route}[st["op"]](st)
    return _named(st, got)


def _named(st, got):
    if st["op"] == "linear" and st["out"] == "bf16":
        return {"y": got}
    named = {"q": got[0].view(torch.float8_e4m3fn), "s": got[1].view(torch.float8_e8m0fnu)}
    if st["op"] == "norm":
        named["residual"], named["y"] = got[2], got[3]
    if st["op"] == "route":
        named["sorted_row"], named["expanded_row_idx"], named["group_list"] = got[2:]
    return named


# ---- the definitions in 64 bits -----------------------------------------------------

def _pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quantise(v):
    """fp64 [R, K] -> e4m3 values as payloads (fp64) and scales (fp64, padding 2^-127)."""
    R, K = v.shape
    scales = torch.full((R, -(-K // 64) * 2), 2.0 ** -127, dtype=torch.float64, device=v.device)
    payload = torch.empty_like(v)
    whole = K - K % BLOCK
    for part, at in ((v[:, :whole].reshape(R, -1, BLOCK), 0), (v[:, whole:].reshape(R, 1, K - whole), whole)):
        if part.numel() == 0:
            continue
        top = part.abs().amax(dim=2)
        e = torch.where(top > 0, torch.frexp(top)[1].long() - 9, -127).clamp(-127, 127)
        t = part * _pow2(-e)[:, :, None]
        step = _pow2((torch.frexp(t)[1].long() - 1).clamp(min=-6) - 3)   # e4m3 spacing at t
        t = (torch.round(t / step) * step).clamp(-448, 448)
        payload[:, at:at + t.shape[1] * t.shape[2]] = t.reshape(R, -1)
        scales[:, at // BLOCK:at // BLOCK + e.shape[1]] = _pow2(e)
    return payload, scales.view(R, -1, 2)


def _exact_values(q, s):
    K = q.shape[1]
    e = s.reshape(s.shape[0], -1).long() - 127
    return q.view(torch.float8_e4m3fn).double() * _pow2(e).repeat_interleave(BLOCK, dim=1)[:, :K]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].double()
        if case["residual"]:
            h += st["r"].double()
        n = h / (h.pow(2).sum(dim=1, keepdim=True) / case["K"] + EPS).sqrt() * st["w"].double()
        q, s = _exact_quantise(n)
        return {"q": q, "s": s, "residual": h if case["residual"] else None, "y": n if case["y"] else None}
    if case["op"] == "linear":
        if case["x"] == "bf16":
            q, s = _exact_quantise(st["x"].double())
            x = q * s.reshape(case["T"], -1).repeat_interleave(BLOCK, dim=1)[:, :case["K"]]
        else:
            x = _exact_values(st["x"], st["xs"])
        z = torch.mm(x, _exact_values(st["w"], st["ws"]).T.contiguous())
        if st["b"] is not None:
            z += st["b"].double()
        if case["act"] == "relu":
            z = torch.where(z > 0, z, 0.0)
        elif case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        elif case["act"] == "gelu_tanh":
            z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3)))
        if st["r"] is not None:
            z += st["r"].double()
        if case["out"] == "bf16":
            return {"y": z}
        q, s = _exact_quantise(z)
        return {"q": q, "s": s}
    # each assignment's place: its expert's first row, then its rank among the expert's assignments
    T, k, E = case["T"], case["k"], case["E"]
    ids = st["ids"].reshape(-1).long()
    mine = torch.nn.functional.one_hot(ids, E)
    count = mine.sum(dim=0)
    first = count.cumsum(0) - count
    place = first[ids] + (mine.cumsum(0) - 1).gather(1, ids[:, None])[:, 0]
    order = torch.zeros_like(place).scatter_(0, place, torch.arange(T * k, device="cuda"))
    return {"q": st["x"].view(torch.float8_e4m3fn).double()[order // k],
            "s": _pow2(st["xs"].long() - 127)[order // k],
            "sorted_row": order, "expanded_row_idx": place, "group_list": count}


# ---- what a pass cannot do without --------------------------------------------------

def _mx_bytes(rows, K):
    return rows * (K + 2 * -(-K // 64))


def work(case):
    T, K = case["T"], case["K"]
    if case["op"] == "norm":
        n = 2 * T * K * (1 + 2 * case["residual"] + case["y"]) + _mx_bytes(T, K) + K * (4 if case["weight"] == "f32" else 2)
        return {"bytes": n, "flops": 6 * T * K}
    if case["op"] == "linear":
        N = case["N"]
        n = (2 * T * K if case["x"] == "bf16" else _mx_bytes(T, K)) + _mx_bytes(N, K)
        n += N * {"none": 0, "bf16": 2, "f32": 4}[case["bias"]] + 2 * T * N * case["residual"]
        n += 2 * T * N if case["out"] == "bf16" else _mx_bytes(T, N)
        return {"bytes": n, "flops": 2 * T * K * N}
    k, E = case["k"], case["E"]
    return {"bytes": _mx_bytes(T, K) + _mx_bytes(T * k, K) + 4 * T * k * 3 + 8 * E, "flops": 0}
