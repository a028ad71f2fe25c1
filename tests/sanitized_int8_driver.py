"""Runs inside a process that preloads the sanitizer runtime and loads the
host-sanitised libmxmoe (see sanitized_build.py): calls the entry points of the
INT8 path and of the expert sort with arguments their host checks must reject --
null pointers, sizes at and past every limit, int64 extremes, overlapping buffers
at the largest sizes -- and checks the returned status.  Nothing reaches the GPU:
every call fails validation first."""

import ctypes
import itertools
import sys

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
BIG = [1 << 31, (1 << 31) + 7, 1 << 40, 1 << 62, (1 << 63) - 1]
NEG = [-1, -(1 << 31), -(1 << 63)]
TOP = (1 << 31) - 1

lib = ctypes.CDLL(sys.argv[1])
SIG = {
    "int8_quantize": (I32, [P, I64, I64, I64, P, P, P]),
    "int8_linear_workspace_size": (SZ, [I64, I64, I64, I32]),
    "int8_linear": (I32, [P, P, P, P, P, I32, I32, P, I64, I64, I64, P, P, SZ, P]),
    "int8_linear_kernel": (I32, [I64, I64, I64, I32]),
    "gmm_int8_kernel": (I32, [I64, I64, I64, I64, I32]),
    "gmm_int8": (I32, [P, P, P, P, P, I32, I32, I64, I64, I64, I64, P, P]),
    "moe_permute": (I32, [P, I64, I64, P, P, I64, I64, I64, I64, P, P, P, P, P, P, SZ, P]),
    "moe_unpermute": (I32, [P, I32, P, P, I64, I64, I64, I64, P, P]),
    "moe_unpermute_backward": (I32, [P, I32, P, P, P, I64, I64, I64, I64, P, P, P]),
    "mx_last_error": (ctypes.c_char_p, []),
}
for name, (res, args) in SIG.items():
    fn = getattr(lib, name)
    fn.restype, fn.argtypes = res, args

n = 0


def expect(got, want, what):
    global n
    n += 1
    if got not in (want if isinstance(want, tuple) else (want,)):
        sys.exit(f"{what}: got {got}, want {want} ({lib.mx_last_error()!r})")


def at(i):
    return ctypes.c_void_p((i + 1) << 44)


def quant(rows=4, kd=64, ld=64, x=at(0), q=at(1), s=at(2)):
    return lib.int8_quantize(x, rows, kd, ld, q, s, None)


for v in NEG:
    for kw in ("rows", "kd", "ld"):
        expect(quant(**{kw: v}), INVALID, f"quantize {kw} {v}")
for v in BIG:
    expect(quant(rows=v), UNSUPPORTED, f"quantize rows {v}")
    expect(quant(ld=v), UNSUPPORTED, f"quantize ld {v}")
    expect(quant(kd=v, ld=v), UNSUPPORTED, f"quantize kd {v}")
for rows, kd, ld in itertools.product((1, 7, TOP), (1, 100, 1 << 24), (1 << 24, TOP)):
    for kw in (dict(q=at(0)), dict(s=at(0)), dict(s=at(1))):
        expect(quant(rows=rows, kd=kd, ld=ld, **kw), INVALID, f"quantize overlap {rows} {kd} {ld} {kw}")
for kw in (dict(x=None), dict(q=None), dict(s=None)):
    expect(quant(**kw), INVALID, f"quantize {kw}")


def lin(T=40, K=64, N=96, x=at(0), xs=at(1), w=at(2), ws=at(3), b=at(4), bt=0, act=0, r=at(5), y=at(6), wsp=at(9),
        wsb=1 << 62):
    return lib.int8_linear(x, xs, w, ws, b, bt, act, r, T, K, N, y, wsp, wsb, None)


for v in NEG:
    for kw in ("T", "K", "N"):
        expect(lin(**{kw: v}), INVALID, f"linear {kw} {v}")
for v in BIG:
    expect(lin(T=v), UNSUPPORTED, f"linear T {v}")
    expect(lin(N=v), UNSUPPORTED, f"linear N {v}")
    expect(lin(K=v), UNSUPPORTED, f"linear K {v}")
    expect(lin(K=v // 16 * 16), UNSUPPORTED, f"linear K {v} rounded")
expect(lin(T=TOP, N=(1 << 27) - 1), UNSUPPORTED, "linear tiles")
for T, K, N in ((1, 16, 1), (1, (1 << 17) - 16, (1 << 27) - 1), (TOP, (1 << 17) - 16, 1), (TOP, 16, 96), (1 << 19, 4096, (1 << 19) - 32)):
    for kw in (dict(y=at(0)), dict(y=at(1)), dict(y=at(2)), dict(y=at(3)), dict(y=at(4)),
               dict(y=at(9), xs=None, T=max(T, 40)), dict(wsp=at(0), xs=None, T=max(T, 40))):
        expect(lin(**{**dict(T=T, K=K, N=N), **kw}), INVALID, f"linear overlap {T} {K} {N} {kw}")
    for form in (0, 1):
        lib.int8_linear_workspace_size(T, K, N, form)
        if lib.int8_linear_kernel(T, K, N, form) not in range(8):
            sys.exit(f"linear kernel {T} {K} {N}")
for kw in (dict(x=None), dict(w=None), dict(ws=None), dict(y=None), dict(bt=9), dict(act=9), dict(act=-1),
           dict(xs=None, wsp=None)):
    expect(lin(**kw), INVALID, f"linear {kw}")
expect(lin(xs=None, wsb=0), WORKSPACE, "linear workspace 0")
for v in NEG + BIG:
    for i in range(3):
        a = [64, 64, 64]
        a[i] = v
        expect(lib.int8_linear_workspace_size(*a, 0), 0, f"linear workspace query {i} = {v}")
        expect(lib.int8_linear_kernel(*a, 0), (INVALID, UNSUPPORTED), f"linear kernel query {i} = {v}")


def experts(M=5, N=96, K=64, E=3, a=at(0), a_s=at(1), w=at(2), ws=at(3), gl=at(4), kind=1, swiglu=0, y=at(5)):
    return lib.gmm_int8(a, a_s, w, ws, gl, kind, swiglu, M, N, K, E, y, None)


for v in NEG:
    for i, kw in enumerate(("M", "N", "K", "E")):
        expect(experts(**{kw: v}), INVALID, f"experts {kw} {v}")
for v in BIG:
    for kw in ("M", "N", "K", "E"):
        expect(experts(**{kw: v}), UNSUPPORTED, f"experts {kw} {v}")
    for i in range(4):
        a = [64, 64, 64, 64]
        a[i] = v
        expect(lib.gmm_int8_kernel(*a, 1), UNSUPPORTED, f"experts kernel query {i} = {v}")
for M, N, K, E, swiglu in itertools.product((1, TOP // 64), (1, 96), (16, (1 << 17) - 16), (1, 1024), (0, 1)):
    for kw in (dict(y=at(0)), dict(y=at(1)), dict(y=at(2)), dict(y=at(3)), dict(y=at(4))):
        expect(experts(M=M, N=N, K=K, E=E, swiglu=swiglu, **kw), INVALID, f"experts overlap {M} {N} {K} {E} {kw}")
    if lib.gmm_int8_kernel(M, N, K, E, swiglu) not in range(7):
        sys.exit(f"experts kernel {M} {N} {K} {E}")
expect(experts(M=1 << 28, N=1 << 10), UNSUPPORTED, "experts tiles")
for kw in (dict(a=None), dict(a_s=None), dict(w=None), dict(ws=None), dict(gl=None), dict(y=None), dict(kind=2)):
    expect(experts(**kw), INVALID, f"experts {kw}")


def permute(T=4, K=64, k=2, E=8, ldx=64, eb=2, x=at(0), xs=None, ids=at(1), xp=at(2), xps=None, sr=at(3), eri=at(4),
            gl=at(5), wsp=at(6), wsb=1 << 62):
    return lib.moe_permute(x, ldx, eb, xs, ids, T, K, k, E, xp, xps, sr, eri, gl, wsp, wsb, None)


for v in NEG:
    for kw in ("T", "K", "k", "E", "ldx", "eb"):
        expect(permute(**{kw: v}), INVALID, f"permute {kw} {v}")
for v in BIG:
    for kw in ("T", "E", "ldx"):
        expect(permute(**{kw: v}), UNSUPPORTED, f"permute {kw} {v}")
    expect(permute(K=v, ldx=v), UNSUPPORTED, f"permute K {v}")
    expect(permute(k=v), INVALID, f"permute k {v}")
    expect(permute(eb=v), INVALID, f"permute elem_bytes {v}")
for T, K, ldx, eb in itertools.product((1, 1 << 26), (1, 1 << 24), (1 << 24, TOP), (1, 2, 4)):
    for kw in (dict(xp=at(0)), dict(sr=at(1)), dict(eri=at(2)), dict(gl=at(3)), dict(xs=at(7), xps=at(7)),
               dict(xs=at(7), xps=at(2))):
        expect(permute(T=T, K=K, ldx=ldx, eb=eb, **kw), INVALID, f"permute overlap {T} {K} {ldx} {eb} {kw}")
for kw in (dict(x=None), dict(ids=None), dict(xp=None), dict(sr=None), dict(eri=None), dict(gl=None), dict(xs=at(7)),
           dict(xps=at(7)), dict(T=300, wsp=None), dict(eb=0), dict(eb=3), dict(eb=8)):
    expect(permute(**kw), INVALID, f"permute {kw}")
expect(permute(T=300, wsb=0), WORKSPACE, "permute workspace 0")


def back(T=4, K=64, k=2, M=8, y=at(0), kind=0, w=at(1), eri=at(2), out=at(3)):
    return lib.moe_unpermute(y, kind, w, eri, T, K, k, M, out, None)


def grad(T=4, K=64, k=2, M=8, d=at(0), kind=0, y=at(1), w=at(2), eri=at(3), dy=at(4), dw=at(5)):
    return lib.moe_unpermute_backward(d, kind, y, w, eri, T, K, k, M, dy, dw, None)


for call in (back, grad):
    for v in NEG:
        for kw in ("T", "K", "k", "M"):
            expect(call(**{kw: v}), INVALID, f"{call.__name__} {kw} {v}")
    for v in BIG:
        for kw in ("T", "K", "k", "M"):
            expect(call(**{kw: v}), UNSUPPORTED, f"{call.__name__} {kw} {v}")
    for kind in (-1, 3, 1 << 30):
        expect(call(kind=kind), INVALID, f"{call.__name__} type {kind}")
    expect(call(T=1 << 30, k=2), UNSUPPORTED, f"{call.__name__} T k")
for T, K, M, kind in itertools.product((1, TOP // 2), (1, 1 << 24), (1, TOP), (0, 1, 2)):
    for kw in (dict(out=at(0)), dict(out=at(1)), dict(out=at(2))):
        expect(back(T=T, K=K, k=2, M=M, kind=kind, **kw), INVALID, f"unpermute overlap {T} {K} {M} {kw}")
    for kw in (dict(dy=at(0)), dict(dy=at(1)), dict(dy=at(2)), dict(dy=at(3)), dict(dw=at(0)), dict(dw=at(2)), dict(dw=at(4))):
        expect(grad(T=T, K=K, k=2, M=M, kind=kind, **kw), INVALID, f"gradient overlap {T} {K} {M} {kw}")
for kw in (dict(y=None), dict(eri=None), dict(out=None)):
    expect(back(**kw), INVALID, f"unpermute {kw}")
for kw in (dict(d=None), dict(y=None), dict(eri=None), dict(dy=None)):
    expect(grad(**kw), INVALID, f"gradient {kw}")

print(f"OK {n} checks")
