"""Runs inside a process that preloads the sanitizer runtime and loads the
host-sanitised libmxmoe (see sanitized_build.py): calls the entry points of the
operators around the expert layer with arguments their host checks must reject
-- null pointers, sizes at and past every limit, int64 extremes, overlapping
buffers at the largest sizes -- and checks the returned status.  Nothing
reaches the GPU: every call fails validation first."""

import ctypes
import itertools
import sys

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P, I64, I32, SZ, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
BIG = [1 << 31, (1 << 31) + 7, 1 << 40, 1 << 62, (1 << 63) - 1]
NEG = [-1, -(1 << 31), -(1 << 63)]
TOP = (1 << 31) - 1

lib = ctypes.CDLL(sys.argv[1])
SIG = {
    "mx_add_rmsnorm": (I32, [P, I64, P, I64, P, I32, F32, I64, I64, P, P, P, P, P]),
    "mx_linear_fused_workspace_size": (SZ, [I64, I64, I64, I32]),
    "mx_linear_fused": (I32, [P, P, P, P, P, I32, I32, P, I64, I64, I64, P, P, P, P, SZ, P]),
    "moe_route_mx": (I32, [P, P, P, I64, I64, I64, I64, P, P, P, P, P, P, SZ, P]),
    "moe_mxfp8_forward_mx": (I32, [P, P, P, P, I32, P, P, P, P, I64, I64, I64, I64, I64, P, P, SZ, P]),
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


def norm(rows=4, kd=64, ldx=64, ldr=64, x=at(0), res=at(1), w=at(2), wt=0, eps=1e-6, ro=at(3), y=at(4), q=at(5),
         s=at(6)):
    return lib.mx_add_rmsnorm(x, ldx, res, ldr, w, wt, eps, rows, kd, ro, y, q, s, None)


for v in NEG:
    for kw in ("rows", "kd", "ldx", "ldr"):
        expect(norm(**{kw: v}), INVALID, f"norm {kw} {v}")
for v in BIG:
    expect(norm(rows=v), UNSUPPORTED, f"norm rows {v}")
    expect(norm(ldx=v), UNSUPPORTED, f"norm ldx {v}")
    expect(norm(ldr=v), UNSUPPORTED, f"norm ldr {v}")
    expect(norm(kd=v, ldx=v, ldr=v), UNSUPPORTED, f"norm kd {v}")
for rows, kd, ld in itertools.product((1, 7, TOP), (1, 100, 1 << 24), (1 << 24, TOP)):
    for kw in (dict(q=at(0)), dict(y=at(2)), dict(ro=at(4)), dict(s=at(5)), dict(q=at(1))):
        expect(norm(rows=rows, kd=kd, ldx=ld, ldr=ld, **kw), INVALID, f"norm overlap {rows} {kd} {ld} {kw}")
for kw in (dict(x=None), dict(w=None), dict(q=None), dict(s=None), dict(res=None), dict(y=None, q=None, s=None),
           dict(wt=7), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf"))):
    expect(norm(**kw), INVALID, f"norm {kw}")


def lin(T=4, K=64, N=96, x=at(0), xs=at(1), w=at(2), ws=at(3), b=at(4), bt=0, act=0, r=at(5), y=at(6), yq=None,
        ys=None, wsp=at(9), wsb=1 << 62):
    return lib.mx_linear_fused(x, xs, w, ws, b, bt, act, r, T, K, N, y, yq, ys, wsp, wsb, None)


for v in NEG:
    for kw in ("T", "K", "N"):
        expect(lin(**{kw: v}), INVALID, f"linear {kw} {v}")
for v in BIG:
    expect(lin(T=v), UNSUPPORTED, f"linear T {v}")
    expect(lin(N=v), UNSUPPORTED, f"linear N {v}")
    expect(lin(K=v), UNSUPPORTED, f"linear K {v}")
    expect(lin(K=v // 32 * 32), UNSUPPORTED, f"linear K {v} rounded")
for T, K, N in itertools.product((1, TOP), (32, 1 << 20), (1, TOP)):
    for kw in (dict(y=at(0)), dict(y=at(2)), dict(y=at(9), xs=None, T=max(T, 100)), dict(y=None, yq=at(7), ys=at(7)),
               dict(y=None, yq=at(5), ys=at(8))):
        expect(lin(**{**dict(T=T, K=K, N=N), **kw}), INVALID, f"linear overlap {T} {K} {N} {kw}")
    lib.mx_linear_fused_workspace_size(T, K, N, 0)
for kw in (dict(x=None), dict(w=None), dict(ws=None), dict(y=None), dict(yq=at(7)), dict(y=None, ys=at(7)),
           dict(bt=9), dict(act=9), dict(act=-1), dict(xs=None, T=100, wsp=None)):
    expect(lin(**kw), INVALID, f"linear {kw}")
expect(lin(xs=None, T=100, wsb=0), WORKSPACE, "linear workspace 0")
for v in NEG + BIG:
    for i in range(3):
        a = [64, 64, 64]
        a[i] = v
        expect(lib.mx_linear_fused_workspace_size(*a, 0), 0, f"linear ws query arg {i} = {v}")


def route(T=64, K=256, k=2, E=8, wsb=1 << 40, q=at(0), s=at(1), gl=at(7)):
    return lib.moe_route_mx(q, s, at(2), T, K, k, E, at(3), at(4), at(5), at(6), gl, at(9), wsb, None)


def forward(T=64, K=256, I=128, E=8, k=2, fmt=0, wsb=1 << 62, ws=at(9), s=at(1)):
    return lib.moe_mxfp8_forward_mx(at(0), s, at(2), at(3), fmt, at(4), at(5), at(6), at(7), T, K, I, E, k, at(8), ws,
                                    wsb, None)


for v in NEG:
    for kw in ("T", "K", "k", "E"):
        expect(route(**{kw: v}), INVALID, f"route {kw} {v}")
        expect(forward(**{kw: v}), INVALID, f"forward {kw} {v}")
    expect(forward(I=v), INVALID, f"forward I {v}")
for v in BIG:
    for kw in ("T", "K", "E"):
        expect(route(**{kw: v}), UNSUPPORTED, f"route {kw} {v}")
    for kw in ("T", "K", "I", "E", "k"):
        expect(forward(**{kw: v}), (INVALID, UNSUPPORTED), f"forward {kw} {v}")
expect(route(q=None), INVALID, "route null q")
expect(route(s=None), INVALID, "route null s")
expect(route(gl=None), INVALID, "route null group_list")
expect(route(T=300, wsb=0), WORKSPACE, "route workspace 0")
for fmt in (-1, 3, 1 << 30):
    expect(forward(fmt=fmt), INVALID, f"forward format {fmt}")
for fmt in (0, 1, 2):
    expect(forward(fmt=fmt, wsb=0), WORKSPACE, "forward workspace 0")
    expect(forward(fmt=fmt, ws=None), INVALID, "forward null workspace")
    expect(forward(fmt=fmt, s=None), INVALID, "forward null scales")

print(f"OK {n} checks")
