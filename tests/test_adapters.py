"""Low-rank adapters of many requests beside the shared projection, and their
gradients: the kernels against the FP64 oracle, and the refusals.

Tolerances count roundings, u = 2^-24 being half a step of fp32.  A sum of k
products on the tensor cores adds 16 of them per step and may drop a step (two
u) of the running sum each time: k / 8 u of the sum of absolute products, which
also covers the CUDA cores' partial sums (at most k / 32 additions in a row).
Where a hidden vector is fed to the tensor cores it is cut into two bf16
pieces for a bf16 output (the rest is below 2^-17 of it; 2^-16 allowed), three
for an fp32 one (below u)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
import post_weight_quantization_09_b200 as Q
from post_weight_quantization_09_b200 import _lib as L
from post_weight_quantization_09_b200.build import build
from quip_synth import Side
from parity_util import dev, host

U = 2.0 ** -24
gpu = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16


@pytest.fixture
def clean():
    Q.load()
    Q.quip_sync_status()
    yield
    assert Q.quip_sync_status() == L.QUIP_OK


# ------------------------------------------------------------------ on the CPU

def test_oracle_gradients_are_the_slopes():
    rng = np.random.default_rng(0)
    T, n, m, r, c = 5, 4, 3, 2, 2
    x, down, up = rng.standard_normal((T, n)), rng.standard_normal((c, r, n)), rng.standard_normal((c, r, m))
    scale, dy, ids = rng.uniform(0.5, 1.5, c), rng.standard_normal((T, m)), np.array([1, -1, 1, 0, 1])
    base = rng.standard_normal((T, m))
    y, h = O.adapter_apply(x, ids, down, up, scale, base)
    dx, d_down, d_up, _ = O.adapter_backward(x, dy, ids, down, up, scale, h, np.zeros((T, n)))

    def loss(x=x, down=down, up=up):
        return np.sum(dy * O.adapter_apply(x, ids, down, up, scale, base)[0])
    for name, a, g in (("x", x, dx), ("down", down, d_down), ("up", up, d_up)):
        for i in np.ndindex(a.shape):
            e = np.zeros_like(a)
            e[i] = 1e-5
            assert abs((loss(**{name: a + e}) - loss(**{name: a - e})) / 2e-5 - g[i]) < 1e-8
    assert np.array_equal(y[1], base[1]) and np.all(h[1] == 0)


def test_refusals_answer_on_the_host():
    build()
    lib = L.load()
    p = lambda i: ctypes.c_void_p(0x1000000 * (i + 1))
    size = ctypes.c_size_t()
    assert lib.quip_adapter_plan_size(8, 4, None) == L.QUIP_ERR_ARG
    for T, c in ((-1, 4), (8, 0), (8, 1025), (1 << 23, 4)):
        assert lib.quip_adapter_plan_size(T, c, ctypes.byref(size)) == L.QUIP_ERR_SHAPE
    assert lib.quip_adapter_plan_size(8, 4, ctypes.byref(size)) == L.QUIP_OK and size.value % 256 == 0
    assert lib.quip_adapter_plan(None, 8, 4, p(0), size, None) == L.QUIP_ERR_ARG
    assert lib.quip_adapter_plan(p(1), 8, 4, p(0), size.value - 1, None) == L.QUIP_ERR_WORKSPACE
    assert lib.quip_adapter_plan(p(1), 8, 4, ctypes.c_void_p(0x1010), size, None) == L.QUIP_ERR_WORKSPACE
    assert lib.quip_adapter_workspace_size(8, 4, 4, 257, 1, 0, ctypes.byref(size)) == L.QUIP_ERR_SHAPE
    assert lib.quip_adapter_workspace_size(8, 0, 4, 1, 1, 0, ctypes.byref(size)) == L.QUIP_ERR_SHAPE

    def fw(x=p(0), xt=0, ldx=64, ids=p(1), T=100, n=64, m=32, down=p(2), up=p(3), wt=0, c=2, r=4, base=p(5), ldb=32,
           y=p(6), yt=0, ldy=32, plan=None, ws=p(8), wsb=1 << 30):
        return lib.quip_adapter_apply(x, xt, ldx, ids, T, n, m, down, up, wt, c, r, None, base, ldb, y, yt, ldy, None,
                                      plan, ws, wsb, None)
    for name in ("x", "ids", "down", "up", "y"):
        assert fw(**{name: None}) == L.QUIP_ERR_ARG, name
    assert fw(xt=2) == fw(wt=7) == fw(yt=-1) == L.QUIP_ERR_ARG
    assert fw(ldx=63) == fw(ldy=31) == fw(ldb=31) == fw(r=0) == fw(r=257) == fw(c=1025) == fw(T=-1) == L.QUIP_ERR_SHAPE
    assert fw(base=p(6), ldy=40) == L.QUIP_ERR_ARG                   # the same buffer, other rows
    assert fw(base=ctypes.c_void_p(p(6).value + 4)) == L.QUIP_ERR_ARG
    assert fw(y=p(0), base=None) == L.QUIP_ERR_ARG                   # y over x
    assert fw(T=1100, ws=None) == fw(T=1100, wsb=16) == fw(T=1100, ws=ctypes.c_void_p(0x1004)) == L.QUIP_ERR_WORKSPACE
    assert fw(T=0, x=None) == L.QUIP_OK

    def bw(x=p(0), xt=0, ldx=64, dy=p(1), dyt=0, lddy=32, ids=p(2), T=100, n=64, m=32, down=p(3), up=p(4), r=4, h=p(5),
           b=p(6), lddb=64, dx=p(7), lddx=64, dd=p(8), du=p(9), ws=p(10), wsb=1 << 30):
        return lib.quip_adapter_backward(x, xt, ldx, dy, dyt, lddy, ids, T, n, m, down, up, 0, 2, r, None, h, b, lddb, dx,
                                         lddx, dd, du, 0, None, ws, wsb, None)
    for name in ("x", "dy", "ids", "down", "up", "h"):
        assert bw(**{name: None}) == L.QUIP_ERR_ARG, name
    assert bw(xt=2) == bw(dyt=2) == L.QUIP_ERR_ARG
    assert bw(ldx=63) == bw(lddy=31) == bw(lddx=63) == bw(lddb=63) == bw(r=0) == L.QUIP_ERR_SHAPE
    assert bw(dx=p(1), b=None) == bw(dx=p(0), b=None) == bw(b=p(7), lddb=65) == L.QUIP_ERR_ARG
    assert bw(wsb=16) == bw(ws=None) == L.QUIP_ERR_WORKSPACE
    assert bw(dx=None, dd=None, du=None, ws=None) == L.QUIP_OK       # nothing is asked for


def test_binding_refuses_host_tensors():
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        Q.quip_adapter_apply(z(2, 8), z(2, dtype=torch.int32), z(1, 2, 8), z(1, 2, 4), None, z(2, 4))
    with pytest.raises(ValueError, match="CUDA"):
        Q.quip_adapter_plan(z(2, dtype=torch.int32), 1)


# ------------------------------------------------------------------ on the GPU

def _ids(T, count, kind, rng):
    if kind == "random":
        return rng.integers(-1, count, T)
    if kind == "runs":
        cuts = np.sort(rng.integers(0, T + 1, 4))
        return rng.integers(-1, count, 5)[np.searchsorted(cuts, np.arange(T), side="right")]
    if kind == "one":
        return np.full(T, count - 1)
    if kind == "none":
        return np.full(T, -1)
    return np.where(np.arange(T) % 3 == 0, -5, np.arange(T) % count)          # "mixed"


class Case:
    def __init__(self, T, n, m, r, count, x=B, w=B, y=B, ids="random", seed=0, pad=0):
        rng = np.random.default_rng(seed + 7 * T + n + m + r)
        g = torch.Generator().manual_seed(seed + T + n)

        def rows(c, t):
            buf = torch.full((T, c + pad), float("nan"))
            buf[:, :c] = torch.randn(T, c, generator=g)
            return buf.to(t).cuda()[:, :c]
        self.T, self.n, self.m, self.r, self.count, self.pad = T, n, m, r, count, pad
        self.x, self.base, self.dy, self.dx_base = rows(n, x), rows(m, y), rows(m, y), rows(n, x)
        self.down = (torch.randn(count, r, n, generator=g) * n ** -0.5).to(w).cuda()
        self.up = (torch.randn(count, r, m, generator=g) * r ** -0.5).to(w).cuda()
        self.scale = (torch.rand(count, generator=g) + 0.5).cuda()
        self.ids = torch.as_tensor(_ids(T, count, ids, rng).astype(np.int32)).cuda()
        self.y = rows(m, y)
        self.dx = rows(n, x)
        self.h = torch.full((T, r), float("nan"), device="cuda")

    def apply(self, **kw):
        Q.quip_adapter_apply(self.x, self.ids, self.down, self.up, self.scale, self.y, base=self.base, h=self.h, **kw)
        return self.y, self.h

    def check_apply(self):
        ids = host(self.ids).astype(int)
        x, down, up, s, base = (host(t) for t in (self.x, self.down, self.up, self.scale, self.base))
        y, h = O.adapter_apply(x, ids, down, up, s, base)
        mag_h = O.adapter_apply(np.abs(x), ids, np.abs(down), np.abs(up), s, np.abs(base))[1]
        tol_h = (self.n / 8 + 64) * U * mag_h
        assert np.all(np.abs(host(self.h) - h) <= tol_h), np.max(np.abs(host(self.h) - h) - tol_h)
        piece = 2.0 ** -16 if self.y.dtype == B else U
        tol = np.zeros_like(y)
        for t, l in enumerate(ids):
            if l >= 0:
                tol[t] = s[l] * ((tol_h[t] + (piece + (self.r / 8 + 16) * U) * np.abs(h[t])) @ np.abs(up[l]))
        tol += 4 * U * np.abs(base) + torch.finfo(self.y.dtype).eps / 2 * (np.abs(y) + tol)
        got = host(self.y)
        assert np.all(np.abs(got - y) <= tol), np.max(np.abs(got - y) / tol)
        none = ids < 0
        assert np.array_equal(got[none], base[none]) and np.all(host(self.h)[none] == 0)
        if self.pad:
            buf = self.y.as_strided((self.T, self.m + self.pad), self.y.stride())
            assert torch.isnan(buf[:, self.m:]).all()

    def backward(self, accumulate=0.0, **kw):
        self.h = torch.as_tensor(O.adapter_apply(host(self.x), host(self.ids).astype(int), host(self.down), host(self.up),
                                                 host(self.scale), host(self.base))[1], dtype=F).cuda()
        self.d_down = torch.full(self.down.shape, accumulate if accumulate else float("nan"), device="cuda")
        self.d_up = torch.full(self.up.shape, accumulate if accumulate else float("nan"), device="cuda")
        self.acc = accumulate
        Q.quip_adapter_backward(self.x, self.dy, self.ids, self.down, self.up, self.scale, self.h, dx=self.dx,
                                dx_base=self.dx_base, d_down=self.d_down, d_up=self.d_up, accumulate=bool(accumulate),
                                **kw)
        return self.dx, self.d_down, self.d_up

    def check_backward(self):
        ids = host(self.ids).astype(int)
        a = [host(t) for t in (self.x, self.dy)], [host(t) for t in (self.down, self.up, self.scale, self.h, self.dx_base)]
        dx, d_down, d_up, dh = O.adapter_backward(*a[0], ids, *a[1])
        mag = [np.abs(t) for t in a[0]], [np.abs(t) for t in a[1]]
        dx_m, dd_m, du_m, dh_m = O.adapter_backward(*mag[0], ids, *mag[1])
        tol_dh = (self.m / 8 + 64) * U * dh_m
        piece = 2.0 ** -16 if self.dx.dtype == B else U
        tol = np.zeros_like(dx)
        tol_dd = np.zeros_like(d_down)
        for t, l in enumerate(ids):
            if l >= 0:
                tol[t] = (tol_dh[t] + (piece + (self.r / 8 + 16) * U) * np.abs(dh[t])) @ mag[1][0][l]
                tol_dd[l] += np.outer(tol_dh[t], mag[0][0][t])
        tol += 4 * U * mag[1][4] + torch.finfo(self.dx.dtype).eps / 2 * (np.abs(dx) + tol)
        assert np.all(np.abs(host(self.dx) - dx) <= tol), np.max(np.abs(host(self.dx) - dx) / tol)
        # sums over tokens: 1024 in a row at most, then one per further chunk
        k = 1024 + 64 + self.T / 1024
        tol_dd += (k + 4) * U * dd_m + 4 * U * abs(self.acc) + 1e-30
        tol_du = (k + 4) * U * du_m + 4 * U * abs(self.acc) + 1e-30
        assert np.all(np.abs(host(self.d_down) - self.acc - d_down) <= tol_dd)
        assert np.all(np.abs(host(self.d_up) - self.acc - d_up) <= tol_du)
        for l in range(self.count):
            if not np.any(ids == l):
                assert torch.all(self.d_down[l] == self.acc) and torch.all(self.d_up[l] == self.acc)


TYPES = [(B, B, B), (B, B, F), (F, F, F), (F, B, F), (B, F, F), (F, B, B), (F, F, B), (B, F, B)]
SHAPES = [(1, 64, 64, 4, 1, "one"), (1, 33, 7, 1, 3, "random"), (5, 100, 36, 3, 2, "mixed"), (64, 512, 200, 16, 9, "random"),
          (300, 256, 128, 16, 4, "random"), (400, 1030, 517, 12, 3, "runs"), (300, 128, 384, 64, 2, "one"),
          (560, 64, 64, 8, 70, "random"), (130, 96, 72, 12, 5, "runs"), (129, 320, 264, 33, 2, "runs"), (600, 72, 40, 8, 3, "none"), (3100, 200, 136, 16, 2, "runs"),
          (1100, 130, 1000, 48, 1, "one")]


@gpu
@pytest.mark.parametrize("T,n,m,r,count,ids", SHAPES)
@pytest.mark.parametrize("x,w,y", TYPES)
def test_apply_matches_oracle(clean, T, n, m, r, count, ids, x, w, y):
    c = Case(T, n, m, r, count, x, w, y, ids)
    c.apply()
    c.check_apply()


@gpu
@pytest.mark.parametrize("T,n,m,r,count,ids", SHAPES)
@pytest.mark.parametrize("x,w,y", TYPES)
def test_backward_matches_oracle(clean, T, n, m, r, count, ids, x, w, y):
    c = Case(T, n, m, r, count, x, w, y, ids)
    c.backward()
    c.check_backward()


@gpu
@pytest.mark.parametrize("x,w,y", [(B, B, B), (B, B, F), (F, F, F)])
@pytest.mark.parametrize("T,n,m,r,count,ids", [(2, 9000, 4100, 256, 2, "one"), (70, 5000, 1024, 128, 2, "random"),
                                               (260, 1024, 2048, 256, 2, "runs"), (150, 2048, 3000, 96, 3, "random"),
                                               (257, 16, 16, 16, 1, "one"), (513, 8, 1, 1, 1, "one")])
def test_large_ranks_and_widths(clean, T, n, m, r, count, ids, x, w, y):
    c = Case(T, n, m, r, count, x, w, y, ids, seed=3)
    c.apply()
    c.check_apply()
    c.backward()
    c.check_backward()


@gpu
@pytest.mark.parametrize("x,y", [(B, B), (B, F), (F, F)])
@pytest.mark.parametrize("pad", [1, 2, 8])
@pytest.mark.parametrize("T", [3, 270])
def test_strided_rows(clean, T, pad, x, y):
    c = Case(T, 264, 136, 16, 3, x, B, y, "random", pad=pad)
    c.apply()
    c.check_apply()
    c.backward()
    c.check_backward()


@gpu
@pytest.mark.parametrize("T,ld", [(4, 2 ** 30 + 8), (300, 2 ** 23 + 8)])
def test_row_offsets_past_32_bits(clean, T, ld):
    c = Case(T, 264, 136, 16, 3)

    def far(t):
        return torch.empty((T - 1) * ld + t.shape[1], dtype=t.dtype, device="cuda").as_strided(t.shape, (ld, 1)).copy_(t)
    c.x, c.y, c.base, c.dy, c.dx, c.dx_base = (far(t) for t in (c.x, c.y, c.base, c.dy, c.dx, c.dx_base))
    c.apply()
    c.check_apply()
    c.backward()
    c.check_backward()


@gpu
@pytest.mark.parametrize("T,r", [(3, 128), (300, 128), (300, 256)])
def test_factor_offsets_past_32_bits(clean, T, r):
    # the last of 1024 adapters starts behind 2^31 values; the others are never read
    n = 2 ** 31 // (1023 * r) + 8 & ~7
    c = Case(T, n, n, r, 1, ids="one")
    down, up = (torch.empty(1024, r, n, dtype=B, device="cuda") for _ in range(2))
    d_down, d_up = (torch.full((1024, r, n), float("nan"), device="cuda") for _ in range(2))
    down[-1], up[-1] = c.down[0], c.up[0]
    scale, ids = c.scale.repeat(1024), torch.full_like(c.ids, 1023)
    Q.quip_adapter_apply(c.x, ids, down, up, scale, c.y, base=c.base, h=c.h)
    c.check_apply()
    Q.quip_adapter_backward(c.x, c.dy, ids, down, up, scale, c.h, dx=c.dx, dx_base=c.dx_base, d_down=d_down, d_up=d_up)
    c.d_down, c.d_up, c.acc = d_down[-1:], d_up[-1:], 0.0
    c.check_backward()
    assert not d_down[:-1].any() and not d_up[:-1].any()


@gpu
def test_unaligned_tensors(clean):
    # every operand one element off its 16-byte boundary
    for T in (4, 300):
        c = Case(T, 256, 128, 16, 2)
        off = lambda t: torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
        c.x, c.base, c.dy, c.dx_base, c.down, c.up = (off(t.contiguous()) for t in (c.x, c.base, c.dy, c.dx_base, c.down, c.up))
        c.y, c.dx = off(c.y.contiguous()), off(c.dx.contiguous())
        c.apply()
        c.check_apply()
        c.backward()
        c.check_backward()


@gpu
@pytest.mark.parametrize("T", [7, 600])
@pytest.mark.parametrize("y", [B, F])
def test_in_place_without_base_without_scale(clean, T, y):
    c = Case(T, 128, 256, 8, 3, y=y)
    want, _ = c.apply()
    want = want.clone()
    both = c.base.clone()
    Q.quip_adapter_apply(c.x, c.ids, c.down, c.up, c.scale, both, base=both)
    assert torch.equal(both, want)
    zero = torch.zeros_like(c.base)
    a, b = torch.empty_like(zero), torch.full_like(zero, float("nan"))
    Q.quip_adapter_apply(c.x, c.ids, c.down, c.up, c.scale, a, base=zero)
    Q.quip_adapter_apply(c.x, c.ids, c.down, c.up, c.scale, b)
    assert torch.equal(a, b)
    one = torch.ones(3, device="cuda")
    Q.quip_adapter_apply(c.x, c.ids, c.down, c.up, one, a)
    Q.quip_adapter_apply(c.x, c.ids, c.down, c.up, None, b)
    assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("T", [20, 2500])
def test_parts_of_the_gradient_and_accumulation(clean, T):
    c = Case(T, 128, 192, 16, 2, ids="runs")
    dx, dd, du = (t.clone() for t in c.backward())
    c.backward(accumulate=3.0)
    c.check_backward()
    only = torch.empty_like(c.dx.contiguous())
    Q.quip_adapter_backward(c.x, c.dy, c.ids, c.down, c.up, c.scale, None, dx=only, dx_base=c.dx_base)
    assert torch.equal(only, dx)
    d = torch.empty_like(dd)
    Q.quip_adapter_backward(c.x, c.dy, c.ids, c.down, c.up, c.scale, None, d_down=d)
    assert torch.equal(d, dd)
    d = torch.empty_like(du)
    Q.quip_adapter_backward(c.x, c.dy, c.ids, c.down, c.up, c.scale, c.h, d_up=d)
    assert torch.equal(d, du)
    with pytest.raises(ValueError):
        Q.quip_adapter_backward(c.x, c.dy, c.ids, c.down, c.up, c.scale, None, d_up=d)


@gpu
@pytest.mark.parametrize("r", [16, 160])
@pytest.mark.parametrize("T", [0, 6, 300])
@pytest.mark.parametrize("accumulate", [0.0, 3.0])
def test_unused_adapters_may_hold_anything(clean, T, r, accumulate):
    c = Case(T, 256, 192, r, 5)
    c.ids[:] = torch.as_tensor(np.where(np.arange(T) % 3 == 0, -1, 2).astype(np.int32))
    for t in (c.down, c.up, c.scale):
        t[[0, 1, 3, 4]] = float("nan")
    c.apply()
    c.check_apply()
    c.backward(accumulate)
    c.check_backward()


@gpu
@pytest.mark.parametrize("T", [6, 300])
def test_other_rows_nan_stays_theirs(clean, T):
    # a request whose activations are NaN or infinite: nobody else sees it
    c = Case(T, 256, 256, 16, 3, ids="mixed")
    clean_y, _ = c.apply()
    clean_y = clean_y.clone()
    dx, dd, du = (t.clone() for t in c.backward())
    ids = host(c.ids)
    x, dy, h = c.x.clone(), c.dy.clone(), c.h.clone()
    bad = np.flatnonzero(ids == 1)
    c.x[bad[0]] = float("nan")
    c.dy[bad[-1]] = float("inf")
    pad = np.flatnonzero(ids < 0)                   # padding rows hold anything
    c.x[pad] = float("nan")
    c.dy[pad] = float("inf")
    c.down[1, 3, 5] = float("nan")
    c.apply()
    assert torch.equal(c.y[ids != 1], clean_y[ids != 1])
    out = [torch.empty_like(t) for t in (dx, dd, du)]
    h[pad] = float("nan")
    Q.quip_adapter_backward(c.x, c.dy, c.ids, c.down, c.up, c.scale, h, dx=out[0], dx_base=c.dx_base, d_down=out[1], d_up=out[2])
    assert torch.equal(out[0][ids != 1], dx[ids != 1])
    for l in (0, 2):
        assert torch.equal(out[1][l], dd[l]) and torch.equal(out[2][l], du[l])


@gpu
@pytest.mark.parametrize("T,count", [(1, 1), (64, 3), (1000, 5), (5000, 1), (5000, 1024), (40000, 7)])
@pytest.mark.parametrize("kind", ["random", "runs", "one", "none", "mixed"])
def test_plan_groups_every_token_once(clean, T, count, kind):
    ids = _ids(T, count, kind, np.random.default_rng(T + count))
    plan = Q.quip_adapter_plan(torch.as_tensor(ids.astype(np.int32)).cuda(), count).view(torch.int32).cpu().numpy()
    up4 = lambda v: (v + 3) // 4 * 4
    start = plan[16:16 + count + 2]
    order = plan[16 + up4(count + 2):][:T]
    key = np.where(ids < 0, count, ids)
    np.testing.assert_array_equal(order, np.argsort(key, kind="stable"))
    np.testing.assert_array_equal(start, np.searchsorted(key[order], np.arange(count + 2)))
    at = 16 + up4(count + 2) + up4(T)
    size = np.bincount(key, minlength=count + 1)
    for tile, head in ((128, 3), (8, 4)):
        want = [(l, start[l] + i) for l in range(count + 1) for i in range(0, size[l], tile)]
        assert plan[head] == len(want)
        np.testing.assert_array_equal(plan[at:at + 2 * len(want)].reshape(-1, 2), np.array(want).reshape(-1, 2))
        at += up4(2 * (T // tile + count + 1))
    want = [(l, start[l] + i) for l in range(count) for i in range(0, max(size[l], 1), 1024)]
    assert plan[5] == len(want)
    got = plan[at:at + 4 * len(want)].reshape(-1, 4)
    np.testing.assert_array_equal(got[:, :2], np.array(want).reshape(-1, 2))
    many = np.array([size[l] > 1024 for l, _ in want])
    np.testing.assert_array_equal(got[many, 2], np.arange(many.sum()))
    assert np.all(got[~many, 2] == -1) and many.sum() <= 2 * (T // 1024)


@gpu
def test_bad_ids_and_plans_are_reported():
    Q.load()
    Q.quip_sync_status()
    for T in (3, 200):
        c = Case(T, 64, 64, 32, 2)
        c.ids[1] = 2
        c.apply()
        assert Q.quip_sync_status() == L.QUIP_ERR_ARG
        c.ids[1] = -1
        c.check_apply()
    c = Case(200, 64, 64, 32, 2)
    plan = Q.quip_adapter_plan(c.ids, 2)
    plan.view(torch.int32)[1] = 199                      # a plan of another batch
    c.y.fill_(7)
    c.apply(plan=plan)
    assert Q.quip_sync_status() == L.QUIP_ERR_ARG and torch.all(c.y == 7)
    c.apply(plan=Q.quip_adapter_plan(c.ids, 3))          # of another count, the same bytes
    assert Q.quip_sync_status() == L.QUIP_ERR_ARG and torch.all(c.y == 7)
    with pytest.raises(ValueError):
        c.apply(plan=Q.quip_adapter_plan(c.ids.repeat(9), 2))        # of another size


@gpu
@pytest.mark.parametrize("T", [50, 900])
def test_plans_replays_streams_and_repeats_agree(clean, T):
    c = Case(T, 256, 320, 16, 4)
    first = [t.clone() for t in (*c.apply(), *c.backward())]
    plan = Q.quip_adapter_plan(c.ids, 4)
    assert all(torch.equal(a, b) for a, b in zip(first[:2], c.apply(plan=plan)))
    assert all(torch.equal(a, b) for a, b in zip(first[2:], c.backward(plan=plan)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [*c.apply(stream=side)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[:2], again))
    # two captured calls, each with its own workspace, replayed in turn and beside each other
    graphs, cases = [], [c, Case(T, 256, 320, 16, 4, seed=9)]
    wants = [[t.clone() for t in k.apply()] for k in cases]
    for k in cases:
        k.d_down, k.d_up = torch.empty(k.down.shape, device="cuda"), torch.empty(k.up.shape, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            k.apply()
            Q.quip_adapter_backward(k.x, k.dy, k.ids, k.down, k.up, k.scale, k.h, dx=k.dx, d_down=k.d_down, d_up=k.d_up)
        graphs.append(g)
    for k in cases:
        k.y.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    for k, want in zip(cases, wants):
        assert torch.equal(k.y, want[0]) and torch.equal(k.h, want[1])


@gpu
def test_empty_batch(clean):
    c = Case(4, 64, 32, 4, 2)
    e = slice(0, 0)
    Q.quip_adapter_apply(c.x[e], c.ids[e], c.down, c.up, c.scale, c.y[e])
    d = torch.full((2, 4, 64), float("nan"), device="cuda")
    Q.quip_adapter_backward(c.x[e], c.dy[e], c.ids[e], c.down, c.up, c.scale, c.h[e], d_down=d)
    assert torch.all(d == 0)


@gpu
def test_quantized_layer_with_adapters_to_the_loss(clean):
    # quantized hidden layer + adapters -> quantized output layer -> log
    # probabilities -> gradients of the adapters, against differences in FP64
    rng = np.random.default_rng(5)
    T, n, m, V, r, count, bits = 6, 64, 32, 50, 4, 2, 4

    def layer(rows, cols, seed):
        C = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
        lo, s = np.full(rows, -0.25), np.full(rows, 0.5 / 15)
        tf = Q.Transform(seed, rows, cols, Side("identity"), Side("hadamard"))
        W = O.incoherence_inverse(O.dequantize(C, host(dev(lo)), host(dev(s))), O.SideTransform("identity", rows),
                                  O.make_side(seed, "n", "hadamard", cols))
        return Q.QuantizedLinear(tf, dev(C, torch.uint8), dev(lo), dev(s), bits, max_batch=8), W
    (hidden, W1), (head, W2) = layer(m, n, 1), layer(V, m, 2)
    x = dev(rng.standard_normal((T, n)))
    ad = Q.Adapters(dev(rng.standard_normal((count, r, n)) / 8), dev(rng.standard_normal((count, r, m)) / 2),
                    dev(np.array([0.5, 1.5])))
    ids = torch.tensor([0, 1, -1, 1, 0, 1], dtype=torch.int32, device="cuda")
    tokens = torch.tensor([3, 11, 7, -1, 49, 0], dtype=torch.int32, device="cuda")
    h = torch.empty(T, r, device="cuda")
    y = hidden(x, adapters=ad, ids=ids, h=h)
    logits = head(y)
    lp, ent, lse = (torch.empty(T, device="cuda") for _ in range(3))
    Q.quip_logprobs(logits, tokens, lp, ent, lse)
    d_logits = torch.empty_like(logits)
    g = torch.full((T,), -1.0 / T, device="cuda")
    Q.quip_logprobs_backward(logits, tokens, lse, d_logits, g_logprob=g)
    dy = (d_logits.double() @ torch.as_tensor(W2, device="cuda")).float()        # through the output layer
    d_down, d_up = torch.empty_like(ad.down), torch.empty_like(ad.up)
    Q.quip_adapter_backward(x, dy, ids, ad.down, ad.up, ad.scale, h, d_down=d_down, d_up=d_up)
    args = [host(x), host(ids).astype(int), host(ad.down), host(ad.up), host(ad.scale)]

    def loss(down, up):
        yy, _ = O.adapter_apply(args[0], args[1], down, up, args[4], args[0] @ W1.T)
        return -np.sum(O.token_logprobs(yy @ W2.T, host(tokens).astype(int))[0]) / T
    assert abs(loss(args[2], args[3]) + float(lp.double().mean())) < 1e-5
    for k, (a, got) in enumerate(((args[2], d_down), (args[3], d_up))):
        for i in [(0, 0, 0), (0, 3, 5), (1, 2, 17), (1, 0, 31)]:
            e = np.zeros_like(a)
            e[i] = 1e-4
            p = [args[2], args[3]]
            p[k] = a + e
            up_ = loss(*p)
            p[k] = a - e
            # central differences: 1e-8 of the third derivative's order, fp32 kernels 1e-5 of the gradient's size
            assert abs((up_ - loss(*p)) / 2e-4 - float(got[i])) < 1e-6 + 1e-4 * float(got.abs().max())
    r2 = head.score(y, tokens, top=2)
    assert torch.equal(r2.logprob, lp)
    with pytest.raises(ValueError):
        hidden(x, adapters=ad)


# ------------------------------------------------------------------ buffers that kernels write

def test_buffers_on_the_host_are_refused():
    from post_weight_quantization_09_b200 import _room
    for name in ("plan", "ws"):
        with pytest.raises(ValueError, match=f"{name} must be a CUDA tensor"):
            _room(name, torch.empty(4096, dtype=torch.uint8), 0)


@gpu
def test_plans_and_workspaces_elsewhere_are_refused(clean):
    c = Case(300, 64, 64, 32, 2)
    nbytes = Q.quip_adapter_workspace_size(300, 64, 64, 32, 2, True)
    plan = Q.quip_adapter_plan(c.ids, 2)
    on_host = [torch.empty(nbytes, dtype=torch.uint8, pin_memory=p) for p in (False, True)]
    gaps = torch.empty(2 * nbytes, dtype=torch.uint8, device="cuda")[::2]
    c.y.fill_(7)
    for bad in (*on_host, gaps):
        with pytest.raises(ValueError, match="plan"):
            Q.quip_adapter_plan(c.ids, 2, plan=bad)
        with pytest.raises(ValueError, match="plan"):
            c.apply(plan=bad[:plan.numel()])
        with pytest.raises(ValueError, match="ws"):
            c.apply(ws=bad)
        with pytest.raises(ValueError, match="ws"):
            c.backward(ws=bad)
    assert torch.all(c.y == 7)
    with pytest.raises(Q.QuipError):
        c.apply(ws=gaps[:1])
    # of any type, as long as the bytes are there
    first = [t.clone() for t in (*c.apply(), *c.backward())]
    ws = torch.empty(nbytes // 4, dtype=F, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(first, (*c.apply(ws=ws), *c.backward(ws=ws))))
    again = Q.quip_adapter_plan(c.ids, 2, plan=torch.empty(plan.numel() // 4, dtype=torch.int32, device="cuda"))
    assert torch.equal(again[:6], plan.view(torch.int32)[:6])          # the header


# ------------------------------------------------------------------ rows that end inside 16 bytes

@gpu
@pytest.mark.parametrize("x,y", [(B, B), (B, F), (F, B)])
@pytest.mark.parametrize("T,n,m", [(1, 100, 36), (20, 100, 36), (70, 257, 999), (1500, 1, 7), (2500, 263, 134)])
def test_widths_that_are_no_vectors_in_aligned_rows(clean, T, n, m, x, y):
    # row strides that are multiples of 16 bytes, widths that are not: the
    # buffers end with the last row's last value, and NaN lies between the rows
    c = Case(T, n, m, 16, 2, x, B, y, "runs" if T > 1 else "one")
    for name in ("x", "y", "base", "dy", "dx", "dx_base"):
        t = getattr(c, name)
        ld = (t.shape[1] + 15) // 8 * 8
        buf = torch.full(((T - 1) * ld + t.shape[1],), float("nan"), dtype=t.dtype, device="cuda")
        setattr(c, name, buf.as_strided(t.shape, (ld, 1)).copy_(t))
        if name in ("y", "dx"):
            setattr(c, name + "_buf", buf)
    c.apply()
    c.check_apply()
    c.backward()
    c.check_backward()
    for buf, width in ((c.y_buf, m), (c.dx_buf, n)):
        between = torch.arange(buf.numel(), device="cuda") % ((width + 15) // 8 * 8) >= width
        assert torch.isnan(buf[between]).all() and not torch.isnan(buf[~between]).any()


def test_column_slices_of_one_buffer_are_accepted():
    # Rows of 200 fp32 values hold x in columns [0, 64) and others beside it:
    # no byte is shared.  Such a call gets as far as its workspace, which is too
    # small here; one column less apart and it is refused.
    lib = L.load()
    at = lambda c: ctypes.c_void_p(0x1000000 + 4 * c)

    def fw(y, base=None, ldx=200, ldy=200, T=1100):
        return lib.quip_adapter_apply(at(0), 0, ldx, at(10 ** 8), T, 64, 32, at(2 * 10 ** 8), at(3 * 10 ** 8), 0, 2, 4, None,
                                      base, 200, y, 0, ldy, None, None, None, 0, None)
    for c in (64, 100, 168):
        assert fw(at(c)) == L.QUIP_ERR_WORKSPACE, c
    for c in (0, 1, 63, 169, 199):                                   # 169: the last column is the next row's first
        assert fw(at(c)) == L.QUIP_ERR_ARG, c
    assert fw(at(64 + 200 * 1099)) == L.QUIP_ERR_WORKSPACE           # beside x's last row, then past it
    assert fw(at(63 + 200 * 1099)) == L.QUIP_ERR_ARG
    assert fw(at(200 * 1100 - 1)) == fw(at(200 * 1100)) == L.QUIP_ERR_WORKSPACE
    assert fw(at(-32 - 200 * 1099)) == fw(at(-32)) == L.QUIP_ERR_WORKSPACE
    assert fw(at(-31)) == fw(at(-200 * 1099)) == L.QUIP_ERR_ARG
    assert fw(at(64), base=at(96)) == L.QUIP_ERR_WORKSPACE           # x, y and base side by side
    assert fw(at(64), base=at(95)) == fw(at(96), base=at(65)) == L.QUIP_ERR_ARG
    assert fw(at(100), ldx=201) == L.QUIP_ERR_ARG                    # rows of other lengths: by their span

    def bw(dx, b=None):
        return lib.quip_adapter_backward(at(0), 0, 200, at(64), 0, 200, at(10 ** 8), 1100, 64, 32, at(2 * 10 ** 8),
                                         at(3 * 10 ** 8), 0, 2, 4, None, None, b, 200, dx, 200, at(4 * 10 ** 8), None, 0,
                                         None, None, 0, None)
    assert bw(at(96)) == bw(at(136)) == bw(at(96), at(96)) == L.QUIP_ERR_WORKSPACE
    assert bw(at(95)) == bw(at(137)) == bw(at(20)) == bw(at(96), at(97)) == L.QUIP_ERR_ARG


@gpu
@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("T", [7, 600])
def test_column_slices_of_one_buffer(clean, T, dtype):
    c = Case(T, 264, 136, 16, 3, dtype, B, dtype)
    want = [t.clone() for t in (*c.apply(), *c.backward())]
    buf = torch.full((T, 2 * 264 + 3 * 136 + 3), float("nan"), dtype=dtype, device="cuda")
    at = 1
    for name, width in (("x", 264), ("y", 136), ("base", 136), ("dy", 136), ("dx", 264)):
        part = buf[:, at:at + width]
        part.copy_(getattr(c, name))
        setattr(c, name, part)
        at += width
    got = (*c.apply(), *c.backward())
    assert all(torch.equal(a, b) for a, b in zip(want[2:], got[2:]))
    c.check_apply()
    assert torch.equal(want[0], got[0]) and torch.isnan(buf[:, 0]).all() and torch.isnan(buf[:, at:]).all()


# ------------------------------------------------------------------ long rows

@gpu
@pytest.mark.parametrize("x,w,r,n,count", [
    (F, F, 12, 28672, 1), (F, F, 12, 28672, 1024), (F, F, 64, 9000, 1024), (F, F, 64, 70000, 1), (F, B, 128, 11008, 1),
    (F, B, 128, 11008, 1024), (F, B, 128, 28700, 1), (F, B, 100, 5003, 1024), (B, B, 16, 28672, 1), (B, B, 16, 28672, 1024),
    (B, B, 33, 20000, 1024), (B, B, 96, 28672, 1), (B, B, 128, 2112, 1024), (B, B, 128, 11008, 1024), (B, B, 128, 11007, 1024)])
def test_long_sums_of_one_sign(clean, x, w, r, n, count):
    # Sums whose every term is positive lose what the tensor core drops at each
    # step in one direction.  A step adds 16 products and may drop 2 u of the
    # running sum; at most 1024 columns (64 steps) meet in an accumulator, then
    # fp32 sums of n / 512 + 8 parts, however many adapters are loaded.
    T, m = 2400, 8
    g = torch.Generator().manual_seed(n)
    xs = (torch.rand(T, n, generator=g) + 0.5).to(x).cuda()
    down = torch.zeros(count, r, n, dtype=w, device="cuda")
    down[-1] = (torch.rand(r, n, generator=g) + 0.5).to(w).cuda()
    up = torch.zeros(count, r, m, dtype=w, device="cuda")
    ids = torch.full((T,), count - 1, dtype=torch.int32, device="cuda")
    y, h = torch.empty(T, m, dtype=x, device="cuda"), torch.empty(T, r, device="cuda")
    Q.quip_adapter_apply(xs, ids, down, up, None, y, h=h)
    want = xs.double() @ down[-1].double().T
    off = ((h.double() - want).abs() / want).max().item()
    assert off <= (128 + 8 + n / 512) * U, off / U


# ------------------------------------------------------------------ arguments without their adapters

def test_layer_refuses_what_only_adapters_take():
    layer = object.__new__(Q.QuantizedLinear)
    layer.max_batch = 8
    x = torch.zeros(2, 8)
    for extra in (dict(h=torch.zeros(2, 4)), dict(plan=torch.zeros(256, dtype=torch.uint8)), dict(ids=torch.zeros(2))):
        with pytest.raises(ValueError, match="adapters"):
            layer(x, **extra)


@gpu
@pytest.mark.parametrize("x,w,y", TYPES)
@pytest.mark.parametrize("T,m,pad", [(1, 11008, 0), (16, 4100, 4), (64, 9001, 1)])
def test_few_tokens_in_place(clean, T, m, pad, x, w, y):
    # base is y itself, several rounds of columns per thread
    c = Case(T, 96, m, 16, 3, x, w, y, pad=pad)
    want = c.apply()[0].clone()
    c.y.copy_(c.base)
    Q.quip_adapter_apply(c.x, c.ids, c.down, c.up, c.scale, c.y, base=c.y, h=c.h)
    assert torch.equal(c.y, want)
    c.check_apply()
