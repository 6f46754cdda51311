"""Log probabilities of given tokens, entropy, top alternatives and their
gradient: the kernels against the FP64 oracle, and the refusals.

Tolerances count the kernels' roundings, u = 2^-24 being half a step of
fp32.  Exponentials carry 2^-22 relative (ex2.approx: two steps) plus 2 u per
unit of the exponent; a thread adds at most V / 256 + 64 of them, and every
addition of these non-negative numbers loses at most u of the sum."""
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


@pytest.fixture
def clean():
    Q.load()
    Q.quip_sync_status()
    yield
    assert Q.quip_sync_status() == L.QUIP_OK


# ------------------------------------------------------------------ on the CPU

def test_oracle_gradient_is_the_slope():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 9)) * 2
    x[1, 3] = -np.inf
    tokens = np.array([2, 5, -1, 0])
    g, ge = rng.standard_normal(4), rng.standard_normal(4)

    def value(z):
        lp, H, *_ = O.token_logprobs(z, tokens)
        return np.sum(g * lp) + np.sum(ge * H)
    lp, H, lse, *_ = O.token_logprobs(x, tokens)
    d = O.token_logprobs_grad(x, tokens, lse, H, g, ge)
    for t in range(4):
        for v in range(9):
            if x[t, v] == -np.inf:
                assert d[t, v] == 0
                continue
            e = np.zeros_like(x)
            e[t, v] = 1e-5
            assert abs((value(x + e) - value(x - e)) / 2e-5 - d[t, v]) < 1e-8


def test_oracle_ties_and_empty_rows():
    x = np.array([[1.0, 3.0, 3.0, 1.0], [-np.inf] * 4])
    lp, H, lse, values, ids = O.token_logprobs(x, np.array([1, 2]), 3)
    assert ids[0].tolist() == [1, 2, 0] and ids[1].tolist() == [0, 1, 2]
    assert lp[1] == -np.inf and H[1] == 0 and lse[1] == -np.inf


def test_refusals_answer_on_the_host():
    build()
    lib = L.load()
    f, o = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x100000)
    fw = lambda x=f, dt=L.QUIP_F32, T=2, V=64, ld=64, tok=f, lp=f, k=2, tv=f, ti=f: lib.quip_logprobs(
        x, dt, T, V, ld, tok, lp, None, None, k, tv, ti, None)
    assert fw(x=None) == fw(dt=L.QUIP_U8) == fw(k=-1) == fw(k=33) == fw(tok=None) == fw(lp=None) == L.QUIP_ERR_ARG
    assert fw(tv=None) == fw(ti=None) == L.QUIP_ERR_ARG
    assert fw(T=-1) == fw(V=0) == fw(ld=63) == fw(V=1, ld=64) == L.QUIP_ERR_SHAPE
    assert fw(V=1 << 29, ld=1 << 29) == fw(T=1 << 23) == L.QUIP_ERR_SHAPE
    assert fw(T=1 << 22, V=1 << 28, ld=1 << 28) == L.QUIP_ERR_SHAPE
    assert fw(T=0) == fw(T=0, x=None) == L.QUIP_OK
    bw = lambda x=f, dt=L.QUIP_F32, T=2, V=64, ld=64, tok=f, lse=f, H=f, g=f, ge=f, d=o, ldd=64: \
        lib.quip_logprobs_backward(x, dt, T, V, ld, tok, lse, H, g, ge, d, ldd, None)
    assert bw(x=None) == bw(dt=7) == bw(tok=None) == bw(lse=None) == bw(H=None) == bw(d=None) == L.QUIP_ERR_ARG
    assert bw(d=ctypes.c_void_p(0x1004)) == L.QUIP_ERR_ARG                       # overlaps the logits
    assert bw(d=f, ldd=65) == L.QUIP_ERR_ARG                                     # in place, other rows
    assert bw(ldd=63) == bw(ld=63) == bw(V=0) == L.QUIP_ERR_SHAPE
    assert bw(T=0) == L.QUIP_OK


def test_binding_refuses_host_tensors():
    x, t, o = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        Q.quip_logprobs(x, t, o)
    with pytest.raises(ValueError, match="CUDA"):
        Q.quip_logprobs_backward(x, t, o, x)


# ------------------------------------------------------------------ on the GPU

def _logits(T, V, dtype, seed, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, V, generator=g) * scale
    x[torch.rand(T, V, generator=g) < 0.02] = float("-inf")
    x[:, V // 2] = 0.5
    tokens = torch.randint(0, V, (T,), generator=g).to(torch.int32)
    tokens[torch.rand(T, generator=g) < 0.1] = -1
    return x.to(dtype).cuda(), tokens.cuda()


def _run(x, tokens, k, stream=None):
    T = x.shape[0]
    out = [torch.full((T,), 7.0, device="cuda") for _ in range(3)]
    tv = torch.full((T, k), 7.0, device="cuda")
    ti = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    Q.quip_logprobs(x, tokens, out[0], out[1], out[2], tv if k else None, ti if k else None, stream)
    return (*out, tv, ti)


def _check(x, tokens, k, got):
    x64, V = host(x), x.shape[1]
    lp, H, lse, values, ids = O.token_logprobs(x64, host(tokens).astype(np.int64), k)
    top = x64.max(1)
    fin = np.where(np.isfinite(x64), x64, 0.0)
    p = np.exp(x64 - lse[:, None])
    spread = np.sum(p * np.where(p > 0, top[:, None] - fin, 0.0), 1)          # sum p (max - x)
    rel = 4 * U + (V / 256 + 64) * U + 3 * U * spread                         # of the sum of exponentials
    mag = np.abs(top) + np.log(V) + 1

    def near(a, b, tol):
        live = np.isfinite(b)
        np.testing.assert_array_equal(a[~live], b[~live])
        off = np.abs(a[live] - b[live])
        assert np.all(off <= np.broadcast_to(tol, b.shape)[live]), np.max(off)
    near(host(got[2]), lse, rel + 4 * U * mag)
    gap = np.where(np.isfinite(lp), np.abs(lp), 0.0)
    near(host(got[0]), lp, rel + 4 * U * (mag + gap))
    # H = ln s - w / s: the errors of ln s, of w (its terms lose rel and 2 U more) and of the quotient
    near(host(got[1]), H, rel + (2 * rel + 8 * U) * (spread + 1) + 8 * U * np.log(V))
    if k:
        np.testing.assert_array_equal(got[4].cpu().numpy(), ids)
        gap = np.where(np.isfinite(values), np.abs(values), 0.0)
        near(host(got[3]), values, (rel + 4 * U * mag)[:, None] + 4 * U * gap)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (1, 1, 0), (2, 7, 7), (3, 33, 32), (5, 100, 20), (1, 4095, 1),
                                   (700, 257, 2), (4, 32000, 8), (1, 50257, 32), (9, 128000, 20), (130, 8193, 5),
                                   (1000, 4096, 3), (891, 4101, 0), (2100, 5001, 32)])
def test_logprobs_match_oracle(clean, T, V, k, dtype):
    x, tokens = _logits(T, V, dtype, 7 * T + V + k)
    _check(x, tokens, k, _run(x, tokens, k))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_unaligned_and_strided_rows(clean, shift, dtype):
    T, V = 6, 4099
    x, tokens = _logits(T, V, dtype, shift)
    buf = torch.full((T, V + 3 + shift), float("nan"), dtype=dtype, device="cuda")
    view = buf[:, shift:shift + V]
    view.copy_(x)
    a, b = _run(view, tokens, 9), _run(x, tokens, 9)
    _check(x, tokens, 9, a)
    assert torch.equal(a[4], b[4])


@gpu
def test_large_magnitudes(clean):
    # logits around 5000: lse and logprob lose U of 5000, entropy nothing of it
    x, tokens = _logits(3, 5000, torch.float32, 1)
    x = torch.where(torch.isfinite(x), (x + 5000), x)
    _check(x, tokens, 4, _run(x, tokens, 4))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masks_of_the_lowest_value(clean, dtype):
    # entries barred by the type's lowest value: beside real logits, alone, and beside -inf
    x, tokens = _logits(5, 6000, dtype, 12)
    low = torch.finfo(dtype).min
    x[0, 100:3000] = low
    x[1] = low
    x[2] = low
    x[2, ::3] = float("-inf")
    x[3] = float("-inf")
    x[3, 4321] = low
    x[4] = 1e30
    x[4, 7:] = -1e30
    tokens[:] = torch.tensor([150, 5, 4, 4321, 3])
    lp, H, lse, tv, ti = _run(x, tokens, 5)
    assert torch.equal(ti[1:].cpu(), torch.tensor([[0, 1, 2, 3, 4], [1, 2, 4, 5, 7], [4321, 0, 1, 2, 3], [0, 1, 2, 3, 4]],
                                                  dtype=torch.int32))
    n = np.array([6000, 4000, 1, 7])
    assert host(lp)[0] == float(low) and np.all(host(lse)[1:4] == float(low))
    np.testing.assert_allclose(host(lp)[1:], -np.log(n), rtol=4 * U, atol=0)
    np.testing.assert_allclose(host(H)[1:], np.log(n), rtol=4 * U, atol=0)
    np.testing.assert_allclose(host(tv)[1:3], -np.log(n[:2, None]) * np.ones(5), rtol=4 * U, atol=0)
    assert host(tv)[3, 0] == 0 and np.all(host(tv)[3, 1:] == -np.inf)


@gpu
@pytest.mark.parametrize("kind", ["constant", "falling", "rising", "one_thread", "two_values", "zeros"])
@pytest.mark.parametrize("V", [255, 9000, 70000])
def test_ties_and_orders_that_crowd_the_candidates(clean, kind, V):
    T = 2 if V != 9000 else 900
    x = {"constant": torch.full((2, V), 1.5),
         "falling": -torch.arange(V).float()[None].repeat(2, 1) / 64,
         "rising": torch.arange(V).float()[None].repeat(2, 1) / 64,
         # the largest logits all in vectors that one thread of a 256-thread CTA reads
         "one_thread": ((torch.arange(V) // 4 % 256) == 3).float()[None].repeat(2, 1) * 4 + torch.linspace(0, 1, V),
         "two_values": (torch.arange(V) % 3 == 1).float()[None].repeat(2, 1),
         "zeros": torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)[None].repeat(2, 1)}[kind].cuda()
    x = x.repeat(T // 2, 1)
    tokens = torch.tensor([0, V - 1], dtype=torch.int32, device="cuda").repeat(T // 2)
    _check(x, tokens, 32, _run(x, tokens, 32))


@gpu
def test_empty_rows_nan_and_infinity(clean):
    x, tokens = _logits(6, 3001, torch.float32, 3)
    tokens.fill_(5)
    x[1] = float("-inf")
    x[2, 77] = float("nan")
    x[3, 5] = float("inf")
    x[4] = float("nan")
    got = [host(t) for t in _run(x, tokens, 4)]
    assert got[0][1] == -np.inf and got[1][1] == 0 and got[2][1] == -np.inf
    assert np.all(got[3][1] == -np.inf) and got[4][1].tolist() == [0, 1, 2, 3]
    for r in (2, 3, 4):
        assert np.isnan(got[0][r]) and np.isnan(got[1][r]) and np.isnan(got[2][r]) and np.all(np.isnan(got[3][r]))
        assert np.all((got[4][r] >= 0) & (got[4][r] < 3001))
    keep = torch.tensor([0, 5], device="cuda")
    _check(x[keep], tokens[keep], 4, [torch.as_tensor(t).cuda()[keep] for t in got])
    d = torch.full_like(x, 7.0)
    lse, H = (torch.as_tensor(got[i], dtype=torch.float32).cuda() for i in (2, 1))
    g = torch.tensor([1.0, 1.0, 1.0, 1.0, 0.0, 0.0], device="cuda")
    Q.quip_logprobs_backward(x, tokens, lse, d, g_logprob=g, g_entropy=torch.zeros(6, device="cuda"), entropy=H)
    assert torch.all(d[1] == 0) and torch.all(d[4] == 0) and torch.all(d[5] == 0)
    assert torch.isnan(d[2]).all() and torch.isnan(d[3]).all() and torch.isfinite(d[0]).all()


@gpu
def test_tokens_out_of_range_are_reported():
    Q.load()
    Q.quip_sync_status()
    x, _ = _logits(2, 100, torch.float32, 3)
    for bad in (100, -2):
        tokens = torch.tensor([4, bad], dtype=torch.int32, device="cuda")
        got = _run(x, tokens, 0)
        assert Q.quip_sync_status() == L.QUIP_ERR_ARG
        assert host(got[0])[1] == 0
        d = torch.empty_like(x)
        Q.quip_logprobs_backward(x, tokens, got[2], d, g_logprob=torch.ones(2, device="cuda"))
        assert Q.quip_sync_status() == L.QUIP_ERR_ARG
        assert torch.all(d[1] == 0)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,pad,inplace", [(1, 1, 0, False), (3, 37, 3, False), (5, 4096, 0, True), (2, 32000, 8, False),
                                             (4, 9001, 1, True), (300, 260, 0, False)])
def test_gradient_matches_oracle(clean, T, V, pad, inplace, dtype):
    x, tokens = _logits(T, V, dtype, T + V)
    buf = torch.full((T, V + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :V] = x
    x = buf[:, :V]
    rng = np.random.default_rng(T)
    g, ge = rng.standard_normal(T).astype(np.float32), rng.standard_normal(T).astype(np.float32)
    g[0], ge[-1] = 0.5, 0.0
    _, H, lse, _, _ = _run(x, tokens, 0)
    x64 = host(x)
    out = x if inplace else torch.empty(T, V, dtype=dtype, device="cuda")
    Q.quip_logprobs_backward(x, tokens, lse, out, g_logprob=dev(g), g_entropy=dev(ge), entropy=H)
    tok = host(tokens).astype(np.int64)
    want = O.token_logprobs_grad(x64, tok, host(lse), host(H), g.astype(np.float64), ge.astype(np.float64))
    g64 = np.where(tok >= 0, np.abs(g), 0.0)[:, None]
    logp = np.where(np.isfinite(x64), x64 - host(lse)[:, None], 0.0)
    p = np.exp(np.where(np.isfinite(x64), x64 - host(lse)[:, None], -np.inf))
    # p loses 4 u + 3 u |ln p|; the factor (g + ge H) + ge ln p 4 u of its parts; the token's g one more u
    size = p * (g64 + np.abs(ge)[:, None] * (host(H)[:, None] + np.abs(logp)))
    tol = size * (8 + 3 * np.abs(logp)) * U + U * np.abs(want) + 1e-37
    tol[np.arange(T), np.maximum(tok, 0)] += 2 * U * g64[:, 0]
    tol += np.abs(want) * torch.finfo(dtype).eps / 2 * (1 + 1e-3)
    assert np.all(np.abs(host(out) - want) <= tol), np.max(np.abs(host(out) - want) / tol)
    if pad:
        assert torch.isnan(buf[:, V:]).all()


@gpu
def test_row_offsets_past_32_bits(clean):
    T, V, ld = 4, 5000, 2 ** 30 + 8
    x, tokens = _logits(T, V, torch.bfloat16, 17)
    far = torch.empty((T - 1) * ld + V, dtype=torch.bfloat16, device="cuda").as_strided((T, V), (ld, 1)).copy_(x)
    got, want = _run(far, tokens, 9), _run(x, tokens, 9)
    _check(x, tokens, 9, got)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.linspace(-1, 1, T, device="cuda")
    d = torch.empty_like(x)
    for logits, out in ((x, d), (far, far)):
        Q.quip_logprobs_backward(logits, tokens, want[2], out, g_logprob=g, g_entropy=g, entropy=want[1])
    assert torch.equal(far, d)


@gpu
def test_gradient_parts_may_be_absent(clean):
    x, tokens = _logits(3, 500, torch.float32, 8)
    _, H, lse, _, _ = _run(x, tokens, 0)
    z, o = torch.zeros(3, device="cuda"), torch.ones(3, device="cuda")
    both, one = torch.empty_like(x), torch.empty_like(x)
    Q.quip_logprobs_backward(x, tokens, lse, both, g_logprob=o, g_entropy=z, entropy=H)
    Q.quip_logprobs_backward(x, tokens, lse, one, g_logprob=o)
    assert torch.equal(both, one)
    Q.quip_logprobs_backward(x, tokens, lse, both, g_logprob=z, g_entropy=o, entropy=H)
    Q.quip_logprobs_backward(x, None, lse, one, g_entropy=o, entropy=H)
    assert torch.equal(both, one)


@gpu
def test_replays_streams_and_repeats_agree(clean):
    x, tokens = _logits(40, 32000, torch.bfloat16, 11)
    want = _run(x, tokens, 20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _run(x, tokens, 20, side)
    torch.cuda.synchronize()
    for a, b in zip(want, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _run(x, tokens, 20)
        d = torch.empty_like(x)
        Q.quip_logprobs_backward(x, tokens, got[2], d, g_logprob=got[0], g_entropy=got[1], entropy=got[1])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    d2 = torch.empty_like(x)
    Q.quip_logprobs_backward(x, tokens, want[2], d2, g_logprob=want[0], g_entropy=want[1], entropy=want[1])
    assert torch.equal(d.view(torch.int16), d2.view(torch.int16))   # bits: a barred token has gradient NaN


@gpu
def test_rows_behind_the_last_are_left_as_they_were(clean):
    x, tokens = _logits(5, 700, torch.float32, 2)
    out = torch.full((8,), 7.0, device="cuda")
    Q.quip_logprobs(x, tokens, out[:5])
    assert torch.all(out[5:] == 7.0)
    Q.quip_logprobs(x[:0], tokens[:0], out[:0])


@gpu
def test_score_of_a_quantized_output_layer(clean):
    m, n, bits, T = 200, 64, 4, 11
    rng = np.random.default_rng(4)
    C = rng.integers(0, 16, (m, n)).astype(np.uint8)
    lo, s = np.full(m, -0.5), np.full(m, 1 / 15)
    tf = Q.Transform(3, m, n, Side("identity"), Side("hadamard"))
    ql = Q.QuantizedLinear(tf, dev(C, torch.uint8), dev(lo), dev(s), bits, max_batch=4)
    x = dev(rng.standard_normal((T, n)))
    tokens = torch.arange(T, dtype=torch.int32, device="cuda") * 3
    tokens[2] = -1
    r = ql.score(x, tokens, top=3)
    logits = torch.cat([ql(x[a:a + 4]) for a in range(0, T, 4)])
    _check(logits, tokens, 3, (r.logprob, r.entropy, r.lse, r.top_values, r.top_ids))
    assert ql.score(x, tokens).top_ids is None
    with pytest.raises(ValueError):
        ql.score(x, tokens, top=33)
    with pytest.raises(ValueError):
        ql.score(x, tokens[:3])
    tf.close()


# ------------------------------------------------------------------ finite masks

def _masked(T, V, dtype, value, seed):
    """Random rows with `value` at, row by row: half the entries, 99 in 100,
    a stretch of up to 4096, all but one."""
    x, tokens = _logits(T, V, dtype, seed)
    g = torch.Generator().manual_seed(seed)
    kind = (torch.arange(T) % 4)[:, None]
    v, start = torch.arange(V)[None], torch.randint(0, max(V - 4096, V // 4), (T, 1), generator=g)
    mask = torch.where(kind == 0, torch.rand(T, V, generator=g) < 0.5, torch.rand(T, V, generator=g) < 0.99)
    mask = torch.where(kind == 2, (v >= start) & (v < start + 4096), mask) | (kind == 3)
    mask[:, V // 2] = False
    x.masked_fill_(mask.cuda(), value)
    return x, tokens


MASKS = [-1e9, -1e10, -1e12, -1e20, -1e30, -1e38, "half", "min"]


def _mask_value(value, dtype):
    return {"half": torch.finfo(dtype).min / 2, "min": torch.finfo(dtype).min}.get(value, value)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", MASKS)
@pytest.mark.parametrize("T,V,k", [(1, 500, 3), (700, 500, 0), (700, 500, 5), (4, 32000, 8), (4, 128000, 20), (600, 9000, 2)])
def test_finite_masks_count_nothing(clean, T, V, k, value, dtype):
    x, tokens = _masked(T, V, dtype, _mask_value(value, dtype), T + V)
    _check(x, tokens, k, _run(x, tokens, k))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", MASKS)
def test_gradient_beside_finite_masks(clean, value, dtype):
    T, V = 8, 9001
    x, tokens = _masked(T, V, dtype, _mask_value(value, dtype), 5)
    tokens.fill_(V // 2)
    _, H, lse, _, _ = _run(x, tokens, 0)
    g, ge = torch.linspace(-1, 1, T, device="cuda"), torch.linspace(0.5, 1.5, T, device="cuda")
    d = torch.empty_like(x)
    Q.quip_logprobs_backward(x, tokens, lse, d, g_logprob=g, g_entropy=ge, entropy=H)
    x64, lse64, H64, g64, ge64 = (host(t) for t in (x, lse, H, g, ge))
    want = O.token_logprobs_grad(x64, host(tokens).astype(np.int64), lse64, H64, g64, ge64)
    logp = np.maximum(x64 - lse64[:, None], -1000.0)
    # as in test_gradient_matches_oracle
    size = np.exp(logp) * (np.abs(g64)[:, None] + ge64[:, None] * (H64[:, None] + np.abs(logp)))
    tol = size * (8 + 3 * np.abs(logp)) * U + np.abs(want) * (U + torch.finfo(dtype).eps / 2 * (1 + 1e-3)) + 1e-37
    tol[:, V // 2] += 2 * U * np.abs(g64)
    assert np.all(np.abs(host(d) - want) <= tol), np.nanmax(np.abs(host(d) - want) / tol)


# ------------------------------------------------------------------ gradients of rows far from 0

def _far_rows(kind, dtype):
    """(x, tokens) of 6 rows of logits whose log-sum-exp is far from 0."""
    x, tokens = _logits(6, 9001, dtype, 21)
    tokens[:] = torch.tensor([9001 // 2, 7, 0, -1, 9000, 4096])
    if kind == "equal":                  # equal logits of any size, beside -inf
        x = torch.where(torch.isfinite(x), torch.tensor([1e9, -1e9, 3e38, -3e38, 300.0, -5e5])[:, None].cuda(), x.float())
    elif kind == "lowest":               # rows of the type's lowest value alone
        x = torch.where(torch.isfinite(x), torch.finfo(dtype).min, x.float())
    else:
        x = x.float() + kind
    x[torch.arange(6), tokens.long().clamp(min=0).cpu()] = x.amax(1)
    return x.to(dtype), tokens


def _far_check(x, tokens, g, ge, got):
    """Against the oracle's own log-sum-exp and entropy: p loses 4 u + 3 u
    |ln p| by its own arithmetic, and what lse lost: its computation (_check)
    and at most half a step below 256, where the row itself is not looked at
    again; else u of each of the few additions that correct it, ln V in size."""
    x64, tok, V = host(x), host(tokens).astype(np.int64), x.shape[1]
    far = np.abs(x64.max(1))
    x64 = x64 - x64.max(1)[:, None]              # the gradient does not see it; FP64 would at 3e38
    _, H, lse, _, _ = O.token_logprobs(x64, tok)
    want = O.token_logprobs_grad(x64, tok, lse, H, host(g), host(ge))
    logp = np.maximum(x64 - lse[:, None], -1000.0)
    p = np.exp(logp)
    spread = np.sum(p * -np.maximum(x64, -1000.0), 1)
    rel = 4 * U + (V / 256 + 64) * U + 3 * U * spread
    err = rel + 4 * U * (np.minimum(far, 256.0) + 2 * np.log(V) + 1)
    err_h = rel + (2 * rel + 8 * U) * (spread + 1) + 8 * U * np.log(V)
    g64 = np.where(tok >= 0, np.abs(host(g)), 0.0)[:, None]
    ge64 = np.abs(host(ge))[:, None]
    size = p * (g64 + ge64 * (H[:, None] + np.abs(logp)))
    tol = size * ((8 + 3 * np.abs(logp)) * U + err[:, None]) + p * ge64 * (err + err_h)[:, None] + 1e-37
    tol[np.arange(len(tok)), np.maximum(tok, 0)] += 2 * U * g64[:, 0]
    tol += (np.abs(want) + tol) * (U + torch.finfo(x.dtype).eps / 2 * (1 + 1e-3))
    off = np.abs(host(got) - want)
    assert np.all(off <= tol), np.nanmax(off / tol)
    assert np.all(host(got)[x64 == -np.inf] == 0)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", [100.0, -300.0, 5000.0, 1e6, -1e6, "equal", "lowest"])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_far_from_zero(clean, kind, dtype, inplace, entropy):
    x, tokens = _far_rows(kind, dtype)
    keep = x.clone()
    _, H, lse, _, _ = _run(x, tokens, 0)
    g = torch.tensor([-1.0, 0.5, 2.0, 1.0, -0.25, 1.0], device="cuda")
    ge = torch.linspace(-1, 1, 6, device="cuda") * entropy
    out = x if inplace else torch.full_like(x, 7.0)
    Q.quip_logprobs_backward(x, tokens, lse, out, g_logprob=g, g_entropy=ge if entropy else None, entropy=H)
    _far_check(keep, tokens, g, ge, out)


@gpu
@pytest.mark.parametrize("V,pad,shift", [(1, 0, 0), (3, 1, 0), (257, 3, 1), (40000, 5, 3)])
def test_gradient_far_from_zero_in_strided_rows(clean, V, pad, shift):
    T = 5
    x, tokens = _logits(T, V, torch.float32, V, scale=1.0)
    x += 7000.0
    buf, out = (torch.full((T, V + pad + shift), float("nan"), device="cuda") for _ in range(2))
    view, d = buf[:, shift:shift + V], out[:, shift:shift + V]
    view.copy_(x)
    _, H, lse, _, _ = _run(view, tokens, 0)
    g = torch.linspace(-1, 1, T, device="cuda")
    Q.quip_logprobs_backward(view, tokens, lse, d, g_logprob=g, g_entropy=g, entropy=H)
    _far_check(x, tokens, g, g, d)
    out[:, shift:shift + V] = float("nan")
    assert torch.isnan(out).all()


@gpu
def test_gradient_with_the_sum_of_a_larger_vocabulary(clean):
    # the rows are shards: lse is that of the whole row, 1 more than the shard's
    x, tokens = _logits(4, 5000, torch.float32, 9)
    x += 5000.0
    lse = _run(x, tokens, 0)[2] + 1.0
    g = torch.ones(4, device="cuda")
    d = torch.empty_like(x)
    Q.quip_logprobs_backward(x, tokens, lse, d, g_logprob=g)
    x64, lse64 = host(x), host(lse)
    want = O.token_logprobs_grad(x64, host(tokens).astype(np.int64), lse64, np.zeros(4), np.ones(4), np.zeros(4))
    p = np.exp(x64 - lse64[:, None])
    tol = p * (8 + 3 * np.maximum(lse64[:, None] - x64, 0).clip(max=1000)) * U + 2 * U * np.abs(want) + 1e-37
    assert np.all(np.abs(host(d) - want) <= tol)


@gpu
def test_gradient_into_other_columns_of_the_logits_buffer(clean):
    x, tokens = _logits(6, 1000, torch.float32, 4)
    _, H, lse, _, _ = _run(x, tokens, 0)
    g = torch.linspace(-1, 1, 6, device="cuda")
    want, buf = torch.empty_like(x), torch.full((6, 2010), float("nan"), device="cuda")
    Q.quip_logprobs_backward(x, tokens, lse, want, g_logprob=g, g_entropy=g, entropy=H)
    buf[:, :1000] = x
    Q.quip_logprobs_backward(buf[:, :1000], tokens, lse, buf[:, 1003:2003], g_logprob=g, g_entropy=g, entropy=H)
    assert torch.equal(buf[:, 1003:2003], want) and torch.equal(buf[:, :1000], x)
    assert torch.isnan(buf[:, 1000:1003]).all() and torch.isnan(buf[:, 2003:]).all()
    with pytest.raises(Q.QuipError):
        Q.quip_logprobs_backward(buf[:, :1000], tokens, lse, buf[:, 999:1999], g_logprob=g)
