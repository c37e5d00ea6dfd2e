"""The int8 products by the forms they are cut in, against 64-bit formulas."""
import pytest
import torch

from activation_sparse_gated_tma_b200 import twell as tw
from tests.test_gpu_int8 import BF16, F16, F32, U, _check, _half_step, _operand, _product64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(5, 300, 256), (200, 300, 256), (700, 300, 256), (2500, 2600, 640), (2049, 5130, 1000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gated_product_of_up_channels_without_a_scale(M, N, K, dtype):
    # h = u ReLU(g): where u is NaN so is h, for any g, and an infinite u gives NaN where ReLU(g) is 0.
    x, xs = _operand(M, K, 1)
    wg, gs = _operand(N, K, 2)
    wu, us = _operand(N, K, 3)
    good = tw.int8_gated(x, xs, wg, gs, wu, us, out_dtype=dtype)
    us[17], us[N - 1], us[40] = float("nan"), float("nan"), float("inf")
    h = tw.int8_gated(x, xs, wg, gs, wu, us, out_dtype=dtype)
    assert bool(h[:, 17].isnan().all()) and bool(h[:, N - 1].isnan().all())
    ref = _product64(x, xs, wg[40:41], gs[40:41]).clamp_min(0) * _product64(x, xs, wu[40:41], us[40:41])
    assert torch.equal(h[:, 40:41].isnan(), ref.isnan()) and bool(ref.isnan().any())
    assert torch.equal(h[:, 40:41].isinf(), ref.isinf())
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[[17, 40, N - 1]] = False
    assert torch.equal(h[:, keep], good[:, keep])


# ---------------------------------------------------------------- every cut
TILES = [(tile, s) for tile in (16, 32, 64, 128) for s in (1, 2, 4, 8)]
PAIRS = (256, 1)


@pytest.fixture
def cut():
    yield tw.int8_cut
    tw.int8_cut()


def _linear_in(cut, how, M, N, K, dtype, bias, gap):
    x, xs = _operand(M, K, 1)
    w, ws = _operand(N, K, 2, gap=16)
    b = torch.randn(N, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") if bias else None
    out = torch.full((M + 2, N + gap), 7.0, device="cuda", dtype=dtype)
    cut(*how)
    y = tw.int8_linear(x, xs, w, ws, bias=b, out=out[1:M + 1, :N])
    ref = _product64(x, xs, w, ws)
    tol = 8 * U * (ref.abs() + (b.double().abs() if bias else 0.0))
    if bias:
        ref = ref + b.double()
    _check(y, ref, tol + _half_step(dtype, ref))
    # A token and a channel without a scale, a token of scale 0: they stay by themselves.
    xs[M // 2], ws[N - 1] = float("nan"), float("nan")
    xs[0] = 0.0
    z = tw.int8_linear(x, xs, w, ws, bias=b, out_dtype=dtype)
    keep = torch.ones((M, N), dtype=torch.bool, device="cuda")
    keep[0], keep[M // 2], keep[:, N - 1] = False, False, False
    assert torch.equal(z[keep], y[keep])
    assert bool(z[M // 2].isnan().all()) and bool(z[:, N - 1].isnan().all())
    assert torch.equal(z[0, :-1], (b[:-1] if bias else torch.zeros(N - 1, device="cuda")).to(dtype))
    out[1:M + 1, :N] = 7.0
    assert bool((out == 7.0).all()), "written outside the output's rows"
    return y


def _gated_in(cut, how, M, N, K, dtype, gap):
    x, xs = _operand(M, K, 1)
    wg, gs = _operand(N, K, 2, gap=48)
    wu, us = _operand(N, K, 3)
    out = torch.full((M + 2, N + gap), 7.0, device="cuda", dtype=dtype)
    cut(*how)
    h = tw.int8_gated(x, xs, wg, gs, wu, us, out=out[1:M + 1, :N])
    ref = _product64(x, xs, wg, gs).clamp_min(0) * _product64(x, xs, wu, us)
    _check(h, ref, 8 * U * ref.abs() + _half_step(dtype, ref))
    xs[M // 2], gs[N - 1], us[N // 3] = float("nan"), float("nan"), float("nan")
    z = tw.int8_gated(x, xs, wg, gs, wu, us, out_dtype=dtype)
    keep = torch.ones((M, N), dtype=torch.bool, device="cuda")
    keep[M // 2], keep[:, N - 1], keep[:, N // 3] = False, False, False
    assert torch.equal(z[keep], h[keep]) and bool(z[~keep].isnan().all())
    out[1:M + 1, :N] = 7.0
    assert bool((out == 7.0).all()), "written outside the output's rows"


@pytest.mark.parametrize("how", TILES + [PAIRS])
@pytest.mark.parametrize("dtype,bias,gap", [(BF16, False, 2), (F32, True, 1), (F16, True, 6)])
def test_int8_linear_in_every_cut(cut, how, dtype, bias, gap):
    # 1000 is eight 128-wide blocks, the last one in part; no tile divides 300 tokens or 390 channels.
    _linear_in(cut, how, 300, 390, 1000, dtype, bias, gap)


@pytest.mark.parametrize("how", [h for h in TILES if h[0] < 128 or h[1] == 1] + [PAIRS])
@pytest.mark.parametrize("dtype,gap", [(BF16, 2), (F32, 1), (F16, 6)])
def test_int8_gated_in_every_cut(cut, how, dtype, gap):
    _gated_in(cut, how, 300, 390, 1000, dtype, gap)


# (More than four tiles a pair of SMs; a last sweep of fewer than eight token blocks; one 128-wide block; one tile.)
PAIR_SHAPES = [(5000, 5130, 640), (2049, 5130, 1000), (2600, 9000, 96), (256, 256, 128), (1, 1, 1), (257, 129, 4093)]


@pytest.mark.parametrize("M,N,K", PAIR_SHAPES)
@pytest.mark.parametrize("dtype,bias,gap", [(BF16, False, 6), (F32, True, 0), (F32, False, 3)])
def test_int8_linear_on_cta_pairs(cut, M, N, K, dtype, bias, gap):
    if M > 1:
        _linear_in(cut, PAIRS, M, N, K, dtype, bias, gap)
    cut(*PAIRS)
    x, xs = _operand(M, K, 1)
    w, ws = _operand(N, K, 2)
    y = tw.int8_linear(x, xs, w, ws, out_dtype=dtype)
    cut(64, 1)
    assert torch.equal(y, tw.int8_linear(x, xs, w, ws, out_dtype=dtype)), "another cut gives other bits"


@pytest.mark.parametrize("M,N,K", PAIR_SHAPES)
@pytest.mark.parametrize("dtype,gap", [(BF16, 0), (BF16, 6), (F32, 3)])
def test_int8_gated_on_cta_pairs(cut, M, N, K, dtype, gap):
    if M > 1:
        _gated_in(cut, PAIRS, M, N, K, dtype, gap)
    cut(*PAIRS)
    x, xs = _operand(M, K, 1)
    wg, gs = _operand(N, K, 2)
    wu, us = _operand(N, K, 3)
    h = tw.int8_gated(x, xs, wg, gs, wu, us, out_dtype=dtype)
    cut(32, 1)
    assert torch.equal(h, tw.int8_gated(x, xs, wg, gs, wu, us, out_dtype=dtype)), "another cut gives other bits"


@pytest.mark.parametrize("M,N", [(3, 130), (300, 600)])
def test_longest_sums_on_cta_pairs(cut, M, N):
    K = 131071
    x = torch.full((M, -(-K // 16) * 16), -128, dtype=torch.int8, device="cuda")[:, :K]
    w = torch.full((N, -(-K // 16) * 16), -128, dtype=torch.int8, device="cuda")[:, :K]
    w[1], w[2, ::2] = 127, 127
    one = torch.ones
    cut(*PAIRS)
    y = tw.int8_linear(x, one(M, device="cuda"), w, one(N, device="cuda"), out_dtype=F32)
    exact = x[:1].double() @ w.double().t()
    assert torch.equal(y, exact.float().expand(M, N))


def test_cuts_that_a_product_does_not_allow(cut):
    x, xs = _operand(20, 256, 1)
    w, ws = _operand(40, 256, 2)
    cut(16, 4)      # two 128-wide blocks for four shares
    with pytest.raises(tw.TwellError):
        tw.int8_linear(x, xs, w, ws)
    cut(128, 2)
    tw.int8_linear(x, xs, w, ws)
    with pytest.raises(tw.TwellError):
        tw.int8_gated(x, xs, w, ws, w, ws)


def test_pairs_replayed_from_a_graph(cut):
    x, xs = _operand(3000, 320, 1)
    w, ws = _operand(2600, 320, 2)
    cut(*PAIRS)

    def step():
        return tw.int8_linear(x, xs, w, ws), tw.int8_gated(x, xs, w, ws, w, ws)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    xs.mul_(2)
    ref = step()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))


# ---------------------------------------------------------------- a wait that gives up
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pairs_whose_wait_gave_up_write_nan_from_then_on(cut, gated, dtype):
    # The MMAs stop after every pair's first tile (host-side injection, waits of 1 ms): those tiles are right, all later
    # ones NaN, however often the accumulators' barriers would have turned over since; the next call is right again.
    M, N, K = 5000, 5130, 640
    x, xs = _operand(M, K, 1)
    wg, gs = _operand(N, K, 2)
    wu, us = _operand(N, K, 3)

    def call():
        return (tw.int8_gated(x, xs, wg, gs, wu, us, out_dtype=dtype) if gated
                else tw.int8_linear(x, xs, wg, gs, out_dtype=dtype))
    cut(*PAIRS)
    good = call()
    tw.test_expire_wait(1_000_000)
    y = call()
    torch.cuda.synchronize()
    units = 128 if gated else 256
    right = 0
    for m in range(0, M, 256):
        for n in range(0, N, units):
            a, b = y[m:m + 256, n:n + units], good[m:m + 256, n:n + units]
            whole = bool(torch.equal(a, b))
            right += whole
            assert whole or bool(a.isnan().all()), (m, n)
    assert right == torch.cuda.get_device_properties(0).multi_processor_count // 2
    assert torch.equal(call(), good)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("how", [(16, 1), (16, 4), (32, 2), (64, 1), (128, 1)])
def test_tiles_whose_wait_gave_up_are_nan(cut, gated, how):
    x, xs = _operand(70, 1000, 1)
    wg, gs = _operand(300, 1000, 2)
    wu, us = _operand(300, 1000, 3)

    def call():
        return tw.int8_gated(x, xs, wg, gs, wu, us) if gated else tw.int8_linear(x, xs, wg, gs)
    cut(*how)
    good = call()
    tw.test_expire_wait(100_000)
    assert bool(call().isnan().all())
    assert torch.equal(call(), good)
