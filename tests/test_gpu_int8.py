"""The int8 products with scales per token and channel on the GPU against
64-bit formulas, and the FFN paths that use them and the norm.

The integer sum is exact; float(sum), two products and the bias are four fp32
roundings (u = 2^-24 each), and the output adds its type's half step."""
import numpy as np
import pytest
import torch

from activation_sparse_gated_tma_b200 import twell as tw
from activation_sparse_gated_tma_b200 import workloads as wl
from oracle import backward as ob
from tests import parity as P
from tests.test_gpu_backward import _active_mask

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _half_step(dtype, v):
    return torch.finfo(dtype).eps / 2 * v.abs() + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def _operand(R, K, seed, gap=0):
    """int8 rows (all values, -128 too) and scales; bytes between rows hold what must not be read."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = -(-K // 16) * 16 + gap
    q = torch.randint(-128, 128, (R, ld), generator=g, device="cuda", dtype=torch.int8)
    s = torch.exp(0.5 * torch.randn(R, generator=g, device="cuda")) / (100 * K ** 0.5)
    return q[:, :K], s


def _product64(x, xs, w, ws):
    return (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()


def _check(y, ref, tol):
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


SHAPES = [(1, 1, 1), (1, 128, 32), (2, 5, 16), (3, 130, 128), (16, 1024, 2048), (17, 129, 127), (31, 64, 100), (33, 300, 640),
          (64, 257, 512), (65, 1000, 333), (127, 128, 4093), (128, 512, 256), (129, 384, 1024), (256, 2048, 1536),
          (300, 257, 640), (513, 1535, 4093), (1000, 130, 96), (2049, 600, 200), (4, 70000, 64), (5000, 17, 31)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype,bias", [(BF16, False), (F32, True)])
def test_int8_linear(M, N, K, dtype, bias):
    x, xs = _operand(M, K, 1)
    w, ws = _operand(N, K, 2, gap=16)
    b = torch.randn(N, device="cuda") if bias else None
    y = tw.int8_linear(x, xs, w, ws, bias=b, out_dtype=dtype)
    assert tw.last_launch_count() == 1
    p = _product64(x, xs, w, ws)
    ref = p if b is None else p + b.double()
    _check(y, ref, (4 * U * p.abs() + U * ref.abs()) * 1.01 + _half_step(dtype, ref))
    assert torch.equal(y, tw.int8_linear(x, xs, w, ws, bias=b, out_dtype=dtype)), "not the same bits twice"


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_int8_gated(M, N, K, dtype):
    x, xs = _operand(M, K, 1)
    wg, gs = _operand(N, K, 2)
    wu, us = _operand(N, K, 3, gap=32)
    h = tw.int8_gated(x, xs, wg, gs, wu, us, out_dtype=dtype)
    ref = _product64(x, xs, wg, gs).clamp_min(0) * _product64(x, xs, wu, us)
    _check(h, ref, 8 * U * ref.abs() + _half_step(dtype, ref))


@pytest.mark.parametrize("M,N", [(3, 130), (40, 129), (200, 256)])
def test_int8_linear_longest_sums(M, N):
    # K = 131071 of +-128 and 127: the largest 32-bit sums, split over CTAs for few tiles.
    K = 131071
    x = torch.full((M, -(-K // 16) * 16), -128, dtype=torch.int8, device="cuda")[:, :K]
    w = torch.full((N, -(-K // 16) * 16), -128, dtype=torch.int8, device="cuda")[:, :K]
    w[1], w[2, ::2] = 127, 127
    one = torch.ones
    y = tw.int8_linear(x, one(M, device="cuda"), w, one(N, device="cuda"), out_dtype=F32)
    exact = x[:1].double() @ w.double().t()
    assert float(exact[0, 0]) == 131071 * 16384
    assert torch.equal(y, exact.float().expand(M, N))


def test_int8_linear_writes_strided_rows_only():
    x, xs = _operand(70, 100, 1)
    w, ws = _operand(130, 100, 2)
    ref = tw.int8_linear(x, xs, w, ws, out_dtype=F32)
    for gap in (1, 6):
        buf = torch.full((72, 130 + gap), 7.0, device="cuda")
        tw.int8_linear(x, xs, w, ws, out=buf[1:71, :130])
        assert torch.equal(buf[1:71, :130], ref)
        buf[1:71, :130] = 7.0
        assert bool((buf == 7.0).all()), "written outside the output's rows"


@pytest.mark.parametrize("M", [5, 200, 700])
def test_rows_without_a_scale_stay_by_themselves(M):
    x, xs = _operand(M, 256, 1)
    w, ws = _operand(300, 256, 2)
    wu, us = _operand(300, 256, 3)
    good = tw.int8_linear(x, xs, w, ws)
    good_h = tw.int8_gated(x, xs, w, ws, wu, us)
    xs[3], ws[17] = float("nan"), float("nan")
    xs[1] = 0
    y, h = tw.int8_linear(x, xs, w, ws), tw.int8_gated(x, xs, w, ws, wu, us)
    keep = torch.ones((M, 300), dtype=torch.bool, device="cuda")
    keep[3], keep[:, 17], keep[1] = False, False, False
    assert torch.equal(y[keep], good[keep]) and torch.equal(h[keep], good_h[keep])
    assert bool(y[3].isnan().all()) and bool(y[:, 17].isnan().all()) and bool(h[3].isnan().all())
    assert bool(h[:, 17].isnan().all())
    row = torch.ones(300, dtype=torch.bool, device="cuda")
    row[17] = False
    assert not y[1][row].any() and not h[1][row].any()


def test_int8_products_on_another_stream_and_in_graphs():
    x, xs = _operand(40, 512, 1)
    w, ws = _operand(700, 512, 2)
    wu, us = _operand(700, 512, 3)

    def step(stream=None):
        return (tw.int8_linear(x, xs, w, ws, stream=stream), tw.int8_gated(x, xs, w, ws, wu, us, stream=stream))
    ref = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    here = step()          # two calls at once
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(ref, got)) and all(torch.equal(a, c) for a, c in zip(ref, here))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    xs.mul_(2)
    ref = step()
    for k in (0, 1, 0):
        graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(ref, outs[k]))


def test_offsets_past_32_bits():
    # Rows 2 GiB apart: the third one's offset passes 2^32 bytes, the output's 2^32 elements' bytes too.
    far = (1 << 31) + 32
    xb = torch.zeros(2 * far + 96, dtype=torch.int8, device="cuda")
    x = torch.as_strided(xb, (3, 96), (far, 1))
    q, xs = _operand(3, 96, 1)
    x.copy_(q)
    w, ws = _operand(40, 96, 2)
    yb = torch.zeros(2 * far + 40, dtype=BF16, device="cuda")
    y = torch.as_strided(yb, (3, 40), (far, 1))
    tw.int8_linear(x, xs, w, ws, out=y)
    assert torch.equal(y, tw.int8_linear(q, xs, w, ws))
    wide = torch.as_strided(xb, (3, 96), (far, 1))
    assert torch.equal(tw.int8_linear(q, xs, wide, xs), tw.int8_linear(q, xs, q, xs))


# ---------------------------------------------------------------- as used together
def _ffn_inputs(M, K, N, seed):
    w = wl.Workload(f"int8_{M}_{K}_{N}", M, K, N, 128, 16, seed, p_mean=0.05)
    d = wl.generate(w)
    return w, d, {k: P.to_dev(d[k]) for k in ("x", "wg_t", "wu_t", "wd")}


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("with_norm", [False, True])
def test_dense_ffn_int8(M, with_norm):
    K, N = 256, 1024
    _, _, dev = _ffn_inputs(M, K, N, 3)
    x = dev["x"].float() * 2 + 0.1
    norm = (1 + 0.1 * torch.randn(K, device="cuda"), 0.1 * torch.randn(K, device="cuda"), 1e-5) if with_norm else None
    W = tw.int8_ffn_weights(dev["wg_t"], dev["wu_t"], dev["wd"])
    y = tw.dense_ffn_int8(x, W, norm=norm)
    assert y.dtype == F32 and y.shape == (M, K)
    # The formula in 64 bits from the same int8 rows; h is rounded to bf16
    # (2^-8) and then to a 127th of its row's largest value (half a step each).
    q, s = tw.quantize_rows(x) if norm is None else tw.layer_norm_int8(x, *norm)
    h = _product64(q, s, W.wg, W.wg_scale).clamp_min(0) * _product64(q, s, W.wu, W.wu_scale)
    wd = W.wd_t.double() * W.wd_scale.double()[:, None]
    off = (2.0 ** -8 + 8 * U) * h.abs() + h.abs().amax(1, keepdim=True) / 127 * 0.51
    ref = h @ wd.t()
    _check(y, ref, off @ wd.abs().t() + 5 * U * (h.abs() @ wd.abs().t()))


def test_norm_sparse_ffn_and_both_backward_passes():
    # The pre-norm block as training runs it: norm -> sparse FFN -> backward -> norm backward.
    M, K, N = 300, 192, 512
    w, d, dev = _ffn_inputs(M, K, N, 5)
    g = torch.Generator(device="cuda").manual_seed(1)
    stream = torch.randn((M, K), generator=g, device="cuda") * 3 + 0.5      # the fp32 residual stream
    nw, nb = 1 + 0.2 * torch.randn(K, generator=g, device="cuda"), 0.2 * torch.randn(K, generator=g, device="cuda")
    nw[K - 1], nb[K - 1] = 0, 1                                              # the gate's bias column
    xn, mean, rstd = tw.layer_norm(stream, nw, nb, 1e-5, out_dtype=BF16, stats=True)
    y, t = tw.sparse_ffn(xn, dev["wg_t"], dev["wu_t"], dev["wd"], w.T, w.C)
    y2, _ = tw.sparse_ffn(stream, dev["wg_t"], dev["wu_t"], dev["wd"], w.T, w.C, norm=(nw, nb, 1e-5))
    # The same pass twice: split rows are added in another order (fp32 atomics).
    torch.testing.assert_close(y, y2, rtol=1e-4, atol=1e-5 * float(y.abs().max()))
    dy = torch.randn((M, K), generator=g, device="cuda")
    dxn, dwg, dwu, dwd = tw.ffn_bwd(xn, dev["wg_t"], dev["wu_t"], dev["wd"], t, dy)
    dx, dnw, dnb = tw.layer_norm_bwd(dxn, stream, mean, rstd, nw)
    mask = _active_mask(t.to_host(), N, w.T, w.C)
    bits = xn.view(torch.int16).cpu().numpy().view(np.uint16)
    ref = ob.ffn_backward(bits, d["wg_t"], d["wu_t"], d["wd"], dy.double().cpu().numpy(), active=mask)
    up = torch.from_numpy(ref["dx"]).cuda()
    hat = (stream.double() - mean.double()[:, None]) * rstd.double()[:, None]
    gr = up * nw.double()
    rx = rstd.double()[:, None] * (gr - gr.mean(1, keepdim=True) - hat * (gr * hat).mean(1, keepdim=True))
    for got, want in ((dx, rx), (dnw, (up * hat).sum(0)), (dnb, up.sum(0))):
        # the rule of the FFN's own gradients, whose error the norm passes on
        assert float((got.double() - want).abs().max()) <= 2e-2 * float(want.pow(2).mean().sqrt())


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("h_dtype", [F32, BF16, F16])
def test_dense_ffn_int8_hidden_rows_of_any_type(M, h_dtype):
    K, N = 256, 1024
    _, _, dev = _ffn_inputs(M, K, N, 3)
    W = tw.int8_ffn_weights(dev["wg_t"], dev["wu_t"], dev["wd"])
    y = tw.dense_ffn_int8(dev["x"], W, h_dtype=h_dtype)
    # As test_dense_ffn_int8, with the half step of h's type.
    q, s = tw.quantize_rows(dev["x"])
    h = _product64(q, s, W.wg, W.wg_scale).clamp_min(0) * _product64(q, s, W.wu, W.wu_scale)
    wd = W.wd_t.double() * W.wd_scale.double()[:, None]
    off = _half_step(h_dtype, h) + 8 * U * h.abs() + h.abs().amax(1, keepdim=True) / 127 * 0.51
    _check(y, h @ wd.t(), off @ wd.abs().t() + 5 * U * (h.abs() @ wd.abs().t()))
    # The int8 rows themselves are those of the fp32 (or rounded) h.
    hh = tw.int8_gated(q, s, W.wg, W.wg_scale, W.wu, W.wu_scale, out_dtype=h_dtype)
    q2, s2 = tw.quantize_rows(hh)
    assert torch.equal(y, tw.int8_linear(q2, s2, W.wd_t, W.wd_scale, out_dtype=F32))
