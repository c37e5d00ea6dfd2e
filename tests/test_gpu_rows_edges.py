"""Rows at the edges of the row kernels' arithmetic and launches: lanes behind a
row, means far above the spread, calls from two host threads, many rows.

u = 2^-24 is fp32's half step; a row sum of terms t is within 64 u sum|t| (see
test_gpu_rows.py, whose helpers and bounds these tests share)."""
import threading

import pytest
import torch

from activation_sparse_gated_tma_b200 import twell as tw
from tests.test_gpu_rows import BF16, EPS, F16, F32, U, _affine, _bwd, _check_norm, _half_step, _norm64, _quant64, _rows

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- lanes behind a row
@pytest.mark.parametrize("D", [64, 63, 33, 96, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_norm_int8_of_large_constant_rows(D, dtype):
    # (0 - mean) rstd passes the fp32 range, the rows' own deviations are 0: y is the bias.
    x = _rows(5, D, dtype)
    x[1], x[3] = 2.0 ** 120, -2.0 ** 121
    w, b = _affine(D, F32)
    y = tw.layer_norm(x, w, b, EPS, out_dtype=F32)
    assert torch.equal(y[1], b) and torch.equal(y[3], b)
    q, scale = tw.layer_norm_int8(x, w, b, EPS)
    ref, s = _quant64(y)
    for r in (1, 3):
        assert float(scale[r]) == float(s[r]) and torch.equal(q[r].double(), ref[r])
    assert bool(scale.isfinite().all())


# ---------------------------------------------------------------- means far above the spread
@pytest.mark.parametrize("D", [1000, 4093, 2047, 1535, 4096])
@pytest.mark.parametrize("dtype,value", [(BF16, 6016.0), (BF16, 8064.0), (F16, 6016.0), (F32, 1234.567), (F32, -3e7)])
def test_layer_norm_of_constant_rows_is_the_bias(D, dtype, value):
    x = _rows(7, D, dtype)
    x[2] = value
    w, b = _affine(D, F32)
    y, mean, _ = tw.layer_norm(x, w, b, EPS, out_dtype=F32, stats=True)
    assert torch.equal(y[2], b) and float(mean[2]) == float(x[2, 0])
    q, scale = tw.layer_norm_int8(x, w, b, EPS)
    ref, s = _quant64(b[None])
    assert torch.equal(q[2].double(), ref[0]) and float(scale[2]) == float(s[0])


@pytest.mark.parametrize("M,D", [(5, 2560), (300, 1000), (3, 2047), (4, 8192), (9, 16383), (700, 300)])
@pytest.mark.parametrize("level,spread", [(1000.0, 0.01), (-3e5, 2.0), (20.0, 1.0)])
def test_layer_norm_of_rows_far_from_zero(M, D, level, spread):
    # The deviations that count are those from the row's true mean.  A first mean is within 64 u |mean| of it, so the
    # deviations from that one are below |x - mean| + 64 u |mean|; their sum, and with it the correction, is within
    # 64 u of their magnitudes' sum, and each deviation adds its own rounding.  Rows whose mean is up to four times
    # the spread (4.1 with what both are off by) need no correction: there the first mean's 64 u |mean| counts.
    x = (_rows(M, D, F32) * spread + level).contiguous()
    w, b = _affine(D, F32)
    y, mean, rstd = tw.layer_norm(x, w, b, 0.0, stats=True)
    ref, m64, r64, hat = _norm64(x, w, b, 0.0)
    off = (x.double() - m64).abs().mean(1, keepdim=True) + 64 * U * m64.abs()
    off += torch.where(m64.abs() * r64 <= 4.1, m64.abs(), 0.0)
    wa, ba = w.double().abs(), b.double().abs()
    tol = _half_step(F32, ref) + 64 * U * (wa * (hat.abs() + r64 * off) + ba) * (1 + 64 * U)
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    assert bool(((mean.double()[:, None] - m64).abs() <= U * m64.abs() + 64 * U * off * (1 + U)).all())
    assert bool(((rstd.double()[:, None] - r64).abs() <= 64 * U * r64 * (1 + (64 * U * off * r64) ** 2 / U)).all())


@pytest.mark.parametrize("D", [2, 64, 1000, 2560, 4093, 8192, 16383, 16384])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_norm_of_rows_whose_sum_passes_the_range(D, dtype):
    x = _rows(6, D, dtype)
    x[1], x[3], x[4] = 3e38, -torch.finfo(dtype).max, torch.finfo(dtype).max
    w, b = _affine(D, F32)
    y, mean, rstd = tw.layer_norm(x, w, b, EPS, out_dtype=F32, stats=True)
    q, scale = tw.layer_norm_int8(x, w, b, EPS)
    ref, s = _quant64(b[None])
    for r in (1, 3, 4):
        assert torch.equal(y[r], b) and float(mean[r]) == float(x[r, 0])
        assert abs(float(rstd[r]) * EPS ** 0.5 - 1) <= 8 * U
        assert torch.equal(q[r].double(), ref[0]) and float(scale[r]) == float(s[0])
    _check_norm(y[::5], mean[::5], rstd[::5], x[::5], w, b)


@pytest.mark.parametrize("D", [64, 63, 33, 1000, 2040, 2047, 4100, 4097])
@pytest.mark.parametrize("M", [7, 1300])
@pytest.mark.parametrize("tx,td", [(F32, F32), (BF16, BF16)])
def test_layer_norm_bwd_of_large_constant_rows(M, D, tx, td):
    # mean rstd passes the fp32 range (2^110 10^6) while x - mean is 0: dx is rstd (g - sum g / D).
    x, dy = _rows(M, D, tx), _rows(M, D, td, seed=5)
    w = _affine(D, F32)[0]
    x[1::3] = 2.0 ** 110
    mean, rstd = x.double().mean(1).float(), torch.ones(M, device="cuda")
    mean[1::3], rstd[1::3] = 2.0 ** 110, 1e6
    dx, dw, db = tw.layer_norm_bwd(dy, x, mean, rstd, w)
    d, m, r = dy.double(), mean.double()[:, None], rstd.double()[:, None]
    hat = (x.double() - m) * r
    gr = d * w.double()
    ref = r * (gr - gr.mean(1, keepdim=True) - hat * (gr * hat).mean(1, keepdim=True))
    tol = _half_step(tx, ref) + 64 * U * r * (
        gr.abs() + gr.abs().mean(1, keepdim=True) + hat.abs() * (gr * hat).abs().mean(1, keepdim=True)) * (
            1 + torch.finfo(tx).eps)
    assert bool(((dx.double() - ref).abs() <= tol).all())
    for got, terms in ((dw, d * hat), (db, d)):
        assert bool(((got.double() - terms.sum(0)).abs() <= 128 * U * terms.abs().sum(0)).all())


def test_layer_norm_bwd_of_rows_without_rstd():
    # Squared deviations past the fp32 range leave rstd 0, and with it dx.
    x, dy = _rows(9, 1000, F32), _rows(9, 1000, F32, seed=5)
    x[4] *= 1e37
    _, mean, rstd = tw.layer_norm(x, stats=True)
    assert float(rstd[4]) == 0
    dx, dw, db = tw.layer_norm_bwd(dy, x, mean, rstd)
    assert not dx[4].any() and bool(dx.isfinite().all())
    keep = torch.arange(9, device="cuda") != 4
    _bwd(x[keep], dy[keep], None)
    assert bool(dw.isfinite().all()) and bool(db.isfinite().all())


# ---------------------------------------------------------------- host threads
def _in_threads(calls, times):
    """Each (library function, arguments before the stream) in two threads of its
    own, on streams of their own: the calls overlap in the library."""
    statuses = []

    def loop(function, args):
        s = torch.cuda.Stream()
        args = (*args, s.cuda_stream)
        bad = [st for st in (function(*args) for _ in range(times)) if st != tw.OK]
        s.synchronize()
        statuses.append((len(bad), (tw.lib().twell_last_error() or b"").decode() if bad else ""))
    threads = [threading.Thread(target=loop, args=c) for c in calls for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(statuses) == len(threads) and not any(n for n, _ in statuses), statuses


def test_threads_that_norm_rows_of_different_lengths():
    # 16384 and 8192 columns are eight chunks a thread in one kernel, with 128 and 64 KB of shared memory.
    keep = []

    def call(D):
        x = _rows(2, D, F32)
        keep.append((x, torch.empty_like(x)))
        return tw.lib().twell_layer_norm_fwd, (x.data_ptr(), 0, D, None, None, 0, 2, D, 1e-5, keep[-1][1].data_ptr(), 0,
                                               D, None, None)
    # (Two rows of 8192 columns would take more warps and fewer chunks: 300 of them do not.)
    a = call(16384)
    x, y = _rows(300, 8192, F32), torch.empty((300, 8192), device="cuda")
    b = (tw.lib().twell_layer_norm_fwd, (x.data_ptr(), 0, 8192, None, None, 0, 300, 8192, 1e-5, y.data_ptr(), 0, 8192,
                                         None, None))
    torch.cuda.synchronize()
    _in_threads([a, b], 10000)
    torch.cuda.synchronize()
    _check_norm(y, None, None, x, None, None)
    _check_norm(keep[0][1], None, None, keep[0][0], None, None)


@pytest.mark.parametrize("lengths", [(2048, 2816), (4096, 3200)])
def test_threads_that_differentiate_rows_of_different_lengths(lengths):
    # One kernel, 48 and 44 KB of sums (64 and 50).
    keep = []

    def call(D):
        M = 900
        x = _rows(M, D, F32)
        _, mean, rstd = tw.layer_norm(x, stats=True)
        dx = torch.empty_like(x)
        keep.append((x, mean, rstd, dx))
        size = tw.lib().twell_layer_norm_bwd_scratch_bytes(M, D)
        scratch = torch.empty(size, dtype=torch.uint8, device="cuda")
        dw = torch.empty(D, device="cuda")
        keep.append((scratch, dw))
        return tw.lib().twell_layer_norm_bwd, (x.data_ptr(), 0, D, x.data_ptr(), 0, D, mean.data_ptr(), rstd.data_ptr(),
                                               None, 0, M, D, dx.data_ptr(), D, dw.data_ptr(), None, scratch.data_ptr(), size)
    calls = [call(D) for D in lengths]
    torch.cuda.synchronize()
    _in_threads(calls, 5000)
    for x, mean, rstd, dx in keep[::2]:   # (dw is left out: two threads use one scratch)
        assert torch.equal(dx, tw.layer_norm_bwd(x, x, mean, rstd, param_grads=False)[0])


# ---------------------------------------------------------------- more rows than groups
@pytest.mark.parametrize("M,D,gap", [(5000, 256, 0), (5000, 2560, 0), (2500, 8192, 0), (1300, 16384, 0),      # aligned
                                     (5003, 255, 0), (5001, 2047, 0), (5000, 2559, 1), (2500, 8191, 0), (1300, 16383, 0)])
@pytest.mark.parametrize("tx,ty", [(F32, BF16), (BF16, BF16), (F16, F32)])
def test_layer_norm_of_many_rows(M, D, gap, tx, ty):
    # Every group of warps takes several rows in turn.
    x = _rows(M, D, tx, gap)
    w, b = _affine(D, F32)
    y, mean, rstd = tw.layer_norm(x, w, b, EPS, out_dtype=ty, stats=True)
    _check_norm(y, mean, rstd, x, w, b)
    # (By 64-bit quotients of fp32 results: those have the kernel's own values, which the tests above check.)
    y = tw.layer_norm(x, w, b, EPS, out_dtype=F32)
    q, scale = tw.layer_norm_int8(x, w, b, EPS)
    ref, s = _quant64(y)
    # The same fp32 operations; were one fused otherwise, y would be off by 8 u of its terms, and q by one step at ties.
    hat = (x.double() - mean.double()[:, None]).abs() * rstd.double()[:, None]
    e = 8 * U * (w.double().abs() * hat + b.double().abs())
    top = e.amax(1)
    assert bool(((scale.double() - s.double()).abs() <= (top + 2 * U * s.double() * 127) / 127).all())
    at = y.double() / s.double()[:, None]
    assert bool(((q.double() - at).abs() <= 0.5 + (e + top[:, None]) / s.double()[:, None] + 1e-4).all())


@pytest.mark.parametrize("M,K,gap", [(5000, 256, 0), (5001, 2047, 0), (4000, 5632, 0), (4000, 5631, 1), (1300, 20480, 0),
                                     (1300, 20479, 0), (700, 20481, 0), (650, 40001, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantize_rows_of_many_rows(M, K, gap, dtype):
    # (Rows of more than 20480 elements are read twice, a block each: 592 blocks.)
    x = _rows(M, K, dtype, gap)
    q, scale = tw.quantize_rows(x)
    for i in range(0, M, 1000):
        part = slice(i, i + 1000)
        ref, s = _quant64(x[part])
        assert torch.equal(q[part].double(), ref) and torch.equal(scale[part], s)
    for t in (F32, BF16):
        assert torch.equal(tw.dequantize_rows(q, scale, t), (q.float() * scale[:, None]).to(t))


@pytest.mark.parametrize("M,D", [(2500, 8192), (2500, 8191), (5001, 2047), (1300, 16384)])
def test_layer_norm_of_many_rows_some_far_from_zero(M, D):
    # Groups take rows with and without the correction's two sums in turn.
    x = _rows(M, D, F32)
    g = torch.Generator(device="cuda").manual_seed(M)
    far = torch.rand(M, generator=g, device="cuda") < 0.4
    level = torch.where(torch.rand(M, generator=g, device="cuda") < 0.5, 6016.0, -1234.567)
    x[far] = level[far, None]
    w, b = _affine(D, F32)
    y, mean, rstd = tw.layer_norm(x, w, b, EPS, stats=True)
    assert torch.equal(y[far], b.expand(int(far.sum()), D)) and torch.equal(mean[far], x[far, 0])
    _check_norm(y[~far], mean[~far], rstd[~far], x[~far], w, b)
    q, scale = tw.layer_norm_int8(x, w, b, EPS)
    ref, s = _quant64(b[None])
    assert torch.equal(q[far].double(), ref.expand(int(far.sum()), D)) and bool((scale[far] == s).all())
