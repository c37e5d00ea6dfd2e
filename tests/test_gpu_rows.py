"""Layer norm, its backward pass and row quantisation on the GPU against plain
64-bit formulas.

Tolerances.  u = 2^-24 is fp32's half step.  A sum over a row is taken in at
most 32 additions per thread and 10 levels of a tree, so a row sum of terms t is
within 42 u sum|t|; 64 u leaves room for the few roundings per term.  An output
of type t adds its own half step, finfo(t).eps / 2 relative to the value."""
import numpy as np
import pytest
import torch

from activation_sparse_gated_tma_b200 import twell as tw

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5


def _half_step(dtype, v):
    # relative half step, and the half step of the subnormals (fp16 rows reach them)
    return torch.finfo(dtype).eps / 2 * v.abs() + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def _rows(M, D, dtype, gap=0, offset=0, seed=0):
    """[M][D] whose rows are D + gap elements apart, `offset` elements into the storage."""
    g = torch.Generator(device="cuda").manual_seed(seed * 1000 + M * 7 + D)
    x = torch.randn((M, D), generator=g, device="cuda", dtype=torch.float64)
    x *= torch.exp(0.5 * torch.randn((M, 1), generator=g, device="cuda", dtype=torch.float64))
    x += 0.2
    buf = torch.full((offset + M * (D + gap),), 7.0, device="cuda", dtype=dtype)
    v = buf[offset:].view(M, D + gap)[:, :D]
    v.copy_(x)
    return v


def _affine(D, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype),
            (0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype))


def _norm64(x, w, b, eps=EPS):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    hat = (x - mean) * rstd
    w = 1.0 if w is None else w.double()
    b = 0.0 if b is None else b.double()
    return hat * w + b, mean, rstd, hat


def _check_norm(y, mean, rstd, x, w, b, eps=EPS):
    ref, m64, r64, hat = _norm64(x, w, b, eps)
    xd = x.double()
    spread = xd.abs().mean(1, keepdim=True)
    wa = 1.0 if w is None else w.double().abs()
    ba = 0.0 if b is None else b.double().abs()
    tol = _half_step(y.dtype, ref) + 64 * U * (wa * (hat.abs() + r64 * spread) + ba) * (1 + torch.finfo(y.dtype).eps)
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    if mean is not None:
        assert bool(((mean.double()[:, None] - m64).abs() <= 64 * U * spread).all())
        # rstd: half of the variance's relative error, the mean's error squared, two roundings
        assert bool(((rstd.double()[:, None] - r64).abs() <= 64 * U * r64 * (1 + (64 * U * spread * r64) ** 2 / U)).all())


SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (9, 63), (1, 64), (17, 255), (4, 256), (3, 257), (33, 1000), (7, 2047), (300, 2048),
          (2, 4096), (3, 4097), (2, 8192), (2, 8200), (3, 16384), (2, 16383), (700, 1536)]
TYPES = [(F32, F32), (F32, BF16), (F32, F16), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)]


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("tx,ty", [(F32, BF16), (BF16, BF16), (F16, F32)])
def test_layer_norm_shapes(M, D, tx, ty):
    x = _rows(M, D, tx)
    w, b = _affine(D, F32)
    y, mean, rstd = tw.layer_norm(x, w, b, EPS, out_dtype=ty, stats=True)
    assert tw.last_launch_count() == 1
    _check_norm(y, mean, rstd, x, w, b)


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("gap,offset", [(0, 0), (1, 0), (8, 0), (8, 3)])
def test_layer_norm_types_strides_and_alignment(tx, ty, gap, offset):
    M, D = 13, 520
    x = _rows(M, D, tx, gap, offset)
    w, b = _affine(D, BF16 if ty is BF16 else F32)
    out = torch.full((M, D + gap), 7.0, device="cuda", dtype=ty)
    assert tw.layer_norm(x, w, b, EPS, out=out[:, :D]).data_ptr() == out.data_ptr()
    _check_norm(out[:, :D], None, None, x, w, b)
    assert bool((out[:, D:] == 7.0).all()), "columns behind the rows were written"


@pytest.mark.parametrize("w_on,b_on", [(False, False), (True, False), (False, True)])
def test_layer_norm_without_weight_or_bias(w_on, b_on):
    x = _rows(6, 384, BF16)
    w, b = _affine(384, F16)
    w, b = w if w_on else None, b if b_on else None
    _check_norm(tw.layer_norm(x, w, b, out_dtype=F32), None, None, x, w, b)


def test_layer_norm_gate_bias_column_both_ways():
    # D = K - 1 with the ones column left alone, and D = K with weight 0, bias 1 there.
    M, K = 37, 256
    buf = torch.ones((M, K), device="cuda", dtype=BF16)
    x = _rows(M, K - 1, F32)
    w, b = _affine(K - 1, F32)
    tw.layer_norm(x, w, b, out=buf[:, :K - 1])
    _check_norm(buf[:, :K - 1], None, None, x, w, b)
    assert bool((buf[:, K - 1] == 1).all())
    x = _rows(M, K, F32)
    w, b = _affine(K, F32)
    w[K - 1], b[K - 1] = 0, 1
    assert bool((tw.layer_norm(x, w, b, out_dtype=BF16)[:, K - 1] == 1).all())


def test_layer_norm_mean_far_above_the_spread():
    # Sums of squares would cancel here: mean 1000, spread 1 (fp32 keeps 2^-14 of a step of the spread).
    x = (_rows(5, 2048, F32) + 1000).contiguous()
    y, mean, rstd = tw.layer_norm(x, eps=0.0, stats=True)
    _check_norm(y, mean, rstd, x, None, None, 0.0)


def test_layer_norm_constant_rows_and_non_finite_rows():
    x = _rows(6, 512, F32)
    x[1] = 0.0
    x[2] = 3.0
    x[3, 100] = float("nan")
    x[4, 7] = float("inf")
    w, b = _affine(512, F32)
    y = tw.layer_norm(x, w, b)
    assert torch.equal(y[1], b) and torch.equal(y[2], b)
    assert bool(y[3:5].isnan().all())
    assert bool(y[[0, 1, 2, 5]].isfinite().all())


@pytest.mark.parametrize("M,D,tx,td", [
    (1, 1, F32, F32), (3, 7, F32, F32), (1, 64, BF16, BF16), (5, 8, F16, F16), (33, 255, BF16, F32), (300, 256, F32, BF16),
    (64, 1000, F16, F32), (4099, 130, F32, F32), (700, 2047, F32, F16), (2500, 2048, BF16, F32), (20, 4096, F32, F32),
    (9, 4100, BF16, BF16), (5, 8192, F32, F32), (3, 16384, F32, F32), (4, 16383, F16, F16)])
def test_layer_norm_bwd(M, D, tx, td):
    _bwd(_rows(M, D, tx), _rows(M, D, td, seed=5), _affine(D, F32)[0])


@pytest.mark.parametrize("M,D,tx,td", [(4099, 2047, F16, F16), (1030, 1535, BF16, F32), (1, 9, F32, F32), (7, 2049, F32, BF16),
                                       (600, 4089, BF16, BF16), (600, 4090, F32, F32), (640, 8188, F16, F32), (601, 16377, F32, F32),
                                       (1300, 12, BF16, BF16), (2000, 514, F32, F32), (11, 16378, BF16, F32), (900, 1, F32, F32),
                                       (777, 7, BF16, F32), (700, 4100, F16, F16)])
def test_layer_norm_bwd_rows_that_start_within_a_chunk(M, D, tx, td):
    _bwd(_rows(M, D, tx), _rows(M, D, td, seed=5), _affine(D, F16)[0])


@pytest.mark.parametrize("warps", range(1, 17))
def test_layer_norm_bwd_every_number_of_warps_a_row(warps):
    # Rows enough to fill every SM, aligned, shifted and by elements: every shape of block.
    for D, gap in ((256 * warps, 0), (256 * warps - 9, 0), (256 * warps - 1, 1)):
        _bwd(_rows(3000, D, BF16, gap), _rows(3000, D, F32, seed=5), None)


def test_layer_norm_bwd_equal_shifts_and_untouched_padding():
    # x, dy and dx start three elements behind a chunk's boundary, rows 2 elements apart.
    M, D, ld = 661, 515, 517
    x, dy = _rows(M, D, BF16, 2, 3), _rows(M, D, F32, 2, 3, seed=5)
    w, b = _affine(D, F32)
    _, mean, rstd = tw.layer_norm(x, w, b, stats=True)
    ref = tw.layer_norm_bwd(dy, x, mean, rstd, w)
    buf = torch.full((3 + M * ld,), 5.0, device="cuda", dtype=BF16)
    dw, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    size = tw.lib().twell_layer_norm_bwd_scratch_bytes(M, D)
    scratch = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert tw.lib().twell_layer_norm_bwd(
        dy.data_ptr(), 0, ld, x.data_ptr(), 1, ld, mean.data_ptr(), rstd.data_ptr(), w.data_ptr(), 0, M, D,
        buf.data_ptr() + 6, ld, dw.data_ptr(), db.data_ptr(), scratch.data_ptr(), size,
        torch.cuda.current_stream().cuda_stream) == tw.OK
    dx = buf[3:].view(M, ld)
    assert bool((buf[:3] == 5).all()) and bool((dx[:, D:] == 5).all())
    # Both are within the bounds of _bwd of the formula; sums in other orders differ by no more than twice those.
    for got, want in ((dx[:, :D], ref[0]), (dw, ref[1]), (db, ref[2])):
        assert torch.allclose(got.float(), want.float(), rtol=2 ** -7, atol=1e-4)


@pytest.mark.parametrize("gap,offset", [(1, 0), (8, 0), (8, 3)])
def test_layer_norm_bwd_strides(gap, offset):
    _bwd(_rows(50, 520, BF16, gap, offset), _rows(50, 520, F32, gap, offset, seed=5), _affine(520, BF16)[0])


def test_layer_norm_bwd_without_weight():
    _bwd(_rows(50, 520, BF16), _rows(50, 520, F32, seed=5), None)


def _bwd(x, dy, w):
    M, D = x.shape
    y, mean, rstd = tw.layer_norm(x, w, stats=True)
    dx, dw, db = tw.layer_norm_bwd(dy, x, mean, rstd, w)
    assert tw.last_launch_count() == 2
    assert dx.dtype == x.dtype and dw.dtype == db.dtype == F32
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    d = dy.double()
    hat = (x.double() - mean) * rstd
    gr = d if w is None else d * w.double()
    ref = rstd * (gr - gr.mean(1, keepdim=True) - hat * (gr * hat).mean(1, keepdim=True))
    tol = _half_step(x.dtype, ref) + 64 * U * rstd * (
        gr.abs() + gr.abs().mean(1, keepdim=True) + hat.abs() * (gr * hat).abs().mean(1, keepdim=True)) * (
            1 + torch.finfo(x.dtype).eps)
    err = (dx.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    # Column sums: rows of one partial row in a chain (M / 148 at most 34 here),
    # every 16th partial row in a chain, 16 sums: under 128 additions each.
    for got, terms in ((dw, d * hat), (db, d)):
        err = (got.double() - terms.sum(0)).abs()
        tol = 128 * U * terms.abs().sum(0)
        assert bool((err <= tol).all()), float((err / tol).max())
    again = tw.layer_norm_bwd(dy, x, mean[:, 0].float(), rstd[:, 0].float(), w)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again)), "not the same bits twice"
    only = tw.layer_norm_bwd(dy, x, mean[:, 0].float(), rstd[:, 0].float(), w, param_grads=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None


def test_layer_norm_bwd_against_differences():
    # d/dx, d/dw, d/db of sum(y dy) by central differences of the 64-bit formula
    # (h = 1e-5: their error is near 1e-9; the kernel's is bounded by 64 u of terms of size < 30).
    M, D, h = 3, 7, 1e-5
    x, dy = _rows(M, D, F32), _rows(M, D, F32, seed=5)
    w, b = _affine(D, F32)
    _, mean, rstd = tw.layer_norm(x, w, b, stats=True)
    got = tw.layer_norm_bwd(dy, x, mean, rstd, w)

    def loss(x, w, b):
        return float((_norm64(x, w, b)[0] * dy.double()).sum())
    args = [x.double().clone(), w.double().clone(), b.double().clone()]
    for k, g in enumerate(got):
        flat = args[k].view(-1)
        for i in range(flat.numel()):
            at = float(flat[i])
            flat[i] = at + h
            up = loss(*args)
            flat[i] = at - h
            down = loss(*args)
            flat[i] = at
            assert abs((up - down) / (2 * h) - float(g.view(-1)[i])) < 2e-4, (k, i)


def test_layer_norm_bwd_no_rows_and_scratch():
    e = torch.empty((0, 96), device="cuda")
    v = torch.empty(0, device="cuda")
    dx, dw, db = tw.layer_norm_bwd(e, e, v, v)
    assert dx.shape == (0, 96) and not dw.any() and not db.any()
    assert tw.layer_norm(e).shape == (0, 96) and tw.quantize_rows(e)[0].shape == (0, 96)
    x = _rows(40, 96, F32)
    _, mean, rstd = tw.layer_norm(x, stats=True)
    need = tw.lib().twell_layer_norm_bwd_scratch_bytes(40, 96)
    with pytest.raises(tw.TwellError):
        tw.layer_norm_bwd(x, x, mean, rstd, scratch=torch.empty(need - 4, dtype=torch.uint8, device="cuda"))
    a = tw.layer_norm_bwd(x, x, mean, rstd, scratch=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(p, q) for p, q in zip(a, tw.layer_norm_bwd(x, x, mean, rstd)))


# ---------------------------------------------------------------- int8 rows
def _quant64(x):
    """The definition, in 64 bits (torch.round: ties to even)."""
    amax = x.abs().amax(1, keepdim=True)
    q = torch.where(amax > 0, x.double() * 127 / torch.where(amax > 0, amax, 1).double(), 0.0).round()
    # The 64-bit quotient rounded to fp32 is the correctly rounded fp32 quotient
    # (53 >= 2 * 24 + 2 bits); fp32 tensor / number would multiply by 1/127 instead.
    return q, (amax.double() / 127).float()[:, 0]


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 16), (4, 100), (33, 2048), (2, 4097), (3, 8192), (2, 12345), (3, 16384),
                                 (2, 16392), (2, 40001), (1, 131071)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantize_rows_is_exact(M, K, dtype):
    x = _rows(M, K, dtype)
    q, scale = tw.quantize_rows(x)
    ref, s = _quant64(x)
    assert q.dtype == torch.int8 and q.stride(0) % 16 == 0
    assert torch.equal(q.double(), ref) and torch.equal(scale, s)
    for t in (F32, BF16, F16):
        assert torch.equal(tw.dequantize_rows(q, scale, t), (q.float() * scale[:, None]).to(t))


@pytest.mark.parametrize("gap,offset", [(1, 0), (8, 0), (8, 3)])
def test_quantize_rows_strides(gap, offset):
    x = _rows(9, 520, F16, gap, offset)
    q, scale = tw.quantize_rows(x)
    ref, s = _quant64(x)
    assert torch.equal(q.double(), ref) and torch.equal(scale, s)
    odd = torch.zeros((9, 523), dtype=torch.int8, device="cuda")
    odd[:, 1:521] = q
    assert torch.equal(tw.dequantize_rows(odd[:, 1:521], scale, F32), tw.dequantize_rows(q, scale, F32))


def test_quantize_rows_ties_zeros_and_extremes():
    x = torch.zeros((9, 40), device="cuda")
    x[0, :4] = torch.tensor([3.0, 1.5, -1.5, 0.75])               # 63.5 and -63.5: ties, to 64
    x[1, :4] = torch.tensor([254.0, 1.0, 3.0, -5.0])              # 0.5, 1.5, -2.5: to 0, 2, -2
    # row 2: zeros
    x[3, :3] = torch.tensor([1e-45, 0.0, -1e-45])                 # subnormals: 127 / amax overflows
    x[4, :3] = torch.tensor([3e38, -1.5e38, 1e38])
    x[5, 3] = float("nan")
    x[6, 5] = float("-inf")
    x[7, :3] = torch.tensor([-2.0, 1.0, 2e-39])
    x[8, :3] = torch.tensor([2e-38, 1e-38, -7e-39])
    q, scale = tw.quantize_rows(x)
    ref, s = _quant64(x)
    good = [0, 1, 2, 3, 4, 7, 8]
    assert torch.equal(q[good].double(), ref[good]) and torch.equal(scale[good], s[good])
    assert q[0, :4].tolist() == [127, 64, -64, 32] and q[1, :4].tolist() == [127, 0, 2, -2]
    assert float(scale[2]) == 0 and not q[2].any()
    assert bool(scale[5:7].isnan().all()) and not q[5:7].any()


@pytest.mark.parametrize("dtype,exponents", [(BF16, [0, 1, 3, 27, 28, 127, 227, 254]), (F16, [0, 1, 2, 15, 30])])
def test_quantize_rows_every_16_bit_value(dtype, exponents):
    """Rows of all values from amax down to below amax / 254, both signs, for
    every mantissa of amax: with them every tie and every quotient next to one."""
    ones = 128 if dtype == BF16 else 1024  # mantissas per exponent
    for e in exponents:
        top = (torch.arange(ones, device="cuda") + e * ones)[:, None]
        bits = (top - torch.arange(9 * ones, device="cuda")[None]).clamp_min_(0).to(torch.int16)
        x = torch.cat((bits, bits | -2 ** 15), 1).view(dtype)
        q, scale = tw.quantize_rows(x)
        ref, s = _quant64(x)
        assert torch.equal(q.double(), ref) and torch.equal(scale, s), e


def test_quantize_rows_leaves_the_padding_alone():
    L = tw.lib()
    x = _rows(5, 33, BF16)
    q = torch.full((5, 48), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(5, device="cuda")
    assert L.twell_quantize_rows(x.data_ptr(), 1, 33, 5, 33, q.data_ptr(), 48, s.data_ptr(),
                                 torch.cuda.current_stream().cuda_stream) == tw.OK
    assert torch.equal(q[:, :33].double(), _quant64(x)[0]) and bool((q[:, 33:] == 99).all())


@pytest.mark.parametrize("M,D,dtype,gap", [(1, 1, F32, 0), (5, 8, BF16, 0), (33, 1535, BF16, 1), (300, 2048, F32, 0),
                                           (7, 2047, F16, 0), (2, 8192, F32, 0), (3, 16384, BF16, 0)])
def test_layer_norm_int8(M, D, dtype, gap):
    x = _rows(M, D, dtype, gap)
    w, b = _affine(D, F32)
    q, scale = tw.layer_norm_int8(x, w, b, EPS)
    ref, m64, r64, hat = _norm64(x, w, b)
    # fp32 error of a value before it is quantised, as for layer_norm's output
    e = 64 * U * (w.double().abs() * (hat.abs() + r64 * x.double().abs().mean(1, keepdim=True)) + b.double().abs())
    amax = ref.abs().amax(1, keepdim=True)
    ea = e.amax(1, keepdim=True)
    assert bool(((scale.double()[:, None] - amax / 127).abs() <= ea / 127 + 2 * U * amax / 127).all())
    # q is the nearest integer to 127 y / amax of nearby y and amax: half a step and what those are off by.
    at = ref * 127 / torch.where(amax > 0, amax, 1)
    slack = 0.5 + torch.where(amax > 0, 127 * (e + ea) / torch.where(amax > 0, amax, 1) * (1 + 1e-3), 0.0) + 1e-12
    assert bool(((q.double() - at).abs() <= slack).all())
    assert int(q.abs().max()) == 127 or not bool(amax.any())


def test_offsets_past_32_bits():
    # Rows 2^31 elements apart: the third one's offset passes 2^32 bytes and elements.
    far = (1 << 31) + 16
    buf = torch.zeros(2 * far + 520, dtype=BF16, device="cuda")
    x = torch.as_strided(buf, (3, 520), (far, 1))
    near = _rows(3, 520, BF16)
    x.copy_(near)
    w, b = _affine(520, F32)
    y, mean, rstd = tw.layer_norm(near, w, b, stats=True)
    assert torch.equal(tw.layer_norm(x, w, b), y)
    assert all(torch.equal(p, q) for p, q in zip(tw.layer_norm_int8(x, w, b), tw.layer_norm_int8(near, w, b)))
    assert all(torch.equal(p, q) for p, q in zip(tw.quantize_rows(x), tw.quantize_rows(near)))
    dy = _rows(3, 520, F32, seed=5)
    assert all(torch.equal(p, q) for p, q in zip(tw.layer_norm_bwd(dy, x, mean, rstd, w),
                                                 tw.layer_norm_bwd(dy, near, mean, rstd, w)))
    tw.layer_norm(near, w, b, out=x)
    assert torch.equal(x, y)


# ---------------------------------------------------------------- streams, graphs
def test_rows_on_another_stream_and_in_graphs():
    x = _rows(64, 1000, F32)
    dy = _rows(64, 1000, F32, seed=5)
    w, b = _affine(1000, F32)

    def step(stream=None):
        y, mean, rstd = tw.layer_norm(x, w, b, out_dtype=BF16, stats=True, stream=stream)
        q, s = tw.quantize_rows(y, stream=stream)
        return (y, q, s, tw.dequantize_rows(q, s, stream=stream), *tw.layer_norm_int8(x, w, b, stream=stream),
                *tw.layer_norm_bwd(dy, x, mean, rstd, w, stream=stream))
    ref = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(ref, got))
    # Two captured graphs, replayed in turn with new inputs: no workspace is shared.
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    x.mul_(1.5).add_(0.1)
    dy.mul_(-0.5)
    ref = step()
    for k in (0, 1, 0):
        for t in outs[k]:
            t.zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(ref, outs[k]))
