"""Refusals of the row kernels and int8 products (no GPU needed): every invalid
call is answered before anything touches CUDA."""
import ctypes

import pytest
import torch

from activation_sparse_gated_tma_b200 import twell as tw

P = 1 << 33   # a 16-byte aligned fake device pointer: validation must fail before any use
F32, BF16, F16, I8 = range(4)


def _norm(L, **kw):
    a = dict(x=P, xt=BF16, ldx=64, w=P, b=P, wt=F32, M=4, D=64, eps=1e-5, y=P, yt=BF16, ldy=64, mean=P, rstd=P)
    a.update(kw)
    return L.twell_layer_norm_fwd(a["x"], a["xt"], a["ldx"], a["w"], a["b"], a["wt"], a["M"], a["D"], a["eps"], a["y"],
                                  a["yt"], a["ldy"], a["mean"], a["rstd"], None)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(D=0), dict(D=16385), dict(ldx=63), dict(ldy=63), dict(x=None), dict(y=None), dict(x=P + 1),
    dict(y=P + 1), dict(yt=I8), dict(xt=I8), dict(yt=F16), dict(xt=7), dict(wt=I8), dict(wt=-1), dict(w=P + 2),
    dict(b=P + 2), dict(mean=P + 2), dict(rstd=P + 2), dict(eps=-1.0), dict(eps=float("nan")), dict(ldx=-64)])
def test_layer_norm_refuses(bad):
    L = tw.lib()
    assert _norm(L, **bad) == tw.ERR_INVALID, bad
    assert L.twell_last_error()


def test_layer_norm_int8_refuses():
    L = tw.lib()

    def call(q=P, ldq=64, scale=P, D=64):
        return L.twell_layer_norm_int8(P, BF16, 64, None, None, F32, 4, D, 1e-5, q, ldq, scale, None, None, None)
    for bad in (dict(q=None), dict(ldq=63), dict(scale=None), dict(scale=P + 2), dict(D=0)):
        assert call(**bad) == tw.ERR_INVALID, bad


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(D=0), dict(D=16385), dict(dyt=BF16, xt=F16), dict(dyt=I8), dict(xt=I8), dict(dy=None), dict(x=None),
    dict(dx=None), dict(mean=None), dict(rstd=None), dict(mean=P + 2), dict(wt=9), dict(w=P + 2), dict(lddy=63),
    dict(ldx=63), dict(lddx=63), dict(dw=P + 2), dict(db=P + 2), dict(scratch=None), dict(scratch=P + 8)])
def test_layer_norm_bwd_refuses(bad):
    L = tw.lib()
    a = dict(dy=P, dyt=F32, lddy=64, x=P, xt=F32, ldx=64, mean=P, rstd=P, w=P, wt=F32, M=4, D=64, dx=P, lddx=64, dw=P,
             db=P, scratch=P, bytes=1 << 20)
    a.update(bad)
    st = L.twell_layer_norm_bwd(a["dy"], a["dyt"], a["lddy"], a["x"], a["xt"], a["ldx"], a["mean"], a["rstd"], a["w"],
                                a["wt"], a["M"], a["D"], a["dx"], a["lddx"], a["dw"], a["db"], a["scratch"], a["bytes"],
                                None)
    assert st == tw.ERR_INVALID, bad


@pytest.mark.parametrize("sizes", [(0, 64), (-1, 64), (4, 0), (4, 16385)])
def test_bwd_scratch_is_zero_for_invalid_sizes(sizes):
    assert tw.lib().twell_layer_norm_bwd_scratch_bytes(*sizes) == 0


def test_quantize_and_dequantize_refuse():
    L = tw.lib()

    def quant(x=P, xt=BF16, ldx=64, M=4, K=64, q=P, ldq=64, scale=P):
        return L.twell_quantize_rows(x, xt, ldx, M, K, q, ldq, scale, None)

    def back(q=P, ldq=64, scale=P, M=4, K=64, y=P, yt=BF16, ldy=64):
        return L.twell_dequantize_rows(q, ldq, scale, M, K, y, yt, ldy, None)
    for bad in (dict(M=-1), dict(K=0), dict(K=131072), dict(xt=I8), dict(x=None), dict(x=P + 1), dict(ldx=63),
                dict(q=None), dict(ldq=63), dict(scale=None), dict(scale=P + 1)):
        assert quant(**bad) == tw.ERR_INVALID, bad
    for bad in (dict(M=-1), dict(K=0), dict(K=131072), dict(yt=I8), dict(y=None), dict(y=P + 1), dict(ldy=63),
                dict(q=None), dict(ldq=63), dict(scale=None), dict(scale=P + 2)):
        assert back(**bad) == tw.ERR_INVALID, bad


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(K=0), dict(K=131072), dict(M=(1 << 31) - 1), dict(N=(1 << 31) - 1), dict(x=None), dict(w=None), dict(xs=None), dict(ws=None),
    dict(y=None), dict(x=P + 8), dict(w=P + 8), dict(ldx=72), dict(ldw=72), dict(ldx=48), dict(ldw=48), dict(xs=P + 2),
    dict(ws=P + 2), dict(bias=P + 2), dict(yt=I8), dict(yt=-1), dict(y=P + 1), dict(ldy=31)])
def test_int8_products_refuse(bad):
    L = tw.lib()
    a = dict(x=P, ldx=64, xs=P, w=P, ldw=64, ws=P, bias=None, M=4, N=32, K=64, y=P, yt=BF16, ldy=32)
    a.update(bad)
    st = L.twell_int8_linear(a["x"], a["ldx"], a["xs"], a["w"], a["ldw"], a["ws"], a["bias"], a["M"], a["N"], a["K"],
                             a["y"], a["yt"], a["ldy"], None)
    assert st == tw.ERR_INVALID, bad
    if "bias" in bad:
        return
    for first in (True, False):   # the refused operand as the gate's and as the up product's
        g = (a["w"], a["ldw"], a["ws"]) if first else (P, 64 if a["K"] == 64 else a["K"], P)
        u = (P, 64 if a["K"] == 64 else a["K"], P) if first else (a["w"], a["ldw"], a["ws"])
        st = L.twell_int8_gated(a["x"], a["ldx"], a["xs"], *g, *u, a["M"], a["N"], a["K"], a["y"], a["yt"], a["ldy"], None)
        assert st == tw.ERR_INVALID, bad


def test_no_rows_is_a_valid_call():
    L = tw.lib()
    assert _norm(L, M=0, x=None, y=None) == tw.OK
    assert L.twell_last_launch_count() == 0
    assert L.twell_quantize_rows(None, BF16, 64, 0, 64, None, 64, None, None) == tw.OK
    assert L.twell_dequantize_rows(None, 64, None, 0, 64, None, BF16, 64, None) == tw.OK
    assert L.twell_int8_linear(None, 64, None, None, 64, None, None, 0, 32, 64, None, BF16, 32, None) == tw.OK
    assert L.twell_layer_norm_bwd(None, F32, 64, None, F32, 64, None, None, None, F32, 0, 64, None, 64, None, None, None,
                                  0, None) == tw.OK


def test_wrappers_refuse_wrong_tensors():
    z, i8, v = torch.zeros(4, 32), torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: tw.layer_norm(z),                                       # not on a CUDA device
                 lambda: tw.layer_norm(z[0]),                                    # not a matrix
                 lambda: tw.layer_norm(z.t()),                                   # rows not contiguous
                 lambda: tw.layer_norm(z.double()),
                 lambda: tw.layer_norm(z, torch.ones(31)),
                 lambda: tw.layer_norm(z, torch.ones(32), torch.ones(32).half()),
                 lambda: tw.layer_norm(z[:1].expand(4, 32)),                     # rows overlap
                 lambda: tw.layer_norm(z, out=z.clone(), out_dtype=torch.bfloat16),
                 lambda: tw.layer_norm_int8(i8),
                 lambda: tw.layer_norm_bwd(z[:3], z, v, v),
                 lambda: tw.quantize_rows(i8),
                 lambda: tw.dequantize_rows(i8, v, torch.int32),
                 lambda: tw.dequantize_rows(z, v),
                 lambda: tw.int8_linear(i8, v, i8[:, :16], v),
                 lambda: tw.int8_linear(z, v, i8, v),
                 lambda: tw.int8_linear(i8, v, i8, v, out_dtype=torch.int8),
                 lambda: tw.int8_gated(i8, v, i8, v, i8[:3], v[:3])):
        with pytest.raises(ValueError):
            call()


def test_ctypes_signatures_cover_the_new_calls():
    L = tw.lib()
    for n in ("twell_layer_norm_fwd", "twell_layer_norm_int8", "twell_layer_norm_bwd", "twell_quantize_rows",
              "twell_dequantize_rows", "twell_int8_linear", "twell_int8_gated"):
        assert n in tw.header_functions() and getattr(L, n).argtypes[-1] is ctypes.c_void_p, n


@pytest.mark.parametrize("shape", [((1 << 32) + 5, 2), (2, (1 << 32) + 5), (1 << 31, 1)])
def test_wrappers_refuse_sizes_past_32_bits(shape):
    # The library takes sizes as 32-bit integers; cut to those, 2^32 + 5 rows would be 5.
    M, D = shape
    z, i8 = torch.empty(shape, device="meta"), torch.empty(shape, dtype=torch.int8, device="meta")
    v, d = torch.empty(M, device="meta"), torch.empty(D, device="meta")
    few, one = torch.empty((3, D), dtype=torch.int8, device="meta"), torch.empty(3, device="meta")
    for call in (lambda: tw.layer_norm(z, d, d), lambda: tw.layer_norm_int8(z, d, d), lambda: tw.quantize_rows(z),
                 lambda: tw.layer_norm_bwd(z, z, v, v), lambda: tw.dequantize_rows(i8, v),
                 lambda: tw.int8_linear(i8, v, few, one), lambda: tw.int8_linear(few, one, i8, v),
                 lambda: tw.int8_gated(few, one, i8, v, i8, v)):
        with pytest.raises(ValueError, match="2147483647"):
            call()
