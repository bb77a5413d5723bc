"""Argument checks of the 8-bit entry points: the C ABI's statuses (no call
here launches anything: every one fails a check or has M == 0) and the
binding's tensor checks."""
import ctypes

import pytest
import torch

import rotated_bit_amd as H
from rotated_bit_amd import _lib as L

FAKE, MIS = 0x10000, 0x10004


def fw(N=256, K=256, experts=1, w=FAKE, s=FAKE):
    return L.harp_fp8_weight(N, K, experts, w, s)


def test_weight_struct_layout():
    f = {n: getattr(L.harp_fp8_weight, n) for n, _ in L.harp_fp8_weight._fields_}
    assert [f[n].offset for n in ("N", "K", "experts", "w", "scale")] == [0, 4, 8, 16, 24]
    assert ctypes.sizeof(L.harp_fp8_weight) == 32


def norm(x=FAKE, xdt=0, r=0, ro=0, w=FAKE, wdt=0, eps=1e-6, y=FAKE, ydt=0, M=1, D=64):
    return L.lib.harp_rmsnorm(x, xdt, r, ro, w, wdt, eps, y, ydt, M, D, None)


def norm8(x=FAKE, xdt=0, r=0, ro=0, w=FAKE, wdt=0, eps=1e-6, q=FAKE, s=FAKE, M=1, D=64):
    return L.lib.harp_rmsnorm_fp8(x, xdt, r, ro, w, wdt, eps, q, s, M, D, None)


@pytest.mark.parametrize("f", [norm, norm8])
@pytest.mark.parametrize("kw,expect", [
    (dict(x=0), L.HARP_ERR_NULL), (dict(w=0), L.HARP_ERR_NULL), (dict(ro=FAKE), L.HARP_ERR_NULL),
    (dict(x=MIS), L.HARP_ERR_ALIGN), (dict(w=MIS), L.HARP_ERR_ALIGN),
    (dict(r=MIS), L.HARP_ERR_ALIGN), (dict(r=FAKE, ro=MIS), L.HARP_ERR_ALIGN),
    (dict(xdt=2), L.HARP_ERR_DTYPE), (dict(wdt=-1), L.HARP_ERR_DTYPE),
    (dict(eps=-1.0), L.HARP_ERR_SHAPE), (dict(eps=float("nan")), L.HARP_ERR_SHAPE),
    (dict(eps=float("inf")), L.HARP_ERR_SHAPE),
    (dict(D=0), L.HARP_ERR_SHAPE), (dict(D=32768 + 16), L.HARP_ERR_SHAPE),
    (dict(M=-1), L.HARP_ERR_SHAPE), (dict(M=65537), L.HARP_ERR_SHAPE),
    (dict(M=0, x=0, w=0), L.HARP_OK), (dict(M=0, D=32768), L.HARP_OK),
])
def test_norm_checks(f, kw, expect):
    assert f(**kw) == expect


def test_norm_output_checks():
    assert norm(y=0) == L.HARP_ERR_NULL and norm(y=MIS) == L.HARP_ERR_ALIGN
    assert norm(ydt=2) == L.HARP_ERR_DTYPE
    assert norm(D=33, M=0) == L.HARP_OK
    assert norm8(D=33, M=0) == L.HARP_ERR_SHAPE and norm8(D=72, M=0) == L.HARP_ERR_SHAPE
    assert norm8(q=0) == L.HARP_ERR_NULL and norm8(s=0) == L.HARP_ERR_NULL
    assert norm8(q=MIS) == L.HARP_ERR_ALIGN and norm8(s=MIS) == L.HARP_ERR_ALIGN


def silu(x=FAKE, xdt=1, q=FAKE, s=FAKE, M=1, D=64):
    return L.lib.harp_silu_mul_fp8(x, xdt, q, s, M, D, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=0), L.HARP_ERR_NULL), (dict(q=0), L.HARP_ERR_NULL), (dict(s=0), L.HARP_ERR_NULL),
    (dict(x=MIS), L.HARP_ERR_ALIGN), (dict(q=MIS), L.HARP_ERR_ALIGN),
    (dict(s=MIS), L.HARP_ERR_ALIGN), (dict(xdt=7), L.HARP_ERR_DTYPE),
    (dict(D=0), L.HARP_ERR_SHAPE), (dict(D=24), L.HARP_ERR_SHAPE),
    (dict(D=262144 + 16), L.HARP_ERR_SHAPE), (dict(M=-1), L.HARP_ERR_SHAPE),
    (dict(M=65537), L.HARP_ERR_SHAPE), (dict(M=0, x=0, q=0, s=0), L.HARP_OK),
])
def test_silu_checks(kw, expect):
    assert silu(**kw) == expect


def gemm(W=None, a=FAKE, sa=FAKE, y=FAKE, ydt=0, M=1):
    W = fw() if W is None else W
    return L.lib.harp_fp8_gemm(ctypes.byref(W), a, sa, y, ydt, M, None)


def grouped(W=None, a=FAKE, sa=FAKE, a_rows=1, rows=0, off=FAKE, y=FAKE, ydt=0, M=1):
    W = fw(experts=4) if W is None else W
    return L.lib.harp_fp8_gemm_grouped(ctypes.byref(W), a, sa, a_rows, rows, off, y, ydt, M,
                                       None)


@pytest.mark.parametrize("f", [gemm, grouped])
@pytest.mark.parametrize("kw,expect", [
    (dict(W=fw(w=0)), L.HARP_ERR_NULL), (dict(W=fw(s=0)), L.HARP_ERR_NULL),
    (dict(W=fw(w=MIS)), L.HARP_ERR_ALIGN), (dict(W=fw(s=MIS)), L.HARP_ERR_ALIGN),
    (dict(W=fw(N=0)), L.HARP_ERR_SHAPE), (dict(W=fw(N=262145)), L.HARP_ERR_SHAPE),
    (dict(W=fw(K=0)), L.HARP_ERR_SHAPE), (dict(W=fw(K=24)), L.HARP_ERR_SHAPE),
    (dict(W=fw(K=262160)), L.HARP_ERR_SHAPE), (dict(W=fw(experts=0)), L.HARP_ERR_SHAPE),
    (dict(W=fw(experts=1025)), L.HARP_ERR_SHAPE),
    (dict(a=0), L.HARP_ERR_NULL), (dict(sa=0), L.HARP_ERR_NULL), (dict(y=0), L.HARP_ERR_NULL),
    (dict(a=MIS), L.HARP_ERR_ALIGN), (dict(sa=MIS), L.HARP_ERR_ALIGN),
    (dict(y=MIS), L.HARP_ERR_ALIGN), (dict(ydt=2), L.HARP_ERR_DTYPE),
    (dict(M=-1), L.HARP_ERR_SHAPE), (dict(M=65537), L.HARP_ERR_SHAPE),
    (dict(M=0, a=0, sa=0, y=0), L.HARP_OK),
])
def test_product_checks(f, kw, expect):
    assert f(**kw) == expect


def test_product_other_checks():
    assert L.lib.harp_fp8_gemm(None, FAKE, FAKE, FAKE, 0, 1, None) == L.HARP_ERR_NULL
    assert gemm(W=fw(experts=2)) == L.HARP_ERR_SHAPE
    assert grouped(off=0) == L.HARP_ERR_NULL and grouped(off=MIS) == L.HARP_ERR_ALIGN
    assert grouped(rows=MIS) == L.HARP_ERR_ALIGN
    assert grouped(a_rows=-1) == L.HARP_ERR_SHAPE and grouped(a_rows=65537) == L.HARP_ERR_SHAPE
    assert grouped(a_rows=0) == L.HARP_ERR_SHAPE
    assert grouped(a_rows=3, M=4) == L.HARP_ERR_SHAPE          # no rows: one a row per y row
    assert grouped(a_rows=0, off=0, M=0) == L.HARP_OK
    # gathered rows are addressed with 32 bits
    wide = fw(K=131072)
    assert grouped(W=wide, a_rows=32768, rows=FAKE, M=0) == L.HARP_ERR_UNSUPPORTED
    assert grouped(W=wide, a_rows=32767, rows=FAKE, M=0) == L.HARP_OK
    assert grouped(W=wide, a_rows=65536, M=0) == L.HARP_OK


def test_binding_rejects_tensors():
    e4 = torch.float8_e4m3fn
    w, s = torch.zeros((256, 144), dtype=e4), torch.zeros((2, 2))
    W = H.FP8Weight(w, s)
    with pytest.raises(ValueError, match="scale"):
        H.FP8Weight(w, torch.zeros((2, 1)))
    with pytest.raises(TypeError, match="w"):
        H.FP8Weight(w.float(), s)
    with pytest.raises(ValueError, match="contiguous"):
        H.FP8Weight(torch.zeros((144, 256), dtype=e4).t(), s)
    with pytest.raises(ValueError):
        H.FP8Weight(torch.zeros(16, dtype=e4), s)
    a, sa, y = torch.zeros((3, 144), dtype=e4), torch.zeros((3, 2)), torch.zeros((3, 256))
    with pytest.raises(ValueError, match="a:"):
        H.harp_fp8_gemm(W, a[:, :128], sa, y)
    with pytest.raises(ValueError, match="a_scale"):
        H.harp_fp8_gemm(W, a, sa[:2], y)
    with pytest.raises(ValueError, match="y"):
        H.harp_fp8_gemm(W, a, sa, y[:, :255])
    with pytest.raises(TypeError):
        H.harp_fp8_gemm(W, a, sa, y.half())
    with pytest.raises(ValueError, match="GPU"):       # CPU tensors never reach the library
        H.harp_fp8_gemm(W, a, sa, y)
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="offsets"):
        H.harp_fp8_gemm_grouped(W, a, sa, off.long(), y)
    with pytest.raises(ValueError, match="offsets"):
        H.harp_fp8_gemm_grouped(W, a, sa, torch.zeros(3, dtype=torch.int32), y)
    with pytest.raises(ValueError, match="rows"):
        H.harp_fp8_gemm_grouped(W, a, sa, off, y, rows=off)
    x = torch.zeros((3, 64))
    with pytest.raises(ValueError, match="weight"):
        H.harp_rmsnorm(x, torch.ones(63), x.clone())
    with pytest.raises(TypeError, match="residual"):
        H.harp_rmsnorm(x, torch.ones(64), x.clone(), residual=x.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        H.harp_rmsnorm(torch.zeros((64, 3)).t(), torch.ones(64), x.clone())
    with pytest.raises(TypeError):
        H.harp_rmsnorm(x.half(), torch.ones(64), x.clone())
    q, qs = torch.zeros((3, 64), dtype=e4), torch.zeros((3, 1))
    with pytest.raises(ValueError, match="gate_up"):
        H.harp_silu_mul_fp8(x, q, qs)
    with pytest.raises(ValueError, match="q_scale"):
        H.harp_silu_mul_fp8(torch.zeros((3, 128)), q, torch.zeros((3, 2)))
