"""Refusals of the grouped products and of the FP8 quantiser: the statuses that include/moe.h
documents, before any device work, and what the binding refuses by itself.

The C calls get NULL or never-dereferenced pointers, so the module runs only where no device is
visible; every call here is rejected, or has nothing to do."""
import ctypes as C

import pytest
import torch

import expert_ffn_layer_top_b200 as moe

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks; run where no device is visible")

OK, INVALID_ARG, UNSUPPORTED = 0, 1, 2
A = 1 << 24          # an aligned address that nothing reads


def _err():
    return moe.lib().moe_last_error_string().decode()


def _gemm(name, x=A, ldx=256, rows=4, off=A, w=A, ldw=256, we=0, E=8, N=256, K=256, y=A, ldy=256, fp32=0):
    return getattr(moe.lib(), name)(x, ldx, rows, off, w, ldw, we, E, N, K, y, ldy, fp32, None)


@pytest.mark.parametrize("name", ["moe_grouped_gemm", "moe_grouped_gemm_dgrad"])
def test_products_check_their_arguments(name):
    g = lambda **kw: _gemm(name, **kw)
    assert g(rows=0, x=None, w=None, y=None) == OK                 # nothing to do
    for E in (0, -1, 1025):
        assert g(E=E) == UNSUPPORTED
    assert g(N=0) == INVALID_ARG and g(K=-5) == INVALID_ARG and g(rows=-1) == INVALID_ARG
    assert g(N=(1 << 24) + 1, ldw=1 << 25) == UNSUPPORTED and g(rows=(1 << 30) + 1) == UNSUPPORTED
    assert g(off=None) == INVALID_ARG and "offsets" in _err()      # more than one expert
    assert g(off=A + 2) == INVALID_ARG
    for p in ("x", "w", "y"):
        assert g(**{p: None}) == INVALID_ARG
    assert g(x=A + 8) == INVALID_ARG and g(w=A + 2) == INVALID_ARG and "16-byte" in _err()
    assert g(ldx=255) == INVALID_ARG and g(ldx=260) == INVALID_ARG   # below a row, not a multiple of 16 bytes
    assert g(ldw=248) == INVALID_ARG and g(ldw=262) == INVALID_ARG
    assert g(we=256 * 255) == INVALID_ARG and g(we=256 * 256 + 4) == INVALID_ARG
    assert g(ldy=255) == INVALID_ARG
    assert g(y=A + 1) == INVALID_ARG and g(y=A + 2, fp32=1) == INVALID_ARG
    for ld in ("ldx", "ldw", "ldy"):                               # no product of strides leaves 64 bits
        assert g(**{ld: 1 << 60}) == INVALID_ARG and g(**{ld: (1 << 63) - 16}) == INVALID_ARG


def test_wgrad_checks_its_arguments():
    def g(dy=A, lddy=256, x=A, ldx=256, rows=4, off=A, E=8, N=256, K=256, dw=A, ld=256, es=0, fp32=1, acc=0):
        return moe.lib().moe_grouped_gemm_wgrad(dy, lddy, x, ldx, rows, off, E, N, K, dw, ld, es, fp32, acc, None)

    assert g(E=1025) == UNSUPPORTED and g(N=0) == INVALID_ARG and g(rows=-1) == INVALID_ARG
    assert g(fp32=0, acc=1) == UNSUPPORTED and "fp32" in _err()
    assert g(off=None) == INVALID_ARG
    for p in ("dy", "x", "dw"):
        assert g(**{p: None}) == INVALID_ARG
    assert g(dy=A + 2) == INVALID_ARG and g(lddy=260) == INVALID_ARG and g(ldx=128) == INVALID_ARG
    assert g(ld=255) == INVALID_ARG and g(es=256 * 255) == INVALID_ARG and g(dw=A + 2) == INVALID_ARG
    assert g(ld=1 << 60) == INVALID_ARG and g(lddy=1 << 62) == INVALID_ARG and g(es=1 << 62) == INVALID_ARG


def test_fp8_product_checks_its_arguments():
    def g(xq=A, ldx=256, xs=A, rows=4, off=A, wq=A, ldw=256, we=0, ws=A, wse=0, E=8, N=256, K=256, y=A, ldy=256, fp32=0):
        return moe.lib().moe_grouped_gemm_fp8(xq, ldx, xs, rows, off, wq, ldw, we, ws, wse, E, N, K, y, ldy, fp32, None)

    assert g(rows=0, xq=None) == OK
    assert g(E=0) == UNSUPPORTED and g(K=0) == INVALID_ARG
    for p in ("xq", "xs", "wq", "ws", "y"):
        assert g(**{p: None}) == INVALID_ARG
    assert g(ldx=264) == INVALID_ARG and g(ldw=264) == INVALID_ARG and g(xq=A + 8) == INVALID_ARG
    assert g(xs=A + 2) == INVALID_ARG and g(wse=256 * 2 - 1) == INVALID_ARG
    assert g(we=256 * 256 + 8) == INVALID_ARG and g(off=None) == INVALID_ARG


def test_quantiser_checks_its_arguments():
    def q(x=A, ldx=256, rows=4, K=256, sw=0, codes=A, ldc=256, scale=A):
        return moe.lib().moe_quantize_fp8(x, ldx, rows, K, sw, codes, ldc, scale, None)

    assert q(rows=0, x=None) == OK
    assert q(rows=-1) == INVALID_ARG
    for K in (0, -16, 8, 100):
        assert q(K=K) == INVALID_ARG
    for p in ("x", "codes", "scale"):
        assert q(**{p: None}) == INVALID_ARG
    assert q(ldx=252) == INVALID_ARG and q(ldx=260) == INVALID_ARG and q(ldc=264) == INVALID_ARG
    assert q(ldx=1 << 60) == INVALID_ARG and q(ldc=1 << 60) == INVALID_ARG
    assert q(sw=1) == INVALID_ARG                                   # gate and up need 512 columns
    assert q(x=A + 8) == INVALID_ARG and q(codes=A + 8) == INVALID_ARG and q(scale=A + 2) == INVALID_ARG


def test_the_binding_refuses_what_the_library_cannot_see():
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(2, 32, 64, dtype=bf)
    off = torch.zeros(3, dtype=torch.int32)
    bad = [
        (ValueError, lambda: moe.moe_grouped_gemm(x.float(), off, w)),                 # dtype
        (ValueError, lambda: moe.moe_grouped_gemm(x, off, w[:, :, :32])),              # K differs
        (ValueError, lambda: moe.moe_grouped_gemm(x, off[:2], w)),                     # offsets of one expert
        (ValueError, lambda: moe.moe_grouped_gemm(x, off.long(), w)),
        (ValueError, lambda: moe.moe_grouped_gemm(x, None, w)),
        (ValueError, lambda: moe.moe_grouped_gemm(torch.zeros(64, 4, dtype=bf).T, off, w)),   # columns first
        (ValueError, lambda: moe.moe_grouped_gemm(x, off, w)),                         # host tensors
        (ValueError, lambda: moe.moe_grouped_gemm_dgrad(x, off, w)),                   # N differs
        (ValueError, lambda: moe.moe_grouped_gemm_wgrad(x, x[:2], off)),
        (ValueError, lambda: moe.moe_grouped_gemm_wgrad(x, x, off, accumulate=True)),  # nothing to add to
        (ValueError, lambda: moe.moe_quantize_fp8(x.float())),
        (ValueError, lambda: moe.moe_quantize_fp8(torch.zeros(4, 33, dtype=bf), swiglu=True)),
    ]
    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    wq, ws = torch.zeros(2, 32, 256, dtype=torch.uint8), torch.zeros(2, 32, 2)
    bad += [
        (ValueError, lambda: moe.moe_grouped_gemm_fp8(q, s[:, :1], off, wq, ws)),
        (ValueError, lambda: moe.moe_grouped_gemm_fp8(q, s, off, wq, ws[:1])),
        (ValueError, lambda: moe.moe_grouped_gemm_fp8(q, s, off, wq, ws.transpose(1, 2).contiguous().transpose(1, 2))),
        (ValueError, lambda: moe.moe_grouped_gemm_fp8(q.to(torch.int8), s, off, wq, ws)),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()
    # one expert's weights seen as several have stride 0, which means "dense" to the library
    with pytest.raises(ValueError, match="expanded"):
        moe.moe_grouped_gemm(x, off, w[:1].expand(2, 32, 64))
    with pytest.raises(ValueError, match="expanded"):
        moe.moe_grouped_gemm_fp8(q, s, off, wq, ws[:1].expand(2, 32, 2))
    assert moe._lib._matrix("x", torch.zeros(1, 40, dtype=bf), (bf,)) == (1, 40, 48)   # a lone row's stride says nothing


def test_the_abi_declares_them():
    for n in ("moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad", "moe_grouped_gemm_fp8",
              "moe_quantize_fp8"):
        assert hasattr(moe, n) and isinstance(getattr(moe.lib(), n), C._CFuncPtr)
