"""What the grouped products answer or refuse before any device work, at their edges.

The C calls get never-dereferenced pointers, so the module runs only where no device is visible."""
import pytest
import torch

import expert_ffn_layer_top_b200 as moe

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks; run where no device is visible")

OK, INVALID_ARG, UNSUPPORTED = 0, 1, 2
A = 1 << 24          # an aligned address that nothing reads


def test_accumulating_no_rows_launches_nothing():
    def g(dw=A, ld=256, dy=None, x=None, fp32=1, acc=1):
        return moe.lib().moe_grouped_gemm_wgrad(dy, 256, x, 256, 0, A, 8, 256, 256, dw, ld, 0, fp32, acc, None)

    before = moe.lib().moe_kernel_launch_count()
    assert g() == OK and g(dy=A, x=A) == OK
    assert moe.lib().moe_kernel_launch_count() == before
    assert g(dw=None) == INVALID_ARG and g(ld=255) == INVALID_ARG and g(fp32=0) == UNSUPPORTED   # still checked


def test_the_binding_refuses_sizes_that_leave_32_bits():
    """Their low bits would name other, smaller sizes. Meta tensors have sizes and no memory."""
    big = 2**32 + 64

    def t(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="meta")

    x, w, off = t(4, 64), t(2, 32, 64), t(3, dtype=torch.int32)
    for call in (
        lambda: moe.moe_grouped_gemm(t(big, 64), off, w),
        lambda: moe.moe_grouped_gemm(t(4, big), off, w),
        lambda: moe.moe_grouped_gemm(x, None, t(big, 64)),
        lambda: moe.moe_grouped_gemm(x, off, t(big, 1, 64)),
        lambda: moe.moe_grouped_gemm_dgrad(t(big, 32), off, w),
        lambda: moe.moe_grouped_gemm_wgrad(t(big, 64), t(big, 64), off),
        lambda: moe.moe_quantize_fp8(t(big, 64)),
        lambda: moe.moe_quantize_fp8(t(4, big), swiglu=True),
        lambda: moe.moe_grouped_gemm_fp8(t(big, 64, dtype=torch.uint8), t(big, 1, dtype=torch.float32), off,
                                         t(2, 32, 64, dtype=torch.uint8), t(2, 32, 1, dtype=torch.float32)),
    ):
        with pytest.raises(ValueError, match="below 2.31"):
            call()
