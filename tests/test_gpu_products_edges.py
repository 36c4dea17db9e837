"""Edges of the grouped products and of the FP8 quantiser: values next to fp32's smallest, signed zeros, experts
without rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import expert_ffn_layer_top_b200 as m

    yield m
    assert m.moe_device_error() == 0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _offsets(counts):
    return torch.tensor([0] + list(counts), device="cuda").cumsum(0).int()


# ---------------------------------------------------------------------------- quantiser


@pytest.mark.parametrize("units", [1, 3, 223, 224, 225, 255])
@pytest.mark.parametrize("K", [256, 144])
def test_swiglu_blocks_next_to_the_smallest_value_stay_finite(moe, K, units):
    """silu(2^-70) = 2^-71 in fp32, so the largest value of the last block is units * 2^-149. units / 448
    rounds to 0 up to 224 (a tie at one half goes to even) and to one unit beyond."""
    x = torch.zeros(3, 2 * K, dtype=BF16)
    at = K - 7
    x[0, at], x[0, K + at] = 2.0**-70, units * 2.0**-78
    x[1, at], x[1, K + at] = 2.0**-70, -units * 2.0**-78
    x[2, at], x[2, K + at] = 1e-22, 1e-21
    codes, scale = moe.moe_quantize_fp8(x.cuda(), swiglu=True)
    values = codes.cpu().view(torch.float8_e4m3fn).float()
    want = torch.ones(3, 2)
    code = torch.zeros(3, K)
    if units > 224:
        want[:2, 1] = 2.0**-149
        code[0, at] = 224.0 if units == 225 else 256.0     # steps of 16 below 256
        code[1, at] = -code[0, at]
    assert torch.equal(scale.cpu(), want) and torch.equal(values, code)
    w = torch.ones(8, K, dtype=torch.float8_e4m3fn, device="cuda")
    y = moe.moe_grouped_gemm_fp8(codes, scale, None, w, torch.ones(8, 2, device="cuda"), y_fp32=True)
    assert torch.equal(y.cpu(), (code.sum(1) * want[:, 1])[:, None].expand(3, 8))


@pytest.mark.parametrize("rows,K", [(3, 144), (40, 1024)])
def test_signs_of_zeros_are_those_of_the_division(moe, rows, K):
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, K, generator=g).to(BF16)
    zeros = torch.rand(rows, K, generator=g)
    x[zeros < 0.2] = 0.0
    x[zeros > 0.8] = -0.0
    x[0, :128] = -0.0
    x[1, 5] = -(2.0**-60)                # a code of 0 from a value that is not
    codes, scale = moe.moe_quantize_fp8(x.cuda())
    blk = torch.nn.functional.pad(x.float(), (0, -K % 128)).view(rows, -1, 128)
    amax = blk.abs().amax(-1)
    s = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    q = (blk / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(rows, -1)[:, :K]
    assert torch.equal(scale.cpu(), s) and torch.equal(codes.cpu(), q.contiguous().view(torch.uint8))


def test_swiglu_keeps_the_sign_of_zeros(moe):
    """silu of a far negative gate is -0."""
    x = torch.ones(2, 256, dtype=BF16)
    x[:, 3] = -200.0
    x[0, 7], x[0, 128 + 7] = 0.0, -1.0
    x[1, 128 + 3] = -1.0
    codes, _ = moe.moe_quantize_fp8(x.cuda(), swiglu=True)
    codes = codes.cpu()
    assert codes[0, 3] == 0x80 and codes[1, 3] == 0x00 and codes[0, 7] == 0x80


# ---------------------------------------------------------------------------- weight gradients


@pytest.mark.parametrize("counts,N,K", [([0, 5, 0, 70], 136, 72), ([0, 900, 0, 1100, 0, 0, 700, 0], 2056, 1160),
                                        ([0, 0, 0], 64, 200)])
def test_accumulating_leaves_experts_without_rows_as_they_are(moe, counts, N, K):
    g = _gen(1)
    E, R = len(counts), sum(counts)
    dy = torch.randint(-3, 4, (R, N), generator=g, device="cuda").to(BF16)
    x = torch.randint(-3, 4, (R, K), generator=g, device="cuda").to(BF16)
    dw = torch.randint(-9, 10, (E, N, K), generator=g, device="cuda").float()
    dw[dw == 0] = -0.0
    before = dw.clone()
    launches = moe.lib().moe_kernel_launch_count()
    moe.moe_grouped_gemm_wgrad(dy, x, _offsets(counts), out=dw, accumulate=True)
    if R == 0:
        assert moe.lib().moe_kernel_launch_count() == launches
    at = 0
    for e, n in enumerate(counts):
        if n == 0:
            assert torch.equal(dw[e].view(torch.int32), before[e].view(torch.int32))
        else:
            want = before[e].double() + dy[at:at + n].double().T @ x[at:at + n].double()
            assert torch.equal(dw[e].double(), want)
        at += n
