"""Edges of the grouped products and of the FP8 quantiser: values next to fp32's smallest, signed zeros, experts
without rows, the accuracy of long sums, sizes that
strides of 16 bytes do not divide, 1024 experts, calls at once."""
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


# ---------------------------------------------------------------------------- accuracy of long sums


def _off(got, want64):
    return float((got.double() - want64).norm() / want64.norm())


# columns of the result and rows per expert: tiles of single CTAs, and CTA pairs
SUMS = [([20], 520), ([300, 301, 255, 0, 513, 100, 1, 700], 2056)]
C = 4096


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("counts,cols", SUMS)
def test_fp32_sums_are_as_exact_as_parts_of_512_make_them(moe, counts, cols, positive):
    """The tensor core cuts the sum off after each step of 16 products: by half a unit in the last place on
    average, which is ln 2 * 2^-24 of the sum on average over a binade, and by a unit at most. (The products
    have 16 bits and a part's sum is at most 2^9 of them, so aligning them with it cuts hardly any.) Around 0
    the sum grows like the square root of the steps: over the 32 steps of a part of 512 it loses no more than
    0.69 * 2^-24 * 2/3 * 32 = 9e-7 of its size were every step to err the same way; parts err by
    themselves, and adding up eight of them in rounded fp32 is below 2e-7: 1.5e-6. One part of 4096 lost
    4.4e-6. Positive operands grow like the steps and all parts err downwards: a whole unit a step is
    2^-23 * 16.5 = 2.0e-6, with the roundings 2.5e-6; a single part would lose half a unit in 256 steps,
    0.69 * 2^-24 * 128 = 5.3e-6."""
    g = _gen(2)
    bound = 2.5e-6 if positive else 1.5e-6
    draw = torch.rand if positive else torch.randn
    E, R, off = len(counts), sum(counts), _offsets(counts)
    at = [0] + torch.tensor(counts).cumsum(0).tolist()
    x = draw(R, C, generator=g, device="cuda").to(BF16)
    w = draw(E, cols, C, generator=g, device="cuda").to(BF16)
    want = torch.cat([x[at[e]:at[e + 1]].double() @ w[e].double().T for e in range(E)])
    wt = w.transpose(1, 2).contiguous()
    assert _off(moe.moe_grouped_gemm(x, off, w, y_fp32=True), want) < bound
    assert _off(moe.moe_grouped_gemm_dgrad(x, off, wt, dx_fp32=True), want) < bound


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("counts,N,K", [([4096], 200, 264), ([4100, 4096], 2056, 1160)])
def test_fp32_weight_gradients_are_as_exact_as_parts_of_512_make_them(moe, counts, N, K, positive):
    """As above, the sum running over an expert's rows."""
    g = _gen(3)
    draw = torch.rand if positive else torch.randn
    R = sum(counts)
    dy = draw(R, N, generator=g, device="cuda").to(BF16)
    x = draw(R, K, generator=g, device="cuda").to(BF16)
    dw = moe.moe_grouped_gemm_wgrad(dy, x, _offsets(counts))
    at = 0
    for e, n in enumerate(counts):
        assert _off(dw[e], dy[at:at + n].double().T @ x[at:at + n].double()) < (2.5e-6 if positive else 1.5e-6)
        at += n


def test_bf16_results_of_long_sums_lean_to_no_side(moe):
    """Positive operands, 2^18 rows: bf16 results add up parts of 8192. Each of a part's 512 steps cuts the
    sum and, that far above them, its 16 products too, each by half a unit at most on average:
    17 * 0.69 * 2^-24 * 256 = 1.8e-4 of the sum. Rounding to bf16 is off by up to 2^-8, 1.66e-3 in the root
    mean square, and leans to no side, so the mean over 256 * 256 results deviates by 6.5e-6: three of them
    make 2e-4. One part of 2^18 would lose more, half a unit of the sum alone in 2^14 steps:
    0.69 * 2^-24 * 2^13 = 3.4e-4."""
    g = _gen(4)
    R, N, K = 1 << 18, 256, 256
    dy = torch.rand(R, N, generator=g, device="cuda")
    dy = (dy * torch.exp2(torch.rand(N, generator=g, device="cuda") * 4)).to(BF16)   # results spread over binades
    x = torch.rand(R, K, generator=g, device="cuda")
    x = (x * torch.exp2(torch.rand(K, generator=g, device="cuda") * 4)).to(BF16)
    want = dy.double().T @ x.double()
    rel = (moe.moe_grouped_gemm_wgrad(dy, x, None, dw_fp32=False)[0].double() - want) / want
    assert abs(float(rel.mean())) < 2e-4 and float(rel.abs().max()) <= 2.0**-8 + 2e-4


# ---------------------------------------------------------------------------- sizes


def _ints(g, rows, cols, *experts, unit=8):
    """Whole numbers in rows whose stride is a multiple of `unit` and whose padding is NaN."""
    wide = torch.full((*experts, rows, -(-cols // unit) * unit), float("nan"), dtype=BF16, device="cuda")
    wide[..., :cols] = torch.randint(-3, 4, (*experts, rows, cols), generator=g, device="cuda").to(BF16)
    return wide[..., :cols]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("K,N", [(1, 1), (5, 3), (3, 129), (131, 7), (577, 257), (1025, 2049)])
@pytest.mark.parametrize("counts", [[1, 0, 2], [37, 0, 5, 300]])
def test_odd_sizes_in_every_direction(moe, counts, K, N, fp32):
    g = _gen(5)
    E, R, off = len(counts), sum(counts), _offsets(counts)
    at = [0] + torch.tensor(counts).cumsum(0).tolist()
    parts = [slice(at[e], at[e + 1]) for e in range(E)]
    x, dy, w = _ints(g, R, K), _ints(g, R, N), _ints(g, N, K, E)
    dt = torch.float32 if fp32 else BF16

    def same(got, want64):
        assert got.dtype == dt and torch.equal(got, want64.float().to(dt))

    same(moe.moe_grouped_gemm(x, off, w, y_fp32=fp32), torch.cat([x[p].double() @ w[e].double().T for e, p in enumerate(parts)]))
    same(moe.moe_grouped_gemm_dgrad(dy, off, w, dx_fp32=fp32), torch.cat([dy[p].double() @ w[e].double() for e, p in enumerate(parts)]))
    same(moe.moe_grouped_gemm_wgrad(dy, x, off, dw_fp32=fp32), torch.stack([dy[p].double().T @ x[p].double() for p in parts]))
    # fp8: codes of the same whole numbers, NaN behind K
    KB = -(-K // 128)

    def codes(t):
        wide = torch.full((*t.shape[:-1], -(-K // 16) * 16), 0x7F, dtype=torch.uint8, device="cuda")
        wide[..., :K] = t.float().to(torch.float8_e4m3fn).view(torch.uint8)
        return wide[..., :K]

    xs = torch.exp2(torch.randint(-3, 2, (R, KB), generator=g, device="cuda").float())
    ws = torch.exp2(torch.randint(-3, 2, (E, N, KB), generator=g, device="cuda").float())
    xf = x.double() * xs.double().repeat_interleave(128, dim=-1)[..., :K]
    wf = w.double() * ws.double().repeat_interleave(128, dim=-1)[..., :K]
    same(moe.moe_grouped_gemm_fp8(codes(x), xs, off, codes(w), ws, y_fp32=fp32),
         torch.cat([xf[p] @ wf[e].T for e, p in enumerate(parts)]))


def test_as_many_experts_as_there_may_be(moe):
    """1024 experts, of which the first, the last and a few between have rows."""
    g = _gen(6)
    counts = [0] * 1024
    for e, n in ((0, 3), (31, 1), (32, 70), (500, 2), (991, 40), (1023, 5)):
        counts[e] = n
    R, K, N, off = sum(counts), 72, 40, _offsets(counts)
    x, dy, w = _ints(g, R, K), _ints(g, R, N), _ints(g, N, K, 1024)
    e = torch.arange(1024, device="cuda").repeat_interleave(torch.tensor(counts, device="cuda"))
    w64 = w[e].double()
    assert torch.equal(moe.moe_grouped_gemm(x, off, w, y_fp32=True).double(), torch.einsum("rk,rnk->rn", x.double(), w64))
    assert torch.equal(moe.moe_grouped_gemm_dgrad(dy, off, w, dx_fp32=True).double(), torch.einsum("rn,rnk->rk", dy.double(), w64))
    dw = torch.zeros(1024, N, K, dtype=torch.float64, device="cuda")
    dw.index_add_(0, e, torch.einsum("rn,rk->rnk", dy.double(), x.double()))
    assert torch.equal(moe.moe_grouped_gemm_wgrad(dy, x, off).double(), dw)
    codes = torch.zeros(R, 80, dtype=torch.uint8, device="cuda")[:, :K]
    codes.copy_(x.float().to(torch.float8_e4m3fn).view(torch.uint8))
    wq = torch.zeros(1024, N, 80, dtype=torch.uint8, device="cuda")[..., :K]
    wq.copy_(w.float().to(torch.float8_e4m3fn).view(torch.uint8))
    one = lambda *s: torch.ones(*s, 1, device="cuda")
    got = moe.moe_grouped_gemm_fp8(codes, one(R), off, wq, one(1024, N), y_fp32=True)
    assert torch.equal(got.double(), torch.einsum("rk,rnk->rn", x.double(), w64))


def test_two_streams_and_two_threads_at_once(moe):
    """Products of all kinds under way together, from two host threads on two streams, on shared inputs."""
    import threading

    g = _gen(7)
    counts, K, N = [300, 301, 255, 0, 513, 100, 1, 700], 512, 1032
    R, off = sum(counts), _offsets(counts)
    x, dy, w = _ints(g, R, K), _ints(g, R, N), _ints(g, N, K, len(counts))
    wq, ws = moe.moe_quantize_fp8(w.reshape(-1, K))
    wq, ws = wq.view(len(counts), N, K), ws.view(len(counts), N, -1)

    def step():
        xq, xs = moe.moe_quantize_fp8(x)
        y = moe.moe_grouped_gemm_fp8(xq, xs, off, wq, ws)
        return [moe.moe_grouped_gemm(x, off, w), moe.moe_grouped_gemm_dgrad(dy, off, w), moe.moe_grouped_gemm_wgrad(dy, x, off),
                xq, xs, y, *moe.moe_quantize_fp8(y[:, :1024].contiguous(), swiglu=True)]

    want = step()
    torch.cuda.synchronize()
    got = [[], []]

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = step()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for outs in got:
        assert len(outs) == len(want) and all(torch.equal(a, b) for a, b in zip(outs, want))
