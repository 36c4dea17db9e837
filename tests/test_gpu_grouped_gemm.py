"""The products grouped by expert, their gradients, the FP8 quantiser and the FP8 product
against the formulas in 64 bits.

Most cases use small whole numbers: bf16 holds them, every product and every partial sum
stays below 2^24, so fp32 sums are exact in any order and the results have to be equal (bf16
results: equal to the exact sum rounded once). E4M3 holds the whole numbers up to 16, and
scales that are powers of two keep the FP8 sums exact as well.

With random values the bound is: a step of the tensor core adds 16 (FP8: 32) products to the
sum, each addition losing at most one unit in the last place of fp32, 2^-23 of the largest
term, so n terms lose at most 1.1 n 2^-23 S, S being the sum of the terms' magnitudes; the
FP8 product adds two multiplications and an addition per block, 3 * 2^-24 of its part each;
a bf16 result adds half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import oracle
import synthetic
from gpu_util import TOL, rel_err

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


def _ints(g, *shape, top=3):
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(BF16)


def _offsets(counts, start=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + start, dtype=torch.int32, device="cuda")


def _per_row(counts, w):
    """w[e(r)] by expert, in 64 bits: a list of (rows, w)."""
    at = 0
    for e, n in enumerate(counts):
        yield slice(at, at + n), w[e].double()
        at += n


def _forward64(x, counts, w):
    return torch.cat([x[s].double() @ we.T for s, we in _per_row(counts, w)]) if counts else x


def _dgrad64(dy, counts, w):
    return torch.cat([dy[s].double() @ we for s, we in _per_row(counts, w)])


def _wgrad64(dy, x, counts):
    out, at = [], 0
    for n in counts:
        out.append(dy[at:at + n].double().T @ x[at:at + n].double())
        at += n
    return torch.stack(out)


def _same(got, want64, fp32):
    want = want64.to(torch.float32) if fp32 else want64.to(torch.float32).to(BF16)
    assert got.dtype == want.dtype and got.shape == want.shape
    assert torch.equal(got, want), f"{(got != want).sum().item()} of {got.numel()} differ, first at " \
                                   f"{(got != want).nonzero()[0].tolist()}"


# rows per expert, K, N: one token, empty experts, tiles that end inside, one under and one over a
# tile, sizes that no tile divides, K and N below one tile, sums of more than one part of 8192
SHAPES = [
    ([1], 64, 128), ([1], 8, 8), ([3, 0, 1], 2048, 256), ([0, 0, 5, 0], 128, 520), ([16, 17, 15], 264, 136),
    ([255, 256, 257], 128, 256), ([511, 1, 513, 0, 31], 192, 384), ([1300], 512, 1000), ([64] * 9, 768, 264),
    ([2, 1] * 40, 256, 512), ([33, 700, 129, 5], 1000, 1160), ([8] * 200, 72, 40), ([30] * 6, 200, 264),
    ([1, 0, 2] * 300, 64, 72), ([9, 40], 8264, 72), ([3, 9], 72, 8264), ([8300, 16500], 72, 136),
]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_forward_is_exact_on_whole_numbers(moe, counts, K, N, fp32):
    g = _gen(1)
    x, w = _ints(g, sum(counts), K), _ints(g, len(counts), N, K)
    y = moe.moe_grouped_gemm(x, _offsets(counts), w, y_fp32=fp32)
    _same(y, _forward64(x, counts, w), fp32)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_dgrad_is_exact_on_whole_numbers(moe, counts, K, N, fp32):
    g = _gen(2)
    dy, w = _ints(g, sum(counts), N), _ints(g, len(counts), N, K)
    dx = moe.moe_grouped_gemm_dgrad(dy, _offsets(counts), w, dx_fp32=fp32)
    _same(dx, _dgrad64(dy, counts, w), fp32)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_wgrad_is_exact_on_whole_numbers(moe, counts, K, N, fp32):
    g = _gen(3)
    dy, x = _ints(g, sum(counts), N), _ints(g, sum(counts), K)
    dw = moe.moe_grouped_gemm_wgrad(dy, x, _offsets(counts), dw_fp32=fp32)
    _same(dw, _wgrad64(dy, x, counts), fp32)
    if fp32:   # added to what is there
        base = _ints(g, *dw.shape).float()
        out = base.clone()
        assert moe.moe_grouped_gemm_wgrad(dy, x, _offsets(counts), out=out, accumulate=True) is out
        assert torch.equal(out, base + dw)


@pytest.mark.parametrize("wide,other", [(4104, 320), (8200, 72)])
def test_wide_results_in_strips(moe, wide, other):
    """More than 4096 columns of the result, whose tiles go in strips, several rows of tiles each."""
    g = _gen(20)
    counts = [700, 0, 300, 513]
    R, E, off = sum(counts), len(counts), _offsets(counts)
    x, w = _ints(g, R, other), _ints(g, E, wide, other)
    _same(moe.moe_grouped_gemm(x, off, w), _forward64(x, counts, w), False)
    dy, w = _ints(g, R, other), _ints(g, E, other, wide)
    _same(moe.moe_grouped_gemm_dgrad(dy, off, w, dx_fp32=True), _dgrad64(dy, counts, w), True)
    x = _ints(g, R, wide)
    _same(moe.moe_grouped_gemm_wgrad(dy, x, off), _wgrad64(dy, x, counts), True)
    K = other // 16 * 16
    xq, xs, xf = _fp8_ints(g, R, K)
    wq, ws, wf = _fp8_ints(g, E, wide, K)
    _same(moe.moe_grouped_gemm_fp8(xq, xs, off, wq, ws), _forward64(xf, counts, wf), False)


FP8_SHAPES = [
    ([1], 128, 128), ([1], 16, 8), ([3, 0, 1], 2048, 256), ([0, 0, 5, 0], 144, 520), ([16, 17, 15], 272, 136),
    ([255, 256, 257], 128, 256), ([511, 1, 513, 0, 31], 640, 384), ([1300], 512, 1000), ([64] * 9, 768, 264),
    ([2, 1] * 40, 256, 512), ([33, 700, 129, 5], 1008, 1160), ([30] * 6, 208, 264), ([1, 0, 2] * 300, 64, 96),
]


def _fp8_ints(g, *shape):
    """Codes of whole numbers up to 4, and scales that are powers of two."""
    v = torch.randint(-4, 5, shape, generator=g, device="cuda").float()
    KB = -(-shape[-1] // 128)
    e = torch.randint(-3, 2, (*shape[:-1], KB), generator=g, device="cuda")
    scale = torch.exp2(e.float())
    full = v * scale.repeat_interleave(128, dim=-1)[..., : shape[-1]]
    return v.to(torch.float8_e4m3fn).view(torch.uint8), scale.contiguous(), full


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("counts,K,N", FP8_SHAPES)
def test_fp8_is_exact_on_whole_numbers(moe, counts, K, N, fp32):
    g = _gen(4)
    xq, xs, x = _fp8_ints(g, sum(counts), K)
    wq, ws, w = _fp8_ints(g, len(counts), N, K)
    y = moe.moe_grouped_gemm_fp8(xq, xs, _offsets(counts), wq, ws, y_fp32=fp32)
    _same(y, _forward64(x, counts, w), fp32)


@pytest.mark.parametrize("rows", [1, 2, 15, 130, 1000])
def test_plain_products_without_experts(moe, rows):
    g = _gen(5)
    K, N = 384, 272
    x, w, dy = _ints(g, rows, K), _ints(g, N, K), _ints(g, rows, N)
    _same(moe.moe_grouped_gemm(x, None, w, y_fp32=True), x.double() @ w.double().T, True)
    _same(moe.moe_grouped_gemm_dgrad(dy, None, w, dx_fp32=True), dy.double() @ w.double(), True)
    _same(moe.moe_grouped_gemm_wgrad(dy, x, None), (dy.double().T @ x.double())[None], True)
    xq, xs, xf = _fp8_ints(g, rows, K)
    wq, ws, wf = _fp8_ints(g, N, K)
    _same(moe.moe_grouped_gemm_fp8(xq.view(torch.float8_e4m3fn), xs, None, wq, ws, y_fp32=True), xf.double() @ wf.double().T,
          True)


# ---------------------------------------------------------------------------- random values


def _within(got, want64, terms, S, extra=0.0):
    tol = (1.1 * terms * 2.0**-23 + extra) * S
    if got.dtype == BF16:
        tol = tol + 2.0**-8 * want64.abs()
    err = (got.double() - want64).abs()
    assert (err <= tol).all(), f"worst {float((err / tol.clamp_min(1e-300)).max()):.2f} of the bound"


COUNTS = [70, 0, 1, 300, 22]
MANY = [300, 301, 255, 0, 513, 100, 1, 700]   # rows that CTA pairs take


@pytest.mark.parametrize("COUNTS,K,N", [(COUNTS, 600, 328), (MANY, 1160, 2056), (MANY, 2056, 1160), ([1300], 600, 1000)])
@pytest.mark.parametrize("fp32", [False, True])
def test_random_values_stay_within_the_bound(moe, fp32, COUNTS, K, N):
    g = _gen(6)
    R, E = sum(COUNTS), len(COUNTS)
    x = torch.randn(R, K, generator=g, device="cuda").to(BF16)
    dy = torch.randn(R, N, generator=g, device="cuda").to(BF16)
    w = (torch.randn(E, N, K, generator=g, device="cuda") * 0.02).to(BF16)
    off = _offsets(COUNTS)
    _within(moe.moe_grouped_gemm(x, off, w, y_fp32=fp32), _forward64(x, COUNTS, w), K, _forward64(x.abs(), COUNTS, w.abs()))
    _within(moe.moe_grouped_gemm_dgrad(dy, off, w, dx_fp32=fp32), _dgrad64(dy, COUNTS, w), N,
            _dgrad64(dy.abs(), COUNTS, w.abs()))
    _within(moe.moe_grouped_gemm_wgrad(dy, x, off, dw_fp32=fp32), _wgrad64(dy, x, COUNTS), max(COUNTS),
            _wgrad64(dy.abs(), x.abs(), COUNTS))


@pytest.mark.parametrize("COUNTS,K,N", [(COUNTS, 640, 328), (COUNTS, 2000, 328), (MANY, 2000, 2056), ([1300], 640, 1000)])
@pytest.mark.parametrize("fp32", [False, True])
def test_fp8_random_values_stay_within_the_bound(moe, fp32, COUNTS, K, N):
    g = _gen(7)
    R, E = sum(COUNTS), len(COUNTS)
    xq, xs = moe.moe_quantize_fp8(torch.randn(R, K, generator=g, device="cuda").to(BF16))
    wq, ws = moe.moe_quantize_fp8((torch.randn(E * N, K, generator=g, device="cuda") * 0.02).to(BF16))
    wq, ws = wq.view(E, N, K), ws.view(E, N, -1)

    def full(q, s):
        return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, dim=-1)[..., :K]

    x, w = full(xq, xs), full(wq, ws)
    y = moe.moe_grouped_gemm_fp8(xq, xs, _offsets(COUNTS), wq, ws, y_fp32=fp32)
    _within(y, _forward64(x, COUNTS, w), K, _forward64(x.abs(), COUNTS, w.abs()), extra=3 * 2.0**-24)


# ---------------------------------------------------------------------------- layouts and neighbours


@pytest.mark.parametrize("N", [1, 3, 130])
@pytest.mark.parametrize("rows", [5, 200])
def test_results_of_few_or_odd_columns(moe, rows, N):
    g = _gen(21)
    x, w = _ints(g, rows, 200), _ints(g, N, 200)
    for fp32 in (False, True):
        _same(moe.moe_grouped_gemm(x, None, w, y_fp32=fp32), x.double() @ w.double().T, fp32)
    xq, xs, xf = _fp8_ints(g, rows, 208)
    wq, ws, wf = _fp8_ints(g, N, 208)
    _same(moe.moe_grouped_gemm_fp8(xq, xs, None, wq, ws, y_fp32=True), xf.double() @ wf.double().T, True)


def _strided(t, pad, fill):
    """The same values with `pad` more elements between rows (and experts), holding `fill`."""
    big = torch.full((*t.shape[:-2], t.shape[-2] + 1, t.shape[-1] + pad), fill, dtype=t.dtype, device=t.device)
    view = big[..., : t.shape[-2], : t.shape[-1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("pad_out", [8, 3])
@pytest.mark.parametrize("fp32", [False, True])
def test_strides_padding_and_rows_outside_the_experts(moe, fp32, pad_out):
    """Row and expert strides; rows before offsets[0] and behind offsets[E] hold NaN and stay as they
    were in the result, as does the space between rows."""
    g = _gen(8)
    counts, K, N, before, after = [40, 0, 300, 7], 200, 264, 5, 11
    E, R = len(counts), sum(counts)
    n = before + R + after
    off = _offsets(counts, before)
    rows = slice(before, before + R)
    dt = torch.float32 if fp32 else BF16
    nan = float("nan")

    def rows_of(cols):
        t = torch.full((n, cols), nan, dtype=BF16, device="cuda")
        t[rows] = _ints(g, R, cols)
        return _strided(t, 8, nan)

    def out_of(*shape):
        big = torch.full((*shape[:-1], shape[-1] + pad_out), 7.0, dtype=dt, device="cuda")
        return big, big[..., : shape[-1]]

    x, dy, w = rows_of(K), rows_of(N), _strided(_ints(g, E, N, K), 8, nan)
    for cols, call, want in ((N, lambda o: moe.moe_grouped_gemm(x, off, w, y_fp32=fp32, out=o), _forward64(x[rows], counts, w)),
                             (K, lambda o: moe.moe_grouped_gemm_dgrad(dy, off, w, dx_fp32=fp32, out=o),
                              _dgrad64(dy[rows], counts, w))):
        big, out = out_of(n, cols)
        assert call(out) is out
        _same(out[rows].contiguous(), want, fp32)
        big[rows, :cols] = 7.0
        assert (big == 7.0).all()
    big, out = out_of(E, N, K)
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw_fp32=fp32, out=out)
    _same(out.contiguous(), _wgrad64(dy[rows], x[rows], counts), fp32)
    assert (big[..., K:] == 7.0).all()
    # fp8, one byte wide: strides of 16
    xq, xs, xf = _fp8_ints(g, n, 208)
    wq, ws, wf = _fp8_ints(g, E, N, 208)
    xs[:before], xs[before + R:] = nan, nan
    big, out = out_of(n, N)
    wss = torch.full((E, N + 1, ws.shape[2]), nan, device="cuda")[:, :N]
    wss.copy_(ws)
    moe.moe_grouped_gemm_fp8(_strided(xq, 16, 0x7F), xs, off, _strided(wq, 16, 0x7F), wss, y_fp32=fp32, out=out)
    _same(out[rows].contiguous(), _forward64(xf[rows], counts, wf), fp32)
    big[rows, :N] = 7.0
    assert (big == 7.0).all()


@pytest.mark.parametrize("pad_out", [0, 1, 2, 4])
@pytest.mark.parametrize("rows", [20, 150])
def test_fp8_results_of_any_alignment(moe, rows, pad_out):
    """Weight rows in whole groups of 32, whose results are stored four at a time where the result allows."""
    g = _gen(19)
    K, N = 256, 160
    xq, xs, x = _fp8_ints(g, rows, K)
    wq, ws, w = _fp8_ints(g, N, K)
    for dt, fp32 in ((BF16, False), (torch.float32, True)):
        for shift in (0, 1, 4):
            big = torch.full((rows * (N + pad_out) + 8,), 7.0, dtype=dt, device="cuda")
            out = big[shift:shift + rows * (N + pad_out)].view(rows, N + pad_out)[:, :N]
            moe.moe_grouped_gemm_fp8(xq, xs, None, wq, ws, y_fp32=fp32, out=out)
            _same(out.contiguous(), x.double() @ w.double().T, fp32)
            out.fill_(7.0)
            assert (big == 7.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_row_and_an_expert_keep_their_values_to_themselves(moe, bad):
    """Expert 1's rows and weights are not finite: nothing of them reaches experts 0 and 2, whose rows
    share tiles and blocks with them in memory."""
    g = _gen(9)
    counts, K, N = [37, 5, 90], 320, 200
    R, mid = sum(counts), slice(37, 42)
    off = _offsets(counts)
    x, dy, w = _ints(g, R, K), _ints(g, R, N), _ints(g, 3, N, K)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[mid] = False
    y0, d0, g0 = _forward64(x, counts, w), _dgrad64(dy, counts, w), _wgrad64(dy, x, counts)
    x[mid], dy[mid], w[1] = bad, bad, bad
    y, d = moe.moe_grouped_gemm(x, off, w, y_fp32=True), moe.moe_grouped_gemm_dgrad(dy, off, w, dx_fp32=True)
    dw = moe.moe_grouped_gemm_wgrad(dy, x, off)
    assert torch.equal(y[keep], y0[keep].float()) and torch.equal(d[keep], d0[keep].float())
    assert torch.equal(dw[[0, 2]], g0[[0, 2]].float())
    assert not torch.isfinite(y[mid]).any() and not torch.isfinite(d[mid]).any() and not torch.isfinite(dw[1]).any()
    # one bad row inside an expert stays in its own row
    x2, w2 = _ints(g, R, K), _ints(g, 3, N, K)
    y2 = _forward64(x2, counts, w2)
    x2[50] = bad
    got = moe.moe_grouped_gemm(x2, off, w2, y_fp32=True)
    keep[mid] = True
    keep[50] = False
    assert torch.equal(got[keep], y2[keep].float()) and not torch.isfinite(got[50]).any()
    # fp8: NaN codes and scales
    xq, xs, xf = _fp8_ints(g, R, K)
    wq, ws, wf = _fp8_ints(g, 3, N, K)
    want = _forward64(xf, counts, wf).float()
    xq[50], xs[51] = 0x7F, bad
    wq[1] = 0x7F
    keep[51] = False
    keep[mid] = False
    got = moe.moe_grouped_gemm_fp8(xq, xs, off, wq, ws, y_fp32=True)
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[50]).all() and torch.isnan(got[mid]).all() and not torch.isfinite(got[51]).any()


# rows per expert and output columns that take each of the tiles (bf16; fp8): of 64; 32, 64; 128, 64;
# 128, 64; pairs; pairs; pairs; 128, 128
TILES = [
    ([40, 0, 33, 70, 12] * 30, 1160), ([45] * 40, 2056), ([64, 100, 128, 60, 90, 70, 110, 33], 2056),
    ([80, 64, 65, 0, 129, 63] * 4, 2056), (MANY, 2056), ([1100, 257, 3, 0] * 3, 2056), ([2500], 1160), ([1300], 1000),
]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("counts,cols", TILES)
def test_every_tile_keeps_to_its_rows(moe, counts, cols, fp32):
    """Exact results from strided operands; rows before the first expert and behind the last hold NaN and
    stay as they were; one expert's rows and weights are NaN, and one row of another."""
    g = _gen(23)
    E, R, before, after, C = len(counts), sum(counts), 5, 11, 272
    n = before + R + after
    off = _offsets(counts, before)
    rows = slice(before, before + R)
    nan = float("nan")
    at = np.concatenate([[0], np.cumsum(counts)])
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    lone = int(at[E // 2]) if E > 1 else 700     # a row that is NaN by itself
    keep[lone] = False
    bad = max(e for e in range(E) if counts[e] and e != E // 2) if E > 1 else None
    if bad is not None:
        keep[at[bad]:at[bad + 1]] = False

    def check(call, want):
        big = torch.full((n, cols + 8), 7.0, dtype=torch.float32 if fp32 else BF16, device="cuda")
        got = call(big[:, :cols])[rows]
        _same(got[keep], want[keep], fp32)
        assert torch.isnan(got[~keep]).all()
        big[rows, :cols] = 7.0
        assert (big == 7.0).all()

    x = torch.full((n, C), nan, dtype=BF16, device="cuda")
    x[rows] = _ints(g, R, C)
    x[rows][~keep] = nan
    x = _strided(x, 8, nan)
    w = _ints(g, E, cols, C)
    if bad is not None:
        w[bad] = nan
    wt = _strided(w.transpose(1, 2).contiguous(), 8, nan)
    w = _strided(w, 8, nan)
    want = _forward64(x[rows], counts, w)
    check(lambda o: moe.moe_grouped_gemm(x, off, w, y_fp32=fp32, out=o), want)
    check(lambda o: moe.moe_grouped_gemm_dgrad(x, off, wt, dx_fp32=fp32, out=o), want)
    xq, xs, xf = _fp8_ints(g, n, C)
    wq, ws, wf = _fp8_ints(g, E, cols, C)
    want = _forward64(xf[rows], counts, wf)
    xq[rows][~keep] = 0x7F
    xq[:before], xs[before + R:] = 0x7F, nan
    if bad is not None:
        ws[bad] = nan
    check(lambda o: moe.moe_grouped_gemm_fp8(_strided(xq, 16, 0x7F), xs, off, _strided(wq, 16, 0x7F), ws, y_fp32=fp32, out=o),
          want)


# tiles of 64 columns, 64, 128, 128, pairs, pairs
WGRAD_TILES = [
    ([1, 17, 0, 63, 130], 200, 264), ([700, 4300], 512, 264), ([100, 64, 65, 0, 128, 129, 1, 112], 512, 1160), ([2500], 1160, 1160),
    (MANY, 2056, 1160), ([1300, 0, 1101], 2056, 1160),
]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("counts,N,K", WGRAD_TILES)
def test_every_tile_of_weight_gradients_keeps_to_its_expert(moe, counts, N, K, fp32):
    """Exact from strided operands, added to what is there or not; the rows around the experts hold NaN,
    and one expert's rows too."""
    g = _gen(24)
    E, R, before, after = len(counts), sum(counts), 3, 11
    off = _offsets(counts, before)
    rows = slice(before, before + R)
    x = torch.full((before + R + after, K), float("nan"), dtype=BF16, device="cuda")
    dy = torch.full((before + R + after, N), float("nan"), dtype=BF16, device="cuda")
    x[rows], dy[rows] = _ints(g, R, K), _ints(g, R, N)
    keep = torch.ones(E, dtype=torch.bool, device="cuda")
    if E > 1:
        keep[1] = False
        x[rows][counts[0]:counts[0] + counts[1]] = float("nan")
    x, dy = _strided(x, 8, float("nan")), _strided(dy, 16, float("nan"))
    want = _wgrad64(dy[rows], x[rows], counts)
    big = torch.full((E, N, K + 8), 7.0, dtype=torch.float32 if fp32 else BF16, device="cuda")
    out = big[..., :K]
    assert moe.moe_grouped_gemm_wgrad(dy, x, off, dw_fp32=fp32, out=out) is out
    _same(out[keep], want[keep], fp32)
    if E > 1:
        assert torch.isnan(out[1]).all() or counts[1] == 0
    if fp32:
        moe.moe_grouped_gemm_wgrad(dy, x, off, out=out, accumulate=True)
        _same(out[keep], 2 * want[keep], fp32)
    assert (big[..., K:] == 7.0).all()


def test_empty_batches(moe):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    w = _ints(_gen(10), 3, 64, 72)
    none = torch.empty(0, 72, dtype=BF16, device="cuda")
    dnone = torch.empty(0, 64, dtype=BF16, device="cuda")
    assert moe.moe_grouped_gemm(none, off, w).shape == (0, 64)
    assert moe.moe_grouped_gemm_dgrad(dnone, off, w).shape == (0, 72)
    assert (moe.moe_grouped_gemm_wgrad(dnone, none, off) == 0).all()
    kept = torch.full((3, 64, 72), 5.0, device="cuda")
    moe.moe_grouped_gemm_wgrad(dnone, none, off, out=kept, accumulate=True)
    assert (kept == 5.0).all()
    codes, scale = moe.moe_quantize_fp8(torch.empty(0, 256, dtype=BF16, device="cuda"))
    assert codes.shape == (0, 256) and scale.shape == (0, 2)
    # rows that belong to no expert
    x = _ints(_gen(11), 9, 72)
    out = torch.full((9, 64), 3.0, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm(x, off, w, out=out)
    assert (out == 3.0).all()
    assert (moe.moe_grouped_gemm_wgrad(_ints(_gen(12), 9, 64), x, off) == 0).all()


def test_offsets_outside_the_rows_are_cut_and_reported(moe):
    g = _gen(13)
    x, w = _ints(g, 50, 128), _ints(g, 3, 96, 128)
    dy = _ints(g, 50, 96)
    off = torch.tensor([-4, 20, 10, 70], dtype=torch.int32, device="cuda")   # rows 0-19, none, 10-49
    y = moe.moe_grouped_gemm(x, off, w, y_fp32=True)
    assert moe.moe_device_error() == 2
    _same(y[20:].contiguous(), x[20:].double() @ w[2].double().T, True)
    _same(y[:10].contiguous(), x[:10].double() @ w[0].double().T, True)
    dw = moe.moe_grouped_gemm_wgrad(dy, x, off)
    assert moe.moe_device_error() == 2
    want = torch.stack([dy[:20].double().T @ x[:20].double(), torch.zeros(96, 128, dtype=torch.float64, device="cuda"),
                        dy[10:].double().T @ x[10:].double()])
    _same(dw, want, True)


def test_results_past_32_bit_offsets(moe):
    """More than 2^31 elements in x and in y."""
    g = _gen(14)
    K = N = 1024
    n = (1 << 31) // K + 300
    x = torch.randint(-3, 4, (n, K), generator=g, device="cuda", dtype=torch.int8).to(BF16)
    counts = [n - 200, 150, 50]
    w = _ints(g, 3, N, K)
    y = moe.moe_grouped_gemm(x, _offsets(counts), w)
    tail = slice(n - 300, n)
    _same(y[tail], _forward64(x[tail], [100, 150, 50], w), False)
    _same(y[:64], x[:64].double() @ w[0].double().T, False)


def test_experts_past_32_bit_offsets(moe):
    """More than 2^31 weights: the last expert's, and its gradient."""
    g = _gen(15)
    E, N, K = 260, 2048, 4096
    w = torch.empty(E, N, K, dtype=BF16, device="cuda")
    w[-1] = _ints(g, N, K)
    counts = [0] * (E - 1) + [33]
    x, dy = _ints(g, 33, K), _ints(g, 33, N)
    off = _offsets(counts)
    _same(moe.moe_grouped_gemm(x, off, w, y_fp32=True), x.double() @ w[-1].double().T, True)
    _same(moe.moe_grouped_gemm_dgrad(dy, off, w, dx_fp32=True), dy.double() @ w[-1].double(), True)
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw_fp32=False, out=w)
    _same(w[-1], dy.double().T @ x.double(), False)
    assert (w[:-1] == 0).all()


# ---------------------------------------------------------------------------- quantiser


def _quant_ref(v):
    """The formula in 32 bits on the CPU, each step rounded once."""
    rows, K = v.shape
    blk = torch.nn.functional.pad(v, (0, -K % 128)).view(rows, -1, 128)
    amax = blk.abs().amax(-1)
    s = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    q = (blk / s.unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :K].contiguous().view(torch.uint8), s


@pytest.mark.parametrize("rows,K", [(1, 16), (1, 128), (7, 144), (300, 2048), (33, 272), (1000, 1024)])
def test_quantise_matches_the_formula_bit_for_bit(moe, rows, K):
    g = torch.Generator().manual_seed(rows + K)
    x = torch.randn(rows, K, generator=g)
    x = (x * torch.exp2(torch.randint(-40, 40, (rows, 1), generator=g).float())).to(BF16)
    x[0, :16] = 0.0
    codes, scale = moe.moe_quantize_fp8(x.cuda())
    q, s = _quant_ref(x.float())
    assert torch.equal(scale.cpu(), s) and torch.equal(codes.cpu(), q)
    # strided rows
    wide = torch.full((rows, K + 24), float("nan"), dtype=BF16, device="cuda")
    wide[:, :K] = x.cuda()
    codes2, scale2 = moe.moe_quantize_fp8(wide[:, :K])
    assert torch.equal(codes, codes2) and torch.equal(scale, scale2)
    if K % 128 == 0:
        # the library's own decoder reads them back; it rounds scale * 2^120 to bf16, which holds scales
        # below 2^7 only, and then the product of the two: (1 + 2^-8)^2 - 1 = 2^-7 + 2^-16
        back = moe.moe_dequantize("fp8", codes, scale, 1.0, rows, K).float().cpu()
        want = q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, dim=1)
        held = (s < 2.0**7).repeat_interleave(128, dim=1)
        assert torch.allclose(back[held], want[held], rtol=2.0**-7 + 2.0**-16, atol=0)


def test_quantise_zeros_extremes_and_values_that_are_not_finite(moe):
    tiny = torch.finfo(BF16).tiny
    x = torch.zeros(6, 256, dtype=BF16)
    x[1, :128] = 2.0**-133            # the smallest bf16
    x[1, 128:] = tiny
    x[2, :128] = torch.finfo(BF16).max
    x[2, 128:] = 1.0
    x[3, 5] = float("nan")
    x[4, 200] = float("inf")
    x[5, 0], x[5, 1] = -3.0, 2.0**-60
    codes, scale = moe.moe_quantize_fp8(x.cuda())
    q, s = _quant_ref(x.float())
    fine = [0, 1, 2, 5]
    assert torch.equal(scale.cpu()[fine], s[fine]) and torch.equal(codes.cpu()[fine], q[fine])
    back = codes.cpu().view(torch.float8_e4m3fn).float() * scale.cpu().repeat_interleave(128, dim=1)
    assert torch.isnan(back[3, :128]).all() and (back[3, 128:] == 0).all()
    assert torch.isnan(back[4, 128:]).all() and (back[4, :128] == 0).all()


@pytest.mark.parametrize("rows,K", [(1, 16), (40, 768), (301, 272)])
def test_swiglu_quantise(moe, rows, K):
    """The scale is amax / 448 within 2^-20 (exp, the sum, the quotient and the product are a few units
    in the last place of fp32); a value is off by half a step of E4M3, 2^-4 of it, or half of the
    smallest step, 2^-10 of the scale."""
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(rows, 2 * K, generator=g) * 3).to(BF16)
    x[0, 0], x[0, K] = -90.0, 1.0
    x[0, 1], x[0, K + 1] = 60.0, 0.5
    if rows > 1:
        x[1, :K], x[1, K:] = -87.5, 3.0     # exp(87.5) is beyond 2^126: the block's values are tiny, not 0
    codes, scale = moe.moe_quantize_fp8(x.cuda(), swiglu=True)
    gate, up = x[:, :K].double(), x[:, K:].double()
    h = gate / (1 + torch.exp(-gate)) * up
    pad = torch.nn.functional.pad(h, (0, -K % 128)).view(rows, -1, 128)
    s = pad.abs().amax(-1) / 448.0
    assert ((scale.cpu().double() - s).abs() <= 2.0**-20 * s).all()
    full = scale.cpu().double().repeat_interleave(128, dim=1)[:, :K]
    back = codes.cpu().view(torch.float8_e4m3fn).double() * full
    assert ((back - h).abs() <= (2.0**-4 + 2.0**-20) * h.abs() + 2.0**-10 * full).all()


# ---------------------------------------------------------------------------- used together


def test_products_are_captured_and_replayed(moe):
    """A training step of one expert projection in a CUDA graph, replayed on new inputs, next to eager
    calls on another stream."""
    g = _gen(16)
    counts, K, N = [50, 0, 201, 9], 256, 384
    R, off = sum(counts), _offsets(counts)
    x, w, dy = _ints(g, R, K), _ints(g, 4, N, K), _ints(g, R, N)

    def step():
        return (moe.moe_grouped_gemm(x, off, w, y_fp32=True), moe.moe_grouped_gemm_dgrad(dy, off, w, dx_fp32=True),
                moe.moe_grouped_gemm_wgrad(dy, x, off), *moe.moe_quantize_fp8(x))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    side = torch.cuda.Stream()
    for i in range(3):
        x.copy_(_ints(g, R, K))
        dy.copy_(_ints(g, R, N))
        moved = [37, 100, 0, R - 137]
        off.copy_(_offsets(moved if i == 1 else counts))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            again = step()
        torch.cuda.synchronize()
        c = moved if i == 1 else counts
        _same(outs[0], _forward64(x, c, w), True)
        _same(outs[1], _dgrad64(dy, c, w), True)
        _same(outs[2], _wgrad64(dy, x, c), True)
        for a, b in zip(outs, again):
            assert torch.equal(a, b)


def test_gradients_agree_with_differences(moe):
    """The product is linear in x and in w, so differences along any direction are its derivative: with
    whole numbers, exactly."""
    g = _gen(17)
    counts, K, N = [20, 3, 0, 140], 136, 72
    R, off = sum(counts), _offsets(counts)
    x, w, dy = _ints(g, R, K, top=2), _ints(g, 4, N, K, top=2), _ints(g, R, N, top=2)
    d, v = _ints(g, R, K, top=1), _ints(g, 4, N, K, top=1)

    def loss(x, w):
        return (moe.moe_grouped_gemm(x, off, w, y_fp32=True).double() * dy.double()).sum()

    along_x = loss(x + d, w) - loss(x, w)
    along_w = loss(x, w + v) - loss(x, w)
    assert along_x == (moe.moe_grouped_gemm_dgrad(dy, off, w, dx_fp32=True).double() * d.double()).sum()
    assert along_w == (moe.moe_grouped_gemm_wgrad(dy, x, off).double() * v.double()).sum()


def _routed(moe, L, T, seed):
    x = synthetic.make_tokens(T, L.H, seed, device="cuda")
    idx, gate = moe.moe_route_topk(x, L.wr, L.k, bias=L.bias)
    off, sorted_pair, pair_row, xp = moe.moe_permute(idx, L.E, x, act="a4")
    return x, off, sorted_pair, pair_row, xp, gate


def test_an_expert_layer_is_trained_with_them(moe):
    """Route, permute, two products with a SwiGLU between them, combine; the gradients of both weights
    and of the rows against autograd in 64 bits on the same rows. bf16 is rounded to in y13, h, their
    gradients and dx: each at most 2^-8 of the value, a handful in a row, so 2e-2 of the largest."""
    cfg = dict(H=256, E=8, k=2, I=256, fmt="bf16", wr_fp32=True)
    L = synthetic.make_layer(cfg, 0, device="cuda")
    x, off, _, pair_row, xp, gate = _routed(moe, L, 77, 1)
    counts = (off[1:] - off[:-1]).tolist()
    g = _gen(18)
    dy = torch.randn(xp.shape[0], L.H, generator=g, device="cuda").to(BF16)

    y13 = moe.moe_grouped_gemm(xp, off, L.w13).requires_grad_()
    a, b = y13.float().chunk(2, dim=1)
    h = (torch.nn.functional.silu(a) * b).to(BF16)
    y = moe.moe_grouped_gemm(h.detach(), off, L.w2)
    out = moe.moe_combine(y, pair_row, gate)
    dh = moe.moe_grouped_gemm_dgrad(dy, off, L.w2)
    dw2 = moe.moe_grouped_gemm_wgrad(dy, h.detach(), off)
    (d13,) = torch.autograd.grad(h, y13, dh)
    dx = moe.moe_grouped_gemm_dgrad(d13, off, L.w13)
    dw13 = moe.moe_grouped_gemm_wgrad(d13, xp, off)

    x64 = xp.double().requires_grad_()
    w13, w2 = L.w13.double().requires_grad_(), L.w2.double().requires_grad_()
    parts = []
    for e, xs in enumerate(x64.split(counts)):
        a, b = (xs @ w13[e].T).chunk(2, dim=1)
        parts.append((torch.nn.functional.silu(a) * b) @ w2[e].T)
    y64 = torch.cat(parts)
    y64.backward(dy.double())
    want = torch.zeros(77, L.H, dtype=torch.float64, device="cuda")
    want.index_add_(0, torch.arange(77, device="cuda").repeat_interleave(L.k),
                    y64.detach()[pair_row.long()] * gate.flatten().double()[:, None])
    for got, ref in ((out, want), (y, y64), (dx, x64.grad), (dw13, w13.grad), (dw2, w2.grad)):
        assert rel_err(got.detach().cpu().double(), ref.detach().cpu()) < TOL


@pytest.mark.parametrize("T", [1, 4, 200])
def test_fp8_experts_are_served_on_fp8_activations(moe, T):
    """Route, permute, quantise, gate/up, SwiGLU and quantise, down, combine, against the layer's oracle,
    whose activations are not quantised. E4M3 leaves at most 2^-4 of a value, about 2^-5.8 in the root mean
    square over a binade (a uniform error of step 2^-3); x, h and their sums over hundreds of terms carry
    that as independent errors, so the outputs' root mean square is off by some 2 * 2^-5 of theirs."""
    cfg = dict(H=512, E=16, k=4, I=256, fmt="fp8", wr_fp32=False)
    L = synthetic.make_layer(cfg, 0)
    Ld = L.to("cuda")
    x, off, _, pair_row, xp, gate = _routed(moe, Ld, T, 2)
    xq, xs = moe.moe_quantize_fp8(xp)
    y13 = moe.moe_grouped_gemm_fp8(xq, xs, off, Ld.w13, Ld.w13_scale)
    hq, hs = moe.moe_quantize_fp8(y13, swiglu=True)
    y = moe.moe_grouped_gemm_fp8(hq, hs, off, Ld.w2, Ld.w2_scale, y_fp32=True)
    out = moe.moe_combine(y, pair_row, gate)
    ref = torch.from_numpy(oracle.layer_forward(x.cpu(), L)["out"]).double()
    err = (out.cpu().double() - ref).square().mean().sqrt() / ref.square().mean().sqrt()
    assert err < 2.0**-4
    # and exactly the formula on the codes: each product against 64 bits
    def full(q, s, K):
        return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, dim=-1)

    counts = (off[1:] - off[:-1]).tolist()
    want = _forward64(full(hq, hs, 256), counts, full(Ld.w2, Ld.w2_scale, 256))
    S = _forward64(full(hq, hs, 256).abs(), counts, full(Ld.w2, Ld.w2_scale, 256).abs())
    _within(y, want, 256, S, extra=3 * 2.0**-24)
