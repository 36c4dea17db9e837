"""The training and FP8 products of the expert layer, as cases to measure.

Rows of x are (token, expert) pairs in expert order, as the permutation of the layer leaves them:
rows offsets[e] .. offsets[e+1]-1 belong to expert e. The operators:

  gemm    y[r] = w[e(r)] x[r]                 bf16 rows and weights w [E, N, K]
  dgrad   dx[r] = w[e(r)]^T dy[r]             its gradient for x
  wgrad   dw[e] = sum_r dy[r] x[r]^T          its gradient for w, over the rows of expert e
  quant   s = amax / 448 over each 128 of a row, codes E4M3(x / s); with swiglu the row is first
          silu(gate) * up of the two halves of the given row
  fp8     y[r, n] = sum_b xs[r, b] ws[e, n, b] sum_{i in block b} xq[r, i] wq[e, n, i], the blocks
          being 128 wide along K; without experts (E = 1) a plain matrix product

Each case has `op`, the tokens T, the experts E, the k experts that each token goes to, the sizes K
and N, the skew `zipf` of the experts' popularity (0: uniform) and `fp32`: whether the result is
stored in 32 bits.
"""
import math

import torch

own = False

BLOCK = 128
FP8_MAX = 448.0


def listed():
    return [
        # one token of a decode step through the gate/up weights of its 8 experts: latency and weight reads
        dict(name="gemm decode T=1", op="gemm", T=1, E=128, k=8, K=2048, N=1536, zipf=0.0, fp32=False),
        # a prompt of 4096 tokens, popular experts: gate/up products from a few to thousands of rows
        dict(name="gemm prefill T=4096", op="gemm", T=4096, E=128, k=8, K=2048, N=1536, zipf=1.1, fp32=False),
        # few wide experts with an odd number of rows: bound by the tensor cores
        dict(name="gemm few experts", op="gemm", T=4099, E=8, k=2, K=4096, N=4096, zipf=0.0, fp32=True),
        # the backward pass of the down projection over the same prompt
        dict(name="dgrad prefill T=4096", op="dgrad", T=4096, E=128, k=8, K=768, N=2048, zipf=1.1, fp32=False),
        # a short, ragged batch on sizes that no tile divides, gradients kept in 32 bits
        dict(name="dgrad ragged", op="dgrad", T=333, E=40, k=6, K=1000, N=1160, zipf=1.0, fp32=True),
        # weight gradients of the gate/up projection in 32 bits, as an optimiser sums them
        dict(name="wgrad prefill T=4096", op="wgrad", T=4096, E=128, k=8, K=2048, N=1536, zipf=1.1, fp32=True),
        # weight gradients of few wide experts in bf16: long sums over the rows
        dict(name="wgrad few experts", op="wgrad", T=8191, E=8, k=2, K=2048, N=4096, zipf=0.0, fp32=False),
        # the activations of the prompt's pairs on their way into the gate/up product
        dict(name="quant prefill", op="quant", T=4096, E=128, k=8, K=2048, N=0, zipf=0.0, fp32=False, swiglu=False),
        # the hidden rows of a decode batch of 64 tokens, gate and up in, E4M3 out
        dict(name="quant swiglu T=64", op="quant", T=64, E=128, k=8, K=768, N=0, zipf=0.0, fp32=False, swiglu=True),
        # a decode batch of 4 tokens on the FP8 experts of a streamed layer, outputs in 32 bits
        dict(name="fp8 decode T=4", op="fp8", T=4, E=128, k=8, K=2048, N=1536, zipf=0.0, fp32=True),
        # the prompt through FP8 gate/up weights
        dict(name="fp8 prefill T=4096", op="fp8", T=4096, E=128, k=8, K=2048, N=1536, zipf=1.1, fp32=False),
        # a plain FP8 product without experts: bound by the tensor cores
        dict(name="fp8 dense", op="fp8", T=8191, E=1, k=1, K=4096, N=4096, zipf=0.0, fp32=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    """One more case of the same ranges: one token to thousands, one expert to 256, sizes that need not fit a tile."""
    op = rng.choice(["gemm", "gemm", "dgrad", "wgrad", "quant", "fp8", "fp8"])
    E = 1 if op == "fp8" and rng.random() < 0.3 else _log(rng, 4, 256)
    k = min(E, rng.choice([1, 2, 6, 8]))
    T = _log(rng, 1, 8192)
    step = 16 if op in ("fp8", "quant") else 8
    K = rng.choice([256, 512, 768, 2048, 4096, _log(rng, 64, 4096, step), _log(rng, 64, 4096, step)])
    N = rng.choice([512, 768, 1536, 2048, 4096, _log(rng, 64, 4096, 8), _log(rng, 64, 4096, 8)])
    # no more weights and no more rows than the largest listed cases hold
    while E * K * N > 128 * 2048 * 1536:
        E = max(1, E // 2)
    k = min(k, E)
    while T * k > 32768 or T * k * K * N > 8191 * 2 * 2048 * 4096:
        T = max(1, T // 2)
    c = dict(op=op, T=T, E=E, k=k, K=K, N=N, zipf=rng.choice([0.0, 1.0, 1.1, 1.2]), fp32=rng.random() < 0.5)
    if op == "quant":
        c.update(N=0, swiglu=rng.random() < 0.5, fp32=False)
    return c


# ------------------------------------------------------------------------------- inputs


def _quantised_weights(w):
    """E4M3 codes and one fp32 scale per (row, 128 of K), as the FP8 experts are stored."""
    K = w.shape[-1]
    pad = -K % BLOCK
    blk = torch.nn.functional.pad(w, (0, pad)).unflatten(-1, (-1, BLOCK))
    amax = blk.abs().amax(-1)
    scale = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
    codes = (blk / scale.unsqueeze(-1)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).flatten(-2)[..., :K].contiguous(), scale.contiguous()


def prepare(case, seed):
    """Rows in expert order with their offsets, and the layer's weights, as the program that calls has them."""
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 9176 + 11)
    T, E, k, K, N = c["T"], c["E"], c["k"], c["K"], c["N"]
    rows = T * k
    s = dict(case=c, rows=rows, E=E)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16) * std

    if c["op"] == "quant":
        s["x"] = normal(rows, 2 * K if c["swiglu"] else K)
        return s
    # routing: each token takes k experts, drawn without replacement by popularity 1 / (rank + 1)^zipf
    rank = torch.randperm(E, generator=g, device=dev).float()
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=dev).clamp(1e-7, 1 - 1e-7)))
    idx = (noise - c["zipf"] * torch.log(rank + 1.0)).topk(k, dim=1).indices
    count = torch.bincount(idx.flatten(), minlength=E)
    s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
    s["most"] = int(count.max())
    if c["op"] == "fp8":
        s["wq"], s["ws"] = _quantised_weights(torch.randn(E, N, K, generator=g, device=dev) * 0.02)
        s["xq"], s["xs"] = _quantised_weights(torch.randn(rows, K, generator=g, device=dev))
        return s
    if c["op"] in ("gemm", "wgrad"):
        s["x"] = normal(rows, K)
    if c["op"] in ("dgrad", "wgrad"):
        s["dy"] = normal(rows, N)
    if c["op"] in ("gemm", "dgrad"):
        s["w"] = normal(E, N, K, std=0.02)
    return s


# ------------------------------------------------------------------------------- one pass


def run(state):
    c = state["case"]
    return _with_framework(state, c) if own else _plain(state, c)


def _with_framework(s, c):
    import expert_ffn_layer_top_b200 as moe

    if c["op"] == "gemm":
        return moe.moe_grouped_gemm(s["x"], s["offsets"], s["w"], y_fp32=c["fp32"])
    if c["op"] == "dgrad":
        return moe.moe_grouped_gemm_dgrad(s["dy"], s["offsets"], s["w"], dx_fp32=c["fp32"])
    if c["op"] == "wgrad":
        return moe.moe_grouped_gemm_wgrad(s["dy"], s["x"], s["offsets"], dw_fp32=c["fp32"])
    if c["op"] == "quant":
        codes, scale = moe.moe_quantize_fp8(s["x"], swiglu=c["swiglu"])
        return codes.view(torch.float8_e4m3fn), scale
    if c["E"] == 1:
        return moe.moe_grouped_gemm_fp8(s["xq"], s["xs"], None, s["wq"], s["ws"], y_fp32=c["fp32"])
    return moe.moe_grouped_gemm_fp8(s["xq"], s["xs"], s["offsets"], s["wq"], s["ws"], y_fp32=c["fp32"])


def _slots(s):
    """For each row its place (expert * most + position) in the rows padded to the largest expert."""
    r = torch.arange(s["rows"], device="cuda")
    e = torch.searchsorted(s["offsets"][1:].contiguous(), r.to(torch.int32), right=True)
    return e * s["most"] + r - s["offsets"][e]


def _padded(s, x):
    out = torch.zeros(s["E"] * s["most"], x.shape[1], device=x.device)
    out[_slots(s)] = x.float()
    return out.view(s["E"], s["most"], -1)


def _decoded(codes, scale):
    K = codes.shape[-1]
    return codes.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(BLOCK, dim=-1)[..., :K]


def _plain(s, c):
    store = torch.float32 if c["fp32"] else torch.bfloat16
    if c["op"] == "quant":
        x = s["x"].float()
        if c["swiglu"]:
            gate, up = x.chunk(2, dim=1)
            x = gate / (1.0 + torch.exp(-gate)) * up
        return _plain_quant(x)
    if c["op"] == "wgrad":
        return torch.bmm(_padded(s, s["dy"]).transpose(1, 2), _padded(s, s["x"])).to(store)
    if c["op"] == "fp8":
        y = torch.bmm(_padded(s, _decoded(s["xq"], s["xs"])), _decoded(s["wq"], s["ws"]).transpose(1, 2))
    elif c["op"] == "gemm":
        y = torch.bmm(_padded(s, s["x"]), s["w"].float().transpose(1, 2))
    else:
        y = torch.bmm(_padded(s, s["dy"]), s["w"].float())
    return y.flatten(0, 1)[_slots(s)].to(store)


def _plain_quant(x):
    rows, K = x.shape
    blk = torch.nn.functional.pad(x, (0, -K % BLOCK)).view(rows, -1, BLOCK)
    amax = blk.abs().amax(-1)
    scale = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
    codes = (blk / scale.unsqueeze(-1)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return codes.view(rows, -1)[:, :K].contiguous(), scale


# ------------------------------------------------------------------------------- what a pass has to do


def work(case):
    c = case
    rows, E, K, N = c["T"] * c["k"], c["E"], c["K"], c["N"]
    if c["op"] == "quant":
        read = rows * K * (4 if c["swiglu"] else 2)
        return {"bytes": read + rows * K + 4 * rows * -(-K // BLOCK), "flops": rows * K * (8 if c["swiglu"] else 3)}
    # experts that receive a row, as uniform routing would reach them
    used = min(E, max(1, round(E * (1 - (1 - c["k"] / E) ** c["T"]))))
    size = 4 if c["fp32"] else 2
    flops = 2.0 * rows * K * N
    if c["op"] == "wgrad":
        return {"bytes": 2 * rows * (K + N) + size * E * K * N, "flops": flops}
    if c["op"] == "fp8":
        per = 1 + 4.0 * -(-K // BLOCK) / K
        return {"bytes": per * (rows * K + used * K * N) + size * rows * N, "flops": flops}
    inner, outer = (K, N) if c["op"] == "gemm" else (N, K)
    return {"bytes": 2 * rows * inner + 2 * used * K * N + size * rows * outer, "flops": flops}


# ------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    """The formulas expert by expert in 64 bits, from the stored inputs."""
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "quant":
        return _exact_quant(s["x"].double(), c["swiglu"])
    edges = s["offsets"].tolist()
    if c["op"] == "fp8":
        out = torch.zeros(s["rows"], c["N"], dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            a, b = edges[e], edges[e + 1]
            for lo in range(0, c["K"], BLOCK):
                if a == b:
                    break
                hi, j = min(c["K"], lo + BLOCK), lo // BLOCK
                xb = s["xq"][a:b, lo:hi].contiguous().view(torch.float8_e4m3fn).double() * s["xs"][a:b, j : j + 1].double()
                wb = s["wq"][e, :, lo:hi].contiguous().view(torch.float8_e4m3fn).double() * s["ws"][e, :, j : j + 1].double()
                out[a:b] += xb @ wb.T
        return out
    if c["op"] == "wgrad":
        out = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            a, b = edges[e], edges[e + 1]
            out[e] = s["dy"][a:b].double().T @ s["x"][a:b].double()
        return out
    src = s["x"] if c["op"] == "gemm" else s["dy"]
    out = torch.zeros(s["rows"], c["N"] if c["op"] == "gemm" else c["K"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        a, b = edges[e], edges[e + 1]
        w = s["w"][e].double()
        out[a:b] = src[a:b].double() @ (w.T if c["op"] == "gemm" else w)
    return out


def _exact_quant(x, swiglu):
    if swiglu:
        half = x.shape[1] // 2
        gate = x[:, :half]
        x = gate * torch.sigmoid(gate) * x[:, half:]
    rows, K = x.shape
    scales, values = [], []
    for lo in range(0, K, BLOCK):
        v = x[:, lo : lo + BLOCK]
        top = v.abs().max(dim=1, keepdim=True).values
        step = torch.where(top > 0, top / FP8_MAX, torch.ones_like(top))
        q = v / step
        # E4M3: three bits after the leading one, the smallest normal 2^-6, ties to even
        unit = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0**-6))) - 3)
        values.append((torch.round(q / unit) * unit).clamp(-FP8_MAX, FP8_MAX))
        scales.append(step)
    return torch.cat(values, dim=1), torch.cat(scales, dim=1)
