"""The linear layers of a decode step and of a prefill: block-scaled FP8 quantize and
matrix product, and the routed-expert layer for few tokens.

``run`` computes each operator in plain torch operations (float32, or float64 where a
code is decided), or, with ``own`` set, calls the library's binding.

Sizes: 5120 -> 25600 and its 8192 tokens, the 2048 -> 151936 lm_head with 128 tokens,
and the 128-expert top-8 (H 2048, I 768) and 512-expert top-10 (H 4096, I 1024) layers
are the workloads of ``moe_nvfp4_quantize_amd/workloads.py``; the rest is generic.
"""

import math

import torch

own = False

BLOCK = 128       # columns of one FP8 scale block
E4M3_MAX = 448.0
# E2M1 magnitudes of codes 0..7; bit 3 of a code is the sign
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's hidden state before its projection: a call that is all latency
        dict(name="quantize 1x5120 bf16", op="quantize", rows=1, cols=5120, block_rows=1, dtype="bf16"),
        # a prefill's activations, one scale per token and 128 channels
        dict(name="quantize 8192x5120 bf16", op="quantize", rows=8192, cols=5120, block_rows=1, dtype="bf16"),
        # a weight quantized when a checkpoint is loaded, one scale per 128 x 128 tile
        dict(name="quantize 25600x5120 tiles", op="quantize", rows=25600, cols=5120, block_rows=128, dtype="bf16"),
        # one sequence's token through a square projection
        dict(name="gemm 1x5120x5120", op="gemm", M=1, N=5120, K=5120, out="bf16"),
        # a decode batch through the widest projection
        dict(name="gemm 32x25600x5120", op="gemm", M=32, N=25600, K=5120, out="bf16"),
        # a batch's logits
        dict(name="gemm 128x151936x2048", op="gemm", M=128, N=151936, K=2048, out="bf16"),
        # odd sizes: no dimension is a multiple of a tile, the last scale block is short
        dict(name="gemm 1000x1552x2064 f32", op="gemm", M=1000, N=1552, K=2064, out="f32"),
        # a prefill through the widest projection
        dict(name="gemm 8192x25600x5120", op="gemm", M=8192, N=25600, K=5120, out="bf16"),
        # one sequence's token through a layer of 128 experts
        dict(name="moe T1 E128 k8", op="moe", T=1, E=128, k=8, H=2048, I=768, dtype="bf16"),
        # a few sequences through a layer of 512 experts
        dict(name="moe T4 E512 k10", op="moe", T=4, E=512, k=10, H=4096, I=1024, dtype="bf16"),
        # odd sizes, float32 activations, several tokens on every expert
        dict(name="moe T37 E24 k5 f32", op="moe", T=37, E=24, k=5, H=2064, I=784, dtype="f32"),
        # a decode batch over which most experts are read
        dict(name="moe T32 E512 k10", op="moe", T=32, E=512, k=10, H=4096, I=1024, dtype="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, even over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm", "moe", "moe"))
    if op == "quantize":
        cols = _log(rng, 256, 8192, 16)
        return dict(op=op, rows=_log(rng, 1, min(25600, 131072000 // cols)), cols=cols,
                    block_rows=rng.choice((1, 1, 128)), dtype=rng.choice(("bf16", "f32")))
    if op == "gemm":
        K = _log(rng, 512, 8192, 16)
        N = _log(rng, 256, 32768)
        M = rng.choice((_log(rng, 1, 64), _log(rng, 1, 8192)))
        return dict(op=op, M=min(M, (8192 * 25600 * 5120) // (N * K)), N=N, K=K, out=rng.choice(("bf16", "f32")))
    E = _log(rng, 8, 512)
    k = rng.randint(1, min(10, E))
    T = _log(rng, 1, min(128, 320 // k))
    return dict(op=op, T=T, E=E, k=k, H=_log(rng, 512, 4096, 16), I=_log(rng, 256, 1024, 16),
                dtype=rng.choice(("bf16", "f32")))


def _torch_dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _blocks(n):
    return -(-n // BLOCK)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dev = "cuda"

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def fp8(rows, cols):
        # codes of normal values under their block's maximum: the largest of 128 is about 2.6 sigma
        return (normal(rows, cols) * (E4M3_MAX / 2.6)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)

    def nvfp4(e, rows, cols):
        # codes of normal values over their block's maximum are close to uniform; block scales
        # sit below the largest (448), the global scale is that of weights of sigma 0.02
        q = torch.randint(0, 256, (e, rows, cols // 2), generator=gen, device=dev, dtype=torch.uint8)
        s = torch.randint(0x68, 0x7D, (e, rows, cols // 16), generator=gen, device=dev, dtype=torch.uint8)
        g = (torch.rand(e, generator=gen, device=dev) + 0.5) * (0.1 / 2688)
        return q, s, g

    if case["op"] == "quantize":
        # channels of unequal size, as the hidden states of a trained model have them
        x = normal(case["rows"], case["cols"]) * torch.exp(normal(case["cols"]))
        state = dict(case, x=x.to(_torch_dtype(case["dtype"])))
    elif case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        a = (fp8(M, K), torch.exp(normal(M, _blocks(K)) * 0.5) * 0.01)
        b = (fp8(N, K), torch.exp(normal(_blocks(N), _blocks(K)) * 0.5) * 0.0002)
        state = dict(case, a=a, b=b)
    else:
        T, E, H, I = case["T"], case["E"], case["H"], case["I"]
        state = dict(case, logits=normal(T, E), x=normal(T, H).to(_torch_dtype(case["dtype"])),
                     w_gate_up=nvfp4(E, 2 * I, H), w_down=nvfp4(E, H, I))
    return state


# ------------------------------------------------------------ the plain forms


def _plain_quantize(x, block_rows):
    rows, cols = x.shape
    rb = -(-rows // block_rows)
    # whole blocks: the rows and columns that are missing count as zeros
    w = torch.zeros((rb * block_rows, _blocks(cols) * BLOCK), dtype=torch.float32, device=x.device)
    w[:rows, :cols] = x
    w = w.view(rb, block_rows, -1, BLOCK)
    amax = w.abs().amax(dim=(1, 3))
    s = (amax.double() / E4M3_MAX).float().clamp(min=2.0 ** -126)
    s = torch.where(amax == 0, torch.ones_like(s), s)
    # the code nearest the quotient: 64 bits, since a quotient rounded to 32 may land on a tie
    y = (w.double() / s.double()[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    step = torch.exp2((torch.frexp(y).exponent - 1).clamp(min=-6).double() - 3)
    v = torch.round(y / step) * step
    return v.reshape(rb * block_rows, -1)[:rows, :cols].float().to(torch.float8_e4m3fn).contiguous(), s


def _plain_gemm(a, b, dtype):
    def values(q, s, rows):
        cols = q.shape[1]
        s = s.repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(BLOCK, 1)[:, :cols]
        return q.view(torch.float8_e4m3fn).float() * s

    return (values(*a, 1) @ values(*b, BLOCK).t()).to(dtype)


def _plain_moe(x, logits, k, w_gate_up, w_down):
    T, H = x.shape
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=x.device)
    pairs = torch.stack((table.repeat(16), table.repeat_interleave(16)), 1)  # byte -> (low, high) nibble

    def product(w, experts, v):
        q, s, g = w
        m = pairs[q[experts].int()].view(experts.numel(), q.shape[1], -1, 16)
        m = m * s[experts].view(torch.float8_e4m3fn).float().unsqueeze(-1)
        return (m.flatten(2) @ v.unsqueeze(-1)).squeeze(-1) * g[experts, None]

    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)  # equal logits: lower id first
    top, ids = top[:, :k], ids[:, :k].reshape(-1)
    p = torch.exp(top - top[:, :1])
    p = p / p.sum(1, keepdim=True)
    gate, up = product(w_gate_up, ids, x.float().repeat_interleave(k, 0)).chunk(2, 1)
    y = product(w_down, ids, gate / (1 + torch.exp(-gate)) * up)
    return (p.unsqueeze(-1) * y.view(T, k, H)).sum(1).to(x.dtype)


def run(state):
    op = state["op"]
    if own:
        from moe_nvfp4_quantize_amd import nvfp4 as F
        if op == "quantize":
            q, s = F.nvfp4_fp8_block_quantize(state["x"], block_rows=state["block_rows"])
            return q.view(torch.float8_e4m3fn), s
        if op == "gemm":
            return F.nvfp4_fp8_block_gemm(state["a"], state["b"], out_dtype=_torch_dtype(state["out"]))
        return F.nvfp4_moe_decode(state["x"], state["logits"], state["k"], state["w_gate_up"], state["w_down"],
                                  out_dtype=state["x"].dtype)
    if op == "quantize":
        return _plain_quantize(state["x"], state["block_rows"])
    if op == "gemm":
        return _plain_gemm(state["a"], state["b"], _torch_dtype(state["out"]))
    return _plain_moe(state["x"], state["logits"], state["k"], state["w_gate_up"], state["w_down"])


# ------------------------------------------------------------ what a pass cannot do without


def work(case):
    if case["op"] == "quantize":
        n, es = case["rows"] * case["cols"], 4 if case["dtype"] == "f32" else 2
        scales = -(-case["rows"] // case["block_rows"]) * _blocks(case["cols"])
        return {"bytes": n * es + n + 4 * scales, "flops": 4 * n}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        scales = _blocks(K) * (M + _blocks(N))
        return {"bytes": M * K + N * K + 4 * scales + M * N * (4 if case["out"] == "f32" else 2), "flops": 2 * M * N * K}
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    es = 4 if case["dtype"] == "f32" else 2
    active = E * (1 - (1 - k / E) ** T)  # experts that at least one token is expected to pick
    return {"bytes": active * (3 * H * I * 9 / 16 + 8) + T * (2 * H * es + 4 * E), "flops": 6 * T * k * H * I}


# ------------------------------------------------------------ the definitions in 64 bits


def _exact_quantize(x, block_rows):
    x = x.double()
    rows, cols = x.shape
    grid = torch.tensor([0.0] + [m * 2.0 ** -9 for m in range(1, 8)]
                        + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=x.device)  # the 127 finite magnitudes, by code
    values, scales = torch.empty_like(x), []
    for r in range(0, rows, 4096 if block_rows == 1 else block_rows):
        part = x[r:r + (4096 if block_rows == 1 else block_rows)]
        line = []
        for c in range(0, cols, BLOCK):
            b = part[:, c:c + BLOCK]
            top = b.abs().amax().view(1, 1) if block_rows > 1 else b.abs().amax(1, keepdim=True)
            s = torch.where(top == 0, 1.0, (top / E4M3_MAX).float().clamp(min=2.0 ** -126).double())
            y = (b.abs() / s).clamp(max=E4M3_MAX).contiguous()
            hi = torch.searchsorted(grid, y).clamp(max=126)  # grid[hi - 1] < y <= grid[hi]
            lo = (hi - 1).clamp(min=0)
            up, down = grid[hi] - y, y - grid[lo]
            code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            values[r:r + b.shape[0], c:c + BLOCK] = torch.copysign(grid[code], b)
            line.append(s)
        scales.append(torch.cat(line, 1))
    return values, torch.cat(scales, 0)


def _exact_gemm(a, b):
    (aq, sa), (bq, sb) = a, b
    out = 0
    for j in range(sa.shape[1]):
        cut = slice(j * BLOCK, (j + 1) * BLOCK)
        at = aq[:, cut].view(torch.float8_e4m3fn).double() * sa[:, j:j + 1].double()
        bt = bq[:, cut].view(torch.float8_e4m3fn).double() * sb.double()[:, j].repeat_interleave(BLOCK)[:bq.shape[0], None]
        out = out + at @ bt.t().contiguous()
    return out


def _exact_moe(x, logits, k, w_gate_up, w_down):
    def weight(w, e):
        q, s, g = (t[e] for t in w)
        code = torch.stack((q & 15, q >> 4), -1).flatten(1).double()
        m = code % 8
        mag = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
        mag = torch.where(code >= 8, -mag, mag)
        exponent, mantissa = (s.double() / 8).floor(), s.double() % 8
        scale = torch.where(exponent == 0, mantissa * 2.0 ** -9, (1 + mantissa / 8) * torch.exp2(exponent - 7))
        return mag * scale.repeat_interleave(16, 1) * g.double()

    lg = logits.cpu().tolist()
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    picked = {}
    for t, row in enumerate(lg):
        best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        p = [math.exp(row[e] - row[best[0]]) for e in best]
        for e, v in zip(best, p):
            picked.setdefault(e, []).append((t, v / math.fsum(p)))
    for e, hits in picked.items():
        tokens = [t for t, _ in hits]
        p = torch.tensor([v for _, v in hits], dtype=torch.float64, device=x.device)
        z = x[tokens].double() @ weight(w_gate_up, e).t().contiguous()
        gate, up = z.chunk(2, 1)
        y = (gate * torch.sigmoid(gate) * up) @ weight(w_down, e).t().contiguous()
        out[tokens] += p[:, None] * y
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantize(state["x"], case["block_rows"])
    if case["op"] == "gemm":
        return _exact_gemm(state["a"], state["b"])
    return _exact_moe(state["x"], state["logits"], case["k"], state["w_gate_up"], state["w_down"])
