"""GPU parity of the block-scaled FP8 quantize and GEMM against their oracle.

Quantized bytes and scales are bit-exact.  GEMM outputs lie within the oracle's bound on a
float32 evaluation, element by element; a bf16 output, whose products go through the FP8
matrix unit, within the bound that counts that unit's cuts, half a bf16 step (2^-8 relative
at most) further, and as a whole within half a bf16 step in norm (the cuts are 2^-16 there).
"""

import numpy as np
import pytest
import torch

from oracle import fp8_block as P
from moe_nvfp4_quantize_amd import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from moe_nvfp4_quantize_amd import nvfp4
    nvfp4.load_library()
    return nvfp4


def _host(t):
    return t.detach().float().cpu().numpy()


def _same(got, want, label):
    np.testing.assert_array_equal(got[1].cpu().numpy(), want[1], err_msg=str(label))
    np.testing.assert_array_equal(got[0].cpu().numpy(), want[0], err_msg=str(label))


def _uneven(rows, cols, seed, dtype):
    x = W.random_matrix(rows, cols, seed=seed, device="cuda") * torch.exp(
        2 * W.random_matrix(1, cols, seed=seed + 1, device="cuda"))
    return x.to(dtype)


# ------------------------------------------------------------------ quantize


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 5120), (3, 128), (127, 272), (128, 256), (129, 2064), (300, 144)])
def test_quantize_bit_exact(B, rows, cols, dtype, block_rows):
    x = _uneven(rows, cols, rows + cols, dtype)
    _same(B.nvfp4_fp8_block_quantize(x, block_rows), P.quantize(_host(x), block_rows), (rows, cols))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_midpoints(B, dtype):
    """Values that sit on midpoints of two codes of the real scale or one unit beside them, for
    block maxima whose scale is no float32; subnormal codes; signed zeros."""
    rng = np.random.default_rng(11)
    from oracle.formats import e4m3_decode
    mids = (e4m3_decode(np.arange(126)) + e4m3_decode(np.arange(1, 127))) / 2
    rows = []
    for amax in (1.0, 0.75, 1.5, 3.0, 5.5, 1e-3, 448.0, 447.0, 2.0 ** -70, 1.3 * 2.0 ** -118, 2.0 ** -130, 3e38):
        s = float(max(np.float32(amax) / np.float32(448.0), np.float32(2.0 ** -126)))
        near = np.float32(mids * s)
        for v in (near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(np.inf)),
                  np.float32(mids * (amax / 448.0))):
            row = np.zeros(128, np.float32)
            row[:126] = np.minimum(v, np.float32(amax)) * rng.choice([-1, 1], 126)
            row[126], row[127] = amax, -0.0
            rows.append(row)
    x = torch.from_numpy(np.stack(rows)).cuda().to(dtype)
    for br in (1, 128):
        _same(B.nvfp4_fp8_block_quantize(x, br), P.quantize(_host(x), br), br)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_strides_alignment_out(B, dtype):
    big = _uneven(140, 700, 5, dtype)
    for x in (big[:, :272], big[:, 3:275], big[::2, 1:401]):
        for br in (1, 128):
            q = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
            s = torch.empty((-(-x.shape[0] // br), -(-x.shape[1] // 128)), device="cuda")
            got = B.nvfp4_fp8_block_quantize(x, br, out=(q, s))
            assert got[0] is q and got[1] is s
            _same(got, P.quantize(_host(x), br), br)
    zero = torch.zeros((130, 144), dtype=dtype, device="cuda")
    q, s = B.nvfp4_fp8_block_quantize(zero, 128)
    assert torch.all(q == 0) and torch.all(s == 1)
    q, s = B.nvfp4_fp8_block_quantize(zero[:0])
    assert q.shape == (0, 144) and s.shape == (0, 2)


# ---------------------------------------------------------------------- GEMM


def _operands(M, N, K, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def codes(rows):
        return (torch.randn((rows, K), generator=g, device="cuda") * 120).clamp(-448, 448) \
            .to(torch.float8_e4m3fn).view(torch.uint8)

    def scales(rows):
        return torch.exp(torch.randn((rows, -(-K // 128)), generator=g, device="cuda")) * 0.01

    return (codes(M), scales(M)), (codes(N), scales(-(-N // 128)))


def _check(B, M, N, K, dtype, out=None, a=None, b=None, seed=0):
    a0, b0 = _operands(M, N, K, seed + M + N + K)
    a, b = a or a0, b or b0
    y = B.nvfp4_fp8_block_gemm(a, b, out_dtype=dtype, out=out)
    args = [t.cpu().numpy() for t in (*a, *b)]
    bf16 = dtype == torch.bfloat16
    ref, tol = P.gemm(*args), P.gemm_bound(*args, fp8_unit=bf16)
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y.double().cpu().numpy() - ref)
    worst = np.max(err / np.maximum(tol, 1e-300))
    rel = np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-300)
    print(f"[fp8 block gemm] {M}x{N}x{K} {dtype}: {worst:.3f} of the bound, rel {rel:.2e}", flush=True)
    assert worst <= 1.0, (M, N, K, worst)
    assert not bf16 or rel <= 2.0 ** -8, (M, N, K, rel)
    return y


SHAPES = [(1, 1, 16), (1, 512, 512), (2, 17, 144), (7, 130, 272), (16, 256, 5120), (17, 300, 1040), (33, 129, 128),
          (64, 640, 2048), (65, 1000, 640), (100, 96, 8192), (128, 384, 1024), (129, 257, 2064), (255, 520, 384),
          (256, 512, 1280), (300, 770, 1552), (513, 1030, 256)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(B, M, N, K, dtype):
    _check(B, M, N, K, dtype)


# Every tile that the launch chooses from (256 compute units): few tiles to many, each with rows and
# columns that end inside a tile and a K that ends inside a block
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(4, 100, 400), (5, 100, 400), (20, 19900, 272), (60, 5100, 400), (61, 19700, 272),
                                   (130, 4990, 400), (257, 6600, 272), (1150, 4500, 400), (64, 10000, 144)])
def test_gemm_every_tile(B, M, N, K, dtype):
    _check(B, M, N, K, dtype)


def test_gemm_long_k(B):
    """K past the tile kernels' 32-bit offsets (256 rows of 2^24 bytes)."""
    M, N, K = 6, 3, 2 ** 24 + 144
    a, b = _operands(M, N, K, 12)
    y = B.nvfp4_fp8_block_gemm(a, b, out_dtype=torch.float32)

    def values(t, rows):
        s = t[1].double().repeat_interleave(rows, 0)[:t[0].shape[0]]
        return t[0].view(torch.float8_e4m3fn).double() * s.repeat_interleave(128, 1)[:, :K]

    av, bv = values(a, 1), values(b, 128)
    ref = torch.stack([(av * row).sum(1) for row in bv], 1)
    tol = (128 + K // 128 + 4) * 2.0 ** -23 * torch.stack([(av * row).abs().sum(1) for row in bv], 1)
    assert torch.all((y.double() - ref).abs() <= tol)


@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_gemm_output_strides(B, M):
    """Rows of a wider buffer, at element alignment; what lies beside them stays."""
    N, K = 200, 384
    for dtype in (torch.bfloat16, torch.float32):
        for first, wide in ((0, 256), (1, 203), (3, 301)):
            buf = torch.full((M, wide + first), 7.0, dtype=dtype, device="cuda")
            _check(B, M, N, K, dtype, out=buf[:, first:first + N])
            assert torch.all(buf[:, :first] == 7) and torch.all(buf[:, first + N:] == 7)


@pytest.mark.parametrize("M", [3, 70, 260])
def test_gemm_zero_scales_and_codes(B, M):
    a, b = _operands(M, 260, 400, 9)
    a[1][:, 1] = 0
    a[0][M // 2] = 0
    b[1][1] = 0
    y = _check(B, M, 260, 400, torch.float32, a=a, b=b)
    assert torch.all(y[M // 2] == 0) and torch.all(y[:, 128:256] == 0)
    assert B.nvfp4_fp8_block_gemm((a[0][:0], a[1][:0]), b).shape == (0, 260)


@pytest.mark.parametrize("M,N,K", [(1, 200, 5120), (32, 640, 2064), (90, 300, 1024), (300, 600, 1024)])
def test_gemm_same_bits_every_time(B, M, N, K):
    a, b = _operands(M, N, K, 1)
    y = B.nvfp4_fp8_block_gemm(a, b, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(y, B.nvfp4_fp8_block_gemm(a, b, out_dtype=torch.float32))


@pytest.mark.parametrize("M", [1, 48, 150])
def test_quantize_then_gemm_graph_and_stream(B, M):
    """The two as a linear layer, on a side stream and captured: replays on rewritten inputs with
    eager work between equal the eager result."""
    K, N = 1280, 390
    w = B.nvfp4_fp8_block_quantize(_uneven(N, K, 4, torch.bfloat16), 128)
    x = _uneven(M, K, 6, torch.bfloat16)
    q = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((M, K // 128), device="cuda")
    y = torch.empty((M, N), device="cuda")

    def layer(stream=None):
        B.nvfp4_fp8_block_quantize(x, out=(q, s), stream=stream)
        return B.nvfp4_fp8_block_gemm((q, s), w, out=y, stream=stream)

    want = layer().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    layer(side)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for i in range(3):
        x.copy_(_uneven(M, K, 60 + i, torch.bfloat16))
        want = layer().clone()
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


@pytest.mark.parametrize("M", [3, 40, 140])
def test_rows_without_numbers_stay_their_own(B, M):
    """Padding rows of a batch that hold NaN or infinity: NaN rows of C, the others' bits as without."""
    K, N = 640, 300
    w = B.nvfp4_fp8_block_quantize(_uneven(N, K, 4, torch.bfloat16), 128)
    x = _uneven(M, K, 6, torch.bfloat16)
    for dt in (torch.bfloat16, torch.float32):
        want = B.nvfp4_fp8_block_gemm(B.nvfp4_fp8_block_quantize(x), w, out_dtype=dt)
        bad = x.clone()
        bad[1, 5] = float("nan")
        bad[M - 1] = float("inf")
        got = B.nvfp4_fp8_block_gemm(B.nvfp4_fp8_block_quantize(bad), w, out_dtype=dt)
        assert torch.isnan(got[1]).all() and torch.isnan(got[M - 1]).all()
        rest = [r for r in range(M) if r not in (1, M - 1)]
        assert torch.equal(got[rest], want[rest])


def test_inputs_freed_behind_a_call_on_another_stream(B):
    """Memory of inputs dropped after a call on a given stream is not handed out before its
    kernels have run: the call waits behind other work while the caller frees and fills."""
    M, K, N = 64, 1280, 390
    x0 = _uneven(M, K, 6, torch.bfloat16)
    w = B.nvfp4_fp8_block_quantize(_uneven(N, K, 4, torch.bfloat16), 128)
    a0 = B.nvfp4_fp8_block_quantize(x0)
    want = B.nvfp4_fp8_block_gemm(a0, w)
    side = torch.cuda.Stream()
    x, a = x0.clone(), tuple(t.clone() for t in a0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    q, s = B.nvfp4_fp8_block_quantize(x, stream=side)
    y = B.nvfp4_fp8_block_gemm(a, w, stream=side)
    del x, a
    fill = [torch.full_like(t, 1) for t in (x0, *a0)]
    side.synchronize()
    assert torch.equal(q, a0[0]) and torch.equal(s, a0[1]) and torch.equal(y, want)
    assert all(torch.all(t == 1) for t in fill)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 4896, 2048), (1, 4897, 2064), (1, 4850, 2064), (4, 4865, 144), (4, 4864, 144),
                                   (3, 4900, 5136), (1, 20000, 16)])
def test_gemm_few_rows_both_kernels(B, M, N, K, dtype):
    """Both sides of the rule for up to four rows."""
    _check(B, M, N, K, dtype)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_offsets_past_32_bits(B, block_rows):
    """4.3e9 elements: the last rows are what those rows alone give."""
    rows, cols = 2 ** 21, 2064
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[:] = torch.arange(cols, device="cuda")
    tail = slice(rows - 256, rows)
    x[tail] = _uneven(256, cols, 3, torch.bfloat16)
    q, s = B.nvfp4_fp8_block_quantize(x, block_rows)
    want = B.nvfp4_fp8_block_quantize(x[tail], block_rows)
    assert torch.equal(q[tail], want[0]) and torch.equal(s[-256 // block_rows:], want[1])
    assert torch.equal(q[:128], q[128 * 1000:128 * 1001])


@pytest.mark.parametrize("M", [1, 3, 40, 130])
def test_gemm_offsets_past_32_bits(B, M):
    """B of more than 2^32 bytes, and (130 rows) a C that reaches past 2^32 bytes: the last columns."""
    N, K = 2 ** 25, 144
    a, _ = _operands(M, 128, K, M)
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    bq = torch.randint(0, 0x7F, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    bs = torch.rand((N // 128, 2), generator=g, device="cuda")
    y = B.nvfp4_fp8_block_gemm(a, (bq, bs), out_dtype=torch.bfloat16)
    for c0 in (0, N - 384):
        args = [t.cpu().numpy() for t in (*a, bq[c0:c0 + 384], bs[c0 // 128:c0 // 128 + 3])]
        ref, tol = P.gemm(*args), P.gemm_bound(*args, fp8_unit=True)
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert np.all(np.abs(y[:, c0:c0 + 384].double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("M", [5, 70])
def test_gemm_long_rows_offsets(B, M):
    """Rows so long that few of them pass 2^32 bytes, on both sides of where the tiles' offsets end."""
    for N, K in ((300, 2 ** 24 - 16), (260, 2 ** 24 + 16)):
        a, b = _operands(M, 128, 256, M)
        aq = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
        bq = torch.zeros((N, K), dtype=torch.uint8, device="cuda")
        kb = -(-K // 128)
        as_ = torch.ones((M, kb), device="cuda")
        bs = torch.ones((-(-N // 128), kb), device="cuda")
        g = torch.Generator(device="cuda")
        g.manual_seed(N)
        cols = torch.tensor([0, 16, 4096, K // 2, K - 16], device="cuda")[:, None] + torch.arange(16, device="cuda")
        cols = cols.reshape(-1)
        aq[:, cols] = torch.randint(0, 0x7F, (M, cols.numel()), generator=g, device="cuda", dtype=torch.uint8)
        bq[:, cols] = torch.randint(0, 0x7F, (N, cols.numel()), generator=g, device="cuda", dtype=torch.uint8)
        y = B.nvfp4_fp8_block_gemm((aq, as_), (bq, bs), out_dtype=torch.float32)
        # unit scales: the same product over the 80 columns that hold anything.  Adding zeros is exact,
        # so an output rounds at most 32 + 5 + 5 + 3 times (codes of a block, blocks, waves, scales),
        # fewer than the 80 + 1 + 3 that the bound of the dense product counts
        small = [aq[:, cols].cpu().numpy(), np.ones((M, 1), np.float32), bq[:, cols].cpu().numpy(),
                 np.ones((-(-N // 128), 1), np.float32)]
        ref, tol = P.gemm(*small), P.gemm_bound(*small)
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol)
        del aq, bq, as_, bs
