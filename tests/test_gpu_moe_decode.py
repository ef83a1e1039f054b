"""GPU parity of the few-token routed-expert layer against its oracle.

Every output lies within the bound that the oracle carries through the layer for a float32
evaluation (h as one f16 value for bf16 outputs, x and h as two otherwise; a bf16 x is exact),
plus half a bf16 step (2^-8 relative at most) where the output is bf16.  Routing is the routed call's own, so a wrong expert or weight
shows as a gross error.
"""

import numpy as np
import pytest
import torch

from oracle import moe_decode as OD
from moe_nvfp4_quantize_amd import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from moe_nvfp4_quantize_amd import nvfp4
    nvfp4.load_library()
    return nvfp4


def _weights(E, rows, cols, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(1, 0x7F, (E, rows, cols // 16), generator=g, device="cuda", dtype=torch.uint8)
    return q, s, (torch.rand(E, generator=g, device="cuda") + 0.5) * 2.0 ** -14


def _case(T, E, k, H, I, seed=0):
    seed = seed + T + E + k + H + I
    return (W.random_matrix(T, H, seed=seed, device="cuda"), W.random_matrix(T, E, seed=seed + 1, device="cuda"), k,
            _weights(E, 2 * I, H, seed + 2), _weights(E, H, I, seed + 3))


def _check(y, x, logits, k, gu, dn):
    bf16 = y.dtype == torch.bfloat16
    ref, tol = OD.forward(x.float().cpu().numpy(), logits.cpu().numpy(), k, [t.cpu().numpy() for t in gu],
                          [t.cpu().numpy() for t in dn], x_bits=None if x.dtype == torch.bfloat16 else 22,
                          h_bits=11 if bf16 else 22)
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y.double().cpu().numpy() - ref)
    worst = np.max(err / np.maximum(tol, 1e-300)) if err.size else 0.0
    rel = np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-300)
    print(f"[moe decode] {tuple(y.shape)} {y.dtype}: {worst:.3f} of the bound, rel {rel:.2e}", flush=True)
    assert worst <= 1.0, worst


SHAPES = [(1, 1, 1, 16, 16), (1, 8, 2, 256, 128), (1, 128, 8, 1024, 384), (2, 5, 3, 48, 80), (4, 512, 10, 320, 256),
          (5, 16, 4, 528, 144), (8, 3, 3, 512, 192), (9, 40, 7, 784, 400), (16, 4, 2, 256, 320), (17, 2, 1, 128, 64),
          (33, 6, 3, 272, 176), (64, 1024, 32, 64, 64), (65, 8, 2, 192, 128), (100, 24, 5, 208, 112),
          (128, 3, 2, 320, 64), (128, 64, 32, 64, 64)]


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k,H,I", SHAPES)
def test_layer(B, T, E, k, H, I, x_dtype, out_dtype):
    x, logits, k, gu, dn = _case(T, E, k, H, I)
    x = x.to(x_dtype)
    _check(B.nvfp4_moe_decode(x, logits, k, gu, dn, out_dtype=out_dtype), x, logits, k, gu, dn)


@pytest.mark.parametrize("T", [1, 3, 20])
def test_strides_and_alignment(B, T):
    """Rows of wider buffers at element alignment; weights whose bases are off 16 bytes; what
    lies beside the output stays."""
    E, k, H, I = 6, 2, 128, 64
    x0, logits, k, gu, dn = _case(T, E, k, H, I, 3)

    def off(t, n):
        buf = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
        buf[n:] = t.reshape(-1)
        return buf[n:].view(t.shape)

    for x_dtype in (torch.bfloat16, torch.float32):
        for first, wide in ((0, 160), (3, 161)):
            xb = torch.zeros((T, wide), dtype=x_dtype, device="cuda")
            x = xb[:, first:first + H]
            x.copy_(x0)
            ob = torch.full((T, wide + 1), 9.0, dtype=x_dtype, device="cuda")
            for n in (0, 1, 4, 8):
                gun = (off(gu[0], n), off(gu[1], n), gu[2])
                dnn = (off(dn[0], n), off(dn[1], n), dn[2])
                _check(B.nvfp4_moe_decode(x, logits, k, gun, dnn, out=ob[:, first:first + H]), x, logits, k, gu, dn)
            assert torch.all(ob[:, :first] == 9) and torch.all(ob[:, first + H:] == 9)


def test_ties_extremes_and_shared_experts(B):
    T, E, k, H, I = 12, 9, 4, 128, 96
    x, logits, k, gu, dn = _case(T, E, k, H, I, 5)
    logits[0] = 0.0                       # all equal: experts 0 .. k-1
    logits[1] = torch.arange(E, device="cuda").float() % 2
    logits[2] = -1e30
    logits[2, 3] = 1e30                   # one weight 1, the others 0
    logits[3:9] = logits[3]               # the same experts for six tokens
    logits[9, 4] = float("-inf")
    logits[10, :] = torch.tensor([3.4e38, -3.4e38] * 4 + [0.0], device="cuda")
    x[11] = 0.0
    x[4] *= 1e4
    x[5] *= 1e-12
    x[6, ::3] *= 1e-9                     # small beside the row's largest
    x[7] *= 1e-30
    for dt in (torch.bfloat16, torch.float32):
        y = B.nvfp4_moe_decode(x.to(dt), logits, k, gu, dn, out_dtype=torch.float32)
        _check(y, x.to(dt), logits, k, gu, dn)
        assert torch.all(y[11] == 0)


def test_matches_the_routed_layer(B):
    """Beside moe_layer, which quantizes x and h to 4 bits: the two agree to what that costs
    (E2M1 steps, at most 1/6 of a block's maximum: well under half in norm)."""
    x, logits, k, gu, dn = _case(16, 8, 2, 256, 128, 8)
    a = B.nvfp4_moe_decode(x, logits, k, gu, dn, out_dtype=torch.float32)
    b = B.moe_layer(x, logits, k, gu, dn).float()
    assert (a - b).norm() < 0.5 * b.norm()


def test_same_bits_every_time_and_empty(B):
    x, logits, k, gu, dn = _case(24, 10, 4, 256, 128, 2)
    y = B.nvfp4_moe_decode(x, logits, k, gu, dn, out_dtype=torch.float32)
    for _ in range(4):
        assert torch.equal(y, B.nvfp4_moe_decode(x, logits, k, gu, dn, out_dtype=torch.float32))
    # a token's result does not depend on how many others share the call
    for t in (0, 7, 23):
        one = B.nvfp4_moe_decode(x[t:t + 1], logits[t:t + 1], k, gu, dn, out_dtype=torch.float32)
        _check(one, x[t:t + 1], logits[t:t + 1], k, gu, dn)
    assert B.nvfp4_moe_decode(x[:0], logits[:0], k, gu, dn).shape == (0, 256)


@pytest.mark.parametrize("T", [1, 4, 30])
def test_graph_and_stream(B, T):
    E, k, H, I = 16, 3, 256, 128
    x, logits, k, gu, dn = _case(T, E, k, H, I, 4)
    x = x.to(torch.bfloat16)
    y = torch.empty((T, H), device="cuda")
    want = B.nvfp4_moe_decode(x, logits, k, gu, dn, out=y).clone()
    side = torch.cuda.Stream()
    y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    B.nvfp4_moe_decode(x, logits, k, gu, dn, out=y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.nvfp4_moe_decode(x, logits, k, gu, dn, out=y)
    for i in range(3):
        x.copy_(W.random_matrix(T, H, seed=70 + i, device="cuda"))
        logits.copy_(W.random_matrix(T, E, seed=80 + i, device="cuda"))
        want = B.nvfp4_moe_decode(x, logits, k, gu, dn, out_dtype=torch.float32)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_decode_step(B):
    """The operators as a decode step uses them: a block-scaled FP8 projection, the router's logits
    from the same product with a float32 result, the routed experts on both."""
    T, K, H, E, k, I = 6, 384, 256, 16, 4, 128
    x = W.random_matrix(T, K, seed=1, dtype=torch.bfloat16, device="cuda")
    wp = B.nvfp4_fp8_block_quantize(W.random_matrix(H, K, seed=2, device="cuda", std=0.05), 128)
    wr = B.nvfp4_fp8_block_quantize(W.random_matrix(E, H, seed=3, device="cuda", std=0.05), 128)
    gu, dn = _weights(E, 2 * I, H, 4), _weights(E, H, I, 5)
    hid = B.nvfp4_fp8_block_gemm(B.nvfp4_fp8_block_quantize(x), wp)
    logits = B.nvfp4_fp8_block_gemm(B.nvfp4_fp8_block_quantize(hid), wr, out_dtype=torch.float32)
    y = B.nvfp4_moe_decode(hid, logits, k, gu, dn)
    # each stage against its oracle, given the stage's own input
    from oracle import fp8_block as P
    for a, w, got in ((x, wp, hid), (hid, wr, logits)):
        aq = P.quantize(a.float().cpu().numpy())
        wq = [t.cpu().numpy() for t in w]
        ref, tol = P.gemm(*aq, *wq), P.gemm_bound(*aq, *wq, fp8_unit=got.dtype == torch.bfloat16)
        if got.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)
    _check(y, hid, logits, k, gu, dn)


@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (24, 40, 3), (100, 6, 2)])
def test_tokens_without_numbers_stay_their_own(B, T, E, k):
    """Padding tokens: NaN or infinity in x, a row of logits that a mask left nothing of.  Their own
    rows are not numbers, the others' bits are as when the padding routes the same way."""
    x, logits, k, gu, dn = _case(T, E, k, 128, 80, 6)
    for dt in (torch.bfloat16, torch.float32):
        want = B.nvfp4_moe_decode(x.to(dt), logits, k, gu, dn, out_dtype=dt)
        bad, lg = x.to(dt), logits.clone()
        bad = bad.clone()
        bad[0, 7] = float("nan")
        bad[1] = float("inf")
        lg[2] = float("-inf")
        got = B.nvfp4_moe_decode(bad, lg, k, gu, dn, out_dtype=dt)
        assert not torch.isfinite(got[:3]).any()
        if T > 3:
            # token 2's experts change where its slots stand, never what others' columns hold
            err = (got[3:].double() - want[3:].double()).abs().max()
            assert torch.equal(got[3:], want[3:]), err


def test_calls_at_once_on_two_streams(B):
    """Two layers in flight together, each on a stream of its own, inputs freed behind them."""
    cases = [_case(20, 16, 3, 256, 128, 4), _case(40, 12, 2, 256, 192, 5)]
    want = [B.nvfp4_moe_decode(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for st, c in zip(streams * 4, cases * 4):
        st.wait_stream(torch.cuda.current_stream())
        x = c[0].clone()
        st.wait_stream(torch.cuda.current_stream())
        got.append(B.nvfp4_moe_decode(x, *c[1:], stream=st))
        del x
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2]), i


def test_one_expert_for_a_whole_batch(B):
    """Every token of the largest batch on the same experts (several passes over its columns)."""
    for T, E, k in ((128, 64, 1), (128, 2, 2), (16, 64, 1), (17, 300, 1)):
        x, logits, k, gu, dn = _case(T, E, k, 192, 80, 9)
        logits[:] = 0.0
        logits[:, E - 1] = 5.0
        _check(B.nvfp4_moe_decode(x, logits, k, gu, dn, out_dtype=torch.float32), x, logits, k, gu, dn)


@pytest.mark.parametrize("T", [1, 20])
def test_offsets_past_32_bits(B, T):
    """1024 experts whose codes pass 2^32 bytes, the last ones routed to: as with those alone."""
    E, k, H, I = 1024, 2, 2048, 2112
    gu, dn = _weights(E, 2 * I, H, 4), _weights(E, H, I, 5)
    assert gu[0].numel() > 2 ** 32
    x = W.random_matrix(T, H, seed=1, dtype=torch.bfloat16, device="cuda")
    logits = torch.full((T, E), -50.0, device="cuda")
    logits[:, -5:] = W.random_matrix(T, 5, seed=2, device="cuda")
    last = [tuple(t[-5:].contiguous() for t in w) for w in (gu, dn)]
    y = B.nvfp4_moe_decode(x, logits, k, gu, dn, out_dtype=torch.float32)
    _check(y, x, logits[:, -5:], k, *last)


def test_captured_on_a_given_stream(B):
    """A capture whose calls name its stream: replays with eager work on the default stream
    between them equal the eager result."""
    x, logits, k, gu, dn = _case(9, 16, 3, 256, 128, 4)
    y = torch.empty((9, 256), device="cuda")
    side = torch.cuda.Stream()
    w = B.nvfp4_fp8_block_quantize(W.random_matrix(300, 256, seed=5, device="cuda"), 128)
    z = torch.empty((9, 300), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.nvfp4_moe_decode(x, logits, k, gu, dn, out=y, stream=side)
        B.nvfp4_fp8_block_gemm(B.nvfp4_fp8_block_quantize(y, stream=side), w, out=z, stream=side)
    for i in range(3):
        x.copy_(W.random_matrix(9, 256, seed=70 + i, device="cuda"))
        want = B.nvfp4_moe_decode(x, logits, k, gu, dn, out_dtype=torch.float32)
        want_z = B.nvfp4_fp8_block_gemm(B.nvfp4_fp8_block_quantize(want), w, out_dtype=torch.float32)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want_z), i
