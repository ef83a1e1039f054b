"""Refusals of the block-scaled FP8 and few-token routed-expert entry points (no GPU: no call
here gets past argument validation, the pointers are fakes), and of their binding."""

import ctypes
import os

import pytest
import torch

from moe_nvfp4_quantize_amd import nvfp4 as B

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1001)
OFF4 = ctypes.c_void_p(0x1004)
INVALID = B.NVFP4_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libnvfp4.so not built (run __graft_entry__.build())")
    return B.load_library()


def test_block_quantize_rejects(lib):
    ok = dict(x=FAKE, t=B.NVFP4_BF16, rows=4, cols=32, ld=32, br=1, q=FAKE, s=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.nvfp4_fp8_block_quantize(a["x"], a["t"], a["rows"], a["cols"], a["ld"], a["br"], a["q"], a["s"], None)
    for bad in [dict(t=7), dict(rows=-1), dict(cols=0), dict(cols=24), dict(ld=16), dict(br=0), dict(br=64), dict(br=2),
                dict(x=None), dict(q=None), dict(s=None), dict(q=OFF4), dict(s=ODD), dict(x=ODD), dict(rows=2 ** 31),
                dict(rows=2 ** 30, cols=64, ld=64), dict(ld=2 ** 40)]:
        assert call(**bad) == INVALID, bad
    assert call(rows=0, x=None, q=None, s=None) == B.NVFP4_OK


def test_block_gemm_rejects(lib):
    ok = dict(aq=FAKE, as_=FAKE, bq=FAKE, bs=FAKE, M=4, N=8, K=64, c=FAKE, t=B.NVFP4_F32, ldc=8)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.nvfp4_fp8_block_gemm(a["aq"], a["as_"], a["bq"], a["bs"], a["M"], a["N"], a["K"], a["c"], a["t"],
                                        a["ldc"], None)
    for bad in [dict(K=24), dict(K=0), dict(M=-1), dict(N=-1), dict(ldc=4), dict(t=5), dict(aq=None), dict(as_=None),
                dict(bq=None), dict(bs=None), dict(c=None), dict(N=2 ** 31, ldc=2 ** 31), dict(aq=OFF4), dict(bq=OFF4),
                dict(as_=ODD), dict(bs=ODD), dict(c=ODD), dict(M=2 ** 31), dict(K=2 ** 31)]:
        assert call(**bad) == INVALID, bad
    assert call(M=0, aq=None, c=None) == B.NVFP4_OK
    assert call(N=0, ldc=0, bq=None, c=None) == B.NVFP4_OK


def test_moe_decode_rejects(lib):
    ok = dict(x=FAKE, t=B.NVFP4_BF16, ldx=64, lg=FAKE, T=4, E=8, k=2, H=64, I=32, gq=FAKE, gs=FAKE, gg=FAKE, dq=FAKE,
              ds=FAKE, dg=FAKE, o=FAKE, ot=B.NVFP4_F32, ldo=64, ws=FAKE, wsb=1 << 24)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.nvfp4_moe_decode(a["x"], a["t"], a["ldx"], a["lg"], a["T"], a["E"], a["k"], a["H"], a["I"], a["gq"],
                                    a["gs"], a["gg"], a["dq"], a["ds"], a["dg"], a["o"], a["ot"], a["ldo"], a["ws"],
                                    a["wsb"], None)
    for bad in [dict(t=3), dict(ot=3), dict(ldx=32), dict(ldo=32), dict(T=-1), dict(E=0), dict(E=1025), dict(k=0),
                dict(k=9), dict(E=64, k=33), dict(H=40, ldx=64), dict(H=0), dict(I=0), dict(I=24), dict(x=None),
                dict(lg=None), dict(gq=None), dict(gs=None), dict(gg=None), dict(dq=None), dict(ds=None), dict(dg=None),
                dict(o=None), dict(ws=None), dict(wsb=64), dict(ws=OFF4), dict(x=ODD), dict(o=ODD), dict(lg=ODD),
                dict(gg=ODD), dict(dg=ODD), dict(I=2 ** 21), dict(H=2 ** 21, ldx=2 ** 21, ldo=2 ** 21)]:
        assert call(**bad) == INVALID, bad
    assert call(T=129) == B.NVFP4_ERR_UNSUPPORTED
    assert call(T=0, x=None, lg=None, o=None, ws=None, wsb=0) == B.NVFP4_OK


def test_moe_decode_workspace_size(lib):
    f = lib.nvfp4_moe_decode_workspace_size
    assert f(0, 8, 2, 64, 32) >= 0
    # at least h in three bf16 planes, and growing with the tokens
    assert f(32, 512, 10, 4096, 1024) >= 3 * 320 * 1024 * 2
    assert f(1, 128, 8, 2048, 768) < f(2, 128, 8, 2048, 768)
    for bad in [(-1, 8, 2, 64, 32), (1, 8, 9, 64, 32), (1, 8, 2, 40, 32), (129, 8, 2, 64, 32)]:
        assert f(*bad) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="CPU tensors: what the binding refuses first")
def test_binding_refuses_cpu_tensors_and_bad_shapes(lib):
    u8, f32 = torch.uint8, torch.float32
    x = torch.zeros((4, 256))
    with pytest.raises(ValueError, match="GPU"):
        B.nvfp4_fp8_block_quantize(x)
    with pytest.raises(ValueError, match="block_rows"):
        B.nvfp4_fp8_block_quantize(x, block_rows=64)
    with pytest.raises(ValueError, match="2-D"):
        B.nvfp4_fp8_block_quantize(x[0])
    with pytest.raises(ValueError, match="unit stride"):
        B.nvfp4_fp8_block_quantize(x.t())
    with pytest.raises(TypeError):
        B.nvfp4_fp8_block_quantize(x.double())
    a = (torch.zeros((4, 256), dtype=u8), torch.zeros((4, 2)))
    b = (torch.zeros((300, 256), dtype=u8), torch.zeros((3, 2)))
    for bad in [((a[0][:, :240], a[1]), b), ((a[0], a[1][:, :1]), b), (a, (b[0], b[1][:2])), ((a[0].float(), a[1]), b),
                (a, (b[0], b[1].double())), (a, (b[0].t().contiguous().t(), b[1])), (a, b)]:
        with pytest.raises(ValueError):
            B.nvfp4_fp8_block_gemm(*bad)
    with pytest.raises(ValueError, match="out"):
        B.nvfp4_fp8_block_gemm(a, b, out=torch.zeros((4, 299)))
    T, E, H, I = 2, 3, 64, 32
    gu = (torch.zeros((E, 2 * I, H // 2), dtype=u8), torch.zeros((E, 2 * I, H // 16), dtype=u8), torch.ones(E))
    dn = (torch.zeros((E, H, I // 2), dtype=u8), torch.zeros((E, H, I // 16), dtype=u8), torch.ones(E))
    x, lg = torch.zeros((T, H)), torch.zeros((T, E))
    with pytest.raises(ValueError, match="GPU"):
        B.nvfp4_moe_decode(x, lg, 2, gu, dn)
    for bad in [(x[:, :48], lg, 2, gu, dn), (x, lg[:1], 2, gu, dn), (x, lg.double(), 2, gu, dn), (x, lg, 2, dn, dn),
                (x, lg, 2, gu, gu), (x, lg, 2, (gu[0], gu[1], gu[2][:1]), dn), (x, lg, 2, gu, (dn[0], dn[1][:, :32], dn[2])),
                (x, lg[:, :2], 2, gu, dn), (x[0], lg, 2, gu, dn)]:
        with pytest.raises(ValueError):
            B.nvfp4_moe_decode(*bad)
    with pytest.raises(ValueError, match="out"):
        B.nvfp4_moe_decode(x, lg, 2, gu, dn, out=torch.zeros((T, H + 16)))


def test_largest_sizes(lib):
    """Shapes whose launches would pass 2^32 threads are refused, whatever the card's memory."""
    q = lib.nvfp4_fp8_block_quantize
    assert q(FAKE, B.NVFP4_BF16, 2 ** 29, 16, 16, 1, FAKE, FAKE, None) == INVALID
    assert q(FAKE, B.NVFP4_BF16, 128, 2 ** 31 - 16, 2 ** 31, 128, FAKE, FAKE, None) == INVALID
    assert q(FAKE, B.NVFP4_BF16, 1, 2 ** 31 - 16, 2 ** 31, 128, FAKE, FAKE, None) == INVALID
    g = lib.nvfp4_fp8_block_gemm
    for M, N in ((2 ** 26, 1), (1, 2 ** 26), (2 ** 19, 2 ** 19), (2 ** 26 - 1, 2 ** 26 - 1)):
        assert g(FAKE, FAKE, FAKE, FAKE, M, N, 16, FAKE, B.NVFP4_F32, N, None) == INVALID, (M, N)
    f = lib.nvfp4_moe_decode_workspace_size
    assert f(1, 1024, 1, 2 ** 18, 16) == 0 and f(1, 1024, 1, 16, 2 ** 18) == 0 and f(1, 1023, 1, 2 ** 18, 16) > 0
