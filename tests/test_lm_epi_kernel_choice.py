"""Which forward kernel og_gemm_nt_epi takes, seen by its workspace (the kernel of few rows needs none), on a host
without a GPU; and results on both sides of the choice."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref

SIXTEEN = [og.BF16, og.F16]


@pytest.mark.parametrize("type", SIXTEEN)
@pytest.mark.parametrize("m,n,k", [(4096, 4096, 16), (2048, 2048, 32), (65536, 64, 64), (1024, 4096, 8), (1, 65536, 100),
                                   (16, 58422, 136), (1 << 24, 16, 1)])
def test_many_thin_blocks_are_tiles(m, n, k, type):
    assert og.gemm_nt_epi_workspace(m, n, k, type) > 0


@pytest.mark.parametrize("m,n,k", [(4096, 4096, 16), (2048, 2048, 32), (1024, 4096, 8)])
def test_many_thin_blocks_are_tiles_in_fp32(m, n, k):
    assert og.gemm_nt_epi_workspace(m, n, k, og.F32) > 0


@pytest.mark.parametrize("type,m,n,k", [(t, *s) for t in SIXTEEN for s in (
    (1, 11008, 4096), (16, 4096, 11008), (1, 32768, 4096), (16, 65536, 512), (1, 1, 1), (16, 16384, 8), (128, 1531, 1000),
    (1000, 128, 1000), (12000, 7, 9))] + [(og.F32, *s) for s in (
        (1, 11008, 4096), (64, 65536, 16), (64, 11008, 4096), (65536, 64, 64), (1024, 1024, 128), (128, 1531, 1000))])
def test_few_rows_and_little_weights_are_not(type, m, n, k):
    assert og.gemm_nt_epi_workspace(m, n, k, type) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("m,n,k", [(1040, 1030, 9), (512, 520, 16), (4100, 64, 24), (5000, 17, 33), (16, 16400, 500),
                                   (16, 16400, 520), (3, 20001, 31), (65, 16385, 8)])
def test_thin_products(m, n, k, dtype):
    import torch as th
    gen = th.Generator().manual_seed(m + n + k)
    kind = getattr(th, dtype)
    a, w, bias = (th.randn(s, generator=gen).to(kind).cuda() for s in ((m, k), (n, k), (n,)))
    print(f"gemm_nt_epi thin {m}x{n}x{k} {dtype}", flush=True)
    out, pre = og.gemm_nt_epi(a, w, bias=bias, act="silu", need_pre=True)
    e = ref.gemm_epi(a, w, bias, "silu", None)
    assert ((out.double() - e["c"]).abs() <= e["e_c"]).all()
    assert ((pre.double() - e["pre"]).abs() <= e["e_pre"]).all()
