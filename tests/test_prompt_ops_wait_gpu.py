"""The prompt and chunk attention's waits are bounded: a call whose limit is shorter than a unit of its work ends with
W4A4_ERR_TIMEOUT once its own copies and products have ended, and the calls after it are right."""
import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.test_layer_ops_gpu import BF16, E4M3, F16, Cache, gen, randn
from tests.test_prompt_ops_gpu import check_chunk, check_prompt, ints, qkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()
    w4.w4a4_device_status()


def runs_out(call):
    """`call` under a limit of a nanosecond: a wait is looked at some 20 us after it began, and a unit takes longer.
    With 20 us more for each tile, a tenth of which it takes, the same wait does not run out."""
    for tile_ns, status in ((0, w4.W4A4_ERR_TIMEOUT), (20000, 0)):
        w4.lib().w4a4_debug_prompt_wait_ns(1, tile_ns)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            w4.lib().w4a4_debug_prompt_wait_ns(0, 0)
        assert w4.w4a4_device_status() == status
        assert w4.w4a4_device_status() == 0  # read and cleared


@pytest.mark.parametrize("dtype, dim, hq, hkv", [(F16, 128, 32, 8), (BF16, 64, 16, 16), (F16, 256, 12, 4), (BF16, 96, 40, 8)])
def test_prompt_wait_runs_out(dtype, dim, hq, hkv):
    """12 heads for 4 and 40 for 8: queries without a tensor map."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((12000, h, dim), generator=g, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    out = torch.empty_like(q)
    runs_out(lambda: w4.w4a4_prompt_attention(q, k, v, ints([0, 12000]), out, causal=False))
    check_prompt(*qkv(3, 300, hq, hkv, dim, dtype), [0, 140, 300], what="after a call that gave up")


@pytest.mark.parametrize("dtype, act, dim, page", [(F16, F16, 128, 16), (E4M3, BF16, 128, 16), (E4M3, F16, 64, 32), (BF16, BF16, 256, 24),
                                                   (F16, F16, 128, 7), (E4M3, F16, 96, 5)])
def test_chunk_wait_runs_out(dtype, act, dim, page):
    """Pages of 7 and 5: keys without tensor maps."""
    c = Cache([300], page, 4, dim, dtype, seed=2)
    far = Cache([40000], page, 4, dim, dtype, seed=2, fill=False)
    q = torch.randn((9000, 8, dim), device="cuda").to(act)
    out = torch.empty_like(q)
    runs_out(lambda: w4.w4a4_chunk_attention(q, far.handle, ints([0, 9000]), ints([40000]), out))
    check_chunk(c, randn(gen(3), 40, 8, dim).to(act), [0, 40], [300], what="after a call that gave up")


def test_one_long_unit_a_cta():
    """D = 256: half of the softmax's warps have no tiles and wait for the others' through the whole unit."""
    far = Cache([40000], 16, 2, 256, F16, seed=2, fill=False)
    q = torch.randn((9000, 2, 256), device="cuda").to(F16)
    out = torch.empty_like(q)
    runs_out(lambda: w4.w4a4_chunk_attention(q, far.handle, ints([0, 9000]), ints([40000]), out))
