"""Which calls of the decoder-layer operators are refused on the host, by the memory that they would write
and the strides that they use; nothing is launched."""
import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.test_layer_ops_cpu import A, GOOD, L, append, attention, cache, norm  # noqa: F401 (L: a fixture)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="good calls would launch on a machine with a GPU")


@pytest.mark.parametrize("over", [dict(out_token_stride=0), dict(out_head_stride=0), dict(out_head_stride=64),
                                  dict(out_token_stride=120)])
def test_overlapping_outputs_are_refused(L, over):
    assert L.w4a4_kv_append(cache(), append(**over), None) == 1
    assert L.w4a4_paged_attention(cache(), attention(**over), None) == 1


@pytest.mark.parametrize("over", [{f"{p}_{d}_stride": s} for p in "kv" for d in ("page", "token", "head") for s in (0, 64)])
def test_append_refuses_pools_whose_rows_overlap(L, over):
    assert L.w4a4_kv_append(cache(**over), append(), None) == 1


def test_norm_in_place_with_another_stride_is_refused(L):
    assert L.w4a4_block_norm(norm(r_out_stride=2048), None) == 1


@no_gpu
def test_inputs_may_share_rows(L):
    for over in (dict(q_token_stride=0), dict(q_head_stride=0), dict(k_token_stride=0), dict(v_head_stride=0)):
        assert L.w4a4_kv_append(cache(), append(**over), None) == GOOD
    for over in (dict(k_page_stride=0), dict(v_token_stride=0), dict(k_head_stride=0)):
        assert L.w4a4_paged_attention(cache(**over), attention(), None) == GOOD
    assert L.w4a4_kv_append(cache(), append(q_heads=1, out_head_stride=0), None) == GOOD
    assert L.w4a4_kv_append(cache(), append(q_heads=0, q=0, q_out=0, out_token_stride=0), None) == GOOD
    assert L.w4a4_block_norm(norm(r_out=A + 4096, r_out_stride=2048), None) == GOOD
