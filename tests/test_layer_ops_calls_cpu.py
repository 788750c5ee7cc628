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


ODD = (0, 3, -5, 1 << 40)


@no_gpu
@pytest.mark.parametrize("odd", ODD)
def test_strides_that_no_index_uses_are_not_looked_at(L, odd):
    one = dict(tokens=1, q_token_stride=odd, k_token_stride=odd, v_token_stride=odd, out_token_stride=odd)
    assert L.w4a4_kv_append(cache(), append(**one), None) == GOOD
    assert L.w4a4_kv_append(cache(), append(**{**one, "q_out": A}), None) == GOOD  # in place: no stride differs
    assert L.w4a4_kv_append(cache(), append(q_heads=1, q_head_stride=odd, out_head_stride=odd), None) == GOOD
    single = dict(kv_heads=1, k_head_stride=odd, v_head_stride=odd)
    assert L.w4a4_kv_append(cache(**single), append(k_head_stride=odd, v_head_stride=odd), None) == GOOD
    assert L.w4a4_paged_attention(cache(**single), attention(), None) == GOOD
    for over in (dict(pages=1, k_page_stride=odd, v_page_stride=odd), dict(page_size=1, k_token_stride=odd, v_token_stride=odd),
                 dict(seqs=1, table_stride=odd)):
        assert L.w4a4_kv_append(cache(**over), append(), None) == GOOD
        assert L.w4a4_paged_attention(cache(**over), attention(), None) == GOOD
    row = dict(q_token_stride=odd, out_token_stride=odd)
    assert L.w4a4_paged_attention(cache(seqs=1), attention(**row), None) == GOOD
    assert L.w4a4_paged_attention(cache(**single), attention(q_heads=1, q_head_stride=odd, out_head_stride=odd), None) == GOOD
    row = dict(rows=1, y_stride=odd, r_stride=odd, r_out_stride=odd, x_stride=odd)
    assert L.w4a4_block_norm(norm(**row), None) == GOOD
    assert L.w4a4_block_norm(norm(gate=A, gate_stride=odd), None) == GOOD
    assert L.w4a4_block_norm(norm(gate=A, gate_stride=odd, rows_per_gate=4), None) == GOOD


@pytest.mark.parametrize("odd", ODD)
def test_strides_that_an_index_uses_are(L, odd):
    assert L.w4a4_kv_append(cache(), append(tokens=2, out_token_stride=odd), None) in (1, 3)
    assert L.w4a4_paged_attention(cache(seqs=2), attention(out_token_stride=odd), None) in (1, 3)
    assert L.w4a4_paged_attention(cache(seqs=2, table_stride=odd), attention(), None) == 1
    assert L.w4a4_block_norm(norm(rows=2, y_stride=odd), None) in (1, 3)
    assert L.w4a4_block_norm(norm(gate=A, gate_stride=odd, rows_per_gate=3), None) in (1, 3)
