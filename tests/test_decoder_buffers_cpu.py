"""The decoder example's buffers for passes over many rows: how they grow and who shares them."""
import math
import random
from types import SimpleNamespace

import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from w4a4_quantized_gemm_gb300 import decoder

SIZES = dict(hidden=512, inner=640, heads=8, kv_heads=2, dim=64, rank=32)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()


def layer(**over):
    """What Buffers looks at in a layer, without weights."""
    s = SimpleNamespace(**{**SIZES, **over})
    shapes = dict(qkv=((s.heads + 2 * s.kv_heads) * s.dim, s.hidden), o=(s.hidden, s.heads * s.dim),
                  gate_up=(2 * s.inner, s.hidden), down=(s.hidden, s.inner))
    packed = {name: SimpleNamespace(N=n, K=k, r=s.rank, packed=torch.empty(0)) for name, (n, k) in shapes.items()}
    return SimpleNamespace(**packed, q_heads=s.heads, kv_heads=s.kv_heads, dim=s.dim, shape=tuple(sorted(vars(s).items())))


def check_held(l, buffers, largest):
    """Sets at least double, and the last has fewer than twice the rows of the largest pass unless that made it: their
    rows are at most 2 * 2 times the largest pass's, and the sets 2 + log2(largest).  (A workspace is no multiple of its rows:
    10 MB of it are the same for all above 32.)"""
    sets = [s for of_shape in buffers._sets.values() for s in of_shape]
    room = sum(t.numel() * t.element_size() for s in sets for t in (getattr(s, name) for name in decoder._ROWS))
    one = decoder.Buffers().rows(l, largest)
    assert room <= 4 * sum(getattr(one, name).numel() * 2 for name in decoder._ROWS)
    assert len(sets) <= 2 + math.log2(largest) and all(s.ws.numel() <= 2 * one.ws.numel() for s in sets)


@pytest.mark.parametrize("lengths", [range(1, 701), range(700, 0, -1), [2000, 2001, 1999, 2002, 2500], [1, 3000, 2, 5999, 6000]])
def test_lengths_do_not_add_up(lengths):
    """However many there are."""
    l, buffers = layer(), decoder.Buffers()
    for n in lengths:
        b = buffers.rows(l, n)
        assert b.qkv_out.shape == (n, 12 * 64) and b.attn.shape == (n, 8, 64) and b.h.shape == (n, 640)
        assert b.ws.numel() == max(w4.act_workspace_bytes(n, k, 32) for k in (512, 640)) and b.qkv_out.is_contiguous()
    check_held(l, buffers, max(lengths))


def test_many_lengths_in_any_order():
    rng, l, buffers = random.Random(1), layer(), decoder.Buffers()
    lengths = [rng.randint(1, 4000) for _ in range(500)]
    for n in lengths:
        buffers.rows(l, n)
    check_held(l, buffers, max(lengths))


def test_what_a_graph_may_hold_stays():
    l, buffers = layer(), decoder.Buffers()
    first = buffers.rows(l, 10)
    first.attn.fill_(3)
    where = first.attn.data_ptr()
    del first
    for n in (11, 40, 300):
        buffers.rows(l, n).attn.fill_(4)
    kept = [s.attn for s in buffers._sets[l.shape] if s.attn.data_ptr() == where]
    assert len(kept) == 1 and torch.all(kept[0] == 3)


def test_layers_of_the_same_shapes_share():
    a, b, other, buffers = layer(), layer(), layer(inner=1280), decoder.Buffers()
    where = buffers.rows(a, 100).h.data_ptr()
    assert buffers.rows(b, 70).h.data_ptr() == where and buffers.rows(other, 70).h.data_ptr() != where
    assert buffers.rows(other, 70).h.shape == (70, 1280)
    assert decoder.Buffers().rows(a, 100).h.data_ptr() != where
    q, k, v = buffers.rows(a, 33).split
    assert q.shape == (33, 8, 64) and k.shape == v.shape == (33, 2, 64)
    assert q.data_ptr() == buffers.rows(a, 33).qkv_out.data_ptr() and k.stride(0) == 12 * 64
