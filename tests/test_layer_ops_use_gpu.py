"""The cache, attention and norm operators as a server uses them: workspaces shared and dropped, host threads,
streams, devices, strides that no index uses; and values at the borders of their types.

References and tolerances as in test_layer_ops_gpu."""
import math
import threading

import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.test_layer_ops_gpu import (BF16, E4M3, F16, F64, SLACK, Cache, attend, attention_ref, check, check_attention, gen,
                                      randn, tiny, u)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()
    w4.w4a4_device_status()


def test_attention_one_workspace_for_calls_of_all_shapes():
    """A buffer that is large enough and was zeroed once serves any sequence of calls: split sequences of one
    batch, a larger batch whose late sequence goes over more than sixteen CTAs, other head dimensions."""
    shapes = [([5000], 8, 2, 128), ([1] * 8 + [40000] + [1] * 55, 8, 2, 128), ([700] * 3, 16, 1, 64), ([3000, 9], 2, 9, 96),
              ([9000], 1, 8, 256), ([2] * 30 + [30000], 4, 1, 64)]
    size = lambda lengths, hkv, group, dim: w4.lib().w4a4_paged_attention_workspace_bytes(len(lengths), hkv * group, hkv, dim)
    ws = torch.zeros(max(size(*s) for s in shapes), dtype=torch.uint8, device="cuda")
    calls = []
    for i, (lengths, hkv, group, dim) in enumerate(shapes):
        c = Cache(lengths, 16, hkv, dim, F16, seed=40 + i)
        q = randn(gen(50 + i), len(lengths), hkv * group, dim).to(F16)
        want, _ = check_attention(c, q, lengths, what=f"shape {i}")
        calls.append((c, q.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), want))
    for turn in range(2):
        for i, (c, q, n, want) in enumerate(calls):
            out = torch.full_like(q, float("nan"))
            w4.w4a4_paged_attention(q, c.handle, n, out, workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(out.view(torch.int16), want.view(torch.int16)), (turn, i)
    assert w4.w4a4_device_status() == 0


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
def test_attention_rows_without_weight_are_zero_whatever_the_values(dtype):
    """Every score -inf: out = 0 and lse = -inf, with infinities and NaN among the values."""
    lengths = [40, 3000]
    c = Cache(lengths, 16, 2, 64, F16 if dtype == E4M3 else dtype, seed=65)
    act = BF16 if dtype == BF16 else F16
    q = randn(gen(66), 2, 4, 64).abs().to(act)
    if dtype == E4M3:  # E4M3 has no infinity: the query brings it
        c = Cache(lengths, 16, 2, 64, E4M3, seed=65, scales=False)
        c.k[..., 0] = torch.full_like(c.k[..., 0].float(), -1.0).to(E4M3)
        q[..., 0] = math.inf
    else:
        c.k[..., 0] = -math.inf
    v = c.v.float()
    v[c.table[0, 1].long(), 3, 0, 5] = float("nan")
    v[c.table[1, 100].long(), 7, 1, 6] = math.inf if dtype != E4M3 else float("nan")
    c.v = v.to(c.dtype)
    c.to_gpu()
    out, lse = attend(c, q, lengths)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)


@pytest.mark.parametrize("dtype, act", [(F16, F16), (BF16, BF16), (E4M3, F16)])
@pytest.mark.parametrize("below", [12, 18, 26])
def test_attention_many_small_weights_beside_a_large_one(dtype, act, below):
    """One token takes nearly all the weight and has zero values, as a first token often does; the others, each
    w = 2^(-1.03 below) of it, make the output: out = n w / (1 + n w) where their values are one.

    Each weight is rounded once to the matrix instruction's type, the output once."""
    tokens, dim, seqs = 8192, 64, 512  # more sequences than CTAs: whole sequences to a CTA
    page = 64
    k = torch.zeros(tokens // page, page, 1, dim)
    v = torch.ones_like(k)
    k[0, 0, 0, 0], v[0, 0] = float(below), 0.0
    table = torch.arange(tokens // page, dtype=torch.int32).repeat(seqs, 1).cuda()  # all read the same pages
    handle = w4.PagedKVCache(k.to(dtype).cuda(), v.to(dtype).cuda(), table)
    q = torch.zeros(seqs, 2, dim)
    q[..., 0] = 1.0
    n = torch.full((seqs,), tokens, dtype=torch.int32, device="cuda")
    out = torch.empty(seqs, 2, dim, dtype=act, device="cuda")
    w4.w4a4_paged_attention(q.to(act).cuda(), handle, n, out, scale=1.03 * math.log(2.0))
    torch.cuda.synchronize()
    mass = (tokens - 1) * 2.0 ** (-1.03 * below)
    ref = torch.full(out.shape, mass / (1 + mass), dtype=F64)
    p_type = BF16 if dtype == BF16 else F16
    err = ref * (u(p_type) + 64 * SLACK)
    check(out, ref, err + u(act) * (ref + err) + tiny(act), f"{dtype} 2^-{below}")


def test_attention_infinite_bf16_query_beside_large_elements():
    """An infinite element of a bf16 query against an 8-bit cache: the score is an infinity of its sign, also with
    other elements outside fp16's range."""
    lengths = [50]
    c = Cache(lengths, 16, 1, 64, E4M3, seed=67, scales=False)
    k = c.k.float()
    k[..., 0], k[..., 1] = -1.0, 1.0
    c.k = k.to(E4M3)
    c.to_gpu()
    q = torch.ones(1, 2, 64)
    q[..., 0], q[..., 1] = math.inf, 1e6
    out, lse = attend(c, q.to(BF16), lengths)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
