"""Chunk attention whose keys and values say which of them counted: one-hot rows by their number in the sequence, so
that an output's elements are the weights of the keys, over work that goes through the rings of shared memory
many times on every SM."""
import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.test_layer_ops_gpu import BF16, E4M3, F16
from tests.test_prompt_ops_gpu import fresh, ints, starts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()
    w4.w4a4_device_status()


@pytest.mark.parametrize("dtype, act", [(E4M3, BF16), (E4M3, F16), (BF16, BF16)])
@pytest.mark.parametrize("dim, page", [(256, 16), (128, 16), (96, 32), (64, 8), (256, 24)])
def test_every_key_counts_in_every_call(dtype, act, dim, page):
    rows, lengths, heads = [500, 300, 300, 3], [600, 305, 700, 703], 80
    need = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(3))
    table = torch.zeros(4, max(need), dtype=torch.int32)
    pool = torch.zeros(sum(need), page, 1, dim)
    for b, (n, count) in enumerate(zip(lengths, need)):
        table[b, :count] = order[sum(need[:b]):sum(need[:b + 1])]
        t = torch.arange(n)
        pool[table[b, t // page].long(), t % page, 0, t % dim] = 1.0
    pool = pool.cuda().to(dtype).view(torch.uint8).expand(-1, -1, heads, -1).contiguous().view(dtype)
    handle = w4.PagedKVCache(pool, pool.clone(), table.cuda())
    starts = starts_of(rows)
    score = ((torch.arange(dim) % 7 - 3) / 2).to(act)  # of a key by its number; exact in every type
    q = score.expand(starts[-1], heads, dim).contiguous().cuda()
    out_ref, lse_ref = torch.zeros(starts[-1], dim, dtype=torch.float64), torch.zeros(starts[-1], dtype=torch.float64)
    for b, n in enumerate(lengths):
        for i in range(rows[b]):
            w = score.double()[torch.arange(n - rows[b] + i + 1) % dim].exp()
            lse_ref[starts[b] + i] = w.sum().log()
            out_ref[starts[b] + i].index_add_(0, torch.arange(len(w)) % dim, w / w.sum())
    out_ref, lse_ref = out_ref.cuda()[:, None], lse_ref.cuda()[:, None]
    # a probability and the output, rounded once each (2^-8 or 2^-11 of themselves), and 2^-12 for fp32 sums;
    # at the least weight of one key lost in 703, e^-1.5 of some 1300, lse would be off by 1.7e-4
    u = torch.finfo(act).eps / 2
    got = [fresh(q) for _ in range(30)]
    for out, lse in got:
        w4.w4a4_chunk_attention(q, handle, ints(starts), ints(lengths), out, lse=lse, scale=1.0)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0
    for i, (out, lse) in enumerate(got):
        assert ((lse.double() - lse_ref).abs() <= 2.0 ** -18 * (4 + lse_ref)).all(), i
        assert ((out.double() - out_ref).abs() <= (2 * u + 2.0 ** -12) * out_ref).all(), i
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1]), i
