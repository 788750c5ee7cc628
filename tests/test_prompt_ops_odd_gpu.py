"""Corners of the prompt and chunk attention: rows, keys and values that are no numbers or lie at the
borders of their types, in units that are whole and in units that are split along the keys.

References and tolerances as in test_prompt_ops_gpu."""
import math

import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.test_layer_ops_gpu import BF16, E4M3, F16, F64, Cache, check, gen, randn
from tests.test_prompt_ops_gpu import check_chunk, check_prompt, fresh, ints, rows_ref, starts_of

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()
    w4.w4a4_device_status()


def put(cache, b, tokens, head, pool, value):
    """Sets rows `tokens` of sequence b of a pool of `cache` (a function of the rows as they are, or a number)."""
    tokens = torch.as_tensor(tokens)
    page, slot = cache.table[b, tokens // cache.page].long(), tokens % cache.page
    x = pool.float()
    x[page, slot, head] = value(x[page, slot, head]) if callable(value) else value
    pool.copy_(x.to(pool.dtype))


# A row of few over a long cache is split into parts of four tiles or more; 256 rows of a short one are not.
SPLIT = [("split", [5, 3], [6000, 3000]), ("whole", [5, 3], [900, 300])]


@pytest.mark.parametrize("dtype, act, dim", [(F16, F16, 128), (BF16, BF16, 64), (E4M3, BF16, 128), (F16, F16, 256)])
@pytest.mark.parametrize("how, rows, lengths", SPLIT)
def test_chunk_rows_whose_scores_are_nan(dtype, act, dim, how, rows, lengths):
    """A query that is NaN, or a cache whose scale of a head is: the row is NaN and so is its lse, however many parts
    its keys are shared out into."""
    c = Cache(lengths, 16, 2, dim, dtype, seed=21)
    q = randn(gen(22), sum(rows), 4, dim).to(act)
    q[1, 0, 3], q[6, 3, 0] = NAN, NAN
    out, lse = check_chunk(c, q, starts_of(rows), lengths, what=f"{how} query")
    assert torch.isnan(out[1, 0]).all() and torch.isnan(lse[1, 0]) and torch.isfinite(out[1, 1:]).all()
    if dtype == E4M3:
        c.ks[1] = NAN
        c.to_gpu()
        out, lse = check_chunk(c, q, starts_of(rows), lengths, what=f"{how} scale")
        assert torch.isnan(out[:, 2:]).all() and torch.isnan(lse[:, 2:]).all()


@pytest.mark.parametrize("dtype, act, dim", [(F16, F16, 128), (BF16, BF16, 64), (E4M3, F16, 64), (BF16, BF16, 256)])
@pytest.mark.parametrize("lo, hi", [(0, 1024), (0, 512), (2048, 4096), (5888, 5995)])
def test_chunk_parts_whose_keys_are_all_nan(dtype, act, dim, lo, hi):
    """A part of a row's keys without one number among its scores."""
    lengths, rows = [6000, 3000], [5, 3]
    c = Cache(lengths, 16, 2, dim, dtype, seed=23)
    put(c, 0, range(lo, hi), 0, c.k, NAN)
    c.to_gpu()
    q = randn(gen(24), 8, 4, dim).to(act)
    out, lse = check_chunk(c, q, starts_of(rows), lengths, what=f"keys {lo} to {hi}")
    assert torch.isnan(out[:5, :2]).all() and torch.isfinite(out[:5, 2:]).all() and torch.isfinite(lse[5:]).all()


@pytest.mark.parametrize("heads, rows, length", [(160, 300, 200), (160, 200, 97), (1, 300, 200), (80, 140, 3)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 50, 100, 1])
def test_chunk_longer_than_its_cache_with_a_window(heads, rows, length, window):
    """Rows before token 0 beside rows that see all tokens, in units of 256 rows (many heads) and of 128."""
    c = Cache([length], 16, heads, 64, F16, seed=27)
    q = randn(gen(28), rows, heads, 64).to(F16)
    out, lse = check_chunk(c, q, [0, rows], [length], window=window, what=f"{heads} heads, window {window}")
    assert torch.all(out[:rows - length] == 0) and torch.isfinite(lse[rows - length:]).all()


@pytest.mark.parametrize("dtype, act, dim", [(F16, F16, 128), (BF16, BF16, 64), (E4M3, BF16, 128), (F16, F16, 256)])
@pytest.mark.parametrize("lengths", [[6000], [900]])
def test_chunk_a_value_that_is_seen_counts_whatever_its_weight(dtype, act, dim, lengths):
    """NaN in a value whose key's weight is far below the smallest number, in another part (or another stream's
    tile) than the keys with weight: the output is NaN, as the sum that it stands for."""
    c = Cache(lengths, 16, 1, dim, dtype, seed=25, scales=False)
    n = lengths[0]
    for at, x in ((range(n), -40.0), (range(650, 760), 40.0)):
        put(c, 0, at, 0, c.k, lambda rows: torch.cat((torch.full_like(rows[..., :1], x), rows[..., 1:]), -1))
    put(c, 0, [3], 0, c.v, lambda rows: torch.cat((torch.full_like(rows[..., :1], NAN), rows[..., 1:]), -1))
    c.to_gpu()
    q = randn(gen(26), 4, 2, dim).to(act) / 8
    q[..., 0] = 4.0
    out, lse = check_chunk(c, q, [0, 4], lengths, scale=1.0, what="a value without weight")
    assert torch.isnan(out[..., 0]).all() and torch.isfinite(out[..., 1:]).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_bf16_values_near_the_largest_number(dim):
    """Scores that exceed the first tile's by a little less than what moves the running maximum, whose values are near
    the largest number: the output is one of them, and the sum on the way to it is a finite number too."""
    n = 300
    q, k, v = (torch.zeros(n, 1, dim) for _ in range(3))
    q[..., 0], k[..., 0] = 1.0, -50.0
    k[:100, :, 0], v[:100] = 0.0, 1.0
    k[270, :, 0], v[270] = 5.0, 2.0e38  # 2^7.2 of the first tile's weights
    q, k, v = (x.to(BF16) for x in (q, k, v))
    out, _ = check_prompt(q, k, v, [0, n], scale=1.0, what="prompt")
    assert torch.isfinite(out).all() and float(out[-1, 0, 0]) > 1e37
    # as a cache's, in whole units and in parts
    for length in (n, 6000):
        c = Cache([length], 16, 1, dim, BF16, seed=29)
        put(c, 0, range(length), 0, c.k, torch.cat((torch.full((1,), -50.0), torch.zeros(dim - 1))))
        put(c, 0, range(length), 0, c.v, 0.0)
        for at, score, value in ((range(100), 0.0, 1.0), ([270], 5.0, 2.0e38)):
            put(c, 0, at, 0, c.k, torch.cat((torch.full((1,), score), torch.zeros(dim - 1))))
            put(c, 0, at, 0, c.v, value)
        c.to_gpu()
        out, _ = check_chunk(c, q[:3], [0, 3], [length], scale=1.0, what=f"chunk behind {length}")
        assert torch.isfinite(out).all() and float(out[-1, 0, 0]) > 1e37


@pytest.mark.parametrize("dtype, act, dim, page, hkv", [
    (F16, F16, 128, 16, 2), (BF16, BF16, 64, 16, 160), (E4M3, BF16, 128, 64, 2), (E4M3, F16, 96, 7, 160), (BF16, BF16, 256, 24, 1)])
@pytest.mark.parametrize("window", [0, 1500])
def test_chunk_rows_beside_a_value_that_they_do_not_see(dtype, act, dim, page, hkv, window):
    """NaN and infinities among the values (and keys) of a chunk's later rows, and before a window, behind a long
    context: in whole units (160 heads) and in parts. The rows around them are computed again from their own keys."""
    length, rows = 4500 if hkv > 2 else 20000, 70
    c = Cache([length], page, hkv, dim, dtype, seed=30)
    odd = 1 if hkv > 2 else 0
    for at, head, pool, value in ((length - 3, odd, c.v, math.inf), (length - 30, odd, c.v, NAN), (length - 9, odd, c.k, NAN),
                                  (length - rows - 1480, odd, c.v, -math.inf)):
        put(c, 0, [at], head, pool, lambda x: torch.cat((x[..., :5], torch.full_like(x[..., :1], value), x[..., 6:]), -1))
    if not window:
        put(c, 0, [length - rows - 1480], odd, c.v, 1.0)
    c.to_gpu()
    q = randn(gen(31), rows, 3 * hkv if hkv < 100 else hkv, dim).to(act)
    out, _ = check_chunk(c, q, [0, rows], [length], window=window, what=f"{dtype} D={dim} window={window}")
    g = q.shape[1] // hkv
    mine = out[:, odd * g:odd * g + g]
    assert torch.isfinite(mine[20 if window else 0:rows - 30]).all() and torch.isnan(mine[rows - 9:]).all()
    assert torch.isfinite(out[:, (odd + 1) * g:]).all()


def test_chunk_rows_beside_a_value_that_they_do_not_see_behind_millions_of_tokens():
    """49 rows beside a NaN value behind 8 million tokens (a page, over and over), in the first unit of CTAs that have a
    second one: computed again for as long as a unit takes, not a row at a time while the other warps wait."""
    heads, dim, page, rows, pages = 160, 64, 64, 50, 1 << 17
    g = gen(32)
    q, k, v = (randn(g, n, heads, dim).to(F16) for n in (rows, 2 * page, 2 * page))
    # all pages but the last: scores of -25.9 and less where the last one's lse is 1.8 and more
    q[..., 0], k[:page, :, 0], k[page:, :, 0] = 16.0, -16.0, 0.0
    v[-1, 140:152] = NAN
    table = torch.zeros(1, pages, dtype=torch.int32)
    table[0, -1] = 1
    handle = w4.PagedKVCache(k.view(2, page, heads, dim).cuda(), v.view(2, page, heads, dim).cuda(), table.cuda())
    out, lse = fresh(q)
    w4.w4a4_chunk_attention(q.cuda(), handle, ints([0, rows]), ints([pages * page]), out, lse=lse)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0
    o, l, ot, lt = rows_ref(q, k[page:].to(F64), v[page:].to(F64), page - rows, dim ** -0.5)
    rest = 2 ** 23 * math.exp(-27)  # the weight of all other pages beside the last one's
    check(out, o, ot + rest * (6 + o.abs().nan_to_num(0, 0, 0)), "out")
    check(lse, l, lt + rest, "lse")
    assert torch.isfinite(out[:-1]).all() and torch.isnan(out[-1, 140:152]).all()


@pytest.mark.parametrize("dtype, dim, hq, hkv, n", [(F16, 128, 80, 40, 700), (BF16, 64, 64, 64, 700), (BF16, 96, 6, 2, 1100),
                                                    (F16, 256, 12, 12, 600), (BF16, 128, 4, 4, 900)])
@pytest.mark.parametrize("window, shared", [(0, False), (200, False), (0, True), (130, True)])
def test_prompt_rows_keep_their_bits_beside_a_value_that_they_do_not_see(dtype, dim, hq, hkv, n, window, shared):
    """Units of 256 rows and of 128, of one sequence and the next, with tensor maps and (values whose heads share
    memory) without: what a row does not see leaves its output and lse bit for bit as they are."""
    g = torch.Generator(device="cuda").manual_seed(n + dim)
    q, k, v = (torch.randn((n, h, dim), generator=g, device="cuda").to(dtype) for h in (hq, hkv, 1 if shared else hkv))
    starts, group = [0, n // 3, n], hq // hkv
    calls = []
    at = {n // 3 - 20: math.inf, n // 3 + 150: NAN, n - 140: -math.inf, n - 1: NAN}
    for odd in (False, True):
        for j, x in at.items():
            v[j, 0, ::3] = x if odd else 0.5
        out, lse = fresh(q)
        w4.w4a4_prompt_attention(q, k, v.expand(n, hkv, dim), ints(starts), out, lse=lse, window=window)
        calls.append((out, lse))
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0
    (out, lse), (odd, lse2) = calls
    assert torch.equal(lse, lse2) and torch.isfinite(out).all()
    row = torch.arange(n, device="cuda")
    sees = torch.zeros(n, dtype=torch.bool, device="cuda")
    for j in at:
        sees |= (row >= j) & (row < (j + window if window else n)) & ((row < n // 3) == (j < n // 3))
    heads = hq if shared else group
    assert torch.equal(out[~sees], odd[~sees]) and torch.equal(out[:, heads:], odd[:, heads:])
    hit = odd[sees][:, :heads]
    assert not torch.isfinite(hit[..., ::3]).any() and torch.equal(hit[..., 1::3], out[sees][:, :heads, 1::3])


@pytest.mark.parametrize("dtype, dim, hq, hkv", [(F16, 128, 4, 2), (BF16, 64, 3, 1), (BF16, 256, 2, 2)])
def test_rows_outside_all_sequences_have_no_part(dtype, dim, hq, hkv):
    """With NaN in them the sequences' rows have the bits that they have with numbers."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    n, starts = 400, [7, 150, 150, 290]
    q, k, v = (torch.randn((n, h, dim), generator=g, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    c = Cache([200, 0, 300], 16, hkv, dim, dtype, seed=33)
    results = []
    for outside in (1.0, NAN):
        for x in (q, k, v):
            x[:starts[0]], x[starts[-1]:] = outside, outside
        got = [fresh(q), fresh(q)]
        w4.w4a4_prompt_attention(q, k, v, ints(starts), got[0][0], lse=got[0][1])
        w4.w4a4_chunk_attention(q, c.handle, ints(starts), ints(c.lengths), got[1][0], lse=got[1][1])
        results.append(got)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0
    for one, other in zip(*results):
        for a, b in zip(one, other):
            assert torch.equal(a[7:290], b[7:290]) and torch.isfinite(a[7:290]).all()
            assert torch.isnan(b[:7]).all() and torch.isnan(b[290:]).all()


def test_odd_values_that_come_and_go_between_replays():
    """A captured prompt and chunk (split and whole units), replayed with numbers, with NaN in the last tokens' values and
    with numbers again."""
    g = torch.Generator(device="cuda").manual_seed(8)
    q, k, v = (torch.randn((600, h, 128), generator=g, device="cuda").half() for h in (8, 4, 4))
    c = Cache([5000, 300], 16, 4, 128, E4M3, seed=34)
    c.handle.workspace(8)
    starts, few = ints([0, 250, 600]), ints([0, 3, 40])
    outs = [torch.empty_like(q), torch.empty_like(q[:40]), torch.empty_like(q)]
    calls = [lambda: w4.w4a4_prompt_attention(q, k, v, starts, outs[0]),
             lambda: w4.w4a4_chunk_attention(q[:40], c.handle, few, ints_of[0], outs[1]),
             lambda: w4.w4a4_chunk_attention(q, c.handle, starts, ints_of[0], outs[2])]
    ints_of = [ints([5000, 300])]
    for call in calls:
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in calls:
            call()
    page, slot = int(c.table[0, 4999 // 16]), 4999 % 16
    held, seen = c.gv[page, slot, 1].clone(), []
    for odd in (False, True, False, True):
        v[599, 1, 7] = NAN if odd else 0.25
        c.gv.view(torch.uint8)[page, slot, 1] = 0x7F if odd else held.view(torch.uint8)
        for out in outs:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert w4.w4a4_device_status() == 0
        seen.append([out.clone() for out in outs])
    for a, b in ((0, 2), (1, 3)):
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(seen[a], seen[b]))
    number, nan = seen[:2]
    rows = [599, 2, 249]  # the rows that see the last token
    for i, row in enumerate(rows):
        assert torch.isfinite(number[i]).all()
        assert torch.equal(number[i][:, :2], nan[i][:, :2]) and torch.equal(number[i][:row], nan[i][:row])
        assert torch.isnan(nan[i][row, 2:4, 7]).all() and torch.equal(number[i][row + 1:], nan[i][row + 1:])
