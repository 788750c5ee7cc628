"""Corners of the prompt and chunk attention: rows, keys and values that are no numbers or lie at the
borders of their types, in units that are whole and in units that are split along the keys.

References and tolerances as in test_prompt_ops_gpu."""
import math

import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.test_layer_ops_gpu import BF16, E4M3, F16, F64, Cache, gen, randn
from tests.test_prompt_ops_gpu import check_chunk, check_prompt, ints, qkv, starts_of

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
