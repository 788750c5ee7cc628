"""Rotation without a cache, attention over packed prompts and of chunks over a paged cache, against plain
definitions in 64 bits.

Tolerances follow from the arithmetic.  An output rounded to type t is off by at most u(t) = finfo(t).eps / 2 of
its value (plus half a subnormal step).  A probability is rounded once to t: u(t) of its share of the output, and
with fp16 half a subnormal step, 2^-25, of a scale that puts the largest at 2^13 or more.  Scores, sums and the
output are fp32 sums, for whose roundings 2^-18 of the terms' absolute sum is allowed (64 of 2^-24 each), and
2^-12 of the output's (a rounding of 2^-23 for each of 2048 steps)."""
import math

import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.test_layer_ops_gpu import BF16, E4M3, F16, F32, F64, SLACK, Cache, attend, check, gen, randn, tiny, u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()
    w4.w4a4_device_status()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts_of(rows, first=0):
    out = [first]
    for n in rows:
        out.append(out[-1] + n)
    return out


# ---------------------------------------------------------------- rotation without a cache
def turn_ref(x, positions, rope, gain, eps, interleaved):
    """Outputs and tolerance in 64 bits of heads x [tokens, heads, dim]."""
    t, y, size = x.dtype, x.to(F64), x.to(F64).abs()
    if gain is not None:
        inv = 1 / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        y, size = y * inv * gain.to(F64), size * inv * gain.to(F64).abs()
    live = positions >= 0
    if rope is not None:
        live &= positions < rope.shape[0]
        rot = 2 * rope.shape[2]
        turn = rope.to(F64)[torch.where(live, positions, 0).long()][:, :, None]
        c, n = turn[:, 0], turn[:, 1]
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        ya, yb, sa, sb = y[..., a], y[..., b], size[..., a], size[..., b]
        y, size = y.clone(), size.clone()
        y[..., a], y[..., b] = ya * c - yb * n, yb * c + ya * n
        size[..., a], size[..., b] = sa * c.abs() + sb * n.abs(), sb * c.abs() + sa * n.abs()
    y = torch.where(live[:, None, None], y, 0.0)
    return y, torch.where(live[:, None, None], u(t) * y.abs() + SLACK * size + tiny(t), 0.0)


def check_turn(q, k, positions, rope, qg, kg, interleaved=False, in_place=False, eps=1e-6, status=0):
    gq, gk = q.cuda(), k.cuda()
    outs = (gq, gk) if in_place else [torch.full_like(x, float("nan")) for x in (gq, gk)]
    dev = [None if x is None else x.cuda() for x in (rope, qg, kg)]
    w4.w4a4_qk_rope(gq, gk, None if positions is None else positions.cuda(), *outs, rope=dev[0], q_gain=dev[1],
                    k_gain=dev[2], eps=eps, interleaved=interleaved)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == status
    at = torch.zeros(q.shape[0], dtype=torch.int32) if positions is None else positions
    for x, out, gain in ((q, outs[0], qg), (k, outs[1], kg)):
        check(out, *turn_ref(x, at, rope, gain, eps, interleaved), "rotation")


def table(rows, rot, seed=5):
    angle = torch.rand(rows, rot // 2, generator=gen(seed)) * 6.28
    return torch.stack((angle.cos(), angle.sin()), dim=1)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim, rot", [(64, 64), (96, 32), (128, 128), (128, 16), (256, 96), (96, 96), (256, 256)])
@pytest.mark.parametrize("hq, hkv, tokens", [(4, 2, 1), (7, 1, 33), (3, 3, 2000), (40, 8, 5)])
def test_rotation(dtype, dim, rot, hq, hkv, tokens):
    g = gen(dim + tokens)
    q, k = randn(g, tokens, hq, dim).to(dtype), (3 * randn(g, tokens, hkv, dim)).to(dtype)
    at = torch.randint(-1, 77, (tokens,), generator=g, dtype=torch.int32)
    gains = [(1 + 0.2 * randn(g, dim)).to(dtype) for _ in range(2)]
    rope = table(77, rot)
    check_turn(q, k, at, rope, *gains, interleaved=tokens % 2 == 0)
    check_turn(q, k, at, rope, None, None, interleaved=tokens % 2 == 1, in_place=True)
    check_turn(q, k, at, rope, None, gains[1], in_place=True)
    check_turn(q, k, None, None, *gains, eps=0.1)


def test_rotation_positions_outside_the_table_are_padding():
    q, k = randn(gen(0), 5, 2, 64).to(F16), randn(gen(1), 5, 1, 64).to(F16)
    check_turn(q, k, torch.tensor([3, 10, -5, 2 ** 31 - 1, 9], dtype=torch.int32), table(10, 32), None, None,
               status=w4.W4A4_ERR_INDEX)


def test_rotation_of_slices_and_of_queries_alone():
    g = gen(4)
    qkv = randn(g, 19, 12, 128).to(BF16)
    at, rope = torch.arange(19, dtype=torch.int32), table(19, 64)
    dev = qkv.cuda()
    q, k, v = dev.split((8, 2, 2), dim=1)
    w4.w4a4_qk_rope(q, k, at.cuda(), q, k, rope=rope.cuda())
    none = torch.empty(19, 0, 128, dtype=BF16, device="cuda")
    alone = qkv.cuda()[:, :8]
    w4.w4a4_qk_rope(alone, none, at.cuda(), alone, none, rope=rope.cuda())
    torch.cuda.synchronize()
    assert torch.equal(v.cpu(), qkv[:, 10:]) and torch.equal(alone, q)
    ref, tol = turn_ref(qkv[:, :10], at, rope, None, 1e-6, False)
    check(dev[:, :10], ref, tol, "in place in the fused rows")


def test_rotation_is_the_cache_appends():
    """The same numbers in the same order as on the way into a cache."""
    g = gen(6)
    c = Cache([9, 4], 4, 2, 128, F16, fill=False)
    q, k, v = (randn(g, 13, h, 128).to(F16).cuda() for h in (4, 2, 2))
    seqs, at = ints([0] * 9 + [1] * 4), ints([*range(9), *range(4)])
    rope, gains = table(9, 128).cuda(), [(1 + 0.2 * randn(g, 128)).to(F16).cuda() for _ in range(2)]
    q1, q2, k2 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)
    w4.w4a4_kv_append(q, k, v, at, c.handle, q1, seqs=seqs, rope=rope, q_gain=gains[0], k_gain=gains[1])
    w4.w4a4_qk_rope(q, k, at, q2, k2, rope=rope, q_gain=gains[0], k_gain=gains[1])
    table_, stored = c.table.long(), c.gk.cpu()
    k1 = torch.stack([stored[table_[s, p // 4], p % 4] for s, p in zip(seqs.tolist(), at.tolist())])
    for a, b in ((q1.cpu(), q2.cpu()), (k1, k2.cpu())):
        err = (a.to(F64) - b.to(F64)).abs()
        assert (err <= 2 * u(F16) * b.to(F64).abs() + 2 * tiny(F16)).all()


# ---------------------------------------------------------------- attention
def rows_ref(q, k, v, first, scale, causal=True, window=0):
    """(out, lse) and their tolerances in 64 bits of rows q [n, q_heads, dim] at places first .. first + n - 1 over
    keys and values [keys, heads, dim] (64 bits; a key that is not there is None's place: `there` [keys])."""
    n, hq, dim = q.shape
    keys, hkv, t = k.shape[0], k.shape[1], q.dtype
    q = q.to(F64).cuda()
    out, otol = torch.zeros(n, hq, dim, dtype=F64, device="cuda"), torch.zeros(n, hq, dim, dtype=F64, device="cuda")
    lse, ltol = torch.full((n, hq), -math.inf, dtype=F64, device="cuda"), torch.zeros(n, hq, dtype=F64, device="cuda")
    if keys == 0:
        return out, lse, otol, ltol
    place, at = first + torch.arange(n, device="cuda")[:, None], torch.arange(keys, device="cuda")
    seen = torch.ones(n, keys, dtype=torch.bool, device="cuda")
    if causal:
        seen = at <= place
        if window:
            seen &= at > place - window
    for h in range(hq):
        kk, vv = k[:, h * hkv // hq].cuda(), v[:, h * hkv // hq].cuda()
        # keys that a row does not see take no part, whatever they hold
        a = torch.where(seen, q[:, h] @ kk.nan_to_num(0, 0, 0).T, 0.0)
        odd = ~torch.isfinite(kk).all(1)
        if odd.any():
            a[:, odd] = (q[:, h, None, :] * kk[odd]).sum(-1)
        a = torch.where(seen, a * scale, -math.inf)
        mass = (q[:, h].nan_to_num(0, 0, 0).abs() @ kk.nan_to_num(0, 0, 0).abs().T * abs(scale)).masked_fill(~seen, 0)
        top = a.amax(1, keepdim=True)
        none = top == -math.inf
        e = torch.where(seen, (a - torch.where(none, 0.0, top)).exp(), 0.0)
        total = e.sum(1, keepdim=True)
        p = e / torch.where(none, 1.0, total)
        wild = ~torch.isfinite(vv).all(1)
        o, size = p @ torch.where(wild[:, None], 0.0, vv), p @ vv.nan_to_num(0, 0, 0).abs()
        for j in torch.nonzero(wild)[:, 0].tolist():
            o = torch.where(seen[:, j, None], o + p[:, j, None] * vv[j], o)
        worst = mass.amax(1, keepdim=True)
        off = u(t) + 2 * SLACK * worst + 64 * SLACK
        small = keys * 2.0 ** -38 * vv.nan_to_num(0, 0, 0).abs().amax() if t == F16 else 0.0
        tol = off * size + small
        out[:, h] = torch.where(none, 0.0, o)
        otol[:, h] = tol + u(t) * (o.abs().nan_to_num(0, 0, 0) + tol) + tiny(t)
        lse[:, h] = torch.where(none, -math.inf, top + total.log())[:, 0]
        ltol[:, h] = (SLACK * worst + SLACK * (4 + top.abs().nan_to_num(0, 0, 0)) + 64 * SLACK)[:, 0]
    return out, lse, otol, ltol


def fresh(q):
    return (torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda"),
            torch.full(q.shape[:2], float("nan"), dtype=F32, device="cuda"))


def check_rows(q, out, lse, starts, held, place, scale, causal, window, what):
    """Each sequence's rows against held(b) at place(b); the rows outside all sequences are as they were."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    for b, (lo, hi) in enumerate(zip(starts, starts[1:])):
        o, l, ot, lt = rows_ref(q[lo:hi], *held(b), place(b), scale, causal, window)
        check(out[lo:hi], o, ot, f"{what} sequence {b} out")
        check(lse[lo:hi], l, lt, f"{what} sequence {b} lse")
    for rows in (slice(0, starts[0]), slice(starts[-1], None)):
        assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all(), what


def check_prompt(q, k, v, starts, scale=None, causal=True, window=0, what=""):
    out, lse = fresh(q)
    w4.w4a4_prompt_attention(q.cuda(), k.cuda(), v.cuda(), ints(starts), out, lse=lse, scale=scale, window=window,
                             causal=causal)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0
    check_rows(q, out, lse, starts, lambda b: (k[starts[b]:starts[b + 1]].to(F64), v[starts[b]:starts[b + 1]].to(F64)),
               lambda b: 0, scale, causal, window, what)
    return out, lse


def check_chunk(cache, q, starts, lengths, scale=None, causal=True, window=0, what="", status=0, **named):
    out, lse = fresh(q)
    w4.w4a4_chunk_attention(q.cuda(), cache.handle, ints(starts), ints(lengths), out, lse=lse, scale=scale,
                            window=window, causal=causal, **named)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == status
    check_rows(q, out, lse, starts, lambda b: cache.held(b, 0, lengths[b]),
               lambda b: lengths[b] - (starts[b + 1] - starts[b]), scale, causal, window, what)
    return out, lse


def qkv(seed, tokens, hq, hkv, dim, dtype, times=2.0):
    g = gen(seed)
    return (times * randn(g, tokens, hq, dim)).to(dtype), randn(g, tokens, hkv, dim).to(dtype), randn(g, tokens, hkv, dim).to(dtype)


ROWS = [1, 0, 2, 127, 128, 129, 0, 64, 17, 300, 255, 1, 385]
DIMS = [64, 96, 128, 256]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("hkv, group", [(2, 1), (1, 2), (2, 3), (1, 8), (1, 37)])
def test_prompt_lengths_types_heads(dtype, dim, hkv, group):
    starts = starts_of(ROWS, 3)
    q, k, v = qkv(dim + group, starts[-1] + 5, hkv * group, hkv, dim, dtype)
    check_prompt(q, k, v, starts, what=f"{dtype} D={dim} {hkv}x{group}")


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("causal, window", [(False, 0), (True, 1), (True, 2), (True, 100), (True, 128), (True, 129),
                                            (True, 384), (True, 10 ** 6)])
def test_prompt_masks(dim, causal, window):
    starts = starts_of(ROWS)
    q, k, v = qkv(window + 7, starts[-1], 6, 2, dim, BF16)
    check_prompt(q, k, v, starts, causal=causal, window=window, what=f"D={dim} causal={causal} window={window}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", DIMS)
def test_prompt_long(dtype, dim):
    """Many tiles: stages and accumulators are used again and again, and sequences follow one another."""
    for rows, hq, hkv, causal in (([1500], 2, 1, True), ([900, 1300], 3, 3, False), ([700] * 3, 16, 8, True)):
        starts = starts_of(rows)
        q, k, v = qkv(sum(rows), starts[-1], hq, hkv, dim, dtype)
        check_prompt(q, k, v, starts, causal=causal, what=f"{dtype} D={dim} {rows}")


def test_prompt_more_work_than_the_gpu_holds_at_once():
    starts = starts_of([513, 700, 90, 1, 1100, 256, 255, 40, 333])
    q, k, v = qkv(2, starts[-1], 64, 16, 64, F16)
    check_prompt(q, k, v, starts, what="many heads")


def test_prompt_many_short_sequences():
    g = gen(8)
    rows = [int(x) for x in torch.randint(0, 9, (700,), generator=g)]
    rows[:200] = [0] * 200
    starts = starts_of(rows)
    q, k, v = qkv(9, starts[-1], 4, 2, 64, F16)
    check_prompt(q, k, v, starts, what="short sequences")


def test_prompt_of_slices_with_other_strides():
    """q, k and v as slices of the fused rows, heads-first outputs, keys whose heads share memory."""
    g = gen(10)
    rows, starts = randn(g, 300, 12, 128).to(F16), [0, 140, 300]
    dev = rows.cuda()
    out = torch.full((8, 300, 128), float("nan"), dtype=F16, device="cuda").transpose(0, 1)
    w4.w4a4_prompt_attention(dev[:, :8], dev[:, 8:10], dev[:, 10:], ints(starts), out)
    shared = dev[:, 8:9].expand(300, 2, 128)
    other = torch.empty_like(out)
    w4.w4a4_prompt_attention(dev[:, :8], shared, dev[:, 10:], ints(starts), other)
    torch.cuda.synchronize()
    for b in range(2):
        s = slice(starts[b], starts[b + 1])
        for got, k in ((out, rows[s, 8:10]), (other, rows[s, 8:9].expand(-1, 2, -1))):
            o, _, tol, _ = rows_ref(rows[s, :8], k.to(F64), rows[s, 10:].to(F64), 0, 128 ** -0.5)
            check(got[s], o, tol, "slices")


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-30, -40.0])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompt_scales(scale, dtype):
    q, k, v = qkv(11, 333, 4, 2, 128, dtype)
    check_prompt(q, k, v, [0, 100, 333], scale=scale, what=f"scale {scale}")
    check_prompt(q, k, v, [0, 100, 333], scale=scale, causal=False, what=f"scale {scale}")


@pytest.mark.parametrize("odd", [float("nan"), math.inf, -math.inf])
@pytest.mark.parametrize("dtype, dim", [(F16, 128), (BF16, 64), (BF16, 256)])
def test_prompt_rows_that_are_not_seen_have_no_part(odd, dtype, dim):
    """Infinities and NaN in keys and values, before, inside and behind what a row sees."""
    rows = [200, 150, 310]
    starts = starts_of(rows)
    q, k, v = qkv(12, starts[-1], 4, 2, dim, dtype)
    k[starts[0] + 190], v[starts[1] + 20, 1, 3], v[starts[2] + 290], k[starts[2] + 5, 0, 0] = odd, odd, odd, odd
    w = check_prompt(q, k, v, starts, window=64, what=f"{odd} window")[0]
    assert torch.isfinite(w[starts[2] + 5 + 64:starts[2] + 290]).all()
    out = check_prompt(q, k, v, starts, what=f"{odd}")[0]
    for seen in (slice(0, 190), slice(starts[1], starts[1] + 20), slice(starts[2], starts[2] + 5)):
        assert torch.isfinite(out[seen]).all()
    assert torch.isfinite(out[starts[1]:starts[2], :2]).all()  # the other key-value head's


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompt_rows_without_weight_are_zero_whatever_the_values(dtype):
    q, k, v = qkv(13, 140, 2, 1, 64, dtype)
    q[:, :, 0], k[:, :, 0] = 1.0, -math.inf
    v[3] = float("nan")
    out, lse = fresh(q)
    w4.w4a4_prompt_attention(q.cuda(), k.cuda(), v.cuda(), ints([0, 140]), out, lse=lse)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("below", [12, 18, 26])
def test_prompt_many_small_weights_beside_a_large_one(dtype, below):
    """The first token takes nearly all the weight and has zero values; the others make the output."""
    n, d = 3000, 64
    q, k, v = torch.zeros(n, 1, d), torch.zeros(n, 1, d), torch.ones(n, 1, d)
    q[..., 0], k[0, :, 0], v[0] = 1.0, below / 1.4427, 0.0
    check_prompt(q.to(dtype), k.to(dtype), v.to(dtype), [0, n], scale=1.03, what="small weights")


def test_prompt_growing_scores():
    """Each tile's scores exceed the last's, so that the running maximum moves at every one."""
    n = 900
    q, k, v = qkv(14, n, 2, 1, 128, F16)
    q[..., 0], k[..., 0] = 4.0, (torch.arange(n) / 20).to(F16)[:, None]
    check_prompt(q, k, v, [0, n], scale=0.5, what="growing")
    check_prompt(q, k.flip(0), v, [0, n], scale=0.5, what="shrinking")


def test_prompt_starts_that_are_no_order():
    q, k, v = qkv(15, 100, 2, 2, 64, F16)
    for starts, good in (([-5, 40, 100], [(0, 40), (40, 100)]), ([0, 60, 200], [(0, 60), (60, 100)]),
                         ([70, 20, 60], [(20, 60)]), ([200, 300], [])):
        out, lse = fresh(q)
        w4.w4a4_prompt_attention(q.cuda(), k.cuda(), v.cuda(), ints(starts), out, lse=lse)
        torch.cuda.synchronize()
        assert w4.w4a4_device_status() == w4.W4A4_ERR_INDEX
        for lo, hi in good:
            o, l, ot, lt = rows_ref(q[lo:hi], k[lo:hi].to(F64), v[lo:hi].to(F64), 0, 0.125)
            check(out[lo:hi], o, ot, "clamped"), check(lse[lo:hi], l, lt, "clamped")
    out = fresh(q)[0]
    w4.w4a4_prompt_attention(q.cuda(), k.cuda(), v.cuda(), ints([30]), out)  # no sequence
    empty = q[:0].cuda()
    w4.w4a4_prompt_attention(empty, k[:0].cuda(), v[:0].cuda(), ints([0, 0]), empty.clone())
    assert torch.isnan(out).all() and w4.w4a4_device_status() == 0


LENGTHS = [300, 5, 64, 1000, 128, 17, 2, 129, 515]
CHUNKS = [1, 5, 0, 130, 128, 16, 2, 64, 33]


@pytest.mark.parametrize("dtype, act", [(F16, F16), (BF16, BF16), (E4M3, F16), (E4M3, BF16)])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("hkv, group, page, layout", [(2, 1, 16, "NHD"), (3, 4, 7, "HND"), (1, 8, 1, "NHD"),
                                                      (2, 9, 64, "HND"), (1, 2, 200, "NHD")])
def test_chunk_lengths_types_heads(dtype, act, dim, hkv, group, page, layout):
    c = Cache(LENGTHS, page, hkv, dim, dtype, seed=dim + group, layout=layout)
    starts = starts_of(CHUNKS, 2)
    q = (2 * randn(gen(1), starts[-1] + 3, hkv * group, dim)).to(act)
    check_chunk(c, q, starts, LENGTHS, what=f"{dtype} {act} D={dim} {hkv}x{group} page={page}")


@pytest.mark.parametrize("dtype", [F16, E4M3])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal, window", [(False, 0), (True, 1), (True, 50), (True, 128), (True, 300), (True, 5000)])
def test_chunk_masks(dtype, dim, causal, window):
    c = Cache(LENGTHS, 24, 2, dim, dtype, seed=window)
    starts = starts_of(CHUNKS)
    q = (2 * randn(gen(2), starts[-1], 4, dim)).to(F16)
    check_chunk(c, q, starts, LENGTHS, causal=causal, window=window, scale=0.1, what=f"{dtype} D={dim} {causal} {window}")


@pytest.mark.parametrize("dtype, act", [(F16, F16), (BF16, BF16), (E4M3, BF16)])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("rows, lengths, window", [([5], [9001], 0), ([61, 3], [5000, 7001], 0), ([200], [4100], 0),
                                                   ([9], [8000], 1000), ([1, 1, 1], [3001, 1, 6000], 0)])
def test_chunk_few_rows_over_a_long_cache(dtype, act, dim, rows, lengths, window):
    """Rows whose keys are shared out, joined in the tokens' order: the same bits every time."""
    c = Cache(lengths, 64, 1, dim, dtype, seed=dim)
    starts = starts_of(rows)
    q = (2 * randn(gen(3), starts[-1], 3, dim)).to(act)
    out, lse = check_chunk(c, q, starts, lengths, window=window, what=f"{dtype} D={dim} {rows} of {lengths}")
    for _ in range(3):
        again, lse2 = fresh(q)
        w4.w4a4_chunk_attention(q.cuda(), c.handle, ints(starts), ints(lengths), again, lse=lse2, window=window)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype, act, dim", [(F16, F16, 128), (F16, F16, 64), (E4M3, BF16, 64), (E4M3, F16, 128), (BF16, BF16, 256)])
def test_chunk_gives_the_same_bits_while_copies_arrive_in_any_order(dtype, act, dim):
    """Few rows, whose tiles two streams take in turns, over keys of which some are in L2 and some are not: a stage
    whose copy is overtaken by the next ones' must be waited for all the same."""
    lengths = [2900, 1000, 4097, 128, 3333, 700]
    c = Cache(lengths, 16, 4, dim, dtype, seed=dim)
    rows = [4, 9, 1, 30, 2, 17]
    q = randn(gen(11), sum(rows), 8, dim).to(act)
    want, _ = check_chunk(c, q, starts_of(rows), lengths)
    args = q.cuda(), c.handle, ints(starts_of(rows)), ints(lengths)
    keys, outs = c.gk.reshape(-1).view(torch.uint8), [fresh(q)[0] for _ in range(40)]
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    for i, out in enumerate(outs):
        flush.zero_()  # out of L2, then every other call some of the keys back into it
        if i % 2:
            keys[: len(keys) // 3].max()
        w4.w4a4_chunk_attention(*args, out)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0 and all(torch.equal(out, want) for out in outs)


def test_chunk_of_one_token_is_the_paged_attention():
    lengths = [700, 33, 1, 0, 2049]
    c = Cache(lengths, 16, 2, 128, F16, seed=4)
    q = randn(gen(4), 5, 4, 128).to(F16)
    one, lse1 = attend(c, q, lengths)
    out, lse = check_chunk(c, q, starts_of([1] * 5), lengths)
    assert torch.allclose(one.float(), out.float(), rtol=2e-3, atol=2e-3) and torch.equal(lse1 == -math.inf, lse == -math.inf)


def test_chunk_longer_than_its_cache():
    """The rows before token 0 see nothing."""
    c = Cache([10, 0, 3], 16, 1, 64, F16)
    q = randn(gen(5), 14 + 140 + 3, 2, 64).to(F16)
    out, lse = check_chunk(c, q, [0, 14, 154, 157], [10, 0, 3])
    assert torch.all(out[:4] == 0) and torch.all(lse[:4] == -math.inf) and torch.all(out[14:154] == 0)
    check_chunk(c, q, [0, 14, 154, 157], [10, 0, 3], causal=False)


def test_chunk_lengths_and_pages_outside_their_tables():
    c = Cache([100, 90], 16, 1, 64, F16)
    q = randn(gen(6), 8, 2, 64).to(F16)
    out, lse = fresh(q)
    top = c.table.shape[1] * c.page
    w4.w4a4_chunk_attention(q.cuda(), c.handle, ints([0, 4, 8]), ints([-3, 90]), out, lse=lse)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == w4.W4A4_ERR_INDEX and torch.all(out[:4] == 0) and torch.all(lse[:4] == -math.inf)
    o, _, tol, _ = rows_ref(q[4:], *c.held(1, 0, 90), 86, 0.125)
    check(out[4:], o, tol, "beside a bad length")
    c.table[0, 2], c.table[1, 0] = 10 ** 6, -1
    c.to_gpu()
    out = fresh(q)[0]
    w4.w4a4_chunk_attention(q.cuda(), c.handle, ints([0, 4, 8]), ints([100, 90]), out, causal=False)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == w4.W4A4_ERR_INDEX
    for b, n in enumerate((100, 90)):
        o, _, tol, _ = rows_ref(q[4 * b:4 * b + 4], *c.held(b, 0, n), 0, 0.125, causal=False)
        check(out[4 * b:4 * b + 4], o, tol, "pages left out")
    assert top >= 100


@pytest.mark.parametrize("dtype, act", [(F16, F16), (E4M3, BF16)])
def test_chunk_rows_that_are_not_seen_have_no_part(dtype, act):
    """The cache's pages hold NaN behind each sequence's tokens (see Cache); here also among those of later rows."""
    lengths = [400, 260]
    c = Cache(lengths, 16, 2, 64, dtype)
    for b, tok in ((0, 390), (0, 300), (1, 259)):
        page, slot = c.table[b, tok // 16].long(), tok % 16
        for pool in (c.k, c.v):
            x = pool.float()
            x[page, slot, 0, 5] = float("nan")
            pool.copy_(x.to(dtype))
    c.to_gpu()
    q = randn(gen(7), 150 + 40, 4, 64).to(act)
    out, _ = check_chunk(c, q, [0, 150, 190], lengths)
    assert torch.isnan(out[50:150, :2]).all() and torch.isfinite(out[:, 2:]).all() and torch.isfinite(out[150:189]).all()
    check_chunk(c, q, [0, 150, 190], lengths, window=60)


def test_chunk_offsets_that_pass_32_bits():
    """Pages 2 GB apart, and a token stride that does not fit 32 bits times a token's number."""
    pages, page, dim = 5, 16, 64
    big = torch.empty(pages * (1 << 30), dtype=F16, device="cuda")  # 10.7 GB, of which rows are used
    pools = [big.as_strided((pages, page, 1, dim), (1 << 29, 1 << 24, dim, 1), off) for off in (0, 1 << 23)]
    g = gen(9)
    k, v = (randn(g, pages, page, 1, dim).to(F16) for _ in range(2))
    for pool, x in zip(pools, (k, v)):
        pool.copy_(x.cuda())
    order = torch.tensor([[3, 1, 4, 0, 2]], dtype=torch.int32)
    handle = w4.PagedKVCache(*pools, order.cuda())
    q = randn(g, 30, 2, dim).to(F16)
    out = fresh(q)[0]
    w4.w4a4_chunk_attention(q.cuda(), handle, ints([0, 30]), ints([77]), out)
    o, _, tol, _ = rows_ref(q, *(x[order[0].long()].flatten(0, 1)[:77].to(F64) for x in (k, v)), 47, dim ** -0.5)
    check(out, o, tol, "far pages")
    del pools, handle
    rows = big.as_strided((150, 1, dim), (1 << 25, dim, 1), 0)  # 150 tokens over 2^32 elements
    x = randn(g, 150, 1, dim).to(F16)
    rows.copy_(x.cuda())
    out = fresh(x)[0]
    w4.w4a4_prompt_attention(rows, rows, rows, ints([0, 150]), out)
    o, _, tol, _ = rows_ref(x, x.to(F64), x.to(F64), 0, dim ** -0.5)
    check(out, o, tol, "far rows")


# ---------------------------------------------------------------- how they are called
def test_in_a_graph_on_another_stream_with_growing_lengths():
    c = Cache([600, 300], 16, 2, 128, F16, seed=1)
    q = randn(gen(10), 12, 4, 128).to(F16)
    gq, starts, lengths = q.cuda(), ints([0, 8, 12]), ints([100, 50])
    out, lse = fresh(q)
    c.handle.workspace(4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        w4.w4a4_chunk_attention(gq, c.handle, starts, lengths, out, lse=lse)  # warm-up
        with torch.cuda.graph(graph, stream=side):
            w4.w4a4_chunk_attention(gq, c.handle, starts, lengths, out, lse=lse)
            w4.w4a4_prompt_attention(gq, gq[:, :2], gq[:, 2:], starts, both := torch.empty_like(gq))
    torch.cuda.synchronize()
    for now, rows in (([100, 50], [0, 8, 12]), ([600, 299], [0, 8, 12]), ([0, 300], [0, 0, 12]), ([32, 4], [0, 11, 12])):
        starts.copy_(ints(rows)), lengths.copy_(ints(now)), out.fill_(float("nan")), lse.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check_rows(q, out, lse, rows, lambda b: c.held(b, 0, now[b]), lambda b: now[b] - (rows[b + 1] - rows[b]), None,
                   True, 0, "replayed")
        for b in range(2):
            s = slice(rows[b], rows[b + 1])
            o, _, tol, _ = rows_ref(q[s], q[s, :2].to(F64), q[s, 2:].to(F64), 0, 128 ** -0.5)
            check(both[s], o, tol, "replayed prompt")
    assert w4.w4a4_device_status() == 0


def test_one_workspace_for_all_shapes_and_both_attentions():
    """Calls one after another on one buffer, whose counters the single-token attention needs zeroed."""
    caches = [Cache([5000, 3000, 64], 16, 2, dim, F16, seed=dim) for dim in (256, 64)]
    ws = torch.zeros(max(w4.lib().w4a4_paged_attention_workspace_bytes(3, 32, 2, d) for d in (64, 256)), dtype=torch.uint8,
                     device="cuda")
    for turn in range(3):
        for c in caches:
            for heads, rows in ((2, [1, 1, 1]), (32, [3, 4, 5]), (8, [60, 10, 64])):
                q = randn(gen(turn), sum(rows), heads, c.dim).to(F16)
                check_chunk(c, q, starts_of(rows), c.lengths, workspace=ws)
            q = randn(gen(turn), 3, 8, c.dim).to(F16)
            out = fresh(q)[0]
            w4.w4a4_paged_attention(q.cuda(), c.handle, ints(c.lengths), out, workspace=ws)
            for b, n in enumerate(c.lengths):
                o, _, tol, _ = rows_ref(q[b:b + 1], *c.held(b, 0, n), n - 1, c.dim ** -0.5)
                check(out[b:b + 1], o, tol, "after chunks")


def test_two_streams_at_once():
    """Calls with a cache object (a workspace) each, at the same time."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    caches = [Cache([4000, 900], 16, 2, 128, F16, seed=s) for s in range(2)]
    q = [randn(gen(s), 40, 8, 128).to(F16) for s in range(2)]
    outs = [[fresh(q[0])[0] for _ in range(10)] for _ in range(2)]
    gq, starts, lengths = [x.cuda() for x in q], ints([0, 30, 40]), ints([4000, 900])
    for c in caches:
        c.handle.workspace(8)
    torch.cuda.synchronize()
    for i in range(10):
        for s in range(2):
            w4.w4a4_chunk_attention(gq[s], caches[s].handle, starts, lengths, outs[s][i], stream=sides[s])
    torch.cuda.synchronize()
    for s in range(2):
        for b, (lo, hi) in enumerate(((0, 30), (30, 40))):
            n = (4000, 900)[b]
            o, _, tol, _ = rows_ref(q[s][lo:hi], *caches[s].held(b, 0, n), n - hi + lo, 128 ** -0.5)
            for out in outs[s]:
                check(out[lo:hi], o, tol, "beside another stream's")
    assert w4.w4a4_device_status() == 0


def test_dispatch_names_the_operators():
    q, k, v = (x.cuda() for x in qkv(1, 10, 4, 2, 64, F16))
    w4.w4a4_qk_rope(q, k, None, torch.empty_like(q), torch.empty_like(k))
    assert w4.w4a4_last_dispatch().startswith("qk_rope tokens=10 heads=4+2 dim=64")
    w4.w4a4_prompt_attention(q, k, v, ints([0, 10]), torch.empty_like(q))
    assert w4.w4a4_last_dispatch().startswith("prompt_attention f16 tokens=10 seqs=1 heads=4/2 dim=64")
    c = Cache([30], 16, 2, 64, E4M3)
    w4.w4a4_chunk_attention(q, c.handle, ints([0, 10]), ints([30]), torch.empty_like(q))
    assert w4.w4a4_last_dispatch().startswith("chunk_attention e4m3 tokens=10 seqs=1 heads=4/2 dim=64")


def test_binding_refuses_what_does_not_fit():
    q, k, v = (x.cuda() for x in qkv(1, 10, 4, 2, 64, F16))
    s, out = ints([0, 10]), torch.empty_like(q)
    for args in ((q, k[:9], v, s, out), (q, k, v[:, :1], s, out), (q, k.bfloat16(), v, s, out), (q, k, v, s.long(), out),
                 (q, k, v, s, out[:9]), (q, k, v, s.cpu(), out), (q, k, v, s, q), (q, k, v, s, out.float())):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_prompt_attention(*args)
    for named in (dict(lse=torch.empty(10, 4, device="cuda", dtype=F16)), dict(window=3, causal=False), dict(window=-1),
                  dict(scale=math.nan), dict(lse=torch.empty(10, 3, device="cuda"))):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_prompt_attention(q, k, v, s, out, **named)
    c = Cache([30], 16, 2, 64, F16)
    n = ints([30])
    for args in ((q, c.handle, s[:1], n, out), (q, c.handle, s, ints([1, 2]), out), (q.bfloat16(), c.handle, s, n, out),
                 (q[:, :3], c.handle, s, n, out[:, :3]), (q, c.handle, s, n, q)):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_chunk_attention(*args)
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_chunk_attention(q, c.handle, s, n, out, workspace=torch.zeros(1000, dtype=torch.uint8, device="cuda"))
    for args in ((q, k, n, out, k), (q, k, ints(range(10)).long(), out, k), (q, k[:9], ints(range(10)), out, k)):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_qk_rope(*args)
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_qk_rope(q, k, None, out, k, rope=table(20, 32).cuda())  # rotation without positions
