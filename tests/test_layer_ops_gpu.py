"""Cache append, paged attention and block norm against plain definitions in 64 bits.

Tolerances follow from the arithmetic: an output rounded to type t is off by at most
u(t) = finfo(t).eps / 2 of its value (plus half a subnormal step); attention also rounds
each probability to the MMA's operand type; what is left is fp32 arithmetic, for which
2^-18 of the terms' absolute sum is allowed (64 roundings of 2^-24 each)."""
import math

import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.layer_structs import pack

pytestmark = pytest.mark.gpu

F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
F64 = torch.float64
SLACK = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()
    w4.w4a4_device_status()


def u(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the subnormals."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def check(got, ref, tol, what):
    """|got - ref| <= tol, with infinities and NaN in the same places."""
    got, ref, tol = got.detach().cpu().to(F64), ref.cpu(), tol.cpu()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN"
    odd = ~fin & ~torch.isnan(ref)
    assert torch.equal(got[odd], ref[odd]), f"{what}: infinities"
    err = (got - ref).abs()[fin]
    over = err > tol[fin]
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} off, worst {float((err / tol[fin]).max()):.2f}x"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g)


# ---------------------------------------------------------------- a paged cache
class Cache:
    """Pools with every slot that holds no token (and spare pages) poisoned with NaN."""

    def __init__(self, lengths, page, hkv, dim, dtype, seed=0, layout="NHD", scales=True, fill=True, spare=2, wide=0):
        g = gen(seed)
        self.lengths, self.page, self.hkv, self.dim, self.dtype = lengths, page, hkv, dim, dtype
        need = [-(-n // page) for n in lengths]
        pages, width = sum(need) + spare, max(need + [1]) + wide
        order = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((len(lengths), width), -7, dtype=torch.int32)  # unused entries are never read
        shape = (pages, page, hkv, dim)
        nan = float("nan")
        self.k, self.v = torch.full(shape, nan), torch.full(shape, nan)
        self.ks = self.vs = None
        if dtype == E4M3 and scales:
            self.ks, self.vs = torch.rand(hkv, generator=g) / 50 + 0.01, torch.rand(hkv, generator=g) / 50 + 0.01
        at = 0
        for b, n in enumerate(lengths):
            mine = order[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = torch.tensor(mine, dtype=torch.int32)
            if fill:
                tok = torch.arange(n)
                for pool, s in ((self.k, self.ks), (self.v, self.vs)):
                    x = randn(g, n, hkv, dim)
                    if dtype == E4M3:
                        x = (x / s[:, None] if s is not None else x).clamp(-448, 448)
                    pool[torch.tensor(mine, dtype=torch.long)[tok // page], tok % page] = x
        self.k, self.v = self.k.to(dtype), self.v.to(dtype)
        self.hnd = layout == "HND"
        self.to_gpu()

    def to_gpu(self):
        def up(t):
            return t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if self.hnd else t.cuda()
        self.gk, self.gv, self.gt = up(self.k), up(self.v), self.table.cuda()
        dev = [None if s is None else s.cuda() for s in (self.ks, self.vs)]
        self.handle = w4.PagedKVCache(self.gk, self.gv, self.gt, *dev)

    def held(self, b, lo, hi):
        """Keys and values [tokens, heads, dim] of sequence b in 64 bits."""
        tok = torch.arange(lo, hi)
        page = self.table[b, tok // self.page].long()
        good = (page >= 0) & (page < self.k.shape[0])
        page, slot = page[good], (tok % self.page)[good]
        out = []
        for pool, s in ((self.k, self.ks), (self.v, self.vs)):
            x = pool.float()[page, slot].to(F64)
            out.append(x if s is None else x * s.to(F64)[:, None])
        return out


def attention_ref(q, cache, lengths, scale, window):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits."""
    S, hq, dim = q.shape
    group = hq // cache.hkv
    p_type = BF16 if cache.dtype == BF16 else F16
    out, tol = torch.zeros(S, hq, dim, dtype=F64), torch.zeros(S, hq, dim, dtype=F64)
    lse, ltol = torch.full((S, hq), -math.inf, dtype=F64), torch.zeros(S, hq, dtype=F64)
    top = cache.table.shape[1] * cache.page
    for b, n in enumerate(lengths):
        n = max(0, min(n, top))
        lo = max(0, n - window) if window else 0
        k, v = cache.held(b, lo, n)
        if k.shape[0] == 0:
            continue
        qq = q[b].to(F64).view(cache.hkv, group, dim)
        a = torch.einsum("hgd,nhd->hgn", qq, k) * scale
        mass = torch.einsum("hgd,nhd->hgn", qq.abs(), k.abs()) * scale
        m = a.amax(-1, keepdim=True)
        none = (m == -math.inf)
        e = torch.where(none, 0.0, (a - torch.where(none, 0.0, m)).exp())
        l = e.sum(-1, keepdim=True)
        p = torch.where(none, 0.0, e / torch.where(none, 1.0, l))
        o = torch.einsum("hgn,nhd->hgd", p, v) if not none.all() else torch.zeros(cache.hkv, group, dim, dtype=F64)
        if none.any():
            o = torch.where(none, 0.0, o)
        pv = torch.einsum("hgn,nhd->hgd", p, v.nan_to_num(0, 0, 0).abs())
        # a score off by d moves its weight by the factor e^d: twice the largest, once for l
        worst = torch.nan_to_num(mass, 0, 0, 0).amax(-1, keepdim=True)
        off = u(p_type) + 2 * SLACK * worst + 64 * SLACK
        vmax = v.nan_to_num(0, 0, 0).abs().amax() if v.numel() else 0.0
        t = off * pv + a.shape[-1] * tiny(F16) * vmax * (p_type == F16)
        out[b], tol[b] = o.reshape(hq, dim), (t + u(q.dtype) * (o.abs() + t) + tiny(q.dtype)).reshape(hq, dim)
        lse[b] = torch.where(none, -math.inf, m + torch.where(none, 1.0, l).log()).reshape(hq)
        ltol[b] = (SLACK * worst + SLACK * (4 + m.abs().nan_to_num(0, 0, 0)) + 64 * SLACK).reshape(hq)
    return out, lse, tol, ltol


def attend(cache, q, lengths, scale=None, window=0, check_status=True):
    gl = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), dtype=F32, device="cuda")
    w4.w4a4_paged_attention(q.cuda(), cache.handle, gl, out, lse=lse, scale=scale, window=window)
    torch.cuda.synchronize()
    if check_status:
        assert w4.w4a4_device_status() == 0
    return out, lse


def check_attention(cache, q, lengths, scale=None, window=0, what="", check_status=True):
    out, lse = attend(cache, q, lengths, scale, window, check_status)
    o, l, t, lt = attention_ref(q, cache, lengths, q.shape[-1] ** -0.5 if scale is None else scale, window)
    check(out, o, t, what + " out")
    check(lse, l, lt, what + " lse")
    return out, lse


LENGTHS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300, 0, 1000]


@pytest.mark.parametrize("dtype, act", [(F16, F16), (BF16, BF16), (E4M3, F16), (E4M3, BF16)])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("hkv, group, page, layout", [(2, 1, 16, "NHD"), (3, 4, 7, "HND"), (1, 8, 1, "NHD"),
                                                      (2, 9, 64, "HND"), (1, 37, 33, "NHD")])
def test_attention_lengths_types_heads(dtype, act, dim, hkv, group, page, layout):
    c = Cache(LENGTHS, page, hkv, dim, dtype, seed=dim + group, layout=layout)
    q = (2 * randn(gen(1), len(LENGTHS), hkv * group, dim)).to(act)
    check_attention(c, q, LENGTHS, what=f"{dtype} {act} D={dim} {hkv}x{group}")


@pytest.mark.parametrize("window", [1, 16, 50, 64, 999, 1000, 5000])
@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_attention_window(window, dtype):
    c = Cache(LENGTHS, 24, 2, 128, dtype, seed=window)
    q = randn(gen(2), len(LENGTHS), 6, 128).to(F16)
    check_attention(c, q, LENGTHS, window=window, scale=0.2)


def test_attention_many_short_sequences():
    """More sequences than threads in a CTA, most of them empty or a few tokens long."""
    g = gen(3)
    lengths = [int(x) for x in torch.randint(0, 6, (777,), generator=g)]
    lengths[:130] = [0] * 130
    c = Cache(lengths, 4, 2, 64, F16)
    check_attention(c, randn(g, len(lengths), 4, 64).to(F16), lengths)
    none = [0] * 5
    out, lse = attend(c2 := Cache(none, 4, 2, 64, F16), randn(g, 5, 4, 64).to(F16), none)
    assert out.abs().max() == 0 and torch.all(lse == -math.inf) and c2 is not None


@pytest.mark.parametrize("dtype, hkv, group", [(F16, 1, 2), (BF16, 4, 8), (E4M3, 1, 16)])
def test_attention_long_split_and_joined(dtype, hkv, group):
    """One sequence over many CTAs beside short ones: parts joined, the same bits every time."""
    lengths = [70001, 3, 0, 5000, 64]
    c = Cache(lengths, 16, hkv, 128, dtype, seed=5)
    q = (1.5 * randn(gen(6), len(lengths), hkv * group, 128)).to(BF16 if dtype == BF16 else F16)
    out, lse = check_attention(c, q, lengths)
    for _ in range(3):
        again, lse2 = attend(c, q, lengths)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(lse2, lse)


@pytest.mark.parametrize("lengths, hkv, group, dim", [
    ([700, 650, 1, 0, 702, 700, 699, 688], 8, 2, 128),   # runs of two or three units: single pieces
    ([3000] * 3, 16, 1, 64), ([5000, 40], 2, 16, 96), ([2000], 1, 11, 256),
    ([4096] * 6, 8, 1, 128),                             # runs over two sequences' heads
    ([1] * 40, 8, 1, 64), ([16] * 45, 4, 2, 128),        # one step a sequence, more of them than CTAs
])
@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_attention_shares_of_the_work(lengths, hkv, group, dim, dtype):
    """Each way the units are shared out among the CTAs, and its joins."""
    c = Cache(lengths, 16, hkv, dim, dtype, seed=sum(lengths) + dim)
    check_attention(c, randn(gen(30), len(lengths), hkv * group, dim).to(F16), lengths)


def test_attention_heads_side_by_side_and_defaults():
    """A page table wide enough for the heads of short adjacent rows to be taken together; E4M3
    without scales; a negative scale."""
    lengths = [100, 3, 900, 64, 0]
    for dtype, dim, hkv in ((F16, 64, 4), (E4M3, 64, 6), (BF16, 96, 2), (E4M3, 128, 8)):
        c = Cache(lengths, 64, hkv, dim, dtype, seed=31, scales=False, wide=40000)
        q = (0.1 * randn(gen(32), 5, 3 * hkv, dim) if dtype == E4M3 else randn(gen(32), 5, 3 * hkv, dim))
        check_attention(c, q.to(BF16 if dtype == BF16 else F16), lengths, what=f"{dtype} {dim}")
    assert "heads/unit=" in w4.w4a4_last_dispatch()
    c = Cache(lengths, 64, 2, 64, F16, seed=33)
    q = randn(gen(34), 5, 4, 64).to(F16)
    out, _ = attend(c, q, lengths, scale=-0.1)
    want, _ = attend(c, -q, lengths, scale=0.1)
    assert torch.equal(out, want)


def test_attention_refuses_more_units_than_it_can_number():
    """Sizes alone, on the host: nothing is launched, so the pointers are never used."""
    args = pack("w4a4_paged_attention_args", q=256, out=256, lengths=256, workspace=256, workspace_bytes=1 << 40,
                q_token_stride=8192, q_head_stride=64, out_token_stride=8192, out_head_stride=64, scale=0.1, q_heads=128)
    cache = pack("w4a4_kv_cache", k=256, v=256, page_table=256, k_page_stride=1024, k_token_stride=64, k_head_stride=64,
                 v_page_stride=1024, v_token_stride=64, v_head_stride=64, table_stride=1 << 27, seqs=64,
                 max_pages=1 << 27, pages=8, page_size=8, kv_heads=128, head_dim=64)
    assert w4.lib().w4a4_paged_attention(cache, args, None) == 2


def test_attention_extreme_scores():
    """Scores up to +-1e4 (one token takes all), queries beyond fp16's range against an 8-bit cache."""
    lengths = [100, 1, 700]
    for dtype, act, mul in ((F16, F16, 300.0), (BF16, BF16, 3e4), (E4M3, BF16, 1e9), (E4M3, BF16, 1e-30)):
        c = Cache(lengths, 16, 2, 64, dtype, seed=8)
        q = (mul * randn(gen(9), 3, 4, 64)).to(act)
        check_attention(c, q, lengths, scale=1.0 if mul < 1e4 else 10.0 / mul, what=f"{dtype} {mul}")


def test_attention_infinities_and_nan():
    """-inf scores drop their tokens (all of them: an empty row); a NaN key, value or +inf
    score reaches the rows that see it and no other."""
    lengths = [40, 40, 40, 40]
    c = Cache(lengths, 16, 2, 64, F16, seed=10)
    at = lambda b, j: (int(c.table[b, j // 16]), j % 16)
    for j in range(40):
        p, s = at(0, j)
        c.k[p, s, 0, 0] = -math.inf       # sequence 0, head 0: every score -inf
        if j % 2:
            c.k[p, s, 1, 0] = -math.inf   # head 1: every second one
    p, s = at(1, 17)
    c.k[p, s, 0, 3] = float("nan")
    p, s = at(2, 39)
    c.v[p, s, 1, 5] = float("nan")
    c.to_gpu()
    q = randn(gen(11), 4, 4, 64).abs().to(F16)  # positive, so that q . k = -inf
    out, lse = attend(c, q, lengths)
    o, l, t, lt = attention_ref(q, c, lengths, 64 ** -0.5, 0)
    assert torch.all(out[0, :2] == 0) and torch.all(lse[0, :2] == -math.inf)
    assert torch.isnan(out[1, :2]).all() and torch.isnan(lse[1, :2]).all()
    assert torch.isnan(out[2, 2:, 5]).all()
    rest = [(0, slice(2, 4)), (1, slice(2, 4)), (2, slice(0, 2)), (3, slice(0, 4))]
    # head 1 of sequence 0: the reference over the finite tokens alone
    k, v = c.held(0, 0, 40)
    a = torch.einsum("gd,nd->gn", q[0, 2:].to(F64), k[::2, 1]) / 8
    o[0, 2:] = torch.softmax(a, -1) @ v[::2, 1]
    l[0, 2:] = torch.logsumexp(a, -1)
    for b, h in rest:
        mass = 64 * SLACK * 8
        check(out[b, h], o[b, h], t[b, h].nan_to_num(0, 0, 0) + (2 * u(F16) + mass) * 4, f"row {b}")
        check(lse[b, h], l[b, h], lt[b, h].nan_to_num(0, 0, 0) + mass, f"lse {b}")


def test_attention_bad_indices_are_left_out_and_reported():
    """Pages outside the pool, lengths outside the table: left out or clamped, and W4A4_ERR_INDEX."""
    lengths = [100, 60, 33]
    q = randn(gen(12), 3, 4, 128).to(F16)
    for bad in (-1, 1 << 20, -(1 << 31), (1 << 31) - 1):
        c = Cache(lengths, 16, 2, 128, F16, seed=13)
        c.table[0, 2], c.table[0, 6], c.table[2, 0] = bad, bad, bad
        c.to_gpu()
        check_attention(c, q, lengths, check_status=False, what=f"page {bad}")
        assert w4.w4a4_device_status() == w4.W4A4_ERR_INDEX
        assert w4.w4a4_device_status() == 0
    c = Cache([112, 60, 33], 16, 2, 128, F16, seed=14)
    for l0 in (-1, -(1 << 31), 113, (1 << 31) - 1):
        check_attention(c, q, [l0, 60, 33], check_status=False, what=f"length {l0}")
        assert w4.w4a4_device_status() == w4.W4A4_ERR_INDEX


def test_attention_strided_queries_other_streams_and_graphs():
    """q and out as slices of wider rows, a side stream, and a captured graph that follows the lengths."""
    lengths = [130, 70, 1]
    c = Cache([400] * 3, 16, 2, 64, F16, seed=15)
    wide_q = randn(gen(16), 3, 12, 64).to(F16)
    gq = wide_q.cuda()
    wide_out = torch.full((3, 9, 64), 7.0, dtype=F16, device="cuda")
    gl = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w4.w4a4_paged_attention(gq[:, 2:8], c.handle, gl, wide_out[:, 1:7])
    side.synchronize()
    o, _, t, _ = attention_ref(wide_q[:, 2:8], c, lengths, 0.125, 0)
    check(wide_out[:, 1:7], o, t, "strided")
    assert torch.all(wide_out[:, 0] == 7) and torch.all(wide_out[:, 7:] == 7)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.w4a4_paged_attention(gq[:, 2:8], c.handle, gl, wide_out[:, 1:7])
    for n in (0, 1, 64, 257, 400):
        gl.copy_(torch.tensor([n, 400 - n, n // 2], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        o, _, t, _ = attention_ref(wide_q[:, 2:8], c, [n, 400 - n, n // 2], 0.125, 0)
        check(wide_out[:, 1:7], o, t, f"graph {n}")
    assert w4.w4a4_device_status() == 0


def test_attention_tables_and_workspaces_it_refuses():
    """One row of the page table for all sequences (stride 0); a workspace first asked for inside a capture."""
    c = Cache([40, 40], 16, 2, 64, F16)
    q = randn(gen(35), 2, 4, 64).to(F16).cuda()
    n, out = torch.full((2,), 40, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    shared = w4.PagedKVCache(c.gk, c.gv, c.gt[:1].expand(2, -1))
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_paged_attention(q, shared, n, out)
    graph, raised = torch.cuda.CUDAGraph(), False
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        torch.zeros_like(q)
        try:
            w4.w4a4_paged_attention(q, c.handle, n, out)
        except w4.W4A4Error as e:
            raised = e.status == 4
    assert raised
    one = w4.PagedKVCache(c.gk, c.gv, c.gt[:1].as_strided((1, c.gt.shape[1]), (1, 1)))  # a single row's stride says nothing
    w4.w4a4_paged_attention(q[:1], one, n[:1], out[:1])
    torch.cuda.synchronize()
    o, _, t, _ = attention_ref(q[:1].cpu(), c, [40], 0.125, 0)
    check(out[:1], o, t, "one row")


def test_attention_offsets_beyond_32_bits():
    """Pages more than 2^31 elements apart (a pool among other data)."""
    page, hkv, dim, stride = 16, 2, 64, 1 << 29
    store = torch.empty(5 * stride + 2 * page * hkv * dim, dtype=F16, device="cuda")
    k = store.as_strided((6, page, hkv, dim), (stride, hkv * dim, dim, 1))
    v = store.as_strided((6, page, hkv, dim), (stride, hkv * dim, dim, 1), storage_offset=page * hkv * dim)
    c = Cache([96], page, hkv, dim, F16, seed=17, spare=0)
    k.copy_(c.k), v.copy_(c.v)
    c.handle = w4.PagedKVCache(k, v, c.gt)
    check_attention(c, randn(gen(18), 1, 4, dim).to(F16), [95])
    assert int((c.table[0].long() * stride).max()) > 1 << 31


def test_attention_refusals_of_the_binding():
    c = Cache([20], 16, 2, 64, F16)
    q = randn(gen(19), 1, 4, 64).to(F16).cuda()
    out, n = torch.empty_like(q), torch.ones(1, dtype=torch.int32, device="cuda")
    good = dict(q=q, cache=c.handle, lengths=n, out=out)
    for bad in (dict(q=q.float()), dict(q=q.bfloat16(), out=out.bfloat16()), dict(out=out[:, :2]), dict(q=q.cpu()),
                dict(lengths=n.long()), dict(lengths=n.repeat(2)), dict(lse=torch.zeros(1, 3, device="cuda")),
                dict(q=q[:, :3], out=out[:, :3]), dict(window=-1),
                dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")),
                dict(q=q[..., :32], out=out[..., :32])):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_paged_attention(**{**good, **bad})
    w4.w4a4_paged_attention(**good)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------- append
def append_ref(x, gain, rope, pos, rot, interleaved, eps):
    """(y, sum of the terms' absolute values) of heads [tokens, heads, dim] in 64 bits."""
    x = x.to(F64)
    if gain is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * gain.to(F64)
    if rope is None:
        return x, x.abs()
    c, s = rope[pos, 0].to(F64)[:, None], rope[pos, 1].to(F64)[:, None]
    y, mass = x.clone(), x.abs()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mass[..., ia], mass[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, mass


def stored_tol(ref, mass, dtype):
    return u(dtype) * (ref.abs() + SLACK * mass) + tiny(dtype) + SLACK * mass


def run_append(act, dtype, dim, rot, interleaved, norm, page, layout, seed, lengths, new, hq, hkv, in_place=False,
               scales=True):
    """Appends the last new[b] tokens of each sequence (in a shuffled order) and checks every slot."""
    g = gen(seed)
    c = Cache(lengths, page, hkv, dim, dtype, seed=seed, layout=layout, scales=scales)
    before_k, before_v = c.gk.clone(), c.gv.clone()
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)])
    pos = torch.cat([torch.arange(l - n, l) for l, n in zip(lengths, new)])
    order = torch.randperm(len(seq), generator=g)
    seq, pos = seq[order], pos[order]
    T = len(seq)
    qkv = (randn(g, T, hq + 2 * hkv, dim) * (8 if dtype != E4M3 else 1)).to(act)
    gains = [(1 + 0.3 * randn(g, dim)).to(act) if norm else None for _ in range(2)]
    rope = None
    if rot:
        ang = torch.arange(max(lengths), dtype=F64)[:, None] * 1e4 ** (-torch.arange(rot // 2, dtype=F64) / (rot // 2))
        rope = torch.stack((ang.cos(), ang.sin()), 1).float()
    dev = qkv.cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    q_out = q if in_place else torch.full((T, hq, dim), float("nan"), dtype=act, device="cuda")
    w4.w4a4_kv_append(q, k, v, pos.int().cuda(), c.handle, q_out, seqs=seq.int().cuda(),
                      rope=None if rope is None else rope.cuda(),
                      q_gain=None if not norm else gains[0].cuda(), k_gain=None if not norm else gains[1].cuda(),
                      eps=1e-5, interleaved=interleaved)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0
    ref, mass = append_ref(qkv[:, :hq], gains[0], rope, pos, rot, interleaved, 1e-5)
    check(q_out, ref, stored_tol(ref, mass, act), "q")
    page_of, slot = c.table[seq, pos // page].long(), pos % page
    for got, before, x, gain, s, turn in ((c.gk, before_k, qkv[:, hq:hq + hkv], gains[1], c.ks, rope),
                                          (c.gv, before_v, qkv[:, hq + hkv:], None, c.vs, None)):
        ref, mass = append_ref(x, gain, turn, pos, rot, interleaved, 1e-5)
        if dtype == E4M3:
            s = torch.ones(hkv) if s is None else s
            ref, mass = ref / s.to(F64)[:, None], mass / s.to(F64)[:, None]
            ref = ref.clamp(-448, 448)
        check(got.float().cpu()[page_of, slot], ref, stored_tol(ref, mass, dtype), "pool")
        now, was = got.float().cpu(), before.float().cpu()
        now[page_of, slot] = was[page_of, slot]
        assert torch.equal(now.nan_to_num(nan=1e9), was.nan_to_num(nan=1e9)), "another slot was touched"


@pytest.mark.parametrize("act, dtype", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("dim, rot, interleaved", [(64, 64, False), (96, 96, False), (96, 32, True), (128, 128, False),
                                                   (128, 128, True), (128, 48, False), (256, 256, False), (256, 64, True),
                                                   (128, 0, False)])
@pytest.mark.parametrize("norm", [False, True])
def test_append_types_and_rotations(act, dtype, dim, rot, interleaved, norm):
    run_append(act, dtype, dim, rot, interleaved, norm, 16, "NHD", dim + rot, [40, 1, 17, 90], [7, 1, 0, 60], 6, 2)


@pytest.mark.parametrize("page, layout, hq, hkv", [(1, "NHD", 1, 1), (7, "HND", 40, 5), (64, "HND", 3, 3), (100, "NHD", 37, 1)])
def test_append_layouts_and_heads(page, layout, hq, hkv):
    run_append(F16, F16, 128, 128, False, True, page, layout, page, [333, 64, 5], [333, 1, 2], hq, hkv)
    run_append(BF16, E4M3, 64, 64, False, False, page, layout, page, [33, 64, 5], [30, 1, 2], hq, hkv, scales=False)


def test_append_one_token_and_in_place():
    run_append(F16, F16, 128, 128, False, True, 16, "NHD", 3, [701], [1], 16, 8)
    run_append(F16, F16, 128, 128, False, True, 16, "NHD", 4, [701, 9], [1, 3], 16, 8, in_place=True)
    run_append(BF16, BF16, 96, 96, False, True, 16, "NHD", 5, [71, 9], [50, 3], 4, 4, in_place=True)


def test_append_defaults_padding_and_bad_indices():
    """seqs None: token t of sequence t.  Padding stores nothing and zeroes its query row; so does an
    index outside its table, which is reported as well."""
    c = Cache([20, 20, 20, 20], 8, 2, 64, F16, seed=20, fill=False)
    g = gen(21)
    qkv = randn(g, 4, 8, 64).to(F16).cuda()
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    rope = w4.w4a4_rope_table(20, 64, 1e4)
    out = torch.full((4, 4, 64), 5.0, dtype=F16, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    w4.w4a4_kv_append(q, k, v, i32(0, 7, 8, 19), c.handle, out, rope=rope)
    assert w4.w4a4_device_status() == 0
    want = out.clone()
    assert torch.equal(out[0], q[0])  # position 0 does not turn
    for s, p in enumerate((0, 7, 8, 19)):
        assert torch.equal(c.gv[c.table[s, p // 8], p % 8], v[s])
    snap_k, snap_v = c.gk.clone(), c.gv.clone()

    def same():
        return torch.equal(c.gk.nan_to_num(9), snap_k.nan_to_num(9)) and torch.equal(c.gv.nan_to_num(9), snap_v.nan_to_num(9))

    w4.w4a4_kv_append(q, k, v, i32(0, 7, 8, 19), c.handle, out, rope=rope, seqs=i32(-1, 1, -5, 3))
    assert w4.w4a4_device_status() == 0 and same()
    assert torch.all(out[0] == 0) and torch.all(out[2] == 0) and torch.equal(out[1], want[1]) and torch.equal(out[3], want[3])
    for pos, seqs in (((0, 7, -1, 20), (0, 1, 2, 3)), ((0, 7, 1 << 30, 24), (0, 1, 2, 3)), ((0, 7, 8, 19), (0, 1, 4, 1 << 30))):
        out.fill_(5.0)
        w4.w4a4_kv_append(q, k, v, i32(*pos), c.handle, out, rope=rope, seqs=i32(*seqs))
        assert w4.w4a4_device_status() == w4.W4A4_ERR_INDEX and same(), (pos, seqs)
        assert torch.all(out[2:] == 0) and torch.equal(out[:2], want[:2])
    for bad in (-1, 1 << 20, c.k.shape[0]):
        c.gt[2, 1] = bad
        out.fill_(5.0)
        w4.w4a4_kv_append(q, k, v, i32(0, 7, 8, 19), c.handle, out, rope=rope)
        assert w4.w4a4_device_status() == w4.W4A4_ERR_INDEX and same()
        assert torch.all(out[2] == 0) and torch.equal(out[3], want[3])
    w4.w4a4_kv_append(q[:0], k[:0], v[:0], i32(), c.handle, out[:0], rope=rope)  # no tokens: nothing
    assert w4.w4a4_device_status() == 0 and same()


def test_append_special_values():
    """NaN stays NaN and infinities saturate in an 8-bit cache; a zero head normalises to zero."""
    c = Cache([4], 8, 1, 64, E4M3, seed=22, scales=False, fill=False)
    x = torch.zeros(1, 3, 64, dtype=F16)
    x[0, 1, :4] = torch.tensor([float("nan"), math.inf, -math.inf, 1000.0])
    x[0, 2, :4] = torch.tensor([-1000.0, 2 ** -9, 2 ** -10, 3 * 2 ** -10])
    d = x.cuda()
    out = torch.full((1, 1, 64), 3.0, dtype=F16, device="cuda")
    one = torch.ones(64, dtype=F16, device="cuda")
    w4.w4a4_kv_append(d[:, :1], d[:, 1:2], d[:, 2:], torch.zeros(1, dtype=torch.int32, device="cuda"), c.handle, out,
                      q_gain=one)
    k, v = (p.float().cpu()[c.table[0, 0], 0, 0, :4] for p in (c.gk, c.gv))
    assert torch.all(out == 0)
    assert torch.isnan(k[0]) and k[1:].tolist() == [448.0, -448.0, 448.0]
    assert v.tolist() == [-448.0, 2 ** -9, 0.0, 2 ** -8]  # ties to even


def test_rope_table_far_positions():
    """Angles in 64 bits: the far end of a long table is as exact as its start."""
    rows, rot = 200001, 128
    got = w4.w4a4_rope_table(rows, rot, 1e6).cpu()
    pos = torch.tensor([0, 1, 2, 4095, 65537, 131071, rows - 1])
    ang = pos.to(F64)[:, None] * 1e6 ** (-torch.arange(rot // 2, dtype=F64) * 2 / rot)
    for i, ref in ((0, ang.cos()), (1, ang.sin())):
        check(got[pos, i], ref, u(F32) * ref.abs() + 2.0 ** -32, "rope")


def test_append_then_attend():
    """What was appended is what attention reads: a step of three sequences against the definition."""
    lengths, dim, hq, hkv = [65, 1, 130], 128, 16, 8
    c = Cache(lengths, 16, hkv, dim, F16, seed=23)
    g = gen(24)
    qkv = randn(g, 3, hq + 2 * hkv, dim).to(F16).cuda()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q = torch.empty(3, hq, dim, dtype=F16, device="cuda")
    rope = w4.w4a4_rope_table(200, dim, 1e6)
    w4.w4a4_kv_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], n - 1, c.handle, q, rope=rope)
    c.k, c.v = c.gk.cpu(), c.gv.cpu()
    assert torch.equal(c.v[c.table[2, 8], 129 % 16], qkv[2, hq + hkv:].cpu())
    check_attention(c, q.cpu(), lengths)


# ------------------------------------------------------------------ block norm
def norm_ref(x, kind, gain, bias, eps):
    """(norm, factor from an error of x to one of the norm) in 64 bits."""
    if kind == w4.NORM_NONE:
        return x, torch.ones_like(x)
    mean = x.mean(-1, keepdim=True) if kind == w4.NORM_LAYER else 0.0
    inv = 1 / ((x - mean).pow(2).mean(-1, keepdim=True) + eps).sqrt()
    g = torch.ones(x.shape[-1], dtype=F64) if gain is None else gain.to(F64)
    y = (x - mean) * inv * g
    return (y + bias.to(F64) if bias is not None and kind == w4.NORM_LAYER else y), (inv * g.abs()).expand_as(x)


def check_norm(act, res, rows, width, post, pre, gate, scale=0.7, gains=True, biases=True, want_x=True, in_place=False,
               pad=0, shift=0.0, seed=0, per=3):
    g = gen(seed)
    y, r = (3 * randn(g, rows, width + pad) + shift).to(act), (4 * randn(g, rows, width + pad) - shift).to(res)
    y_in, r_in = y[:, :width], r[:, :width]
    gates = {"none": None, "shared": randn(g, width).to(act), "rows": randn(g, max(1, -(-rows // per)), width + pad).to(act)}[gate]
    v = lambda on, base: (base + 0.3 * randn(g, width)).to(act) if on else None
    pg, pb, ng, nb = v(gains, 1), v(biases, 0), v(gains, 1), v(biases, 0)
    dev = lambda t: None if t is None else t.cuda()
    gy, gr = dev(y)[:, :width], dev(r)[:, :width]
    gg = dev(gates)[:, :width] if gate == "rows" else dev(gates)
    x = torch.full((rows, width + pad), float("nan"), dtype=act, device="cuda")[:, :width] if want_x else None
    r_out = gr if in_place else torch.full((rows, width), float("nan"), dtype=res, device="cuda")
    w4.w4a4_block_norm(gy, gr, x, r_out, gate=gg, rows_per_gate=per if gate == "rows" else 0, scale=scale, post=post,
                       post_gain=dev(pg), post_bias=dev(pb), pre=pre, pre_gain=dev(ng), pre_bias=dev(nb), eps=1e-5)
    torch.cuda.synchronize()
    y64, r64 = y_in.to(F64), r_in.to(F64)
    block, slope = norm_ref(y64, post, pg, pb, 1e-5)
    # fp32 steps of a norm: relative to its terms, the mean's own terms among them
    b_err = SLACK * (block.abs() + slope * (y64.abs() + y64.abs().mean(-1, keepdim=True)))
    if gate != "none":
        gv = gates.to(F64) if gate == "shared" else gates.to(F64)[:, :width][torch.arange(rows) // per]
        block, b_err = block * gv, b_err * gv.abs()
    block, b_err = block * scale, b_err * abs(scale)
    ref = r64 + block
    r_err = b_err + SLACK * (r64.abs() + block.abs())
    check(r_out, ref, r_err + u(res) * (ref.abs() + r_err) + tiny(res), "r")
    if want_x:
        nx, slope = norm_ref(ref, pre, ng, nb, 1e-5)
        # an error of one element moves its own output, and all through the mean and the scale
        spread = (r_err.mean(-1, keepdim=True) + r_err) * slope
        spread = spread + nx.abs() * (r_err * ref.abs()).mean(-1, keepdim=True) / (ref.pow(2).mean(-1, keepdim=True) + 1e-30) \
            if pre != w4.NORM_LAYER else spread + nx.abs() * slope * (r_err.mean(-1, keepdim=True) + r_err)
        t = spread + SLACK * (nx.abs() + slope * (ref.abs() + ref.abs().mean(-1, keepdim=True)))
        check(x, nx, t + u(act) * (nx.abs() + t) + tiny(act), "x")


@pytest.mark.parametrize("act, res", [(F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)])
@pytest.mark.parametrize("post", [0, 1, 2])
@pytest.mark.parametrize("pre", [0, 1, 2])
@pytest.mark.parametrize("gate", ["none", "shared", "rows"])
def test_norm_kinds(act, res, post, pre, gate):
    check_norm(act, res, 7, 1024, post, pre, gate, seed=post * 3 + pre)


@pytest.mark.parametrize("width", [8, 72, 256, 264, 1000, 1024, 1032, 2048, 2056, 4096, 5000, 8192, 8200, 16384])
@pytest.mark.parametrize("rows", [1, 33])
def test_norm_widths(width, rows):
    check_norm(F16, F16, rows, width, 1, 1, "rows", seed=width)
    check_norm(BF16, F32, rows, width, 2, 2, "shared", seed=width)


@pytest.mark.parametrize("rows, width", [(1301, 1024), (1500, 520), (20011, 64), (9001, 200), (5003, 512), (2503, 2048),
                                         (1999, 4096), (400, 16384)])
def test_norm_many_rows(rows, width):
    """More rows than CTAs hold at once: each takes several, with the next one's loads in flight."""
    check_norm(F16, F16, rows, width, 1, 1, "rows", seed=rows, per=7)
    check_norm(BF16, F32, rows, width, 2, 2, "shared", seed=rows, in_place=True)


def test_norm_options():
    check_norm(F16, F16, 700, 1024, 1, 1, "none", scale=1.0, gains=False, biases=False)
    check_norm(F16, F16, 50, 512, 2, 2, "rows", pad=24)
    check_norm(F16, F32, 50, 512, 1, 2, "rows", pad=8, in_place=True, per=1000)
    check_norm(BF16, BF16, 9, 256, 1, 1, "shared", in_place=True)
    check_norm(F16, F16, 9, 256, 2, 1, "shared", want_x=False)
    check_norm(F16, F32, 9, 2048, 2, 2, "none", shift=500.0)  # a mean far above the spread
    check_norm(F16, F16, 0, 256, 1, 1, "none")


def test_norm_special_rows():
    """A zero row stays zero through both norms; a NaN or infinity stays in its row."""
    y = torch.zeros(4, 128, dtype=F16)
    r = torch.zeros(4, 128, dtype=F16)
    y[1, 5], r[2, 7], y[3] = float("nan"), math.inf, 2.0
    x, ro = torch.empty_like(y).cuda(), torch.empty_like(r).cuda()
    w4.w4a4_block_norm(y.cuda(), r.cuda(), x, ro)
    assert torch.all(ro[0] == 0) and torch.all(x[0] == 0)
    assert torch.isnan(ro[1]).all() and torch.isnan(x[1]).all()
    assert ro[2, 7] == math.inf and torch.isnan(x[2, 7]) and torch.all(ro[2, :7] == 0)
    assert torch.all((ro[3] - 1).abs() <= 2 ** -11) and torch.all((x[3] - 1).abs() <= 2 ** -11)


@pytest.mark.parametrize("width", [1032, 1200, 1536, 1544, 2288, 2560, 3064, 3080, 4104, 5120, 6144, 6152])
@pytest.mark.parametrize("rows", [1, 40, 1999])
def test_norm_widths_between_powers_of_two(width, rows):
    check_norm(F16, F16, rows, width, 2, 1, "rows", seed=width)
    check_norm(BF16, F32, rows, width, 1, 2, "none", seed=width, in_place=True)


@pytest.mark.parametrize("rows, width", [(6, 64), (6, 120), (6, 200), (6, 512), (6, 1000), (1301, 1000), (6, 1536), (6, 2288),
                                         (6, 4096), (6, 4104), (6, 8192), (6, 16384)])
def test_layernorm_of_rows_far_from_their_first_elements(rows, width):
    """The statistics are summed about a row's first eight elements and joined about its first warp's mean.

    With squares (p - mean)^2 <= 128 variances at the pivot and 16 at the join, each rounding of the sums (a depth of
    20) counts 146 times against the variance, half of that against its root."""
    g = gen(width)
    r = randn(g, rows, width)
    r[0, :8] += 1000.0
    r[1] += 30000.0
    r[2, : width // 2] -= 500.0
    r[3] = 7.25
    r[4, -8:] -= 2000.0
    if rows > 6:
        r[6:, :8] += 100.0 * torch.arange(rows - 6)[:, None]
    y = torch.zeros(rows, width, dtype=F16)
    x = torch.empty_like(y).cuda()
    w4.w4a4_block_norm(y.cuda(), r.cuda(), x, torch.empty_like(r).cuda(), post=w4.NORM_NONE, pre=w4.NORM_LAYER, eps=1e-5)
    nx, slope = norm_ref(r.to(F64), w4.NORM_LAYER, None, None, 1e-5)
    t = nx.abs() * 146 * 20 / 2 * u(F32) + SLACK * (nx.abs() + slope * (r.abs().to(F64) + r.abs().to(F64).mean(-1, keepdim=True)))
    check(x, nx, t + u(F16) * (nx.abs() + t) + tiny(F16), "x")


@pytest.mark.parametrize("width", [64, 512, 1536, 4096])
def test_layernorm_special_rows(width):
    """NaN and infinities, at the pivot or not, make their own row NaN and no other."""
    r = randn(gen(width), 8, width).to(F16)
    r[0, 0], r[1, -1], r[2, 3], r[3, width // 2], r[5] = float("nan"), float("nan"), math.inf, -math.inf, 0.0
    y = torch.zeros_like(r)
    x = torch.empty_like(r).cuda()
    w4.w4a4_block_norm(y.cuda(), r.cuda(), x, torch.empty_like(r).cuda(), post=w4.NORM_NONE, pre=w4.NORM_LAYER)
    assert torch.isnan(x[:4]).all() and torch.isfinite(x[4:]).all() and torch.all(x[5] == 0)


def test_norm_refusals_of_the_binding():
    y = torch.zeros(4, 64, dtype=F16, device="cuda")
    good = dict(y=y, r=y, x=y.clone(), r_out=y.clone())
    for bad in (dict(r=y.bfloat16()), dict(r=y.bfloat16(), r_out=y.bfloat16()), dict(x=y.float()), dict(r=y[:2]),
                dict(gate=y[0].float()), dict(gate=y[:1], rows_per_gate=2), dict(gate=y[0, :32]),
                dict(pre_gain=y[0, :8]), dict(post=5), dict(y=y.t(), r=y.t(), x=y.t(), r_out=y.t()), dict(r=y.cpu())):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_block_norm(**{**good, **bad})
    w4.w4a4_block_norm(**good)
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens", [2500, 3100, 4200, 5600])
def test_append_tokens_that_share_ctas_out(tokens):
    """Many tokens of many heads: one or two CTAs a token, by how full the GPU's last time over is."""
    run_append(F16, F16, 64, 64, False, True, 64, "NHD", tokens, [tokens - 697, 700], [tokens - 700, 700], 56, 4)


@pytest.mark.parametrize("seqs, longest, hkv, group, dim, dtype, window", [
    (200, 588, 1, 16, 96, E4M3, 400), (140, 300, 2, 4, 128, F16, 0), (152, 700, 1, 1, 64, F16, 0), (300, 200, 1, 4, 128, BF16, 0),
    (150, 900, 1, 7, 256, E4M3, 0), (440, 150, 1, 2, 64, E4M3, 100), (1000, 70, 1, 2, 64, F16, 0)])
def test_attention_short_runs_of_many_sequences(seqs, longest, hkv, group, dim, dtype, window):
    """More sequences than a CTA has threads, some empty, some long: single pieces as long as there are CTAs for them."""
    g = gen(seqs)
    lengths = torch.randint(0, longest + 1, (seqs,), generator=g).tolist()
    lengths[0], lengths[1], lengths[-1], lengths[-2] = 0, 4 * longest, longest, 0
    c = Cache(lengths, 16, hkv, dim, dtype, seed=seqs)
    check_attention(c, randn(g, seqs, hkv * group, dim).to(BF16 if dtype == BF16 else F16), lengths, window=window)
    c = Cache([longest] * seqs, 16, hkv, dim, dtype, seed=seqs)
    check_attention(c, randn(g, seqs, hkv * group, dim).to(BF16 if dtype == BF16 else F16), [longest] * seqs, window=window)
