"""The cache, attention and norm operators as a server uses them: workspaces shared and dropped, host threads,
streams, devices, strides that no index uses; and values at the borders of their types.

References and tolerances as in test_layer_ops_gpu."""
import ctypes
import math
import re
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


def test_append_to_an_8_bit_cache_divides_by_the_scale():
    """The stored code is that of the quotient y / scale: ties go to even, and the smallest scales keep zeros."""
    hkv = 6
    c = Cache([64], 16, hkv, 64, E4M3, seed=68, fill=False)
    scale = torch.tensor([3 / 64, 5 / 64, 7 / 64, 49 / 1024, 0.7, 2.0 ** -130])
    c.ks, c.vs = scale, scale.flip(0).contiguous()
    c.to_gpu()
    ties = torch.tensor([m + 0.5 for m in range(8, 16)])  # halfway between neighbours of E4M3
    x = torch.empty(64, hkv, 64)
    for h in range(hkv):
        e = torch.arange(64) % 4
        x[:, h] = torch.where(torch.rand(64, 64, generator=gen(h)) < 0.5, 1.0, -1.0) * ties[torch.arange(64) % 8] * 2.0 ** -e * (
            scale[h] if h < 5 else 1.0)
    x[::3, 5] = 0.0
    x = x.to(F16)
    xv = x.flip(1).contiguous()
    tok = torch.arange(64, dtype=torch.int32, device="cuda")
    none = torch.empty(64, 0, 64, dtype=F16, device="cuda")
    w4.w4a4_kv_append(none, x.cuda(), xv.cuda(), tok, c.handle, none, seqs=torch.zeros_like(tok))
    torch.cuda.synchronize()
    at = c.table[0, torch.arange(64) // 16].long(), torch.arange(64) % 16
    for pool, y, s in ((c.gk, x, c.ks), (c.gv, xv, c.vs)):
        want = (y.float() / s[:, None]).clamp(-448, 448).to(E4M3).float()
        assert torch.equal(pool.float().cpu()[at], want)

    # bf16 rows over fp32's range, and scales at its ends, zero among them
    scale = torch.tensor([2.0 ** 120, 3e-30, 1.1, 0.0, 1.7e38, 2.0 ** -149])
    c.ks.copy_(scale), c.vs.copy_(scale.flip(0))
    c.to_gpu()
    x = randn(gen(9), 64, hkv, 64) * 10.0 ** (60 * torch.rand(64, hkv, 64, generator=gen(10)) - 30)
    x[0], x[1], x[2], x[3] = 0.0, math.inf, -math.inf, float("nan")
    x[4:, 2] = 300 * randn(gen(11), 60, 64)
    x = x.to(BF16)
    w4.w4a4_kv_append(none.to(BF16), x.cuda(), x.cuda(), tok, c.handle, none.to(BF16), seqs=torch.zeros_like(tok))
    torch.cuda.synchronize()
    for pool, s in ((c.gk, c.ks), (c.gv, c.vs)):
        want = (x.float() / s[:, None]).clamp(-448, 448).to(E4M3).float()
        assert torch.equal(pool.float().cpu()[at].nan_to_num(nan=1e9), want.nan_to_num(nan=1e9))
    assert w4.w4a4_device_status() == 0


def test_operators_called_first_in_a_fresh_thread():
    """A thread whose first CUDA work is one of the operators, on tensors that another thread made."""
    c = Cache([40], 16, 2, 64, F16, seed=62)
    c.handle.workspace(4)
    qkv = randn(gen(63), 1, 8, 64).to(F16).cuda()
    pos, n = torch.tensor([39], dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda")
    y = randn(gen(64), 3, 64).to(F16).cuda()

    def run(op):
        q, out = torch.zeros(1, 4, 64, dtype=F16, device="cuda"), torch.zeros(1, 4, 64, dtype=F16, device="cuda")
        x, r = torch.zeros_like(y), torch.zeros_like(y)
        torch.cuda.synchronize()
        calls = {"append": lambda: w4.w4a4_kv_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], pos, c.handle, q),
                 "attend": lambda: w4.w4a4_paged_attention(qkv[:, :4], c.handle, n, out),
                 "norm": lambda: w4.w4a4_block_norm(y, y, x, r)}
        return calls[op], (q, out, x, r)

    for op in ("append", "attend", "norm"):
        call, want = run(op)
        call()  # handles, attributes and sizes are known from here on
        call, got = run(op)
        raised = []

        def body():
            try:
                call()
            except BaseException as e:
                raised.append(e)

        t = threading.Thread(target=body)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not raised, (op, raised)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), op


def on_device(t, index):
    """`t`'s memory as a tensor that says it is on GPU `index`."""
    class Tensor(ctypes.Structure):
        _fields_ = [("data", ctypes.c_void_p), ("device_type", ctypes.c_int32), ("device_id", ctypes.c_int32),
                    ("ndim", ctypes.c_int32), ("code", ctypes.c_uint8), ("bits", ctypes.c_uint8), ("lanes", ctypes.c_uint16),
                    ("shape", ctypes.POINTER(ctypes.c_int64)), ("strides", ctypes.POINTER(ctypes.c_int64)),
                    ("byte_offset", ctypes.c_uint64)]

    class Managed(ctypes.Structure):
        _fields_ = [("t", Tensor), ("ctx", ctypes.c_void_p), ("deleter", ctypes.c_void_p)]

    shape, strides = (ctypes.c_int64 * t.dim())(*t.shape), (ctypes.c_int64 * t.dim())(*t.stride())
    code = 2 if t.is_floating_point() else 0
    m = Managed(Tensor(t.data_ptr(), 2, index, t.dim(), code, 8 * t.element_size(), 1, shape, strides, 0), None, None)
    on_device.kept = getattr(on_device, "kept", []) + [(m, shape, strides, t)]
    new = ctypes.pythonapi.PyCapsule_New
    new.restype, new.argtypes = ctypes.py_object, [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p]
    return torch.utils.dlpack.from_dlpack(new(ctypes.addressof(m), b"dltensor", None))


def test_operators_do_not_run_on_another_device_than_their_tensors():
    """Tensors that name another GPU than the current one, and a stream's handle, which says nothing of a device."""
    there = torch.cuda.device_count()  # a GPU that the machine does not have; the memory is the current one's
    y = torch.zeros(4, 64, dtype=F16, device="cuda")
    x, r = torch.zeros_like(y), torch.zeros_like(y)
    a = [on_device(t, there) for t in (y, y, x, r)]
    assert all(t.get_device() == there for t in a)
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_block_norm(*a, stream=0)
    assert torch.cuda.current_device() == 0


def test_strides_that_no_index_uses():
    """One row, token or head: its stride is whatever torch left there."""
    g = gen(70)
    wide = randn(g, 4, 67).to(F16).cuda()
    y, r = wide[:1, :64], torch.randn(64, 1, generator=g).cuda().t()  # strides 67 and 1
    x, ro = torch.empty(1, 64, dtype=F16, device="cuda"), torch.empty(1, 64, device="cuda")
    want_x, want_r = torch.empty_like(x), torch.empty_like(ro)
    w4.w4a4_block_norm(y, r, x, ro, gate=wide[:1, :64], rows_per_gate=5)
    w4.w4a4_block_norm(y.clone(), r.clone(memory_format=torch.contiguous_format), want_x, want_r, gate=y.clone())
    assert torch.equal(x, want_x) and torch.equal(ro, want_r)

    c = Cache([40], 16, 2, 64, F16, seed=71)
    rows = randn(g, 2, 8 * 64 + 1).to(F16).cuda()
    q = rows[:1, :256].unflatten(1, (4, 64))  # a token stride of 513
    n, pos = torch.tensor([40], dtype=torch.int32, device="cuda"), torch.tensor([39], dtype=torch.int32, device="cuda")
    out = torch.empty(2, 4 * 64 + 3, dtype=F16, device="cuda")[:1, :256].unflatten(1, (4, 64))
    w4.w4a4_paged_attention(q, c.handle, n, out)
    check(out, attention_ref(q.cpu(), c, [40], 0.125, 0)[0], attention_ref(q.cpu(), c, [40], 0.125, 0)[2], "one sequence")
    k, v = rows[:1, 256:384].unflatten(1, (2, 64)), rows[:1, 384:512].unflatten(1, (2, 64))
    w4.w4a4_kv_append(q, k, v, pos, c.handle, out)
    assert torch.equal(out, q) and torch.equal(c.gk[c.table[0, 2], 7], k[0]) and torch.equal(c.gv[c.table[0, 2], 7], v[0])

    one = torch.randn(3, 16, 65, generator=g).to(F16).cuda()[:1, :, :64].unsqueeze(2)  # one page of one head, odd strides
    pool = one.as_strided((1, 16, 1, 64), (1041, 64, 3, 1))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    n = torch.tensor([16], dtype=torch.int32, device="cuda")
    got, want = torch.empty(1, 1, 64, dtype=F16, device="cuda"), torch.empty(1, 1, 64, dtype=F16, device="cuda")
    w4.w4a4_paged_attention(q[:, :1], w4.PagedKVCache(pool, pool, table), n, got)
    w4.w4a4_paged_attention(q[:, :1].clone(), w4.PagedKVCache(pool.clone(memory_format=torch.contiguous_format),
                                                              pool.clone(memory_format=torch.contiguous_format), table), n, want)
    assert torch.equal(got, want)
    assert w4.w4a4_device_status() == 0


def test_attention_workspace_outlives_the_cache_object():
    """A cache object dropped while a side stream still runs its attention: the memory of its workspace is not
    handed out before that has ended."""
    c = Cache([700], 16, 2, 64, F16, seed=60)
    q = randn(gen(61), 1, 4, 64).to(F16).cuda()
    n, out = torch.full((1,), 700, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    side = torch.cuda.Stream()
    for given in (False, True):  # the side stream as the current one, and as an argument
        handle = w4.PagedKVCache(c.gk, c.gv, c.gt)
        ws = handle.workspace(4)
        at, size = ws.data_ptr(), ws.numel()
        del ws
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # a tenth of a second
            if not given:
                w4.w4a4_paged_attention(q, handle, n, out)
        if given:
            w4.w4a4_paged_attention(q, handle, n, out, stream=side)
        del handle
        again = torch.empty(size, dtype=torch.uint8, device="cuda")
        busy = not side.query()
        torch.cuda.synchronize()
        assert busy and again.data_ptr() != at
        del again


def test_rope_table_made_on_a_side_stream():
    """The table's memory belongs to the stream that fills it: no memory whose last use on the current stream is
    still to come."""
    rows, rot = 4096, 128
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        held = torch.full((rows, 2, rot // 2), 7.0, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)
        copy = held.clone()
        del held
        table = w4.w4a4_rope_table(rows, rot, 1e4, stream=stream)
        torch.cuda.synchronize()
        assert torch.all(copy == 7)
        assert torch.equal(table, w4.w4a4_rope_table(rows, rot, 1e4))
        del copy, table


def test_numbers_outside_an_int_are_refused():
    y = torch.zeros(4, 64, dtype=F16, device="cuda")
    for over in (dict(post=1 << 32), dict(pre=(1 << 32) + 2), dict(post=-(1 << 32))):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_block_norm(y, y, y.clone(), y.clone(), **over)


def heads_of_a_unit():
    return int(re.search(r"heads/unit=(\d+)", w4.w4a4_last_dispatch()).group(1))


@pytest.mark.parametrize("dtype, dim, hkv, group, side_by_side", [
    (F16, 256, 2, 11, 4), (E4M3, 256, 1, 16, 2), (F16, 256, 3, 9, 2),       # chunks of 8 query heads, the last one short
    (F16, 64, 2, 37, 2), (BF16, 128, 2, 20, 2), (E4M3, 96, 4, 17, 2),       # chunks of 16
    (F16, 96, 4, 3, 4), (E4M3, 64, 6, 3, 2), (E4M3, 128, 8, 5, 4), (BF16, 64, 2, 8, 2)])  # adjacent heads
def test_attention_chunks_side_by_side(dtype, dim, hkv, group, side_by_side):
    """Tables with room for much work: the warps of a CTA take several chunks of heads and the same tokens."""
    lengths = [100, 3, 3000, 64, 0, 17]
    c = Cache(lengths, 64, hkv, dim, dtype, seed=dim + group, wide=40000)
    q = randn(gen(72), len(lengths), hkv * group, dim).to(BF16 if dtype == BF16 else F16)
    check_attention(c, q, lengths, what=f"{dtype} {dim} {hkv}x{group}")
    assert heads_of_a_unit() == side_by_side


@pytest.mark.parametrize("dtype, dim, tokens", [(F16, 128, 16), (E4M3, 64, 32)])
def test_attention_one_step_a_sequence_of_more_than_the_ctas(dtype, dim, tokens):
    lengths = [tokens] * 90 + [1, 0, 5] * 30
    c = Cache(lengths, tokens, 4, dim, dtype, seed=73)
    check_attention(c, randn(gen(74), len(lengths), 8, dim).to(F16), lengths)
    assert heads_of_a_unit() == 4


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim, group", [(64, 2), (128, 12), (256, 3)])
def test_attention_weights_keep_more_bits_than_their_type(dtype, dim, group):
    """Tokens of weight 1 and value 1 beside tokens whose weight w, next below 1, rounds to 1, and of value -1: the
    output is (1 - w) / (1 + w), all of it what the weights' rounding would take away.

    Rounded twice, a weight is off by u^2 at most; fp32 sums of 256 terms by 256 roundings of 2^-24; the output is
    rounded once."""
    tokens, page = 256, 16
    w = 1 - 0.35 * torch.finfo(dtype).eps / 2
    k = torch.zeros(tokens // page, page, 1, dim)
    v = torch.ones_like(k)
    k[:, 1::2, 0, 0], v[:, 1::2] = -1.0, -1.0
    table = torch.arange(tokens // page, dtype=torch.int32).repeat(2, 1).cuda()
    handle = w4.PagedKVCache(k.to(dtype).cuda(), v.to(dtype).cuda(), table)
    q = torch.zeros(2, group, dim)
    q[..., 0] = 1.0
    n = torch.full((2,), tokens, dtype=torch.int32, device="cuda")
    out = torch.empty(2, group, dim, dtype=dtype, device="cuda")
    w4.w4a4_paged_attention(q.to(dtype).cuda(), handle, n, out, scale=-math.log(w))
    torch.cuda.synchronize()
    ref = torch.full(out.shape, (1 - w) / (1 + w), dtype=F64)
    err = u(dtype) ** 2 + 2.0 ** -16
    check(out, ref, ref * u(dtype) + err * (1 + u(dtype)) + tiny(dtype), f"{dtype}")
