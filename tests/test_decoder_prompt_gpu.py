"""The decoder layer's pass over whole prompts and over chunks into the cache: what lies between the quantised
linears, from the linears' own outputs, against definitions in 64 bits; chunks of a prompt against the whole of
it; and a decode step after them."""
import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.test_decoder_gpu import F64, U16, close, rms, turn
from w4a4_quantized_gemm_gb300 import decoder

pytestmark = pytest.mark.gpu
HIDDEN, HQ, HKV, DIM = 512, 8, 2, 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()
    w4.w4a4_device_status()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def layer_and_inputs(rows, seqs, seed):
    layer = decoder.random_layer(HIDDEN, 640, HQ, HKV, DIM, seqs)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    return layer, rand(rows, HIDDEN).half(), 3 * rand(rows, HIDDEN), (1 + 0.1 * rand(HIDDEN)).half()


def attended(q, k, v, first):
    """Causal attention in 64 bits of q [n, heads, dim], row i at place first + i, over k, v [keys, heads, dim]."""
    k, v = (x.repeat_interleave(HQ // HKV, dim=1) for x in (k, v))
    a = torch.einsum("ihd,jhd->hij", q, k) * DIM ** -0.5
    place = first + torch.arange(q.shape[0], device="cuda")
    a.masked_fill_(torch.arange(k.shape[0], device="cuda") > place[:, None], float("-inf"))
    return torch.einsum("hij,jhd->ihd", a.softmax(-1), v)


def check_rest(layer, b, r_before, r, x_next, gain):
    """The two block norms from the linears' outputs."""
    r1 = r_before.to(F64) + b.o_out.to(F64)
    close(b.x_mlp, rms(r1, layer.mlp_gain), 4 * U16, "norm before the MLP")
    r2 = r1 + b.down_out.to(F64)
    close(r, r2, 4 * U16, "residual stream")
    close(x_next, rms(r2, gain), 4 * U16, "next layer's input")


def test_prompts_without_a_cache():
    lengths = [70, 1, 200, 129]
    rows, starts = sum(lengths), [0, 70, 71, 271, 400]
    layer, x, r, gain = layer_and_inputs(rows, 4, 1)
    rope, at = w4.w4a4_rope_table(200, DIM, 1e6), ints([i for n in lengths for i in range(n)])
    b = layer.rows(rows)
    w4.w4a4_forward(x, layer.qkv.packed, layer.qkv.colscale, layer.qkv.bias, b.qkv_out, layer.qkv.r, b.ws)
    q, k, v = (t.to(F64) for t in b.split)
    before, x_next = r.clone(), torch.empty_like(x)
    layer.prompt(x, r, at, ints(starts), rope, gain, x_next)
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0
    q, k = turn(rms(q, layer.q_gain), rope, at), turn(rms(k, layer.k_gain), rope, at)
    close(b.split[0], q, 4 * U16, "queries"), close(b.split[1], k, 4 * U16, "keys")
    for lo, hi in zip(starts, starts[1:]):
        # scores off by the queries' and keys' roundings, probabilities and outputs by theirs
        ref = attended(*(t[lo:hi].to(F64) for t in b.split), 0)
        close(b.attn[lo:hi], ref, 4 * U16, "attention")
    check_rest(layer, b, before, r, x_next, gain)


def test_chunks_of_a_prompt_are_the_prompt():
    """Two sequences' prompts in three chunks through the cache, with one decode step behind them, against the whole
    prompts without a cache."""
    lengths, cuts = [150, 90], ([0, 64, 65, 150], [0, 0, 90, 90])  # a chunk without rows of the second, and the other way
    rope = w4.w4a4_rope_table(200, DIM, 1e6)
    layer, x, r, gain = layer_and_inputs(242, 2, 2)  # 240 of the prompts, then one token each
    cache = decoder.paged_cache(2, 200, HKV, DIM, page_size=8)
    first = [0, 150]
    whole = torch.empty(240, HQ, DIM, dtype=torch.float16, device="cuda")
    at = ints([*range(150), *range(90)])
    layer.prompt(x[:240], r[:240].clone(), at, ints([0, 150, 240]), rope, gain, torch.empty_like(x[:240]))
    whole.copy_(layer.rows(240).attn)
    for c in range(3):
        part = [(cuts[b][c], cuts[b][c + 1]) for b in range(2)]
        index = torch.tensor([first[b] + i for b in range(2) for i in range(*part[b])], device="cuda")
        places = ints([i for b in range(2) for i in range(*part[b])])
        owners = ints([b for b in range(2) for _ in range(*part[b])])
        n = part[0][1] - part[0][0]
        starts, now = ints([0, n, len(index)]), ints([p[1] for p in part])
        x_next = torch.empty(len(index), HIDDEN, dtype=torch.float16, device="cuda")
        before = r[index]
        after = before.clone()
        layer.chunk(x[index], after, places, owners, starts, now, cache, rope, gain, x_next)
        torch.cuda.synchronize()
        assert w4.w4a4_device_status() == 0
        b = layer.rows(len(index))
        close(b.attn, whole[index].to(F64), 8 * U16, "chunk")  # both off by what the other is
        check_rest(layer, b, before, after, x_next, gain)
    k, v, table = cache._keep[:3]
    x_next, rr = torch.empty(2, HIDDEN, dtype=torch.float16, device="cuda"), r[240:].clone()
    layer.step(x[240:], rr, ints([150, 90]), ints([151, 91]), cache, rope, gain, x_next)
    torch.cuda.synchronize()
    for b, n in enumerate((151, 91)):
        tok = torch.arange(n, device="cuda")
        held = [p[table[b, tok // 8].long(), tok % 8].to(F64) for p in (k, v)]
        close(layer.attn[b:b + 1], attended(layer.q[b:b + 1].to(F64), *held, n - 1), 4 * U16, "decode step")
    assert w4.w4a4_device_status() == 0


def test_a_captured_prompt_and_chunk():
    rows, starts = 100, ints([0, 60, 100])
    layer, x, r, gain = layer_and_inputs(rows, 2, 3)
    cache = decoder.paged_cache(2, 64, HKV, DIM)
    rope, at = w4.w4a4_rope_table(64, DIM, 1e6), ints([*range(60), *range(40)])
    owners, lengths = ints([0] * 60 + [1] * 40), ints([60, 40])
    outs = [torch.empty_like(x) for _ in range(2)]
    streams = [r.clone() for _ in range(2)]

    def both():
        layer.prompt(x, streams[0], at, starts, rope, gain, outs[0])
        layer.chunk(x, streams[1], at, owners, starts, lengths, cache, rope, gain, outs[1])

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    want = None
    for _ in range(3):
        for s in streams:
            s.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        assert w4.w4a4_device_status() == 0
        b = layer.rows(rows)  # of the chunk, the later one
        for lo, hi in ((0, 60), (60, 100)):
            k = turn(rms(b.split[1][lo:hi].to(F64), layer.k_gain), rope, at[lo:hi]).half().to(F64)  # as the cache holds them
            close(b.attn[lo:hi], attended(b.q[lo:hi].to(F64), k, b.split[2][lo:hi].to(F64), 0), 8 * U16, "replayed chunk")
        assert want is None or all(torch.equal(a, c) for a, c in zip(want, outs))
        want = [o.clone() for o in outs]


def test_main_runs(capsys):
    decoder.main(2, 40, 2)
    assert "a prompt of 40 tokens" in capsys.readouterr().out
