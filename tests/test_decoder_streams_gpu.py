"""The decoder layer's passes on another stream than the current one: the memory of their buffers."""
import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.test_decoder_prompt_gpu import DIM, HKV, HQ, ints, layer_and_inputs
from w4a4_quantized_gemm_gb300 import decoder

pytestmark = pytest.mark.gpu
ROWS = 2000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a4_quantized_gemm_gb300 import build
    build.build()
    w4.lib()
    w4.w4a4_device_status()


def a_pass(kind, layer, x, r, gain):
    """A prompt, or the same tokens as a chunk into a cache, on a stream: returns a function of it and its results."""
    rope, at, starts = w4.w4a4_rope_table(ROWS, DIM, 1e6), ints(list(range(ROWS))), ints([0, ROWS])
    owners, lengths = ints([0] * ROWS), ints([ROWS])
    cache = decoder.paged_cache(1, ROWS, HKV, DIM)
    cache.workspace(HQ)

    def run(stream=None):
        stream_r, out = streams.pop(), outs.pop()
        if kind == "prompt":
            layer.prompt(x, stream_r, at, starts, rope, gain, out, stream=stream)
        else:
            layer.chunk(x, stream_r, at, owners, starts, lengths, cache, rope, gain, out, stream=stream)
        return stream_r, out

    streams, outs = [r.clone() for _ in range(4)], [torch.empty_like(x) for _ in range(4)]
    return run


@pytest.mark.parametrize("kind", ["prompt", "chunk"])
@pytest.mark.parametrize("handle", [False, True])
def test_buffers_made_for_a_side_stream(kind, handle):
    """No memory whose last use on the current stream is still to come."""
    layer, x, r, gain = layer_and_inputs(ROWS, 1, 4)
    run = a_pass(kind, layer, x, r, gain)
    side = torch.cuda.Stream()
    width = (HQ + 2 * HKV) * DIM  # what the fused q|k|v output takes
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((ROWS, w), 7.0, dtype=torch.float16, device="cuda") for w in (width, HQ * DIM, HQ * DIM)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second
    copies = [h.clone() for h in held]
    del held
    got = run(side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert all(torch.all(c == 7) for c in copies)
    want = run()
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["prompt", "chunk"])
@pytest.mark.parametrize("first", ["side", "current"])
def test_buffers_outlive_the_layer(kind, first):
    """A layer dropped while a side stream still runs its pass, whose buffers were made for it or for the current one."""
    layer, x, r, gain = layer_and_inputs(ROWS, 1, 5)
    run = a_pass(kind, layer, x, r, gain)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if first == "current":
        run()
        torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    run(side)
    b = layer.rows(ROWS, side)
    buffers = [(t.data_ptr(), t.numel() * t.element_size()) for t in (b.qkv_out, b.attn, b.o_out, b.h, b.ws)]
    weights = layer.qkv, layer.o, layer.gate_up, layer.down, layer.q_gain, layer.k_gain, layer.mlp_gain
    del layer, run, b
    again = [torch.empty(size, dtype=torch.uint8, device="cuda") for _, size in buffers]
    busy = not side.query()
    torch.cuda.synchronize()
    spans = [(p, p + n) for p, n in buffers]
    assert busy and not any(lo < t.data_ptr() + t.numel() and t.data_ptr() < hi for t in again for lo, hi in spans)
    assert len(weights) == 7  # they are the caller's to keep, as tensors are


def test_passes_over_many_lengths_in_one_room():
    """Prompts of growing and shrinking length through two layers that share their buffers: each the same as through
    layers that hold no others."""
    shared = decoder.Buffers()
    g = torch.Generator(device="cuda").manual_seed(6)
    made = [decoder.random_layer(512, 640, HQ, HKV, DIM, 1, seed=i, buffers=shared) for i in range(2)]
    rope, gain = w4.w4a4_rope_table(500, DIM, 1e6), torch.ones(512, dtype=torch.float16, device="cuda")
    for n in (300, 20, 301, 500, 1, 299):
        x, r = torch.randn(n, 512, generator=g, device="cuda").half(), torch.randn(n, 512, generator=g, device="cuda")
        results = []
        for rooms in (shared, decoder.Buffers()):
            stream, xs = r.clone(), [x, torch.empty_like(x), torch.empty_like(x)]
            for i, layer in enumerate(made):
                layer.prompt(xs[i], stream, ints(list(range(n))), ints([0, n]), rope, gain, xs[i + 1],
                             buffers=None if rooms is shared else rooms)
            results.append((stream, xs[2]))
        assert all(torch.equal(a, b) for a, b in zip(*results)), n
    assert w4.w4a4_device_status() == 0


def test_two_streams_with_buffers_of_their_own():
    """A prompt of one layer on each of two streams at the same time, and a decode step on a third."""
    layer, x, r, gain = layer_and_inputs(ROWS, 1, 7)
    rope, at, starts = w4.w4a4_rope_table(ROWS, DIM, 1e6), ints(list(range(ROWS))), ints([0, ROWS])
    cache = decoder.paged_cache(1, 16, HKV, DIM)
    cache.workspace(HQ)
    sides, rooms = [torch.cuda.Stream() for _ in range(3)], [decoder.Buffers() for _ in range(2)]
    inputs = [x, x.flip(0).contiguous()]
    one, first, place = x[:1].contiguous(), ints([1]), ints([0])

    def prompt(i, streams, outs, stream=None):
        layer.prompt(inputs[i], streams[i], at, starts, rope, gain, outs[i], stream=stream, buffers=rooms[i])

    def step(streams, outs, stream=None):
        layer.step(one, streams[2], place, first, cache, rope, gain, outs[2], stream=stream)

    def fresh():
        return ([r.clone(), r.clone(), r[:1].clone()], [torch.empty_like(x), torch.empty_like(x), torch.empty_like(one)])

    want = fresh()
    for i in range(2):
        prompt(i, *want)
    step(*want)
    torch.cuda.synchronize()
    for turn in range(5):
        got = fresh()
        torch.cuda.synchronize()
        for i in range(2):
            prompt(i, *got, stream=sides[i])
        step(*got, stream=sides[2])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g)), turn
    assert w4.w4a4_device_status() == 0
