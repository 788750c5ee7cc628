"""The operators that take a prompt through a layer (rotation without a cache, prompt and chunk attention)
refuse bad calls on the host, before any launch; their argument structs have the header's layout."""
import os
import re
import struct
import subprocess

import pytest
import torch

import w4a4_quantized_gemm_gb300 as w4
from tests.layer_structs import fields
from tests.test_layer_ops_cpu import A, GOOD, L, cache  # noqa: F401 (L: a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="good calls would launch on a machine with a GPU")
FORMATS = {  # Q: a size or pointer, q: a stride, i: an int, f: a float
    "w4a4_qk_rope_args": struct.Struct("=Q8Q8q8ifi"),
    "w4a4_prompt_attention_args": struct.Struct("=Q6Q8qf9i"),
    "w4a4_chunk_attention_args": struct.Struct("=Q6QQ4qf5i"),
}


def pack(name, values, over):
    values = {"bytes": FORMATS[name].size, **values, **over}
    names = fields(name)
    assert set(values) <= set(names), set(values) - set(names)
    return FORMATS[name].pack(*[values.get(n, 0) for n in names])


def turn(**over):
    return pack("w4a4_qk_rope_args", dict(
        q=A, k=A + 4096, q_out=A + 8192, k_out=A + 16384, positions=A, rope=A, q_token_stride=4096, q_head_stride=128,
        k_token_stride=4096, k_head_stride=128, q_out_token_stride=2048, q_out_head_stride=128, k_out_token_stride=1024,
        k_out_head_stride=128, tokens=4, q_heads=16, kv_heads=8, head_dim=128, rope_rows=100, rot_dim=128, eps=1e-6), over)


def prompt(**over):
    return pack("w4a4_prompt_attention_args", dict(
        q=A, k=A + 4096, v=A + 6144, out=A + 65536, starts=A, q_token_stride=4096, q_head_stride=128, k_token_stride=4096,
        k_head_stride=128, v_token_stride=4096, v_head_stride=128, out_token_stride=2048, out_head_stride=128, scale=0.1,
        tokens=700, seqs=2, q_heads=16, kv_heads=8, head_dim=128, causal=1), over)


def chunk(**over):
    return pack("w4a4_chunk_attention_args", dict(
        q=A + 64, out=A + 65536, starts=A, lengths=A, workspace=A, workspace_bytes=1 << 40, q_token_stride=2048,
        q_head_stride=128, out_token_stride=2048, out_head_stride=128, scale=0.1, tokens=40, q_heads=16, causal=1), over)


def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    header = re.sub(r"#include <cuda_runtime_api.h>", "", open(os.path.join(ROOT, "include", "w4a4.h")).read())
    lines = [f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for n in FORMATS for f in fields(n)]
    lines += [f'printf("{n} %zu\\n", sizeof({n}));' for n in FORMATS]
    src.write_text("#include <stdio.h>\n#include <stddef.h>\ntypedef void* cudaStream_t;\n" + header +
                   "int main(void) {\n" + "\n".join(lines) + "return 0; }\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-o", str(exe), str(src)], check=True)
    want = dict(l.split() for l in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for name, fmt in FORMATS.items():
        codes = [c for n, c in re.findall(r"(\d*)([Qqif])", fmt.format) for _ in range(int(n or 1))]
        names, at = fields(name), 0
        assert len(codes) == len(names), name
        for c, f in zip(codes, names):
            assert int(want[f"{name}.{f}"]) == at, f"{name}.{f}"
            at += 8 if c in "Qq" else 4
        assert at == fmt.size == int(want[name])


@pytest.mark.parametrize("over, status", [
    (dict(bytes=8), 1), (dict(tokens=-1), 1), (dict(q_heads=-1), 1), (dict(kv_heads=-1), 1), (dict(dtype=2), 1),
    (dict(dtype=3), 1), (dict(head_dim=112), 2), (dict(rot_dim=0), 1), (dict(rope_rows=0), 1), (dict(positions=0), 1),
    (dict(rot_dim=24), 2), (dict(rot_dim=144), 2), (dict(q=0), 1), (dict(k=0), 1), (dict(q_out=0), 1), (dict(k_out=0), 1),
    (dict(q=A + 2), 3), (dict(k_out=A + 8), 3), (dict(q_gain=A + 4), 3), (dict(rope=A + 8), 3), (dict(positions=A + 2), 3),
    (dict(q_token_stride=4100), 3), (dict(k_out_head_stride=-128), 3), (dict(k_token_stride=1 << 40), 3),
    (dict(q_out_token_stride=0), 1), (dict(q_out_head_stride=64), 1), (dict(k_out_token_stride=120), 1),
    (dict(q_out=A), 1), (dict(k_out=A + 4096), 1),  # in place with other strides
    (dict(q_out=A + 16384), 1), (dict(q_out=A + 4096), 1), (dict(k_out=A), 1),  # an output that is another's or another's input
    (dict(q_out_token_stride=128), 1), (dict(k_out_token_stride=896), 1),  # rows of two tokens in one place
    (dict(q_heads=1 << 17), 2), (dict(tokens=0), 0), (dict(q_heads=0, kv_heads=0), 0),
])
def test_rope_refusals(L, over, status):
    assert L.w4a4_qk_rope(turn(**over), None) == status
    assert L.w4a4_qk_rope(None, None) == 1


@pytest.mark.parametrize("over, status", [
    (dict(bytes=8), 1), (dict(tokens=-1), 1), (dict(seqs=-1), 1), (dict(dtype=2), 1), (dict(dtype=3), 1),
    (dict(window=-1), 1), (dict(window=5, causal=0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(q_heads=0), 1), (dict(kv_heads=0), 1), (dict(q_heads=12), 2), (dict(q_heads=1 << 16), 2), (dict(head_dim=80), 2),
    (dict(tokens=1 << 28), 2), (dict(seqs=1 << 21), 2),
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(out=0), 1), (dict(starts=0), 1), (dict(q=A + 2), 3),
    (dict(v=A + 8), 3), (dict(out=A + 4), 3), (dict(lse=A + 2), 3), (dict(starts=A + 1), 3),
    (dict(v_token_stride=4100), 3), (dict(q_head_stride=-128), 3), (dict(k_token_stride=1 << 30), 3),
    (dict(out_token_stride=0), 1), (dict(out_head_stride=120), 1), (dict(out=A), 1), (dict(out=A + 4096), 1),
    (dict(out_token_stride=1920), 1), (dict(out_token_stride=128, out_head_stride=699 * 128), 1),  # two rows in one place
    (dict(out=A + 6144), 1), (dict(tokens=0), 0), (dict(seqs=0), 0), (dict(tokens=0, q=0), 0),
])
def test_prompt_refusals(L, over, status):
    assert L.w4a4_prompt_attention(prompt(**over), None) == status
    assert L.w4a4_prompt_attention(None, None) == 1


@pytest.mark.parametrize("over, status", [
    (dict(bytes=8), 1), (dict(tokens=-1), 1), (dict(dtype=1), 1), (dict(dtype=2), 1), (dict(window=-1), 1),
    (dict(window=5, causal=0), 1), (dict(scale=float("inf")), 1), (dict(q_heads=0), 1), (dict(q_heads=12), 2),
    (dict(q_heads=1 << 16), 2), (dict(tokens=1 << 28), 2), (dict(q=0), 1), (dict(out=0), 1), (dict(starts=0), 1),
    (dict(lengths=0), 1), (dict(workspace=0), 1), (dict(workspace_bytes=1000), 4), (dict(workspace=A + 8), 3),
    (dict(q=A + 4), 3), (dict(lse=A + 2), 3), (dict(starts=A + 2), 3), (dict(lengths=A + 1), 3), (dict(q_head_stride=4), 3),
    (dict(out_token_stride=0), 1), (dict(out_head_stride=64), 1), (dict(out=A + 64), 1), (dict(out=A), 1),
    (dict(out_token_stride=128), 1), (dict(out_token_stride=2040), 1),
    (dict(tokens=0), 0),
])
def test_chunk_refusals(L, over, status):
    assert L.w4a4_chunk_attention(cache(), chunk(**over), None) == status
    assert L.w4a4_chunk_attention(None, chunk(), None) == 1
    assert L.w4a4_chunk_attention(cache(), None, None) == 1
    assert L.w4a4_chunk_attention(cache(seqs=0), chunk(), None) == 0


@pytest.mark.parametrize("over, status", [
    (dict(bytes=8), 1), (dict(seqs=-1), 1), (dict(page_size=0), 1), (dict(dtype=2), 1), (dict(head_dim=112), 2),
    (dict(k=0), 1), (dict(page_table=0), 1), (dict(k=A + 8), 3), (dict(k_scale=A + 1), 3), (dict(v_head_stride=-128), 3),
    (dict(table_stride=9), 1), (dict(max_pages=1 << 28, table_stride=1 << 28), 2),
])
def test_chunk_refuses_bad_caches(L, over, status):
    assert L.w4a4_chunk_attention(cache(**over), chunk(), None) == status


@no_gpu
def test_good_calls_reach_the_device_check(L):
    assert L.w4a4_qk_rope(turn(), None) == GOOD
    assert L.w4a4_qk_rope(turn(q_out=A, q_out_token_stride=4096, k_out=A + 4096, k_out_token_stride=4096), None) == GOOD
    assert L.w4a4_qk_rope(turn(rope=0, positions=0), None) == GOOD
    assert L.w4a4_qk_rope(turn(kv_heads=0, k=0, k_out=0), None) == GOOD
    assert L.w4a4_qk_rope(turn(q_heads=0, q=0, q_out=0), None) == GOOD
    assert L.w4a4_qk_rope(turn(q_token_stride=0, k_head_stride=0), None) == GOOD  # inputs may share rows
    assert L.w4a4_prompt_attention(prompt(), None) == GOOD
    assert L.w4a4_prompt_attention(prompt(causal=0, scale=-1.0, dtype=1, lse=A), None) == GOOD
    assert L.w4a4_prompt_attention(prompt(window=1 << 30, k_head_stride=0, v_token_stride=0), None) == GOOD
    heads_first = dict(out_token_stride=128, out_head_stride=700 * 128)
    assert L.w4a4_prompt_attention(prompt(**heads_first), None) == GOOD
    assert L.w4a4_chunk_attention(cache(), chunk(**heads_first), None) == GOOD
    for kind in (0, 1, 3):
        act = 1 if kind == 1 else 0
        assert L.w4a4_chunk_attention(cache(dtype=kind), chunk(dtype=act), None) == GOOD
    assert L.w4a4_chunk_attention(cache(dtype=3), chunk(dtype=1, causal=0), None) == GOOD


@no_gpu
@pytest.mark.parametrize("odd", (0, 3, -5, 1 << 40))
def test_strides_that_no_index_uses_are_not_looked_at(L, odd):
    names = ("q_token_stride", "k_token_stride", "q_out_token_stride", "k_out_token_stride")
    assert L.w4a4_qk_rope(turn(tokens=1, **{n: odd for n in names}), None) == GOOD
    names = ("q_head_stride", "k_head_stride", "q_out_head_stride", "k_out_head_stride")
    assert L.w4a4_qk_rope(turn(q_heads=1, kv_heads=1, **{n: odd for n in names}), None) == GOOD
    names = ("q_token_stride", "k_token_stride", "v_token_stride", "out_token_stride")
    assert L.w4a4_prompt_attention(prompt(tokens=1, **{n: odd for n in names}), None) == GOOD
    names = ("q_head_stride", "k_head_stride", "v_head_stride", "out_head_stride")
    assert L.w4a4_prompt_attention(prompt(q_heads=1, kv_heads=1, **{n: odd for n in names}), None) == GOOD
    assert L.w4a4_chunk_attention(cache(), chunk(tokens=1, q_token_stride=odd, out_token_stride=odd), None) == GOOD


def test_the_workspace_is_paged_attentions(L):
    need = L.w4a4_paged_attention_workspace_bytes(4, 16, 8, 128)
    assert L.w4a4_chunk_attention(cache(), chunk(workspace_bytes=need - 1), None) == 4


def test_binding_refuses_tensors_it_cannot_describe(L):
    """On the host, from shapes and types alone: no device is touched."""
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    for args in ((x, x, i, x, x), (x, None, i, x, x), ("q", x, i, x, x), (x.to_sparse(), x, i, x, x)):  # not on a GPU
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_qk_rope(*args)
    for args in ((x, x, x, i, x), (x, x, x, None, x), (x, 3, x, i, x), (x, x, x, torch.zeros(0, dtype=torch.int32), x)):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_prompt_attention(*args)
    for handle in (None, object(), 3):
        with pytest.raises(w4.W4A4Error):
            w4.w4a4_chunk_attention(x, handle, i, i, x)
    for f, n in ((w4.w4a4_qk_rope, 11), (w4.w4a4_prompt_attention, 10), (w4.w4a4_chunk_attention, 11)):
        for args, named in (((x,), {}), ((x,) * (n + 1), {}), ((x, x, x, x, x), dict(q=x)), ((x, x, x, x, x), dict(mask=x))):
            with pytest.raises(TypeError):
                f(*args, **named)
    assert "starts" in w4.w4a4_prompt_attention.__doc__ and "lengths" in w4.w4a4_chunk_attention.__doc__
