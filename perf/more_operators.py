"""What is measured of the operators that take a prompt through a decoder layer: queries and keys
normalised and rotated where they lie, attention over whole prompts packed one behind the other,
and attention of a chunk of new tokens over a paged cache.

`run` computes a case in plain torch operations, or with `own` through this package's entry
points; `exact` computes the same from the definitions in 64 bits."""
import math
import random

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"fp16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-6
THETA = 1e6  # base of the rotation's wavelengths
BLOCK = 1 << 28  # scores that the plain form holds at once


# ------------------------------------------------------------------ the cases
# tokens: of all sequences; seqs: how many share them ("mix" draws their lengths, 0: equal shares).
# past: tokens that the cache holds of each sequence before its chunk (with "mix": at most).
def listed():
    turn = dict(op="turn", hq=16, hkv=8, dim=128, rot=128, type="fp16", qk_norm=True, interleaved=False)
    prompt = dict(op="prompt", seqs=1, mix=0, hq=16, hkv=8, dim=128, type="fp16", causal=True, window=0, lse=False)
    chunk = dict(op="chunk", seqs=1, mix=0, hq=16, hkv=8, dim=128, type="fp16", cache="fp16", page=16, layout="NHD",
                 window=0, lse=False)
    return [
        # one token of a 1024-wide layer
        dict(turn, name="turn_one", tokens=1),
        # its 700-token prompt
        dict(turn, name="turn_prompt", tokens=700),
        # a long prompt of a wider layer, pairs side by side
        dict(turn, name="turn_long", tokens=8192, hq=32, type="bf16", qk_norm=False, interleaved=True),
        # the 700-token prompt of the 1024-wide layer
        dict(prompt, name="prompt_700", tokens=700),
        # every position sees the whole text: an encoder's batch with small heads
        dict(prompt, name="prompt_both_ways", tokens=12000, seqs=8, mix=3, hq=16, hkv=16, dim=64, causal=False),
        # prompts of all lengths in one call, with what a later join needs
        dict(prompt, name="prompt_packed", tokens=8192, seqs=19, mix=5, hq=32, type="bf16", lse=True),
        # the largest: one long document
        dict(prompt, name="prompt_long", tokens=16384, hq=32, type="bf16"),
        # five tokens proposed to one stream after its 700
        dict(chunk, name="chunk_verify", tokens=5, past=700),
        # four proposed tokens of each of many streams over an 8-bit cache
        dict(chunk, name="chunk_verify_e4m3", tokens=256, seqs=64, past=8191, mix=7, hq=32, type="bf16", cache="e4m3",
             page=32, layout="HND"),
        # one stream's next sixty-odd tokens behind a very long context: few rows, a long axis
        dict(chunk, name="chunk_long_past", tokens=61, past=100000, hq=32, type="bf16", cache="bf16", page=64,
             layout="HND"),
        # a prefill step that serves pieces of several prompts, wide heads
        dict(chunk, name="chunk_wide_heads", tokens=2500, seqs=6, past=3000, mix=9, hkv=4, dim=256, page=24, lse=True),
        # a piece of a long prompt
        dict(chunk, name="chunk_prefill", tokens=2048, past=30000, hq=32, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST = {"turn": 7 * 8192 * 40 * 128, "prompt": 4 * 16384 * 16385 // 2 * 32 * 128, "chunk": 4 * 2048 * 31024 * 32 * 128}


def draw(rng):
    op = rng.choice(["turn", "prompt", "prompt", "chunk", "chunk"])
    kind = rng.choice(["fp16", "bf16"])
    hkv, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 7, 8])
    dim = rng.choice([64, 96, 128, 128, 256])
    case = dict(op=op, hq=hkv * group, hkv=hkv, dim=dim, type=kind)
    if op == "turn":
        return dict(case, rot=rng.choice([dim, dim, 32]), qk_norm=rng.random() < 0.5, interleaved=rng.random() < 0.3,
                    tokens=_log(rng, 1, min(8192, MOST[op] // (7 * (hkv + case["hq"]) * dim))))
    if op == "prompt":
        tokens = _log(rng, 1, 16384)
        seqs = rng.choice([1, _log(rng, 1, min(64, tokens))])
        causal = rng.random() < 0.75
        case |= dict(tokens=tokens, seqs=seqs, mix=rng.randint(1, 10 ** 6), causal=causal, lse=rng.random() < 0.4,
                     window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]) if causal else 0)
    else:
        tokens, past = _log(rng, 1, 4096), _log(rng, 1, 100000)
        seqs = rng.choice([1, _log(rng, 1, min(128, tokens))])
        case |= dict(tokens=tokens, seqs=seqs, mix=rng.randint(1, 10 ** 6), past=past, cache=rng.choice([kind, kind, "e4m3"]),
                     page=rng.choice([1, 8, 16, 24, 32, 64, 100]), layout=rng.choice(["NHD", "HND"]),
                     window=rng.choice([0, 0, 0, max(1, past // 3)]), lse=rng.random() < 0.4)
    while work(case)["flops"] > MOST[op] or (op == "chunk" and work(case)["bytes"] > 1.5e9):
        if op == "chunk" and case["past"] > 1000:
            case["past"] //= 2
        else:
            case["tokens"] = max(1, case["tokens"] // 2)
            case["seqs"] = min(case["seqs"], case["tokens"])
    return case


def _lengths(case):
    """New tokens of each sequence, and what the cache holds of it before them."""
    seqs, tokens, past = case["seqs"], case["tokens"], case.get("past", 0)
    if not case["mix"]:
        return [tokens * (i + 1) // seqs - tokens * i // seqs for i in range(seqs)], [past] * seqs
    mix = random.Random(case["mix"])
    cut = [0] + sorted(mix.sample(range(1, tokens), seqs - 1)) + [tokens]
    if "past" in case and tokens == 4 * seqs:  # as many proposed tokens of each
        cut = list(range(0, tokens + 1, 4))
    return [b - a for a, b in zip(cut, cut[1:])], [mix.randint(0, past) if past else 0 for _ in range(seqs)]


# ------------------------------------------------------------------ a program's data
def _starts(new):
    return [sum(new[:i]) for i in range(len(new) + 1)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind, hq, hkv, dim, tokens = TYPES[case["type"]], case["hq"], case["hkv"], case["dim"], case["tokens"]

    def randn(*shape, times=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(times).to(kind)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    qkv = randn(tokens, (hq + 2 * hkv) * dim)  # the output of the fused q|k|v linear
    qkv[:, :hq * dim] *= 2
    q, k, v = (x.unflatten(1, (-1, dim)) for x in qkv.split((hq * dim, hkv * dim, hkv * dim), dim=1))
    s = {"case": case, "q": q, "out": torch.empty(tokens, hq, dim, dtype=kind, device="cuda")}
    if case["op"] == "turn":
        half = case["rot"] // 2
        angle = torch.arange(10000, device="cuda", dtype=torch.float64)[:, None] * \
            THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s |= {"k": k, "k_out": torch.empty(tokens, hkv, dim, dtype=kind, device="cuda"),
              "position": torch.randint(0, 10000, (tokens,), generator=gen, device="cuda", dtype=torch.int32),
              "rope": torch.stack((angle.cos(), angle.sin()), dim=1).float()}
        for name in ("q_gain", "k_gain"):
            s[name] = 1 + randn(dim, times=0.2) if case["qk_norm"] else None
        return s
    new, past = _lengths(case)
    s |= {"new": new, "past": past, "starts": ints(_starts(new)),
          "lse": torch.empty(tokens, hq, device="cuda") if case["lse"] else None}
    if case["op"] == "prompt":
        return s | {"k": k, "v": v}
    # pools that hold past and new tokens of each sequence, pages in any order
    page, hnd = case["page"], case["layout"] == "HND"
    lengths = [n + p for n, p in zip(new, past)]
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    count, at = torch.tensor(need, device="cuda"), torch.arange(max(need), device="cuda")
    first = torch.cumsum(count, 0) - count
    s["table"] = torch.where(at < count[:, None], order[(first[:, None] + at).clamp_(max=pages - 1)], 0).to(torch.int32)
    s["lengths"] = ints(lengths)
    for name in ("k", "v"):
        pool = torch.randn((pages, hkv, page, dim) if hnd else (pages, page, hkv, dim), generator=gen, device="cuda",
                           dtype=torch.float16)
        scale = None
        if case["cache"] == "e4m3":  # an 8-bit pool holds unit-variance rows over scale[head]
            scale = (torch.rand(hkv, generator=gen, device="cuda") + 0.5) / 64
            pool.div_((scale[:, None, None] if hnd else scale[:, None]).half()).clamp_(-E4M3_MAX, E4M3_MAX)
        pool = pool.to(TYPES[case["cache"]])
        s[name], s[name + "_scale"] = pool.transpose(1, 2) if hnd else pool, scale
    if own:  # the program's handle on its cache
        import w4a4_quantized_gemm_gb300 as w4
        s["cache"] = w4.PagedKVCache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------------ the plain form
def _turned(x, gain, s):
    """Heads [tokens, heads, dim] normalised and rotated by their positions, in 32 bits."""
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()
    rot, turn = s["case"]["rot"], s["rope"][s["position"].long()][:, :, None]
    c, t, head = turn[:, 0], turn[:, 1], x[..., :rot]
    if s["case"]["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * c - b * t, b * c + a * t), dim=-1).flatten(-2)
    else:
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        head = torch.cat((a * c - b * t, b * c + a * t), dim=-1)
    return torch.cat((head, x[..., rot:]), dim=-1)


def _bits(pool):
    """A pool as something torch can index: it has no indexing of 8-bit floats."""
    return pool.view(torch.uint8) if pool.element_size() == 1 else pool


def _held(s, name, b, n):
    """What the cache holds of sequence b, [tokens, heads, dim] in 32 bits."""
    page = s["case"]["page"]
    x = _bits(s[name])[s["table"][b, : -(-n // page)].long()].view(s[name].dtype).flatten(0, 1)[:n].float()
    return x if s[name + "_scale"] is None else x * s[name + "_scale"][:, None]


def _attend(s):
    case = s["case"]
    hkv, scale, window = case["hkv"], 1.0 / math.sqrt(case["dim"]), case["window"]
    group, at = case["hq"] // hkv, 0
    for b, (n, past) in enumerate(zip(s["new"], s["past"])):
        m = n + past  # keys
        if case["op"] == "prompt":
            k, v = s["k"][at:at + n].float(), s["v"][at:at + n].float()
        else:
            k, v = _held(s, "k", b, m), _held(s, "v", b, m)
        k, v = k.transpose(0, 1)[:, None], v.transpose(0, 1)[:, None]  # [heads, 1, keys, dim]
        key = torch.arange(m, device="cuda")
        rows = max(1, min(n, BLOCK // (m * hkv * group)))
        for i in range(0, n, rows):
            j = min(n, i + rows)
            q = s["q"][at + i:at + j].float().unflatten(1, (hkv, group)).permute(1, 2, 0, 3)
            a = (q @ k.transpose(2, 3)).mul_(scale)  # [heads, group, rows, keys]
            place = past + torch.arange(i, j, device="cuda")[:, None]
            if case.get("causal", True):
                hidden = key > place
                if window:
                    hidden |= key <= place - window
                a.masked_fill_(hidden, -math.inf)
            top = a.amax(-1, keepdim=True)
            a = a.sub_(top).exp_()
            total = a.sum(-1, keepdim=True)
            s["out"][at + i:at + j] = ((a @ v) / total).permute(2, 0, 1, 3).flatten(1, 2).to(s["q"].dtype)
            if s["lse"] is not None:
                s["lse"][at + i:at + j] = (top + total.log()).squeeze(-1).permute(2, 0, 1).flatten(1, 2)
        at += n
    return (s["out"], s["lse"]) if s["lse"] is not None else s["out"]


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "turn":
            return tuple(_turned(s[x], s[x + "_gain"], s).to(s["q"].dtype) for x in ("q", "k"))
        return _attend(s)
    import w4a4_quantized_gemm_gb300 as w4
    if case["op"] == "turn":
        w4.w4a4_qk_rope(s["q"], s["k"], s["position"], s["out"], s["k_out"], rope=s["rope"], q_gain=s["q_gain"],
                        k_gain=s["k_gain"], eps=EPS, interleaved=case["interleaved"])
        return s["out"], s["k_out"]
    if case["op"] == "prompt":
        w4.w4a4_prompt_attention(s["q"], s["k"], s["v"], s["starts"], s["out"], lse=s["lse"], window=case["window"],
                                 causal=case["causal"])
    else:
        w4.w4a4_chunk_attention(s["q"], s["cache"], s["starts"], s["lengths"], s["out"], lse=s["lse"],
                                window=case["window"])
    return (s["out"], s["lse"]) if s["lse"] is not None else s["out"]


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64, dim = torch.float64, case["dim"]
    if case["op"] == "turn":
        rot, out = case["rot"], []
        wave = torch.tensor([THETA ** (-2.0 * i / rot) for i in range(rot // 2)], device="cuda", dtype=f64)
        wave = s["position"].to(f64)[:, None] * wave
        wave = torch.polar(torch.ones_like(wave), wave)[:, None]
        for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
            x = x.to(f64)
            if gain is not None:
                x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * gain.to(f64)
            pair = x[..., :rot].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
            axis = -1 if case["interleaved"] else -2
            z = torch.complex(pair.select(axis, 0), pair.select(axis, 1)) * wave
            out.append(torch.cat((torch.stack((z.real, z.imag), dim=axis).flatten(-2), x[..., rot:]), -1))
        return tuple(out)
    hkv, hq, page = case["hkv"], case["hq"], case.get("page")
    out = torch.empty(case["tokens"], hq, dim, device="cuda", dtype=f64)
    lse = torch.empty(case["tokens"], hq, device="cuda", dtype=f64)
    starts = s["starts"].tolist()
    for b, (lo, hi) in enumerate(zip(starts, starts[1:])):
        if case["op"] == "prompt":
            keys, values = s["k"][lo:hi], s["v"][lo:hi]
            before = 0
        else:
            length = int(s["lengths"][b])
            before = length - (hi - lo)
            place = torch.arange(length, device="cuda")
            slot = s["table"][b].long()[place // page] * page + place % page
            keys, values = (_bits(s[x]).flatten(0, 1)[slot].view(s[x].dtype) for x in ("k", "v"))
        for h in range(hq):
            g = h * hkv // hq
            k, v = keys[:, g].to(f64), values[:, g].to(f64)
            if case["op"] == "chunk" and s["k_scale"] is not None:
                k, v = k * s["k_scale"][g].to(f64), v * s["v_scale"][g].to(f64)
            for i in range(lo, hi, 4096):
                j = min(hi, i + 4096)
                first, last = 0, len(k)
                if case.get("causal", True):  # the keys that any of these rows sees
                    last = before + j - lo
                    first = max(0, before + i - lo + 1 - case["window"]) if case["window"] else 0
                a = s["q"][i:j, h].to(f64) @ k[first:last].T / dim ** 0.5
                if case.get("causal", True):
                    far = torch.arange(before + i - lo, before + j - lo, device="cuda")[:, None] - \
                        torch.arange(first, last, device="cuda")  # how far back a key lies
                    a[(far < 0) | ((far >= case["window"]) if case["window"] else (far < 0))] = -math.inf
                lse[i:j, h] = torch.logsumexp(a, 1)
                out[i:j, h] = torch.softmax(a, 1) @ v[first:last]
    return (out, lse) if case["lse"] else out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es, hq, hkv, dim, t = SIZE[case["type"]], case["hq"], case["hkv"], case["dim"], case["tokens"]
    if case["op"] == "turn":
        return {"bytes": 2 * t * (hq + hkv) * dim * es + min(t, 10000) * case["rot"] * 4 + 4 * t,
                "flops": t * (hq + hkv) * dim * 7}
    pairs = keys = 0  # of query and key that see each other; keys that some query sees
    window = case["window"]
    for n, past in zip(*_lengths(case)):
        m = n + past
        if not case.get("causal", True):
            pairs += n * m
            keys += m
            continue
        w = min(window or m, m)
        full = max(0, min(n, m - w + 1))  # queries at places >= w - 1, which see w keys each
        short = n - full
        pairs += full * w + short * (past + 1) + short * (short - 1) // 2
        keys += min(m, n + w - 1)
    ec = SIZE[case["cache"]] if case["op"] == "chunk" else es
    table = 4 * keys / case["page"] if case["op"] == "chunk" else 0
    return {"bytes": 2 * t * hq * dim * es + 2 * keys * hkv * dim * ec + table + (4 * t * hq if case["lse"] else 0),
            "flops": 4 * pairs * hq * dim}
