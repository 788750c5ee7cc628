"""What is measured of the decoder layer's operators around the quantised linears: appending
rotated keys and values to a paged cache, attention of one new token per sequence over that
cache, and the norms after and before a block fused with its gate and residual scale.

`run` computes a case in plain torch operations, or with `own` through this package's entry
points; `exact` computes the same from the definitions in 64 bits."""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-6
THETA = 1e6  # base of the rotation's wavelengths


# ------------------------------------------------------------------ the cases
def listed():
    append = dict(op="append", hq=16, hkv=8, dim=128, rot=128, type="fp16", cache="fp16", page=16, layout="NHD",
                  qk_norm=True, interleaved=False)
    attend = dict(op="attend", hq=16, hkv=8, dim=128, type="fp16", cache="fp16", page=16, layout="NHD", ragged=False,
                  window=0, lse=False)
    norm = dict(op="norm", type="fp16", residual="fp16", post="rms", pre="rms", gate="none", span=1, scale=1.0)
    return [
        # one token of one sequence: the step that a single stream of a 1024-wide layer waits for
        dict(append, name="append_one", tokens=1, seqs=1, past=700),
        # a 700-token prompt of that layer
        dict(append, name="append_prompt", tokens=700, seqs=1, past=0),
        # a decode step of many streams into an 8-bit cache
        dict(append, name="append_decode_e4m3", tokens=250, seqs=250, past=1000, hq=32, type="bf16", cache="e4m3",
             page=32, layout="HND", qk_norm=False),
        # chunked prefill: the largest
        dict(append, name="append_chunks", tokens=8192, seqs=5, past=3000, hq=32, page=64, qk_norm=False),
        # one stream that has just had its 700-token prompt
        dict(attend, name="attend_one", seqs=1, length=700),
        # a batch of streams of all lengths, the ordinary serving step
        dict(attend, name="attend_ragged", seqs=76, length=4096, ragged=True, lse=True),
        # one stream with a very long context, few heads to share it out by
        dict(attend, name="attend_long", seqs=1, length=131071, hq=32, type="bf16", cache="bf16", page=64, layout="HND"),
        # 8-bit cache, small heads, a sliding window
        dict(attend, name="attend_window_e4m3", seqs=64, length=9001, ragged=True, hq=64, dim=64, type="bf16",
             cache="e4m3", page=32, window=4096),
        # the largest: a full batch at a full context
        dict(attend, name="attend_full", seqs=128, length=8192, hq=32),
        # one token of a 1024-wide layer
        dict(norm, name="norm_one", rows=1, width=1024),
        # the 700-token prompt, with a gate per channel and a residual scale
        dict(norm, name="norm_prompt", rows=700, width=1024, gate="shared", scale=0.7),
        # a prefill step of a 4096-wide layer on an fp32 residual stream, a gate row per sequence, layer norms
        dict(norm, name="norm_prefill", rows=8192, width=4096, type="bf16", residual="fp32", post="layer", pre="layer",
             gate="rows", span=1000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "norm"])
    kind = rng.choice(["fp16", "bf16"])
    if op == "norm":
        width = 8 * _log(rng, 8, 1024)
        return dict(op=op, type=kind, residual=rng.choice([kind, "fp32"]), post=rng.choice(["none", "rms", "layer"]),
                    pre=rng.choice(["rms", "layer"]), gate=rng.choice(["none", "shared", "rows"]),
                    span=_log(rng, 1, 1000), scale=rng.choice([1.0, 0.7, 0.25]), width=width,
                    rows=_log(rng, 1, min(8192, 8192 * 4096 // width)))
    hkv, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 7, 8, 16])
    dim = rng.choice([64, 96, 128, 256])
    case = dict(op=op, hq=hkv * group, hkv=hkv, dim=dim, type=kind, cache=rng.choice([kind, kind, "e4m3"]),
                page=rng.choice([1, 8, 16, 24, 32, 64, 100]), layout=rng.choice(["NHD", "HND"]))
    if op == "append":
        tokens = _log(rng, 1, min(8192, 8192 * 48 * 128 // (hkv * (group + 2) * dim)))
        seqs = tokens if rng.random() < 0.5 and tokens <= 256 else rng.randint(1, min(tokens, 8))
        return dict(case, rot=rng.choice([dim, dim, 32]), qk_norm=rng.random() < 0.5, interleaved=rng.random() < 0.3,
                    tokens=tokens, seqs=seqs, past=rng.randint(0, 1000))
    most = 128 * 8192 * 8 * 128 // (hkv * dim * max(1, (group + 3) // 4))  # keys of all sequences together
    length = _log(rng, 1, min(131072, most))
    return dict(case, length=length, seqs=_log(rng, 1, max(1, min(256, most // length))), ragged=rng.random() < 0.6,
                window=rng.choice([0, 0, 0, max(1, length // 3)]), lse=rng.random() < 0.5)


# ------------------------------------------------------------------ a program's data
def _cache(case, lengths, most, gen):
    """Pools, page table and scales that hold `lengths` (a list) tokens of each sequence, pages in any order, in pools
    with room for `most` tokens in all."""
    page, hkv, dim = case["page"], case["hkv"], case["dim"]
    need = [-(-n // page) for n in lengths]
    pages, wide = -(-most // page) + len(need), max(need)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    count = torch.tensor(need, device="cuda")
    at = torch.arange(wide, device="cuda")
    first = torch.cumsum(count, 0) - count
    table = torch.where(at < count[:, None], order[(first[:, None] + at).clamp_(max=pages - 1)], 0).to(torch.int32)
    s, hnd = {"table": table}, case["layout"] == "HND"
    for name in ("k", "v"):
        pool = torch.randn((pages, hkv, page, dim) if hnd else (pages, page, hkv, dim), generator=gen, device="cuda",
                           dtype=torch.float16)
        scale = None
        if case["cache"] == "e4m3":  # an 8-bit pool holds unit-variance rows over scale[head]
            scale = (torch.rand(hkv, generator=gen, device="cuda") + 0.5) / 64
            pool.div_((scale[:, None, None] if hnd else scale[:, None]).half()).clamp_(-E4M3_MAX, E4M3_MAX)
        pool = pool.to(TYPES[case["cache"]])
        s[name], s[name + "_scale"] = pool.transpose(1, 2) if hnd else pool, scale
    if own:  # the program's handle on its cache: pointers, strides, and the workspace of the split
        import w4a4_quantized_gemm_gb300 as w4
        s["cache"] = w4.PagedKVCache(s["k"], s["v"], table, s["k_scale"], s["v_scale"])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    kind = TYPES[case["type"]]

    def randn(*shape, dtype=kind, times=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(times).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        rows, width = case["rows"], case["width"]
        gates = {"none": 0, "shared": 1, "rows": -(-rows // case["span"])}[case["gate"]]
        s |= {"y": randn(rows, width, times=3.0), "r": randn(rows, width, dtype=TYPES[case["residual"]], times=4.0),
              "gate": randn(gates, width) if gates else None, "x": torch.empty(rows, width, dtype=kind, device="cuda")}
        s["r_new"] = torch.empty_like(s["r"])
        for name in ("post", "pre"):
            s[name + "_gain"] = 1 + randn(width, times=0.2) if case[name] != "none" else None
            s[name + "_bias"] = randn(width, times=0.2) if case[name] == "layer" else None
        return s
    hq, hkv, dim, seqs = case["hq"], case["hkv"], case["dim"], case["seqs"]
    if case["op"] == "attend":
        n = case["length"]
        lengths = torch.randint(1, n + 1, (seqs,), generator=host).tolist() if case["ragged"] else [n] * seqs
        s |= _cache(case, lengths, n * seqs, gen)
        s |= {"q": randn(seqs, hq, dim, times=2.0), "lengths": torch.tensor(lengths, dtype=torch.int32, device="cuda"),
              "out": torch.empty(seqs, hq, dim, dtype=kind, device="cuda"),
              "lse": torch.empty(seqs, hq, device="cuda") if case["lse"] else None}
        return s
    tokens = case["tokens"]
    cut = sorted((torch.randperm(tokens - 1, generator=host)[: seqs - 1] + 1).tolist())  # a token at least of each
    starts, ends = [0] + cut, cut + [tokens]
    past = torch.randint(0, case["past"] + 1, (seqs,), generator=host).tolist()
    s |= _cache(case, [p + e - b for p, b, e in zip(past, starts, ends)], tokens + seqs * case["past"], gen)
    count = torch.tensor([e - b for b, e in zip(starts, ends)])
    seq = torch.repeat_interleave(torch.arange(seqs), count)
    position = torch.arange(tokens) - torch.tensor(starts)[seq] + torch.tensor(past)[seq]
    half = case["rot"] // 2
    angle = torch.arange(case["past"] + tokens, device="cuda", dtype=torch.float64)[:, None] * \
        THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    qkv = randn(tokens, (hq + 2 * hkv) * dim)  # the output of the fused q|k|v linear
    q, k, v = (x.unflatten(1, (-1, dim)) for x in qkv.split((hq * dim, hkv * dim, hkv * dim), dim=1))
    s |= {"q": q, "new_k": k, "new_v": v, "seq": seq.to(torch.int32).cuda(), "position": position.to(torch.int32).cuda(),
          "rope": torch.stack((angle.cos(), angle.sin()), dim=1).float(),
          "q_gain": 1 + randn(dim, times=0.2) if case["qk_norm"] else None,
          "k_gain": 1 + randn(dim, times=0.2) if case["qk_norm"] else None,
          "q_out": torch.empty(tokens, hq, dim, dtype=kind, device="cuda")}
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


def _stored(pool, x, scale, page, slot):
    if scale is not None:
        x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    _bits(pool)[page, slot] = _bits(x.to(pool.dtype))


def _append(s):
    position = s["position"].long()
    page, slot = s["table"][s["seq"].long(), position // s["case"]["page"]].long(), position % s["case"]["page"]
    _stored(s["k"], _turned(s["new_k"], s["k_gain"], s), s["k_scale"], page, slot)
    _stored(s["v"], s["new_v"].float(), s["v_scale"], page, slot)
    return _turned(s["q"], s["q_gain"], s).to(s["q"].dtype), s["k"], s["v"]


def _held(pool, scale, table):
    """What the pages of `table` [sequences, pages] hold, [sequences, heads, tokens, dim] in 32 bits."""
    x = _bits(pool)[table].view(pool.dtype).float()
    x = x.flatten(1, 2).transpose(1, 2)
    return x if scale is None else x * scale[:, None, None]


def _attend(s):
    table, n, window = s["table"].long(), s["lengths"][:, None], s["case"]["window"]
    q = s["q"].float().unflatten(1, (s["case"]["hkv"], -1))
    score = q @ _held(s["k"], s["k_scale"], table).transpose(2, 3) / math.sqrt(q.shape[-1])
    at = torch.arange(score.shape[-1], device="cuda")
    seen = (at < n) & (at >= n - window) if window else at < n
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = ((p @ _held(s["v"], s["v_scale"], table)) / total).flatten(1, 2).to(s["q"].dtype)
    return (out, (top + total.log()).flatten(1)) if s["case"]["lse"] else out


def _normed(x, kind, gain, bias):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
    return x if bias is None else x + bias


def _norm(s):
    case = s["case"]
    up = {k: s[k].float() for k in ("y", "r", "gate", "post_gain", "post_bias", "pre_gain", "pre_bias") if s[k] is not None}
    block = _normed(up["y"], case["post"], up.get("post_gain"), up.get("post_bias")) * case["scale"]
    if case["gate"] == "rows":
        block = block * up["gate"][torch.arange(case["rows"], device="cuda") // case["span"]]
    elif case["gate"] == "shared":
        block = block * up["gate"]
    r = up["r"] + block
    return r.to(s["r"].dtype), _normed(r, case["pre"], up.get("pre_gain"), up.get("pre_bias")).to(s["y"].dtype)


def run(s):
    case = s["case"]
    if not own:
        return {"append": _append, "attend": _attend, "norm": _norm}[case["op"]](s)
    import w4a4_quantized_gemm_gb300 as w4
    if case["op"] == "append":
        w4.w4a4_kv_append(s["q"], s["new_k"], s["new_v"], s["position"], s["cache"], s["q_out"], seqs=s["seq"],
                          rope=s["rope"], q_gain=s["q_gain"], k_gain=s["k_gain"], eps=EPS,
                          interleaved=case["interleaved"])
        return s["q_out"], s["k"], s["v"]
    if case["op"] == "attend":
        w4.w4a4_paged_attention(s["q"], s["cache"], s["lengths"], s["out"], lse=s["lse"], window=case["window"])
        return (s["out"], s["lse"]) if case["lse"] else s["out"]
    kinds = {"none": w4.NORM_NONE, "rms": w4.NORM_RMS, "layer": w4.NORM_LAYER}
    w4.w4a4_block_norm(s["y"], s["r"], s["x"], s["r_new"], gate=s["gate"],
                       rows_per_gate=case["span"] if case["gate"] == "rows" else 0, scale=case["scale"],
                       post=kinds[case["post"]], post_gain=s["post_gain"], post_bias=s["post_bias"],
                       pre=kinds[case["pre"]], pre_gain=s["pre_gain"], pre_bias=s["pre_bias"], eps=EPS)
    return s["r_new"], s["x"]


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        out = []
        for i in range(0, case["rows"], 1024):
            j = min(case["rows"], i + 1024)
            y, r = s["y"][i:j].to(f64), s["r"][i:j].to(f64)
            for name in ("post", "pre"):
                x = y if name == "post" else r
                if case[name] != "none":
                    mean = x.mean(1, keepdim=True) if case[name] == "layer" else 0.0
                    x = (x - mean) / ((x - mean).pow(2).mean(1, keepdim=True) + EPS).sqrt() * s[name + "_gain"].to(f64)
                    x = x + s[name + "_bias"].to(f64) if case[name] == "layer" else x
                if name == "post":
                    if s["gate"] is not None:
                        span = case["span"] if case["gate"] == "rows" else case["rows"]
                        x = x * s["gate"].to(f64)[[m // span for m in range(i, j)]]
                    r = r + case["scale"] * x
            out.append((r, x))
        return tuple(torch.cat(x) for x in zip(*out))
    hkv, dim, page = case["hkv"], case["dim"], case["page"]
    one = torch.ones(hkv, device="cuda")
    k_scale, v_scale = ((one if s[n] is None else s[n]).to(f64)[:, None] for n in ("k_scale", "v_scale"))
    if case["op"] == "attend":
        outs, lses = [], []
        for b, n in enumerate(s["lengths"].tolist()):
            lo = max(0, n - case["window"]) if case["window"] else 0
            use = s["table"][b, lo // page:-(-n // page)].long()
            part = slice(lo % page, lo % page + n - lo)
            k, v = (_bits(s[x])[use].view(s[x].dtype).flatten(0, 1)[part].to(f64) * w
                    for x, w in (("k", k_scale), ("v", v_scale)))
            q = s["q"][b].to(f64).view(hkv, -1, dim)
            a = torch.einsum("hgd,nhd->hgn", q, k) / dim ** 0.5
            lse = torch.logsumexp(a, 2)
            outs.append(torch.einsum("hgn,nhd->hgd", (a - lse[..., None]).exp(), v).reshape(-1, dim))
            lses.append(lse.reshape(-1))
        return (torch.stack(outs), torch.stack(lses)) if case["lse"] else torch.stack(outs)
    rot = case["rot"]
    wave = torch.tensor([THETA ** (-2.0 * i / rot) for i in range(rot // 2)], device="cuda", dtype=f64)
    wave = s["position"].to(f64)[:, None] * wave
    wave = torch.polar(torch.ones_like(wave), wave)[:, None]

    def turned(x, gain):
        x = x.to(f64)
        if gain is not None:
            x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * gain.to(f64)
        pair = x[..., :rot].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
        axis = -1 if case["interleaved"] else -2
        z = torch.complex(pair.select(axis, 0), pair.select(axis, 1)) * wave
        return torch.cat((torch.stack((z.real, z.imag), dim=axis).flatten(-2), x[..., rot:]), -1)

    pools = []
    position = s["position"].cpu().long()
    slots = s["table"].cpu()[s["seq"].cpu().long(), position // page] * page + position % page
    for name, x, scale in (("k", turned(s["new_k"], s["k_gain"]), k_scale), ("v", s["new_v"].to(f64), v_scale)):
        pool = s[name].float().flatten(0, 1)  # the other slots keep what they hold
        if case["cache"] == "e4m3":
            x = (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        pool[slots.long().cuda()] = x.float()
        pools.append(pool.view(s[name].shape))
    return turned(s["q"], s["q_gain"]), *pools


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es = SIZE[case["type"]]
    if case["op"] == "norm":
        n, er = case["rows"] * case["width"], SIZE[case["residual"]]
        gates = {"none": 0, "shared": 1, "rows": -(-case["rows"] // case["span"])}[case["gate"]]
        vectors = {"none": 0, "rms": 1, "layer": 2}
        return {"bytes": n * (2 * es + 2 * er) + (gates + vectors[case["post"]] + vectors[case["pre"]]) * case["width"] * es,
                "flops": n * 12}
    hq, hkv, dim, ec = case["hq"], case["hkv"], case["dim"], SIZE[case["cache"]]
    if case["op"] == "append":
        t = case["tokens"]
        table = min(t, case["past"] + t) * case["rot"] * 4
        return {"bytes": t * dim * ((2 * hq + 2 * hkv) * es + 2 * hkv * ec) + table + 12 * t, "flops": t * (hq + hkv) * dim * 7}
    n = case["length"]
    # a ragged batch's lengths are uniform over 1..n; a window cuts those over it
    w = min(n, case["window"] or n)
    keys = case["seqs"] * ((w * (w + 1) / 2 + (n - w) * w) / n if case["ragged"] else w)
    return {"bytes": keys * hkv * dim * 2 * ec + 2 * case["seqs"] * hq * dim * es + 4 * keys / case["page"],
            "flops": 4 * keys * hq * dim}
