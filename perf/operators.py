"""The attention operators of the hybrid model's full-attention layers, as a user calls them: per-head
normalisation of queries and keys with the rotation of their positions and the write into the paged cache,
the cache's read-back, attention over whole prompts, and attention of single tokens over the cache.

`run` computes each in elementary torch operations, or (where `own` is set) by the library's calls.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6

# ------------------------------------------------------------------ cases


def _prepare(name, tokens, seqs, first, hq, hkv, dim, rot, layout, stretch, cache, page, keys_too):
    return {"name": name, "op": "prepare", "tokens": tokens, "seqs": seqs, "first": first, "hq": hq, "hkv": hkv,
            "dim": dim, "rot": rot, "layout": layout, "stretch": stretch, "cache": cache, "page": page,
            "keys_too": keys_too}


def _read(name, lens, hkv, dim, cache, page):
    return {"name": name, "op": "read", "lens": lens, "hkv": hkv, "dim": dim, "cache": cache, "page": page}


def _prefill(name, lens_q, lens_k, hq, hkv, dim, causal):
    return {"name": name, "op": "prefill", "lens_q": lens_q, "lens_k": lens_k, "hq": hq, "hkv": hkv, "dim": dim,
            "causal": causal}


def _decode(name, lens, new, hq, hkv, dim, cache, page):
    return {"name": name, "op": "decode", "lens": lens, "new": new, "hq": hq, "hkv": hkv, "dim": dim,
            "cache": cache, "page": page}


def _ragged(n, top):
    """n lengths between 1 and top that no rule of tiles or pages divides, as a text."""
    return ",".join(str(1 + (i * 2654435761 + 12345) % top) for i in range(n))


def listed():
    return [
        # one decode step of one sequence far into its context: 16 query and 2 key heads, latency alone
        _prepare("prepare_step", 1, 1, 100003, 16, 2, 128, 128, "half", 1.0, "e4m3", 64, False),
        # a prompt of the prefill benchmark's length; a quarter of each head is rotated, keys also go to the attention
        _prepare("prepare_prompt", 2048, 1, 0, 16, 2, 256, 64, "half", 1.0, "e4m3", 64, True),
        # the longest chunk of tokens, positions stretched for a long context, neighbouring pairs, 16-bit cache
        _prepare("prepare_chunk", 16384, 3, 65536, 16, 2, 128, 128, "pairs", 8.0, "bf16", 16, True),
        # a short prefix read back before its prompt's next chunk
        _read("read_prefix", "777", 2, 256, "bf16", 64),
        # many prefixes of ragged lengths, one of them empty, held in 8 bits
        _read("read_ragged", _ragged(15, 8192) + ",0", 2, 128, "e4m3", 16),
        # short packed prompts of ragged lengths, the shortest a single token
        _prefill("prefill_packed", "1,37,128,300,129,64,511", "1,37,128,300,129,64,511", 16, 2, 128, True),
        # one prompt of the prefill benchmark's length
        _prefill("prefill_prompt", "2048", "2048", 16, 2, 128, True),
        # one prompt of the longest benchmark length
        _prefill("prefill_long", "16384", "16384", 16, 2, 128, True),
        # the next chunks of two prompts after their prefixes, wide heads
        _prefill("prefill_chunks", "2048,1000", "10240,4999", 16, 2, 256, True),
        # one sequence of ordinary length: latency
        _decode("decode_one", "4096", 1, 16, 2, 128, "bf16", 64),
        # a batch of ragged sequences held in 8 bits, verification rows of 4 tokens each
        _decode("decode_batch", _ragged(64, 16384), 4, 16, 2, 128, "e4m3", 16),
        # one sequence at the longest context, wide heads
        _decode("decode_long", "131072", 1, 16, 2, 256, "e4m3", 64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv = rng.choice([(16, 2), (16, 2), (32, 8), (8, 8), (12, 4), (5, 1)])
    dim = rng.choice([64, 128, 128, 256])
    cache, page = rng.choice(["bf16", "e4m3"]), rng.choice([16, 32, 64, 128])
    op = rng.choice(["prepare", "read", "prefill", "prefill", "decode", "decode"])
    if op == "prepare":
        tokens = _log(rng, 1, 8192 if dim < 256 else 4096)
        c = _prepare("", tokens, min(tokens, _log(rng, 1, 64)), rng.randrange(0, 1 << 17), hq, hkv, dim,
                     16 * rng.randrange(1, dim // 16 + 1), rng.choice(["half", "pairs"]),
                     rng.choice([1.0, 4.0, 8.0]), cache, page, rng.random() < 0.5)
    elif op == "read":
        n = _log(rng, 1, 32)
        c = _read("", ",".join(str(_log(rng, 1, 4096) - rng.randrange(2) * (i > 0)) for i in range(n)), hkv, dim, cache, page)
    elif op == "prefill":
        n = _log(rng, 1, 16)
        top = int(4096 / math.sqrt(n))
        lens_q = [_log(rng, 1, top) for _ in range(n)]
        more = [_log(rng, 1, top) - 1 if rng.random() < 0.3 else 0 for _ in range(n)]
        c = _prefill("", ",".join(map(str, lens_q)), ",".join(str(a + b) for a, b in zip(lens_q, more)), hq, hkv, dim,
                     rng.random() < 0.8)
    else:
        n = _log(rng, 1, 64)
        new = rng.choice([1, 1, 1, 2, 4, 5, 8])
        top = max(64, 65536 // n)
        c = _decode("", ",".join(str(new + _log(rng, 1, top) - 1) for _ in range(n)), new, hq, hkv, dim, cache, page)
    del c["name"]
    return c


def _lens(text):
    return [int(v) for v in text.split(",")]


def _row_bytes(case):
    """Bytes of one head's row in the cache."""
    return case["dim"] * 2 if case["cache"] == "bf16" else case["dim"] + 4


def _pairs(case):
    """(query, key) pairs that a prompt's attention looks at, over all sequences."""
    n = 0
    for a, b in zip(_lens(case["lens_q"]), _lens(case["lens_k"])):
        n += a * b - a * (a - 1) // 2 if case["causal"] else a * b
    return n


def work(case):
    hkv, dim = case["hkv"], case["dim"]
    if case["op"] == "prepare":
        T, hq = case["tokens"], case["hq"]
        b = T * (hq + 2 * hkv) * dim * 2 + T * hq * dim * 2 + 2 * T * hkv * _row_bytes(case) + T * 8
        b += T * hkv * dim * 2 if case["keys_too"] else 0
        return {"bytes": b, "flops": T * (hq + hkv) * (4 * dim + 3 * case["rot"])}
    if case["op"] == "read":
        n = sum(_lens(case["lens"]))
        return {"bytes": 2 * n * hkv * (_row_bytes(case) + dim * 2), "flops": 2 * n * hkv * dim}
    hq = case["hq"]
    if case["op"] == "prefill":
        q, k = sum(_lens(case["lens_q"])), sum(_lens(case["lens_k"]))
        return {"bytes": 2 * q * hq * dim * 2 + q * hq * 4 + 2 * k * hkv * dim * 2, "flops": 4 * dim * hq * _pairs(case)}
    n, rows = sum(_lens(case["lens"])), len(_lens(case["lens"])) * case["new"]
    return {"bytes": 2 * n * hkv * _row_bytes(case) + 2 * rows * hq * dim * 2 + rows * hq * 4,
            "flops": 4 * dim * hq * case["new"] * n}


# ------------------------------------------------------------------ inputs


def _starts(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return c


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _pages(g, lens, page):
    """A table of pages in shuffled order for sequences of these lengths, and the number of pages."""
    need = [(n + page - 1) // page for n in lens]
    width, total = max(1, max(need)), sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _filled(g, case, pages):
    """K and V caches [pages, hkv, page, dim] with their scales [pages, hkv, page] (None in 16 bits)."""
    shape = (pages, case["hkv"], case["page"], case["dim"])
    k, v = _randn(g, *shape), _randn(g, *shape)
    if case["cache"] == "bf16":
        return k.to(torch.bfloat16), v.to(torch.bfloat16), None, None
    k8, ks = _quantised(k)
    v8, vs = _quantised(v)
    return k8, v8, ks, vs


def _quantised(x):
    """(e4m3 codes, fp32 scales) of rows along the last dimension: the scale takes the largest magnitude to 448."""
    top = x.abs().amax(dim=-1)
    s = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    return (x / s.unsqueeze(-1)).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    hkv, dim = case["hkv"], case["dim"]
    s = {"case": case}
    if case["op"] == "prepare":
        T, hq, page = case["tokens"], case["hq"], case["page"]
        s["qkv"] = (_randn(g, T, (hq + 2 * hkv) * dim) * 3).to(torch.bfloat16)
        s["qw"] = (1 + 0.2 * _randn(g, dim)).to(torch.bfloat16)
        s["kw"] = (1 + 0.2 * _randn(g, dim)).to(torch.bfloat16)
        i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = (10000.0 ** (-i / case["rot"]) / case["stretch"]).to(torch.float32)
        s["rope_scale"] = 1.0 if case["stretch"] == 1.0 else 0.1 * math.log(case["stretch"]) + 1.0
        lens = [T // case["seqs"] + (b < T % case["seqs"]) for b in range(case["seqs"])]
        s["positions"] = torch.cat([torch.arange(n, device="cuda") + case["first"] + 7 * b
                                    for b, n in enumerate(lens)]).to(torch.int32)
        pages = (T + page - 1) // page + 2
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        s["slots"] = (order[t // page] * page + t % page).to(torch.int32)   # each page filled in order
        shape = (pages, hkv, page, dim)
        kind = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
        s["pages"], s["k"], s["v"] = pages, torch.zeros(shape, device="cuda").to(kind), torch.zeros(shape, device="cuda").to(kind)
        s["ks"] = s["vs"] = None
        if case["cache"] == "e4m3":
            s["ks"], s["vs"] = torch.ones(shape[:3], device="cuda"), torch.ones(shape[:3], device="cuda")
    elif case["op"] == "prefill":
        s["lens_q"], s["lens_k"] = _lens(case["lens_q"]), _lens(case["lens_k"])
        s["cu_q"], s["cu_k"] = _int(_starts(s["lens_q"])), _int(_starts(s["lens_k"]))
        # normalised queries against keys: logits a few units wide, as a trained layer's are
        s["q"] = (_randn(g, sum(s["lens_q"]), case["hq"], dim) * 1.5).to(torch.bfloat16)
        s["k"] = (_randn(g, sum(s["lens_k"]), hkv, dim) * 1.5).to(torch.bfloat16)
        s["v"] = _randn(g, sum(s["lens_k"]), hkv, dim).to(torch.bfloat16)
    else:
        s["lens"] = _lens(case["lens"])
        s["table"], s["pages"] = _pages(g, s["lens"], case["page"])
        s["k"], s["v"], s["ks"], s["vs"] = _filled(g, case, s["pages"])
        if case["op"] == "read":
            s["cu"] = _int(_starts(s["lens"]))
        else:
            s["len"] = _int(s["lens"])
            s["q"] = (_randn(g, len(s["lens"]) * case["new"], case["hq"], dim) * 1.5).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ the library's calls


def _config(m, case):
    return m.attn_config(case.get("hq", case["hkv"]), case["hkv"], case["dim"], case.get("page", 64),
                         m.ATTN_CACHE_E4M3 if case.get("cache") == "e4m3" else m.ATTN_CACHE_BF16)


def _own(s):
    import bit_dequant_expert_b200 as m
    case = s["case"]
    cfg, hkv, dim = _config(m, case), case["hkv"], case["dim"]
    if case["op"] == "prepare":
        T, hq = case["tokens"], case["hq"]
        q = torch.empty(T, hq, dim, dtype=torch.bfloat16, device="cuda")
        k = torch.empty(T, hkv, dim, dtype=torch.bfloat16, device="cuda") if case["keys_too"] else None
        m.attn_qkv_prepare(cfg, T, s["qkv"], s["qkv"].stride(0), s["qw"], s["kw"], EPS, s["inv_freq"], case["rot"],
                           m.ATTN_ROPE_HALF if case["layout"] == "half" else m.ATTN_ROPE_PAIRS, s["rope_scale"],
                           s["positions"], s["slots"], s["pages"], s["k"], s["v"], s["ks"], s["vs"], q, k)
        return [q, k, s["k"], s["v"], s["ks"], s["vs"]]
    if case["op"] == "read":
        n = sum(s["lens"])
        k = torch.empty(n, hkv, dim, dtype=torch.bfloat16, device="cuda")
        v = torch.empty(n, hkv, dim, dtype=torch.bfloat16, device="cuda")
        m.attn_kv_read(cfg, len(s["lens"]), n, s["table"], s["table"].stride(0), s["cu"], s["pages"], s["k"], s["v"],
                       s["ks"], s["vs"], k, v)
        return [k, v]
    q = s["q"]
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    if case["op"] == "prefill":
        m.attn_prefill(cfg, len(s["lens_q"]), q.shape[0], s["k"].shape[0], s["cu_q"], s["cu_k"], q, q.stride(0),
                       s["k"], s["k"].stride(0), s["v"], s["v"].stride(0), dim ** -0.5, case["causal"], out, lse)
        return [out, lse]
    top = max(s["lens"])
    ws = torch.empty(m.attn_decode_workspace_size(cfg, len(s["lens"]), case["new"], top), dtype=torch.uint8, device="cuda")
    m.attn_decode(cfg, len(s["lens"]), case["new"], top, q, q.stride(0), s["table"], s["table"].stride(0), s["len"],
                  s["pages"], s["k"], s["v"], s["ks"], s["vs"], dim ** -0.5, out, lse, ws)
    return [out, lse]


# ------------------------------------------------------------------ plain forms


def _turned(x, case, s):
    """The first rot elements of each head rotated by its token's angles (which 32 bits do not hold)."""
    rot = case["rot"]
    ang = s["positions"].double().unsqueeze(-1) * s["inv_freq"].double()
    cos = (ang.cos() * s["rope_scale"]).float().unsqueeze(1)
    sin = (ang.sin() * s["rope_scale"]).float().unsqueeze(1)
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        t = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        t = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([t, x[..., rot:]], dim=-1)


def _normed(x, w):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w.float()


def _plain_prepare(s):
    case = s["case"]
    T, hq, hkv, dim, page = case["tokens"], case["hq"], case["hkv"], case["dim"], case["page"]
    x = s["qkv"].float().view(T, hq + 2 * hkv, dim)
    q = _turned(_normed(x[:, :hq], s["qw"]), case, s)
    k = _turned(_normed(x[:, hq:hq + hkv], s["kw"]), case, s)
    v = x[:, hq + hkv:]
    slot = s["slots"].long()
    p, o = slot // page, slot % page
    if case["cache"] == "bf16":
        s["k"][p, :, o] = k.to(torch.bfloat16)
        s["v"][p, :, o] = v.to(torch.bfloat16)
    else:
        k8, ks = _quantised(k)
        v8, vs = _quantised(v)
        s["k"].view(torch.uint8)[p, :, o] = k8.view(torch.uint8)
        s["v"].view(torch.uint8)[p, :, o] = v8.view(torch.uint8)
        s["ks"][p, :, o] = ks
        s["vs"][p, :, o] = vs
    return [q.to(torch.bfloat16), k.to(torch.bfloat16) if case["keys_too"] else None, s["k"], s["v"], s["ks"], s["vs"]]


def _gathered(cache, scales, p, o):
    x = cache.float() if scales is None else cache.float() * scales.unsqueeze(-1)
    return x[p, :, o]


def _plain_read(s):
    page = s["case"]["page"]
    lens = torch.diff(s["cu"]).long()
    b = torch.repeat_interleave(torch.arange(len(s["lens"]), device="cuda"), lens, output_size=sum(s["lens"]))
    j = torch.arange(sum(s["lens"]), device="cuda") - s["cu"].long()[b]
    p, o = s["table"].long()[b, j // page], j % page
    return [_gathered(s["k"], s["ks"], p, o).to(torch.bfloat16), _gathered(s["v"], s["vs"], p, o).to(torch.bfloat16)]


def _softmax_av(x, v, visible):
    """Scores [.., q, k] -> (outputs [.., q, d], log of the sum of exponentials): a row that sees no key gives zeros."""
    x.masked_fill_(~visible, -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(m).exp_()
    z = x.sum(dim=-1, keepdim=True)
    return (x @ v) / torch.where(z > 0, z, torch.ones_like(z)), (z.log() + m).squeeze(-1)


def _plain_prefill(s):
    case = s["case"]
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    G, n = hq // hkv, len(s["lens_q"])
    top_q, top_k = max(s["lens_q"]), max(s["lens_k"])
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = torch.diff(cu_q), torch.diff(cu_k)
    i, j = torch.arange(top_q, device="cuda"), torch.arange(top_k, device="cuda")
    # every sequence padded to the longest, rows past its end those of its last token
    rq = (cu_q[:-1, None] + torch.minimum(i[None], lq[:, None] - 1)).clamp(0)
    rk = (cu_k[:-1, None] + torch.minimum(j[None], lk[:, None] - 1)).clamp(0)
    q = s["q"].float()[rq].view(n, top_q, hkv, G, dim).permute(0, 2, 3, 1, 4)
    k = s["k"].float()[rk].permute(0, 2, 3, 1).unsqueeze(2)
    v = s["v"].float()[rk].permute(0, 2, 1, 3).unsqueeze(2)
    seen = j[None, None] < lk[:, None, None]
    if case["causal"]:
        seen = seen & (j[None, None] <= i[None, :, None] + (lk - lq)[:, None, None])
    o, lse = _softmax_av((q * dim ** -0.5) @ k, v, seen[:, None, None])
    inside = i[None] < lq[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, top_q, hq, dim)[inside]
    return [o.to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(n, top_q, hq)[inside]]


def _plain_decode(s):
    case = s["case"]
    hq, hkv, dim, new, page = case["hq"], case["hkv"], case["dim"], case["new"], case["page"]
    G, n, top = hq // hkv, len(s["lens"]), max(s["lens"])
    j, lens = torch.arange(top, device="cuda"), s["len"].long()
    p = s["table"].long()[:, j // page]
    o = (j % page).expand(n, top)
    k = _gathered(s["k"], s["ks"], p, o).permute(0, 2, 3, 1).unsqueeze(2)
    v = _gathered(s["v"], s["vs"], p, o).permute(0, 2, 1, 3).unsqueeze(2)
    q = s["q"].float().view(n, new, hkv, G, dim).permute(0, 2, 3, 1, 4)
    last = lens[:, None] - new + torch.arange(new, device="cuda")
    o, lse = _softmax_av((q * dim ** -0.5) @ k, v, (j[None, None] <= last[..., None])[:, None, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(n * new, hq, dim)
    return [o.to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(n * new, hq)]


def run(state):
    if own:
        return _own(state)
    return {"prepare": _plain_prepare, "read": _plain_read, "prefill": _plain_prefill,
            "decode": _plain_decode}[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits, from the definition


def _exact_rows(x, w, case, s):
    """Heads [T, h, dim] normed and rotated in 64 bits: each pair as a complex number times its angle's."""
    x = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS) * w.double()
    rot = case["rot"]
    ang = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.full_like(ang, s["rope_scale"]), ang)[:, None]
    y = x.clone()
    if case["layout"] == "half":
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def _e4m3(x):
    """Each value rounded to the nearest with four significant bits (halves to even), steps of 2^-9 at the least."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60)))
    step = torch.exp2(torch.clamp(e, min=-6) - 3)
    return torch.round(x / step) * step


def _exact_one(q, k, v, causal):
    """One sequence and head in 64 bits: q [a, d], k and v [b, d]."""
    a, b = q.shape[0], k.shape[0]
    if a == 0 or b == 0:
        return torch.zeros(a, v.shape[-1], dtype=torch.float64, device="cuda"), torch.full((a,), -math.inf, dtype=torch.float64, device="cuda")
    x = q @ k.T * q.shape[-1] ** -0.5
    if causal:
        x = x.masked_fill(torch.ones(a, b, dtype=torch.bool, device="cuda").triu(b - a + 1), -math.inf)
    lse = torch.logsumexp(x, dim=-1)
    w = torch.where(torch.isinf(lse)[:, None], torch.zeros_like(x), torch.exp(x - lse[:, None]))
    return w @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    hkv, dim, page = case["hkv"], case["dim"], case.get("page", 1)
    if case["op"] == "prepare":
        T, hq = case["tokens"], case["hq"]
        x = s["qkv"].double().view(T, hq + 2 * hkv, dim)
        q = _exact_rows(x[:, :hq], s["qw"], case, s)
        k = _exact_rows(x[:, hq:hq + hkv], s["kw"], case, s)
        rows = [k, x[:, hq + hkv:]]
        caches, scales = [], []
        flat = s["slots"].long()
        for row in rows:
            cache = torch.zeros(s["pages"] * page, hkv, dim, dtype=torch.float64, device="cuda")
            scale = torch.ones(s["pages"] * page, hkv, dtype=torch.float64, device="cuda")
            if case["cache"] == "bf16":
                cache[flat] = row
            else:
                scale[flat] = row.abs().amax(-1) / E4M3_MAX
                cache[flat] = _e4m3(row / scale[flat][..., None])
            caches.append(cache.view(s["pages"], page, hkv, dim).transpose(1, 2).contiguous())
            scales.append(scale.view(s["pages"], page, hkv).transpose(1, 2).contiguous())
        if case["cache"] == "bf16":
            scales = [None, None]
        return [q, k if case["keys_too"] else None, *caches, *scales]

    def keys(cache, scale, b, n):
        """[n, hkv, dim]: the first n rows of sequence b, page by page."""
        x = cache[s["table"][b, :(n + page - 1) // page].long()].double()
        if scale is not None:
            x = x * scale[s["table"][b, :(n + page - 1) // page].long()].double()[..., None]
        return x.transpose(1, 2).reshape(-1, hkv, dim)[:n]

    if case["op"] == "read":
        return [torch.cat([keys(c, z, b, n) for b, n in enumerate(s["lens"])]) for c, z in ((s["k"], s["ks"]), (s["v"], s["vs"]))]
    hq = case["hq"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    lens_q = s["lens_q"] if case["op"] == "prefill" else [case["new"]] * len(s["lens"])
    at = at_k = 0
    for b, a in enumerate(lens_q):
        if case["op"] == "prefill":
            k, v = (s[n][at_k:at_k + s["lens_k"][b]].double() for n in ("k", "v"))
            at_k += s["lens_k"][b]
        else:
            k, v = keys(s["k"], s["ks"], b, s["lens"][b]), keys(s["v"], s["vs"], b, s["lens"][b])
        for h in range(hq):
            o, z = _exact_one(s["q"][at:at + a, h].double(), k[:, h * hkv // hq], v[:, h * hkv // hq],
                              case["op"] == "decode" or case["causal"])
            out[at:at + a, h], lse[at:at + a, h] = o, z
        at += a
    return [out, lse]
