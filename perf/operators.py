"""Measured cases of the decoder-layer operators that run next to the
projections: rotary positions, the append of new keys and values to the paged
8-bit cache (rotated on the way), attention over that cache, and the linear
layer with 4-bit weights and group scales.

``listed`` names the cases, ``draw`` gives more of the same ranges, ``prepare``
makes the inputs a program holds before the call, ``run`` makes one pass --
the operator's plain form in elementary torch operations, or (``own``) the
framework's call -- and ``exact`` gives the same outputs from the definition in
64 bits.  ``work`` counts what one pass has to read, write and compute.

Shapes: 32 and 40 heads of 128 (hidden sizes 4096 and 5120) with MLP widths
11008 and 13824 are the linear layers of this repository's workloads; grouped
heads, other head sizes and page sizes are generic.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
SMALLEST = 2.0 ** -126  # the scale of a block that holds only zeros


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # the q and k heads of one token in flight: the smallest call, all latency
        _rope("rotate one token", "bf16", tokens=1, heads=64, dim=128, rot=128, layout="half", inverse=False, context=4096),
        # gradient of the rotation over a training batch's q and k heads
        _rope("rotate back 2048 tokens", "bf16", tokens=2048, heads=80, dim=128, rot=128, layout="half", inverse=True,
              context=4096),
        # a long prompt, half of each head rotated, interleaved pairs, far positions
        _rope("rotate 16383 tokens in part", "f16", tokens=16383, heads=40, dim=128, rot=64, layout="interleaved",
              inverse=False, context=131072),
        # one token for each of 64 running sequences
        _append("append a token to 64", "bf16", seqs=64, new=(1, 1), past=(100, 4000), heads=32, kv_heads=32, dim=128,
                page=64, rot=128, layout="half"),
        # prompts of odd lengths entering the cache
        _append("append 8 prompts", "f16", seqs=8, new=(500, 2100), past=(0, 300), heads=32, kv_heads=8, dim=128, page=32,
                rot=64, layout="interleaved"),
        # one user, a short conversation: latency
        _attend("attend one short", "bf16", seqs=1, new=(1, 1), past=(699, 699), heads=32, kv_heads=32, dim=128, page=64,
                window=0, out="bf16"),
        # a serving batch of uneven lengths, grouped heads
        _attend("attend batch of 48", "bf16", seqs=48, new=(1, 1), past=(200, 4000), heads=32, kv_heads=8, dim=128,
                page=64, window=0, out="bf16"),
        # two very long contexts
        _attend("attend two long", "f16", seqs=2, new=(1, 1), past=(100000, 130000), heads=40, kv_heads=8, dim=128,
                page=128, window=0, out="f16"),
        # a chunk of each of three prompts over what is cached already
        _attend("attend prompt chunks", "bf16", seqs=3, new=(700, 1100), past=(1500, 5000), heads=32, kv_heads=8, dim=128,
                page=64, window=0, out="bf16"),
        # one token through an attention projection
        _w4("w4 one token", "bf16", rows=1, n=4096, k=4096, group=128, zero=False, out="bf16"),
        # sixteen tokens through an MLP projection, groups with a zero point
        _w4("w4 sixteen tokens", "f16", rows=16, n=11008, k=4096, group=64, zero=True, out="f16"),
        # a few tokens through the wider model's MLP projection, 32-bit result
        _w4("w4 five tokens, wide", "bf16", rows=5, n=13824, k=5120, group=32, zero=False, out="f32"),
    ]


def _rope(name, type, **k):
    return {"name": name, "op": "rope", "type": type, **k}


def _append(name, type, new, past, **k):
    return {"name": name, "op": "append", "type": type, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0],
            "past_hi": past[1], **k}


def _attend(name, type, new, past, **k):
    return {"name": name, "op": "attend", "type": type, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0],
            "past_hi": past[1], **k}


def _w4(name, type, **k):
    return {"name": name, "op": "w4", "type": type, **k}


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, dim):
    kv = rng.choice([1, 2, 4, 5, 8, 8, 16, 32] if dim <= 128 else [1, 2, 4, 8])
    return kv * rng.choice([1, 1, 2, 3, 4, 5, 8] if kv <= 8 else [1, 1, 2]), kv


def _drawn(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "w4"])
    t = rng.choice(["bf16", "f16"])
    layout = rng.choice(["half", "interleaved"])
    dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    rot = rng.choice([dim, dim, dim // 2])
    if op == "rope":
        return {"op": op, "type": rng.choice(["bf16", "f16", "f32"]), "tokens": _log(rng, 1, 16383), "heads": _log(rng, 1, 80),
                "dim": dim, "rot": rot, "layout": layout, "inverse": rng.random() < 0.5, "context": _log(rng, 16384, 131072)}
    if op == "append":
        heads, kv = _heads(rng, dim)
        if rng.random() < 0.5:
            new = (1, 1)
        else:
            hi = _log(rng, 2, 4000)
            new = (_log(rng, 1, hi), hi)
        return {"op": op, "type": t, "seqs": _log(rng, 1, 128), "new_lo": new[0], "new_hi": new[1], "past_lo": 0,
                "past_hi": _log(rng, 1, 5000), "heads": heads, "kv_heads": kv, "dim": dim, "page": rng.choice([16, 32, 64, 128]),
                "rot": rot, "layout": layout}
    if op == "attend":
        heads, kv = _heads(rng, dim)
        past = _log(rng, 1, 130000)
        kind = rng.random()
        new = 1 if kind < 0.5 else _log(rng, 2, 8) if kind < 0.7 else _log(rng, 9, 1100)
        return {"op": op, "type": t, "seqs": _log(rng, 1, 128), "new_lo": max(1, new // 2), "new_hi": new,
                "past_lo": past // 4, "past_hi": past, "heads": heads, "kv_heads": kv, "dim": dim,
                "page": rng.choice([16, 32, 64, 128]), "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)]),
                "out": rng.choice([t, t, "f32"])}
    g = rng.choice([32, 64, 128])
    return {"op": op, "type": t, "rows": _log(rng, 1, 32), "n": _log(rng, 64, 13824), "k": g * _log(rng, 1, 13824 // g),
            "group": g, "zero": rng.random() < 0.5, "out": rng.choice([t, t, "f32"])}


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = tuple(max(a, b) for a, b in zip(most.get(c["op"], (0, 0)), (w["bytes"], w["flops"])))
    while True:
        c = _drawn(rng)
        w = work(c)
        if w["bytes"] > most[c["op"]][0] or w["flops"] > most[c["op"]][1]:
            continue
        if c["op"] == "attend":  # the plain form holds every score and a padded copy of the cache
            new, total = _lens(c)
            if c["seqs"] * max(total) * max(c["heads"] * max(new), 4 * c["kv_heads"] * c["dim"]) > 2.5e9:
                continue
        return c


def _lens(case):
    """New tokens of each sequence and its length with them: a part of the case, not of the inputs."""
    r = random.Random("%d %d %d %d %d" % (case["seqs"], case["new_lo"], case["new_hi"], case["past_lo"], case["past_hi"]))
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    past = [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["seqs"])]
    return new, [n + p for n, p in zip(new, past)]


def _seen(new, total, window):
    """Pairs of a query and a key that it attends to, and keys that some query of the sequence attends to."""
    pairs = keys = 0
    for n, t in zip(new, total):
        if window <= 0:
            pairs += n * (t - n) + n * (n + 1) // 2
            keys += t
        else:
            pairs += sum(min(p + 1, window) for p in range(t - n, t))
            keys += min(t, window + n - 1)
    return pairs, keys


def work(case):
    c, size = case, {"bf16": 2, "f16": 2, "f32": 4}
    if c["op"] == "rope":
        x = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 2 * x * size[c["type"]] + c["tokens"] * (4 * c["rot"] + 4),
                "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    if c["op"] == "append":
        new, _ = _lens(c)
        t = sum(new)
        kv = t * c["kv_heads"] * c["dim"]
        blocks = sum(-(-n // c["page"]) for n in new) * c["kv_heads"]
        return {"bytes": 2 * kv * size[c["type"]] + 2 * kv + 8 * blocks + 2 * t * c["heads"] * c["dim"] * size[c["type"]]
                + 4 * t * c["rot"], "flops": t * (3 * (c["heads"] + c["kv_heads"]) * c["rot"] + 2 * 2 * c["kv_heads"] * c["dim"])}
    if c["op"] == "attend":
        new, total = _lens(c)
        pairs, keys = _seen(new, total, c["window"])
        t = sum(new)
        return {"bytes": 2 * keys * c["kv_heads"] * c["dim"] + 8 * (keys // c["page"] + len(new)) * c["kv_heads"]
                + t * c["heads"] * c["dim"] * (size[c["type"]] + size[c["out"]]) + 4 * (keys // c["page"] + 2 * len(new)),
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    groups = c["k"] // c["group"]
    return {"bytes": c["n"] * (c["k"] // 2 + groups * (3 if c["zero"] else 2)) + c["rows"] * c["k"] * size[c["type"]]
            + c["rows"] * c["n"] * size[c["out"]], "flops": 2 * c["rows"] * c["n"] * c["k"]}


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "rope":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        # the heads to rotate lie beside others in one projection's output
        s["x"] = _normal(g, (t, h + 2, d), case["type"])[:, :h]
        start = int(torch.randint(0, case["context"] - t + 1, (1,), generator=g, device="cuda"))
        s["positions"] = torch.arange(start, start + t, dtype=torch.int32, device="cuda")
        s["table"] = _table(case["context"], case["rot"])
    elif case["op"] == "append":
        new, total = _lens(case)
        t, h, hk, d = sum(new), case["heads"], case["kv_heads"], case["dim"]
        qkv = _normal(g, (t, h + 2 * hk, d), case["type"])
        qkv *= torch.exp(0.5 * torch.randn((h + 2 * hk, 1), generator=g, device="cuda")).to(qkv.dtype)
        s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        s["table"] = _table(max(total), case["rot"])
        _cache(s, case, g, new, total)
    elif case["op"] == "attend":
        new, total = _lens(case)
        s["q"] = _normal(g, (sum(new), case["heads"], case["dim"]), case["type"], 1.5)
        s["most_new"], s["most"] = max(new), max(total)
        _cache(s, case, g, new, total)
    else:
        m, n, k, gr = case["rows"], case["n"], case["k"], case["group"]
        s["x"] = _normal(g, (m, k), case["type"])
        w = 0.02 * torch.randn((n, k // gr, gr), generator=g, device="cuda")
        if case["zero"]:
            w += 0.01 * torch.randn((n, k // gr, 1), generator=g, device="cuda")
            lo, hi = w.amin(-1, keepdim=True).clamp(max=0.0), w.amax(-1, keepdim=True).clamp(min=0.0)
            scale = ((hi - lo) / 15).to(TYPES[case["type"]])
            zero = torch.round(-lo / scale.float()).clamp(0, 15)
            s["zero"] = zero.squeeze(-1).to(torch.uint8)
        else:
            scale = (w.abs().amax(-1, keepdim=True) / 7).to(TYPES[case["type"]])
            zero = 8.0
            s["zero"] = None
        q = (torch.round(w / scale.float()) + zero).clamp(0, 15).to(torch.uint8).view(n, k // 2, 2)
        s["q"] = (q[..., 0] | (q[..., 1] << 4)).contiguous()  # the even column in the low half of a byte
        s["scale"] = scale.squeeze(-1).contiguous()
        if own:
            from sparse_gemm_amd import patch
            s["weight"] = patch.w4_pack(s["q"], s["scale"], s["zero"], gr)
    return s


def _normal(g, shape, type, std=1.0):
    return (std * torch.randn(shape, generator=g, device="cuda")).to(TYPES[type])


def _table(context, rot):
    """cos (first half of a row) and sin (second half) of each position's angles, computed in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(context, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _cache(s, case, g, new, total):
    """Cache pages with the sequences' earlier tokens, in a shuffled order, and the tables that find them."""
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["page_table"] = torch.full((len(need), max(need)), -1, dtype=torch.int32, device="cuda")
    row = torch.repeat_interleave(torch.arange(len(need)), torch.tensor(need))
    first = torch.tensor([0] + need).cumsum(0)
    col = torch.arange(sum(need)) - first[row]
    s["page_table"][row.cuda(), col.cuda()] = order[:sum(need)]
    s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["cu_new"] = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    for name in ("k", "v"):
        x = torch.randn((pages, hk, page, d), generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn((pages, hk, 1, 1), generator=g, device="cuda"))
        scale = _scale_for(x.abs().amax((2, 3)))
        s[name + "_cache"] = (x / scale[:, :, None, None]).to(E4M3)
        s[name + "_scale"] = scale
    if own:
        from sparse_gemm_amd import patch
        s["cache"] = patch.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])


def _scale_for(most):
    """The smallest power of two that brings `most` to 448 or less."""
    m, e = torch.frexp(most / E4M3_MAX)
    return torch.ldexp(torch.ones_like(most), torch.where(m == 0.5, e - 1, e)).clamp(min=SMALLEST)


# ---------------------------------------------------------------------------- one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_rope(s):
    from sparse_gemm_amd import patch
    c = s["case"]
    return patch.rope(s["x"], s["positions"], s["table"], layout=c["layout"], inverse=c["inverse"])


def _own_append(s):
    from sparse_gemm_amd import patch
    q = patch.kv_append(s["k"], s["v"], s["cache"], s["page_table"], s["lens"], s["cu_new"], table=s["table"],
                        layout=s["case"]["layout"], q=s["q"])
    return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _own_attend(s):
    from sparse_gemm_amd import patch
    c = s["case"]
    return patch.attention(s["q"], s["cache"], s["page_table"], s["lens"], s["cu_new"], window=c["window"],
                           out_dtype=TYPES[c["out"]])


def _own_w4(s):
    from sparse_gemm_amd import patch
    return patch.w4_gemm(s["x"], s["weight"], out_dtype=TYPES[s["case"]["out"]])


def _rotate(x, cos, sin, layout, rot):
    """x [..., heads, dim] in 32 bits; cos, sin [..., 1, rot / 2]."""
    r = x[..., :rot]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([r, x[..., rot:]], dim=-1)


def _plain_rope(s):
    c = s["case"]
    row = s["table"][s["positions"].long()][:, None]
    cos, sin = row[..., :c["rot"] // 2], row[..., c["rot"] // 2:]
    return _rotate(s["x"].float(), cos, -sin if c["inverse"] else sin, c["layout"], c["rot"]).to(s["x"].dtype)


def _plain_append(s):
    c = s["case"]
    page, rot, t = c["page"], c["rot"], s["k"].shape[0]
    at = torch.arange(t, device="cuda")
    seq = torch.searchsorted(s["cu_new"].long(), at, right=True) - 1
    n = (s["cu_new"][1:] - s["cu_new"][:-1]).long()
    past = s["lens"].long() - n
    pos = past[seq] + at - s["cu_new"].long()[seq]
    row = s["table"][pos][:, None]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    q = _rotate(s["q"].float(), cos, sin, c["layout"], rot).to(s["q"].dtype)
    block = s["page_table"][seq, pos // page].long()  # each token's page
    first = s["page_table"][torch.arange(len(n), device="cuda"), past // page].long()  # the page that may hold earlier tokens
    held = past % page
    for name, x in (("k", _rotate(s["k"].float(), cos, sin, c["layout"], rot)), ("v", s["v"].float())):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        most = torch.zeros_like(scale).scatter_reduce(0, block[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
        want = _scale_for(most)
        keep = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda")
        keep[first[(held > 0) & (n > 0)]] = True
        want = torch.where(keep[:, None], torch.maximum(want, scale), want)
        written = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda")
        written[block] = True
        want = torch.where(written[:, None], want, scale)
        old = cache[first].float() * (scale[first] / want[first])[:, :, None, None]  # earlier tokens under the new scale
        stays = torch.arange(page, device="cuda")[None] < held[:, None]
        i, j = torch.nonzero(stays & (n > 0)[:, None], as_tuple=True)
        bits = cache.view(torch.uint8)
        bits[first[i], :, j] = old[i, :, j].to(E4M3).view(torch.uint8)
        bits[block, :, pos % page] = (x / want[block][:, :, None]).to(E4M3).view(torch.uint8)
        scale.copy_(want)
    return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain_attend(s):
    c = s["case"]
    page, h, hk, d = c["page"], c["heads"], c["kv_heads"], c["dim"]
    seqs, most, most_new = len(s["lens"]), s["most"], s["most_new"]
    pages = s["page_table"].long().clamp(min=0)
    start, n, total = s["cu_new"][:-1].long(), (s["cu_new"][1:] - s["cu_new"][:-1]).long(), s["lens"].long()
    i = torch.arange(most_new, device="cuda")
    token = (start[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][token].float().view(seqs, most_new, hk, h // hk, d).permute(0, 2, 3, 1, 4)  # seq, kv head, head, new, dim

    def values(name):
        x = s[name + "_cache"][pages].float() * s[name + "_scale"][pages][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(seqs, hk, -1, d)

    score = torch.matmul(q.reshape(seqs, hk, -1, d), values("k").transpose(2, 3)) * d ** -0.5
    score = score.view(seqs, hk, h // hk, most_new, -1)
    key = torch.arange(score.shape[-1], device="cuda")
    pos = (total - n)[:, None] + i
    hidden = key > pos[..., None]
    if c["window"] > 0:
        hidden = hidden | (key <= pos[..., None] - c["window"])
    score = score.masked_fill(hidden[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = values("v").masked_fill((key >= total[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.view(seqs, hk, -1, p.shape[-1]), v).view(seqs, hk, h // hk, most_new, d)
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, most_new, h, d)
    return o[i < n[:, None]].to(TYPES[c["out"]])


def _plain_w4(s):
    c = s["case"]
    q = torch.stack([s["q"] & 15, s["q"] >> 4], dim=-1).view(c["n"], -1, c["group"]).float()
    zero = 8.0 if s["zero"] is None else s["zero"].float()[..., None]
    w = ((q - zero) * s["scale"].float()[..., None]).view(c["n"], c["k"])
    return torch.matmul(s["x"].float(), w.t()).to(TYPES[c["out"]])


_plain = {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "w4": _plain_w4}
_own = {"rope": _own_rope, "append": _own_append, "attend": _own_attend, "w4": _own_w4}


# ---------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    return _exact[case["op"]](case, prepare(case, seed))


def _turn(x, table, pos, layout, back=False):
    """Each pair of x [tokens, heads, dim] (64 bits) as a complex number, turned by its position's angle."""
    row = table[pos].double()
    half = row.shape[1] // 2
    by = torch.complex(row[:, :half], -row[:, half:] if back else row[:, half:])[:, None]
    out = x.clone()
    if layout == "half":
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * by
        out[..., :half], out[..., half:2 * half] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:2 * half:2], x[..., 1:2 * half:2]) * by
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = z.real, z.imag
    return out


def _exact_rope(case, s):
    return _turn(s["x"].double(), s["table"], s["positions"].long(), case["layout"], case["inverse"])


def _e4m3(x):
    """Round to the nearest value of three fraction bits (even on a tie), least exponent -6."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_append(case, s):
    page = case["page"]
    new, total = _lens(case)
    cache = {m: s[m + "_cache"].double() for m in "kv"}
    scale = {m: s[m + "_scale"].double() for m in "kv"}
    q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    table = s["page_table"].tolist()
    t = 0
    for r, (n, end) in enumerate(zip(new, total)):
        begin = end - n
        pos = torch.arange(begin, end, device="cuda")
        q[t:t + n] = _turn(s["q"][t:t + n].double(), s["table"], pos, case["layout"])
        x = {"k": _turn(s["k"][t:t + n].double(), s["table"], pos, case["layout"]), "v": s["v"][t:t + n].double()}
        for b in range(begin // page, (end - 1) // page + 1):
            p, lo, hi = table[r][b], max(begin, b * page), min(end, (b + 1) * page)
            for m in "kv":
                y = x[m][lo - begin:hi - begin].transpose(0, 1)  # heads, tokens, dim
                want = torch.exp2(torch.ceil(torch.log2(y.abs().amax((1, 2)) / E4M3_MAX))).clamp(min=SMALLEST)
                if lo > b * page:
                    want = torch.maximum(want, scale[m][p])
                    kept = cache[m][p][:, :lo - b * page]
                    cache[m][p][:, :lo - b * page] = _e4m3(kept * (scale[m][p] / want)[:, None, None])
                scale[m][p] = want
                cache[m][p][:, lo - b * page:hi - b * page] = _e4m3(y / want[:, None, None])
        t += n
    return q, cache["k"], cache["v"], scale["k"], scale["v"]


def _exact_attend(case, s):
    page, h, hk, d, w = case["page"], case["heads"], case["kv_heads"], case["dim"], case["window"]
    new, total = _lens(case)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    t = 0
    for r, (n, end) in enumerate(zip(new, total)):
        pages = s["page_table"][r, :-(-end // page)].long()
        pos = torch.arange(end - n, end, device="cuda")[:, None]
        key = torch.arange(end, device="cuda")[None]
        seen = (key <= pos) & ((key > pos - w) if w > 0 else True)
        for j in range(hk):
            k, v = (s[m + "_cache"][pages, j].double() * s[m + "_scale"][pages, j].double()[:, None, None] for m in "kv")
            k, v = k.reshape(-1, d)[:end], v.reshape(-1, d)[:end]
            for i in range(j * (h // hk), (j + 1) * (h // hk)):
                a = (s["q"][t:t + n, i].double() @ k.t()) / math.sqrt(d)
                out[t:t + n, i] = torch.softmax(a.masked_fill(~seen, -math.inf), dim=-1) @ v
        t += n
    return out


def _exact_w4(case, s):
    k = torch.arange(case["k"], device="cuda")
    q = ((s["q"][:, k // 2].int() >> (4 * (k % 2))) & 15).double()
    z = torch.full_like(s["scale"], 8).double() if s["zero"] is None else s["zero"].double()
    g = k // case["group"]
    return s["x"].double() @ ((q - z[:, g]) * s["scale"].double()[:, g]).t()


_exact = {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend, "w4": _exact_w4}
