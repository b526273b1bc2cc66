"""Plain 64-bit implementations of the decoder-layer operators (rotary
positions, cache append, attention over the cache, 4-bit linear layer), on the
CPU, and the error bounds the GPU results are held to.

Every bound is built from roundings: one to a type t costs at most eps(t) / 2
of the value (bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4), fp32 sums of n
terms at most n roundings of the sum of the terms' sizes.
"""
import math

import numpy as np
import torch

U32 = 2.0 ** -24
HALF_EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the least subnormal
E4M3_MAX = 448.0


def f64(t):
    return t.detach().cpu().double()


# ---------------------------------------------------------------------------- rotary positions
def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        turns = original * f / (2 * math.pi)
        g = np.clip((turns - low) / (high - low), 0.0, 1.0)
        f = g * f + (1 - g) * f / factor
    return f


def table(positions, rot, magnitude=1.0, **kw):
    a = np.arange(positions, dtype=np.float64)[:, None] * frequencies(rot, **kw)
    return magnitude * torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], axis=1))


def pairs(x, rot, layout):
    if layout == "half":
        return x[..., :rot // 2], x[..., rot // 2:rot]
    return x[..., 0:rot:2], x[..., 1:rot:2]


def rope(x, positions, tab, layout, inverse=False):
    """x [T, H, D] in 64 bits; returns the result and the error bound of an
    fp32 computation of it (two products and a sum a value)."""
    rot = tab.shape[1]
    row = tab[positions.long().clamp(0, tab.shape[0] - 1)][:, None]
    bad = (positions < 0) | (positions >= tab.shape[0])
    row = torch.where(bad[:, None, None], torch.full_like(row, math.nan), row)
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    if inverse:
        s = -s
    a, b = pairs(x, rot, layout)
    y, err = x.clone(), torch.zeros_like(x)
    ya, yb = pairs(y, rot, layout)
    ea, eb = pairs(err, rot, layout)
    ya_, yb_ = a * c - b * s, b * c + a * s
    ea.copy_(3 * U32 * ((a * c).abs() + (b * s).abs()))
    eb.copy_(3 * U32 * ((b * c).abs() + (a * s).abs()))
    ya.copy_(ya_)
    yb.copy_(yb_)
    return y, err


def assert_within(got, want, bound, what=""):
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN at other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]) and not torch.isinf(got[~inf]).any(), f"{what}: infinite at other places"
    fine = torch.isfinite(want)
    d = (got - want).abs()
    over = fine & ~(d <= bound)
    if over.any():
        i = tuple(int(v) for v in torch.nonzero(over)[0])
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} values off, first at {i}: {got[i]} for "
                             f"{want[i]}, bound {bound[i]}; worst {float((d / bound)[fine].max()):.3g} times the bound")


def rounded(want, dtype, err=0.0):
    """The bound of a value computed within err and rounded to dtype."""
    return HALF_EPS[dtype] * (want.abs() + err) + err + TINY[dtype]


# ---------------------------------------------------------------------------- cache append
def scale_for(amax):
    """2^ceil(log2(amax / 448)), at least 2^-126, exactly."""
    if amax == 0:
        return 2.0 ** -126
    m, e = math.frexp(amax / E4M3_MAX)  # 448 is a sum of three powers of two: the quotient is near exact in 64 bits
    return max(2.0 ** (e - 1 if m == 0.5 else e), 2.0 ** -126)


def e4m3(x):
    """Nearest e4m3 value in 64 bits, even on a tie; not finite: NaN."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where((a > 0) & torch.isfinite(a), a, torch.ones_like(a)))).clamp(min=-6)
    step = torch.pow(2.0, e - 3)
    r = torch.round(a / step) * step
    r = torch.where(torch.isfinite(a), r, torch.full_like(a, math.nan))
    return torch.copysign(r, x)


def append(k, v, q, cache, page_table, kv_lens, cu_new, tab, layout):
    """cache: dict of k, v (64-bit e4m3 values [pages, heads, page, dim]),
    k_scale, v_scale, changed in place.  Returns the rotated q and its bound,
    and for k and v each the lowest and highest value a place may hold
    (fp32 rotation may fall on the other side of an 8-bit border)."""
    T = k.shape[0]
    P, H, B, D = cache["k"].shape
    pos = torch.full((T,), -1, dtype=torch.long)
    seq = torch.full((T,), -1, dtype=torch.long)
    for s in range(len(kv_lens)):
        c0, c1 = int(cu_new[s]), int(cu_new[s + 1])
        for t in range(max(c0, 0), min(c1, T)):
            pos[t] = int(kv_lens[s]) - (c1 - t)
            seq[t] = s
    zero = torch.zeros_like
    if tab is not None:
        kr, ke = rope(k, pos, tab, layout)
        qr, qe = rope(q, pos, tab, layout) if q is not None else (None, None)
    else:
        kr, ke = k.clone(), zero(k)
        qr, qe = (q.clone(), zero(q)) if q is not None else (None, None)
    lo = {"k": cache["k"].clone(), "v": cache["v"].clone()}
    hi = {"k": cache["k"].clone(), "v": cache["v"].clone()}
    for s in range(len(kv_lens)):
        c0, c1 = int(cu_new[s]), int(cu_new[s + 1])
        by_page = {}
        for t in range(max(c0, 0), min(c1, T)):
            p = int(pos[t])
            if p < 0 or p // B >= page_table.shape[1]:
                continue
            page = int(page_table[s, p // B])
            if 0 <= page < P:
                by_page.setdefault((page, p // B), []).append(t)
        for (page, index), ts in by_page.items():
            first = int(pos[ts[0]]) % B
            for name, x, e in (("k", kr, ke), ("v", v, zero(v))):
                for h in range(H):
                    y = x[ts, h]
                    fin = y[torch.isfinite(y)].abs()
                    want = scale_for(float(fin.max()) if fin.numel() else 0.0)
                    old = float(cache[name + "_scale"][page, h])
                    if first > 0:
                        if want > old:
                            held = e4m3(cache[name][page, h, :first] * (old / want))
                            for c in (cache[name], lo[name], hi[name]):
                                c[page, h, :first] = held
                        else:
                            want = old
                    cache[name + "_scale"][page, h] = want
                    inv = float(np.float32(1.0) / np.float32(want))
                    d = e[ts, h] + U32 * y.abs()
                    cache[name][page, h, first:first + len(ts)] = e4m3(y * inv)
                    lo[name][page, h, first:first + len(ts)] = e4m3((y - d) * inv)
                    hi[name][page, h, first:first + len(ts)] = e4m3((y + d) * inv)
    return qr, qe, lo, hi


# ---------------------------------------------------------------------------- attention
def attention(q, cache, page_table, kv_lens, cu_new, scale, window):
    """q in 64 bits; cache: dict as above.  Returns out and lse, the sum of p
    |v| (out's size) and the largest error of a score in fp32."""
    T, Hq, D = q.shape
    P, H, B, _ = cache["k"].shape
    group = Hq // H
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    size = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    ds = torch.zeros(T, Hq, dtype=torch.float64)
    for s in range(len(kv_lens)):
        c0, c1, L = int(cu_new[s]), int(cu_new[s + 1]), int(kv_lens[s])
        n = c1 - c0
        if n <= 0:
            continue
        if L > page_table.shape[1] * B:
            out[c0:c1], lse[c0:c1], size[c0:c1] = math.nan, math.nan, math.nan
            continue
        for i in range(n):
            p = L - n + i
            if p < 0:
                continue
            key = torch.arange(max(0, p - window + 1) if window > 0 else 0, p + 1)
            page = page_table[s, key // B].long()
            if ((page < 0) | (page >= P)).any():
                out[c0 + i], lse[c0 + i], size[c0 + i] = math.nan, math.nan, math.nan
                continue
            for h in range(H):
                k = cache["k"][page, h, key % B] * cache["k_scale"][page, h][:, None]
                v = cache["v"][page, h, key % B] * cache["v_scale"][page, h][:, None]
                x = q[c0 + i, h * group:(h + 1) * group]
                a = (x @ k.T) * scale
                m = a.max(dim=1, keepdim=True).values
                e = torch.exp(a - m)
                l = e.sum(1, keepdim=True)
                sl = slice(h * group, (h + 1) * group)
                pr = e / l
                out[c0 + i, sl] = pr @ v
                size[c0 + i, sl] = pr @ v.abs()
                lse[c0 + i, sl] = (m + torch.log(l))[:, 0]
                ds[c0 + i, sl] = ((x.abs() @ k.abs().T) * abs(scale)).max(1).values * (D + 8) * U32 + a.abs().max(
                    1).values * 4 * U32
    return out, lse, size, ds


def attention_bound(out, size, ds, n_keys, dtype):
    """p is e^score in fp32 (an error of ds in the score is one of ds in p;
    the exponential's own and the scalings' some fp32 roundings), rounded to
    11 bits; the sums of n_keys terms are fp32."""
    err = size * (2.0 ** -11 + 2 * ds[..., None] + (2 * n_keys + 32) * U32)
    return rounded(out, dtype, err)


# ---------------------------------------------------------------------------- 4-bit weights
def w4_weight(q, scale, zero, group):
    q = q.cpu()
    n = q.shape[0]
    x = torch.stack([q & 15, q >> 4], dim=-1).reshape(n, -1, group).double()
    z = 8.0 if zero is None else zero.cpu().double()[..., None]
    s = f64(scale)[..., None]
    size = (x + 16 + z + 16).reshape(n, -1) * s.abs().expand_as(x).reshape(n, -1)
    return ((x - z) * s).reshape(n, -1), size


def w4_bound(x, want, size, group, dtype):
    """Sums of x (16 + q) and x (16 + z) in fp32: at most a rounding a term,
    and one a group after the scale."""
    err = (x.abs() @ size.T) * U32 * (group + x.shape[1] // group + 16)
    return rounded(want, dtype, err)


def w4_quantize(w, group, with_zero, dtype):
    """The stated rounding, fp32 as the definition has it (numpy)."""
    w = w.float().cpu().numpy().reshape(w.shape[0], -1, group)
    f = np.float32
    if with_zero:
        lo, hi = np.minimum(w.min(-1), f(0)), np.maximum(w.max(-1), f(0))
        st = torch.from_numpy((hi - lo) / f(15)).to(dtype)
        s = st.float().numpy()
        ok = s > 0
        sd = np.where(ok, s, f(1))
        z = np.where(ok, np.clip(np.rint(-lo / sd), 0, 15), f(8)).astype(f)
        least = 0
    else:
        st = torch.from_numpy(np.abs(w).max(-1) / f(7)).to(dtype)
        s = st.float().numpy()
        ok = s > 0
        sd = np.where(ok, s, f(1))
        z = np.full_like(s, 8)
        least = 1
    q = np.where(ok[..., None], np.clip(np.rint(w / sd[..., None]) + z[..., None], least, 15), 8).astype(np.uint8)
    q = q.reshape(w.shape[0], -1)
    return (torch.from_numpy(q[:, 0::2] | (q[:, 1::2] << 4)), st,
            torch.from_numpy(z.astype(np.uint8)) if with_zero else None)
