"""CPU checks of the decoder-layer operators: what their entry points refuse
before any GPU call, and the properties of the 64-bit reference the GPU
results are compared with."""
import ctypes
import math

import pytest
import torch

from sparse_gemm_amd import patch
from tests import layer_ref as ref

V = ctypes.c_void_p
P = 4096  # an address that is never read: every call below is refused


def _name(rc):
    return patch.STATUS[rc]


def _rope(**kw):
    f = dict(dtype=1, layout=0, inverse=0, T=4, H=2, D=64, rot=64, context=16, x=P, xt=128, xh=64, out=P + 4096, ot=128,
             oh=64, pos=P, table=P)
    f.update(kw)
    return _name(patch.load().patch_rope(patch._ROPE_ARGS.pack(*f.values()), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), "INVALID_ARG"), (dict(layout=2), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"),
    (dict(H=0), "SHAPE"), (dict(D=63), "SHAPE"), (dict(rot=66), "SHAPE"), (dict(rot=63), "SHAPE"), (dict(rot=0), "SHAPE"),
    (dict(context=0), "INVALID_ARG"), (dict(x=0), "INVALID_ARG"), (dict(out=0), "INVALID_ARG"),
    (dict(pos=0), "INVALID_ARG"), (dict(table=0), "INVALID_ARG"), (dict(table=P + 4), "INVALID_ARG"),
    (dict(x=P + 1), "INVALID_ARG"), (dict(pos=P + 2), "INVALID_ARG"), (dict(out=P, ot=64), "INVALID_ARG"),
    (dict(T=1 << 40), "SHAPE"),
])
def test_rope_refuses(change, status):
    assert _rope(**change) == "PATCH_ERR_" + status


def test_rope_of_nothing_is_a_no_op():
    assert _rope(T=0) == "PATCH_OK"


@pytest.mark.parametrize("args,status", [
    ((0, 64, 1e4, 0, 1., 0., 1., 32., 1., V(P)), "SHAPE"), ((16, 63, 1e4, 0, 1., 0., 1., 32., 1., V(P)), "SHAPE"),
    ((16, 64, 1.0, 0, 1., 0., 1., 32., 1., V(P)), "INVALID_ARG"),
    ((16, 64, math.nan, 0, 1., 0., 1., 32., 1., V(P)), "INVALID_ARG"),
    ((16, 64, 1e4, 4, 1., 0., 1., 32., 1., V(P)), "INVALID_ARG"),
    ((16, 64, 1e4, 1, 0.5, 0., 1., 32., 1., V(P)), "INVALID_ARG"),
    ((16, 2, 1e4, 2, 4., 0., 1., 32., 1., V(P)), "SHAPE"),
    ((16, 64, 1e4, 3, 4., 0., 1., 32., 1., V(P)), "INVALID_ARG"),
    ((16, 64, 1e4, 3, 4., 64., 32., 32., 1., V(P)), "INVALID_ARG"),
    ((16, 64, 1e4, 0, 1., 0., 1., 32., math.inf, V(P)), "INVALID_ARG"),
    ((16, 64, 1e4, 0, 1., 0., 1., 32., 1., None), "INVALID_ARG"),
    ((16, 64, 1e4, 0, 1., 0., 1., 32., 1., V(P + 4)), "INVALID_ARG"),
])
def test_rope_table_refuses(args, status):
    assert _name(patch.load().patch_rope_table(*args, None)) == "PATCH_ERR_" + status


def _cache(**kw):
    f = dict(k=P, v=P, ks=P, vs=P, pages=8, heads=2, page=16, dim=64)
    f.update(kw)
    return patch._CACHE_ARGS.pack(*f.values())


BAD_CACHE = [(dict(page=24), "SHAPE"), (dict(page=8), "SHAPE"), (dict(page=256), "SHAPE"), (dict(dim=72), "SHAPE"),
             (dict(dim=272), "SHAPE"), (dict(dim=0), "SHAPE"), (dict(pages=0), "SHAPE"), (dict(heads=0), "SHAPE"),
             (dict(k=0), "INVALID_ARG"), (dict(vs=0), "INVALID_ARG"), (dict(v=P + 8), "INVALID_ARG"),
             (dict(ks=P + 2), "INVALID_ARG")]
BAD_SEQS = [(dict(T=-1), "INVALID_ARG"), (dict(S=-1), "INVALID_ARG"), (dict(S=4097), "SHAPE"), (dict(T=1 << 30), "SHAPE"),
            (dict(heads=3), "SHAPE"), (dict(heads=0), "SHAPE"), (dict(max_pages=-1), "SHAPE"),
            (dict(max_pages=1 << 28, row=1 << 28), "SHAPE"), (dict(row=3), "SHAPE"), (dict(pt=0), "INVALID_ARG"),
            (dict(lens=0), "INVALID_ARG"), (dict(cu=0), "INVALID_ARG"), (dict(cu=P + 2), "INVALID_ARG"),
            (dict(q=P + 1), "INVALID_ARG")]


def _append(cache=None, **kw):
    f = dict(dtype=1, layout=0, T=4, S=2, heads=4, rot=64, context=16, max_pages=4, k=P, kt=128, kh=64, v=P, vt=128, vh=64,
             q=P, qt=256, qh=64, qo=P + 4096, qot=256, qoh=64, pt=P, row=4, lens=P, cu=P, table=P)
    f.update(kw)
    return _name(patch.load().patch_kv_append(patch._APPEND_ARGS.pack(*f.values()), _cache(**(cache or {})), None))


def _attend(cache=None, ws=(0, 0), **kw):
    f = dict(dtype=1, out_dtype=1, T=4, S=2, heads=4, max_pages=4, window=0, scale=0.125, q=P, qt=256, qh=64, out=P, ot=256,
             oh=64, lse=0, pt=P, row=4, lens=P, cu=P)
    f.update(kw)
    return _name(patch.load().patch_attention(patch._ATTENTION_ARGS.pack(*f.values()), _cache(**(cache or {})),
                                              ws[0] or None, ws[1], None))


@pytest.mark.parametrize("change,status", BAD_SEQS + [
    (dict(dtype=2), "INVALID_ARG"), (dict(layout=-1), "INVALID_ARG"), (dict(rot=66), "SHAPE"), (dict(rot=7), "SHAPE"),
    (dict(context=0), "INVALID_ARG"), (dict(table=P + 8), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"),
    (dict(v=0), "INVALID_ARG"), (dict(qo=0), "INVALID_ARG"), (dict(qo=P, qot=64), "INVALID_ARG"),
    (dict(k=P + 1), "INVALID_ARG")])
def test_append_refuses(change, status):
    assert _append(**change) == "PATCH_ERR_" + status


@pytest.mark.parametrize("change,status", BAD_SEQS + [
    (dict(dtype=2), "INVALID_ARG"), (dict(out_dtype=0), "INVALID_ARG"), (dict(scale=math.nan), "INVALID_ARG"),
    (dict(scale=1e300), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"), (dict(q=0), "INVALID_ARG"),
    (dict(out=0), "INVALID_ARG"), (dict(out=P + 1), "INVALID_ARG"), (dict(lse=P + 2), "INVALID_ARG"),
    (dict(ws=(0, 64)), "INVALID_ARG"), (dict(ws=(P + 8, 64)), "INVALID_ARG"),
    (dict(T=(1 << 30) - 1, heads=8), "SHAPE"), (dict(scale=-1e31), "INVALID_ARG")])
def test_attention_refuses(change, status):
    assert _attend(**change) == "PATCH_ERR_" + status


@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_a_bad_cache_is_refused(change, status):
    assert _append(cache=change) == "PATCH_ERR_" + status
    assert _attend(cache=change) == "PATCH_ERR_" + status


def test_no_tokens_or_sequences_is_a_no_op():
    for kw in (dict(T=0), dict(S=0)):
        assert _append(**kw) == "PATCH_OK"
        assert _attend(**kw) == "PATCH_OK"


@pytest.mark.parametrize("N,K,group,status", [(0, 128, 32, "SHAPE"), (16, 0, 32, "SHAPE"), (16, 96, 64, "SHAPE"),
                                              (16, 128, 48, "SHAPE"), (1 << 23, 128, 32, "SHAPE")])
def test_w4_shapes_refused(N, K, group, status):
    lib = patch.load()
    assert lib.patch_w4_bytes(N, K, group, 0) == 0
    assert _name(lib.patch_w4_quantize(1, N, K, group, V(P), V(P), V(P), None, None)) == "PATCH_ERR_" + status
    assert _name(lib.patch_w4_pack(1, N, K, group, V(P), V(P), None, V(P), 1 << 40, None)) == "PATCH_ERR_" + status
    assert _name(lib.patch_w4_gemm(1, N, K, group, 0, V(P), 1 << 40, V(P), 1, V(P), 1, None)) == "PATCH_ERR_" + status


def test_w4_arguments_refused():
    lib = patch.load()
    n = lib.patch_w4_bytes(40, 160, 32, 1)
    # 3 bands of 2 blocks of 1 KB, 3 x 16 rows of 8 groups (K padded to 256) of a 2-byte scale and a zero byte
    assert n == 3 * 2 * 1024 + 48 * 8 * 3
    g = lambda dt=1, z=1, p=P, b=n, x=P, m=1, y=P, yd=1: _name(  # noqa: E731
        lib.patch_w4_gemm(dt, 40, 160, 32, z, V(p), b, V(x), m, V(y), yd, None))
    assert g(dt=2) == g(yd=0) == g(m=-1) == g(p=0) == g(x=0) == g(y=0) == g(p=P + 8) == g(x=P + 2) == "PATCH_ERR_INVALID_ARG"
    assert g(b=n - 1) == "PATCH_ERR_BUFFER_TOO_SMALL"
    assert g(m=0) == "PATCH_OK"
    assert _name(lib.patch_w4_pack(1, 40, 160, 32, V(P), V(P), V(P), V(P), n - 1, None)) == "PATCH_ERR_BUFFER_TOO_SMALL"
    assert _name(lib.patch_w4_pack(1, 40, 160, 32, V(P + 2), V(P), V(P), V(P), n, None)) == "PATCH_ERR_INVALID_ARG"
    assert _name(lib.patch_w4_quantize(2, 40, 160, 32, V(P), V(P), V(P), None, None)) == "PATCH_ERR_INVALID_ARG"
    assert _name(lib.patch_w4_quantize(1, 40, 160, 32, None, V(P), V(P), None, None)) == "PATCH_ERR_INVALID_ARG"


# ---------------------------------------------------------------------------- the binding, on CPU tensors
def _cpu_cache(pages=4, heads=2, page=16, dim=32):
    z = lambda: torch.zeros((pages, heads, page, dim), dtype=torch.uint8)  # noqa: E731
    return z(), z(), torch.zeros(pages, heads), torch.zeros(pages, heads)


def test_binding_checks_types_and_shapes():
    x = torch.zeros(3, 2, 32, dtype=torch.bfloat16)
    pos, tab = torch.zeros(3, dtype=torch.int32), torch.zeros(8, 32)
    for bad, msg in ((lambda: patch.rope(x[0], pos, tab), "3-D"), (lambda: patch.rope(x.long(), pos, tab), "dtype"),
                     (lambda: patch.rope(x, pos.long(), tab), "int32"), (lambda: patch.rope(x, pos[:2], tab), "int32"),
                     (lambda: patch.rope(x, pos, tab.double()), "table"), (lambda: patch.rope(x, pos, None), "table"),
                     (lambda: patch.rope(x, pos, tab, layout="pairs"), "layout"),
                     (lambda: patch.rope(x.transpose(1, 2), pos, tab), "contiguous"),
                     (lambda: patch.rope(x, pos, tab), "device")):
        with pytest.raises((ValueError, TypeError), match=msg):
            bad()
    k, v, ks, vs = _cpu_cache()
    for bad, msg in ((lambda: patch.KVCache(k[0], v, ks, vs), "4-D"), (lambda: patch.KVCache(k.float(), v, ks, vs), "uint8"),
                     (lambda: patch.KVCache(k, v[:2], ks, vs), "shape"), (lambda: patch.KVCache(k, v, ks[:1], vs), "shape"),
                     (lambda: patch.KVCache(k, v, ks.double(), vs), "float32"),
                     (lambda: patch.KVCache(k.transpose(1, 2), v, ks, vs), "contiguous"),
                     (lambda: patch.KVCache(*_cpu_cache(page=24)), "16, 32, 64 or 128"),
                     (lambda: patch.KVCache(*_cpu_cache(dim=40)), "multiple of 16"),
                     (lambda: patch.KVCache(k, v, ks, vs), "device")):
        with pytest.raises(ValueError, match=msg):
            bad()
    with pytest.raises(ValueError, match="itself"):
        patch.rope(x, pos, tab, out=x[:, :1].expand(3, 2, 32))
    for fn in (patch.kv_append, patch.attention):
        with pytest.raises(ValueError, match="KVCache"):
            fn(x, x, *(None,) * 4) if fn is patch.kv_append else fn(x, None, None, None, None)
    with pytest.raises(ValueError, match="group"):
        patch.w4_pack(torch.zeros(4, 24, dtype=torch.uint8), torch.zeros(4, 1), None, 48)
    with pytest.raises(ValueError, match="W4Weight"):
        patch.w4_gemm(x[0], None)


# ---------------------------------------------------------------------------- the reference itself
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [2, 6, 16])
def test_reference_rotation_keeps_lengths_and_turns_back(layout, rot):
    g = torch.Generator().manual_seed(rot)
    x = torch.randn(5, 3, 16, generator=g, dtype=torch.float64)
    pos = torch.tensor([0, 1, 7, 100, 4095])
    tab = ref.table(4096, rot)
    y, _ = ref.rope(x, pos, tab, layout)
    assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-13)
    assert torch.equal(y[..., rot:], x[..., rot:]) and torch.equal(y[0], x[0])
    back, _ = ref.rope(y, pos, tab, layout, inverse=True)
    assert torch.allclose(back, x, rtol=0, atol=1e-13)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_reference_gradient_is_the_inverse_rotation(layout):
    """d(sum g . rope(x)) / dx by differences is the inverse rotation of g,
    times the table's magnitude."""
    gen = torch.Generator().manual_seed(1)
    x, g = (torch.randn(3, 2, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    pos, tab = torch.tensor([3, 0, 50]), ref.table(64, 6, magnitude=1.25)
    grad, _ = ref.rope(g, pos, tab, layout, inverse=True)
    for i in range(x.numel()):
        d = torch.zeros_like(x)
        d.view(-1)[i] = 1e-4
        up, down = (ref.rope(x + e * d, pos, tab, layout)[0] for e in (1, -1))
        assert abs(float(((up - down) * g).sum() / 2e-4) - float(grad.view(-1)[i])) < 1e-8


def test_reference_scalings():
    f = ref.frequencies(8)
    assert (ref.frequencies(8, scaling="linear", factor=4.0) * 4 == f).all()
    n = ref.frequencies(8, scaling="ntk", factor=4.0)
    assert n[0] == f[0] and abs(n[-1] * 4 / f[-1] - 1) < 1e-12  # the fastest pair untouched, the slowest interpolated
    b = ref.frequencies(64, scaling="by_parts", factor=8.0, original=4096.0)
    f = ref.frequencies(64)
    turns = 4096 * f / (2 * math.pi)
    assert (b[turns >= 32] == f[turns >= 32]).all() and abs(b[turns <= 1] * 8 / f[turns <= 1] - 1).max() < 1e-12
    assert ((b <= f) & (b >= f / 8 * (1 - 1e-12))).all()


def test_reference_e4m3_is_the_type():
    """Against torch's own float8_e4m3fn on every value and midpoint."""
    bits = torch.arange(0, 127, dtype=torch.uint8)
    vals = bits.view(torch.float8_e4m3fn).double()
    assert torch.equal(ref.e4m3(vals), vals) and vals.max() == 448
    mid = (vals[1:] + vals[:-1]) / 2
    for x in (mid, mid * (1 + 1e-9), mid * (1 - 1e-9), -mid):
        # through float32 a nudge of 1e-9 would be lost: compare the nudged ones by their neighbours
        got = ref.e4m3(x)
        assert ((got - x).abs() <= (x.abs() * 2.0 ** -4).clamp(min=2.0 ** -10)).all()
    assert torch.equal(ref.e4m3(mid), mid.float().to(torch.float8_e4m3fn).double())
    assert torch.isnan(ref.e4m3(torch.tensor([math.inf, math.nan], dtype=torch.float64))).all()


@pytest.mark.parametrize("amax,scale", [(0.0, 2.0 ** -126), (448.0, 1.0), (449.0, 2.0), (1.75, 2.0 ** -8), (1e-40, 2.0 ** -126),
                                        (3.4e38, 2.0 ** 120)])
def test_reference_scale(amax, scale):
    assert ref.scale_for(amax) == scale
