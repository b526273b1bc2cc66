"""Rotary positions on the GPU against the 64-bit reference."""
import pytest
import torch

from sparse_gemm_amd import patch
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _x(T, H, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, D, generator=g).to(dtype).cuda()


def _check(x, pos, tab, layout, inverse, got, what=""):
    want, err = ref.rope(ref.f64(x), pos.cpu(), ref.f64(tab), layout, inverse)
    ref.assert_within(got, want, torch.where(err > 0, ref.rounded(want, x.dtype, err), torch.zeros_like(want)), what)


@pytest.mark.parametrize("scaling", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                     dict(scaling="by_parts", factor=8.0, original=4096.0, magnitude=1.2),
                                     dict(scaling="by_parts", factor=4.0, original=64.0, low=1.0, high=4.0, base=5e5)])
@pytest.mark.parametrize("rot,n", [(2, 3), (4, 1), (64, 300), (128, 131072), (40, 5000)])
def test_table(rot, n, scaling):
    if scaling.get("scaling") == "ntk" and rot < 4:
        with pytest.raises(patch.PatchError, match="SHAPE"):
            patch.rope_table(n, rot, **scaling)
        return
    tab = patch.rope_table(n, rot, **scaling)
    kw = dict(scaling)
    want = ref.table(n, rot, magnitude=kw.pop("magnitude", 1.0), **kw)
    # the angle: a few 64-bit roundings of up to n radians; the result: one of fp32
    ref.assert_within(tab, want, ref.U32 * want.abs() + n * 2.0 ** -49 + 2.0 ** -150)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 2, 2), (1, 64, 128, 128), (7, 3, 80, 40), (33, 5, 64, 6), (130, 8, 128, 64),
                                       (5, 2, 256, 256), (1000, 9, 96, 96), (3, 1, 18, 10), (2, 300, 16, 16)])
def test_rope(T, H, D, rot, layout, inverse, dtype):
    x = _x(T, H, D, TYPES[dtype], T)
    tab = patch.rope_table(4096, rot)
    pos = torch.randint(0, 4096, (T,), generator=torch.Generator().manual_seed(T), dtype=torch.int32).cuda()
    _check(x, pos, tab, layout, inverse, patch.rope(x, pos, tab, layout=layout, inverse=inverse))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_strides_alignment_and_in_place(dtype, layout, shift):
    """Heads inside a wider row, at an odd address, tokens in reverse strides
    of others; in place writes only the rotated elements."""
    T, H, D, rot = 19, 4, 48, 32
    base = _x(T, 3 * H, D + 8, TYPES[dtype], 3)
    x = base[:, 1:1 + H, shift:shift + D]
    tab, pos = patch.rope_table(64, rot), torch.arange(T, dtype=torch.int32, device="cuda")
    y = patch.rope(x, pos, tab, layout=layout)
    _check(x, pos, tab, layout, False, y)
    before = base.clone()
    out = torch.full((H, T, D), 7.0, dtype=x.dtype, device="cuda").transpose(0, 1)  # head-major
    assert patch.rope(x, pos, tab, layout=layout, out=out) is out
    assert torch.equal(out, y) and torch.equal(base, before)
    patch.rope(x, pos, tab, layout=layout, out=x)
    assert torch.equal(x, y)
    before[:, 1:1 + H, shift:shift + D] = y
    assert torch.equal(base, before)


def test_positions_outside_the_table_are_nan_in_the_rotated_part():
    x, tab = _x(4, 2, 32, torch.bfloat16), patch.rope_table(10, 16)
    pos = torch.tensor([-1, 9, 10, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    y = patch.rope(x, pos, tab)
    _check(x, pos, tab, "half", False, y)
    assert torch.equal(y[..., 16:], x[..., 16:]) and torch.isnan(y[0, :, :16]).all()


def test_infinities_and_nan_stay_in_their_pair():
    x, tab = _x(3, 2, 16, torch.float16), patch.rope_table(10, 16)
    x[0, 0, 1], x[1, 1, 3] = float("inf"), float("nan")
    pos = torch.tensor([2, 3, 4], dtype=torch.int32, device="cuda")
    _check(x, pos, tab, "half", False, patch.rope(x, pos, tab))


def test_gradient_turns_back():
    """inverse=True on the gradient, against differences of the forward
    rotation in fp32 along random directions."""
    T, H, D, rot = 9, 3, 64, 48
    x, g, d = (_x(T, H, D, torch.float32, s) for s in (1, 2, 3))
    tab = patch.rope_table(2048, rot, scaling="by_parts", factor=4.0, original=512.0, magnitude=1.1)
    pos = torch.randint(0, 2048, (T,), dtype=torch.int32).cuda()
    grad = patch.rope(g, pos, tab, inverse=True)
    want, err = ref.rope(ref.f64(g), pos.cpu(), ref.f64(tab), "half", True)
    ref.assert_within(grad, want, ref.rounded(want, torch.float32, err))
    # the map is linear: (rope(x + d) - rope(x - d)) / 2 = rope(d), and <g, rope(d)> = <grad, d>
    up, down = patch.rope(x + d, pos, tab), patch.rope(x - d, pos, tab)
    lhs = float((ref.f64(g) * (ref.f64(up) - ref.f64(down)) / 2).sum())
    rhs = float((ref.f64(grad) * ref.f64(d)).sum())
    terms = float((ref.f64(g).abs() * (ref.f64(x).abs() + ref.f64(d).abs()) * 2 * 1.1).sum())
    assert abs(lhs - rhs) <= 16 * ref.U32 * terms


def test_streams_graphs_and_no_tokens():
    T, H, D = 12, 4, 64
    tab = patch.rope_table(256, D)
    x, pos = _x(T, H, D, torch.bfloat16), torch.arange(T, dtype=torch.int32, device="cuda")
    want = patch.rope(x, pos, tab)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = patch.rope(x, pos, tab)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        patch.rope(x, pos, tab, out=out)
    for k in range(3):  # positions change between replays
        pos.copy_(torch.arange(T, dtype=torch.int32) * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, patch.rope(x, pos, tab)), k
    assert patch.rope(x[:0], pos[:0], tab).shape == (0, H, D)
