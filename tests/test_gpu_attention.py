"""Attention over the paged 8-bit cache on the GPU against the 64-bit reference."""
import math

import pytest
import torch

from sparse_gemm_amd import patch
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


class Case:
    def __init__(self, new, total, heads, kv_heads, D, page, dtype, seed=0, q_std=1.0, extra_rows=0, pages_wide=0):
        g = torch.Generator().manual_seed(seed + D + len(new))
        need = [-(-t // page) for t in total]
        P = sum(need) + 3
        order = torch.randperm(P, generator=g).int()
        self.pt = torch.full((len(new), max(max(need), 1) + pages_wide), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            self.pt[s, :n] = order[at:at + n]
            at += n
        self.cu, self.lens = torch.tensor([0] + new).cumsum(0).int(), torch.tensor(total).int()
        self.q = (q_std * torch.randn(sum(new) + extra_rows, heads, D, generator=g)).to(TYPES[dtype]).cuda()
        self.cache = patch.kv_cache(P, kv_heads, D, page)
        for c, sc in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            x = torch.randn(P, kv_heads, page, D, generator=g) * 100
            c.copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn))
            # any finite scale, powers of two and others, three orders of magnitude apart
            sc.copy_(0.01 * torch.exp(1.5 * torch.randn(P, kv_heads, generator=g)))
        self.unseen_is_nan()

    def unseen_is_nan(self):
        """Every place that no sequence holds is NaN."""
        page = self.cache._shape[2]
        hold = torch.zeros(self.cache._shape[0], page, dtype=torch.bool)
        for s in range(len(self.lens)):
            for i in range(min(int(self.lens[s]), self.pt.shape[1] * page)):
                p = int(self.pt[s, i // page])
                if 0 <= p < hold.shape[0]:
                    hold[p, i % page] = True
        for c in (self.cache.k, self.cache.v):
            b = c.view(torch.uint8)
            b.copy_(torch.where(hold[:, None, :, None].cuda(), b, torch.full_like(b, 0x7f)))

    def want(self, scale, window):
        plain = {n: ref.f64(getattr(self.cache, n).float()) for n in ("k", "v", "k_scale", "v_scale")}
        return ref.attention(ref.f64(self.q), plain, self.pt, self.lens, self.cu, scale, window)

    def run(self, window=0, out_dtype=None, scale=None, check=True, **kw):
        lse = torch.full((self.q.shape[0], self.q.shape[1]), 9.0, device="cuda")
        out = patch.attention(self.q, self.cache, self.pt.cuda(), self.lens.cuda(), self.cu.cuda(), scale=scale,
                              window=window, out_dtype=out_dtype, lse=lse, **kw)
        if check:
            self.check(out, lse, window, scale)
        return out, lse

    def check(self, out, lse, window=0, scale=None):
        scale = self.q.shape[2] ** -0.5 if scale is None else scale
        n = int(self.cu[-1])
        want, wl, size, ds = (t[:n] for t in self.want(scale, window))
        keys = int(self.lens.max())
        ref.assert_within(out[:n], want, ref.attention_bound(want, size, ds, keys, out.dtype), "out")
        bound = ds + (2 * keys + 32) * ref.U32 + 4 * ref.U32 * wl.abs()
        ref.assert_within(lse[:n], wl, torch.where(torch.isfinite(bound), bound, torch.zeros_like(bound)), "lse")


@pytest.mark.parametrize("workspace", ["auto", None])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("new,total,heads,kv_heads,D,page,window", [
    ([1], [1], 1, 1, 16, 16, 0),
    ([1], [33], 4, 4, 128, 16, 0),
    ([1, 1, 1], [31, 32, 700], 32, 8, 128, 64, 0),
    ([1] * 5, [1, 130, 2, 64, 1000], 8, 1, 64, 128, 0),
    ([1, 1], [90, 2000], 12, 2, 128, 32, 50),
    ([0, 3, 0, 1, 17], [9, 40, 0, 1, 300], 6, 3, 96, 16, 0),
    ([5, 2], [5, 64], 40, 8, 80, 64, 0),
    ([33, 70], [33, 150], 4, 2, 128, 64, 0),
    ([40], [200], 8, 8, 256, 32, 0),
    ([64, 1, 20], [300, 301, 20], 4, 1, 64, 16, 37),
    ([129], [129], 2, 2, 112, 128, 1),
    ([100, 90], [400, 90], 16, 2, 128, 64, 64),
    ([300, 17], [1500, 700], 8, 2, 128, 64, 0),
    ([260], [2100], 2, 1, 64, 16, 300),
    ([40, 1, 150], [1200, 1300, 400], 4, 2, 112, 32, 0),
])
def test_attention(new, total, heads, kv_heads, D, page, window, dtype, out, workspace):
    Case(new, total, heads, kv_heads, D, page, dtype).run(window, TYPES[out], workspace=workspace)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,total,heads,kv_heads,D,window", [
    ([1, 1], [700, 40], 4, 4, 128, 0), ([5, 1], [90, 300], 8, 2, 80, 0), ([9], [1000], 8, 2, 64, 100),
    ([3], [200], 2, 1, 256, 0), ([90, 70], [400, 70], 4, 2, 128, 0), ([130], [500], 2, 1, 48, 200)])
def test_float32_outputs_keep_22_bits(new, total, heads, kv_heads, D, window, dtype):
    """Probabilities are 2^6 at the largest and held as two fp16 values: 2^-22
    of each, and 2^-25 (the second's least step) of each of the n keys' |v| <=
    448 v_scale, over a sum of 2^6 or more."""
    c = Case(new, total, heads, kv_heads, D, 32, dtype)
    c.cache.v_scale.fill_(2.0 ** -6)
    out, _ = c.run(window, torch.float32)
    want, _, size, ds = c.want(D ** -0.5, window)
    n = max(total)
    err = size * (2.0 ** -21 + 2 * ds[..., None] + (2 * n + 32) * ref.U32) + n * 2.0 ** -31 * 448 * 2.0 ** -6
    ref.assert_within(out, want, ref.rounded(want, torch.float32, err), "out")


def test_long_cache():
    Case([1, 1], [20011, 7], 2, 1, 128, 64, "f16").run()


def test_sharp_scores_and_scale():
    """Scores of hundreds, and of exactly one key; a scale of 0 is the mean."""
    Case([1, 4], [500, 200], 4, 2, 64, 32, "bf16", q_std=40.0).run(scale=1.0)
    Case([1, 4], [500, 200], 4, 2, 64, 32, "bf16").run(scale=0.0)
    Case([3], [70], 4, 2, 64, 32, "f16").run(scale=-0.2)


def test_scales_far_apart():
    """Blocks whose scales differ by 2^60, the large ones first, last, or of
    one key: no overflow, and the large values win."""
    for where in (0, 1, -1):
        c = Case([1], [100], 2, 1, 64, 16, "bf16")
        c.cache.v_scale.fill_(2.0 ** -30)
        c.cache.v_scale[c.pt[0, where].item()] = 2.0 ** 30
        c.run()
    c = Case([1], [100], 2, 1, 64, 16, "bf16")
    c.cache.v_scale.fill_(0.0)
    c.cache.k_scale.fill_(2.0 ** -126)
    c.run()


def test_tokens_that_see_nothing_and_rows_behind_the_last():
    c = Case([6, 4], [40, 9], 4, 2, 64, 16, "bf16", extra_rows=5)
    c.lens[0] = 4  # six new tokens in a sequence of four: two see nothing
    out = torch.full(c.q.shape, 3.0, dtype=c.q.dtype, device="cuda")
    out, lse = c.run(out=out)
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
    assert (out[10:] == 3.0).all() and (lse[10:] == 9.0).all()


def test_bad_pages_and_lengths_are_nan_for_who_sees_them():
    c = Case([3, 2, 1], [70, 50, 33], 4, 2, 64, 16, "bf16")
    c.pt[0, 4] = c.cache._shape[0]  # places 64 .. of the first: seen by all of its tokens
    c.pt[1, 0] = -5                 # not seen within the window
    c.lens[2] = 16 * c.pt.shape[1] + 1
    for window in (0, 20):
        out, _ = c.run(window)
        assert torch.isnan(out[0]).all() and torch.isnan(out[5]).all()
        assert torch.isnan(out[3]).all() == (window == 0)


@pytest.mark.parametrize("new,total", [([20], [45]), ([20, 90], [45, 300])])
@pytest.mark.parametrize("window", [0, 9])
def test_nan_reaches_only_the_tokens_that_see_it(window, new, total):
    """NaN keys and values among the new tokens: earlier tokens and those whose
    window has passed them stay clean."""
    c = Case(new, total, 4, 2, 64, 16, "bf16")
    for name, place, h, d in (("v", 35, 0, 7), ("v", 40, 1, 63), ("k", 38, 1, 3), ("v", 31, 0, 0)):
        getattr(c.cache, name).view(torch.uint8)[c.pt[0, place // 16].item(), h, place % 16, d] = 0xff
    out, _ = c.run(window)
    assert not torch.isnan(out[:5]).any() and torch.isnan(out[-1 if len(new) == 1 else 12]).any()


def test_nan_and_infinite_queries_stay_in_their_row():
    c = Case([4], [50], 4, 2, 64, 16, "bf16")
    c.q[1, 2, 5], c.q[2, 0, 0] = float("nan"), float("nan")
    out, _ = c.run()
    assert torch.isnan(out[1, 2]).all() and not torch.isnan(out[1, 1]).any()


@pytest.mark.parametrize("shift", [0, 1])
def test_strides_and_alignment(shift):
    c = Case([1, 30], [70, 200], 4, 2, 64, 32, "bf16")
    want, lse = c.run()
    q = torch.zeros(31, 9, 70, dtype=torch.bfloat16, device="cuda")[:, 2:6, shift:shift + 64]
    q.copy_(c.q)
    pt = torch.full((2, 20), -9, dtype=torch.int32, device="cuda")[:, 3:3 + c.pt.shape[1]]
    pt.copy_(c.pt)
    out = torch.full((4, 31, 66), 5.0, dtype=torch.bfloat16, device="cuda")
    view = out.transpose(0, 1)[:, :, shift:shift + 64]
    patch.attention(q, c.cache, pt, c.lens.cuda(), c.cu.cuda(), out=view)
    assert torch.equal(view, want)
    assert (out[:, :, 64 + shift:] == 5.0).all() and (out[:, :, :shift] == 5.0).all()


def test_results_do_not_change_between_runs_or_with_the_workspace_contents():
    c = Case([1, 1, 1], [3000, 20, 700], 8, 2, 128, 64, "bf16")
    args = (c.q, c.cache, c.pt.cuda(), c.lens.cuda(), c.cu.cuda())
    want = patch.attention(*args)
    n = patch.attention_workspace_bytes(3, 3, 8, 2, 128)
    for fill in (0, 255, 77):
        ws = torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            assert torch.equal(patch.attention(*args, workspace=ws), want), fill


def test_graph_follows_lengths():
    """A captured call whose lengths, pages and queries change between
    replays, other work in between, and two graphs with a workspace each."""
    c = Case([1, 1, 1], [3000, 1500, 700], 8, 2, 64, 32, "bf16")
    full = c.lens.clone()
    lens, pt, cu = c.lens.cuda(), c.pt.cuda(), c.cu.cuda()
    n = max(16, patch.attention_workspace_bytes(3, 3, 8, 2, 64))
    outs, graphs = [], []
    spaces = [torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for ws in spaces:
        out = torch.empty_like(c.q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            patch.attention(c.q, c.cache, pt, lens, cu, out=out, workspace=ws)
        outs.append(out)
        graphs.append(g)
    for step, by in enumerate((0, 1, 650, 33, 0)):
        lens.copy_(full - by)
        c.q.copy_(torch.randn(c.q.shape, generator=torch.Generator().manual_seed(step)))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        eager = patch.attention(c.q, c.cache, pt, lens, cu)
        for out in outs:
            assert torch.equal(out, eager), step
        c.lens = full - by
        torch.cuda.synchronize()
    lse = torch.empty(3, 8, device="cuda")
    out = patch.attention(c.q, c.cache, pt, lens, cu, lse=lse)
    c.check(out, lse)


def test_graph_of_chunks_follows_lengths():
    c = Case([150, 90], [700, 400], 4, 2, 128, 64, "bf16")
    full, lens, pt, cu = c.lens.clone(), c.lens.cuda(), c.pt.cuda(), c.cu.cuda()
    out = torch.empty_like(c.q)
    ws = torch.randint(0, 256, (patch.attention_workspace_bytes(240, 2, 4, 2, 128),), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        patch.attention(c.q, c.cache, pt, lens, cu, out=out, workspace=ws)
    for by in (0, 130, 200, 0):
        lens.copy_(full - by)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, patch.attention(c.q, c.cache, pt, lens, cu)), by


@pytest.mark.parametrize("new,total", [([1, 1, 3], [9000, 40, 700]), ([130, 260], [2000, 260]), ([1, 0], [1, 5])])
def test_in_place(new, total):
    c = Case(new, total, 8, 2, 128, 64, "bf16")
    want = c.run(check=False)[0]
    for workspace in ("auto", None):
        q = c.q.clone()
        out = patch.attention(q, c.cache, c.pt.cuda(), c.lens.cuda(), c.cu.cuda(), out=q, workspace=workspace)
        assert out is q and (workspace is None or torch.equal(q, want))
    n = int(c.cu[-1])
    wantd, _, size, ds = (t[:n] for t in c.want(128 ** -0.5, 0))
    ref.assert_within(q[:n], wantd, ref.attention_bound(wantd, size, ds, int(c.lens.max()), q.dtype), "in place")


def test_offsets_beyond_32_bits():
    """Pages whose bytes lie behind the first 4 GiB of a cache, appended to and
    attended to by one token and by a chunk."""
    pages, hk, page, D = 70000, 4, 128, 128
    cache = patch.kv_cache(pages, hk, D, page)
    assert cache.k.numel() > 1 << 32
    g = torch.Generator().manual_seed(0)
    table = patch.rope_table(512, D)
    for n in (1, 140):
        total, start = 300, 300 - n
        pt = torch.tensor([[pages - 1, 0, pages - 7]], dtype=torch.int32, device="cuda")
        small = patch.kv_cache(3, hk, D, page)
        spt = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
        outs = []
        x = torch.randn(total, 3 * hk, D, generator=g).bfloat16().cuda()
        for c, t in ((cache, pt), (small, spt)):
            for at, m in ((0, start), (start, n)):
                lens = torch.tensor([at + m], dtype=torch.int32, device="cuda")
                cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
                y = x[at:at + m]
                q = patch.kv_append(y[:, :hk], y[:, hk:2 * hk], c, t, lens, cu, table=table, q=y[:, 2 * hk:])
            outs.append(patch.attention(q, c, t, lens, cu))
        assert torch.equal(outs[0], outs[1]) and torch.equal(cache.k.view(torch.uint8)[pages - 1], small.k.view(torch.uint8)[0])


def test_two_streams_at_once():
    a, b = Case([1, 1], [2500, 900], 8, 2, 128, 64, "bf16"), Case([1], [3100], 8, 2, 128, 64, "bf16", seed=5)
    want = [c.run(check=False)[0] for c in (a, b)]
    args = [(c.q, c.cache, c.pt.cuda(), c.lens.cuda(), c.cu.cuda()) for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(patch.attention(*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_many_sequences():
    """More sequences than a wave, most of them short, some empty."""
    new = [1 if i % 7 else 0 for i in range(300)]
    total = [(i * 37) % 90 + 1 for i in range(300)]
    Case(new, total, 2, 1, 32, 16, "bf16").run()
    new = [(i * 29) % 90 for i in range(70)]  # and chunks of them
    Case(new, [n + (i * 53) % 200 for i, n in enumerate(new)], 2, 1, 64, 16, "f16").run()


def test_no_tokens():
    c = Case([0, 0], [5, 9], 2, 2, 32, 16, "bf16")
    assert c.run(check=False)[0].shape == (0, 2, 32)
