"""Appending to the paged 8-bit cache on the GPU against the 64-bit reference."""
import pytest
import torch

from sparse_gemm_amd import patch
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Case:
    """A cache with earlier tokens, and new ones for some sequences."""

    def __init__(self, new, past, heads, kv_heads, D, page, dtype, seed=0, spare=3, extra_rows=0, pages_wide=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.total = new, [n + p for n, p in zip(new, past)]
        need = [-(-max(t, 0) // page) for t in self.total]
        P = sum(need) + spare
        order = torch.randperm(P, generator=g).int()
        self.pt = torch.full((len(new), max(max(need), 1) + pages_wide), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            self.pt[s, :n] = order[at:at + n]
            at += n
        T = sum(new) + extra_rows
        qkv = torch.randn(T, heads + 2 * kv_heads, D, generator=g).to(dtype).cuda()
        self.q, self.k, self.v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
        self.cu = torch.tensor([0] + new).cumsum(0).int()
        self.lens = torch.tensor(self.total).int()
        self.cache = patch.kv_cache(P, kv_heads, D, page)
        for c, sc in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            bits = torch.randint(0, 256, (P, kv_heads, page, D), generator=g, dtype=torch.uint8)
            bits[(bits & 127) == 127] = 0
            c.view(torch.uint8).copy_(bits)
            sc.copy_(2.0 ** torch.randint(-12, -6, (P, kv_heads), generator=g).float())
        self.plain = {"k": ref.f64(self.cache.k.float()), "v": ref.f64(self.cache.v.float()),
                      "k_scale": ref.f64(self.cache.k_scale), "v_scale": ref.f64(self.cache.v_scale)}

    def run(self, table=None, layout="half", with_q=True, **kw):
        return patch.kv_append(self.k, self.v, self.cache, self.pt.cuda(), self.lens.cuda(), self.cu.cuda(), table=table,
                               layout=layout, q=self.q if with_q else None, **kw)

    def check(self, q_out, table=None, layout="half"):
        tab = None if table is None else ref.f64(table)
        qr, qe, lo, hi = ref.append(ref.f64(self.k), ref.f64(self.v), ref.f64(self.q), self.plain, self.pt, self.lens,
                                    self.cu, tab, layout)
        n = int(self.cu[-1])
        if q_out is not None:
            bound = torch.where(qe > 0, ref.rounded(qr, self.q.dtype, qe), torch.zeros_like(qr))
            ref.assert_within(q_out[:n], qr[:n], bound[:n], "q")
        for name in "kv":
            got = ref.f64(getattr(self.cache, name).float())
            scale = ref.f64(getattr(self.cache, name + "_scale"))
            assert torch.equal(scale, self.plain[name + "_scale"]), name + "_scale"
            nan = torch.isnan(self.plain[name])
            assert torch.equal(torch.isnan(got), nan), name + ": NaN at other places"
            ok = ((got >= torch.minimum(lo[name], hi[name])) & (got <= torch.maximum(lo[name], hi[name]))) | nan
            assert ok.all(), (name, int((~ok).sum()), torch.nonzero(~ok)[0].tolist())
            self.plain[name] = got  # for a further step: the 8-bit values as they are


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("new,past,heads,kv_heads,D,page,rot,layout", [
    ([1], [0], 1, 1, 16, 16, 16, "half"),
    ([1, 1, 1], [0, 15, 16], 8, 2, 64, 16, 64, "half"),
    ([1] * 9, [3, 63, 64, 65, 127, 0, 200, 1, 31], 32, 32, 128, 64, 128, "half"),
    ([0, 5, 0, 1, 40], [7, 12, 0, 16, 30], 6, 3, 96, 32, 48, "interleaved"),
    ([130, 1, 257], [0, 100, 127], 4, 1, 128, 128, 128, "half"),
    ([33], [17], 10, 5, 80, 16, 80, "interleaved"),
    ([70, 2], [5, 9], 2, 2, 256, 128, 256, "half"),
    ([300], [1], 3, 3, 48, 64, 6, "half"),
    ([2, 3, 1, 2], [62, 61, 63, 64], 4, 2, 80, 64, 40, "interleaved"),
])
def test_append(new, past, heads, kv_heads, D, page, rot, layout, dtype):
    c = Case(new, past, heads, kv_heads, D, page, TYPES[dtype], seed=len(new) + D)
    table = patch.rope_table(max(c.total), rot)
    c.check(c.run(table, layout), table, layout)


@pytest.mark.parametrize("new,past,heads,kv_heads,D,page,rows", [
    ([2050], [3], 2, 1, 32, 64, 0), ([4099], [30], 2, 1, 32, 16, 7), ([1900, 0, 2300, 61], [0, 9, 100, 15], 6, 2, 48, 128, 0)])
def test_many_tokens(new, past, heads, kv_heads, D, page, rows):
    """q's workgroups of two tokens, behind the others and among them."""
    c = Case(new, past, heads, kv_heads, D, page, torch.bfloat16, extra_rows=rows)
    table = patch.rope_table(max(c.total), 32)
    c.check(c.run(table), table)


def test_token_by_token_through_pages():
    """Twenty steps of one token a sequence over two page borders: scales that
    grow take the earlier tokens with them."""
    c = Case([1, 1], [10, 0], 4, 2, 64, 16, torch.bfloat16, pages_wide=3, spare=8)
    c.pt[0, :3], c.pt[1, :3] = torch.tensor([0, 1, 2]), torch.tensor([3, 4, 5])
    table = patch.rope_table(64, 64)
    for step in range(20):
        # every third token ten times as large as any before
        c.k.copy_(torch.randn(c.k.shape, generator=torch.Generator().manual_seed(step)).to(c.k.dtype)
                  * (10.0 ** (step // 3 - 3)))
        c.v.copy_(c.k * 0.5)
        c.check(c.run(table), table)
        c.lens += 1


def test_values_that_are_no_numbers():
    """Infinite and NaN values are stored as NaN and do not reach the scale;
    zeros take the least scale; a block of NaN alone likewise."""
    c = Case([20, 3], [3, 0], 2, 2, 32, 16, torch.bfloat16)
    c.k[2, 0, 5], c.k[3, 1, 0], c.v[0, 0, 0], c.v[15, 1, 31] = float("inf"), float("nan"), float("-inf"), float("nan")
    c.v[20:] = 0.0
    c.k[20:, 1] = float("nan")
    c.check(c.run(None), None)
    assert float(c.cache.v_scale[c.pt[1, 0].item()].max()) == 2.0 ** -126
    c = Case([2], [0], 2, 2, 32, 16, torch.bfloat16)
    c.k.fill_(3.3895e38)  # the largest bf16
    c.v.fill_(1e-40)
    c.check(c.run(None), None)


@pytest.mark.parametrize("tokens", ["few", "many"])
def test_bad_pages_places_and_positions_write_nothing(tokens):
    """Page numbers outside the cache, lengths behind the page table, places
    before 0 and positions outside the rotary table; rows behind the last
    sequence: none of them may write anywhere else."""
    new = [1, 2, 2, 1, 1] if tokens == "few" else [40, 20, 40, 9, 33]
    c = Case(new, [20, 30, 33, 5, 2], 4, 2, 64, 16, torch.float16, extra_rows=5)
    c.pt[0, 1] = c.cache._shape[0]  # one page behind the cache
    c.pt[1, 1:3] = -1
    c.lens[2] = 3 * new[2] // 4     # shorter than its new tokens: the first have negative places
    c.lens[3] = 16 * c.pt.shape[1] + 2  # longer than the page table holds
    table = patch.rope_table(24, 64)    # shorter than the sequences
    q_out = torch.full((c.q.shape[0], 4, 64), 5.0, dtype=torch.float16, device="cuda")
    c.run(table, q_out=q_out)
    c.check(q_out, table)
    assert (q_out[int(c.cu[-1]):] == 5.0).all()


def test_cu_new_beyond_the_tokens_is_not_followed():
    c = Case([4, 4], [0, 0], 2, 2, 32, 16, torch.bfloat16)
    before = c.cache.k.view(torch.uint8).clone()
    c.cu = torch.tensor([0, 4, 1000000], dtype=torch.int32)  # tokens 8 .. do not exist
    c.lens = torch.tensor([4, 16], dtype=torch.int32)
    c.run(None, with_q=True)
    torch.cuda.synchronize()
    p = int(c.pt[0, 0])
    rest = [i for i in range(before.shape[0]) if i != p and i != int(c.pt[1, 0])]
    assert torch.equal(c.cache.k.view(torch.uint8)[rest], before[rest])


def test_without_q_in_place_q_and_wide_page_table_rows():
    c = Case([3, 1], [14, 15], 4, 2, 64, 16, torch.bfloat16)
    table = patch.rope_table(64, 64)
    wide = torch.full((2, 9), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.pt.shape[1]] = c.pt.cuda()
    q0 = c.q.clone()
    q = patch.kv_append(c.k, c.v, c.cache, wide[:, 2:2 + c.pt.shape[1]], c.lens.cuda(), c.cu.cuda(), table=table, q=c.q,
                        q_out=c.q)
    assert q.data_ptr() == c.q.data_ptr()
    got, c.q = q.clone(), q0
    c.check(got, table)
    d = Case([3, 1], [14, 15], 4, 2, 64, 16, torch.bfloat16)
    assert d.run(table, with_q=False) is None
    d.check(None, table)


def test_same_twice_other_stream_and_graph():
    """Appending the same tokens again changes nothing; a captured append
    follows lengths that change between replays."""
    c, table = Case([1, 1, 1], [15, 16, 40], 4, 4, 64, 16, torch.bfloat16, pages_wide=1), patch.rope_table(128, 64)
    c.pt[0, 1] = c.cache._shape[0] - 1
    c.pt[1, 2] = c.cache._shape[0] - 2
    pt, lens, cu = c.pt.cuda(), c.lens.cuda(), c.cu.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q = patch.kv_append(c.k, c.v, c.cache, pt, lens, cu, table=table, q=c.q)
    torch.cuda.current_stream().wait_stream(s)
    c.check(q, table)
    first = [t.view(torch.uint8).clone() for t in (c.cache.k, c.cache.v)]
    patch.kv_append(c.k, c.v, c.cache, pt, lens, cu, table=table, q=c.q)
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(first, (c.cache.k, c.cache.v)))
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        patch.kv_append(c.k, c.v, c.cache, pt, lens, cu, table=table, q=c.q, q_out=out)
    for step in range(3):
        lens += 1
        c.lens += 1
        c.k.copy_(torch.randn(c.k.shape, generator=torch.Generator().manual_seed(step)).to(c.k.dtype) * (step + 1))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, table)


def test_no_tokens():
    c = Case([0, 0], [3, 5], 2, 2, 32, 16, torch.bfloat16)
    before = c.cache.k.view(torch.uint8).clone()
    c.run(None)
    assert torch.equal(before, c.cache.k.view(torch.uint8))
