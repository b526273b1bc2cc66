"""The decoder-layer operators as a program uses them together: tile-sparse
q/k/v projections in one launch, keys and values appended to the paged 8-bit
cache with the rotation on the way, attention over it, and an output projection
with 4-bit weights -- a prompt, then tokens one at a time, then a captured step
-- against the same chain in 64 bits."""
import numpy as np
import pytest
import torch

from sparse_gemm_amd import inputs, patch
from tests import layer_ref as ref
from tests.gpu_util import dev_bits, dev_u8

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, PAGE, GROUP = 256, 4, 2, 64, 16, 64


class Layer:
    def __init__(self):
        sizes = (HEADS * DIM, KV * DIM, KV * DIM)
        probs = [inputs.make_custom("bf16", n, HIDDEN, 50 + i, "bernoulli", 0.5, "top2") for i, n in enumerate(sizes)]
        self.qkv = patch.pack_concat([dev_bits(p.w, "bf16") for p in probs], [p.tile_map for p in probs],
                                     [dev_u8(p.mask) for p in probs])
        self.wq = self._weights(probs)
        g = torch.Generator().manual_seed(3)
        wo = (0.05 * torch.randn(HIDDEN, HEADS * DIM, generator=g)).to(torch.bfloat16).cuda()
        q, s, z = patch.w4_quantize(wo, GROUP, zero=True)
        self.out = patch.w4_pack(q, s, z, GROUP)
        self.out64 = ref.w4_weight(q, s, z, GROUP)[0]
        self.table = patch.rope_table(128, DIM)
        self.cache = patch.kv_cache(16, KV, DIM, PAGE)

    @staticmethod
    def _weights(probs):
        ws = []
        for p in probs:
            sparse = np.repeat(np.repeat(p.tile_map != 0, 128, axis=0), 128, axis=1)
            keep = np.where(sparse, p.mask != 0, True)
            ws.append(inputs.bits_to_f32(p.w, "bf16").astype(np.float64) * keep)
        return torch.from_numpy(np.concatenate(ws))

    def step(self, x, pt, lens, cu):
        y = patch.gemm(x, self.qkv).view(x.shape[0], HEADS + 2 * KV, DIM)
        q = patch.kv_append(y[:, HEADS:HEADS + KV], y[:, HEADS + KV:], self.cache, pt, lens, cu, table=self.table,
                            q=y[:, :HEADS])
        o = patch.attention(q, self.cache, pt, lens, cu)
        return patch.w4_gemm(o.view(x.shape[0], -1), self.out, out_dtype=torch.float32)


def _chain64(layer, xs, total):
    """The newest tokens' outputs for one sequence whose inputs so far are xs,
    every value in 64 bits, nothing rounded to 8."""
    x = torch.cat([ref.f64(t) for t in xs])
    y = (x @ layer.wq.T).view(len(x), HEADS + 2 * KV, DIM)
    pos, tab = torch.arange(len(x)), ref.table(128, DIM)
    q, k, v = (y[:, :HEADS], y[:, HEADS:HEADS + KV], y[:, HEADS + KV:])
    q, k = ref.rope(q, pos, tab, "half")[0], ref.rope(k, pos, tab, "half")[0]
    rep = HEADS // KV
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    a = torch.einsum("thd,shd->hts", q, k) * DIM ** -0.5
    a = a.masked_fill(torch.arange(len(x))[None, :] > torch.arange(len(x))[:, None], -float("inf"))
    o = torch.einsum("hts,shd->thd", torch.softmax(a, -1), v).reshape(len(x), -1)
    return (o @ layer.out64.T)[-total:]


def test_a_prompt_then_tokens_then_a_captured_token():
    layer = Layer()
    g = torch.Generator().manual_seed(9)
    draw = lambda n: (0.3 * torch.randn(n, HIDDEN, generator=g)).to(torch.bfloat16).cuda()  # noqa: E731
    pt = torch.tensor([[3, 7, 1, 9], [2, 12, 5, 0]], dtype=torch.int32, device="cuda")
    seen = [[], []]

    def feed(news):
        parts = [draw(n) for n in news]
        for s, p in enumerate(parts):
            seen[s].append(p)
        return torch.cat(parts)

    def lens_of():
        return torch.tensor([sum(len(t) for t in s) for s in seen], dtype=torch.int32, device="cuda")

    def check(y, news, what):
        at = 0
        for s, n in enumerate(news):
            if n:
                want = _chain64(layer, seen[s], n)
                err = (ref.f64(y[at:at + n]) - want).norm() / want.norm()
                # q, k and o are rounded to bf16 once each (2^-9 rms about), k and v to e4m3 (a relative error
                # uniform up to 2^-4: 0.6 * 2^-4 rms of each, and the softmax averages over keys): their sum is
                # below 2 * 0.6 * 2^-4
                assert err <= 1.2 * 2.0 ** -4, (what, s, float(err))
            at += n

    news = [37, 20]
    cu = torch.tensor([0, 37, 57], dtype=torch.int32, device="cuda")
    check(layer.step(feed(news), pt, lens_of(), cu), news, "prompt")
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for k in range(5):
        check(layer.step(feed([1, 1]), pt, lens_of(), one), [1, 1], k)

    # the same step captured: inputs, lengths and cache change between replays
    x, lens = draw(2), lens_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, pt, lens, one)  # the current last places again: the real tokens follow below
    torch.cuda.current_stream().wait_stream(side)
    # put back what the warm-up wrote over
    last = torch.cat([s[-1][-1:] for s in seen])
    layer.step(last, pt, lens, one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.step(x, pt, lens, one)
    for k in range(4):
        x.copy_(feed([1, 1]))
        lens.copy_(lens_of())
        graph.replay()
        torch.cuda.synchronize()
        check(y, [1, 1], f"replay {k}")
        assert torch.equal(y, layer.step(x, pt, lens, one))  # the same places, the same values


def test_mixed_batch_of_a_prompt_and_single_tokens():
    """One sequence's prompt beside others' single tokens gives each the values
    it gets alone (but for the order of fp32 sums)."""
    layer, alone = Layer(), Layer()
    g = torch.Generator().manual_seed(4)
    draw = lambda n: (0.3 * torch.randn(n, HIDDEN, generator=g)).to(torch.bfloat16).cuda()  # noqa: E731
    pt = torch.tensor([[0, 1, 2], [3, 4, 5], [6, 7, 8]], dtype=torch.int32, device="cuda")
    first, news = [9, 30, 0], [1, 1, 33]
    x0, x1 = draw(sum(first)), draw(sum(news))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for lay in (layer, alone):
        lay.step(x0, pt, i32(first), i32([0, 9, 39, 39]))
    lens = [a + b for a, b in zip(first, news)]
    y = layer.step(x1, pt, i32(lens), i32([0, 1, 2, 35]))
    at = 0
    for s, n in enumerate(news):
        z = alone.step(x1[at:at + n], pt[s:s + 1], i32([lens[s]]), i32([0, n]))
        d = (y[at:at + n] - z).double()
        # o is rounded to bf16 after sums in another order, q the same
        assert d.norm() <= 2.0 ** -7 * z.double().norm(), s
        at += n
