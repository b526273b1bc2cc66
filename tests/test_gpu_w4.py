"""The linear layer with 4-bit weights on the GPU against the 64-bit reference."""
import pytest
import torch

from sparse_gemm_amd import patch
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _weight(N, K, group, zero, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + N + K)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scale = (0.002 + 0.01 * torch.rand(N, K // group, generator=g)).to(dtype)
    z = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zero else None
    return q.cuda(), scale.cuda(), None if z is None else z.cuda()


def _check(x, q, scale, z, group, y, what=""):
    w, size = ref.w4_weight(q, scale, z, group)
    xd = ref.f64(x)
    want = xd @ w.T
    ref.assert_within(y, want, ref.w4_bound(xd, want, size, group, y.dtype), what)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (16, 128, 128), (7, 96, 32), (40, 160, 32), (129, 192, 64),
                                       (64, 64, 64), (250, 1152, 128), (34, 4096, 128), (96, 2080, 32)])
def test_gemm(N, K, group, zero, dtype):
    q, scale, z = _weight(N, K, group, zero, TYPES[dtype])
    w = patch.w4_pack(q, scale, z, group)
    for M in (1, 2, 16, 17, 33, 70):
        x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(TYPES[dtype]).cuda()
        for od in (None, torch.float32):
            _check(x, q, scale, z, group, patch.w4_gemm(x, w, out_dtype=od), f"M={M} {od}")


@pytest.mark.parametrize("N,K,group,zero", [(4100, 256, 64, True), (8300, 288, 32, False), (13001, 128, 128, True),
                                            (20000, 160, 32, True)])
def test_many_bands(N, K, group, zero):
    """Two to four bands a workgroup, and more than one round of the GPU."""
    q, scale, z = _weight(N, K, group, zero, torch.bfloat16)
    w = patch.w4_pack(q, scale, z, group)
    for M in (1, 7, 20):
        x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).bfloat16().cuda()
        _check(x, q, scale, z, group, patch.w4_gemm(x, w), f"M={M}")


@pytest.mark.parametrize("N,K,group,zero,M", [(4100, 256, 64, False, 40), (8300, 160, 32, True, 20), (4100, 384, 128, True, 90),
                                              (2000, 256, 32, True, 530), (1000, 224, 32, False, 1101)])
def test_many_tokens(N, K, group, zero, M):
    """Two to four bands a workgroup for blocks of 32 tokens, and many rounds."""
    q, scale, z = _weight(N, K, group, zero, torch.float16)
    w = patch.w4_pack(q, scale, z, group)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.float16).cuda()
    for od in (None, torch.float32):
        _check(x, q, scale, z, group, patch.w4_gemm(x, w, out_dtype=od), f"{od}")


def test_more_tokens_than_a_launch_has():
    q, scale, z = _weight(20, 32, 32, True, torch.bfloat16)
    w = patch.w4_pack(q, scale, z, 32)
    x = torch.randn(64, 32, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want = patch.w4_gemm(x, w)
    y = patch.w4_gemm(x.repeat(32768, 1), w)  # 2^21 rows
    assert torch.equal(y.view(32768, 64, 20), want.expand(32768, 64, 20))


def test_packed_bytes_are_as_stated():
    """The layout of patch_w4_pack, byte by byte, and its padding."""
    N, K, group = 20, 160, 32
    q, scale, z = _weight(N, K, group, True, torch.float16)
    p = patch.w4_pack(q, scale, z, group).packed.cpu()
    qc = q.cpu()
    val = torch.zeros(32, 256, dtype=torch.uint8)
    val[:N, :K] = torch.stack([qc & 15, qc >> 4], dim=-1).reshape(N, K)
    words = p[:2 * 2 * 1024].view(torch.int32).view(2, 2, 64, 4)
    for band in range(2):
        for block in range(2):
            for l in (0, 3, 16, 17, 33, 63):
                for j in range(4):
                    word = int(words[band, block, l, j]) & 0xffffffff
                    for i in range(4):
                        k = block * 128 + 32 * j + 8 * (l // 16) + 2 * i
                        row = band * 16 + l % 16
                        assert (word >> (4 * i)) & 15 == int(val[row, k]) and (word >> (16 + 4 * i)) & 15 == int(val[row, k + 1])
    # band, block, quad of rows, group, row of the quad
    s = torch.zeros(32, 8, dtype=torch.float16)
    s[:N, :5] = scale.cpu()
    order = lambda t: t.view(2, 4, 4, 2, 4).permute(0, 3, 1, 4, 2)  # noqa: E731
    at = 4096
    assert torch.equal(p[at:at + 32 * 8 * 2].view(torch.float16).view(2, 2, 4, 4, 4), order(s))
    zz = torch.zeros(32, 8, dtype=torch.uint8)
    zz[:N, :5] = z.cpu()
    assert torch.equal(p[at + 512:].view(2, 2, 4, 4, 4), order(zz))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize(group, zero, dtype):
    """Bit for bit the stated rounding; within half a step (and the scale's own
    rounding) of the weight; a group of zeros, of one sign, of one value."""
    g = torch.Generator().manual_seed(group)
    w = (0.02 * torch.randn(33, 3 * group, generator=g)).to(TYPES[dtype])
    w[0, :group] = 0
    w[1] = w[1].abs()
    w[2, group:2 * group] = -0.5
    q, s, z = patch.w4_quantize(w.cuda(), group, zero)
    qr, sr, zr = ref.w4_quantize(w, group, zero, TYPES[dtype])
    assert torch.equal(s.cpu(), sr) and torch.equal(q.cpu(), qr) and (not zero or torch.equal(z.cpu(), zr))
    back, _ = ref.w4_weight(q, s, z, group)
    step = ref.f64(s).repeat_interleave(group, 1)
    # half a step for the rounding of w / s, half for the zero's, 7 or 15 steps of the scale's own rounding
    slack = (1.0 if zero else 0.5) + 16 * ref.HALF_EPS[TYPES[dtype]]
    assert ((back - w.double()).abs() <= slack * step).all()


def test_quantized_weight_multiplies():
    w = (0.02 * torch.randn(96, 512, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).cuda()
    x = torch.randn(3, 512, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    for zero in (False, True):
        q, s, z = patch.w4_quantize(w, 64, zero)
        _check(x, q, s, z, 64, patch.w4_gemm(x, patch.w4_pack(q, s, z, 64)))


def test_activations_far_from_zero():
    """A mean of 30 in X: what is taken off for the offset of the weights is
    large, and the fp32 bound still holds."""
    q, scale, z = _weight(64, 512, 128, True, torch.float16)
    x = (30 + torch.randn(4, 512, generator=torch.Generator().manual_seed(2))).half().cuda()
    _check(x, q, scale, z, 128, patch.w4_gemm(x, patch.w4_pack(q, scale, z, 128), out_dtype=torch.float32))


def test_nan_rows_stay_rows_and_out_is_used():
    q, scale, z = _weight(48, 256, 64, False, torch.bfloat16)
    w = patch.w4_pack(q, scale, z, 64)
    x = torch.randn(20, 256, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    want = patch.w4_gemm(x, w)
    x[3, 5], x[19, 255] = float("nan"), float("inf")
    out = torch.empty(20, 48, dtype=torch.bfloat16, device="cuda")
    y = patch.w4_gemm(x, w, out=out)
    assert y is out and torch.isnan(y[3]).all() and torch.isnan(y[19]).all()
    keep = [i for i in range(20) if i not in (3, 19)]
    assert torch.equal(y[keep], want[keep])


def test_stream_graph_and_no_tokens():
    q, scale, z = _weight(160, 384, 128, True, torch.bfloat16)
    w = patch.w4_pack(q, scale, z, 128)
    x = torch.randn(5, 384, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    want = patch.w4_gemm(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = patch.w4_gemm(x, w)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        patch.w4_gemm(x, w, out=out)
    for k in range(3):
        x.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, patch.w4_gemm(x, w)), k
    assert patch.w4_gemm(x[:0], w).shape == (0, 160)
