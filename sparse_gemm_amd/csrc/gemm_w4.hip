// gemm_w4.hip -- linear layer with 4-bit weights and group scales, for few
// tokens: Y = X W^T, W = (q - z) s per group of columns.
//
// Decode reads every weight once, so the product is bound by the N K / 2
// bytes of the weights (plus scales); the matrix cores do the arithmetic, 16
// columns of which only the M tokens count.  W is the A operand of
// v_mfma_f32_16x16x32 (16 rows of W), X the B operand (16 tokens).
//
//   * Weights become 16-bit values by OR alone: 16 + q has q in the top four
//     fraction bits of 16.0 (fp16 0x4c00 | q << 6, bf16 0x4180 | q << 3), so a
//     shift and a v_and_or_b32 make two operand elements.
//   * The 16 + z too much is taken off per group: sum x (16 + q) - (16 + z) sum
//     x, the second sum by the same instruction with an A operand of ones --
//     both exact products added in fp32 -- and the difference is multiplied by
//     the group's scale in fp32.  16 is the smallest such offset, so the
//     cancellation costs three bits of an fp32 sum at most.
//   * A band's weights lie in lane order (patch_w4_pack), 1 KB for 128 columns:
//     one 16-byte load a lane feeds four matrix instructions.
//   * A workgroup has one to four bands of 16 rows; its waves take the 128-column
//     blocks in turn, the next block's bytes on their way while one is used, and
//     join their sums through LDS in a fixed order.
//
// GPU time: 4096 x 4096, one token, 8.7 MB in 5.1 us; 11008 x 4096 in groups of
// 64 with zeros, 16 tokens, 25 MB in 11.5 us (2.2 TB/s); 13824 x 5120 in groups
// of 32, 5 tokens, 40 MB in 14.2 us (2.8 TB/s).  A launch alone takes about 3
// us of each; behind it the last workgroups' waits and joins.
#include <algorithm>

#include "device_common.h"
#include "layer_common.h"

namespace patch {
namespace {

constexpr int kMaxWaves = 8;

// The eight operand elements 16 + q of a packed word.
template <bool BF16>
__device__ __forceinline__ u32x4 widen4(uint32_t w) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (BF16) {
      const uint32_t b = i == 0 ? w << 3 : w >> (4 * i - 3);
      r[i] = (b & 0x00780078u) | 0x41804180u;
    } else {
      const uint32_t b = i < 2 ? w << (6 - 4 * i) : w >> (4 * i - 6);
      r[i] = (b & 0x03c003c0u) | 0x4c004c00u;
    }
  }
  return r;
}

struct W4Args {
  const uint8_t* w;      // bands of blocks
  const uint8_t* scale;  // [band][block][4 quads of rows][group][4 rows] 16-bit
  const uint8_t* zero;   // likewise, bytes
  const void* X;
  void* Y;
  int64_t M, N, K;
  int bands, blocks;  // of 16 rows, of 128 columns
  int group;
};

// The bytes of one 128-column block of RB bands and MT blocks of 16 tokens.
template <int MT, int RB, int G, bool ZERO>
struct Block {
  static constexpr int kGroups = 128 / G;  // groups of a block
  u32x4 w[RB];
  Vec<uint32_t, 2 * kGroups> s[RB];  // four rows' scales, group by group
  Vec<uint32_t, kGroups> z[RB];
  u32x4 x[MT][4];
};
template <int MT, int RB, int G, bool ZERO>
__device__ __forceinline__ Block<MT, RB, G, ZERO> load_block(const W4Args& a, int64_t band, const uint16_t* const (&xp)[MT],
                                                             int b) {
  using B = Block<MT, RB, G, ZERO>;
  const int lane = (int)threadIdx.x & 63, g = lane >> 4;
  B r;
#pragma unroll
  for (int i = 0; i < RB; i++) {
    const int64_t at = min(band + i, (int64_t)a.bands - 1) * a.blocks + b;  // a band behind the last: not stored
    r.w[i] = ld16(a.w + at * 1024 + lane * 16);
    r.s[i] = *reinterpret_cast<const Vec<uint32_t, 2 * B::kGroups>*>(a.scale + (at * 4 + g) * (8 * B::kGroups));
    if constexpr (ZERO)
      r.z[i] = *reinterpret_cast<const Vec<uint32_t, B::kGroups>*>(a.zero + (at * 4 + g) * (4 * B::kGroups));
  }
#pragma unroll
  for (int t = 0; t < MT; t++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t k = (int64_t)b * 128 + 32 * j + 8 * g;
      r.x[t][j] = ld16_pred(xp[t] + k, k < a.K);  // columns behind K are zeros in X too
    }
  return r;
}

template <bool BF16, int MT, int RB, int G, bool ZERO>
__device__ __forceinline__ void multiply(const Block<MT, RB, G, ZERO>& b, f32x4 (&y)[RB][MT]) {
  constexpr int kGroups = 128 / G, kJ = G / 32;  // instructions of a group
  const uint32_t one2 = BF16 ? 0x3f803f80u : 0x3c003c00u;
  const u32x4 ones = {one2, one2, one2, one2};
#pragma unroll
  for (int q = 0; q < kGroups; q++) {
    f32x4 sum[MT];
#pragma unroll
    for (int t = 0; t < MT; t++) {
      sum[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kJ; j++) sum[t] = mma_dense<BF16>(ones, b.x[t][q * kJ + j], sum[t]);
    }
#pragma unroll
    for (int i = 0; i < RB; i++) {
      float s[4], z[4];
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const uint16_t h = (uint16_t)(b.s[i].v[2 * q + (r >> 1)] >> (16 * (r & 1)));
        s[r] = BF16 ? __uint_as_float((uint32_t)h << 16) : (float)__builtin_bit_cast(_Float16, h);
        z[r] = ZERO ? 16.0f + (float)((b.z[i].v[q] >> (8 * r)) & 15u) : 24.0f;
      }
      u32x4 w[kJ];
#pragma unroll
      for (int j = 0; j < kJ; j++) w[j] = widen4<BF16>(b.w[i][q * kJ + j]);
#pragma unroll
      for (int t = 0; t < MT; t++) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kJ; j++) acc = mma_dense<BF16>(w[j], b.x[t][q * kJ + j], acc);
#pragma unroll
        for (int r = 0; r < 4; r++) y[i][t][r] += s[r] * (acc[r] - z[r] * sum[t][r]);
      }
    }
  }
}

// MT blocks of 16 tokens, RB bands, G columns a group.
template <bool BF16, bool OUT_F32, int MT, int RB, int G, bool ZERO>
__global__ __launch_bounds__(kMaxWaves * 64) void k_w4(W4Args a) {
  extern __shared__ f32x4 part[];  // [wave][RB][MT][lane]
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6, waves = (int)blockDim.x >> 6, n = lane & 15;
  const int64_t band = (int64_t)blockIdx.x * RB, m0 = (int64_t)blockIdx.y * (16 * MT);
  const uint16_t* xp[MT];
#pragma unroll
  for (int t = 0; t < MT; t++)  // rows behind M: the last, not stored
    xp[t] = reinterpret_cast<const uint16_t*>(a.X) + min(m0 + 16 * t + n, a.M - 1) * a.K;
  f32x4 y[RB][MT];
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int t = 0; t < MT; t++) y[i][t] = (f32x4){0.f, 0.f, 0.f, 0.f};

  if (wave < a.blocks) {
    Block<MT, RB, G, ZERO> cur = load_block<MT, RB, G, ZERO>(a, band, xp, wave);
    for (int b = wave; b < a.blocks; b += waves) {
      // the next block's bytes are on their way while this one's are used
      const Block<MT, RB, G, ZERO> next = load_block<MT, RB, G, ZERO>(a, band, xp, b + waves < a.blocks ? b + waves : b);
      multiply<BF16, MT, RB, G, ZERO>(cur, y);
      cur = next;
    }
  }
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int t = 0; t < MT; t++) part[((wave * RB + i) * MT + t) * 64 + lane] = y[i][t];
  __syncthreads();
  // lane l of block t holds rows 4 (l / 16) .. + 3, token l % 16
  for (int e = (int)threadIdx.x; e < RB * MT * 64; e += (int)blockDim.x) {
    const int i = e / (MT * 64), t = (e >> 6) % MT, l = e & 63;
    f32x4 v = part[e];
    for (int w = 1; w < waves; w++) v += part[w * RB * MT * 64 + e];
    const int64_t m = m0 + 16 * t + (l & 15), row = (band + i) * 16 + 4 * (l >> 4);
    if (m >= a.M || row >= a.N) continue;
    if (row + 4 <= a.N && (a.N & 3) == 0) {
      store4<BF16, OUT_F32>(a.Y, m * a.N + row, v);
    } else {
      for (int c = 0; c < 4 && row + c < a.N; c++) {
        if constexpr (OUT_F32)
          reinterpret_cast<float*>(a.Y)[m * a.N + row + c] = v[c];
        else if constexpr (BF16)
          reinterpret_cast<__bf16*>(a.Y)[m * a.N + row + c] = (__bf16)v[c];
        else
          reinterpret_cast<_Float16*>(a.Y)[m * a.N + row + c] = (_Float16)v[c];
      }
    }
  }
}

// ---- layout ----
__host__ __device__ inline int64_t n_bands(int64_t N) { return (N + 15) / 16; }
__host__ __device__ inline int64_t n_blocks(int64_t K) { return (K + 127) / 128; }
inline int64_t scale_offset(int64_t N, int64_t K) { return n_bands(N) * n_blocks(K) * 1024; }
inline int64_t n_scales(int64_t N, int64_t K, int64_t G) { return n_bands(N) * 16 * n_blocks(K) * (128 / G); }
inline int64_t zero_offset(int64_t N, int64_t K, int64_t G) { return scale_offset(N, K) + n_scales(N, K, G) * 2; }

// One thread a 32-bit word of the weights, then one a scale and zero.
__global__ __launch_bounds__(256) void k_w4_pack(int64_t N, int64_t K, int64_t G, const uint8_t* __restrict__ q,
                                                 const uint16_t* __restrict__ scale, const uint8_t* __restrict__ zero,
                                                 uint32_t* __restrict__ w, uint16_t* __restrict__ so,
                                                 uint8_t* __restrict__ zo) {
  const int64_t words = n_bands(N) * n_blocks(K) * 256, groups = K / G, per = 128 / G;
  const int64_t extra = n_bands(N) * 16 * n_blocks(K) * per;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < words + extra; e += (int64_t)gridDim.x * 256) {
    if (e < words) {
      const int64_t block = e >> 8, band = block / n_blocks(K);
      const int j = (int)e & 3, l = (int)(e >> 2) & 63;
      const int64_t row = band * 16 + (l & 15), k = (block - band * n_blocks(K)) * 128 + 32 * j + 8 * (l >> 4);
      uint32_t v = 0;
      if (row < N && k < K) {  // K and k are multiples of 8
        const uint32_t b = *reinterpret_cast<const uint32_t*>(q + row * (K / 2) + k / 2);
#pragma unroll
        for (int i = 0; i < 4; i++)
          v |= ((b >> (8 * i)) & 15u) << (4 * i) | ((b >> (8 * i + 4)) & 15u) << (16 + 4 * i);
      }
      w[e] = v;
    } else {
      // place f = (((band, block), quad), group of the block), row of the quad
      const int64_t f = e - words, block = f / (16 * per), band = block / n_blocks(K);
      const int r = (int)(f - block * 16 * per), quad = r / (4 * (int)per), c = r - quad * 4 * (int)per;
      const int64_t row = band * 16 + 4 * quad + (c & 3), gr = (block - band * n_blocks(K)) * per + (c >> 2);
      const bool ok = row < N && gr < groups;
      so[f] = ok ? scale[row * groups + gr] : (uint16_t)0;
      if (zo) zo[f] = ok ? zero[row * groups + gr] & 15 : 0;
    }
  }
}

// One wave a group at a time: G = 32, 64 or 128 columns, two neighbours a lane.
template <typename T>
__global__ __launch_bounds__(256) void k_w4_quantize(int64_t N, int64_t K, int G, const T* __restrict__ W,
                                                     uint8_t* __restrict__ q, T* __restrict__ scale,
                                                     uint8_t* __restrict__ zero) {
  const int lane = (int)threadIdx.x & 63, per = 128 / G, sub = lane / (G / 2);  // groups of a wave
  const int64_t groups = K / G, all = N * groups;
  for (int64_t g0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * per; g0 < all; g0 += (int64_t)gridDim.x * 4 * per) {
    const int64_t gi = g0 + sub;
    const bool ok = gi < all;
    const int64_t at = gi * G + 2 * (lane % (G / 2));  // rows are whole groups: element index = group index * G + column
    const float x = ok ? (float)W[at] : 0.f, y = ok ? (float)W[at + 1] : 0.f;
    float hi = fmaxf(x, y), lo = fminf(x, y);
    for (int d = 1; d < G / 2; d *= 2) {
      hi = fmaxf(hi, __shfl_xor(hi, d));
      lo = fminf(lo, __shfl_xor(lo, d));
    }
    T st;
    float z = 8.0f;
    float s;
    if (zero) {
      hi = fmaxf(hi, 0.f);
      lo = fminf(lo, 0.f);
      st = (T)((hi - lo) / 15.0f);
      s = (float)st;
      z = s > 0.f ? fminf(15.f, fmaxf(0.f, rintf(-lo / s))) : 8.f;
    } else {
      st = (T)(fmaxf(hi, -lo) / 7.0f);
      s = (float)st;
    }
    const float least = zero ? 0.f : 1.f;
    const float qx = s > 0.f ? fminf(15.f, fmaxf(least, rintf(x / s) + z)) : 8.f;
    const float qy = s > 0.f ? fminf(15.f, fmaxf(least, rintf(y / s) + z)) : 8.f;
    if (ok) {
      q[at / 2] = (uint8_t)((uint32_t)qx | (uint32_t)qy << 4);
      if (lane % (G / 2) == 0) {
        scale[gi] = st;
        if (zero) zero[gi] = (uint8_t)z;
      }
    }
  }
}

template <bool BF16, bool OUT_F32, int MT, int RB, int G, bool ZERO>
hipError_t go(const W4Args& a, hipStream_t s) {
  const int64_t my = (a.M + 16 * MT - 1) / (16 * MT);
  // a wave takes two blocks or more where there are enough
  const int waves = std::max(1, std::min(kMaxWaves, a.blocks / 2));
  const size_t lds = (size_t)waves * RB * MT * 1024;
  hipLaunchKernelGGL((k_w4<BF16, OUT_F32, MT, RB, G, ZERO>), dim3((unsigned)((a.bands + RB - 1) / RB), (unsigned)my),
                     dim3(64 * waves), lds, s, a);
  return hipGetLastError();
}
template <bool BF16, bool OUT_F32, int MT, int RB, int G>
hipError_t by_zero(const W4Args& a, hipStream_t s) {
  return a.zero ? go<BF16, OUT_F32, MT, RB, G, true>(a, s) : go<BF16, OUT_F32, MT, RB, G, false>(a, s);
}
template <bool BF16, bool OUT_F32, int MT, int RB>
hipError_t by_group(const W4Args& a, hipStream_t s) {
  switch (a.group) {
    case 32: return by_zero<BF16, OUT_F32, MT, RB, 32>(a, s);
    case 64: return by_zero<BF16, OUT_F32, MT, RB, 64>(a, s);
    default: return by_zero<BF16, OUT_F32, MT, RB, 128>(a, s);
  }
}
template <bool BF16, bool OUT_F32, int MT>
hipError_t by_bands(const W4Args& a, hipStream_t s) {
  // A workgroup reads its tokens whole from L2 and has a CU to itself: as many
  // bands as make one round of the GPU, so that tokens are read seldom and no
  // second round waits, up to what its registers hold.  11008 x 4096 (688
  // bands), 16 tokens: 16.1 us with two bands, 11.5 with three, 12.9 with four;
  // 4096 x 4096 (256 bands), 64 tokens: 22.9 us with one, 14.0 with two, 15.4
  // with four; 2048 tokens: 598 us with one, 346 with two, 209 with four.
  const int64_t wide = (a.M + 16 * MT - 1) / (16 * MT);
  switch (std::min<int64_t>((a.bands * wide + cu_count() - 1) / cu_count(), 4)) {
    case 0:
    case 1: return by_group<BF16, OUT_F32, MT, 1>(a, s);
    case 2: return by_group<BF16, OUT_F32, MT, 2>(a, s);
    case 3: return by_group<BF16, OUT_F32, MT, 3>(a, s);
    default: return by_group<BF16, OUT_F32, MT, 4>(a, s);
  }
}
template <bool BF16, bool OUT_F32>
hipError_t by_tokens(const W4Args& a, hipStream_t s) {
  return a.M > 16 ? by_bands<BF16, OUT_F32, 2>(a, s) : by_bands<BF16, OUT_F32, 1>(a, s);
}

}  // namespace

uint64_t w4_bytes(int64_t N, int64_t K, int64_t G, bool zero) {
  return (uint64_t)(zero_offset(N, K, G) + (zero ? n_scales(N, K, G) : 0));
}

hipError_t launch_w4_quantize(bool bf16, int64_t N, int64_t K, int group, const void* W, uint8_t* q, void* scale,
                              uint8_t* zero, hipStream_t s) {
  const int64_t waves = (N * (K / group) + 128 / group - 1) / (128 / group);
  const unsigned blocks = (unsigned)std::min<int64_t>((waves + 3) / 4, 65536);
  if (bf16)
    hipLaunchKernelGGL((k_w4_quantize<__bf16>), dim3(blocks), dim3(256), 0, s, N, K, group,
                       reinterpret_cast<const __bf16*>(W), q, reinterpret_cast<__bf16*>(scale), zero);
  else
    hipLaunchKernelGGL((k_w4_quantize<_Float16>), dim3(blocks), dim3(256), 0, s, N, K, group,
                       reinterpret_cast<const _Float16*>(W), q, reinterpret_cast<_Float16*>(scale), zero);
  return hipGetLastError();
}

hipError_t launch_w4_pack(int64_t N, int64_t K, int group, const uint8_t* q, const void* scale, const uint8_t* zero,
                          uint8_t* packed, hipStream_t s) {
  const int64_t all = n_bands(N) * n_blocks(K) * 256 + n_scales(N, K, group);
  const unsigned blocks = (unsigned)std::min<int64_t>((all + 255) / 256, 65536);
  hipLaunchKernelGGL(k_w4_pack, dim3(blocks), dim3(256), 0, s, N, K, (int64_t)group, q,
                     reinterpret_cast<const uint16_t*>(scale), zero, reinterpret_cast<uint32_t*>(packed),
                     reinterpret_cast<uint16_t*>(packed + scale_offset(N, K)),
                     zero ? packed + zero_offset(N, K, group) : nullptr);
  return hipGetLastError();
}

hipError_t launch_w4_gemm(bool bf16, bool out_f32, bool zero, int64_t N, int64_t K, int group, const uint8_t* packed,
                          const void* X, int64_t M, void* Y, hipStream_t s) {
  W4Args a;
  a.w = packed;
  a.scale = packed + scale_offset(N, K);
  a.zero = zero ? packed + zero_offset(N, K, group) : nullptr;
  a.N = N;
  a.K = K;
  a.bands = (int)n_bands(N);
  a.blocks = (int)n_blocks(K);
  a.group = group;
  constexpr int64_t kMost = int64_t(32) * 65535;  // rows of a launch, by the grid's second extent
  for (int64_t m = 0; m < M; m += kMost) {
    a.X = reinterpret_cast<const uint16_t*>(X) + m * K;
    a.Y = reinterpret_cast<char*>(Y) + m * N * (out_f32 ? 4 : 2);
    a.M = std::min(M - m, kMost);
    const hipError_t e = bf16 ? (out_f32 ? by_tokens<true, true>(a, s) : by_tokens<true, false>(a, s))
                              : (out_f32 ? by_tokens<false, true>(a, s) : by_tokens<false, false>(a, s));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace patch
