// attention.hip -- attention over the paged 8-bit cache.
//
// out = softmax(scale q k^T) v, one pass over the keys with the running
// maximum m, sum l and output o of each row: a step's scores s give m' =
// max(m, s), and l and o are multiplied by 2^(m - m') before the step's 2^(s -
// m') and 2^(s - m') v are added (scores in units of log2).
//
// Rows are the query tokens times the query heads that share a cache head:
// row r of a (sequence, cache head) is token r / group, head r % group, so
// grouped heads read the cache once.  A workgroup has 16 R rows; its four
// waves take its 32-key steps in turn, each with m, l, o of its own, and join
// them at the end through LDS.
//
// Operands of v_mfma_f32_16x16x32 (A: lane l = row l % 16, 8 of the 32 k's; B
// likewise by column; D: row 4 (l / 16) + i, column l % 16):
//   scores^T = K Q^T   A = 16 keys, B = 16 rows of Q: a lane then holds the
//                      scores of 4 keys for ONE row, l % 16, and so do the
//                      three lanes 16 apart: maxima and sums cross lanes
//                      twice, not four times, and m, l are one register.
//   out^T = V^T P^T    B = P^T: its lane holds 8 keys of its row.  The order of
//                      the k's is free if both operands share it: slots 0-3
//                      are the keys 4g + i, slots 4-7 the keys 16 + 4g + i (g =
//                      l / 16), which are the scores the lane already holds.
// V^T wants 8 keys of one element in a lane, but a cache row holds the
// elements of one key: a lane loads DP / 16 neighbouring bytes of 8 rows and
// zips them pairwise with v_perm_b32 before the conversion (a quarter of an
// instruction a byte); row l % 16 of matrix instruction j is then element (l
// % 16) * DP / 16 + j.
//
// 8-bit values become 16-bit ones exactly (q's type for the scores; fp16 for
// the second product, whose probabilities keep 11 bits: 2^(s - m + 14), up to
// 16384, so that small ones do not fall under fp16's normal range).  A block's
// k scale multiplies the scores, its v scale the probabilities, relative to
// the largest v scale so far (vref), o being kept in units of it.
#include <algorithm>

#include "device_common.h"
#include "layer_common.h"

namespace patch {
namespace {

constexpr int kWaves = 4;
constexpr int kStep = 32;       // keys of a step
constexpr float kBias = 14.0f;  // probabilities are 2^(s - m + kBias)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Eight e4m3 bytes as eight 16-bit values.
template <bool BF16>
__device__ __forceinline__ u32x4 widen8(uint32_t lo, uint32_t hi) {
  u32x4 r;
  if constexpr (BF16) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
  }
  return r;
}

// A sequence's newest tokens and what its rows see.
struct Seq {
  int c0, n;        // tokens c0 .. c0 + n - 1
  int64_t past;     // position of the first
  bool bad;         // its length does not fit its page table
};

__device__ __forceinline__ Seq seq_of(const patch_attention_args& a, const patch_kv_cache& c, int s) {
  Seq q;
  const int e = min(a.cu_new_dev[s + 1], (int)a.T);
  q.c0 = max(a.cu_new_dev[s], 0);
  q.n = max(e - q.c0, 0);
  const int64_t len = a.kv_lens_dev[s];
  q.past = len - q.n;
  q.bad = len > a.max_pages * c.page;
  return q;
}

template <bool BF16, int DP, int R>
struct Tile {
  static constexpr int kRows = 16 * R;
  static constexpr int kLd = DP + 4;  // floats of an LDS row
  u32x4 q[R][DP / 32];
  f32x4 o[R][DP / 16];
  float m[R], l[R];
  int hi[R], lo[R];  // the last and first key this lane's row sees
  float vref;
};

// One task: rows r0 .. r0 + 16 R - 1 of (sequence s, cache head h), the steps
// from begin to end.
template <bool BF16, int DP, int R>
__device__ void run_task(const patch_attention_args& a, const patch_kv_cache& c, const Seq& sq, int s, int h, int r0,
                         int begin, int end, float* lds) {
  using TL = Tile<BF16, DP, R>;
  TL x;
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
  const int D = (int)c.dim, B = (int)c.page, group = (int)(a.heads / c.kv_heads);
  const int rows = sq.n * group;
  const int shift = 31 - __clz(B);
  const float scale = (float)a.scale * kLog2e;
  const int32_t* table = a.page_table_dev + s * a.page_table_row;

  int first_pos, last_pos;  // positions of the task's first and last token
  {
    const int last = min(r0 + TL::kRows, rows) - 1;
    first_pos = (int)(sq.past + r0 / group);
    last_pos = (int)(sq.past + last / group);
  }
  const int w = a.window > 0 ? (int)min(a.window, (int64_t)0x7fffffff) : 0;
  const int all_from = w > 0 ? max(last_pos - w + 1, 0) : 0;  // every row sees the keys all_from .. first_pos
  const int any_from = w > 0 ? max(first_pos - w + 1, 0) : 0;

#pragma unroll
  for (int r = 0; r < R; r++) {
    const int row = r0 + r * 16 + n, tok = row / group;
    const bool ok = row < rows;
    x.hi[r] = ok ? (int)(sq.past + tok) : 0x7fffffff;  // rows that are none see everything and are not stored
    x.lo[r] = ok && w > 0 ? x.hi[r] - w + 1 : (int)0x80000000;
    const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q_dev) +
                         (ok ? (int64_t)(sq.c0 + tok) * a.q_token + (int64_t)(h * group + row - tok * group) * a.q_head : 0);
    const bool wide = ((a.q_token | a.q_head) & 7) == 0 && ((uintptr_t)a.q_dev & 15) == 0;
#pragma unroll
    for (int j = 0; j < DP / 32; j++) {
      const int d = (j >> 1) * 64 + g * 16 + (j & 1) * 8;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (ok && d < D) {
        if (wide) {
          v = ld16(qp + d);
        } else {
#pragma unroll
          for (int i = 0; i < 4; i++) v[i] = (uint32_t)qp[d + 2 * i] | (uint32_t)qp[d + 2 * i + 1] << 16;
        }
      }
      x.q[r][j] = v;
    }
#pragma unroll
    for (int j = 0; j < DP / 16; j++) x.o[r][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    x.m[r] = -__builtin_inff();
    x.l[r] = 0.f;
  }
  x.vref = 0.f;

  const int64_t head_bytes = (int64_t)B * D, page_bytes = c.kv_heads * head_bytes;
  const uint8_t* kc = reinterpret_cast<const uint8_t*>(c.k_dev) + h * head_bytes;
  const uint8_t* vc = reinterpret_cast<const uint8_t*>(c.v_dev) + h * head_bytes;
  constexpr int VB = DP / 16;  // bytes of a V row in a lane

  for (int step = begin + wave; step < end; step += kWaves) {
    const int key0 = step * kStep;
    // the page of each half of the step (16 keys lie in one page); a half behind the last key reads the last page
    const uint8_t *kp[2], *vp[2];
    float ks[2], vs[2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      const int key = min(key0 + 16 * t, last_pos & ~15);
      int page = __builtin_amdgcn_readfirstlane(table[key >> shift]);
      const bool bad_page = page < 0 || page >= c.pages;
      page = bad_page ? 0 : page;
      const int64_t at = page * page_bytes + (int64_t)(key & (B - 1)) * D;
      kp[t] = kc + at;
      vp[t] = vc + at;
      ks[t] = bad_page ? __builtin_nanf("") : c.k_scale_dev[page * c.kv_heads + h] * scale;
      vs[t] = bad_page ? 0.f : c.v_scale_dev[page * c.kv_heads + h];
    }
    const bool partial = key0 < all_from || key0 + kStep - 1 > first_pos;

    u32x4 kr[2][DP / 64];
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int j = 0; j < DP / 64; j++) {
        const int d = j * 64 + g * 16;
        kr[t][j] = ld16_pred(kp[t] + n * D + d, d < D);
      }
    Vec<uint32_t, VB / 4> vr[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int slot = 4 * g + (i & 3);
#pragma unroll
      for (int b = 0; b < VB / 4; b++) vr[i].v[b] = 0u;
      if (n * VB < D) vr[i] = *reinterpret_cast<const Vec<uint32_t, VB / 4>*>(vp[i >> 2] + slot * D + n * VB);
    }

    // scores
    f32x4 sc[R][2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
#pragma unroll
      for (int r = 0; r < R; r++) sc[r][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < DP / 64; j++) {
        const u32x4 a0 = widen8<BF16>(kr[t][j][0], kr[t][j][1]), a1 = widen8<BF16>(kr[t][j][2], kr[t][j][3]);
#pragma unroll
        for (int r = 0; r < R; r++) {
          sc[r][t] = mma_dense<BF16>(a0, x.q[r][2 * j], sc[r][t]);
          sc[r][t] = mma_dense<BF16>(a1, x.q[r][2 * j + 1], sc[r][t]);
        }
      }
    }
    bool nan_v = false;
    if (partial) {
      // V rows that no row of the task sees hold anything at all: take zeros.
      // A NaN in a row that some see must not reach the others through 0 *
      // NaN: it is taken out here and put back below, row by row.
      bool has = false;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int key = key0 + (i >> 2) * 16 + 4 * g + (i & 3);
        const bool seen = key >= any_from && key <= last_pos;
#pragma unroll
        for (int b = 0; b < VB / 4; b++) {
          uint32_t v = seen ? vr[i].v[b] : 0u;
          // a byte is NaN where its low seven bits are all set
          const uint32_t hit = ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
          has |= hit != 0;
          v &= ~((hit >> 7) * 0xffu);
          vr[i].v[b] = v;
        }
      }
      nan_v = __ballot(has) != 0;
    }

    // running maximum and sum, probabilities
    const float vmax = fmaxf(fabsf(vs[0]), fabsf(vs[1]));
    float ratio = 1.0f;
    if (vmax > x.vref) {
      ratio = x.vref / vmax;
      x.vref = vmax;
    }
    const float inv = x.vref > 0.f ? 1.0f / x.vref : 0.f;
    const float vf[2] = {vs[0] * inv, vs[1] * inv};
    u32x4 pr[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      float p[8];
      float mx = x.m[r];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        p[i] = sc[r][i >> 2][i & 3] * ks[i >> 2];
        if (partial) {
          const int key = key0 + (i >> 2) * 16 + 4 * g + (i & 3);
          if (key > x.hi[r] || key < x.lo[r] || key > last_pos) p[i] = -__builtin_inff();
        }
        mx = fmaxf(mx, p[i]);
      }
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float mu = mx == -__builtin_inff() ? 0.f : mx;
      const float alpha = exp2f(x.m[r] - mu);
      x.m[r] = mx;
      float sum = 0.f;
      f16x8 ph;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float e = exp2f(p[i] - mu + kBias);
        sum += e;
        ph[i] = (_Float16)(e * vf[i >> 2]);
      }
      pr[r] = __builtin_bit_cast(u32x4, ph);
      x.l[r] = x.l[r] * alpha + sum;
      const float f = alpha * ratio;
      if (__ballot(f != 1.0f)) {
#pragma unroll
        for (int j = 0; j < DP / 16; j++) x.o[r][j] *= f;
      }
    }

    // o += V^T P^T
#pragma unroll
    for (int b = 0; b < VB / 4; b++) {
      u32x4 e[4];
#pragma unroll
      for (int p = 0; p < 4; p++) {
        const uint32_t k0 = vr[2 * p].v[b], k1 = vr[2 * p + 1].v[b];
        const uint32_t z0 = __builtin_amdgcn_perm(k1, k0, 0x05010400u), z1 = __builtin_amdgcn_perm(k1, k0, 0x07030602u);
        e[0][p] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(z0, 1.0f, false));
        e[1][p] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(z0, 1.0f, true));
        e[2][p] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(z1, 1.0f, false));
        e[3][p] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(z1, 1.0f, true));
      }
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int r = 0; r < R; r++) x.o[r][4 * b + j] = mma_dense<false>(e[j], pr[r], x.o[r][4 * b + j]);
    }
    if (nan_v) {  // rare: a NaN value in a row of V that not every row of the task sees
      for (int k = 0; k < kStep; k++) {
        const int key = key0 + k;
        if (key < any_from || key > last_pos) continue;
        const uint8_t* row = vp[k >> 4] + (k & 15) * D;
#pragma unroll
        for (int j = 0; j < VB; j++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int d = (4 * g + i) * VB + j;
            const bool is_nan = d < D && (row[d] & 0x7f) == 0x7f;
#pragma unroll
            for (int r = 0; r < R; r++)
              if (is_nan && key <= x.hi[r] && key >= x.lo[r]) x.o[r][j][i] = __builtin_nanf("");
          }
      }
    }
  }

  // the lanes of a row hold parts of its sum
#pragma unroll
  for (int r = 0; r < R; r++) {
    x.l[r] += __shfl_xor(x.l[r], 16);
    x.l[r] += __shfl_xor(x.l[r], 32);
  }

  // ---- join the waves: o, m, l, vref through LDS ----
  float* lo = lds + wave * TL::kRows * TL::kLd;
  float* lml = lds + kWaves * TL::kRows * TL::kLd;  // [wave][row][m, l], then [wave] vref
#pragma unroll
  for (int r = 0; r < R; r++) {
    float* at = lo + (r * 16 + n) * TL::kLd + 4 * g * VB;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < VB; j += 4)
        *reinterpret_cast<f32x4*>(at + i * VB + j) =
            (f32x4){x.o[r][j][i], x.o[r][j + 1][i], x.o[r][j + 2][i], x.o[r][j + 3][i]};
    if (g == 0) {
      lml[(wave * TL::kRows + r * 16 + n) * 2] = x.m[r];
      lml[(wave * TL::kRows + r * 16 + n) * 2 + 1] = x.l[r];
    }
  }
  if (lane == 0) lml[kWaves * TL::kRows * 2 + wave] = x.vref;
  __syncthreads();

  const int chunks = D / 8;
  const bool wide = ((a.out_token | a.out_head) & 7) == 0 && ((uintptr_t)a.out_dev & 15) == 0;
  for (int e = tid; e < TL::kRows * chunks; e += kWaves * 64) {
    const int row = e / chunks, d = (e - row * chunks) * 8;
    if (r0 + row >= rows) break;
    float mx = -__builtin_inff();
#pragma unroll
    for (int v = 0; v < kWaves; v++) mx = fmaxf(mx, lml[(v * TL::kRows + row) * 2]);
    const float mu = mx == -__builtin_inff() ? 0.f : mx;
    float sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kWaves; v++) {
      const float f = exp2f(lml[(v * TL::kRows + row) * 2] - mu);
      sum += f * lml[(v * TL::kRows + row) * 2 + 1];
      const float fo = f * lml[kWaves * TL::kRows * 2 + v];
      const float* p = lds + (v * TL::kRows + row) * TL::kLd + d;
#pragma unroll
      for (int i = 0; i < 8; i++) acc[i] += fo * p[i];
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    const int tok = (r0 + row) / group, head = h * group + (r0 + row) - tok * group;
    if (a.lse_dev && d == 0)
      a.lse_dev[(int64_t)(sq.c0 + tok) * a.heads + head] = (mx + log2f(sum) - kBias) * kLn2;
    const int64_t at = (int64_t)(sq.c0 + tok) * a.out_token + (int64_t)head * a.out_head + d;
    if (a.out_dtype == PATCH_F32) {
      float* op = reinterpret_cast<float*>(a.out_dev) + at;
      if (wide) {
        *reinterpret_cast<f32x4*>(op) = (f32x4){acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
        *reinterpret_cast<f32x4*>(op + 4) = (f32x4){acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv};
      } else {
        for (int i = 0; i < 8; i++) op[i] = acc[i] * inv;
      }
    } else {
      typedef std::conditional_t<BF16, __bf16, _Float16> T;
      Vec<T, 8> v;
#pragma unroll
      for (int i = 0; i < 8; i++) v.v[i] = (T)(acc[i] * inv);
      T* op = reinterpret_cast<T*>(a.out_dev) + at;
      if (wide) {
        *reinterpret_cast<Vec<T, 8>*>(op) = v;
      } else {
        for (int i = 0; i < 8; i++) op[i] = v.v[i];
      }
    }
  }
  __syncthreads();
}

// Rows that see no key, or whose sequence does not fit its page table.
template <bool BF16>
__device__ void fill_rows(const patch_attention_args& a, int c0, int h, int r0, int r1, int group, int D, float o,
                          float lse) {
  for (int e = threadIdx.x; e < (r1 - r0) * D; e += kWaves * 64) {
    const int row = r0 + e / D, d = e % D, tok = row / group, head = h * group + row - tok * group;
    const int64_t at = (int64_t)(c0 + tok) * a.out_token + (int64_t)head * a.out_head + d;
    if (a.out_dtype == PATCH_F32)
      reinterpret_cast<float*>(a.out_dev)[at] = o;
    else if (BF16)
      reinterpret_cast<__bf16*>(a.out_dev)[at] = (__bf16)o;
    else
      reinterpret_cast<_Float16*>(a.out_dev)[at] = (_Float16)o;
    if (a.lse_dev && d == 0) a.lse_dev[(int64_t)(c0 + tok) * a.heads + head] = lse;
  }
}

// A workgroup a task: sequence s has the tasks floor(cu[s] group / rows) + s
// up to the same of s + 1 for each head, at least as many as its rows need.
template <bool BF16, int DP, int R>
__global__ __launch_bounds__(kWaves * 64) void k_attention(patch_attention_args a, patch_kv_cache c) {
  extern __shared__ __align__(16) float lds[];
  constexpr int kRows = 16 * R;
  const int heads = (int)c.kv_heads, group = (int)(a.heads / c.kv_heads);
  const int h = (int)(blockIdx.x % (uint32_t)heads);
  const int64_t slot = blockIdx.x / (uint32_t)heads;
  const int32_t* cu = a.cu_new_dev;
  const int s = find_last((int)a.S, [&](int i) { return (int64_t)cu[i] * group / kRows + i <= slot; });
  const int64_t first = (int64_t)cu[s] * group / kRows + s;
  const Seq sq = seq_of(a, c, s);
  const int64_t r0w = (slot - first) * kRows;
  if (slot < first || r0w >= (int64_t)sq.n * group) return;
  const int r0 = (int)r0w, r1 = min(r0 + kRows, sq.n * group);
  const int64_t last_pos = sq.past + (r1 - 1) / group;
  if (sq.bad || last_pos < 0) {
    fill_rows<BF16>(a, sq.c0, h, r0, r1, group, (int)c.dim, sq.bad ? __builtin_nanf("") : 0.f,
                    sq.bad ? __builtin_nanf("") : -__builtin_inff());
    return;
  }
  const int64_t first_pos = sq.past + r0 / group;
  const int64_t from = a.window > 0 && first_pos - a.window + 1 > 0 ? first_pos - a.window + 1 : 0;
  run_task<BF16, DP, R>(a, c, sq, s, h, r0, (int)(from / kStep), (int)(last_pos / kStep) + 1, lds);
}

template <bool BF16, int DP, int R>
hipError_t go(const patch_attention_args& a, const patch_kv_cache& c, hipStream_t s) {
  constexpr int kRows = 16 * R;
  const int64_t group = a.heads / c.kv_heads;
  const int64_t blocks = (a.T * group / kRows + a.S) * c.kv_heads;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  const size_t lds = sizeof(float) * (size_t)(kWaves * kRows * (DP + 4) + kWaves * kRows * 2 + kWaves);
  if (lds > 65536) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_attention<BF16, DP, R>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_attention<BF16, DP, R>), dim3((unsigned)blocks), dim3(kWaves * 64), lds, s, a, c);
  return hipGetLastError();
}

template <bool BF16>
hipError_t by_dim(const patch_attention_args& a, const patch_kv_cache& c, hipStream_t s) {
  if (c.dim <= 64) return go<BF16, 64, 1>(a, c, s);
  if (c.dim <= 128) return go<BF16, 128, 1>(a, c, s);
  return go<BF16, 256, 1>(a, c, s);
}

}  // namespace

uint64_t attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_attention(const patch_attention_args& a, const patch_kv_cache& c, void*, uint64_t, hipStream_t s) {
  return a.dtype == PATCH_BF16 ? by_dim<true>(a, c, s) : by_dim<false>(a, c, s);
}

}  // namespace patch
