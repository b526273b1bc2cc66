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
// the second product, whose probabilities keep 11 bits, or 22 in two values and
// products where the output is fp32).  A block's
// k scale multiplies the scores, its v scale the probabilities, relative to
// the largest v scale so far (vref), o being kept in units of it.
//
// Which work a workgroup gets is settled on the device, since lengths change
// between replays of a graph: the steps of all tasks (16 R rows of a sequence
// and cache head) lie on one line, and workgroup w of W takes the w-th of W
// equal pieces, whatever mix of long and short sequences that is.  A task
// that falls to several workgroups leaves parts (o, m, l) in the workspace,
// written and read with the agent-coherent policy (what every XCD sees);
// each part's flag is set after its data has arrived, and a workgroup that
// then finds all flags of the task set joins the parts, in order.  Nobody
// waits: setting a flag and then reading all means that the last to set one
// sees them all.  Two may; they write the same values.  A flag is a 64-bit
// value of the launch, put back to 0 by who joins, so the workspace's
// contents do not matter and a captured launch replays.
//
// Bound by the cache's bytes from a few megabytes on, below that by the chain
// lengths -> page table -> scales -> keys -> parts -> join, which is a handful
// of trips to memory.  Heads of 128, GPU time: 48 sequences of 200 to 4000
// tokens, 8 cache heads, 224 MB in 53.6 us (4.2 TB/s); two of 100 000 to 130
// 000, 486 MB in 110 us (4.4 TB/s; a copy of 1 GiB reaches 5.1); one of 700,
// 32 cache heads, 5.7 MB in 11.4 us.
#include <algorithm>
#include <atomic>
#include <chrono>
#include <random>

#include "attention_common.h"

namespace patch {
using namespace attn;
namespace {

constexpr int kStep = 32;  // keys of a step
constexpr int kWaves = 4, kThreads = 64 * kWaves;

// The pages of a wave's next 64 steps, one step a lane; h: halves of a step
// (16 keys lie in one page).  A page outside the cache reads page 0 with a
// NaN scale.
struct Pages {
  int page[2];
  float ks[2], vs[2];
};
__device__ __forceinline__ Pages load_pages(const Args& a, const int32_t* table, int h, int first, int last_pos) {
  Pages p;
  const int step = first + kWaves * (int)(threadIdx.x & 63);
#pragma unroll
  for (int t = 0; t < 2; t++) {
    const int64_t key = min((int64_t)step * kStep + 16 * t, (int64_t)(last_pos & ~15));  // behind the last key: its page
    const int page = table[key >> a.shift];
    const bool ok = page >= 0 && page < a.pages;
    p.page[t] = ok ? page : 0;
    const int64_t at = (int64_t)p.page[t] * a.kv_heads + h;
    const float ks = a.ks[at], vs = a.vs[at];
    p.ks[t] = ok ? ks * a.scale : __builtin_nanf("");
    p.vs[t] = ok ? vs : 0.f;
  }
  return p;
}
// The bytes of a step: K as A operands, V in bytes [key slot][element].
template <int DP>
struct Bytes {
  static constexpr int VB = DP / 16;  // bytes of a V row in a lane
  u32x4 k[2][DP / 64];
  Vec<uint32_t, VB / 4> v[8];
  const uint8_t* vp[2];
  float ks[2], vs[2];
};
template <int DP>
__device__ __forceinline__ Bytes<DP> load_step(const Args& a, const Pages& p, int i, int h, int step, int last_pos) {
  constexpr int VB = Bytes<DP>::VB;
  const int lane = (int)threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  Bytes<DP> b;
#pragma unroll
  for (int t = 0; t < 2; t++) {
    const int key = min(step * kStep + 16 * t, last_pos & ~15);
    const int64_t at = (((int64_t)lane_of(p.page[t], i) * a.kv_heads + h) * a.B + (key & (a.B - 1))) * a.D;
    b.vp[t] = a.v + at;
    b.ks[t] = lane_of(p.ks[t], i);
    b.vs[t] = lane_of(p.vs[t], i);
    const uint8_t* kp = a.k + at;
    // Behind element D - 1 the same key's first ones: q is zero there (and a
    // NaN among them would make the score NaN in any case).
#pragma unroll
    for (int j = 0; j < DP / 64; j++)
      b.k[t][j] = ld16(kp + (uint32_t)(n * a.D + (j * 64 + g * 16 < a.D ? j * 64 + g * 16 : 0)));
  }
  // likewise; those outputs are not stored
  const uint32_t vo = (uint32_t)(4 * g * a.D + (n * VB < a.D ? n * VB : 0));
#pragma unroll
  for (int i8 = 0; i8 < 8; i8++)
    b.v[i8] = *reinterpret_cast<const Vec<uint32_t, VB / 4>*>(b.vp[i8 >> 2] + (i8 & 3) * a.D + vo);
  return b;
}

// Rows of Q as B operands, and their running state.
template <bool BF16, int DP, int R>
struct Rows {
  u32x4 q[R][DP / 32];
  f32x4 o[R][DP / 16];
  float m[R], l[R];
  int hi[R], lo[R];  // the last and first key this lane's row sees
  float vref;
};
template <bool BF16, int DP, int R>
__device__ __forceinline__ void start_rows(const Args& a, const Seq& sq, const Task& t, int h, Rows<BF16, DP, R>& x) {
  const int lane = (int)threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
  for (int r = 0; r < R; r++) {
    const int row = t.r0 + r * 16 + n, tok = row / a.group;
    const bool ok = row < t.r1;
    x.hi[r] = ok ? sq.past + tok : 0x7fffffff;  // rows that are none see everything and are not stored
    x.lo[r] = ok && a.window > 0 ? x.hi[r] - a.window + 1 : (int)0x80000000;
    const uint16_t* qp =
        a.q + (ok ? (int64_t)(sq.c0 + tok) * a.q_token + (int64_t)(h * a.group + row - tok * a.group) * a.q_head : 0);
#pragma unroll
    for (int j = 0; j < DP / 32; j++) {
      const int d = (j >> 1) * 64 + g * 16 + (j & 1) * 8;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (ok && d < a.D) {
        if (a.q_wide) {
          v = ld16(qp + d);
        } else {
#pragma unroll
          for (int i = 0; i < 4; i++) v[i] = (uint32_t)qp[d + 2 * i] | (uint32_t)qp[d + 2 * i + 1] << 16;
        }
      }
      x.q[r][j] = v ^ a.q_flip;
    }
#pragma unroll
    for (int j = 0; j < DP / 16; j++) x.o[r][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    x.m[r] = -kInf;
    x.l[r] = 0.f;
  }
  x.vref = 0.f;
}

template <bool BF16, int DP, int R, bool WIDE>
__device__ __forceinline__ void do_step(const Args& a, const Task& task, int step, Bytes<DP>& b,
                                        Rows<BF16, DP, R>& x) {
  constexpr int VB = Bytes<DP>::VB;
  const int lane = (int)threadIdx.x & 63, g = lane >> 4;
  const int key0 = step * kStep;
  // every row sees the keys all_from .. first_pos, some row any_from .. last_pos
  const int all_from = a.window > 0 ? max(task.last_pos - a.window + 1, 0) : 0;
  const int any_from = a.window > 0 ? max(task.first_pos - a.window + 1, 0) : 0;
  const bool partial = key0 < all_from || key0 + kStep - 1 > task.first_pos;

  f32x4 sc[R][2];
#pragma unroll
  for (int t = 0; t < 2; t++) {
#pragma unroll
    for (int r = 0; r < R; r++) sc[r][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < DP / 64; j++) {
      const u32x4 a0 = widen8<BF16>(b.k[t][j][0], b.k[t][j][1]), a1 = widen8<BF16>(b.k[t][j][2], b.k[t][j][3]);
#pragma unroll
      for (int r = 0; r < R; r++) {
        sc[r][t] = mma_dense<BF16>(a0, x.q[r][2 * j], sc[r][t]);
        sc[r][t] = mma_dense<BF16>(a1, x.q[r][2 * j + 1], sc[r][t]);
      }
    }
  }
  bool nan_v = false;
  if (partial) {
    const int from = seldom(key0);
    // V rows that no row of the task sees hold anything at all: take zeros.  A
    // NaN in a row that some see must not reach the others through 0 * NaN: it
    // is taken out here and put back below, row by row.
    bool has = false;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int key = from + (i >> 2) * 16 + 4 * g + (i & 3);
      const bool seen = key >= any_from && key <= task.last_pos;
#pragma unroll
      for (int w = 0; w < VB / 4; w++) {
        uint32_t v = seen ? b.v[i].v[w] : 0u;
        // a byte is NaN where its low seven bits are all set
        const uint32_t hit = ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
        has |= hit != 0;
        b.v[i].v[w] = v & ~((hit >> 7) * 0xffu);
      }
    }
    nan_v = __ballot(has) != 0;
  }

  const float vmax = fmaxf(fabsf(b.vs[0]), fabsf(b.vs[1]));
  if (vmax > x.vref) {
    const float f = x.vref / vmax;
    x.vref = vmax;
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
      for (int j = 0; j < DP / 16; j++) x.o[r][j] *= f;
  }
  const float inv = x.vref > 0.f ? 1.0f / x.vref : 0.f;
  const float vf[2] = {b.vs[0] * inv, b.vs[1] * inv};
  u32x4 pr[R], rest[WIDE ? R : 1];
#pragma unroll
  for (int r = 0; r < R; r++) {
    float p[8];
    float mx = -kInf;
#pragma unroll
    for (int i = 0; i < 8; i++) p[i] = sc[r][i >> 2][i & 3] * b.ks[i >> 2];
    if (partial) {
      const int from = seldom(key0);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int key = from + (i >> 2) * 16 + 4 * g + (i & 3);
        if (key > x.hi[r] || key < x.lo[r] || key > task.last_pos) p[i] = -kInf;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) mx = fmaxf(mx, p[i]);
    if (__ballot(mx > x.m[r] + kSlack)) {
      mx = fmaxf(x.m[r], quad_max(mx));
      const float f = exp2_(x.m[r] - finite_or_0(mx));
      x.m[r] = mx;
      x.l[r] *= f;
#pragma unroll
      for (int j = 0; j < DP / 16; j++) x.o[r][j] *= f;
    }
    const float off = finite_or_0(x.m[r]) - kBias;
    float sum = 0.f;
    f16x8 ph, pl;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float e = exp2_(p[i] - off);
      sum += e;
      ph[i] = (_Float16)(e * vf[i >> 2]);
      if constexpr (WIDE) pl[i] = (_Float16)(e * vf[i >> 2] - (float)ph[i]);
    }
    pr[r] = __builtin_bit_cast(u32x4, ph);
    if constexpr (WIDE) rest[r] = __builtin_bit_cast(u32x4, pl);
    x.l[r] += sum;
  }

#pragma unroll
  for (int w = 0; w < VB / 4; w++) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = b.v[i].v[w];
    u32x4 e[4];
    zip4(v, e);
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int r = 0; r < R; r++) {
        x.o[r][4 * w + j] = mma_dense<false>(e[j], pr[r], x.o[r][4 * w + j]);
        if constexpr (WIDE) x.o[r][4 * w + j] = mma_dense<false>(e[j], rest[r], x.o[r][4 * w + j]);
      }
  }
  if (nan_v) {
    // rare: V holds NaN in a row that not every row of the task sees.  A sum of
    // 0/1 products says which outputs see one: 2^-9 (byte 1) where V is NaN,
    // 1 where the row sees the key.
    u32x4 see[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      f16x8 one;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int key = key0 + (i >> 2) * 16 + 4 * g + (i & 3);
        one[i] = key <= x.hi[r] && key >= x.lo[r] && key <= task.last_pos ? (_Float16)1.0f : (_Float16)0.0f;
      }
      see[r] = __builtin_bit_cast(u32x4, one);
    }
    const int vd = (lane & 15) * VB < a.D ? (lane & 15) * VB : 0;
#pragma unroll
    for (int w = 0; w < VB / 4; w++) {
      uint32_t nan[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int key = key0 + (i >> 2) * 16 + 4 * g + (i & 3);
        const uint32_t v = *reinterpret_cast<const uint32_t*>(b.vp[i >> 2] + (4 * g + (i & 3)) * a.D + vd + 4 * w);
        nan[i] = key >= any_from && key <= task.last_pos ? (((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7 : 0u;
      }
      u32x4 e[4];
      zip4(nan, e);
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int r = 0; r < R; r++) {
          const f32x4 hit = mma_dense<false>(e[j], see[r], (f32x4){0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int i = 0; i < 4; i++)
            if (hit[i] > 0.f) x.o[r][4 * w + j][i] = __builtin_nanf("");
        }
    }
  }
}

// WIDE: the probabilities in two fp16 values, 22 bits, for fp32 outputs.
template <bool BF16, int DP, int R, bool WIDE = false>
struct Few {
  static constexpr bool kBf16 = BF16;
  static constexpr int kWaves = patch::kWaves, kDim = DP, kRows = 16 * R, kStep = patch::kStep;
  // Measured: pieces of at least 8 steps, 4 sequences of 1500 tokens 12.6 us,
  // of 4 steps 15.8, of 16 steps 13.7.  A task's own cost of 16 steps, 48
  // sequences of 200 to 4000 tokens 40.5 us, of 8 steps 42.3, of 2 steps 49.7.
  static constexpr int kMinSteps = 8, kTaskCost = 16;
  static constexpr int kPerCu = R == 1 && DP <= 128 ? 2 : 1;
  static constexpr int kLds = kWaves * kRows * (DP + 4) + kWaves * kRows * 2 + kWaves;

  static __device__ __forceinline__ void run(const Args& a, const Seq& sq, const Task& task, int s, int h, int begin,
                                             int end, const Part& part, float* lds) {
  constexpr int kLd = DP + 4, VB = DP / 16;
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15,
            g = lane >> 4;
  Rows<BF16, DP, R> x;
  const int32_t* table = a.table + s * a.table_row;
  int step = begin + wave;
  if (step < end) {
    Pages pages = load_pages(a, table, h, step, task.last_pos);
    start_rows(a, sq, task, h, x);
    Bytes<DP> cur = load_step<DP>(a, pages, 0, h, step, task.last_pos);
    for (int i = 1; step < end; i++, step += kWaves) {
      Bytes<DP> next = cur;
      if (step + kWaves < end) {  // the next step's bytes are on their way while this one's are used
        if ((i & 63) == 0) pages = load_pages(a, table, h, step + kWaves, task.last_pos);
        next = load_step<DP>(a, pages, i & 63, h, step + kWaves, task.last_pos);
      }
      do_step<BF16, DP, R, WIDE>(a, task, step, cur, x);
      cur = next;
    }
  } else {
    start_rows(a, sq, task, h, x);
  }

  // ---- join the waves through LDS ----
  float* lml = lds + kWaves * kRows * kLd;  // [wave][row][m, l], then [wave] vref
#pragma unroll
  for (int r = 0; r < R; r++) {
    x.l[r] = quad_sum(x.l[r]);  // the lanes of a row hold parts of its sum
    float* at = lds + (wave * kRows + r * 16 + n) * kLd + 4 * g * VB;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < VB; j += 4)
        *reinterpret_cast<f32x4*>(at + i * VB + j) =
            (f32x4){x.o[r][j][i], x.o[r][j + 1][i], x.o[r][j + 2][i], x.o[r][j + 3][i]};
    if (g == 0) {
      lml[(wave * kRows + r * 16 + n) * 2] = x.m[r];
      lml[(wave * kRows + r * 16 + n) * 2 + 1] = x.l[r];
    }
  }
  if (lane == 0) lml[kWaves * kRows * 2 + wave] = x.vref;
  __syncthreads();

  const int chunks = a.D / 8;
  float* slot = a.parts + part.slot((int)blockIdx.x - part.w0) * (kRows * (DP + 2));
  const __amdgpu_buffer_rsrc_t rs = rsrc(slot, kRows * (DP + 2) * 4);
  for (int e = tid; e < (task.r1 - task.r0) * chunks; e += kThreads) {
    const int row = e / chunks, d = (e - row * chunks) * 8;
    float mx = -kInf;
#pragma unroll
    for (int v = 0; v < kWaves; v++) mx = fmaxf(mx, lml[(v * kRows + row) * 2]);
    const float mu = finite_or_0(mx);
    float sum = 0.f, f[kWaves], acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kWaves; v++) {
      f[v] = exp2_(lml[(v * kRows + row) * 2] - mu);
      sum += f[v] * lml[(v * kRows + row) * 2 + 1];
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int v = 0; v < kWaves; v++) {
      const float fo = f[v] * inv * lml[kWaves * kRows * 2 + v];
      const float* p = lds + (v * kRows + row) * kLd + d;
#pragma unroll
      for (int i = 0; i < 8; i++) acc[i] += fo * p[i];
    }
    if (part.count == 1) {
      store8<BF16>(a, out_at(a, sq, h, task.r0 + row, d), acc);
      if (a.lse && d == 0) store_lse(a, sq, h, task.r0 + row, lse_of(mx, sum));
    } else {
      const int at = (row * DP + d) * 4;
      const f32x4 lo = {acc[0], acc[1], acc[2], acc[3]}, hi = {acc[4], acc[5], acc[6], acc[7]};
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, lo), rs, at, 0, kCoherent);
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, hi), rs, at + 16, 0, kCoherent);
      if (d == 0) {
        const u32x2 ml = {__float_as_uint(mx), __float_as_uint(sum)};
        __builtin_amdgcn_raw_buffer_store_b64(ml, rs, (kRows * DP + 2 * row) * 4, 0, kCoherent);
      }
    }
  }
}
};

// Many rows a sequence on average: attention_chunk.hip, whose workgroup reads a
// key once for 128 rows.  8 sequences of 4096 keys, 32 query and 8 cache heads
// of 128, this file's against that one's: 64 rows 41 us to 51, 96 rows 64 to
// 57, 256 rows 115 to 85.
bool many_rows(int64_t T, int64_t S, int64_t group, int64_t dim) { return dim <= 128 && T * group > 64 * S; }

// Sixteens of rows of a task, by the rows a sequence has on average.  As above,
// one against two: 4 rows 23.1 us to 25.6, 16 rows 25.4 to 26.9, 24 rows 32.9
// to 29.6, 64 rows 56 to 41.
int tile_rows(int64_t T, int64_t S, int64_t group, int64_t dim) { return T * group <= 16 * S || dim > 128 ? 1 : 2; }

template <bool BF16, bool WIDE>
hipError_t by_shape(Args& a, void* ws, uint64_t ws_bytes, hipStream_t s) {
  if (many_rows(a.T, a.S, a.group, a.D)) return launch_attention_chunk(BF16, a, ws, ws_bytes, s);
  const int R = tile_rows(a.T, a.S, a.group, a.D);
  if (a.D <= 64)
    return R == 1 ? go<Few<BF16, 64, 1, WIDE>>(a, ws, ws_bytes, s) : go<Few<BF16, 64, 2, WIDE>>(a, ws, ws_bytes, s);
  if (a.D <= 128)
    return R == 1 ? go<Few<BF16, 128, 1, WIDE>>(a, ws, ws_bytes, s) : go<Few<BF16, 128, 2, WIDE>>(a, ws, ws_bytes, s);
  return go<Few<BF16, 256, 1, WIDE>>(a, ws, ws_bytes, s);
}

}  // namespace

namespace attn {
// A value of this launch for the flags: a counter mixed with a random salt of
// the process (splitmix64's finaliser), never 0.
uint64_t launch_token() {
  static const uint64_t salt = []() -> uint64_t {
    try {
      std::random_device rd;
      return ((uint64_t)rd() << 32) ^ (uint64_t)rd();
    } catch (...) {  // no source of entropy
      return (uint64_t)std::chrono::steady_clock::now().time_since_epoch().count();
    }
  }();
  static std::atomic<uint64_t> counter{1};
  uint64_t z = salt + 0x9e3779b97f4a7c15ull * counter.fetch_add(1, std::memory_order_relaxed);
  z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
  z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
  z ^= z >> 31;
  return z == 0 ? 1 : z;
}

}  // namespace attn

uint64_t attention_workspace_bytes(int64_t T, int64_t S, int64_t heads, int64_t kv_heads, int64_t dim) {
  if (many_rows(T, S, heads / kv_heads, dim)) return attention_chunk_workspace_bytes(T, S, heads / kv_heads, dim);
  const int R = tile_rows(T, S, heads / kv_heads, dim);
  if (dim <= 64) return R == 1 ? workspace_bytes<Few<true, 64, 1>>() : workspace_bytes<Few<true, 64, 2>>();
  if (dim <= 128) return R == 1 ? workspace_bytes<Few<true, 128, 1>>() : workspace_bytes<Few<true, 128, 2>>();
  return workspace_bytes<Few<true, 256, 1>>();
}

hipError_t launch_attention(const patch_attention_args& p, const patch_kv_cache& c, void* ws, uint64_t ws_bytes,
                            hipStream_t s) {
  Args a;
  a.q = reinterpret_cast<const uint16_t*>(p.q_dev);
  a.out = p.out_dev;
  a.lse = p.lse_dev;
  a.table = p.page_table_dev;
  a.lens = p.kv_lens_dev;
  a.cu = p.cu_new_dev;
  a.k = reinterpret_cast<const uint8_t*>(c.k_dev);
  a.v = reinterpret_cast<const uint8_t*>(c.v_dev);
  a.ks = c.k_scale_dev;
  a.vs = c.v_scale_dev;
  a.parts = nullptr;
  a.flags = nullptr;
  a.token = 0;
  a.q_token = p.q_token;
  a.q_head = p.q_head;
  a.o_token = p.out_token;
  a.o_head = p.out_head;
  a.table_row = p.page_table_row;
  a.T = (int)p.T;
  a.S = (int)p.S;
  a.heads = (int)p.heads;
  a.kv_heads = (int)c.kv_heads;
  a.group = (int)(p.heads / c.kv_heads);
  a.D = (int)c.dim;
  a.B = (int)c.page;
  a.shift = 31 - __builtin_clz((unsigned)c.page);
  a.pages = (int)c.pages;
  a.max_pages = (int)p.max_pages;
  a.window = (int)std::min<int64_t>(p.window, 0x3fffffff);
  a.scale = fabsf((float)p.scale * kLog2e);
  a.q_flip = p.scale < 0 ? 0x80008000u : 0u;
  a.q_wide = ((p.q_token | p.q_head) & 7) == 0 && ((uintptr_t)p.q_dev & 15) == 0;
  a.o_wide = ((p.out_token | p.out_head) & 7) == 0 && ((uintptr_t)p.out_dev & 15) == 0;
  a.out_f32 = p.out_dtype == PATCH_F32;
  if (a.out_f32)
    return p.dtype == PATCH_BF16 ? by_shape<true, true>(a, ws, ws_bytes, s) : by_shape<false, true>(a, ws, ws_bytes, s);
  return p.dtype == PATCH_BF16 ? by_shape<true, false>(a, ws, ws_bytes, s) : by_shape<false, false>(a, ws, ws_bytes, s);
}

}  // namespace patch
