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
#include <algorithm>
#include <atomic>
#include <random>

#include "device_common.h"
#include "layer_common.h"

namespace patch {
namespace {

#ifndef KW
#define KW 4
#endif
#ifndef KM
#define KM 8
#endif
constexpr int kWaves = KW;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;       // keys of a step
#ifndef KC
#define KC 8
#endif
constexpr int kTaskCost = KC;   // of a task beside its steps, in steps
constexpr int kMinSteps = KM;    // steps of a workgroup, at least
constexpr float kBias = 14.0f;  // probabilities are 2^(s - m + kBias)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();

struct Args {
  const uint16_t* q;
  void* out;
  float* lse;
  const int32_t *table, *lens, *cu;
  const uint8_t *k, *v;
  const float *ks, *vs;
  float* parts;     // [worker][2][rows][DP + 2]
  uint64_t* flags;  // [worker][2]
  uint64_t token;
  int64_t q_token, q_head, o_token, o_head, table_row;
  int T, S, heads, kv_heads, group, D, B, shift, pages, max_pages, window;
  float scale;  // with log2(e)
  bool q_wide, o_wide, out_f32;
};

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float finite_or_0(float m) { return m == -kInf ? 0.f : m; }

// Two (lo or hi half of a word) e4m3 bytes as two 16-bit values.
template <bool BF16, bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  if constexpr (BF16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
}
template <bool BF16>
__device__ __forceinline__ u32x4 widen8(uint32_t lo, uint32_t hi) {
  return (u32x4){widen2<BF16, false>(lo), widen2<BF16, true>(lo), widen2<BF16, false>(hi), widen2<BF16, true>(hi)};
}

// Four neighbouring elements of 8 keys (a word a key) as four A operands of
// V^T, a byte of each key.
__device__ __forceinline__ void zip4(const uint32_t (&v)[8], u32x4 (&e)[4]) {
#pragma unroll
  for (int p = 0; p < 4; p++) {
    const uint32_t z0 = __builtin_amdgcn_perm(v[2 * p + 1], v[2 * p], 0x05010400u);
    const uint32_t z1 = __builtin_amdgcn_perm(v[2 * p + 1], v[2 * p], 0x07030602u);
    e[0][p] = widen2<false, false>(z0);
    e[1][p] = widen2<false, true>(z0);
    e[2][p] = widen2<false, false>(z1);
    e[3][p] = widen2<false, true>(z1);
  }
}

// A sequence's newest tokens c0 .. c0 + n - 1, the position of the first, and
// whether its length does not fit its page table.
struct Seq {
  int c0, n, past;
  bool bad;
};
__device__ __forceinline__ Seq seq_of(const Args& a, int s) {
  Seq q;
  const int e = min(a.cu[s + 1], a.T), len = a.lens[s];
  q.c0 = max(a.cu[s], 0);
  q.n = max(e - q.c0, 0);
  q.past = max(len, -0x40000000) - q.n;
  q.bad = len > a.max_pages << a.shift;
  return q;
}

// The rows r0 .. r1 - 1 of a task and the steps of the keys they see.
struct Task {
  int r0, r1, first_pos, last_pos, begin, end;
  bool fill;  // nothing to attend to: rows are filled
};
template <int ROWS>
__device__ __forceinline__ Task task_of(const Args& a, const Seq& sq, int rt) {
  Task t;
  t.r0 = rt * ROWS;
  t.r1 = min(t.r0 + ROWS, sq.n * a.group);
  t.first_pos = sq.past + t.r0 / a.group;
  t.last_pos = sq.past + (t.r1 - 1) / a.group;
  t.fill = sq.bad || t.last_pos < 0;
  const int from = a.window > 0 ? max(t.first_pos - a.window + 1, 0) : 0;
  t.begin = t.fill ? 0 : from / kStep;
  t.end = t.fill ? 1 : t.last_pos / kStep + 1;
  return t;
}
// A head's cost on the line: its tasks' steps, and kTaskCost for each task.
template <int ROWS>
__device__ __forceinline__ int cost_of(const Args& a, const Seq& sq) {
  const int tiles = (sq.n * a.group + ROWS - 1) / ROWS;
  int n = 0;
  for (int i = 0; i < tiles; i++) {
    const Task t = task_of<ROWS>(a, sq, i);
    n += t.end - t.begin + kTaskCost;
  }
  return n;
}
// The pieces a head's tasks make at kMinSteps or more steps each.
__device__ __forceinline__ int pieces_of(const Task& t) { return (t.end - t.begin + kMinSteps - 1) / kMinSteps; }
template <int ROWS>
__device__ __forceinline__ int pieces_of(const Args& a, const Seq& sq) {
  const int tiles = (sq.n * a.group + ROWS - 1) / ROWS;
  int n = 0;
  for (int i = 0; i < tiles; i++) n += pieces_of(task_of<ROWS>(a, sq, i));
  return n;
}

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
__device__ __forceinline__ int lane_of(int v, int i) { return __builtin_amdgcn_readlane(v, i); }
__device__ __forceinline__ float lane_of(float v, int i) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), i));
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
    const uint8_t* kp = a.k + at + n * a.D;
    // Behind element D - 1 the same key's first ones: q is zero there (and a
    // NaN among them would make the score NaN in any case).
#pragma unroll
    for (int j = 0; j < DP / 64; j++) b.k[t][j] = ld16(kp + (j * 64 + g * 16 < a.D ? j * 64 + g * 16 : 0));
  }
  const int vd = n * VB < a.D ? n * VB : 0;  // likewise; those outputs are not stored
#pragma unroll
  for (int i8 = 0; i8 < 8; i8++)
    b.v[i8] = *reinterpret_cast<const Vec<uint32_t, VB / 4>*>(b.vp[i8 >> 2] + (4 * g + (i8 & 3)) * a.D + vd);
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
      x.q[r][j] = v;
    }
#pragma unroll
    for (int j = 0; j < DP / 16; j++) x.o[r][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    x.m[r] = -kInf;
    x.l[r] = 0.f;
  }
  x.vref = 0.f;
}

template <bool BF16, int DP, int R>
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
    // V rows that no row of the task sees hold anything at all: take zeros.  A
    // NaN in a row that some see must not reach the others through 0 * NaN: it
    // is taken out here and put back below, row by row.
    bool has = false;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int key = key0 + (i >> 2) * 16 + 4 * g + (i & 3);
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

  float ratio = 1.0f;
  const float vmax = fmaxf(fabsf(b.vs[0]), fabsf(b.vs[1]));
  if (vmax > x.vref) {
    ratio = x.vref / vmax;
    x.vref = vmax;
  }
  const float inv = x.vref > 0.f ? 1.0f / x.vref : 0.f;
  const float vf[2] = {b.vs[0] * inv, b.vs[1] * inv};
  u32x4 pr[R];
#pragma unroll
  for (int r = 0; r < R; r++) {
    float p[8];
    float mx = x.m[r];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      p[i] = sc[r][i >> 2][i & 3] * b.ks[i >> 2];
      if (partial) {
        const int key = key0 + (i >> 2) * 16 + 4 * g + (i & 3);
        if (key > x.hi[r] || key < x.lo[r] || key > task.last_pos) p[i] = -kInf;
      }
      mx = fmaxf(mx, p[i]);
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mu = finite_or_0(mx);
    const float f = exp2_(x.m[r] - mu);
    x.m[r] = mx;
    float sum = 0.f;
    f16x8 ph;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float e = exp2_(p[i] - (mu - kBias));
      sum += e;
      ph[i] = (_Float16)(e * vf[i >> 2]);
    }
    pr[r] = __builtin_bit_cast(u32x4, ph);
    x.l[r] = x.l[r] * f + sum;
    if (__ballot(f * ratio != 1.0f)) {
#pragma unroll
      for (int j = 0; j < DP / 16; j++) x.o[r][j] *= f * ratio;
    }
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
      for (int r = 0; r < R; r++) x.o[r][4 * w + j] = mma_dense<false>(e[j], pr[r], x.o[r][4 * w + j]);
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

// Eight neighbouring outputs.
template <bool BF16>
__device__ __forceinline__ void store8(const Args& a, int64_t at, const float (&v)[8]) {
  if (a.out_f32) {
    float* op = reinterpret_cast<float*>(a.out) + at;
    if (a.o_wide) {
      *reinterpret_cast<f32x4*>(op) = (f32x4){v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(op + 4) = (f32x4){v[4], v[5], v[6], v[7]};
    } else {
      for (int i = 0; i < 8; i++) op[i] = v[i];
    }
  } else {
    typedef std::conditional_t<BF16, __bf16, _Float16> T;
    Vec<T, 8> o;
#pragma unroll
    for (int i = 0; i < 8; i++) o.v[i] = (T)v[i];
    T* op = reinterpret_cast<T*>(a.out) + at;
    if (a.o_wide) {
      *reinterpret_cast<Vec<T, 8>*>(op) = o;
    } else {
      for (int i = 0; i < 8; i++) op[i] = o.v[i];
    }
  }
}
__device__ __forceinline__ int64_t out_at(const Args& a, const Seq& sq, int h, int row, int d) {
  const int tok = row / a.group, head = h * a.group + row - tok * a.group;
  return (int64_t)(sq.c0 + tok) * a.o_token + (int64_t)head * a.o_head + d;
}
__device__ __forceinline__ void store_lse(const Args& a, const Seq& sq, int h, int row, float v) {
  const int tok = row / a.group, head = h * a.group + row - tok * a.group;
  a.lse[(int64_t)(sq.c0 + tok) * a.heads + head] = v;
}
__device__ __forceinline__ float lse_of(float m, float l) { return (m + __log2f(l) - kBias) * kLn2; }

template <bool BF16>
__device__ __forceinline__ void fill_rows(const Args& a, const Seq& sq, const Task& t, int h) {
  const float o = sq.bad ? __builtin_nanf("") : 0.f, lse = sq.bad ? __builtin_nanf("") : -kInf;
  const int chunks = a.D / 8;
  for (int e = threadIdx.x; e < (t.r1 - t.r0) * chunks; e += kThreads) {
    const int row = t.r0 + e / chunks, d = e % chunks * 8;
    store8<BF16>(a, out_at(a, sq, h, row, d), {o, o, o, o, o, o, o, o});
    if (a.lse && d == 0) store_lse(a, sq, h, row, lse);
  }
}

constexpr int kCoherent = 16;  // cache policy bits of a buffer access: sc1
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

// The steps begin .. end - 1 of a task, by the whole workgroup.  part < 0:
// they are all of its steps, and the rows are stored.  Else o / l, m and l go
// to slot `part` of the workspace.
template <bool BF16, int DP, int R>
__device__ __forceinline__ void run_steps(const Args& a, const Seq& sq, const Task& task, int s, int h, int begin,
                                          int end, int part, float* lds) {
  constexpr int kRows = 16 * R, kLd = DP + 4, VB = DP / 16;
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
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
      do_step<BF16, DP, R>(a, task, step, cur, x);
      cur = next;
    }
  } else {
    start_rows(a, sq, task, h, x);
  }

  // ---- join the waves through LDS ----
  float* lml = lds + kWaves * kRows * kLd;  // [wave][row][m, l], then [wave] vref
#pragma unroll
  for (int r = 0; r < R; r++) {
    // the lanes of a row hold parts of its sum
    x.l[r] += __shfl_xor(x.l[r], 16);
    x.l[r] += __shfl_xor(x.l[r], 32);
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
  float* slot = a.parts + (int64_t)part * (kRows * (DP + 2));
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
    if (part < 0) {
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

// Join the parts of a task: slot 1 of worker w0, then slot 0 of the next.
template <bool BF16, int DP, int R>
__device__ __forceinline__ void join_parts(const Args& a, const Seq& sq, const Task& task, int h, int w0, int count) {
  constexpr int kRows = 16 * R, kSlot = kRows * (DP + 2);
  const int chunks = a.D / 8;
  for (int e = threadIdx.x; e < (task.r1 - task.r0) * chunks; e += kThreads) {
    const int row = e / chunks, d = (e - row * chunks) * 8;
    float mx = -kInf, sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = 0; p < count; p++) {
      const int64_t slot = 2 * ((int64_t)w0 + p) + (p == 0);
      const __amdgpu_buffer_rsrc_t rs = rsrc(a.parts + slot * kSlot, kSlot * 4);
      const int at = (row * DP + d) * 4;
      const u32x2 ml = __builtin_amdgcn_raw_buffer_load_b64(rs, (kRows * DP + 2 * row) * 4, 0, kCoherent);
      const f32x4 lo = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, kCoherent));
      const f32x4 hi = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at + 16, 0, kCoherent));
      const float m = __uint_as_float(ml[0]), l = __uint_as_float(ml[1]);
      const float mn = fmaxf(mx, m), mu = finite_or_0(mn);
      const float f = exp2_(mx - mu), w = exp2_(m - mu) * l;
      mx = mn;
      sum = sum * f + w;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        acc[i] = acc[i] * f + w * lo[i];
        acc[4 + i] = acc[4 + i] * f + w * hi[i];
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < 8; i++) acc[i] *= inv;
    store8<BF16>(a, out_at(a, sq, h, task.r0 + row, d), acc);
    if (a.lse && d == 0) store_lse(a, sq, h, task.r0 + row, lse_of(mx, sum));
  }
}

template <int DP, int R>
constexpr int lds_floats() {
  return kWaves * 16 * R * (DP + 4) + kWaves * 16 * R * 2 + kWaves;
}

// A sequence, where it begins and ends on a line.
struct Place {
  int s, from, to;
};

// A line over up to 64 sequences, one a lane; every wave has its own.
struct LaneLine {
  int from, to, total;
  __device__ __forceinline__ explicit LaneLine(int n) {
    const int lane = (int)threadIdx.x & 63;
    to = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(to, d);
      if (lane >= d) to += v;
    }
    from = to - n;
    total = lane_of(to, 63);
  }
  __device__ __forceinline__ Place find(int u) const {
    const int s = __builtin_ctzll(__ballot(to > u));  // the first that ends behind u
    return Place{s, lane_of(from, s), lane_of(to, s)};
  }
};

// For more sequences: a prefix sum in LDS, by the whole workgroup.
struct LdsLine {
  int* line;  // [S + 1]: where sequence s begins
  int total, S;
  template <typename F>
  __device__ __forceinline__ LdsLine(int n_seqs, int* l, int* wave_sum, F cost) : line(l), total(0), S(n_seqs) {
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int each = (S + kThreads - 1) / kThreads, s1 = min((tid + 1) * each, S);
    int mine = 0;
    for (int s = tid * each; s < s1; s++) {
      line[s] = cost(s);
      mine += line[s];
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 63) wave_sum[wave] = upto;
    __syncthreads();
    int at = upto - mine;
    for (int w = 0; w < kWaves; w++) {
      if (w < wave) at += wave_sum[w];
      total += wave_sum[w];
    }
    for (int s = tid * each; s < s1; s++) {
      const int n = line[s];
      line[s] = at;
      at += n;
    }
    if (tid == 0) line[S] = total;
    __syncthreads();
  }
  __device__ __forceinline__ Place find(int u) const {
    // the last that begins at or before u: of equal ones the one with steps
    const int s = find_last(S, [&](int i) { return line[i] <= u; });
    return Place{s, line[s], line[s + 1]};
  }
};

// Steps begin .. end - 1 of a task by this workgroup, one of the task's
// `count` parts, which the workgroups w0 .. w0 + count - 1 have: part 0 in
// slot 1 of its workgroup, the others in slot 0.
template <bool BF16, int DP, int R>
__device__ __forceinline__ void run_piece(const Args& a, const Seq& sq, const Task& task, int s, int h, int begin,
                                          int end, int w0, int count, float* lds, int* joined) {
  if (task.fill) {
    fill_rows<BF16>(a, sq, task, h);
    return;
  }
  const int lane = (int)threadIdx.x & 63;
  const int mine = count == 1 ? -1 : 2 * (int)blockIdx.x + ((int)blockIdx.x == w0 ? 1 : 0);
  run_steps<BF16, DP, R>(a, sq, task, s, h, begin, end, mine, lds);
  if (count > 1) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's share of the part has arrived
    __syncthreads();
    if (threadIdx.x < 64) {
      if (lane == 0) {
        const uint64_t old =
            __hip_atomic_exchange(a.flags + mine, a.token, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("" ::"v"(old));
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // and its flag, before the others' are read
      bool all = true;
      for (int p = lane; p < count; p += 64)
        all &= __hip_atomic_load(a.flags + 2 * (w0 + p) + (p == 0), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               a.token;
      const bool done = __ballot(!all) == 0;
      if (lane == 0) *joined = done;
      if (done)
        for (int p = lane; p < count; p += 64)
          __hip_atomic_store(a.flags + 2 * (w0 + p) + (p == 0), (uint64_t)0, __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (*joined) join_parts<BF16, DP, R>(a, sq, task, h, w0, count);
  }
}

// All work on one line (see the top).  Where there are fewer pieces of
// kMinSteps steps than workgroups, each task is cut evenly and every piece
// has a workgroup.  Else workgroup w takes the w-th equal piece of the line,
// on which a task begins with kTaskCost places that stand for what it costs
// beside its steps: about what that many steps take.
template <bool BF16, int DP, int R, bool MANY>
__global__ __launch_bounds__(kThreads, (R == 1 && DP <= 128 ? 8 : 4) / kWaves) void k_attention_line(Args a) {
  extern __shared__ __align__(16) float lds[];
  __shared__ int wave_sum[kWaves];
  __shared__ int joined;
  constexpr int kRows = 16 * R;
  Seq mine{0, 0, 0, false};  // of this lane's sequence
  if constexpr (!MANY) {
    const int lane = (int)threadIdx.x & 63;
    if (lane < a.S) mine = seq_of(a, lane);
    const LaneLine pieces(lane < a.S ? pieces_of<kRows>(a, mine) * a.kv_heads : 0);
    if (pieces.total <= (int)gridDim.x) {
      if ((int)blockIdx.x >= pieces.total) return;
      const Place pl = pieces.find((int)blockIdx.x);
      const Seq sq{lane_of(mine.c0, pl.s), lane_of(mine.n, pl.s), lane_of(mine.past, pl.s), lane_of((int)mine.bad, pl.s) != 0};
      const int per_head = (pl.to - pl.from) / a.kv_heads, h = ((int)blockIdx.x - pl.from) / per_head;
      int w0 = pl.from + h * per_head, rt = 0;
      Task task = task_of<kRows>(a, sq, 0);
      int count = pieces_of(task);
      while (w0 + count <= (int)blockIdx.x) {
        w0 += count;
        task = task_of<kRows>(a, sq, ++rt);
        count = pieces_of(task);
      }
      const int i = (int)blockIdx.x - w0, steps = task.end - task.begin;
      const int each = steps / count, more = steps - each * count;  // the first `more` pieces have one step more
      const int begin = task.begin + i * each + min(i, more);
      run_piece<BF16, DP, R>(a, sq, task, pl.s, h, begin, begin + each + (i < more ? 1 : 0), w0, count, lds, &joined);
      return;
    }
  }
  const auto line = [&] {
    if constexpr (MANY)
      return LdsLine(a.S, reinterpret_cast<int*>(lds + lds_floats<DP, R>()), wave_sum,
                     [&](int s) { return cost_of<kRows>(a, seq_of(a, s)) * a.kv_heads; });
    else
      return LaneLine(((int)threadIdx.x & 63) < a.S ? cost_of<kRows>(a, mine) * a.kv_heads : 0);
  }();
  const int per = (line.total + (int)gridDim.x - 1) / (int)gridDim.x;
  int u = per * (int)blockIdx.x;
  const int u_end = min(u + per, line.total);
  while (u < u_end) {
    const Place pl = line.find(u);
    const Seq sq = MANY ? seq_of(a, pl.s)
                        : Seq{lane_of(mine.c0, pl.s), lane_of(mine.n, pl.s), lane_of(mine.past, pl.s),
                              lane_of((int)mine.bad, pl.s) != 0};
    const int per_head = (pl.to - pl.from) / a.kv_heads, h = (u - pl.from) / per_head;
    int at = pl.from + h * per_head, rt = 0;  // where the task begins on the line
    Task task = task_of<kRows>(a, sq, 0);
    while (at + (task.end - task.begin) + kTaskCost <= u) {
      at += task.end - task.begin + kTaskCost;
      task = task_of<kRows>(a, sq, ++rt);
    }
    at += kTaskCost;  // its first step
    const int task_end = at + (task.end - task.begin), from = max(u, at), to = min(u_end, task_end);
    if (from < to) {
      const int w0 = at / per;
      run_piece<BF16, DP, R>(a, sq, task, pl.s, h, task.begin + from - at, task.begin + to - at, w0,
                             (task_end - 1) / per - w0 + 1, lds, &joined);
      __syncthreads();  // LDS is used again
    }
    u = task_end;
  }
}

// Without a workspace: a workgroup a task.  Sequence s has the tasks
// floor(cu[s] group / rows) + s up to the same of s + 1 for each head, at
// least as many as its rows need.
template <bool BF16, int DP, int R>
__global__ __launch_bounds__(kThreads) void k_attention_task(Args a) {
  extern __shared__ __align__(16) float lds[];
  constexpr int kRows = 16 * R;
  const int h = (int)(blockIdx.x % (uint32_t)a.kv_heads);
  const int64_t slot = blockIdx.x / (uint32_t)a.kv_heads;
  const int s = find_last(a.S, [&](int i) { return (int64_t)a.cu[i] * a.group / kRows + i <= slot; });
  const int64_t first = (int64_t)a.cu[s] * a.group / kRows + s;
  const Seq sq = seq_of(a, s);
  if (slot < first || (slot - first) * kRows >= (int64_t)sq.n * a.group) return;
  const Task task = task_of<kRows>(a, sq, (int)(slot - first));
  if (task.fill)
    fill_rows<BF16>(a, sq, task, h);
  else
    run_steps<BF16, DP, R>(a, sq, task, s, h, task.begin, task.end, -1, lds);
}

// A value of this launch for the flags: a counter mixed with a random salt of
// the process (splitmix64's finaliser), never 0.
uint64_t launch_token() {
  static const uint64_t salt = [] {
    std::random_device rd;
    return ((uint64_t)rd() << 32) ^ (uint64_t)rd();
  }();
  static std::atomic<uint64_t> counter{1};
  uint64_t z = salt + 0x9e3779b97f4a7c15ull * counter.fetch_add(1, std::memory_order_relaxed);
  z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
  z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
  z ^= z >> 31;
  return z == 0 ? 1 : z;
}

// Rows of a task in sixteens: by the rows a sequence has on average.
int tile_rows(int64_t T, int64_t S, int64_t group, int64_t dim) {
  const int64_t rows = T * group;
  return rows <= 16 * S || dim > 128 ? 1 : 2;
}
int workers_of(int R, int DP) { return cu_count() * (R == 1 && DP <= 128 ? 8 : 4) / kWaves; }
constexpr int padded_dim(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
uint64_t slot_bytes(int R, int DP) { return (uint64_t)(16 * R * (DP + 2)) * 4; }

hipError_t launch(const void* fn, int64_t blocks, size_t lds, Args& a, hipStream_t s) {
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  if (lds > 65536) {
    hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  void* args[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(kThreads), args, lds, s);
}

template <bool BF16, int DP, int R>
hipError_t go(Args& a, void* ws, uint64_t ws_bytes, hipStream_t s) {
  const uint64_t workers = (uint64_t)workers_of(R, DP);
  const size_t lds = sizeof(float) * (size_t)lds_floats<DP, R>();
  // the line's places are 32-bit numbers
  const int64_t tasks = ((int64_t)a.T * a.group / (16 * R) + a.S) * a.kv_heads;
  const int64_t steps = (((int64_t)a.max_pages << a.shift) + kStep - 1) / kStep + 1 + kTaskCost;
  const bool fits = tasks < 0x40000000 && tasks * steps < 0x40000000;
  if (fits && ws && ws_bytes >= workers * 2 * (slot_bytes(R, DP) + 8)) {
    a.flags = reinterpret_cast<uint64_t*>(ws);
    a.parts = reinterpret_cast<float*>(a.flags + 2 * workers);
    a.token = launch_token();
    return a.S > 64 ? launch(reinterpret_cast<const void*>(k_attention_line<BF16, DP, R, true>), (int64_t)workers,
                             lds + 4 * (size_t)(a.S + 1), a, s)
                    : launch(reinterpret_cast<const void*>(k_attention_line<BF16, DP, R, false>), (int64_t)workers, lds,
                             a, s);
  }
  return launch(reinterpret_cast<const void*>(k_attention_task<BF16, DP, R>),
                tasks, lds, a, s);
}

template <bool BF16>
hipError_t by_shape(Args& a, void* ws, uint64_t ws_bytes, hipStream_t s) {
  const int R = tile_rows(a.T, a.S, a.group, a.D);
  if (a.D <= 64) return R == 1 ? go<BF16, 64, 1>(a, ws, ws_bytes, s) : go<BF16, 64, 2>(a, ws, ws_bytes, s);
  if (a.D <= 128) return R == 1 ? go<BF16, 128, 1>(a, ws, ws_bytes, s) : go<BF16, 128, 2>(a, ws, ws_bytes, s);
  return go<BF16, 256, 1>(a, ws, ws_bytes, s);
}

}  // namespace

uint64_t attention_workspace_bytes(int64_t T, int64_t S, int64_t heads, int64_t kv_heads, int64_t dim) {
  const int R = tile_rows(T, S, heads / kv_heads, dim), DP = padded_dim(dim);
  return (uint64_t)workers_of(R, DP) * 2 * (slot_bytes(R, DP) + 8);
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
  a.scale = (float)p.scale * kLog2e;
  a.q_wide = ((p.q_token | p.q_head) & 7) == 0 && ((uintptr_t)p.q_dev & 15) == 0;
  a.o_wide = ((p.out_token | p.out_head) & 7) == 0 && ((uintptr_t)p.out_dev & 15) == 0;
  a.out_f32 = p.out_dtype == PATCH_F32;
  return p.dtype == PATCH_BF16 ? by_shape<true>(a, ws, ws_bytes, s) : by_shape<false>(a, ws, ws_bytes, s);
}

}  // namespace patch
