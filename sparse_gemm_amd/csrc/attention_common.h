// attention_common.h -- what the attention kernels share: arguments, tasks,
// how work is given to workgroups and parts of a task are joined, stores.
//
// A kernel's body says how a workgroup attends to a range of keys for the
// rows of one task:
//   kBf16, kWaves (of a workgroup), kDim (elements of a head, padded), kRows (of
//   a task), kStep (keys of a step), kMinSteps (of a workgroup, at least),
//   kTaskCost (what a task costs beside its steps, in steps), kPerCu
//   (workgroups a CU), kLds (its LDS, floats),
//   run(a, sq, task, s, h, begin, end, part, lds): the steps begin .. end - 1.
//   Of a task in one part the rows are stored, else o / l, m and l go to this
//   workgroup's slot of the workspace.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "layer_common.h"

namespace patch {
namespace attn {

// Probabilities are 2^(s - m + kBias), m being within kSlack of the running
// maximum: sums and outputs are only scaled anew when it grows by more.  2^14
// at most, and 2^-20 of the maximum still in fp16's normal range.
constexpr float kBias = 6.0f, kSlack = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();

template <class Body>
constexpr int threads_of = 64 * Body::kWaves;

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
  uint32_t q_flip;  // sign bits: of a negative scale, which the rows of q take
  bool q_wide, o_wide, out_f32;
};

__device__ __forceinline__ int lane_of(int v, int i) { return __builtin_amdgcn_readlane(v, i); }
__device__ __forceinline__ float lane_of(float v, int i) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), i));
}

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

// A value for use in a block that seldom runs: what is computed from it stays
// in the block (the compiler would rather compute it every time and select).
__device__ __forceinline__ int seldom(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The largest of a row's four lanes (16 apart), and their sum.  A swap of two
// copies' rows of 16 (halves of 32) leaves each lane both values.
__device__ __forceinline__ void swapped(float x, float& a, float& b, bool by32) {
  const uint32_t u = __float_as_uint(x);
  const auto r = by32 ? __builtin_amdgcn_permlane32_swap(u, u, false, false)
                      : __builtin_amdgcn_permlane16_swap(u, u, false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ float quad_max(float x) {
  float a, b;
  swapped(x, a, b, false);
  swapped(fmaxf(a, b), a, b, true);
  return fmaxf(a, b);
}
__device__ __forceinline__ float quad_sum(float x) {
  float a, b;
  swapped(x, a, b, false);
  swapped(a + b, a, b, true);
  return a + b;
}

// Four neighbouring elements of two keys (a word each) as pairs: a word of
// each element's two.
__device__ __forceinline__ void zip2(uint32_t k0, uint32_t k1, uint32_t& e0, uint32_t& e1, uint32_t& e2, uint32_t& e3) {
  const uint32_t z0 = __builtin_amdgcn_perm(k1, k0, 0x05010400u), z1 = __builtin_amdgcn_perm(k1, k0, 0x07030602u);
  e0 = widen2<false, false>(z0);
  e1 = widen2<false, true>(z0);
  e2 = widen2<false, false>(z1);
  e3 = widen2<false, true>(z1);
}
// Four neighbouring elements of 8 keys as four A operands of V^T.
__device__ __forceinline__ void zip4(const uint32_t (&v)[8], u32x4 (&e)[4]) {
#pragma unroll
  for (int p = 0; p < 4; p++) {
    uint32_t w0, w1, w2, w3;
    zip2(v[2 * p], v[2 * p + 1], w0, w1, w2, w3);
    e[0][p] = w0;
    e[1][p] = w1;
    e[2][p] = w2;
    e[3][p] = w3;
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
  const int e = max(min(a.cu[s + 1], a.T), 0), len = a.lens[s];
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
template <class Body>
__device__ __forceinline__ Task task_of(const Args& a, const Seq& sq, int rt) {
  Task t;
  t.r0 = rt * Body::kRows;
  t.r1 = min(t.r0 + Body::kRows, sq.n * a.group);
  t.first_pos = sq.past + t.r0 / a.group;
  t.last_pos = sq.past + (t.r1 - 1) / a.group;
  t.fill = sq.bad || t.last_pos < 0;
  const int from = a.window > 0 ? max(t.first_pos - a.window + 1, 0) : 0;
  t.begin = t.fill ? 0 : from / Body::kStep;
  t.end = t.fill ? 1 : t.last_pos / Body::kStep + 1;
  return t;
}
// What a task takes of a line: `even`, the pieces it makes at kMinSteps or more
// steps each; else its steps and kTaskCost.
template <class Body>
__device__ __forceinline__ int size_of(const Task& t, bool even) {
  const int steps = t.end - t.begin;
  return even ? (steps + Body::kMinSteps - 1) / Body::kMinSteps : steps + Body::kTaskCost;
}
template <class Body>
__device__ __forceinline__ int tiles_of(const Args& a, const Seq& sq) {
  return (sq.n * a.group + Body::kRows - 1) / Body::kRows;
}
// Of a head's tasks together, by one lane.
template <class Body>
__device__ __forceinline__ int head_size(const Args& a, const Seq& sq, bool even) {
  const int tiles = tiles_of<Body>(a, sq);
  int n = 0;
  for (int i = 0; i < tiles; i++) n += size_of<Body>(task_of<Body>(a, sq, i), even);
  return n;
}

// Sums over the lanes before this one, and this one's own with them.
__device__ __forceinline__ int wave_scan(int v) {
  const int lane = (int)threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int x = __shfl_up(v, d);
    if (lane >= d) v += x;
  }
  return v;
}

// The task at place u of a head's tasks (0 <= u < head_size), and where it
// begins: 64 tasks at a time, one a lane.
template <class Body>
__device__ __forceinline__ Task find_task(const Args& a, const Seq& sq, bool even, int u, int& at) {
  const int tiles = tiles_of<Body>(a, sq), lane = (int)threadIdx.x & 63;
  at = 0;
  if (tiles == 1) return task_of<Body>(a, sq, 0);
  for (int i0 = 0;; i0 += 64) {
    const int i = i0 + lane;
    const int n = i < tiles ? size_of<Body>(task_of<Body>(a, sq, i), even) : 0;
    const int upto = wave_scan(n);
    const uint64_t past = __ballot(at + upto > u);
    if (past || i0 + 64 >= tiles) {
      const int l = past ? __builtin_ctzll(past) : 0;
      at += lane_of(upto - n, l);
      return task_of<Body>(a, sq, i0 + l);
    }
    at += lane_of(upto, 63);
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

template <class Body>
__device__ __forceinline__ void fill_rows(const Args& a, const Seq& sq, const Task& t, int h) {
  const float o = sq.bad ? __builtin_nanf("") : 0.f, lse = sq.bad ? __builtin_nanf("") : -kInf;
  const int chunks = a.D / 8;
  for (int e = threadIdx.x; e < (t.r1 - t.r0) * chunks; e += threads_of<Body>) {
    const int row = t.r0 + e / chunks, d = e % chunks * 8;
    store8<Body::kBf16>(a, out_at(a, sq, h, row, d), {o, o, o, o, o, o, o, o});
    if (a.lse && d == 0) store_lse(a, sq, h, row, lse);
  }
}

constexpr int kCoherent = 16;  // cache policy bits of a buffer access: sc1
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

// A task's parts: part p of `count` by workgroup w0 + p, part 0 in slot 1 of
// its workgroup, the others in slot 0.
struct Part {
  int w0, count;
  __device__ __forceinline__ int64_t slot(int p) const { return 2 * ((int64_t)w0 + p) + (p == 0); }
};

// Whether the flags of all parts are set; if so they are put back.  By the
// whole workgroup, with a word of LDS that is not in use.
__device__ __forceinline__ bool all_there(const Args& a, const Part& part, int* word) {
  if (threadIdx.x < 64) {
    bool all = true;
    for (int p = (int)threadIdx.x; p < part.count; p += 64)
      all &= __hip_atomic_load(a.flags + part.slot(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.token;
    const bool done = __ballot(!all) == 0;
    if (threadIdx.x == 0) *word = done;
    if (done)
      for (int p = (int)threadIdx.x; p < part.count; p += 64)
        __hip_atomic_store(a.flags + part.slot(p), (uint64_t)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *word != 0;
}

// Join the parts of a task and store its rows.
template <class Body>
__device__ __forceinline__ void join_parts(const Args& a, const Seq& sq, const Task& task, int h, const Part& part) {
  constexpr int kRows = Body::kRows, DP = Body::kDim, kSlot = kRows * (DP + 2);
  const int chunks = a.D / 8;
  for (int e = threadIdx.x; e < (task.r1 - task.r0) * chunks; e += threads_of<Body>) {
    const int row = e / chunks, d = (e - row * chunks) * 8;
    float mx = -kInf, sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const auto load = [&](int p, float& m, float& l, f32x4& lo, f32x4& hi) {
      const __amdgpu_buffer_rsrc_t rs = rsrc(a.parts + part.slot(p) * kSlot, kSlot * 4);
      const int at = (row * DP + d) * 4;
      const u32x2 ml = __builtin_amdgcn_raw_buffer_load_b64(rs, (kRows * DP + 2 * row) * 4, 0, kCoherent);
      lo = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, kCoherent));
      hi = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at + 16, 0, kCoherent));
      m = __uint_as_float(ml[0]);
      l = __uint_as_float(ml[1]);
    };
#pragma unroll 4
    for (int p = 0; p < part.count; p++) {
      float m, l;
      f32x4 x[2];
      load(p, m, l, x[0], x[1]);
      const float mn = fmaxf(mx, m), mu = finite_or_0(mn);
      const float f = exp2_(mx - mu), w = exp2_(m - mu) * l;
      mx = mn;
      sum = sum * f + w;
#pragma unroll
      for (int i = 0; i < 8; i++) acc[i] = acc[i] * f + w * x[i / 4][i % 4];
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < 8; i++) acc[i] *= inv;
    store8<Body::kBf16>(a, out_at(a, sq, h, task.r0 + row, d), acc);
    if (a.lse && d == 0) store_lse(a, sq, h, task.r0 + row, lse_of(mx, sum));
  }
}

// A sequence, where it begins and ends on a line.
struct Place {
  int s, from, to;
};

// A line over up to 64 sequences, one a lane; every wave has its own.
struct LaneLine {
  int from, to, total;
  __device__ __forceinline__ explicit LaneLine(int n) : to(wave_scan(n)) {
    from = to - n;
    // cu_new that decreases can count tokens until the sum overflows (the first
    // sum that does is negative): nothing is on the line then.
    total = __any(to < 0) ? 0 : lane_of(to, 63);
  }
  __device__ __forceinline__ Place find(int u) const {
    const int s = __builtin_ctzll(__ballot(to > u));  // the first that ends behind u
    return Place{s, lane_of(from, s), lane_of(to, s)};
  }
};

// For more sequences: a prefix sum in LDS, by the whole workgroup.
template <class Body>
struct LdsLine {
  int* line;  // [S + 1]: where sequence s begins
  int total, S;
  template <typename F>
  __device__ __forceinline__ LdsLine(int n_seqs, int* l, int* wave_sum, F cost) : line(l), total(0), S(n_seqs) {
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int each = (S + threads_of<Body> - 1) / threads_of<Body>, s1 = min((tid + 1) * each, S);
    int mine = 0;
    bool bad = false;  // the sum overflows, see LaneLine
    for (int s = tid * each; s < s1; s++) {
      line[s] = cost(s);
      mine += line[s];
      bad |= mine < 0;
    }
    const int upto = wave_scan(mine);
    bad = __any(bad || upto < 0);
    if (lane == 63) wave_sum[wave] = bad ? -1 : upto;
    __syncthreads();
    int at = upto - mine;
    bad = false;
    for (int w = 0; w < Body::kWaves; w++) {
      if (w < wave) at += wave_sum[w];
      total += wave_sum[w];
      bad |= wave_sum[w] < 0 || total < 0;
    }
    if (bad) total = 0;
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

// n places in `pieces` pieces that differ by one at most, the longer ones first.
struct Cut {
  int pieces, each, more;
  __device__ __forceinline__ Cut(int n, int p) : pieces(p), each(p > 0 ? n / p : 0), more(p > 0 ? n - each * p : 0) {}
  __device__ __forceinline__ int start(int i) const { return i * each + min(i, more); }
  __device__ __forceinline__ int piece(int u) const {  // the piece of place u
    const int longer = more * (each + 1);
    return u < longer ? u / (each + 1) : more + (u - longer) / max(each, 1);
  }
};

// Steps begin .. end - 1 of a task by this workgroup.
template <class Body>
__device__ __forceinline__ void run_piece(const Args& a, const Seq& sq, const Task& task, int s, int h, int begin,
                                          int end, const Part& part, float* lds, int* joined) {
  if (task.fill) {
    fill_rows<Body>(a, sq, task, h);
    return;
  }
  Body::run(a, sq, task, s, h, begin, end, part, lds);
  if (part.count == 1) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's share of them has arrived
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint64_t old = __hip_atomic_exchange(a.flags + part.slot((int)blockIdx.x - part.w0), a.token, __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::"v"(old));
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // and the flag, before the others' are read
  if (all_there(a, part, joined)) join_parts<Body>(a, sq, task, h, part);
}

// All work on one line (see the top).  Where there are fewer pieces of
// Body::kMinSteps steps than workgroups, each task is cut evenly and every piece
// has a workgroup.  Else workgroup w takes the w-th equal piece of the line,
// on which a task begins with Body::kTaskCost places that stand for what it costs
// beside its steps: about what that many steps take.
template <class Body, bool MANY>
__global__ __launch_bounds__(threads_of<Body>, Body::kPerCu* Body::kWaves / 4) void k_attention_line(Args a) {
  extern __shared__ __align__(16) float lds[];
  __shared__ int wave_sum[Body::kWaves];
  __shared__ int joined;
  constexpr int kTaskCost = Body::kTaskCost;
  const int lane = (int)threadIdx.x & 63;
  Seq mine{0, 0, 0, false};  // of this lane's sequence
  if (!MANY && lane < a.S) mine = seq_of(a, lane);
  const auto seq_at = [&](int s) {
    return MANY ? seq_of(a, s)
                : Seq{lane_of(mine.c0, s), lane_of(mine.n, s), lane_of(mine.past, s), lane_of((int)mine.bad, s) != 0};
  };
  const auto make = [&](bool even) {
    if constexpr (MANY) {
      return LdsLine<Body>(a.S, reinterpret_cast<int*>(lds + Body::kLds), wave_sum,
                           [&](int s) { return head_size<Body>(a, seq_of(a, s), even) * a.kv_heads; });
    } else {
      int n = 0;
      if (__ballot(tiles_of<Body>(a, mine) > 2) == 0) {
        n = head_size<Body>(a, mine, even);
      } else {  // a sequence at a time, a task a lane
        for (int s = 0; s < a.S; s++) {
          const Seq sq = seq_at(s);
          const int tiles = tiles_of<Body>(a, sq);
          int x = 0;
          for (int i = lane; i < tiles; i += 64) x += size_of<Body>(task_of<Body>(a, sq, i), even);
          x = lane_of(wave_scan(x), 63);
          if (lane == s) n = x;
        }
      }
      return LaneLine(n * a.kv_heads);
    }
  };
  auto line = make(true);
  const bool even = line.total <= (int)gridDim.x;  // a piece a workgroup
  if (!even) line = make(false);
  const Cut cut(line.total, even ? line.total : (int)gridDim.x);
  if (line.total == 0 || (int)blockIdx.x >= cut.pieces) return;
  int u = cut.start((int)blockIdx.x);
  const int u_end = cut.start((int)blockIdx.x + 1);
  while (u < u_end) {
    const Place pl = line.find(u);
    const Seq sq = seq_at(pl.s);
    const int per_head = (pl.to - pl.from) / a.kv_heads, h = (u - pl.from) / per_head;
    int at;  // where the task begins on the line
    const Task task = find_task<Body>(a, sq, even, u - pl.from - h * per_head, at);
    at += pl.from + h * per_head;
    const int steps = task.end - task.begin, size = size_of<Body>(task, even);
    int begin, end;
    Part part;
    if (even) {
      const Cut of(steps, size);
      begin = task.begin + of.start(u - at);
      end = task.begin + of.start(u - at + 1);
      part = Part{at, size};
      u = u_end;
    } else {
      const int first = at + kTaskCost, last = at + size;  // the task's steps on the line
      begin = task.begin + max(u - first, 0);
      end = task.begin + min(u_end, last) - first;
      part.w0 = cut.piece(first);
      part.count = cut.piece(last - 1) - part.w0 + 1;
      u = last;
    }
    if (begin < end) {
      run_piece<Body>(a, sq, task, pl.s, h, begin, end, part, lds, &joined);
      __syncthreads();  // LDS is used again
    }
  }
}

// Without a workspace: a workgroup a task.  Sequence s has the tasks
// floor(cu[s] group / rows) + s up to the same of s + 1 for each head, at
// least as many as its rows need.
template <class Body>
__global__ __launch_bounds__(threads_of<Body>, Body::kPerCu* Body::kWaves / 4) void k_attention_task(Args a) {
  extern __shared__ __align__(16) float lds[];
  constexpr int kRows = Body::kRows;
  const int h = (int)(blockIdx.x % (uint32_t)a.kv_heads);
  const int64_t slot = blockIdx.x / (uint32_t)a.kv_heads;
  const int s = find_last(a.S, [&](int i) { return (int64_t)a.cu[i] * a.group / kRows + i <= slot; });
  const int64_t first = (int64_t)a.cu[s] * a.group / kRows + s;
  const Seq sq = seq_of(a, s);
  if (slot < first || (slot - first) * kRows >= (int64_t)sq.n * a.group) return;
  const Task task = task_of<Body>(a, sq, (int)(slot - first));
  if (task.fill)
    fill_rows<Body>(a, sq, task, h);
  else
    Body::run(a, sq, task, s, h, task.begin, task.end, Part{0, 1}, lds);
}

// ---- launch ----
inline hipError_t launch(const void* fn, int threads, int64_t blocks, size_t lds, Args& a, hipStream_t s) {
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  if (lds > 65536) {
    hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  void* args[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)blocks), dim3((unsigned)threads), args, lds, s);
}

template <class Body>
uint64_t workers() {
  return (uint64_t)cu_count() * Body::kPerCu;
}
template <class Body>
uint64_t workspace_bytes() {
  return workers<Body>() * 2 * ((uint64_t)(Body::kRows * (Body::kDim + 2)) * 4 + 8);
}

uint64_t launch_token();

template <class Body>
hipError_t go(Args& a, void* ws, uint64_t ws_bytes, hipStream_t s) {
  const size_t lds = sizeof(float) * (size_t)Body::kLds;
  // the line's places are 32-bit numbers
  const int64_t tasks = ((int64_t)a.T * a.group / Body::kRows + a.S) * a.kv_heads;
  const int64_t steps = ((int64_t)a.max_pages << a.shift) / Body::kStep + 2 + Body::kTaskCost;
  const bool fits = tasks < 0x40000000 && tasks * steps < 0x40000000;
  if (fits && ws && ws_bytes >= workspace_bytes<Body>()) {
    const int64_t n = (int64_t)workers<Body>();
    a.flags = reinterpret_cast<uint64_t*>(ws);
    a.parts = reinterpret_cast<float*>(a.flags + 2 * n);
    a.token = launch_token();
    return a.S > 64 ? launch(reinterpret_cast<const void*>(k_attention_line<Body, true>), threads_of<Body>, n, lds + 4 * (size_t)(a.S + 1), a, s)
                    : launch(reinterpret_cast<const void*>(k_attention_line<Body, false>), threads_of<Body>, n, lds, a, s);
  }
  return launch(reinterpret_cast<const void*>(k_attention_task<Body>), threads_of<Body>, tasks, lds, a, s);
}

}  // namespace attn

// attention_chunk.hip
uint64_t attention_chunk_workspace_bytes(int64_t T, int64_t S, int64_t group, int64_t dim);
hipError_t launch_attention_chunk(bool bf16, attn::Args& a, void* ws, uint64_t ws_bytes, hipStream_t s);

}  // namespace patch
