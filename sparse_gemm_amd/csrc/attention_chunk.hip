// attention_chunk.hip -- attention over the paged 8-bit cache for many new
// tokens a sequence (prompts and their chunks).
//
// Here the matrix cores and the exponentials bound the work, not the cache:
// every row tile reads the same keys, mostly from L2.  So the eight waves of a
// workgroup have 16 R rows each and share the keys: a tile of 128 keys is
// loaded once, each wave widening 16 of them into LDS as ready matrix
// operands (lane order, 16 bytes a lane: reads and writes without bank
// conflicts), and every wave then runs all 128 against its rows.  LDS holds two
// tiles (128 KB at 128 elements, so one workgroup a CU): one is used while the
// next is filled, whose bytes were loaded a tile earlier; one barrier a tile.
// Rows are a wave's own, so nothing is joined at a task's end.
//
// The products, the running maximum and sum, and the order of the keys inside
// an operand are those of attention.hip.
//
// Three sequences, 700 to 1100 new tokens behind 1500 to 5000, 32 query and 8
// cache heads of 128: 152 GFLOP in 253 us, 603 TFLOP/s, where a large bf16
// product reaches 1239.  A wave's matrix instructions take 74 us of that and
// its other arithmetic (exponentials, widening, maxima, sums) 116, and two
// waves a SIMD (256 registers each) overlap them little.  Measured instead:
// two workgroups of four waves with a tile each, 16 rows a wave at four waves a
// SIMD (434 us, registers spill), 64 keys of scores before the exponentials
// (263 us against 262 then), wave priorities around the second product (271)
// and prescribed interleavings of matrix and other instructions (276 to 300).
#include "attention_common.h"

namespace patch {
using namespace attn;
namespace {

constexpr int kTile = 128;           // keys of a tile (a step of the line)
constexpr float kNoScale = -200.0f;  // log2 of a scale that is 0
constexpr int kSubs = kTile / 16;    // its sub-tiles of 16 keys, each in one page

// Waits for this wave's LDS traffic, not for loads from memory, and meets the others.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// FULL: dim is DP, and a row's distance a constant.  WIDE: the probabilities in
// two fp16 values, 22 bits, for fp32 outputs.
template <bool BF16, int DP, int R, bool FULL, bool WIDE = false>
struct Chunk {
  static constexpr bool kBf16 = BF16;
  static constexpr int kWaves = 8, kDim = DP, kRows = kWaves * 16 * R, kStep = kTile;
  // Measured: pieces of at least 4 tiles, a prompt of 600 tokens 53.6 us, of 2
  // tiles 55.3, of 8 tiles 51.2.  A task's own cost (its rows' q, the first
  // tiles' way into LDS, its part) of 6 tiles, prompts of 1500, 300, 2000 and
  // 800 tokens 183 us, of 2 tiles 212, of 12 tiles 199.
  static constexpr int kMinSteps = 4, kTaskCost = 6;
  static constexpr int kPerCu = 1;
  static constexpr int kFrags = DP / 16;                        // operands (1 KB) of 32 keys, of K as of V
  static constexpr int kBuf = kTile / 32 * 2 * kFrags * 64;       // 16-byte words of a tile
  static constexpr int kLds = 2 * (kBuf * 4 + 1) + 2;             // two, each with a word that says that V held a NaN
  static constexpr int VB = DP / 16;                            // bytes of a V row in a lane

  // Pages of eight tiles, a sub-tile a lane.
  struct Pages {
    int64_t at;        // where the sub-tile's rows begin in k and v
    float ks, vs;      // k scale (with the softmax's), log2 of the v scale
    float vmax;        // the largest vs of the lane's tile
    float lv, vi;      // vs relative to vref with kBias, and 2^ of minus the former
  };
  static __device__ __forceinline__ Pages load_pages(const Args& a, const int32_t* table, int h, int tile, int last_pos) {
    Pages p;
    const int key = (int)min((int64_t)tile * kTile + 16 * (int64_t)(threadIdx.x & 63), (int64_t)(last_pos & ~15));
    const int page = table[key >> a.shift];
    const bool ok = page >= 0 && page < a.pages;
    const int64_t block = (int64_t)(ok ? page : 0) * a.kv_heads + h;
    p.at = (block * a.B + (key & (a.B - 1))) * a.D;
    p.ks = ok ? a.ks[block] * a.scale : __builtin_nanf("");
    // a scale of 0 (or a page outside the cache) counts as a very small one
    p.vs = fmaxf(ok ? __log2f(a.vs[block]) : kNoScale, kNoScale);
    p.vmax = p.vs;
#pragma unroll
    for (int d = 1; d < kSubs; d *= 2) p.vmax = fmaxf(p.vmax, __shfl_xor(p.vmax, d));
    p.lv = p.vi = 0.f;
    return p;
  }
  static __device__ __forceinline__ void relative(Pages& p, float vref) {
    const float v = fmaxf(p.vs - vref, -100.0f);
    p.lv = v + kBias;
    p.vi = exp2_(-v);
  }
  static __device__ __forceinline__ int64_t at_of(const Pages& p, int i) {
    return (int64_t)(uint32_t)lane_of((int)p.at, i) | (int64_t)lane_of((int)(p.at >> 32), i) << 32;
  }
  static __device__ __forceinline__ int dim(const Args& a) { return FULL ? DP : a.D; }

  // The bytes of this wave's sub-tile of a tile.
  struct Bytes {
    u32x4 k[DP / 64];
    Vec<uint32_t, VB / 4> v[4];
  };
  static __device__ __forceinline__ Bytes load(const Args& a, int64_t at) {
    const int lane = (int)threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    Bytes b;
    // uniform addresses, and a lane's 32-bit offset from them; behind element D
    // - 1 the same key's first ones: q is zero there
    const int D = dim(a);
    const uint32_t vo = (uint32_t)(4 * g * D + (FULL || n * VB < D ? n * VB : 0));
#pragma unroll
    for (int j = 0; j < DP / 64; j++)
      b.k[j] = ld16(a.k + at + (uint32_t)(n * D + (FULL || j * 64 + g * 16 < D ? j * 64 + g * 16 : 0)));
#pragma unroll
    for (int i = 0; i < 4; i++)
      b.v[i] = *reinterpret_cast<const Vec<uint32_t, VB / 4>*>(a.v + at + (uint32_t)(vo + i * D));
    return b;
  }
  // Into LDS: operands of K, and halves of operands of V.  `mask`: V rows that
  // no row of the task sees hold anything at all: take zeros.  A NaN in a row
  // that some see must not reach the others through 0 * NaN: it is taken out
  // here and put back after the products, row by row.  Returns whether V held one.
  static __device__ __forceinline__ bool widen(Bytes& b, u32x4* frags, int sub, bool mask, int key0, int any_from,
                                               int last_pos) {
    const int lane = (int)threadIdx.x & 63, g = lane >> 4;
    bool has = false;
    if (mask) {
      const int from = seldom(key0 + sub * 16);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int key = from + 4 * g + i;
        const bool seen = key >= any_from && key <= last_pos;
#pragma unroll
        for (int w = 0; w < VB / 4; w++) {
          const uint32_t v = seen ? b.v[i].v[w] : 0u;
          const uint32_t hit = ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
          has |= hit != 0;
          b.v[i].v[w] = v & ~((hit >> 7) * 0xffu);
        }
      }
    }
    u32x4* kf = frags + ((sub >> 1) * 2 * kFrags + (sub & 1) * (DP / 32)) * 64 + lane;
#pragma unroll
    for (int j = 0; j < DP / 64; j++) {
      kf[(2 * j) * 64] = widen8<BF16>(b.k[j][0], b.k[j][1]);
      kf[(2 * j + 1) * 64] = widen8<BF16>(b.k[j][2], b.k[j][3]);
    }
    u32x2* vf = reinterpret_cast<u32x2*>(frags + ((sub >> 1) * 2 + 1) * kFrags * 64 + lane) + (sub & 1);
#pragma unroll
    for (int w = 0; w < VB / 4; w++) {
      u32x2 e[4];
#pragma unroll
      for (int p = 0; p < 2; p++) {
        uint32_t w0, w1, w2, w3;
        zip2(b.v[2 * p].v[w], b.v[2 * p + 1].v[w], w0, w1, w2, w3);
        e[0][p] = w0;
        e[1][p] = w1;
        e[2][p] = w2;
        e[3][p] = w3;
      }
#pragma unroll
      for (int j = 0; j < 4; j++) vf[(4 * w + j) * 128] = e[j];
    }
    return __ballot(has) != 0;
  }

  // Scores of 32 keys, whose operands begin at `at`, for the wave's rows.
  template <int RR>
  static __device__ __forceinline__ void scores(const u32x4* at, const u32x4 (&q)[RR][DP / 32], f32x4 (&sc)[RR][2]) {
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int r = 0; r < RR; r++) sc[r][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < DP / 32; j++)
#pragma unroll
      for (int t = 0; t < 2; t++) {
        const u32x4 k = at[(t * (DP / 32) + j) * 64];
#pragma unroll
        for (int r = 0; r < RR; r++) sc[r][t] = mma_dense<BF16>(k, q[r][j], sc[r][t]);
      }
  }

  static __device__ __forceinline__ void run(const Args& a, const Seq& sq, const Task& task, int s, int h, int begin,
                                             int end, const Part& part, float* lds) {
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, g = lane >> 4;
    u32x4* const bufs = reinterpret_cast<u32x4*>(lds);  // two tiles: [32 keys][K, V][operand][lane]
    int* const nan_words = reinterpret_cast<int*>(lds + 2 * kBuf * 4);
    const int32_t* table = a.table + s * a.table_row;
    const int row0 = task.r0 + wave * 16 * R;

    // ---- this wave's rows ----
    u32x4 q[R][DP / 32];
    f32x4 o[R][DP / 16];
    float m[R], l[R];
    int hi[R], lo[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      const int row = row0 + r * 16 + n, tok = row / a.group;
      const bool ok = row < task.r1;
      hi[r] = ok ? sq.past + tok : 0x7fffffff;
      lo[r] = ok && a.window > 0 ? hi[r] - a.window + 1 : (int)0x80000000;
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
        q[r][j] = v ^ a.q_flip;
      }
#pragma unroll
      for (int j = 0; j < DP / 16; j++) o[r][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
      m[r] = -kInf;
      l[r] = 0.f;
    }
    float vref = -kInf;  // log2 of what o is in units of: the largest v scale so far
    const int all_from = a.window > 0 ? max(task.last_pos - a.window + 1, 0) : 0;
    const int any_from = a.window > 0 ? max(task.first_pos - a.window + 1, 0) : 0;

    const auto is_partial = [&](int tile) { return tile * kTile < all_from || (tile + 1) * kTile - 1 > task.first_pos; };
    const auto bring = [&](Bytes& b, int tile) {
      const int i = (tile - begin) & 1;
      if (widen(b, bufs + i * kBuf, wave, is_partial(tile), tile * kTile, any_from, task.last_pos) && lane == 0)
        nan_words[i] = tile;
    };

    // Tile i is used from one half of LDS while tile i + 1 is widened into the
    // other and the bytes of tile i + 2 are on their way.
    Pages pages = load_pages(a, table, h, begin, task.last_pos), next_pages = pages;
    Bytes raw = load(a, at_of(pages, wave));
    bring(raw, begin);
    if (begin + 1 < end) raw = load(a, at_of(pages, kSubs + wave));
    meet();
    for (int tile = begin; tile < end; tile++) {
      const int i = tile - begin, base = (i & 7) * kSubs;
      const int key0 = tile * kTile;
      const bool partial = is_partial(tile);
      const u32x4* const frags = bufs + (i & 1) * kBuf;
      const bool nan_v = partial && nan_words[i & 1] == tile;
      if (tile + 1 < end) {
        bring(raw, tile + 1);
        if (tile + 2 < end) {
          if (((i + 2) & 7) == 0) next_pages = load_pages(a, table, h, tile + 2, task.last_pos);
          const int64_t at = ((i + 2) >> 3) == (i >> 3) ? at_of(pages, ((i + 2) & 7) * kSubs + wave)
                                                        : at_of(next_pages, ((i + 2) & 7) * kSubs + wave);
          raw = load(a, at);
        }
      }

      const float vmax = lane_of(pages.vmax, base);
      if (vmax > vref) {
        const float f = exp2_(vref - vmax);
        vref = vmax;
        relative(pages, vref);
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
          for (int j = 0; j < DP / 16; j++) o[r][j] *= f;
      }

      // 32 keys at a time; the next ones' scores are computed between this
      // one's exponentials
      f32x4 sc[2][R][2];
      scores<R>(frags + lane, q, sc[0]);
#pragma unroll
      for (int st = 0; st < kTile / 32; st++) {
        f32x4(&cur)[R][2] = sc[st & 1];
        const int sub0 = base + st * 2, from0 = key0 + st * 32;
        float ks[2], lv[2], vi[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
          ks[t] = lane_of(pages.ks, sub0 + t);
          lv[t] = lane_of(pages.lv, sub0 + t);
          vi[t] = lane_of(pages.vi, sub0 + t);
        }
        if (partial) {
          const int from = seldom(from0);
#pragma unroll
          for (int t = 0; t < 2; t++) {
#pragma unroll
            for (int r = 0; r < R; r++)
#pragma unroll
              for (int i = 0; i < 4; i++) {
                const int key = from + 16 * t + 4 * g + i;
                const bool seen = key <= hi[r] && key >= lo[r] && key <= task.last_pos;
                cur[r][t][i] = seen ? cur[r][t][i] * ks[t] : -kInf;
              }
            ks[t] = 1.0f;
          }
        }
        float mx[R];
        bool grows = false;
#pragma unroll
        for (int r = 0; r < R; r++) {
          float mt[2];
#pragma unroll
          for (int t = 0; t < 2; t++)
            mt[t] = fmaxf(fmaxf(cur[r][t][0], cur[r][t][1]), fmaxf(cur[r][t][2], cur[r][t][3])) * ks[t];
          mx[r] = fmaxf(mt[0], mt[1]);
          grows |= mx[r] > m[r] + kSlack;
        }
        if (__ballot(grows)) {
#pragma unroll
          for (int r = 0; r < R; r++) {
            const float mn = fmaxf(m[r], quad_max(mx[r]));
            const float f = exp2_(m[r] - finite_or_0(mn));
            m[r] = mn;
            l[r] *= f;
#pragma unroll
            for (int j = 0; j < DP / 16; j++) o[r][j] *= f;
          }
        }
        if (st + 1 < kTile / 32) scores<R>(frags + (st + 1) * 2 * kFrags * 64 + lane, q, sc[(st + 1) & 1]);
        // probabilities times the v scale (relative to vref): 2^(s + log2(vs) - m
        // + kBias), one multiply-add and the exponential; the sum takes them
        // divided by it again
        u32x4 pr[R], rest[WIDE ? R : 1];
#pragma unroll
        for (int r = 0; r < R; r++) {
          const float mu = finite_or_0(m[r]);
          f16x8 ph, pl;
#pragma unroll
          for (int t = 0; t < 2; t++) {
            const float off = lv[t] - mu;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
              const float e = exp2_(fmaf(cur[r][t][i], ks[t], off));
              sum += e;
              ph[4 * t + i] = (_Float16)e;
              if constexpr (WIDE) pl[4 * t + i] = (_Float16)(e - (float)ph[4 * t + i]);
            }
            l[r] = fmaf(sum, vi[t], l[r]);
          }
          pr[r] = __builtin_bit_cast(u32x4, ph);
          if constexpr (WIDE) rest[r] = __builtin_bit_cast(u32x4, pl);
        }
        const u32x4* vf = frags + (st * 2 + 1) * kFrags * 64 + lane;
#pragma unroll
        for (int j = 0; j < DP / 16; j++) {
          const u32x4 v = vf[j * 64];
#pragma unroll
          for (int r = 0; r < R; r++) {
            o[r][j] = mma_dense<false>(v, pr[r], o[r][j]);
            if constexpr (WIDE) o[r][j] = mma_dense<false>(v, rest[r], o[r][j]);
          }
        }
      }
      if (nan_v) {
        // rare: V holds NaN in a row that not every row of the task sees (as in attention.hip)
        const int vd = n * VB < a.D ? n * VB : 0;
#pragma unroll 1
        for (int st = 0; st < kTile / 32; st++) {
          u32x4 see[R];
          const int from0 = seldom(key0 + st * 32);
#pragma unroll
          for (int r = 0; r < R; r++) {
            f16x8 one;
#pragma unroll
            for (int i = 0; i < 8; i++) {
              const int key = from0 + (i >> 2) * 16 + 4 * g + (i & 3);
              one[i] = key <= hi[r] && key >= lo[r] && key <= task.last_pos ? (_Float16)1.0f : (_Float16)0.0f;
            }
            see[r] = __builtin_bit_cast(u32x4, one);
          }
#pragma unroll
          for (int w = 0; w < VB / 4; w++) {
            uint32_t nan[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
              const int key = from0 + (i >> 2) * 16 + 4 * g + (i & 3);
              const uint32_t v = *reinterpret_cast<const uint32_t*>(
                  a.v + at_of(pages, base + st * 2 + (i >> 2)) + (4 * g + (i & 3)) * a.D + vd + 4 * w);
              nan[i] =
                  key >= any_from && key <= task.last_pos ? (((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7 : 0u;
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
                  if (hit[i] > 0.f) o[r][4 * w + j][i] = __builtin_nanf("");
              }
          }
        }
      }
      if (((i + 1) & 7) == 0) {
        pages = next_pages;
        relative(pages, vref);
      }
      meet();
    }

    // ---- a lane holds elements 4g VB .. 4g VB + 4 VB - 1 of its row ----
    const int me = (int)blockIdx.x - part.w0;
    const bool store = part.count == 1;
    const __amdgpu_buffer_rsrc_t rs = rsrc(a.parts + part.slot(me) * (kRows * (DP + 2)), kRows * (DP + 2) * 4);
#pragma unroll
    for (int r = 0; r < R; r++) {
      const int row = (wave * R + r) * 16 + n;  // of the task
      l[r] = quad_sum(l[r]);
      if (task.r0 + row >= task.r1) continue;
      const float by = l[r] == 0.f || vref <= kNoScale ? 0.f : exp2_(vref) / l[r];
      if (g == 0) {
        if (store) {
          if (a.lse) store_lse(a, sq, h, task.r0 + row, lse_of(m[r], l[r]));
        } else {
          const u32x2 ml = {__float_as_uint(m[r]), __float_as_uint(l[r])};
          __builtin_amdgcn_raw_buffer_store_b64(ml, rs, (kRows * DP + 2 * row) * 4, 0, kCoherent);
        }
      }
#pragma unroll
      for (int e = 0; e < 4 * VB; e += 8) {
        const int d = 4 * g * VB + e;
        if (d >= a.D) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = o[r][(e + i) % VB][(e + i) / VB] * by;
        if (store) {
          store8<BF16>(a, out_at(a, sq, h, task.r0 + row, d), v);
        } else {
          const f32x4 v0 = {v[0], v[1], v[2], v[3]}, v1 = {v[4], v[5], v[6], v[7]};
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v0), rs, (row * DP + d) * 4, 0, kCoherent);
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v1), rs, (row * DP + d + 4) * 4, 0, kCoherent);
        }
      }
    }
  }
};


// Rows of a wave in sixteens, by the rows a sequence has on average.  8
// sequences of 4096 keys, 32 query and 8 cache heads of 128, one against two:
// 128 rows 63 us to 78, 256 rows 85 to 101, 512 rows 140 to 127.
int wave_rows(int64_t T, int64_t S, int64_t group) { return T * group <= 256 * S ? 1 : 2; }

template <bool BF16, int R>
hipError_t by_dim(Args& a, void* ws, uint64_t ws_bytes, hipStream_t s) {
  if (a.D == 64) return go<Chunk<BF16, 64, R, true>>(a, ws, ws_bytes, s);
  if (a.D == 128) return go<Chunk<BF16, 128, R, true>>(a, ws, ws_bytes, s);
  if (a.D < 64) return go<Chunk<BF16, 64, R, false>>(a, ws, ws_bytes, s);
  return go<Chunk<BF16, 128, R, false>>(a, ws, ws_bytes, s);
}
template <bool BF16>
hipError_t by_rows(Args& a, void* ws, uint64_t ws_bytes, hipStream_t s) {
  return wave_rows(a.T, a.S, a.group) == 1 ? by_dim<BF16, 1>(a, ws, ws_bytes, s) : by_dim<BF16, 2>(a, ws, ws_bytes, s);
}

// fp32 outputs: 16 rows a wave, whose registers hold the second half of the
// probabilities as well (a workspace for 32 is large enough).
template <bool BF16>
hipError_t wide(Args& a, void* ws, uint64_t ws_bytes, hipStream_t s) {
  return a.D <= 64 ? go<Chunk<BF16, 64, 1, false, true>>(a, ws, ws_bytes, s)
                   : go<Chunk<BF16, 128, 1, false, true>>(a, ws, ws_bytes, s);
}

}  // namespace

uint64_t attention_chunk_workspace_bytes(int64_t T, int64_t S, int64_t group, int64_t dim) {
  if (wave_rows(T, S, group) == 1)
    return dim <= 64 ? workspace_bytes<Chunk<true, 64, 1, true>>() : workspace_bytes<Chunk<true, 128, 1, true>>();
  return dim <= 64 ? workspace_bytes<Chunk<true, 64, 2, true>>() : workspace_bytes<Chunk<true, 128, 2, true>>();
}

hipError_t launch_attention_chunk(bool bf16, Args& a, void* ws, uint64_t ws_bytes, hipStream_t s) {
  if (a.out_f32) return bf16 ? wide<true>(a, ws, ws_bytes, s) : wide<false>(a, ws, ws_bytes, s);
  return bf16 ? by_rows<true>(a, ws, ws_bytes, s) : by_rows<false>(a, ws, ws_bytes, s);
}

}  // namespace patch
