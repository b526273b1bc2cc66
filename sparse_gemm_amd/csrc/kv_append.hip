// kv_append.hip -- new keys and values into the paged 8-bit cache, keys (and
// queries) rotated on the way.
//
// The unit of work is one block of the cache: the tokens of one sequence that
// fall into one page, for one head, of k or of v.  Its scale 2^ceil(log2(amax
// / 448)) needs every new value of the block before any is written, so a
// group of lanes owns the block: it reads and rotates the values once, keeps
// them in registers where they fit (else reads them again, from L2), reduces
// amax over its lanes, rounds and writes.  Nothing is shared between groups,
// so there are no atomics.
//
// Which sequence and page a group has is found on the device, since lengths
// change between replays of a graph: sequence s may take units floor(cu[s] /
// page) + 2 s up to the same of s + 1, at least as many as pages its new
// tokens can touch.  The unused ones end at once.
//
// Bound by HBM for prompts and by latency for a token a sequence, where a
// block has a single row: there 8 lanes own a block and a wave 8 heads.  Heads
// of 128, GPU time: a token to each of 64 sequences, 32 heads, in 5 us; 8
// prompts of 500 to 2100 tokens, 8 cache and 32 query heads, 191 MB in 46.9
// us (4.1 TB/s; a copy of 1 GiB reaches 5.1).
#include <algorithm>

#include "rotate.h"

namespace patch {
namespace {

constexpr int kThreads = 256;

// 2^ceil(log2(amax / 448)), at least 2^-126: 448 = 1.75 * 2^8, so amax = 1.m
// * 2^e needs 2^(e - 8), one more where 1.m > 1.75.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int k = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased exponent of the scale
  k = max(k, 1);
  return __uint_as_float((uint32_t)k << 23);
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __builtin_inff() ? a : 0.0f;  // infinities and NaN do not count
}

// Two values times r as e4m3 bytes; what is not finite becomes NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}
__device__ __forceinline__ float nan_unless_finite(float x) {
  return fabsf(x) < __builtin_inff() ? x : __builtin_nanf("");
}

// Store an item's values, scaled and rounded, into a cache row.
template <int V>
__device__ __forceinline__ void store_item_e4m3(uint8_t* row, const ItemPlace& p, const Item<V>& r, float inv) {
  float x[V], y[V];
  runs_of(p, r, x, y);
#pragma unroll
  for (int i = 0; i < V; i++) {
    x[i] = nan_unless_finite(x[i] * inv);
    y[i] = nan_unless_finite(y[i] * inv);
  }
  if constexpr (V == 1) {
    const uint32_t w = to_e4m3x4(x[0], y[0], 0.f, 0.f);
    row[p.first] = (uint8_t)w;
    row[p.second] = (uint8_t)(w >> 8);
  } else {
    Vec<uint32_t, V / 4> u, w;
#pragma unroll
    for (int i = 0; i < V / 4; i++) {
      u.v[i] = to_e4m3x4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      w.v[i] = to_e4m3x4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    }
    *reinterpret_cast<Vec<uint32_t, V / 4>*>(row + p.first) = u;
    *reinterpret_cast<Vec<uint32_t, V / 4>*>(row + p.second) = w;
  }
}

template <int GW>
__device__ __forceinline__ float group_max(float x, float* lds) {
#pragma unroll
  for (int d = 1; d < (GW < 64 ? GW : 64); d *= 2) x = fmaxf(x, __shfl_xor(x, d));
  if constexpr (GW > 64) {  // the group is the workgroup
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < GW / 64; w++) x = fmaxf(x, lds[w]);
  }
  return x;
}

// GW lanes a block, KEEP items of a lane held in registers.
template <typename T, int V, int GW, int KEEP>
__global__ __launch_bounds__(kThreads) void k_kv_append(patch_kv_append_args a, patch_kv_cache c, uint32_t kv_blocks,
                                                        uint32_t q_share, int q_tokens) {
  __shared__ float lds[kThreads / 64];
  const int rot = (int)a.rot, D = (int)c.dim, items = D / (2 * V), B = (int)c.page;
  const bool inter = a.layout == PATCH_ROPE_INTERLEAVED;
  const int S = (int)a.S;
  const int32_t* cu = a.cu_new_dev;

  uint32_t q_before = __umulhi(blockIdx.x, q_share), q_upto = __umulhi(blockIdx.x + 1, q_share);
  if (blockIdx.x - q_before >= kv_blocks) {
    q_before = blockIdx.x - kv_blocks;
    q_upto = q_before + 1;
  }
  if (q_upto > q_before) {  // q of q_tokens tokens
    const int ta = (int)q_before * q_tokens, tb = min(ta + q_tokens, (int)a.T);
    int s = find_last(S, [&](int i) { return cu[i] <= ta; });
    const int per = kThreads / items;  // heads at a time (items <= 128)
    const int ci = (int)threadIdx.x % items;
    if ((int)threadIdx.x >= per * items) return;
    const ItemPlace p = item_place<V>(ci, a.table_dev ? rot : 0, D, inter);
    for (int t = ta; t < tb; t++) {
      while (s + 1 < S && t >= cu[s + 1]) s++;
      if (t < cu[s] || t >= cu[s + 1]) continue;
      const int64_t pos = (int64_t)a.kv_lens_dev[s] - (cu[s + 1] - t);
      const float* row = a.table_dev && pos >= 0 && pos < a.context ? a.table_dev + pos * rot : nullptr;
      const T* x = reinterpret_cast<const T*>(a.q_dev) + (int64_t)t * a.q_token;
      T* o = reinterpret_cast<T*>(a.q_out_dev) + (int64_t)t * a.q_out_token;
      Angles<V> g;
      if (p.turned) g = load_angles<V>(row, p, rot, false);
      for (int h = (int)threadIdx.x / items; h < (int)a.heads; h += per) {
        Item<V> r = load_item<T, V>(x + h * a.q_head, p);
        if (p.turned) turn(r, g);
        store_item<T, V>(o + h * a.q_out_head, p, r);
      }
    }
    return;
  }

  // ---- which block: unit (sequence, page), head, k or v ----
  constexpr int kGroups = GW < 64 ? 64 / GW : 1;  // groups of a wave, all of one unit
  const int lane = (int)threadIdx.x % GW;
  const int kinds = 2 * (int)c.kv_heads;
  const uint32_t kv_block = blockIdx.x - q_before;
  int64_t unit;
  int kind;
  if constexpr (GW > 64) {
    unit = kv_block / (uint32_t)kinds;
    kind = (int)(kv_block % (uint32_t)kinds);
  } else {
    const uint32_t wave = kv_block * (kThreads / 64) + threadIdx.x / 64, per = (uint32_t)(kinds + kGroups - 1) / kGroups;
    unit = wave / per;
    kind = (int)(wave % per) * kGroups + (int)(threadIdx.x & 63) / GW;
  }
  const int s = find_last(S, [&](int i) { return (int64_t)cu[i] / B + 2 * i <= unit; });
  const int c0 = cu[s], n = cu[s + 1] - c0;
  const int64_t past = (int64_t)a.kv_lens_dev[s] - n;  // place of the first new token
  if (c0 < 0 || n <= 0 || past + n <= 0) return;       // (the whole wave or workgroup)
  const int64_t page_i = (past > 0 ? past / B : 0) + (unit - ((int64_t)c0 / B + 2 * s));
  const int64_t lo = past > page_i * B ? past : page_i * B;  // places lo .. hi - 1 are filled
  const int64_t hi = past + n < (page_i + 1) * B ? past + n : (page_i + 1) * B;
  if (unit < (int64_t)c0 / B + 2 * s || lo >= hi || page_i >= a.max_pages) return;
  const int page = a.page_table_dev[s * a.page_table_row + page_i];
  if (page < 0 || page >= c.pages) return;
  if (GW <= 64 && kind >= kinds) return;  // behind the last head; the lanes that shuffle below are whole groups

  const int head = kind >> 1;
  const bool is_k = (kind & 1) == 0;
  const bool rotates = is_k && a.table_dev;
  const int64_t block = (int64_t)page * c.kv_heads + head;
  uint8_t* cache = reinterpret_cast<uint8_t*>(is_k ? c.k_dev : c.v_dev) + block * B * D;
  float* scale_at = (is_k ? c.k_scale_dev : c.v_scale_dev) + block;
  const T* src = reinterpret_cast<const T*>(is_k ? a.k_dev : a.v_dev) + head * (is_k ? a.k_head : a.v_head);
  const int64_t stride = is_k ? a.k_token : a.v_token;
  const int first_slot = (int)(lo - page_i * B), count = (int)(hi - lo);
  const int64_t t0 = c0 + (lo - past);  // token of place lo
  // tokens outside 0 .. T - 1 (a bad cu_new) are not read
  const int total = t0 + count <= a.T ? count * items : t0 < a.T ? (int)(a.T - t0) * items : 0;
  if (total <= 0) return;

  auto get = [&](int e, ItemPlace& p) {
    const int r = e / items, ci = e - r * items;
    p = item_place<V>(ci, rotates ? rot : 0, D, inter);
    Item<V> x = load_item<T, V>(src + (t0 + r) * stride, p);
    if (p.turned) {
      const int64_t pos = lo + r;
      turn(x, load_angles<V>(pos < a.context ? a.table_dev + pos * rot : nullptr, p, rot, false));
    }
    return x;
  };
  const float held = first_slot > 0 ? *scale_at : 0.0f;
  Item<V> kept[KEEP];
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < KEEP; k++) {
    const int e = k * GW + lane;
    if (e < total) {
      ItemPlace p;
      kept[k] = get(e, p);
#pragma unroll
      for (int i = 0; i < V; i++) amax = fmaxf(amax, fmaxf(finite_abs(kept[k].a[i]), finite_abs(kept[k].b[i])));
    }
  }
  for (int e = KEEP * GW + lane; e < total; e += GW) {
    ItemPlace p;
    const Item<V> x = get(e, p);
#pragma unroll
    for (int i = 0; i < V; i++) amax = fmaxf(amax, fmaxf(finite_abs(x.a[i]), finite_abs(x.b[i])));
  }
  amax = group_max<GW>(amax, lds);
  float scale = scale_for(amax);
  if (first_slot > 0) {
    if (scale > held) {  // the values held so far, under the new scale
      const float by = held / scale;
      for (int e = lane; e < first_slot * (D / 16); e += GW) {
        uint32_t* w = reinterpret_cast<uint32_t*>(cache + (int64_t)e * 16);
        Vec<uint32_t, 4> x = *reinterpret_cast<Vec<uint32_t, 4>*>(w);
#pragma unroll
        for (int i = 0; i < 4; i++)
          x.v[i] = to_e4m3x4(by * __builtin_amdgcn_cvt_f32_fp8((int)x.v[i], 0), by * __builtin_amdgcn_cvt_f32_fp8((int)x.v[i], 1),
                             by * __builtin_amdgcn_cvt_f32_fp8((int)x.v[i], 2), by * __builtin_amdgcn_cvt_f32_fp8((int)x.v[i], 3));
        *reinterpret_cast<Vec<uint32_t, 4>*>(w) = x;
      }
    } else {
      scale = held;
    }
  }
  const float inv = 1.0f / scale;
#pragma unroll
  for (int k = 0; k < KEEP; k++) {
    const int e = k * GW + lane;
    if (e < total) {
      const int r = e / items;
      store_item_e4m3<V>(cache + (first_slot + r) * D, item_place<V>(e - r * items, rotates ? rot : 0, D, inter), kept[k],
                         inv);
    }
  }
  for (int e = KEEP * GW + lane; e < total; e += GW) {
    ItemPlace p;
    const Item<V> x = get(e, p);
    store_item_e4m3<V>(cache + (first_slot + e / items) * D, p, x, inv);
  }
  // every lane has read the old scale (a workgroup's waves have used it above)
  if constexpr (GW > 64) __syncthreads();
  if (lane == 0) *scale_at = scale;
}

template <typename T, int V, int GW, int KEEP>
hipError_t go(const patch_kv_append_args& a, const patch_kv_cache& c, hipStream_t s) {
  const int64_t units = a.T / c.page + 2 * a.S, kinds = 2 * c.kv_heads;
  int64_t blocks;
  if (GW > 64) {
    blocks = units * kinds;
  } else {
    constexpr int groups = 64 / (GW < 64 ? GW : 64);
    blocks = (units * ((kinds + groups - 1) / groups) + kThreads / 64 - 1) / (kThreads / 64);
  }
  // Tokens whose q a workgroup rotates, one against two, with 8 cache and 32
  // query heads: 1024 tokens 8.1 us to 8.6, 2048 tokens 12.7 to 11.8, 16384
  // tokens 89 to 86.
  const int q_tokens = a.T >= 2048 ? 2 : 1;
  const int64_t qs = a.q_dev ? (a.T + q_tokens - 1) / q_tokens : 0, all = blocks + qs;
  if (all > 0x7fffffff) return hipErrorInvalidValue;
  // From 4096 tokens on three quarters of q's workgroups lie evenly among the
  // others, whose waits they fill (before workgroup i lie i q_share / 2^32 of
  // them); the rest, and all of fewer tokens, follow.  8 prompts as above 46.9
  // us against 48.4, 8 of 1024 tokens 36.1 to 36.8; of 128 tokens 8.9 to 8.2.
  const uint64_t mixed = a.T >= 4096 ? (uint64_t)qs * 3 / 4 : 0, first = (uint64_t)blocks + mixed;
  const uint32_t q_share = (uint32_t)((mixed * 0x100000000ull + first - 1) / first);
  hipLaunchKernelGGL((k_kv_append<T, V, GW, KEEP>), dim3((unsigned)all), dim3(kThreads), 0, s, a, c, (uint32_t)blocks,
                     q_share, q_tokens);
  return hipGetLastError();
}

// A sequence brings up to two tokens on average: 8 lanes a block.  More: a
// workgroup a block, which keeps the whole block in registers, 2V values an
// item.  64 sequences of 8 cache heads, 8 lanes against a workgroup: a token
// each 4.6 us to 8.8, two 6.3 to 8.0, four 9.4 to 7.6.
template <typename T, int V>
hipError_t by_tokens(const patch_kv_append_args& a, const patch_kv_cache& c, hipStream_t s) {
  if (a.T <= 2 * a.S) return go<T, V, 8, 1>(a, c, s);
  if constexpr (V == 1) {
    return go<T, 1, 256, 4>(a, c, s);
  } else {
    const int64_t values = c.page * c.dim / kThreads;  // of a thread
    return values <= 16   ? go<T, V, 256, 8 / V>(a, c, s)
           : values <= 32 ? go<T, V, 256, 16 / V>(a, c, s)
                          : go<T, V, 256, 32 / V>(a, c, s);
  }
}

template <typename T>
hipError_t by_width(const patch_kv_append_args& a, const patch_kv_cache& c, hipStream_t s) {
  uintptr_t p = (uintptr_t)a.k_dev | (uintptr_t)a.v_dev;
  int64_t st = a.k_token | a.k_head | a.v_token | a.v_head;
  if (a.q_dev) {
    p |= (uintptr_t)a.q_dev | (uintptr_t)a.q_out_dev;
    st |= a.q_token | a.q_head | a.q_out_token | a.q_out_head;
  }
  switch (choose_v(a.table_dev ? a.rot : 0, c.dim, st, p, (int)sizeof(T))) {
    case 8: return by_tokens<T, 8>(a, c, s);
    case 4: return by_tokens<T, 4>(a, c, s);
    default: return by_tokens<T, 1>(a, c, s);
  }
}

}  // namespace

hipError_t launch_kv_append(const patch_kv_append_args& a, const patch_kv_cache& c, hipStream_t s) {
  return a.dtype == PATCH_BF16 ? by_width<__bf16>(a, c, s) : by_width<_Float16>(a, c, s);
}

}  // namespace patch
