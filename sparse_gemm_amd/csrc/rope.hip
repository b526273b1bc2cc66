// rope.hip -- rotary positions: the table of cos and sin, and the rotation.
//
// k_rope: (a, b) -> (a cos - b sin, b cos + a sin) per pair, in fp32.  It
// reads and writes every element once and is bound by HBM: 340 MB (16383
// tokens, 40 heads of 128, fp16) in 61 us, 5.5 TB/s, where a copy of 1 GiB
// reaches 5.1.
#include <algorithm>

#include "rotate.h"

namespace patch {
namespace {

constexpr int kThreads = 256;

// One thread a pair, walking down the positions: its frequency is computed
// once.  64-bit arithmetic throughout: at position 10^6 an fp32 angle would
// be off by 0.06.
__global__ __launch_bounds__(kThreads) void k_rope_table(int64_t positions, int rot, double base, int scaling,
                                                         double factor, double original, double low, double high,
                                                         double magnitude, float* __restrict__ table) {
  const int half = rot / 2;
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double e = -2.0 * i / rot;
    double f = pow(base, e);
    if (scaling == PATCH_ROPE_LINEAR) f /= factor;
    if (scaling == PATCH_ROPE_NTK) f *= pow(factor, e * rot / (rot - 2.0));
    if (scaling == PATCH_ROPE_BY_PARTS) {
      const double r = original * f / 6.283185307179586476925286766559;
      const double g = fmin(1.0, fmax(0.0, (r - low) / (high - low)));
      f = g * f + (1.0 - g) * (f / factor);
    }
    for (int64_t p = blockIdx.x; p < positions; p += gridDim.x) {
      double s, c;
      sincos((double)p * f, &s, &c);
      table[p * rot + i] = (float)(magnitude * c);
      table[p * rot + half + i] = (float)(magnitude * s);
    }
  }
}

// A thread has item c of head h (and h + step, ...) of one token; neighbouring
// threads have neighbouring items, then heads, so that a wave reads in one run.
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void k_rope(patch_rope_args a, uint32_t threads, uint32_t items, uint32_t step) {
  const uint32_t e = blockIdx.x * kThreads + threadIdx.x;
  if (e >= threads) return;
  const uint32_t u = e / items, c = e - u * items, t = u / step, h0 = u - t * step;
  const int rot = (int)a.rot;
  const ItemPlace p = item_place<V>((int)c, rot, (int)a.D, a.layout == PATCH_ROPE_INTERLEAVED);
  const T* x = reinterpret_cast<const T*>(a.x_dev) + (int64_t)t * a.x_token;
  T* o = reinterpret_cast<T*>(a.out_dev) + (int64_t)t * a.out_token;
  Angles<V> g;
  if (p.turned) {
    const int pos = a.positions_dev[t];
    g = load_angles<V>(pos >= 0 && pos < a.context ? a.table_dev + (int64_t)pos * rot : nullptr, p, rot, a.inverse != 0);
  } else if (a.x_dev == a.out_dev) {
    return;  // in place: the elements behind rot are there already
  }
  for (int64_t h = h0; h < a.H; h += step) {
    Item<V> r = load_item<T, V>(x + h * a.x_head, p);
    if (p.turned) turn(r, g);
    store_item<T, V>(o + h * a.out_head, p, r);
  }
}

template <typename T, int V>
hipError_t go(const patch_rope_args& a, hipStream_t s) {
  const uint64_t items = (uint64_t)a.D / (2 * V);
  // One head a thread; all of a token's heads only where that would be too many
  // threads.  Sharing the angles of a token between 2, 4 or 8 heads of a thread
  // saves nothing (they come from L1) and costs runs of that many times fewer
  // bytes: 16383 x 40 heads of 128, 61 us with one, 71, 75 and 79.
  uint64_t step = (uint64_t)a.H, threads = items * (uint64_t)a.T * step;
  if (threads > 0x7fffffffull) {
    step = 1;
    threads = items * (uint64_t)a.T;
    if (threads > 0x7fffffffull) return hipErrorInvalidValue;
  }
  hipLaunchKernelGGL((k_rope<T, V>), dim3((unsigned)((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, a,
                     (uint32_t)threads, (uint32_t)items, (uint32_t)step);
  return hipGetLastError();
}

template <typename T>
hipError_t by_width(const patch_rope_args& a, hipStream_t s) {
  const uintptr_t p = (uintptr_t)a.x_dev | (uintptr_t)a.out_dev;
  switch (choose_v(a.rot, a.D, a.x_token | a.x_head | a.out_token | a.out_head, p, (int)sizeof(T))) {
    case 8: return go<T, 8>(a, s);
    case 4: return go<T, 4>(a, s);
    default: return go<T, 1>(a, s);
  }
}

}  // namespace

hipError_t launch_rope_table(int64_t positions, int rot, double base, int scaling, double factor, double original,
                             double low, double high, double magnitude, float* table, hipStream_t s) {
  const unsigned blocks = (unsigned)std::min<int64_t>(positions, 4096);
  hipLaunchKernelGGL(k_rope_table, dim3(blocks), dim3(kThreads), 0, s, positions, rot, base, scaling, factor, original,
                     low, high, magnitude, table);
  return hipGetLastError();
}

hipError_t launch_rope(const patch_rope_args& a, hipStream_t s) {
  switch (a.dtype) {
    case PATCH_F16: return by_width<_Float16>(a, s);
    case PATCH_BF16: return by_width<__bf16>(a, s);
    default: return by_width<float>(a, s);
  }
}

}  // namespace patch
