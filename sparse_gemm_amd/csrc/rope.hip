// rope.hip -- rotary positions: the table of cos and sin, and the rotation.
//
// k_rope: (a, b) -> (a cos - b sin, b cos + a sin) per pair, in fp32.  It
// reads and writes every element once and is bound by HBM; a token's table
// row (4 rot bytes) is shared by its heads, so a thread keeps its item's
// angles in registers and walks over several heads.
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

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void k_rope(patch_rope_args a, uint32_t threads, uint32_t items, int heads_each) {
  const uint32_t e = blockIdx.x * kThreads + threadIdx.x;
  if (e >= threads) return;
  const uint32_t t = e / items, c = e - t * items;
  const int rot = (int)a.rot;
  const ItemPlace p = item_place<V>((int)c, rot, (int)a.D, a.layout == PATCH_ROPE_INTERLEAVED);
  const T* x = reinterpret_cast<const T*>(a.x_dev) + (int64_t)t * a.x_token;
  T* o = reinterpret_cast<T*>(a.out_dev) + (int64_t)t * a.out_token;
  Angles<V> g;
  if (p.turned) {
    const int pos = a.positions_dev[t];
    g = load_angles<V>(pos >= 0 && pos < a.context ? a.table_dev + (int64_t)pos * rot : nullptr, p, rot,
                       a.inverse != 0);
  } else if (a.x_dev == a.out_dev) {
    return;  // in place: the elements behind rot are there already
  }
  const int h1 = min((int)a.H, ((int)blockIdx.y + 1) * heads_each);
#pragma unroll 4
  for (int h = (int)blockIdx.y * heads_each; h < h1; h++) {
    Item<V> r = load_item<T, V>(x + h * a.x_head, p);
    if (p.turned) turn(r, g);
    store_item<T, V>(o + h * a.out_head, p, r);
  }
}

template <typename T, int V>
hipError_t go(const patch_rope_args& a, hipStream_t s) {
  const uint64_t items = (uint64_t)a.D / (2 * V), threads = items * (uint64_t)a.T;
  if (threads > 0x7fffffffull) return hipErrorInvalidValue;
  const uint32_t blocks = (uint32_t)((threads + kThreads - 1) / kThreads);
  // heads of one thread: as many as leave 2048 workgroups (8 a CU), at most 8
  int64_t each = std::max<int64_t>(1, std::min<int64_t>(8, (int64_t)blocks * a.H / 2048));
  each = std::max(each, (a.H + 65534) / 65535);
  const dim3 grid(blocks, (unsigned)((a.H + each - 1) / each));
  hipLaunchKernelGGL((k_rope<T, V>), grid, dim3(kThreads), 0, s, a, (uint32_t)threads, (uint32_t)items, (int)each);
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
