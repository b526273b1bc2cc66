// rotate.h -- loading and rotating a slice of a head, shared by the rotary
// kernel and the cache append.
//
// A head of D elements is cut into D / 2V items of 2V elements, one item a
// thread, in two runs of V: the c-th run of the first half and of the second
// half of the rotated elements, or of those behind them, which pass unchanged.
// So neighbouring threads read neighbouring runs, in either layout.  HALF:
// the runs are the two elements of V pairs; INTERLEAVED: each holds V / 2
// pairs (V = 1: the runs are neighbours, one pair).  V is 8 where sizes and
// addresses allow 16-byte accesses of 16-bit elements, else 4, else 1
// (choose_v).
#pragma once

#include "layer_common.h"

namespace patch {

template <int V>
struct Item {
  float a[V], b[V];  // first and second element of each pair (rotated items), or the two runs (others)
};

// Where an item's runs begin, and its first pair and that of its second run's.
struct ItemPlace {
  int first, second, pair0, pair1;
  bool turned, interleaved;
};

template <int V>
__device__ __forceinline__ ItemPlace item_place(int c, int rot, int D, bool interleaved) {
  ItemPlace p;
  const int turning = rot / (2 * V);
  p.turned = c < turning;
  p.interleaved = interleaved && p.turned;
  const int from = p.turned ? 0 : rot, size = p.turned ? rot : D - rot, i = p.turned ? c : c - turning;
  p.first = from + i * V;
  p.second = p.first + size / 2;
  p.pair0 = p.pair1 = c * V;
  if (p.interleaved) {
    if constexpr (V == 1) {
      p.first = 2 * c;
      p.second = 2 * c + 1;
    } else {
      p.pair0 = p.first / 2;
      p.pair1 = p.second / 2;
    }
  }
  return p;
}

template <typename T, int V>
__device__ __forceinline__ Item<V> load_item(const T* head, const ItemPlace& p) {
  const Vec<T, V> x = *reinterpret_cast<const Vec<T, V>*>(head + p.first);
  const Vec<T, V> y = *reinterpret_cast<const Vec<T, V>*>(head + p.second);
  Item<V> r;
  if (V > 1 && p.interleaved) {
#pragma unroll
    for (int i = 0; i < V / 2; i++) {
      r.a[i] = (float)x.v[2 * i];
      r.b[i] = (float)x.v[2 * i + 1];
      r.a[V / 2 + i] = (float)y.v[2 * i];
      r.b[V / 2 + i] = (float)y.v[2 * i + 1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) {
      r.a[i] = (float)x.v[i];
      r.b[i] = (float)y.v[i];
    }
  }
  return r;
}

// An item's two runs of values.
template <int V>
__device__ __forceinline__ void runs_of(const ItemPlace& p, const Item<V>& r, float (&x)[V], float (&y)[V]) {
  if (V > 1 && p.interleaved) {
#pragma unroll
    for (int i = 0; i < V / 2; i++) {
      x[2 * i] = r.a[i];
      x[2 * i + 1] = r.b[i];
      y[2 * i] = r.a[V / 2 + i];
      y[2 * i + 1] = r.b[V / 2 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) {
      x[i] = r.a[i];
      y[i] = r.b[i];
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_item(T* head, const ItemPlace& p, const Item<V>& r) {
  float x[V], y[V];
  runs_of(p, r, x, y);
  Vec<T, V> u, w;
#pragma unroll
  for (int i = 0; i < V; i++) {
    u.v[i] = (T)x[i];
    w.v[i] = (T)y[i];
  }
  *reinterpret_cast<Vec<T, V>*>(head + p.first) = u;
  *reinterpret_cast<Vec<T, V>*>(head + p.second) = w;
}

template <int V>
struct Angles {
  Vec<float, V> c, s;
};

// The angles of an item's pairs from the table row (NULL: a position outside the table, all NaN).
template <int V>
__device__ __forceinline__ Angles<V> load_angles(const float* row, const ItemPlace& p, int rot, bool inverse) {
  Angles<V> g;
  if (row) {
    if constexpr (V == 1) {
      g.c.v[0] = row[p.pair0];
      g.s.v[0] = row[rot / 2 + p.pair0];
    } else {  // V / 2 at either place; in the half layout they are neighbours
      using H = Vec<float, V / 2>;
      const int p1 = p.interleaved ? p.pair1 : p.pair0 + V / 2;
      const H c0 = *reinterpret_cast<const H*>(row + p.pair0), c1 = *reinterpret_cast<const H*>(row + p1);
      const H s0 = *reinterpret_cast<const H*>(row + rot / 2 + p.pair0), s1 = *reinterpret_cast<const H*>(row + rot / 2 + p1);
#pragma unroll
      for (int i = 0; i < V / 2; i++) {
        g.c.v[i] = c0.v[i];
        g.c.v[V / 2 + i] = c1.v[i];
        g.s.v[i] = s0.v[i];
        g.s.v[V / 2 + i] = s1.v[i];
      }
    }
    if (inverse) {
#pragma unroll
      for (int i = 0; i < V; i++) g.s.v[i] = -g.s.v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) g.c.v[i] = g.s.v[i] = __builtin_nanf("");
  }
  return g;
}

template <int V>
__device__ __forceinline__ void turn(Item<V>& r, const Angles<V>& g) {
#pragma unroll
  for (int i = 0; i < V; i++) {
    const float a = r.a[i], b = r.b[i];
    r.a[i] = a * g.c.v[i] - b * g.s.v[i];
    r.b[i] = b * g.c.v[i] + a * g.s.v[i];
  }
}

// The widest V whose accesses are aligned: `all` is the bitwise or of every
// size and stride in elements, addresses the or of the base addresses, es the
// element size.  A V of 1 asks for even rot and D only.
inline int choose_v(int64_t rot, int64_t D, int64_t strides_or, uintptr_t addresses_or, int es) {
  for (int v : {8, 4})
    if (rot % (2 * v) == 0 && D % (2 * v) == 0 && strides_or % v == 0 && addresses_or % (uintptr_t)(v * es) == 0)
      return v;
  return 1;
}

}  // namespace patch
