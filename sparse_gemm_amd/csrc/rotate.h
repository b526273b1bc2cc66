// rotate.h -- loading and rotating a slice of a head, shared by the rotary
// kernel and the cache append.
//
// A head of D elements is cut into D / 2V items of 2V elements, one item a
// thread: an item c < rot / 2V is V pairs (HALF: elements cV.. and rot/2 +
// cV..; INTERLEAVED: 2cV .. 2cV + 2V - 1), a later one 2V elements that pass
// unchanged.  Either way pair i of the head takes entry i of the table row's
// cos half and of its sin half, so an item reads V consecutive floats of each.
// V is 8 where the sizes and addresses allow 16-byte accesses of 16-bit
// elements, else 4, else 1 (choose_v).
#pragma once

#include "layer_common.h"

namespace patch {

template <int V>
struct Item {
  float a[V], b[V];  // first and second element of each pair (rotated items), or elements 0.. and V.. (others)
};

// first element of an item's first and second run of V (pairs) elements
struct ItemPlace {
  int first, second;
  bool turned, interleaved;
};

template <int V>
__device__ __forceinline__ ItemPlace item_place(int c, int rot, bool interleaved) {
  ItemPlace p;
  p.turned = c < rot / (2 * V);
  p.interleaved = interleaved && p.turned;
  if (p.turned && !interleaved) {
    p.first = c * V;
    p.second = rot / 2 + c * V;
  } else {
    p.first = 2 * c * V;
    p.second = p.first + V;
  }
  return p;
}

template <typename T, int V>
__device__ __forceinline__ Item<V> load_item(const T* head, const ItemPlace& p) {
  const Vec<T, V> x = *reinterpret_cast<const Vec<T, V>*>(head + p.first);
  const Vec<T, V> y = *reinterpret_cast<const Vec<T, V>*>(head + p.second);
  Item<V> r;
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < V; i++) {  // pair i = elements 2i, 2i + 1 of the 2V
      const int e = 2 * i, o = 2 * i + 1;
      r.a[i] = (float)(e < V ? x.v[e % V] : y.v[e % V]);
      r.b[i] = (float)(o < V ? x.v[o % V] : y.v[o % V]);
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

template <typename T, int V>
__device__ __forceinline__ void store_item(T* head, const ItemPlace& p, const Item<V>& r) {
  Vec<T, V> x, y;
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int e = 2 * i, o = 2 * i + 1;
      (e < V ? x.v[e % V] : y.v[e % V]) = (T)r.a[i];
      (o < V ? x.v[o % V] : y.v[o % V]) = (T)r.b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) {
      x.v[i] = (T)r.a[i];
      y.v[i] = (T)r.b[i];
    }
  }
  *reinterpret_cast<Vec<T, V>*>(head + p.first) = x;
  *reinterpret_cast<Vec<T, V>*>(head + p.second) = y;
}

template <int V>
struct Angles {
  Vec<float, V> c, s;
};

// The angles of item c from the table row (NULL: a position outside the table, all NaN).
template <int V>
__device__ __forceinline__ Angles<V> load_angles(const float* row, int c, int rot, bool inverse) {
  Angles<V> g;
  if (row) {
    g.c = *reinterpret_cast<const Vec<float, V>*>(row + c * V);
    g.s = *reinterpret_cast<const Vec<float, V>*>(row + rot / 2 + c * V);
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
