// layer_common.h -- argument structures and device helpers shared by the
// decoder-layer kernels (rotary positions, cache append, attention, 4-bit
// linear layer) and their host side.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "patch.h"

namespace patch {

// ---- launches (each kernel file) ----
hipError_t launch_rope_table(int64_t positions, int rot, double base, int scaling, double factor, double original,
                             double low, double high, double magnitude, float* table, hipStream_t s);
hipError_t launch_rope(const patch_rope_args& a, hipStream_t s);
hipError_t launch_kv_append(const patch_kv_append_args& a, const patch_kv_cache& c, hipStream_t s);
uint64_t attention_workspace_bytes(int64_t T, int64_t S, int64_t heads, int64_t kv_heads, int64_t dim);
hipError_t launch_attention(const patch_attention_args& a, const patch_kv_cache& c, void* ws, uint64_t ws_bytes,
                            hipStream_t s);
hipError_t launch_w4_quantize(bool bf16, int64_t N, int64_t K, int group, const void* W, uint8_t* q, void* scale,
                              uint8_t* zero, hipStream_t s);
hipError_t launch_w4_pack(int64_t N, int64_t K, int group, const uint8_t* q, const void* scale, const uint8_t* zero,
                          uint8_t* packed, hipStream_t s);
hipError_t launch_w4_gemm(bool bf16, bool out_f32, bool zero, int64_t N, int64_t K, int group, const uint8_t* packed,
                          const void* X, int64_t M, void* Y, hipStream_t s);

constexpr int64_t kMaxSeqs = 4096;  // attention keeps a sum per sequence in LDS

// ---- device helpers ----
#if defined(__HIP__)

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

// The largest index i in [0, n) with base(i) <= x, for base not decreasing
// and base(0) <= x; called by whole waves with the same x.  Each step looks
// at 64 places at once, so 4096 sequences take two dependent loads.  Any
// contents of base end with an index in [0, n).
template <typename F>
__device__ __forceinline__ int find_last(int n, F base_le) {
  const int lane = (int)(threadIdx.x & 63);
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) >> 6;
    const int i = lo + lane * step;
    const uint64_t m = __ballot(i < hi && base_le(i));
    const int c = m ? 63 - __builtin_clzll(m) : 0;
    lo += c * step;
    hi = min(hi, lo + step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

#endif  // __HIP__

}  // namespace patch
