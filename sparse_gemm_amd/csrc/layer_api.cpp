// layer_api.cpp -- host side of the decoder-layer operators of the C ABI
// (rotary positions, cache append, attention, 4-bit linear layer): argument
// checks before anything is launched.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "layer_common.h"
#include "patch.h"

namespace patch {
// sets the text patch_last_error() returns on this thread (patch_api.cpp)
patch_status set_last_error(patch_status s, const char* msg);
uint64_t w4_bytes(int64_t N, int64_t K, int64_t G, bool zero);
}  // namespace patch

namespace {

constexpr int64_t kMaxSize = int64_t(1) << 31;  // of any one count or index
constexpr int64_t kMaxW4 = int64_t(1) << 22;    // N and K of a 4-bit weight

patch_status fail(patch_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return patch::set_last_error(s, buf);
}

patch_status launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return PATCH_OK;
  if (e == hipErrorInvalidValue) return fail(PATCH_ERR_SHAPE, "%s: too large for one launch", what);
  return fail(PATCH_ERR_HIP, "launch %s: %s (%d)", what, hipGetErrorString(e), (int)e);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool is16(int64_t dt) { return dt == PATCH_F16 || dt == PATCH_BF16; }

patch_status check_rot(int64_t rot, int64_t D) {
  if (rot < 2 || rot % 2 || rot > D)
    return fail(PATCH_ERR_SHAPE, "rot=%lld must be even, at least 2 and at most %lld", (long long)rot, (long long)D);
  return PATCH_OK;
}

patch_status check_layout(int64_t layout) {
  if (layout != PATCH_ROPE_HALF && layout != PATCH_ROPE_INTERLEAVED)
    return fail(PATCH_ERR_INVALID_ARG, "layout %lld is unknown", (long long)layout);
  return PATCH_OK;
}

patch_status check_cache(const patch_kv_cache* c) {
  if (!c) return fail(PATCH_ERR_INVALID_ARG, "null cache");
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
    return fail(PATCH_ERR_SHAPE, "page=%lld must be 16, 32, 64 or 128", (long long)c->page);
  if (c->dim < 16 || c->dim > 256 || c->dim % 16)
    return fail(PATCH_ERR_SHAPE, "dim=%lld must be a multiple of 16 up to 256", (long long)c->dim);
  if (c->pages < 1 || c->pages >= kMaxSize || c->kv_heads < 1 || c->kv_heads > 4096)
    return fail(PATCH_ERR_SHAPE, "pages=%lld kv_heads=%lld out of range", (long long)c->pages, (long long)c->kv_heads);
  if (!c->k_dev || !c->v_dev || !c->k_scale_dev || !c->v_scale_dev)
    return fail(PATCH_ERR_INVALID_ARG, "null cache pointer");
  if (!aligned(c->k_dev, 16) || !aligned(c->v_dev, 16) || !aligned(c->k_scale_dev, 4) || !aligned(c->v_scale_dev, 4))
    return fail(PATCH_ERR_INVALID_ARG, "cache pointers must be 16-byte and scales 4-byte aligned");
  return PATCH_OK;
}

// What append and attention share: sequences, page tables and head counts.
patch_status check_seqs(int64_t T, int64_t S, int64_t heads, const patch_kv_cache* c, int64_t max_pages, int64_t row,
                        const void* table, const void* lens, const void* cu) {
  if (T < 0 || S < 0) return fail(PATCH_ERR_INVALID_ARG, "T=%lld or S=%lld is negative", (long long)T, (long long)S);
  if (T >= kMaxSize / 2 || S > patch::kMaxSeqs)
    return fail(PATCH_ERR_SHAPE, "T=%lld S=%lld: less than 2^30 tokens and at most %lld sequences", (long long)T, (long long)S,
                (long long)patch::kMaxSeqs);
  if (heads < 1 || heads > 65536 || heads % c->kv_heads)
    return fail(PATCH_ERR_SHAPE, "heads=%lld must be a multiple of kv_heads=%lld", (long long)heads,
                (long long)c->kv_heads);
  if (max_pages < 0 || max_pages * c->page >= kMaxSize || row < max_pages)
    return fail(PATCH_ERR_SHAPE, "max_pages=%lld rows of %lld out of range", (long long)max_pages, (long long)row);
  if (!table || !lens || !cu) return fail(PATCH_ERR_INVALID_ARG, "null page table, lengths or cu_new");
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(cu, 4))
    return fail(PATCH_ERR_INVALID_ARG, "page table, lengths and cu_new must be 4-byte aligned");
  return PATCH_OK;
}

patch_status check_w4(int64_t N, int64_t K, int64_t group) {
  if (group != 32 && group != 64 && group != 128)
    return fail(PATCH_ERR_SHAPE, "group=%lld must be 32, 64 or 128", (long long)group);
  if (N < 1 || K < 1 || N > kMaxW4 || K > kMaxW4 || K % group)
    return fail(PATCH_ERR_SHAPE, "N=%lld K=%lld: positive, at most %lld, K a multiple of the group (%lld)", (long long)N,
                (long long)K, (long long)kMaxW4, (long long)group);
  return PATCH_OK;
}

}  // namespace

extern "C" {

patch_status patch_rope_table(int64_t positions, int64_t rot, double base, int32_t scaling, double factor,
                              double original, double low, double high, double magnitude, float* table_dev,
                              void* stream) {
  if (positions < 1 || rot < 2 || rot % 2 || rot > 65536 || positions >= kMaxSize)
    return fail(PATCH_ERR_SHAPE, "positions=%lld rot=%lld: positive, rot even", (long long)positions, (long long)rot);
  if (!table_dev || !aligned(table_dev, 16)) return fail(PATCH_ERR_INVALID_ARG, "null or unaligned table");
  if (!std::isfinite(base) || !(base > 1.0) || !std::isfinite(magnitude))
    return fail(PATCH_ERR_INVALID_ARG, "base must be above 1 and the magnitude finite");
  switch (scaling) {
    case PATCH_ROPE_UNSCALED: break;
    case PATCH_ROPE_LINEAR:
    case PATCH_ROPE_NTK:
    case PATCH_ROPE_BY_PARTS:
      if (!std::isfinite(factor) || !(factor >= 1.0)) return fail(PATCH_ERR_INVALID_ARG, "factor must be at least 1");
      if (scaling == PATCH_ROPE_NTK && rot < 4) return fail(PATCH_ERR_SHAPE, "this scaling needs rot >= 4");
      if (scaling == PATCH_ROPE_BY_PARTS &&
          (!std::isfinite(original) || !(original > 0.0) || !std::isfinite(low) || !std::isfinite(high) || !(low < high)))
        return fail(PATCH_ERR_INVALID_ARG, "scaling by parts needs original > 0 and low < high");
      break;
    default: return fail(PATCH_ERR_INVALID_ARG, "scaling %d is unknown", (int)scaling);
  }
  return launched(patch::launch_rope_table(positions, (int)rot, base, scaling, factor, original, low, high, magnitude,
                                           table_dev, reinterpret_cast<hipStream_t>(stream)),
                  "rope_table");
}

patch_status patch_rope(const patch_rope_args* a, void* stream) {
  if (!a) return fail(PATCH_ERR_INVALID_ARG, "null arguments");
  patch_status s;
  if (!is16(a->dtype) && a->dtype != PATCH_F32) return fail(PATCH_ERR_INVALID_ARG, "dtype %lld", (long long)a->dtype);
  if ((s = check_layout(a->layout))) return s;
  if (a->T < 0) return fail(PATCH_ERR_INVALID_ARG, "T=%lld is negative", (long long)a->T);
  if (a->T >= kMaxSize || a->H < 1 || a->H >= kMaxSize || a->D < 2 || a->D % 2 || a->D > 65536)
    return fail(PATCH_ERR_SHAPE, "T=%lld H=%lld D=%lld out of range (D even)", (long long)a->T, (long long)a->H,
                (long long)a->D);
  if ((s = check_rot(a->rot, a->D))) return s;
  if (a->context < 1) return fail(PATCH_ERR_INVALID_ARG, "context=%lld: an empty table", (long long)a->context);
  if (a->T == 0) return PATCH_OK;
  if (!a->x_dev || !a->out_dev || !a->positions_dev || !a->table_dev)
    return fail(PATCH_ERR_INVALID_ARG, "null pointer argument");
  const uintptr_t es = a->dtype == PATCH_F32 ? 4 : 2;
  if (!aligned(a->x_dev, es) || !aligned(a->out_dev, es) || !aligned(a->positions_dev, 4) || !aligned(a->table_dev, 16))
    return fail(PATCH_ERR_INVALID_ARG, "misaligned pointer (table: 16 bytes, others their element)");
  if (a->x_dev == a->out_dev && (a->x_token != a->out_token || a->x_head != a->out_head))
    return fail(PATCH_ERR_INVALID_ARG, "in place, x and out need the same strides");
  return launched(patch::launch_rope(*a, reinterpret_cast<hipStream_t>(stream)), "rope");
}

patch_status patch_kv_append(const patch_kv_append_args* a, const patch_kv_cache* c, void* stream) {
  if (!a) return fail(PATCH_ERR_INVALID_ARG, "null arguments");
  patch_status s;
  if (!is16(a->dtype)) return fail(PATCH_ERR_INVALID_ARG, "dtype %lld is not F16 or BF16", (long long)a->dtype);
  if ((s = check_layout(a->layout)) || (s = check_cache(c))) return s;
  if ((s = check_seqs(a->T, a->S, a->q_dev ? a->heads : c->kv_heads, c, a->max_pages, a->page_table_row,
                      a->page_table_dev, a->kv_lens_dev, a->cu_new_dev)))
    return s;
  if (a->table_dev) {
    if ((s = check_rot(a->rot, c->dim))) return s;
    if (a->context < 1) return fail(PATCH_ERR_INVALID_ARG, "context=%lld: an empty table", (long long)a->context);
    if (!aligned(a->table_dev, 16)) return fail(PATCH_ERR_INVALID_ARG, "the rope table must be 16-byte aligned");
  }
  if (a->T == 0 || a->S == 0) return PATCH_OK;
  if (!a->k_dev || !a->v_dev || (a->q_dev && !a->q_out_dev)) return fail(PATCH_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(a->k_dev, 2) || !aligned(a->v_dev, 2) || !aligned(a->q_dev, 2) || !aligned(a->q_out_dev, 2))
    return fail(PATCH_ERR_INVALID_ARG, "misaligned k, v or q");
  if (a->q_dev && a->q_dev == a->q_out_dev && (a->q_token != a->q_out_token || a->q_head != a->q_out_head))
    return fail(PATCH_ERR_INVALID_ARG, "in place, q and q_out need the same strides");
  return launched(patch::launch_kv_append(*a, *c, reinterpret_cast<hipStream_t>(stream)), "kv_append");
}

uint64_t patch_attention_workspace_bytes(int64_t T, int64_t S, int64_t heads, int64_t kv_heads, int64_t dim) {
  if (T <= 0 || S <= 0 || T >= kMaxSize || S > patch::kMaxSeqs || kv_heads < 1 || heads < 1 || heads % kv_heads ||
      heads > 65536 || dim < 16 || dim > 256 || dim % 16)
    return 0;
  return patch::attention_workspace_bytes(T, S, heads, kv_heads, dim);
}

patch_status patch_attention(const patch_attention_args* a, const patch_kv_cache* c, void* workspace_dev,
                             uint64_t workspace_bytes, void* stream) {
  if (!a) return fail(PATCH_ERR_INVALID_ARG, "null arguments");
  patch_status s;
  if (!is16(a->dtype)) return fail(PATCH_ERR_INVALID_ARG, "dtype %lld is not F16 or BF16", (long long)a->dtype);
  if (a->out_dtype != a->dtype && a->out_dtype != PATCH_F32)
    return fail(PATCH_ERR_INVALID_ARG, "out_dtype %lld must equal dtype %lld or be F32", (long long)a->out_dtype,
                (long long)a->dtype);
  if ((s = check_cache(c))) return s;
  if ((s = check_seqs(a->T, a->S, a->heads, c, a->max_pages, a->page_table_row, a->page_table_dev, a->kv_lens_dev,
                      a->cu_new_dev)))
    return s;
  if (!(std::fabs(a->scale) <= 1e30)) return fail(PATCH_ERR_INVALID_ARG, "scale must be finite, at most 1e30 in size");
  if (a->window < 0) return fail(PATCH_ERR_INVALID_ARG, "window=%lld is negative", (long long)a->window);
  if (a->T * (a->heads / c->kv_heads) >= kMaxSize / 2)
    return fail(PATCH_ERR_SHAPE, "T=%lld times %lld heads a cache head is too large", (long long)a->T,
                (long long)(a->heads / c->kv_heads));
  if (workspace_bytes > 0 && (!workspace_dev || !aligned(workspace_dev, 16)))
    return fail(PATCH_ERR_INVALID_ARG, "null or unaligned workspace");
  if (a->T == 0 || a->S == 0) return PATCH_OK;
  if (!a->q_dev || !a->out_dev) return fail(PATCH_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(a->q_dev, 2) || !aligned(a->out_dev, a->out_dtype == PATCH_F32 ? 4 : 2) || !aligned(a->lse_dev, 4))
    return fail(PATCH_ERR_INVALID_ARG, "misaligned q, out or lse");
  return launched(patch::launch_attention(*a, *c, workspace_dev, workspace_bytes, reinterpret_cast<hipStream_t>(stream)),
                  "attention");
}

uint64_t patch_w4_bytes(int64_t N, int64_t K, int64_t group, int32_t with_zero) {
  return check_w4(N, K, group) ? 0 : patch::w4_bytes(N, K, group, with_zero != 0);
}

patch_status patch_w4_quantize(patch_dtype dtype, int64_t N, int64_t K, int64_t group, const void* W_dev,
                               uint8_t* q_dev, void* scale_dev, uint8_t* zero_dev, void* stream) {
  patch_status s;
  if (!is16(dtype)) return fail(PATCH_ERR_INVALID_ARG, "dtype %d is not F16 or BF16", (int)dtype);
  if ((s = check_w4(N, K, group))) return s;
  if (!W_dev || !q_dev || !scale_dev) return fail(PATCH_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(W_dev, 2) || !aligned(scale_dev, 2)) return fail(PATCH_ERR_INVALID_ARG, "misaligned W or scale");
  return launched(patch::launch_w4_quantize(dtype == PATCH_BF16, N, K, (int)group, W_dev, q_dev, scale_dev, zero_dev,
                                            reinterpret_cast<hipStream_t>(stream)),
                  "w4_quantize");
}

patch_status patch_w4_pack(patch_dtype dtype, int64_t N, int64_t K, int64_t group, const uint8_t* q_dev,
                           const void* scale_dev, const uint8_t* zero_dev, void* packed_dev, uint64_t packed_bytes,
                           void* stream) {
  patch_status s;
  if (!is16(dtype)) return fail(PATCH_ERR_INVALID_ARG, "dtype %d is not F16 or BF16", (int)dtype);
  if ((s = check_w4(N, K, group))) return s;
  if (!q_dev || !scale_dev || !packed_dev) return fail(PATCH_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q_dev, 4) || !aligned(scale_dev, 2) || !aligned(packed_dev, 16))
    return fail(PATCH_ERR_INVALID_ARG, "q must be 4-byte, scale 2-byte and packed 16-byte aligned");
  if (packed_bytes < patch::w4_bytes(N, K, group, zero_dev != nullptr))
    return fail(PATCH_ERR_BUFFER_TOO_SMALL, "packed buffer of %llu bytes is too small", (unsigned long long)packed_bytes);
  return launched(patch::launch_w4_pack(N, K, (int)group, q_dev, scale_dev, zero_dev,
                                        reinterpret_cast<uint8_t*>(packed_dev), reinterpret_cast<hipStream_t>(stream)),
                  "w4_pack");
}

patch_status patch_w4_gemm(patch_dtype dtype, int64_t N, int64_t K, int64_t group, int32_t with_zero,
                           const void* packed_dev, uint64_t packed_bytes, const void* X_dev, int64_t M, void* Y_dev,
                           patch_dtype y_dtype, void* stream) {
  patch_status s;
  if (!is16(dtype)) return fail(PATCH_ERR_INVALID_ARG, "dtype %d is not F16 or BF16", (int)dtype);
  if (y_dtype != dtype && y_dtype != PATCH_F32)
    return fail(PATCH_ERR_INVALID_ARG, "y_dtype %d must equal the input dtype %d or be F32", (int)y_dtype, (int)dtype);
  if ((s = check_w4(N, K, group))) return s;
  if (M < 0) return fail(PATCH_ERR_INVALID_ARG, "M=%lld is negative", (long long)M);
  if (M == 0) return PATCH_OK;
  if (!packed_dev || !X_dev || !Y_dev) return fail(PATCH_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(packed_dev, 16) || !aligned(X_dev, 16) || !aligned(Y_dev, 16))
    return fail(PATCH_ERR_INVALID_ARG, "packed, X and Y must be 16-byte aligned");
  if (packed_bytes < patch::w4_bytes(N, K, group, with_zero != 0))
    return fail(PATCH_ERR_BUFFER_TOO_SMALL, "packed buffer of %llu bytes is too small", (unsigned long long)packed_bytes);
  return launched(patch::launch_w4_gemm(dtype == PATCH_BF16, y_dtype == PATCH_F32, with_zero != 0, N, K, (int)group,
                                        reinterpret_cast<const uint8_t*>(packed_dev), X_dev, M, Y_dev,
                                        reinterpret_cast<hipStream_t>(stream)),
                  "w4_gemm");
}

}  // extern "C"
