// paged_api.cu -- the C ABI of the packed and paged entry points: argument
// validation on the host, before any launch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "extkv.h"
#include "internal.h"
#include "paged.h"

namespace extkv {
namespace {

int fail(int code, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  set_error(msg);
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(EXTKV_ERR_CUDA, "%s: CUDA error %d (%s)", what, static_cast<int>(e), cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool valid_dtype(int dtype) { return dtype == EXTKV_F32 || dtype == EXTKV_BF16; }
int64_t elem_size(int dtype) { return dtype == EXTKV_F32 ? 4 : 2; }

// Products of sizes below stay far from 2^63 for sizes up to this.
constexpr int64_t kMaxCount = 0x7fffff00;  // rows, sequences, pages, slots
constexpr int64_t kMaxHeads = 1 << 16;

int check_heads(const char* who, int64_t Hq, int64_t Hkv, int64_t D, int dtype) {
  if (!valid_dtype(dtype)) return fail(EXTKV_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
  if (Hq <= 0 || Hkv <= 0 || D <= 0)
    return fail(EXTKV_ERR_INVALID_ARG, "%s: bad sizes Hq=%lld Hkv=%lld D=%lld", who, (long long)Hq, (long long)Hkv,
                (long long)D);
  if (Hq > kMaxHeads || Hkv > kMaxHeads)
    return fail(EXTKV_ERR_UNSUPPORTED, "%s: more than %lld heads", who, (long long)kMaxHeads);
  return EXTKV_OK;
}

int check_attention(const char* who, int64_t Hq, int64_t Hkv, int64_t D, float scale) {
  if (Hq % Hkv)
    return fail(EXTKV_ERR_INVALID_ARG, "%s: Hq=%lld is not a multiple of Hkv=%lld", who, (long long)Hq, (long long)Hkv);
  if (D % 8 || D > 512)
    return fail(EXTKV_ERR_UNSUPPORTED, "%s: D=%lld unsupported (need D %% 8 == 0, D <= 512)", who, (long long)D);
  if (!(scale > 0.f) || std::isinf(scale))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: scale must be finite and positive", who);
  return EXTKV_OK;
}

int check_row_bytes(const char* who, int64_t D, int dtype) {
  if ((D * elem_size(dtype)) % 16 || D > 512)
    return fail(EXTKV_ERR_UNSUPPORTED, "%s: D=%lld unsupported (need D*sizeof(T) a multiple of 16, D <= 512)", who,
                (long long)D);
  return EXTKV_OK;
}

int check_stride(const char* who, const char* name, int64_t stride, int64_t row, int dtype) {
  if (stride < row || (stride * elem_size(dtype)) % 16 || stride > (int64_t(1) << 32))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: %s=%lld (need at least %lld elements and a multiple of 16 bytes)", who, name,
                (long long)stride, (long long)row);
  return EXTKV_OK;
}

int check_pages(const char* who, int64_t Hkv, int64_t num_pages, int64_t page_size, int64_t max_pages) {
  if (num_pages <= 0 || page_size <= 0 || max_pages < 0)
    return fail(EXTKV_ERR_INVALID_ARG, "%s: bad sizes num_pages=%lld page_size=%lld max_pages=%lld", who,
                (long long)num_pages, (long long)page_size, (long long)max_pages);
  if (num_pages > kMaxCount || page_size > kMaxCount || max_pages > kMaxCount || max_pages * page_size > kMaxCount ||
      num_pages * page_size > 0xfffffffell / Hkv)
    return fail(EXTKV_ERR_UNSUPPORTED,
                "%s: num_pages*Hkv*page_size must be below 2^32 - 1 and max_pages*page_size at most 2^31 - 256", who);
  return EXTKV_OK;
}

int check_rotary(const char* who, const extkv_rotary* r, int64_t D) {
  if (r->n_axes < 1 || r->n_axes > 4)
    return fail(EXTKV_ERR_INVALID_ARG, "%s: n_axes=%d outside [1, 4]", who, r->n_axes);
  if (r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > D)
    return fail(EXTKV_ERR_INVALID_ARG, "%s: rotary_dim=%d (need an even number in [2, D=%lld])", who, r->rotary_dim,
                (long long)D);
  int64_t sum = 0;
  for (int i = 0; i < r->n_axes; ++i) {
    if (r->sections[i] < 0) return fail(EXTKV_ERR_INVALID_ARG, "%s: negative section", who);
    sum += r->sections[i];
  }
  if (sum != r->rotary_dim / 2)
    return fail(EXTKV_ERR_INVALID_ARG, "%s: sections sum to %lld, not rotary_dim/2=%d", who, (long long)sum,
                r->rotary_dim / 2);
  if (!r->positions || !r->inv_freq) return fail(EXTKV_ERR_INVALID_ARG, "%s: null positions or inv_freq", who);
  if (!aligned(r->positions, 8) || !aligned(r->inv_freq, 4))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: misaligned positions or inv_freq", who);
  return EXTKV_OK;
}

int check_workspace(const char* who, const void* ws, size_t bytes, size_t need) {
  if (bytes < need || (need && !ws))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: workspace of %zu bytes required (got %zu); query %s_workspace_size", who, need,
                bytes, who);
  if (!aligned(ws, 256)) return fail(EXTKV_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  return EXTKV_OK;
}

RowTensor bnsh(const void* src, void* dst, int64_t H, int64_t S, int64_t D) {
  return RowTensor{src, dst, H * S * D, D, S * D, H * S * D, D, S * D, static_cast<int>(src ? H : 0)};
}

}  // namespace
}  // namespace extkv

using namespace extkv;

extern "C" {

int rotary_multi_axis(void* q_out, void* k_out, const void* q, const void* k, const extkv_rotary* rotary, int64_t B,
                      int64_t Hq, int64_t Hkv, int64_t S, int64_t D, int dtype, void* stream) {
  static const char who[] = "rotary_multi_axis";
  set_error("");
  if (int rc = check_heads(who, Hq, Hkv, D, dtype)) return rc;
  if (int rc = check_row_bytes(who, D, dtype)) return rc;
  if (B < 0 || S < 0 || B > kMaxCount || S > kMaxCount || (B > 0 && S > kMaxCount / B))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: bad sizes B=%lld S=%lld", who, (long long)B, (long long)S);
  if (!rotary) return fail(EXTKV_ERR_INVALID_ARG, "%s: null rotary", who);
  if (B == 0 || S == 0) return EXTKV_OK;
  if (int rc = check_rotary(who, rotary, D)) return rc;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: an input without its output, or an output without its input", who);
  if (!q && !k) return EXTKV_OK;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  RotaryArgs a{};
  a.q = bnsh(q, q_out, Hq, S, D);
  a.k = bnsh(k, k_out, Hkv, S, D);
  a.B = B;
  a.S = S;
  a.D = D;
  a.rotary = rotary;
  a.dtype = dtype;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_rotary(a);
  return e == cudaSuccess ? EXTKV_OK : cuda_fail(e, "rotary_multi_axis launch");
}

int paged_kv_append(void* k_pages, void* v_pages, const void* k_new, const void* v_new, const int64_t* page_table,
                    const int64_t* write_idx, const int64_t* cu_seqlens, void* q_out, const void* q,
                    const extkv_rotary* rotary, int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                    int64_t num_pages, int64_t page_size, int64_t max_pages, int64_t q_stride, int64_t k_stride,
                    int64_t v_stride, int dtype, int32_t* status, void* stream) {
  static const char who[] = "paged_kv_append";
  set_error("");
  if (int rc = check_heads(who, q ? Hq : 1, Hkv, D, dtype)) return rc;
  if (int rc = check_row_bytes(who, D, dtype)) return rc;
  if (T < 0 || B < 0 || T > kMaxCount || B > kMaxCount)
    return fail(EXTKV_ERR_INVALID_ARG, "%s: bad sizes T=%lld B=%lld", who, (long long)T, (long long)B);
  if (!cu_seqlens && T != B)
    return fail(EXTKV_ERR_INVALID_ARG, "%s: without cu_seqlens there is one row per sequence (T=%lld, B=%lld)", who,
                (long long)T, (long long)B);
  if (int rc = check_pages(who, Hkv, num_pages, page_size, max_pages)) return rc;
  if ((q == nullptr) != (q_out == nullptr))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: q and q_out must be given together", who);
  if (q && !rotary) return fail(EXTKV_ERR_INVALID_ARG, "%s: q is rotated; it needs rotary", who);
  if (T == 0 || B == 0) return EXTKV_OK;
  if (rotary)
    if (int rc = check_rotary(who, rotary, D)) return rc;
  if (!k_pages || !v_pages || !k_new || !v_new || !write_idx || (max_pages > 0 && !page_table))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: null pointer", who);
  if (int rc = check_stride(who, "k_stride", k_stride, Hkv * D, dtype)) return rc;
  if (int rc = check_stride(who, "v_stride", v_stride, Hkv * D, dtype)) return rc;
  if (q)
    if (int rc = check_stride(who, "q_stride", q_stride, Hq * D, dtype)) return rc;
  if (q && q == q_out && q_stride != Hq * D)
    return fail(EXTKV_ERR_INVALID_ARG, "%s: q_out is dense; rotating in place needs a dense q", who);
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q, 16) ||
      !aligned(q_out, 16) || !aligned(page_table, 8) || !aligned(write_idx, 8) || !aligned(cu_seqlens, 8) ||
      !aligned(status, 4))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  RotaryArgs a{};
  a.q = RowTensor{q, q_out, 0, q_stride, D, 0, Hq * D, D, static_cast<int>(q ? Hq : 0)};
  a.k = RowTensor{k_new, k_pages, 0, k_stride, D, 0, 0, page_size * D, static_cast<int>(Hkv)};
  a.v = RowTensor{v_new, v_pages, 0, v_stride, D, 0, 0, page_size * D, static_cast<int>(Hkv)};
  a.B = 1;
  a.S = T;
  a.D = D;
  a.rotary = rotary;
  a.paged = 1;
  a.page_table = page_table;
  a.write_idx = write_idx;
  a.cu_seqlens = cu_seqlens;
  a.n_seqs = B;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.dtype = dtype;
  a.status = status;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_rotary(a);
  return e == cudaSuccess ? EXTKV_OK : cuda_fail(e, "paged_kv_append launch");
}

size_t attention_paged_decode_workspace_size(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int dtype) {
  if (!valid_dtype(dtype) || B <= 0 || B > kMaxCount || Hq <= 0 || Hkv <= 0 || Hq % Hkv || D <= 0 || D > 512) return 0;
  return paged_decode_workspace_bytes(B, Hq, Hkv, D, dtype);
}

int attention_paged_decode(void* y, const void* q, const void* k_pages, const void* v_pages, const int64_t* page_table,
                           const int64_t* nonpad, float scale, int32_t window, int64_t B, int64_t Hq, int64_t Hkv,
                           int64_t D, int64_t num_pages, int64_t page_size, int64_t max_pages, int64_t q_stride,
                           int dtype, void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  static const char who[] = "attention_paged_decode";
  set_error("");
  if (int rc = check_heads(who, Hq, Hkv, D, dtype)) return rc;
  if (int rc = check_attention(who, Hq, Hkv, D, scale)) return rc;
  if (B < 0 || B > kMaxCount / Hq) return fail(EXTKV_ERR_INVALID_ARG, "%s: bad size B=%lld", who, (long long)B);
  if (int rc = check_pages(who, Hkv, num_pages, page_size, max_pages)) return rc;
  if (B == 0) return EXTKV_OK;
  if (!y || !q || !k_pages || !v_pages || !nonpad || (max_pages > 0 && !page_table))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: null pointer", who);
  if (int rc = check_stride(who, "q_stride", q_stride, Hq * D, dtype)) return rc;
  if (!aligned(y, 16) || !aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(page_table, 8) ||
      !aligned(nonpad, 8) || !aligned(status, 4))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  if (int rc = check_workspace(who, workspace, ws_bytes, paged_decode_workspace_bytes(B, Hq, Hkv, D, dtype))) return rc;
  PagedDecodeArgs a{y,      q,         k_pages,   v_pages,  page_table, nonpad,    scale,  window, B, Hq, Hkv, D,
                    num_pages, page_size, max_pages, q_stride, dtype,      workspace, status, static_cast<cudaStream_t>(stream),
                    wait_limit_setting(),
                    algo_setting() == EXTKV_ALGO_DECODE_STREAMK   ? kDecodeStreamK
                    : algo_setting() == EXTKV_ALGO_DECODE_CLUSTER ? kDecodeCluster
                                                                  : kDecodeAuto};
  const char* name = "";
  note_launches(0);
  const cudaError_t e = launch_paged_decode(a, &name);
  if (e == cudaErrorNotSupported)
    return fail(EXTKV_ERR_UNSUPPORTED, "%s: the cluster kernel cannot run this shape/type", who);
  if (e != cudaSuccess) return cuda_fail(e, "attention_paged_decode launch");
  note_last_call(name);
  return EXTKV_OK;
}

size_t attention_packed_prefill_workspace_size(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int dtype) {
  if (!valid_dtype(dtype) || T <= 0 || T > kMaxCount || B <= 0 || B > kMaxCount || Hq <= 0 || Hkv <= 0 || Hq % Hkv ||
      D <= 0 || D > 512)
    return 0;
  return packed_workspace_bytes(T, B, Hq, Hkv, D, dtype);
}

int attention_packed_prefill(void* y, const void* q, const void* k, const void* v, const int64_t* cu_seqlens,
                             float scale, int32_t causal, int32_t window, int64_t T, int64_t B, int64_t Hq, int64_t Hkv,
                             int64_t D, int64_t q_stride, int64_t k_stride, int64_t v_stride, int dtype,
                             void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  static const char who[] = "attention_packed_prefill";
  set_error("");
  if (int rc = check_heads(who, Hq, Hkv, D, dtype)) return rc;
  if (int rc = check_attention(who, Hq, Hkv, D, scale)) return rc;
  if (T < 0 || B < 0) return fail(EXTKV_ERR_INVALID_ARG, "%s: bad sizes T=%lld B=%lld", who, (long long)T, (long long)B);
  // rows, and query tiles of the list, are counted in 32 bits
  if (T > kMaxCount || B > kMaxCount || T + B > kMaxCount)
    return fail(EXTKV_ERR_UNSUPPORTED, "%s: T + B must be at most 2^31 - 256", who);
  if (T == 0 || B == 0) return EXTKV_OK;
  if (!y || !q || !k || !v || !cu_seqlens) return fail(EXTKV_ERR_INVALID_ARG, "%s: null pointer", who);
  if (int rc = check_stride(who, "q_stride", q_stride, Hq * D, dtype)) return rc;
  if (int rc = check_stride(who, "k_stride", k_stride, Hkv * D, dtype)) return rc;
  if (int rc = check_stride(who, "v_stride", v_stride, Hkv * D, dtype)) return rc;
  if (!aligned(y, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(cu_seqlens, 8) ||
      !aligned(status, 4))
    return fail(EXTKV_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  if (int rc = check_workspace(who, workspace, ws_bytes, packed_workspace_bytes(T, B, Hq, Hkv, D, dtype))) return rc;
  PackedArgs a{y,   q, k,  v,   cu_seqlens, scale,    causal,   window,   T,     B,
               Hq,  Hkv, D, q_stride, k_stride, v_stride, dtype, workspace, status, static_cast<cudaStream_t>(stream),
               wait_limit_setting()};
  const char* name = "";
  note_launches(0);
  const cudaError_t e = launch_packed(a, &name);
  if (e != cudaSuccess) return cuda_fail(e, "attention_packed_prefill launch");
  note_last_call(name);
  return EXTKV_OK;
}

}  // extern "C"
