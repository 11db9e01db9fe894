// C ABI of the serving operators (declared in include/pulsar_serving.h):
// host-side argument validation, workspace carving and kernel launches, by
// the rules of api.cu.
#include <cmath>

#include "serving.h"
#include "../../include/pulsar_testing.h"

using namespace pa;

namespace {

constexpr uint64_t kWaitLimitNs = 1000000000ull;   // of every bounded device wait

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr || !aligned(ws, kAlign) || ws_bytes < need) return PA_ERR_WORKSPACE;
  return PA_OK;
}

int clear_status(void* ws, cudaStream_t s) {
  return cudaMemsetAsync(ws, 0, kStatusBytes, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int check_heads(int32_t hq, int32_t hkv, int32_t d, int dtype) {
  if (hq <= 0 || hkv <= 0 || hq % hkv != 0) return PA_ERR_INVALID;
  if (d != 64 && d != 128) return PA_ERR_UNSUPPORTED;
  if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (hq / hkv > kMaxGroup || hkv > 65535) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// the stride of packed [heads][d] rows: room for the row, 16-byte multiple
int check_ld(int64_t ld, int32_t heads, int32_t d, int dtype) {
  if (ld < static_cast<int64_t>(heads) * d) return PA_ERR_INVALID;
  if (ld % (dtype == PA_BF16 ? 8 : 4) != 0) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

int check_pages(int32_t max_pages, int32_t page_size) {
  if (max_pages < 1 || page_size < 1) return PA_ERR_INVALID;
  if (page_size < 16 || page_size > 32768 || (page_size & (page_size - 1)) != 0) return PA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_pages) * page_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

int check_batch(int32_t B, int64_t N) {
  if (B < 0 || N < 0) return PA_ERR_INVALID;
  if (B > kMaxRequests || N > INT32_MAX) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

int32_t log2_of(int32_t power) {
  int32_t s = 0;
  while ((1 << s) < power) ++s;
  return s;
}

AttendArgs attend_args(int dtype, int64_t N, int32_t B, int32_t max_q, int32_t max_pages, int32_t page_size,
                       int32_t hq, int32_t hkv, int32_t d) {
  AttendArgs a = {};
  a.dtype = dtype;
  a.N = N; a.B = B; a.max_q = max_q;
  a.max_pages = max_pages; a.page_size = page_size;
  a.page_shift = log2_of(page_size);
  a.hq = hq; a.hkv = hkv; a.d = d;
  a.wait_limit_ns = kWaitLimitNs;
  return a;
}

int paged_attend(const void* q, int dtype, int64_t N, int64_t ldq, const int32_t* cu_q, const int32_t* kv_len,
                    int32_t B, int32_t max_q, const int32_t* block_table, int64_t table_stride,
                    int32_t max_pages, int32_t page_size, const void* k_pages, const void* v_pages,
                    int32_t n_pages, int32_t hq, int32_t hkv, int32_t d, void* o, float* lse_opt, void* ws,
                    size_t ws_bytes, void* stream, uint64_t wait_limit_ns, int stall) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int rc = check_heads(hq, hkv, d, dtype);
  if (!rc) rc = check_batch(B, N);
  if (!rc) rc = check_pages(max_pages, page_size);
  if (rc) return rc;
  if (max_q < 1 || n_pages < 0 || !cu_q || (B > 1 && table_stride < max_pages)) return PA_ERR_INVALID;
  if (static_cast<int64_t>(n_pages) * page_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (B > 0 && N > 0) {
    if (!q || !o || !kv_len || !block_table) return PA_ERR_INVALID;
    if (n_pages > 0 && (!k_pages || !v_pages)) return PA_ERR_INVALID;
    rc = check_ld(ldq, hq, d, dtype);
    if (rc) return rc;
  }
  const void* ptrs[] = {q, k_pages, v_pages, o};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return PA_ERR_UNSUPPORTED;
  const int64_t max_kv = static_cast<int64_t>(max_pages) * page_size;
  AttendArgs a = attend_args(dtype, N, B, max_q, max_pages, page_size, hq, hkv, d);
  rc = check_ws(ws, ws_bytes, plan_attend(a, max_kv, nullptr));
  if (rc) return rc;
  plan_attend(a, max_kv, ws);
  if (static_cast<int64_t>(a.piece_cap) * hkv > INT32_MAX) return PA_ERR_UNSUPPORTED;   // blocks of one launch
  if (B == 0 || N == 0) return clear_status(ws, s);
  a.q = q; a.k = k_pages; a.v = v_pages;
  a.ldq = ldq;
  a.ldk = a.ldv = static_cast<int64_t>(hkv) * d;
  a.n_slots = static_cast<int64_t>(n_pages) * page_size;
  a.cu_q = cu_q; a.kv_len = kv_len;
  a.block_table = block_table; a.table_stride = table_stride;
  a.o = o; a.lse = lse_opt;
  a.wait_limit_ns = wait_limit_ns;
  a.stall = stall;
  return launch_attend(a, s);
}

}  // namespace

extern "C" {

size_t pa_paged_schedule_workspace_size(int32_t B) { return B < 0 || B > kMaxRequests ? 0 : kStatusBytes; }

int pa_paged_schedule(const int32_t* q_len, const int32_t* kv_len, int32_t B, int32_t* block_table,
                      int64_t table_stride, int32_t max_pages, const int32_t* free_pages, int32_t n_free,
                      int32_t page_size, int64_t n_tokens, int32_t* cu_q, int32_t* kv_len_out,
                      int32_t* positions, int32_t* slots, int32_t* n_used, void* ws, size_t ws_bytes,
                      void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int rc = check_batch(B, n_tokens);
  if (rc) return rc;
  rc = check_pages(max_pages, page_size);
  if (rc) return rc;
  if (n_free < 0 || (B > 1 && table_stride < max_pages)) return PA_ERR_INVALID;
  if (B > 0 && (!q_len || !kv_len || !block_table || !kv_len_out)) return PA_ERR_INVALID;
  if (!cu_q || !n_used || (n_free > 0 && !free_pages)) return PA_ERR_INVALID;
  if (n_tokens > 0 && (!positions || !slots)) return PA_ERR_INVALID;
  rc = check_ws(ws, ws_bytes, kStatusBytes);
  if (rc) return rc;
  ScheduleArgs a;
  a.q_len = q_len; a.kv_len = kv_len; a.B = B;
  a.block_table = block_table; a.table_stride = table_stride; a.max_pages = max_pages;
  a.free_pages = free_pages; a.n_free = n_free; a.page_shift = log2_of(page_size);
  a.n_tokens = n_tokens;
  a.cu_q = cu_q; a.kv_len_out = kv_len_out; a.positions = positions; a.slots = slots; a.n_used = n_used;
  a.status = static_cast<DeviceStatus*>(ws);
  return launch_paged_schedule(a, s);
}

size_t pa_paged_append_workspace_size(int64_t N) { return N < 0 || N > INT32_MAX ? 0 : kStatusBytes; }

int pa_paged_append(const void* q, const void* k, const void* v, int dtype, int64_t N, int64_t ldq,
                    int64_t ldk, int64_t ldv, int32_t hq, int32_t hkv, int32_t d, double rope_theta,
                    const int32_t* positions, const int32_t* slots, void* k_pages, void* v_pages,
                    int64_t n_slots, void* q_out, void* k_out_opt, void* ws, size_t ws_bytes, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int rc = check_heads(hq, hkv, d, dtype);
  if (rc) return rc;
  rc = check_batch(0, N);
  if (rc) return rc;
  if (!std::isfinite(rope_theta) || rope_theta < 0) return PA_ERR_INVALID;
  if (n_slots < 0 || n_slots > INT32_MAX) return PA_ERR_INVALID;
  const bool pages = slots != nullptr;
  if (N > 0) {
    // (an empty cache may have no address)
    if (pages ? n_slots > 0 && (!k_pages || !v_pages) : k_pages != nullptr || v_pages != nullptr)
      return PA_ERR_INVALID;
    if (!k || (pages && !v) || (rope_theta > 0 && !positions)) return PA_ERR_INVALID;
    if ((q == nullptr) != (q_out == nullptr)) return PA_ERR_INVALID;
    if (q) rc = check_ld(ldq, hq, d, dtype);
    if (!rc) rc = check_ld(ldk, hkv, d, dtype);
    if (!rc && pages) rc = check_ld(ldv, hkv, d, dtype);
    if (rc) return rc;
  }
  const void* ptrs[] = {q, k, v, k_pages, v_pages, q_out, k_out_opt};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return PA_ERR_UNSUPPORTED;
  rc = check_ws(ws, ws_bytes, kStatusBytes);
  if (rc) return rc;
  if (N == 0) return clear_status(ws, s);
  AppendArgs a;
  a.q = q; a.k = k; a.v = v; a.dtype = dtype;
  a.N = N; a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
  a.hq = hq; a.hkv = hkv; a.d = d; a.rope_theta = rope_theta;
  a.positions = positions; a.slots = slots;
  a.k_pages = k_pages; a.v_pages = v_pages; a.n_slots = n_slots;
  a.q_out = q_out; a.k_out = k_out_opt;
  a.status = static_cast<DeviceStatus*>(ws);
  a.small = N <= 4096;
  return launch_paged_append(a, s);
}

size_t pa_prompt_attend_workspace_size(int32_t B, int64_t N, int32_t hq, int32_t hkv, int32_t d, int dtype) {
  if (check_heads(hq, hkv, d, dtype) || check_batch(B, N)) return 0;
  AttendArgs a = attend_args(dtype, N, B, 0, 0, 1, hq, hkv, d);
  return plan_attend(a, N, nullptr);
}

int pa_prompt_attend(const void* q, const void* k, const void* v, int dtype, int64_t N, int64_t ldq,
                     int64_t ldk, int64_t ldv, const int32_t* cu_q, int32_t B, int32_t hq, int32_t hkv,
                     int32_t d, void* o, float* lse_opt, void* ws, size_t ws_bytes, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int rc = check_heads(hq, hkv, d, dtype);
  if (!rc) rc = check_batch(B, N);
  if (rc) return rc;
  if (!cu_q) return PA_ERR_INVALID;
  if (N > 0) {
    if (!q || !k || !v || !o) return PA_ERR_INVALID;
    rc = check_ld(ldq, hq, d, dtype);
    if (!rc) rc = check_ld(ldk, hkv, d, dtype);
    if (!rc) rc = check_ld(ldv, hkv, d, dtype);
    if (rc) return rc;
  }
  const void* ptrs[] = {q, k, v, o};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return PA_ERR_UNSUPPORTED;
  AttendArgs a = attend_args(dtype, N, B, 0, 0, 1, hq, hkv, d);
  rc = check_ws(ws, ws_bytes, plan_attend(a, N, nullptr));
  if (rc) return rc;
  plan_attend(a, N, ws);
  if (static_cast<int64_t>(a.piece_cap) * hkv > INT32_MAX) return PA_ERR_UNSUPPORTED;   // blocks of one launch
  if (B == 0 || N == 0) return clear_status(ws, s);
  a.q = q; a.k = k; a.v = v;
  a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
  a.n_slots = N;
  a.cu_q = cu_q;
  a.o = o; a.lse = lse_opt;
  return launch_attend(a, s);
}

size_t pa_paged_attend_workspace_size(int32_t B, int64_t N, int32_t max_q, int32_t max_pages, int32_t page_size,
                                      int32_t hq, int32_t hkv, int32_t d, int dtype) {
  if (check_heads(hq, hkv, d, dtype) || check_batch(B, N) || check_pages(max_pages, page_size) || max_q < 1)
    return 0;
  AttendArgs a = attend_args(dtype, N, B, max_q, max_pages, page_size, hq, hkv, d);
  return plan_attend(a, static_cast<int64_t>(max_pages) * page_size, nullptr);
}

int pa_paged_attend(const void* q, int dtype, int64_t N, int64_t ldq, const int32_t* cu_q, const int32_t* kv_len,
                    int32_t B, int32_t max_q, const int32_t* block_table, int64_t table_stride,
                    int32_t max_pages, int32_t page_size, const void* k_pages, const void* v_pages,
                    int32_t n_pages, int32_t hq, int32_t hkv, int32_t d, void* o, float* lse_opt, void* ws,
                    size_t ws_bytes, void* stream) {
  return paged_attend(q, dtype, N, ldq, cu_q, kv_len, B, max_q, block_table, table_stride, max_pages, page_size,
                      k_pages, v_pages, n_pages, hq, hkv, d, o, lse_opt, ws, ws_bytes, stream, kWaitLimitNs, 0);
}

int pa_testing_paged_stall(const void* q, int64_t N, const int32_t* cu_q, const int32_t* kv_len, int32_t B,
                           int32_t max_q, const int32_t* block_table, int32_t max_pages, int32_t page_size,
                           const void* k_pages, const void* v_pages, int32_t n_pages, int32_t hq, int32_t hkv,
                           int32_t d, void* o, void* ws, size_t ws_bytes, int32_t wait_limit_us, void* stream) {
  if (wait_limit_us <= 0 || wait_limit_us > 10000000) return PA_ERR_INVALID;
  return paged_attend(q, PA_BF16, N, static_cast<int64_t>(hq) * d, cu_q, kv_len, B, max_q, block_table, max_pages,
                      max_pages, page_size, k_pages, v_pages, n_pages, hq, hkv, d, o, nullptr, ws, ws_bytes, stream,
                      static_cast<uint64_t>(wait_limit_us) * 1000ull, 1);
}

}  // extern "C"
