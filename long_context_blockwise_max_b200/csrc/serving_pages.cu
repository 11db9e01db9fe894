// The page tables and slot map of a serving step, and the rotation of its
// new tokens with their append to the paged cache.
#include <cmath>

#include "serving.h"

namespace pa {

namespace {

__device__ __forceinline__ int32_t sat32(int64_t x) {
  return static_cast<int32_t>(x < INT32_MAX ? x : INT32_MAX);
}

// The status of a step whose blocks all report to it, cleared before they
// start.  A memset does not overlap the next kernel's set-up: 8.3 us in a graph for
// the tables of 512 requests, 5.5 us with this.
__global__ void clear_status_kernel(DeviceStatus* status) {
  grid_dep_wait();
  grid_dep_launch();
  reinterpret_cast<int32_t*>(status)[threadIdx.x] = 0;
}
int clear_status(DeviceStatus* status, cudaStream_t s) {
  return launch_overlapped(clear_status_kernel, dim3(1), static_cast<int>(kStatusBytes / 4), 0, s, status);
}

// Two prefix sums over the requests (new tokens, new pages), then one entry
// per token and per new page, each found by bisection in them.  Every block
// builds the sums by itself (B is at most 8192: a few loads per thread that
// hit L2), which saves a kernel for them and a grid-wide wait; tokens and pages
// are spread over the blocks.  A step of one block is one launch, one of more has
// its status cleared by another before it.  Latency-bound: 64 requests with a token each
// take 2.8 us in a graph (their loads, one scan and one look-up), 512 requests
// with 150K tokens 5.5 us.
__global__ void __launch_bounds__(1024) paged_schedule_kernel(ScheduleArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* cu = sm;                  // [B + 1] new tokens before request b
  int32_t* pages = cu + a.B + 1;     // [B + 1] new pages asked for before it
  int32_t* cached = pages + a.B + 1; // [B] tokens it has
  uint8_t* granted = reinterpret_cast<uint8_t*>(cached + a.B);   // [B]
  __shared__ int64_t tmp[2][64];
  __shared__ int32_t used;
  const int shift = a.page_shift, page = 1 << shift;
  grid_dep_wait();
  // one block: it clears the status itself (more have it cleared before them)
  if (gridDim.x == 1 && threadIdx.x < kStatusBytes / 4) reinterpret_cast<int32_t*>(a.status)[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    cu[0] = 0;
    pages[0] = 0;
    used = 0;
  }
  __syncthreads();
  const bool first = blockIdx.x == 0;
  int64_t tok_base = 0, page_base = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int64_t q = 0, kv = 0;
    bool bad = false;
    if (b < a.B) {
      q = a.q_len[b];
      kv = a.kv_len[b];
      bad = q < 0 || kv < 0;
      q = q < 0 ? 0 : q;
      kv = kv < 0 ? 0 : kv;
    }
    const int64_t held = (kv + page - 1) >> shift, all = (kv + q + page - 1) >> shift;
    const int64_t need = q > 0 ? all - held : 0;
    const bool fits = q == 0 || all <= a.max_pages;
    int64_t toks = q, pgs = fits ? need : 0, tok_all, page_all;
    block_incl_scan2<int64_t>(toks, pgs, tmp[(b0 / blockDim.x) & 1], &tok_all, &page_all);
    toks += tok_base;
    pgs += page_base;
    if (b < a.B) {
      const bool ok = fits && (need == 0 || pgs <= a.n_free);
      cu[b + 1] = sat32(toks);
      pages[b + 1] = sat32(pgs);
      cached[b] = static_cast<int32_t>(kv);
      granted[b] = ok;
      if (ok && need > 0) atomicMax(&used, sat32(pgs));
      if (first) {
        a.cu_q[b + 1] = sat32(toks);
        a.kv_len_out[b] = sat32(ok ? kv + q : kv);
        if (bad) set_status(a.status, PA_ERR_INVALID, b);
        else if (!ok) set_status(a.status, PA_ERR_CAPACITY, b);
      }
    }
    tok_base += tok_all;
    page_base += page_all;
  }
  __syncthreads();
  if (first && threadIdx.x == 0) {
    a.cu_q[0] = 0;
    *a.n_used = used;
    if (tok_base > a.n_tokens) set_status(a.status, PA_ERR_INVALID, a.B);
  }
  auto held_of = [&](int b) { return (static_cast<int64_t>(cached[b]) + page - 1) >> shift; };
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  // the new pages into their requests' rows
  for (int64_t x = id; x < used; x += step) {
    const int b = upper_index(pages, a.B + 1, static_cast<int32_t>(x));
    a.block_table[b * a.table_stride + held_of(b) + (x - pages[b])] = a.free_pages[x];
  }
  // a position and a slot for each token
  for (int64_t t = id; t < a.n_tokens; t += step) {
    int32_t pos = 0, slot = -1;
    if (t < cu[a.B]) {
      const int b = upper_index(cu, a.B + 1, static_cast<int32_t>(t));
      const int64_t p = static_cast<int64_t>(cached[b]) + (t - cu[b]);
      pos = sat32(p);
      if (granted[b]) {
        const int64_t i = p >> shift, held = held_of(b);
        const int64_t pg = i < held ? a.block_table[b * a.table_stride + i] : a.free_pages[pages[b] + (i - held)];
        const int64_t s = (pg << shift) + (p & (page - 1));
        if (pg < 0 || s > INT32_MAX) set_status(a.status, PA_ERR_INVALID, b, static_cast<int>(pg));
        else slot = static_cast<int32_t>(s);
      }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
}

// RoPE and append.  HBM-bound: each element is read once and written once,
// in 16-byte accesses.  A block takes `tpb` tokens; the angles of a token
// are computed once (fp64 product and reduction to one turn, fp32 sine and
// cosine of the rest) and shared by its heads through shared memory.
// 32K tokens, 32 / 8 heads of 128, bf16: 127 us = 6.33 TB/s, 97 % of a copy's
// rate; 16 tokens: 2.9 us in a graph.  Blocks of 8 tokens take 133 us, of 2 or 16
// more still; two or four tokens' loads in flight per thread took 240.
template <typename T>
__global__ void __launch_bounds__(256) paged_append_kernel(AppendArgs a, RopeFreqs turns, int tpb) {
  constexpr int V = 16 / sizeof(T);            // elements per access
  // (cos, sin) of angle m of token t at [t][m % V][m / V]: the threads of a head
  // read neighbours ([t][m] cost four times the shared-memory cycles, and bound
  // the kernel)
  extern __shared__ float2 cs[];
  const int half = a.d / 2, cpr = half / V;    // cpr: accesses per half row
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tpb;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tpb), a.N - t0));
  const bool rope = a.rope_theta != 0.0;
  grid_dep_wait();
  if (a.small && blockIdx.x == 0) {
    if (threadIdx.x < kStatusBytes / 4) reinterpret_cast<int32_t*>(a.status)[threadIdx.x] = 0;
    __syncthreads();
    if (a.slots)
      for (int64_t t = threadIdx.x; t < a.N; t += 256)
        if (a.slots[t] >= a.n_slots) set_status(a.status, PA_ERR_INVALID, static_cast<int>(t), a.slots[t]);
  }
  if (rope) {
    for (int e = threadIdx.x; e < nt * half; e += 256) {
      const double x = a.positions[t0 + e / half] * turns.omega[e % half];   // angle in turns
      const float f = static_cast<float>(x - rint(x));                       // in [-1/2, 1/2]
      float sn, cn;
      sincospif(2.f * f, &sn, &cn);
      const int m = e % half;
      cs[e - m + (m % V) * cpr + m / V] = make_float2(cn, sn);
    }
    __syncthreads();
  }
  const int hq = a.q ? a.hq : 0;
  const int hv = a.slots ? a.hkv : 0;
  const int per_tok = (hq + a.hkv + hv) * cpr;
  for (int e = threadIdx.x; e < nt * per_tok; e += 256) {
    const int t = e / per_tok, i = e % per_tok;
    const int head = i / cpr, m = (i % cpr) * V;
    const int64_t tok = t0 + t;
    int64_t slot = a.slots ? a.slots[tok] : -1;
    if (slot >= a.n_slots) {
      if (i == 0 && !a.small) set_status(a.status, PA_ERR_INVALID, static_cast<int>(tok), static_cast<int>(slot));
      slot = -1;
    }
    const T* src;
    T *dst, *page = nullptr;
    if (head < hq) {
      src = static_cast<const T*>(a.q) + tok * a.ldq + head * a.d;
      dst = static_cast<T*>(a.q_out) + (tok * a.hq + head) * a.d;
    } else if (head < hq + a.hkv) {
      const int h = head - hq;
      src = static_cast<const T*>(a.k) + tok * a.ldk + h * a.d;
      dst = a.k_out ? static_cast<T*>(a.k_out) + (tok * a.hkv + h) * a.d : nullptr;
      if (slot >= 0) page = static_cast<T*>(a.k_pages) + (slot * a.hkv + h) * a.d;
    } else {
      const int h = head - hq - a.hkv;
      if (slot < 0) continue;
      src = static_cast<const T*>(a.v) + tok * a.ldv + h * a.d;
      dst = nullptr;
      page = static_cast<T*>(a.v_pages) + (slot * a.hkv + h) * a.d;
    }
    alignas(16) T x1[V], x2[V];
    *reinterpret_cast<uint4*>(x1) = *reinterpret_cast<const uint4*>(src + m);
    *reinterpret_cast<uint4*>(x2) = *reinterpret_cast<const uint4*>(src + m + half);
    if (rope && head < hq + a.hkv) {
      const float2* c = cs + t * half + m / V;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float y1 = to_f32(x1[j]), y2 = to_f32(x2[j]);
        const float2 r = c[j * cpr];
        x1[j] = from_f32<T>(y1 * r.x - y2 * r.y);
        x2[j] = from_f32<T>(y2 * r.x + y1 * r.y);
      }
    }
    if (dst) {
      *reinterpret_cast<uint4*>(dst + m) = *reinterpret_cast<uint4*>(x1);
      *reinterpret_cast<uint4*>(dst + m + half) = *reinterpret_cast<uint4*>(x2);
    }
    if (page) {
      *reinterpret_cast<uint4*>(page + m) = *reinterpret_cast<uint4*>(x1);
      *reinterpret_cast<uint4*>(page + m + half) = *reinterpret_cast<uint4*>(x2);
    }
  }
}

}  // namespace

int launch_paged_schedule(const ScheduleArgs& a, cudaStream_t s) {
  const size_t smem = 13 * static_cast<size_t>(a.B) + 8;
  if (smem > 46 * 1024) {   // beside 1 KB of static arrays
    const int rc = allow_smem<paged_schedule_kernel>(13 * kMaxRequests + 8);
    if (rc != PA_OK) return rc;
  }
  // one thread per token up to a block per SM; a small step's block has no
  // more threads than its requests and tokens need
  const int64_t most = a.n_tokens > a.B ? a.n_tokens : a.B;
  const int threads = most <= 256 ? 256 : 1024;
  const int64_t want = (a.n_tokens + threads - 1) / threads;
  const int grid = static_cast<int>(want < 1 ? 1 : want > kSms ? kSms : want);
  const int rc = grid > 1 ? clear_status(a.status, s) : PA_OK;
  if (rc != PA_OK) return rc;
  return launch_overlapped(paged_schedule_kernel, dim3(grid), threads, smem, s, a);
}

int launch_paged_append(const AppendArgs& a, cudaStream_t s) {
  constexpr double kTwoPi = 6.283185307179586476925;
  RopeFreqs f;
  for (int m = 0; m < kMaxHalfDim; ++m)
    f.omega[m] = (m < a.d / 2 && a.rope_theta > 0) ? pow(a.rope_theta, -2.0 * m / a.d) / kTwoPi : 0.0;
  const int tpb = a.N >= 8 * kSms ? 4 : 1;
  const int64_t grid = (a.N + tpb - 1) / tpb;
  const size_t smem = sizeof(float2) * tpb * (a.d / 2);
  const int rc = a.small ? PA_OK : clear_status(a.status, s);
  if (rc != PA_OK) return rc;
  const dim3 blocks(static_cast<unsigned>(grid));
  return a.dtype == PA_F32 ? launch_overlapped(paged_append_kernel<float>, blocks, 256, smem, s, a, f, tpb)
                           : launch_overlapped(paged_append_kernel<__nv_bfloat16>, blocks, 256, smem, s, a, f, tpb);
}

}  // namespace pa
