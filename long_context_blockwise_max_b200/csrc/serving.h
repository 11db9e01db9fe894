// Internal interface of the serving operators (include/pulsar_serving.h):
// kernel arguments, the work plan of an attention call and the launchers.
#pragma once

#include <atomic>

#include "pa_internal.h"
#include "../../include/pulsar_serving.h"

namespace pa {

constexpr int kMaxRequests = 8192;   // prefix sums of a step are staged in shared memory
constexpr int kMaxGroup = 64;        // query heads per kv head: a tile holds at least one token
constexpr int kSms = 148;
constexpr int kPlanTile = 128;       // keys per unit of planned work
constexpr int kDecodeRows = 16;      // most rows per kv head of the decode kernel (one MMA's)
constexpr int kFoldTiles = 2048;     // key tiles after which the tile kernel takes O out of its accumulator

struct ScheduleArgs {
  const int32_t *q_len, *kv_len;
  int32_t B;
  int32_t* block_table;
  int64_t table_stride;
  int32_t max_pages;
  const int32_t* free_pages;
  int32_t n_free, page_shift;
  int64_t n_tokens;
  int32_t *cu_q, *kv_len_out, *positions, *slots, *n_used;
  DeviceStatus* status;
};
int launch_paged_schedule(const ScheduleArgs& a, cudaStream_t s);

struct AppendArgs {
  const void *q, *k, *v;
  int dtype;
  int64_t N, ldq, ldk, ldv;
  int32_t hq, hkv, d;
  double rope_theta;
  const int32_t *positions, *slots;
  void *k_pages, *v_pages;
  int64_t n_slots;
  void *q_out, *k_out;
  DeviceStatus* status;
  int small;   // few tokens: the first block clears the status and checks every slot
};
int launch_paged_append(const AppendArgs& a, cudaStream_t s);

// One unit of attention work: the rows of up to `tokens` new tokens of a
// request (all query heads of one kv head) against key tiles [kt0, kt1).
struct Piece {
  int32_t b, tok0;    // request, first of its new tokens
  int32_t kt0, kt1;   // key tiles of kPlanTile keys
  int32_t part;       // slot of its partial result, or -1: it has all the keys
  int32_t row0;       // cu_q[b]
  int32_t q_len, kv_len;
};
static_assert(sizeof(Piece) == 32, "a piece is two 16-byte loads");

// Rows whose keys were cut into several pieces (merged afterwards).
struct MergeItem {
  int32_t row0, n_tok;      // first packed row, tokens
  int32_t part0, n_parts;
};

// One block's range of decode work, all that it has to know to start: the
// request, kv head and key group of its first unit, and how the units are
// shared out.
struct DecodeStart {
  int32_t b, kvh, unit, n_units;     // n_units: key groups of that request
  int32_t kv, q, row0, steps;        // its lengths; units of this block
  int64_t first;                     // this block's first unit
  int64_t each;                      // units per block; the first `more` blocks have one more
  int32_t more, pad[3];
};
static_assert(sizeof(DecodeStart) == 64, "four 16-byte loads");

struct PlanHead {
  int32_t n_pieces;     // pieces of the tile kernels, per kv head
  int32_t n_items;      // entries of the merge list
  int32_t abort;        // a bounded wait ran out somewhere
  int32_t heads_inner;  // order of the tile kernels' work (piece_at)
  uint32_t next;        // units of work taken beyond each block's first
  int32_t pad;
};

struct AttendArgs {
  int dtype;
  const void *q, *k, *v;          // k, v: packed rows or pages
  int64_t N, ldq, ldk, ldv;       // ldk, ldv: packed rows only
  const int32_t* cu_q;
  const int32_t* kv_len;          // null: prompts (kv_len = q_len)
  int32_t B, max_q;
  const int32_t* block_table;     // null: packed rows
  int64_t table_stride;
  int32_t max_pages, page_size, page_shift;
  int64_t n_slots;                // rows of k, v
  int32_t hq, hkv, d;
  void* o;
  float* lse;
  // ------------------------------------------------ plan (serving_plan.cu)
  int32_t tile_tokens;            // new tokens per piece
  int32_t tile_rows;              // rows a partial result has room for
  int32_t small_rows;             // requests of at most so many rows go to the decode kernel
  int32_t tiles;                  // whether a tile kernel runs
  int32_t slots;                  // blocks of it that run at once
  float piece_cost, merge_cost;   // fixed costs of a piece and of cutting, in key tiles
  int32_t piece_cap;              // pieces the workspace has room for
  int32_t part_cap;               // partial results it has room for, per kv head; 0: never cut
  int32_t item_cap;
  int32_t decode_ctas;            // 0: no decode kernel
  DeviceStatus* status;
  PlanHead* head;
  Piece* pieces;
  MergeItem* items;
  DecodeStart* starts;            // [decode_ctas]
  int32_t* done;                  // [decode_ctas] arrivals at a cut (request, kv head)
  float* part_o;                  // [part_cap][hkv][tile_rows][d]
  float* part_lse;                // [part_cap][hkv][tile_rows]
  float* fold;                    // [slots][2][256][d + 4] O so far of long pieces (tile kernel), or null: none is
  float* dec_o;                   // [2 * decode_ctas][16][d]
  float* dec_lse;                 // [2 * decode_ctas][16]
  uint64_t wait_limit_ns = 1000000000ull;
  int stall = 0;                  // test only: one barrier per block expects 16 bytes more than are copied
};
// Fills the plan's sizes and returns the workspace bytes; with `ws` set,
// carves it.  `max_kv` is the longest cache a request may have.
size_t plan_attend(AttendArgs& a, int64_t max_kv, void* ws);
int launch_attend(const AttendArgs& a, cudaStream_t s);

int launch_attend_simt(const AttendArgs& a, cudaStream_t s);   // fp32
int simt_blocks_per_sm(const AttendArgs& a);
int launch_attend_tc(const AttendArgs& a, cudaStream_t s);     // bf16
int launch_attend_decode(const AttendArgs& a, cudaStream_t s); // bf16, few rows

// keys of a request that the first `n` of its new tokens see
__host__ __device__ inline int64_t keys_seen(int64_t kv_len, int64_t q_len, int64_t n) {
  const int64_t k = kv_len - q_len + n;
  return k < 0 ? 0 : k;
}

// Launch attribute of a kernel that may be set up while the one before it
// in the stream still runs; it calls grid_dep_wait() before it reads anything
// that kernel (or one before) wrote.
inline cudaLaunchAttribute overlap_attr() {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  return at;
}
template <typename... P, typename... A>
int launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute at = overlap_attr();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Sets a kernel's dynamic shared memory once per device.
template <auto* kernel>
int allow_smem(size_t bytes) {
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (set.load(std::memory_order_relaxed) & bit)) return PA_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess)
    return PA_ERR_CUDA;
  set.fetch_or(bit, std::memory_order_relaxed);
  return PA_OK;
}

// Units of work of a tile kernel: the most pieces the arguments allow, times kv heads.
inline unsigned tile_blocks(const AttendArgs& a) {
  return static_cast<unsigned>(a.piece_cap) * static_cast<unsigned>(a.hkv);
}

// TMA map (a CUtensorMap; serving_tc.cu) of a 16-bit tensor
// [rows][heads][d] with a row stride of ld elements, boxes of 64 columns x
// `box_heads` x `box_rows`, 128-byte swizzle.
bool rows_map(void* map, const void* base, int64_t rows, int heads, int d, int64_t ld, int box_heads, int box_rows);

#ifdef __CUDACC__
// Piece and kv head of the i-th unit of work (of n_pieces * hkv).  Units that
// run together share one kv head's K and V (which then stay in L2 however
// long the caches are), or, when all of K and V fit there anyway, are the
// deepest pieces of every head first, so that the launch ends with short ones.
__device__ __forceinline__ void piece_at(const AttendArgs& a, unsigned i, int* at, int* kvh) {
  const unsigned n = static_cast<unsigned>(a.head->n_pieces), h = static_cast<unsigned>(a.hkv);
  if (a.head->heads_inner) {
    *at = static_cast<int>(i / h);
    *kvh = static_cast<int>(i % h);
  } else {
    *at = static_cast<int>(i % n);
    *kvh = static_cast<int>(i / n);
  }
}

// Waits until the kernels before this one in the stream have ended and their
// writes are visible.
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel of the stream be set up.
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

// Slot of key `key` of request b, or -1 (recorded) when its page is not in
// the cache.
__device__ __forceinline__ int64_t key_slot(const AttendArgs& a, int b, int64_t key) {
  const int page = a.block_table[static_cast<int64_t>(b) * a.table_stride + (key >> a.page_shift)];
  const int64_t slot = (static_cast<int64_t>(page) << a.page_shift) + (key & (a.page_size - 1));
  if (page < 0 || slot >= a.n_slots) {
    set_status(a.status, PA_ERR_INVALID, b, page);
    return -1;
  }
  return slot;
}

template <typename T>
__device__ __forceinline__ T warp_incl_scan(T x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Inclusive scans of x and y over the block (a multiple of 32 threads, at most
// 1024); *x_all and *y_all receive the sums.  Every warp scans the warps' sums
// for itself, so that one barrier is enough.  `tmp` has 64 elements and must
// not be in use by an earlier scan (alternate two).
template <typename T>
__device__ __forceinline__ void block_incl_scan2(T& x, T& y, T* tmp, T* x_all, T* y_all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  x = warp_incl_scan(x);
  y = warp_incl_scan(y);
  if (lane == 31) {
    tmp[warp] = x;
    tmp[32 + warp] = y;
  }
  __syncthreads();
  const T wx = warp_incl_scan(lane < warps ? tmp[lane] : T(0));
  const T wy = warp_incl_scan(lane < warps ? tmp[32 + lane] : T(0));
  const int before = warp > 0 ? warp - 1 : 0;
  const T bx = __shfl_sync(0xffffffffu, wx, before), by = __shfl_sync(0xffffffffu, wy, before);
  *x_all = __shfl_sync(0xffffffffu, wx, 31);
  *y_all = __shfl_sync(0xffffffffu, wy, 31);
  if (warp > 0) {
    x += bx;
    y += by;
  }
}

// Largest i in [0, n) with pre[i] <= x (pre[0] <= x; pre non-decreasing).
template <typename T>
__device__ __forceinline__ int upper_index(const T* pre, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
#endif

}  // namespace pa
