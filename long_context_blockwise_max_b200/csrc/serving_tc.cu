// Causal attention of packed prompts, and of new tokens over a paged cache,
// on the sm_100a tensor cores (tcgen05 + TMEM + TMA), bf16.
//
// One block per SM walks the plan's pieces (serving_plan.cu), each for one kv
// head: up to two tiles of 128 packed rows (a tile holds 128 / g tokens x the g
// query heads of the group, so every K / V tile serves all of them and a
// request's ragged end wastes less than one tile) against 128-key tiles.  12
// warps, each walking the same pieces on its own:
//   warp 0      TMA producer: Q of a piece, then K / V tiles through 2-stage
//               rings that run on across pieces.  Packed rows are one box per
//               64 columns; a paged tile is one box per page, issued by as
//               many lanes.
//   warp 1      MMA issuer (one thread): S = Q K^T (bf16 x bf16 -> fp32 in
//               TMEM, exact products) and O += P V (P bf16 from TMEM).
//   warps 2-3   guard of V tiles that hold masked keys (below); warp 2 also
//               allocates TMEM (512 columns: S0 | O0 | S1 | O1).
//   warps 4-11  two softmax warpgroups, one thread per row; online softmax
//               in log2 units, O rescaled only when the running maximum
//               grows by more than 2^8.
// With two row tiles, the warpgroups take one each and share every K / V
// tile: while one runs its softmax the tensor core works on the other.  With
// one (a chunk of at most 128 rows), they take alternate key tiles of the same
// rows, each with its own maximum, sum and O, joined at the end, so a short
// query streams its keys at the same rate per block.
//
// The next piece's Q, first keys and first scores are under way while the
// softmax warps store a piece's output: one block per piece took 8 us of
// set-up and output per piece beside 2.1 us per key tile.
//
// What bounds it: the chain of a row tile's softmax (2300 clocks: TMEM load 120,
// maximum 410, exponentials 1290, sums and P 500) and its PV and next QK^T
// (1230), 3600 to 3900 clocks per pair of row tiles and key tile, in which the
// tensor pipe and the exponentials are each 54 % busy; TMEM has no room for a
// second S.  A piece's output takes another 3800 (64 KB out of one SM).  32 / 8
// heads of 128: one 32K prompt 8.0 to 8.2 ms = 1070 to 1100 TFLOP/s at the power
// cap (7.0 ms before it sets in); 24 prompts of 1 to 4096 tokens 160 to 165 us; a
// 64-token query over 128K keys 168 to 181 us with its plan and merge.
//
// A sum in TMEM loses the bits that one addition cannot hold, always towards
// zero: o was 3e-4 too small over 512K keys in one accumulator, 1e-3 over 1M, 2 % over
// 4M (equal weights).  So where a piece may be longer than kFoldTiles tiles, O goes
// to a row in the workspace after every so many, added in fp32, and the next P V
// starts anew (FOLD).  Calls whose tables or prompts cannot be that long have a
// kernel without it: the same code cost them 2 to 4 % (ragged prompts 161 -> 167 us, one
// 32K prompt 7.97 -> 8.18 ms, 32 mixed requests 97.4 -> 101.4).
//
// P is rounded to bf16 (half a step, 2^-8 of each probability; the row sum is taken
// before it), as its product with V needs: a second product with the residual would
// add half of the tensor pipe's work, and TMEM has no columns for it.
//
// Guard: P is zero at a masked key, but zero times an infinity or NaN in its
// V is NaN.  In tiles with keys that some row does not see, rows past the
// request's last key are zeroed in shared memory, and a non-finite V element
// is replaced by zero with its key noted per column (first +inf, -inf, NaN);
// the epilogue gives rows that do see it the value the sum would have.
//
// Every wait on an mbarrier is bounded; on expiry the block records
// PA_ERR_TIMEOUT, drains its copies and MMAs, frees TMEM and returns.  (A wait may
// last as long as a piece, so its limit grows with the deepest that the arguments
// allow.)  No barrier runs more than one phase ahead of a waiter: those that a role could
// pass a whole piece early come in pairs, used in turn.
#include <cudaTypedefs.h>

#include "serving.h"
#include "sm100.cuh"

namespace pa {
using namespace sm100;

namespace {

constexpr int kKeyTile = 128;
static_assert(kKeyTile == kPlanTile, "the plan counts this kernel's key tiles");

template <int D>
struct SvCfg {
  static constexpr int NKB = D / 64;                 // 128-byte column blocks along d
  static constexpr int KB_BYTES = 128 * 128;         // 128 rows x 128 B
  static constexpr int TILE_BYTES = NKB * KB_BYTES;  // 128 rows x D x 2 B
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + 2 * TILE_BYTES;
  static constexpr int OFF_OUT = OFF_V + 2 * TILE_BYTES;   // output staging, 2 KB per softmax warp
  static constexpr int OFF_BAR = OFF_OUT + 8 * 2048;
  static constexpr int SMEM_BYTES = OFF_BAR + 13 * 1024;
  // log2(e) / sqrt(d)
  static constexpr float SCALE = static_cast<float>(kLog2e / (D == 128 ? 11.31370849898476039 : 8.0));
  static constexpr uint32_t IDESC_QK = idesc_f16(128, 128, 1, 1, 0, 0);  // bf16 Q . bf16 K
  static constexpr uint32_t IDESC_PV = idesc_f16(128, D, 1, 1, 0, 1);    // bf16 P . bf16 V (MN-major)
};

struct SvBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t vg_full[2];    // a guarded V tile has landed
  uint64_t v_ready[2];    // ... and has been checked
  uint64_t s_full[2], p_full[2], o_final[2];
  uint64_t noted[2];      // the guard is through with a piece's tiles; pieces in turn
  uint64_t done[2];       // the softmax warps have read a piece's O; pieces in turn
  uint64_t read[2];       // they and the issuer have read its item, maxima and notes; pieces in turn
  uint64_t ml_full[2][2]; // a warpgroup's maxima and sums are written (one row tile); pieces in turn
  uint64_t work_full[2];  // `work` holds a piece; pieces in turn
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int odd[2];             // 1 + number of the piece that met a non-finite V
  // per column: first key with +inf, -inf, NaN, below the complement of 1 + the
  // piece's number, so that a later piece's entry is always the smaller
  unsigned long long first[2][3][128];
  float ml[2][2][2][128]; // [pieces in turn][warpgroup][maximum, sum][row]
  struct {
    int4 rows;            // row0, tok0, q_len, kv_len
    int4 keys;            // kt0, n, part, kvh (-1: no more)
    int4 tiles;           // nt0, nt1, g0, 2 * request + two
  } work[2];
};
static_assert(sizeof(SvBars) + 1024 <= 13 * 1024, "barriers and alignment slack");

struct SvParams {
  AttendArgs a;
  int box_rows;     // keys per TMA box (a page, or a whole tile)
  int oob_row;      // a row coordinate past the end of K and V: reads zeros
};

__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// An arrival that orders no memory (the caller's global stores need not be
// done first): for O in TMEM alone, whose reads tcgen05 fences order.
__device__ __forceinline__ void mbar_arrive_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool bf16_nonfinite(uint32_t two) {
  return (two & 0x7f80u) == 0x7f80u || (two & 0x7f800000u) == 0x7f800000u;
}

// One guarded V tile in shared memory (column blocks of 128 rows x 128 B,
// 128-byte swizzle): rows from `first_row` on may be masked, rows from
// `n_keys` on hold no key.  Run by 64 threads.
template <int D>
__device__ void guard_tile(uint8_t* v, int first_row, int n_keys, int key0, int piece, SvBars* bars, int tid) {
  using C = SvCfg<D>;
  constexpr int CH = D / 8;   // 16-byte chunks of a row
  constexpr int STEP = 64 / CH;   // rows that the threads take together
  const int c = tid % CH;
  auto at = [&](int r) {
    return reinterpret_cast<uint4*>(v + (c >> 3) * C::KB_BYTES + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  };
#pragma unroll 4
  for (int r = max(n_keys, 0) + tid / CH; r < 128; r += STEP) *at(r) = make_uint4(0, 0, 0, 0);
  const int end = min(n_keys, 128);
  // (eight loads at a time: one by one, their latency made a full tile take longer than its softmax)
  for (int r0 = first_row + tid / CH; r0 < end; r0 += 8 * STEP) {
    uint4 x[8];
    uint32_t odd = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = make_uint4(0, 0, 0, 0);
      if (r0 + j * STEP < end) x[j] = *at(r0 + j * STEP);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      odd |= (bf16_nonfinite(x[j].x) || bf16_nonfinite(x[j].y) || bf16_nonfinite(x[j].z) || bf16_nonfinite(x[j].w))
             << j;
    for (; odd != 0; odd &= odd - 1) {
      const int r = r0 + (__ffs(odd) - 1) * STEP;
      uint16_t* e = reinterpret_cast<uint16_t*>(at(r));
      for (int k = 0; k < 8; ++k)
        if ((e[k] & 0x7f80) == 0x7f80) {
          const int kind = (e[k] & 0x7f) ? 2 : (e[k] >> 15);
          atomicMin(&bars->first[piece & 1][kind][8 * c + k],
                    (static_cast<unsigned long long>(~static_cast<uint32_t>(piece + 1)) << 32) |
                        static_cast<uint32_t>(key0 + r));
          e[k] = 0;
        }
      bars->odd[piece & 1] = piece + 1;
    }
  }
}

// A piece as its roles see it.
struct Item {
  int row0, tok0, q_len, kv_len;   // as in Piece
  int kt0, n;                      // first key tile, key tiles
  int part, kvh;
  int nt0, nt1;                    // key tiles of each warpgroup: with two row tiles those up to
                                   // its last row's limit, of all; with one, every other
  int g0;                          // first guarded tile: those from it on hold a key that the first row does not see
  bool two;                        // two row tiles
  int b;                           // request
  int ctx;                         // position of the first new token (may be negative)
};

// Row `row` (of both warpgroups' 256) of the O so far of this block's pieces,
// taken in turn: D sums and, behind them, the maximum that they are relative to.
template <int D>
__device__ __forceinline__ float* fold_row(const AttendArgs& a, int k, int row) {
  return a.fold + ((static_cast<int64_t>(blockIdx.x) * 2 + (k & 1)) * 256 + row) * (D + 4);
}
// 2^((from - to) * scale): what a sum relative to the maximum `from` weighs in one
// relative to `to`.
__device__ __forceinline__ float reweight(float from, float to, float scale) {
  return from == to ? 1.f : fast_exp2((from - to) * scale);
}

// The k-th piece of this block, once it is there; false: no more.
__device__ __forceinline__ bool get_item(const SvBars* bars, int k, Item& it) {
  const int4 x = bars->work[k & 1].rows, y = bars->work[k & 1].keys, z = bars->work[k & 1].tiles;
  it = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, z.z, (z.w & 1) != 0, z.w >> 1, x.w - x.z};
  return it.kvh >= 0;
}

// Puts piece `pc` (kv head -1: the end) where get_item finds it.
__device__ __forceinline__ void put_item(SvBars* bars, int k, int tpt, const Piece& pc, int kvh) {
  const int ctx = pc.kv_len - pc.q_len, n = pc.kt1 - pc.kt0;
  const bool two = pc.tok0 + tpt < pc.q_len;
  // keys that tile 0 sees (it is full); with a tile's more they may pass 2^31
  const int64_t seen = keys_seen(pc.kv_len, pc.q_len, static_cast<int64_t>(pc.tok0) + tpt);
  const int deep = static_cast<int>((seen + kKeyTile - 1) / kKeyTile);
  const int nt0 = two ? max(0, min(n, deep - pc.kt0)) : (n + 1) / 2;
  bars->work[k & 1].rows = make_int4(pc.row0, pc.tok0, pc.q_len, pc.kv_len);
  bars->work[k & 1].keys = make_int4(pc.kt0, n, pc.part, kvh);
  bars->work[k & 1].tiles = make_int4(nt0, two ? n : n / 2, max(0, max(0, ctx + pc.tok0 + 1) / kKeyTile - pc.kt0),
                                         2 * pc.b + two);
}

template <int D, bool PAGED, bool FOLD>
__global__ void __launch_bounds__(384, 1) attend_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                           const __grid_constant__ CUtensorMap tmK,
                                                           const __grid_constant__ CUtensorMap tmV,
                                                           const __grid_constant__ SvParams p) {
  using C = SvCfg<D>;
  const AttendArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  SvBars* bars = reinterpret_cast<SvBars*>(smem + C::OFF_BAR);
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
      mbar_init(&bars->vg_full[s], 1);
      mbar_init(&bars->v_ready[s], 2);
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->p_full[s], 4);
      mbar_init(&bars->o_final[s], 1);
      mbar_init(&bars->noted[s], 2);
      mbar_init(&bars->done[s], 8);
      mbar_init(&bars->read[s], 9);
      mbar_init(&bars->ml_full[s][0], 4);
      mbar_init(&bars->ml_full[s][1], 4);
      mbar_init(&bars->work_full[s], 1);
      bars->odd[s] = 0;
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < 2 * 3 * 128; i += 384) (&bars->first[0][0][0])[i] = ~0ull;
  if (warp == 2) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();      // the set-up above overlaps the plan
  grid_dep_launch();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort = &bars->abort;
  volatile int* gabort = &a.head->abort;
  const int g = a.hq / a.hkv;
  const int tpt = 128 / g;                           // tokens per row tile
  auto fail = [&](int where) {
    *abort = 1;
    *gabort = 1;
    set_status(a.status, PA_ERR_TIMEOUT, static_cast<int>(blockIdx.x), where);
  };
  auto wait_one = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait(bar, parity & 1, abort, a.wait_limit_ns, gabort);
  };
  // the same for a whole warp, one answer for all lanes
  auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_one(bar, parity)) != 0; };

  // Registers from the first four warps to the softmax: 128 x 128 + 256 x 184 =
  // 63488 of the 384 x 168 = 64512 that the block was launched with.
  if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    // -------------------------------------------------------------- softmax
    const int t = warp >= 8 ? 1 : 0;
    const int sub = warp & 3;
    const int rl = sub * 32 + lane;
    const uint32_t ginv = 65536u / g + 1;            // row / g for rows below 128, g <= 64: exact
    const int rt = static_cast<int>((rl * ginv) >> 16), rh = rl - rt * g;   // token and head of this thread's row
    const uint32_t s_tmem = tmem + (static_cast<uint32_t>(sub * 32) << 16) + t * 256;
    const uint32_t o_tmem = s_tmem + 128;
    const uint32_t o_oth = tmem + (static_cast<uint32_t>(sub * 32) << 16) + (t ^ 1) * 256 + 128;
    const uint64_t sc2 = f2_pack(C::SCALE, C::SCALE);
    uint8_t* stage = smem + C::OFF_OUT + (warp - 4) * 2048;
    uint32_t n_s = 0, n_own = 0, n_oth = 0;   // phases: scores, both final O's
    uint32_t ph_ml = 0;                       // and of both pairs of exchanged maxima, one bit each
    bool ok = true;
    for (int k = 0; ok; ++k) {
      // (read again for the output, so that little of it is held in registers beside the scores)
      int my, lim, lim_w, key_first, key_step;
      {
        if (!wait(&bars->work_full[k & 1], k >> 1)) { ok = false; break; }
        Item it;
        if (!get_item(bars, k, it)) break;
        const int tok_t = it.tok0 + (it.two ? t * tpt : 0);   // first token of this warpgroup's rows
        const bool valid = rl < tpt * g && tok_t + rt < it.q_len;
        lim = valid ? it.ctx + tok_t + rt : it.kv_len - 1;                   // last visible key
        lim_w = it.ctx + tok_t + static_cast<int>((sub * 32 * ginv) >> 16);   // the smallest of this warp's rows
        my = t == 0 ? it.nt0 : it.nt1;
        key_first = (it.kt0 + (it.two ? 0 : t)) * kKeyTile;
        key_step = it.two ? kKeyTile : 2 * kKeyTile;
      }
      float m_run = -INFINITY, l_run = 0.f;
      for (int i = 0; i < my; ++i) {
        const int key0 = key_first + i * key_step;
        if (!wait(&bars->s_full[t], n_s++)) { ok = false; break; }
        tc_fence_after();
        uint32_t sr[128];
        tmem_ld_x128(s_tmem, sr);
        if (key0 + kKeyTile - 1 > lim_w) {
          const int rel = lim - key0;                      // columns <= rel are visible
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (e > rel) sr[e] = __float_as_uint(-INFINITY);
        }
        float mx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mx[e] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 64; ++e)
          mx[e & 7] = fmax3(mx[e & 7], __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
        const float mt = fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(fmax3(mx[3], mx[4], mx[5]), mx[6], mx[7]));
        const float m_new = fmaxf(m_run, mt);
        const bool need = (m_new - m_run) * C::SCALE > 8.f;   // lazy rescale: only when P could exceed 2^8
        float alpha = 1.f;
        if (need) {
          alpha = fast_exp2((m_run - m_new) * C::SCALE);
          m_run = m_new;
        }
        const float m_use = (m_run == -INFINITY) ? 0.f : m_run * C::SCALE;
        const uint64_t nm2 = f2_pack(-m_use, -m_use);
        uint64_t acc2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc2[e] = 0ull;   // two 0.0f
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x0, x1, p0, p1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[32 * c + 2 * e]), __uint_as_float(sr[32 * c + 2 * e + 1])),
                             sc2, nm2), x0, x1);
            p0 = fast_exp2(x0);
            p1 = fast_exp2(x1);
            acc2[e & 3] = f2_add(acc2[e & 3], f2_pack(p0, p1));
            pk[e] = pack2(p0, p1);
          }
          tmem_st_x16(s_tmem + 16 * c, pk);
        }
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float a0, a1;
          f2_unpack(acc2[e], a0, a1);
          sum += a0 + a1;
        }
        l_run = l_run * alpha + sum;
        // O was last written by the previous PV, which completed before this S (the
        // commit signalling S covers every earlier MMA).
        if (FOLD && i > 0 && i % kFoldTiles == 0) {
          // O to its row, with what is there; this tile's PV writes O anew
          float* row = fold_row<D>(a, k, t * 128 + rl);
          const float old = i > kFoldTiles ? reweight(row[D], m_run, C::SCALE) : 0.f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t ov[32];
            tmem_ld_x32(o_tmem + c, ov);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float4* d4 = reinterpret_cast<float4*>(row + c) + e;
              float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
              if (i > kFoldTiles) x = *d4;
              x.x = x.x * old + __uint_as_float(ov[4 * e]) * alpha;
              x.y = x.y * old + __uint_as_float(ov[4 * e + 1]) * alpha;
              x.z = x.z * old + __uint_as_float(ov[4 * e + 2]) * alpha;
              x.w = x.w * old + __uint_as_float(ov[4 * e + 3]) * alpha;
              *d4 = x;
            }
          }
          row[D] = m_run;
        } else if (i > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld_x32(o_tmem + 32 * c, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st_x32(o_tmem + 32 * c, ov);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[t]);
      }
      if (!ok) break;
      // ---- the piece's output: its own O (two row tiles), or half of the
      // columns of both O's joined (one)
      if (!wait(&bars->noted[k & 1], k >> 1)) { ok = false; break; }
      Item it;
      get_item(bars, k, it);
      const bool two = it.two;
      const int tok_t = it.tok0 + (two ? t * tpt : 0);
      const bool valid = rl < tpt * g && tok_t + rt < it.q_len;
      const int n_other = t == 0 ? it.nt1 : it.nt0;
      float w_own = 1.f, w_oth = 0.f;
      // weights of what was folded, relative to O's
      const bool folded = FOLD && (my > kFoldTiles || (!two && n_other > kFoldTiles));
      float f_own = 0.f, f_oth = 0.f;
      if (FOLD && my > kFoldTiles) f_own = reweight(fold_row<D>(a, k, t * 128 + rl)[D], m_run, C::SCALE);
      if (!two) {
        float (*ml)[2][128] = bars->ml[k & 1];
        ml[t][0][rl] = m_run;
        ml[t][1][rl] = l_run;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->ml_full[k & 1][t]);
        if (!wait(&bars->ml_full[k & 1][t ^ 1], ph_ml >> (k & 1))) { ok = false; break; }
        ph_ml ^= 1u << (k & 1);
        const float m2 = ml[t ^ 1][0][rl], l2 = ml[t ^ 1][1][rl];
        if (FOLD && n_other > kFoldTiles) f_oth = reweight(fold_row<D>(a, k, (t ^ 1) * 128 + rl)[D], m2, C::SCALE);
        const float m = fmaxf(m_run, m2);
        if (m != -INFINITY) {
          w_own = fast_exp2((m_run - m) * C::SCALE);
          w_oth = fast_exp2((m2 - m) * C::SCALE);
        }
        l_run = l_run * w_own + l2 * w_oth;
        m_run = m;
      }
      if (my > 0 && !wait(&bars->o_final[t], n_own)) { ok = false; break; }
      if (!two && n_other > 0 && !wait(&bars->o_final[t ^ 1], n_oth)) { ok = false; break; }
      n_own += my > 0;
      n_oth += n_other > 0;
      tc_fence_after();
      const bool empty = l_run == 0.f;               // no visible key (a NaN sum is not zero)
      const float inv = empty ? 0.f : 1.f / l_run;
      const float lse = empty ? -INFINITY : ((m_run == -INFINITY ? 0.f : m_run * C::SCALE) + log2f(l_run)) * kLn2f;
      w_own *= inv;
      w_oth *= inv;
      f_own *= w_own;
      f_oth *= w_oth;
      const bool odd = *reinterpret_cast<volatile int*>(&bars->odd[k & 1]) == k + 1;
      const int64_t prow =
          (static_cast<int64_t>(it.part) * a.hkv + it.kvh) * a.tile_rows + (two ? t * tpt * g : 0) + rl;
      const int rows = min(tpt, it.q_len - tok_t) * g;     // rows of this tile
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) +
                           ((static_cast<int64_t>(it.row0) + tok_t) * a.hq + it.kvh * g) * D;
      if (valid && (two || t == 0)) {
        if (it.part >= 0) a.part_lse[prow] = lse;
        else if (a.lse) a.lse[(static_cast<int64_t>(it.row0) + tok_t + rt) * a.hq + it.kvh * g + rh] = lse;
      }
      // What is read of shared memory is handed back by an ordinary arrival, which
      // orders the reads before whoever writes there next: before the output,
      // whose stores it would wait for, unless there are notes, or rows that were
      // folded, to read behind it.
      auto hand_back = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->read[k & 1]);
      };
      if (!odd && !folded) hand_back();
      // 32 columns at a time; with one row tile each warpgroup writes half of them
      const int c_lo = two ? 0 : t * (D / 2), c_hi = two ? D : c_lo + D / 2;
      // (below, four lanes write 64 bytes of a row: rows 8 x + lane / 4 of the warp)
      int at[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = sub * 32 + 8 * x + (lane >> 2), tk = static_cast<int>((row * ginv) >> 16);
        at[x] = row < rows ? (tk * a.hq + (row - tk * g)) * D + 8 * (lane & 3) : -1;
      }
#pragma unroll 1
      for (int c = c_lo; c < c_hi; c += 32) {
        uint32_t ov[32];
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0.f;
        if (my > 0) {
          tmem_ld_x32(o_tmem + c, ov);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(ov[e]) * w_own;
        }
        if (!two && n_other > 0) {
          tmem_ld_x32(o_oth + c, ov);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] += __uint_as_float(ov[e]) * w_oth;
        }
        if (FOLD && folded) {
          auto add = [&](int row, float w) {
            const float4* s4 = reinterpret_cast<const float4*>(fold_row<D>(a, k, row) + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 x = s4[e];
              v[4 * e] += x.x * w;
              v[4 * e + 1] += x.y * w;
              v[4 * e + 2] += x.z * w;
              v[4 * e + 3] += x.w * w;
            }
          };
          if (my > kFoldTiles) add(t * 128 + rl, f_own);
          if (!two && n_other > kFoldTiles) add((t ^ 1) * 128 + rl, f_oth);
        }
        if (it.part >= 0) {
          if (valid) {
            float4* d4 = reinterpret_cast<float4*>(a.part_o + prow * D + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) d4[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          }
        } else {
          // through shared memory, so that a store writes 64-byte pieces of rows
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(pack2(v[8 * e], v[8 * e + 1]), pack2(v[8 * e + 2], v[8 * e + 3]),
                           pack2(v[8 * e + 4], v[8 * e + 5]), pack2(v[8 * e + 6], v[8 * e + 7]));
          __syncwarp();
          uint4 w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = *reinterpret_cast<const uint4*>(stage + (8 * x + (lane >> 2)) * 64 +
                                                   (((lane & 3) ^ ((lane >> 3) & 3)) << 4));
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (at[x] >= 0) *reinterpret_cast<uint4*>(out + at[x] + c) = w[x];
        }
      }
      if (odd) {
        // columns with a non-finite value that this row sees: what the sum would be
        __syncwarp();
        const unsigned long long tag = static_cast<unsigned long long>(~static_cast<uint32_t>(k + 1)) << 32;
        auto seen = [&](int kind, int col) {
          const unsigned long long x = bars->first[k & 1][kind][col];
          return (x & 0xffffffff00000000ull) == tag && static_cast<int>(x & 0xffffffffu) <= lim;
        };
        for (int c = c_lo; valid && c < c_hi; ++c) {
          const bool pos = seen(0, c), neg = seen(1, c), nan = seen(2, c) || (pos && neg);
          if (!pos && !neg && !nan) continue;
          const float add = nan ? __int_as_float(0x7fc00000) : pos ? INFINITY : -INFINITY;
          if (it.part >= 0) {
            a.part_o[prow * D + c] += add;
          } else {
            __nv_bfloat16* x = out + (static_cast<int64_t>(rt) * a.hq + rh) * D + c;
            *x = __float2bfloat16_rn(__bfloat162float(*x) + add);
          }
        }
      }
      if (odd || folded) hand_back();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(&bars->done[k & 1]);   // O has been read
    }
    if (!ok) fail(9);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 128;");
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      const int nbox = kKeyTile / p.box_rows;
      const int q_bytes = tpt * g * 128 * C::NKB;
      uint32_t tile = 0;                  // K and V tiles before this one
      uint32_t n_q = 0, n_k = 0;          // copies issued: Q's and K tiles,
      uint32_t n_v0 = 0, n_v1 = 0, n_g0 = 0, n_g1 = 0;   // V tiles of each stage, guarded ones
      // Units of work: this block's first, then whichever comes next over all
      // blocks (the deepest come first, so the blocks end together).
      const unsigned total = static_cast<unsigned>(a.head->n_pieces) * static_cast<unsigned>(a.hkv);
      unsigned unit = blockIdx.x;
      int at = 0, kvh = -1;
      Piece after = {};                   // the piece after the current one
      auto fetch = [&]() {
        kvh = -1;
        if (unit < total) {
          piece_at(a, unit, &at, &kvh);
          const int4* src = reinterpret_cast<const int4*>(a.pieces + at);
          const int4 x = src[0], y = src[1];
          after = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        }
      };
      fetch();
      bool ok = true;
      Item it;
      for (int k = 0; ok; ++k) {
        // the slot's previous piece (two before) is finished
        if (k >= 2 && !(wait(&bars->done[k & 1], (k >> 1) - 1) && wait(&bars->read[k & 1], (k >> 1) - 1))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          put_item(bars, k, tpt, after, kvh);
          mbar_arrive(&bars->work_full[k & 1]);
        }
        __syncwarp();
        if (!get_item(bars, k, it)) break;
        // row coordinate of this lane's box of tile j
        auto row_of = [&](int j) -> int {
          if (!PAGED) return it.row0 + j * kKeyTile;
          const int64_t key = static_cast<int64_t>(j) * kKeyTile + lane * p.box_rows;
          if (lane >= nbox || key >= it.kv_len) return p.oob_row;
          const int64_t slot = key_slot(a, it.b, key);
          return slot < 0 ? p.oob_row : static_cast<int>(slot);
        };
        int row = it.n > 0 ? row_of(it.kt0) : 0;
        if (k > 0 && !wait(&bars->q_empty, k - 1)) { ok = false; break; }
        if (lane == 0) {
          const int qt = it.two ? 2 : 1;
          mbar_arrive_expect_tx(&bars->q_full, qt * q_bytes + (a.stall ? 16 : 0));
          for (int t = 0; t < qt; ++t)
            for (int kb = 0; kb < C::NKB; ++kb)
              tma_load_3d(sQ + t * C::TILE_BYTES + kb * C::KB_BYTES, &tmQ, &bars->q_full, kb * 64, it.kvh * g,
                          it.row0 + it.tok0 + t * tpt);
        }
        ++n_q;
        for (int jj = 0; jj < it.n; ++jj, ++tile) {
          const int st = tile & 1;
          const uint32_t ph = tile >> 1;
          const int next = jj + 1 < it.n ? row_of(it.kt0 + jj + 1) : 0;
          if (!wait(&bars->k_empty[st], ph + 1)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&bars->k_full[st], C::TILE_BYTES);
          __syncwarp();
          if (lane < nbox)
            for (int kb = 0; kb < C::NKB; ++kb)
              tma_load_3d(sK + st * C::TILE_BYTES + kb * C::KB_BYTES + lane * p.box_rows * 128, &tmK,
                          &bars->k_full[st], kb * 64, it.kvh, row);
          ++n_k;
          if (!wait(&bars->v_empty[st], ph + 1)) { ok = false; break; }
          const bool guarded = jj >= it.g0;
          uint64_t* full = guarded ? &bars->vg_full[st] : &bars->v_full[st];
          if (lane == 0) mbar_arrive_expect_tx(full, C::TILE_BYTES);
          __syncwarp();
          if (lane < nbox)
            for (int kb = 0; kb < C::NKB; ++kb)
              tma_load_3d(sV + st * C::TILE_BYTES + kb * C::KB_BYTES + lane * p.box_rows * 128, &tmV, full, kb * 64,
                          it.kvh, row);
          n_v0 += !guarded && st == 0;
          n_v1 += !guarded && st == 1;
          n_g0 += guarded && st == 0;
          n_g1 += guarded && st == 1;
          row = next;
        }
        // (not before: a unit taken early would wait here while other blocks run out of work)
        if (lane == 0) unit = gridDim.x + atomicAdd(&a.head->next, 1u);
        unit = __shfl_sync(0xffffffffu, unit, 0);
        fetch();
      }
      if (lane == 0) {
        if (!ok) fail(1);
        // Drain: every copy this warp started has landed before the block ends.
        int zero = 0;
        auto landed = [&](uint64_t* bar, uint32_t count) {
          if (count > 0) mbar_wait(bar, (count - 1) & 1, &zero, a.wait_limit_ns);
        };
        landed(&bars->q_full, n_q);
        landed(&bars->k_full[0], (n_k + 1) >> 1);
        landed(&bars->k_full[1], n_k >> 1);
        landed(&bars->v_full[0], n_v0);
        landed(&bars->v_full[1], n_v1);
        landed(&bars->vg_full[0], n_g0);
        landed(&bars->vg_full[1], n_g1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issue
      if (lane == 0) {
        const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t k_desc = sdesc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t v_desc = sdesc_sw128(smem_u32(sV), C::KB_BYTES, 1024);
        // scores of warpgroup t from row tile qt
        auto qk = [&](int t, int qt, int st) {
          const uint32_t d_tmem = tmem + t * 256;
          const uint64_t qd = sdesc_add(q_desc, qt * C::TILE_BYTES);
          const uint64_t kd = sdesc_add(k_desc, st * C::TILE_BYTES);
  #pragma unroll
          for (int kb = 0; kb < C::NKB; ++kb)
  #pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ss(d_tmem, sdesc_add(qd, kb * C::KB_BYTES + ks * 32), sdesc_add(kd, kb * C::KB_BYTES + ks * 32),
                     C::IDESC_QK, (kb | ks) != 0);
          mma_commit(&bars->s_full[t]);
        };
        auto pv = [&](int t, int st, int acc) {
          const uint32_t d_tmem = tmem + t * 256 + 128;
          const uint64_t vd = sdesc_add(v_desc, st * C::TILE_BYTES);
  #pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ts(d_tmem, tmem + t * 256 + ks * 8, sdesc_add(vd, ks * 2048), C::IDESC_PV, (acc | ks) != 0);
        };
        uint32_t tile = 0;                        // K and V tiles before this piece
        // phases, one bit each: of each warpgroup's P, and of each stage's V
        // tiles and guarded V tiles
        uint32_t ph_p = 0, ph_v = 0, ph_g = 0;
        auto next = [](uint32_t& bits, int i) {
          const uint32_t b = (bits >> i) & 1;
          bits ^= 1u << i;
          return b;
        };
        auto wait_k = [&](uint32_t x) { return wait_one(&bars->k_full[x & 1], x >> 1); };
        bool ok = true;
        Item it;
        for (int k = 0; ok; ++k, tile += it.n) {
          if (!wait_one(&bars->work_full[k & 1], k >> 1)) { fail(2); break; }
          if (!get_item(bars, k, it)) break;
          mbar_arrive(&bars->read[k & 1]);
          const int n = it.n;
          auto wait_v = [&](int jj) {
            const int st = (tile + jj) & 1;
            return jj < it.g0 ? wait_one(&bars->v_full[st], next(ph_v, st))
                              : wait_one(&bars->v_ready[st], next(ph_g, st));
          };
          // the previous piece's O has been read before the first P V of this one
          auto wait_o = [&]() { return k == 0 || wait_one(&bars->done[(k - 1) & 1], (k - 1) >> 1); };
          if (!wait_one(&bars->q_full, k)) { fail(3); break; }
          if (n == 0) {
            mma_commit(&bars->q_empty);
          } else if (it.two) {
            if (!wait_k(tile)) { fail(4); break; }
            tc_fence_after();
            if (it.nt0 > 0) qk(0, 0, tile & 1);
            qk(1, 1, tile & 1);
            mma_commit(&bars->k_empty[tile & 1]);
            if (n == 1) mma_commit(&bars->q_empty);
            for (int jj = 0; ok && jj < n; ++jj) {
              const int st = (tile + jj) & 1, st1 = st ^ 1;
              // V_j and K_{j+1} first, while the tensor pipe still runs the other
              // tile's MMAs, so that nothing stands between P and its products
              if (!wait_v(jj)) { fail(6); ok = false; break; }
              if (jj + 1 < n && !wait_k(tile + jj + 1)) { fail(7); ok = false; break; }
              if (jj == 0 && !wait_o()) { fail(12); ok = false; break; }
  #pragma unroll
              for (int t = 0; t < 2; ++t) {
                const int nt = t == 0 ? it.nt0 : n;
                if (jj < nt) {
                  if (!wait_one(&bars->p_full[t], next(ph_p, t))) { fail(5); ok = false; break; }
                  tc_fence_after();
                  pv(t, st, FOLD ? jj % kFoldTiles != 0 : jj > 0);
                  if (jj == nt - 1) mma_commit(&bars->o_final[t]);
                }
                if (t == 1) mma_commit(&bars->v_empty[st]);
                if (jj + 1 < nt) qk(t, t, st1);
              }
              if (ok && jj + 1 < n) {
                mma_commit(&bars->k_empty[st1]);
                if (jj + 2 == n) mma_commit(&bars->q_empty);
              }
            }
          } else {
            for (int jj = 0; jj < min(n, 2); ++jj) {
              if (!wait_k(tile + jj)) { fail(4); ok = false; break; }
              tc_fence_after();
              qk(jj, 0, (tile + jj) & 1);
              mma_commit(&bars->k_empty[(tile + jj) & 1]);
            }
            if (!ok) break;
            if (n <= 2) mma_commit(&bars->q_empty);
            for (int jj = 0; jj < n; ++jj) {
              const int t = jj & 1, i = jj >> 1, st = (tile + jj) & 1;
              if (!wait_v(jj)) { fail(6); ok = false; break; }
              if (jj + 2 < n && !wait_k(tile + jj + 2)) { fail(7); ok = false; break; }
              if (jj == 0 && !wait_o()) { fail(12); ok = false; break; }
              if (!wait_one(&bars->p_full[t], next(ph_p, t))) { fail(5); ok = false; break; }
              tc_fence_after();
              pv(t, st, FOLD ? i % kFoldTiles != 0 : i > 0);
              if (jj + 2 >= n) mma_commit(&bars->o_final[t]);
              mma_commit(&bars->v_empty[st]);
              if (jj + 2 < n) {
                qk(t, 0, st);
                mma_commit(&bars->k_empty[st]);
                if (jj + 3 == n) mma_commit(&bars->q_empty);
              }
            }
          }
        }
        // Drain: all MMAs issued by this thread complete before TMEM is freed.
        int zero = 0;
        mma_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, &zero, a.wait_limit_ns);
      }
    } else if (warp < 4) {
      // ---------------------------------------------------------- V guard
      const int tid = threadIdx.x - 64;
      uint32_t tile = 0, ph_g = 0;   // ph_g: phase bit of each stage's guarded tiles
      bool ok = true;
      Item it;
      for (int k = 0; ok; ++k, tile += it.n) {
        // (a piece is there only when the one two before, whose notes it takes over, is finished)
        if (!wait(&bars->work_full[k & 1], k >> 1)) { ok = false; break; }
        if (!get_item(bars, k, it)) break;
        const int lim_first = it.ctx + it.tok0;
        for (int jj = it.g0; jj < it.n; ++jj) {
          const int st = (tile + jj) & 1;
          if (!wait(&bars->vg_full[st], ph_g >> st)) { ok = false; break; }
          ph_g ^= 1u << st;
          const int key0 = (it.kt0 + jj) * kKeyTile;
          guard_tile<D>(sV + st * C::TILE_BYTES, max(0, lim_first + 1 - key0), it.kv_len - key0, key0, k, bars, tid);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->v_ready[st]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->noted[k & 1]);
      }
      if (!ok && lane == 0) fail(11);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool PAGED, bool FOLD>
int launch_tc(const AttendArgs& a, cudaStream_t s) {
  using C = SvCfg<D>;
  const int g = a.hq / a.hkv;
  SvParams p;
  p.a = a;
  // roles wait for one another for up to a piece: 10 us for each of its key tiles,
  // which take 2 us (0.01 s for 128K keys)
  const int64_t deepest = PAGED ? static_cast<int64_t>(a.max_pages) * a.page_size : a.N;
  p.a.wait_limit_ns += static_cast<uint64_t>(deepest / kKeyTile) * 10000u;
  p.box_rows = PAGED && a.page_size < kKeyTile ? a.page_size : kKeyTile;
  // an empty cache has no page to read: every box is out of range, and the
  // map is made over q only to have an address
  const int64_t rows = a.n_slots > 0 ? a.n_slots : 1;
  p.oob_row = static_cast<int>(rows);
  CUtensorMap mq, mk, mv;
  const void* k = a.n_slots > 0 ? a.k : a.q;
  const void* v = a.n_slots > 0 ? a.v : a.q;
  if (!rows_map(&mq, a.q, a.N, a.hq, D, a.ldq, g, 128 / g) ||
      !rows_map(&mk, k, rows, a.hkv, D, a.ldk, 1, p.box_rows) ||
      !rows_map(&mv, v, rows, a.hkv, D, a.ldv, 1, p.box_rows))
    return PA_ERR_CUDA;
  const int rc = allow_smem<attend_tc_kernel<D, PAGED, FOLD>>(C::SMEM_BYTES);
  if (rc != PA_OK) return rc;
  const unsigned units = tile_blocks(a);
  return launch_overlapped(attend_tc_kernel<D, PAGED, FOLD>, dim3(units < kSms ? units : kSms), 384, C::SMEM_BYTES, s, mq,
                           mk, mv, p);
}
template <int D>
int launch_tc_for(const AttendArgs& a, cudaStream_t s) {
  if (a.block_table) return a.fold ? launch_tc<D, true, true>(a, s) : launch_tc<D, true, false>(a, s);
  return a.fold ? launch_tc<D, false, true>(a, s) : launch_tc<D, false, false>(a, s);
}

}  // namespace

bool rows_map(void* map, const void* base, int64_t rows, int heads, int d, int64_t ld, int box_heads,
              int box_rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(static_cast<CUtensorMap*>(map), CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_attend_tc(const AttendArgs& a, cudaStream_t s) {
  return a.d == 128 ? launch_tc_for<128>(a, s) : launch_tc_for<64>(a, s);
}

}  // namespace pa
