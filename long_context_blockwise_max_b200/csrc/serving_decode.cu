// Attention of few rows per request (generated tokens) over the paged cache,
// bf16: the HBM-streaming path.
//
// At most 16 (token, query head) rows share a kv head's keys, so the cache's
// bytes are the cost and warp-level MMAs (mma.sync m16n8k16) have ample
// rate.  The work of a call is a row of 128-key groups, over requests, kv
// heads and keys; the plan gives each of the 148 blocks an equal range of it,
// whatever the lengths, so that no SM waits for the longest request.
//
// Each of the 4 warps takes 32 keys of a group and streams them through its
// own 3-stage ring of TMA copies (one box per page or 32 keys and 64 columns;
// copies by the warps' own 16-byte accesses kept each warp busy for a third of
// a tile's time).  The ring runs across the ends of requests and heads: the
// copies of the next range are in flight while a finished one is merged.  A
// key's page is looked up one group ahead of its copy.
//
// With at most 8 rows, the probabilities go in as a bf16 pair, high part in
// MMA rows 0-7 and residual in rows 8-15, at no extra MMA; with 9 to 16 rows
// they are rounded to bf16.
//
// An accumulator of the MMA loses the bits that one addition cannot hold, always
// towards zero (o 9e-3 too small over 1.8M keys in one warp, equal weights): where
// a warp may have more keys of a pair than kFoldKeys, it adds its o to its part of
// the merge memory after every so many and starts anew (FOLD, a kernel of its own).
//
// Rows whose keys lie in several blocks' ranges leave partial results in the
// workspace; the last block to arrive merges them in block order, so results
// do not depend on which block that is.
//
// HBM-bound when long: 16 tokens over 128K keys each, 32 / 8 heads of 128, 1226
// to 1290 us (between boxes) for 8.59 GB = 6.66 to 7.0 TB/s, 1.02 to 1.07 of a copy's
// rate.  Latency-bound when short: 8 tokens behind up to 1467 keys 13.6 to 14.1 us, of
// which 7 are a block's own (table, copies and 32 keys' chain 2 us, parts and arrival
// 2 us, the last one's merge 1 us) and the rest the plan and two launches.
#include "serving.h"
#include "sm100.cuh"

namespace pa {
using namespace sm100;


namespace {

constexpr int kWarps = 4;
constexpr int kKT = 32;      // keys per warp tile
constexpr int kStages = 3;
constexpr int kMergeAhead = 8;   // parts of a cut pair that are loaded together
constexpr int kFoldKeys = kFoldTiles * kPlanTile;   // keys that an accumulator adds up at most
static_assert(kWarps * kKT == kPlanTile, "a block's step is one planned key group");

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
struct DecCfg {
  static constexpr int CH = D / 8;                    // 16-byte chunks per key row
  static constexpr int NKB = D / 64;                  // column blocks of 32 keys x 128 B
  static constexpr int KB = kKT * 128;
  static constexpr int TILE = NKB * KB;               // K (or V) tile bytes
  static constexpr int STAGE = 2 * TILE;              // K + V
  static constexpr int RING = kStages * STAGE;        // per warp
  static constexpr int OFF_RED = kWarps * RING;       // [warp][16][D] floats
  static constexpr int OFF_ML = OFF_RED + kWarps * 16 * D * 4;   // [2][warp][16] floats
  static constexpr int OFF_BAD = OFF_ML + 2 * kWarps * 16 * 4;   // [3][D] first key with +inf, -inf, NaN
  static constexpr int OFF_BAR = OFF_BAD + 3 * D * 4;            // [warp][stage] copies have landed
  static constexpr int OFF_FLAG = OFF_BAR + kWarps * kStages * 8;
  static constexpr int SMEM = OFF_FLAG + 16 + 768;    // the base is aligned to 1024 bytes (it is to 256 already)
  static constexpr float SCALE = static_cast<float>(kLog2e / (D == 128 ? 11.31370849898476039 : 8.0));
};

// byte offset of (key row, 16-byte chunk) inside a tile (128-byte swizzle)
template <int D>
__device__ __forceinline__ uint32_t swz(int key, int chunk) {
  return (chunk >> 3) * DecCfg<D>::KB + key * 128 + (((chunk & 7) ^ (key & 7)) << 4);
}

// A place in the row of key groups: request, kv head, group of that pair.
struct Cursor {
  int b, kvh, unit, n_units;
  int kv, q, row0;

  __device__ __forceinline__ void load(const AttendArgs& a) {
    row0 = a.cu_q[b];
    const int64_t rows = static_cast<int64_t>(a.cu_q[b + 1]) - row0;
    q = rows > 0 && rows <= a.max_q ? static_cast<int>(rows) : 0;
    kv = a.kv_len[b];
    n_units = kv > 0 ? (kv - 1) / kPlanTile + 1 : 1;   // (kv may be as large as the type allows)
  }
  // requests that are not this kernel's (or were found invalid by the plan)
  // have no groups; the caller steps at most as many times as there are groups
  __device__ __forceinline__ bool mine(const AttendArgs& a, int64_t max_kv) const {
    return row0 >= 0 && q > 0 && static_cast<int64_t>(row0) + q <= a.N && kv >= 0 && kv <= max_kv &&
           static_cast<int64_t>(q) * (a.hq / a.hkv) <= a.small_rows;
  }
  __device__ __forceinline__ void step(const AttendArgs& a, int64_t max_kv) {
    if (++unit < n_units) return;
    unit = 0;
    if (++kvh < a.hkv) return;
    kvh = 0;
    do {
      if (++b >= a.B) return;
      load(a);
    } while (!mine(a, max_kv));
  }
};

template <int D, bool FOLD>
__global__ void __launch_bounds__(kWarps * 32, 1) attend_decode_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                       const __grid_constant__ CUtensorMap tmV,
                                                                       const __grid_constant__ AttendArgs a,
                                                                       int box_rows, int oob_row) {
  using C = DecCfg<D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * C::RING;
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
  float* red_m = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* red_l = red_m + kWarps * 16;
  int* bad = reinterpret_cast<int*>(smem + C::OFF_BAD);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * kStages;
  // [0] non-finite V, [1] last to arrive, [2] a wait ran out
  volatile int* flag = reinterpret_cast<volatile int*>(smem + C::OFF_FLAG);
  for (int i = threadIdx.x; i < 3 * D; i += kWarps * 32) bad[i] = INT32_MAX;
  if (threadIdx.x == 0) flag[0] = flag[2] = 0;
  if (lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  grid_dep_wait();      // the set-up above overlaps the plan
  grid_dep_launch();

  const DecodeStart ds = a.starts[blockIdx.x];
  const int steps = ds.steps;
  if (steps == 0) return;
  const int64_t u_lo = ds.first;
  auto block_of = [&](int64_t u) {   // the block whose range holds group u
    const int64_t cut = ds.more * (ds.each + 1);
    if ((u >> 31) == 0) {            // (32-bit divisions, unless there are that many groups)
      const uint32_t v = static_cast<uint32_t>(u), e = static_cast<uint32_t>(ds.each);
      return u < cut ? static_cast<int>(v / (e + 1)) : ds.more + static_cast<int>((v - static_cast<uint32_t>(cut)) / e);
    }
    return static_cast<int>(u < cut ? u / (ds.each + 1) : ds.more + (u - cut) / ds.each);
  };
  const int64_t max_kv = static_cast<int64_t>(a.max_pages) * a.page_size;
  const int g = a.hq / a.hkv;
  Cursor ahead = {ds.b, ds.kvh, ds.unit, ds.n_units, ds.kv, ds.q, ds.row0};   // the next group to be issued
  Cursor cur = ahead;                                                         // the computation's place
  // row coordinate of this lane's box of the group at `ahead`
  const int nbox = kKT / box_rows;
  auto look_up = [&]() -> int {
    const int64_t key = static_cast<int64_t>(ahead.unit) * kPlanTile + warp * kKT + lane * box_rows;
    if (lane >= nbox || key >= ahead.kv) return oob_row;
    const int64_t slot = key_slot(a, ahead.b, key);
    return slot < 0 ? oob_row : static_cast<int>(slot);
  };
  int row = look_up();
  int issued = 0;
  auto issue = [&](int it) {
    if (it >= steps || __any_sync(0xffffffffu, flag[2])) return;   // (one answer for the warp)
    ++issued;
    uint8_t* dst = ring + (it % kStages) * C::STAGE;
    uint64_t* bar = &full[it % kStages];
    if (lane == 0) mbar_arrive_expect_tx(bar, C::STAGE + (a.stall && it == 0 ? 16 : 0));
    __syncwarp();
    if (lane < nbox)
#pragma unroll
      for (int kb = 0; kb < C::NKB; ++kb) {
        tma_load_3d(dst + kb * C::KB + lane * box_rows * 128, &tmK, bar, kb * 64, ahead.kvh, row);
        tma_load_3d(dst + C::TILE + kb * C::KB + lane * box_rows * 128, &tmV, bar, kb * 64, ahead.kvh, row);
      }
    if (it + 1 < steps) {
      ahead.step(a, max_kv);
      row = look_up();
    }
  };

  const int qi = lane >> 2, qc = (lane & 3) * 2;
  uint32_t qa[D / 16][4];
  float o[D / 8][4];
  float m0 = -INFINITY, l0 = 0.f, m1 = -INFINITY, l1 = 0.f;   // rows qi and qi + 8
  int rows = 0, ctx = 0;
  int lim0 = -1, lim1 = -1;
  bool pair = true;             // at most 8 rows: P as a high part and a residual
  int since = 0;                // FOLD: tiles in o; whether there are more in the merge memory
  bool folded = false;
  auto begin = [&]() {
    rows = cur.q * g;
    ctx = cur.kv - cur.q;
    pair = rows <= 8;
    const int r1 = qi + 8;
    lim0 = qi < rows ? ctx + qi / g : -1;
    lim1 = r1 < rows ? ctx + r1 / g : -1;
    const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.q);
    const __nv_bfloat16* q0 = Q + (static_cast<int64_t>(cur.row0) + qi / g) * a.ldq + (cur.kvh * g + qi % g) * D + qc;
    const __nv_bfloat16* q1 = Q + (static_cast<int64_t>(cur.row0) + r1 / g) * a.ldq + (cur.kvh * g + r1 % g) * D + qc;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qa[ks][0] = qi < rows ? *reinterpret_cast<const uint32_t*>(q0 + 16 * ks) : 0u;
      qa[ks][1] = r1 < rows ? *reinterpret_cast<const uint32_t*>(q1 + 16 * ks) : 0u;
      qa[ks][2] = qi < rows ? *reinterpret_cast<const uint32_t*>(q0 + 16 * ks + 8) : 0u;
      qa[ks][3] = r1 < rows ? *reinterpret_cast<const uint32_t*>(q1 + 16 * ks + 8) : 0u;
    }
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
    if (FOLD) {
      since = 0;
      folded = false;
    }
  };
  // o so far, with what was folded before: to this warp's part of the merge memory
  // (each thread its own elements of it), o being relative to the maxima m0, m1
  auto put = [&]() {
    float f0 = 0.f, f1 = 0.f;
    if (FOLD && folded) {
      const float a0 = red_m[warp * 16 + qi], a1 = red_m[warp * 16 + qi + 8];
      f0 = a0 == m0 ? 1.f : fast_exp2((a0 - m0) * C::SCALE);
      f1 = a1 == m1 ? 1.f : fast_exp2((a1 - m1) * C::SCALE);
    }
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      float2 lo = make_float2(o[j][0], o[j][1]);
      float2* r0 = reinterpret_cast<float2*>(red + (warp * 16 + qi) * D + 8 * j + qc);
      if (pair) {
        lo.x += o[j][2];
        lo.y += o[j][3];
      } else {
        float2 hi = make_float2(o[j][2], o[j][3]);
        float2* r1 = reinterpret_cast<float2*>(red + (warp * 16 + qi + 8) * D + 8 * j + qc);
        if (FOLD && folded) hi = make_float2(r1->x * f1 + hi.x, r1->y * f1 + hi.y);
        *r1 = hi;
      }
      if (FOLD && folded) lo = make_float2(r0->x * f0 + lo.x, r0->y * f0 + lo.y);
      *r0 = lo;
    }
    __syncwarp();   // the old maxima have been read
    if ((lane & 3) == 0) {
      red_m[warp * 16 + qi] = m0;
      red_m[warp * 16 + qi + 8] = m1;
    }
  };

#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  begin();
  for (int it = 0; it < steps; ++it) {
    issue(it + kStages - 1);
    const int st = it % kStages;
    if (!mbar_wait(&full[st], (it / kStages) & 1, flag + 2, a.wait_limit_ns, &a.head->abort)) {
      // every warp keeps to its steps (they share barriers), on whatever is there
      flag[2] = 1;
      a.head->abort = 1;
      set_status(a.status, PA_ERR_TIMEOUT, static_cast<int>(blockIdx.x), warp);
    }
    __syncwarp();
    const uint32_t sK = smem_u32(ring + st * C::STAGE);
    const uint32_t sV = sK + C::TILE;
    const int key0 = cur.unit * kPlanTile + warp * kKT;
    if (key0 < cur.kv) {
      const bool edge = key0 + kKT - 1 > ctx;   // some row does not see some key of this tile
      if (edge) {
        // V of keys that not every row sees: rows without a key are zeroed,
        // and a non-finite value is taken out of the product and noted (the
        // rows that see it get it at the end)
        uint8_t* v = ring + st * C::STAGE + C::TILE;
        const int n_keys = cur.kv - key0;
#pragma unroll
        for (int i = 0; i < C::CH; ++i) {
          const int x = i * 32 + lane;
          if (x / C::CH >= n_keys) *reinterpret_cast<uint4*>(v + swz<D>(x / C::CH, x % C::CH)) = make_uint4(0, 0, 0, 0);
        }
        // (a single new token sees every key there is)
        const int hidden = max(0, ctx + 1 - key0), end = min(n_keys, kKT);
        for (int i = hidden * C::CH + lane; i < end * C::CH; i += 32) {
          const int key = key0 + i / C::CH, c = i % C::CH;
          uint16_t* e = reinterpret_cast<uint16_t*>(v + swz<D>(i / C::CH, c));
          for (int k = 0; k < 8; ++k)
            if ((e[k] & 0x7f80) == 0x7f80) {
              atomicMin(&bad[((e[k] & 0x7f) ? 2 : (e[k] >> 15)) * D + 8 * c + k], key);
              flag[0] = 1;
              e[k] = 0;
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the next copy into this stage
        __syncwarp();
      }
      // S = Q K^T over 32 keys: 4 n8 tiles
      float s[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
          uint32_t kb[4];
          ldsm_x4(sK + swz<D>(nt * 8 + (lane & 7), kk * 4 + (lane >> 3)), kb);
          mma_bf16(s[nt], qa[2 * kk], kb[0], kb[1]);
          mma_bf16(s[nt], qa[2 * kk + 1], kb[2], kb[3]);
        }
      }
      float t0 = m0, t1 = m1;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (edge) {
            const int key = key0 + nt * 8 + qc + e;
            if (key > lim0) s[nt][e] = -INFINITY;
            if (key > lim1) s[nt][e + 2] = -INFINITY;
          }
          t0 = fmaxf(t0, s[nt][e]);
          t1 = fmaxf(t1, s[nt][e + 2]);
        }
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
      // a row that has seen no key: nothing to scale, exponents of -inf
      const float sub0 = t0 == -INFINITY ? 0.f : t0 * C::SCALE, sub1 = t1 == -INFINITY ? 0.f : t1 * C::SCALE;
      const float al0 = fast_exp2(m0 * C::SCALE - sub0);
      const float al1 = pair ? al0 : fast_exp2(m1 * C::SCALE - sub1);
      const bool grew = t0 != m0 || (!pair && t1 != m1);
      m0 = t0;
      m1 = t1;
      if (__any_sync(0xffffffffu, grew)) {
        l0 *= al0;
        l1 *= al1;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= al0;
          o[j][1] *= al0;
          o[j][2] *= al1;
          o[j][3] *= al1;
        }
      }
      uint32_t pf[2][4];        // P as A fragments, two k16 steps
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float p0 = fast_exp2(fmaf(s[nt][0], C::SCALE, -sub0)), p1 = fast_exp2(fmaf(s[nt][1], C::SCALE, -sub0));
        l0 += p0 + p1;
        const uint32_t hi = pack_bf16(p0, p1);
        pf[nt >> 1][(nt & 1) * 2] = hi;
        if (pair) {
          pf[nt >> 1][(nt & 1) * 2 + 1] =
              pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
        } else {
          const float p2 = fast_exp2(fmaf(s[nt][2], C::SCALE, -sub1)), p3 = fast_exp2(fmaf(s[nt][3], C::SCALE, -sub1));
          l1 += p2 + p3;
          pf[nt >> 1][(nt & 1) * 2 + 1] = pack_bf16(p2, p3);
        }
      }
      // O += P V over 32 keys: 2 k16 steps x D / 8 n8 tiles
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
        for (int cj = 0; cj < D / 16; ++cj) {
          uint32_t vb[4];
          const int mtx = lane >> 3;
          ldsm_x4_t(sV + swz<D>(k2 * 16 + (mtx & 1) * 8 + (lane & 7), cj * 2 + (mtx >> 1)), vb);
          mma_bf16(o[2 * cj], pf[k2], vb[0], vb[1]);
          mma_bf16(o[2 * cj + 1], pf[k2], vb[2], vb[3]);
        }
      if (FOLD && ++since == kFoldKeys / kKT) {
        put();
        folded = true;
        since = 0;
        __syncwarp();   // its maxima are written
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      }
    }
    __syncwarp();   // the stage is refilled by the next issue
    const bool item_end = cur.unit == cur.n_units - 1;
    if (!item_end && it != steps - 1) {
      ++cur.unit;
      continue;
    }
    // ---- this block's keys of the pair are done: merge the warps -----------
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    put();
    if ((lane & 3) == 0) {
      red_l[warp * 16 + qi] = l0;
      red_l[warp * 16 + qi + 8] = l1;
    }
    __syncthreads();
    // the range of blocks that share this pair's keys
    const int64_t item_lo = u_lo + it - cur.unit;
    const bool whole = item_lo >= u_lo && item_lo + cur.n_units <= u_lo + steps;
    const int c_lo = whole || item_lo >= u_lo ? static_cast<int>(blockIdx.x) : block_of(item_lo);
    const int c_hi = whole || item_end ? static_cast<int>(blockIdx.x) : block_of(item_lo + cur.n_units - 1);
    // a block's partial slots: 0 for a pair that begins before its range, 1 for one that begins in it
    auto slot_of = [&](int c) { return 2 * c + (c == c_lo ? 1 : 0); };
    const int64_t out0 = static_cast<int64_t>(slot_of(blockIdx.x)) * 16;
    const bool odd = flag[0] != 0;
    for (int i = threadIdx.x; i < rows * C::CH; i += kWarps * 32) {
      const int r = i / C::CH, c = i % C::CH;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_m[w * 16 + r]);
      const float sub = M == -INFINITY ? 0.f : M * C::SCALE;
      float L = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = fast_exp2(red_m[w * 16 + r] * C::SCALE - sub);
        L += f * red_l[w * 16 + r];
        const float4* src = reinterpret_cast<const float4*>(red + (w * 16 + r) * D + 8 * c);
        const float4 x = src[0], y = src[1];
        acc[0] += f * x.x; acc[1] += f * x.y; acc[2] += f * x.z; acc[3] += f * x.w;
        acc[4] += f * y.x; acc[5] += f * y.y; acc[6] += f * y.z; acc[7] += f * y.w;
      }
      const bool empty = L == 0.f;
      const float inv = empty ? 0.f : 1.f / L;
      const float lse = empty ? -INFINITY : (sub + log2f(L)) * kLn2f;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= inv;
      if (odd) {
        const int lim = ctx + r / g;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int col = 8 * c + e;
          const bool pos = bad[col] <= lim, neg = bad[D + col] <= lim;
          if (bad[2 * D + col] <= lim || (pos && neg)) acc[e] = __int_as_float(0x7fc00000);
          else if (pos) acc[e] += INFINITY;
          else if (neg) acc[e] -= INFINITY;
        }
      }
      if (whole) {
        const int64_t row = (static_cast<int64_t>(cur.row0) + r / g) * a.hq + cur.kvh * g + r % g;
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + row * D + 8 * c) =
            make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]), pack_bf16(acc[4], acc[5]),
                       pack_bf16(acc[6], acc[7]));
        if (c == 0 && a.lse) a.lse[row] = lse;
      } else {
        float4* dst = reinterpret_cast<float4*>(a.dec_o + (out0 + r) * D + 8 * c);
        dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (c == 0) a.dec_lse[out0 + r] = lse;
      }
    }
    if (!whole) {
      __syncthreads();
      if (threadIdx.x == 0) {
        __threadfence();   // the whole block's part, behind the barrier
        const bool last = atomicAdd(&a.done[c_lo], 1) == c_hi - c_lo;
        if (last) __threadfence();   // the other blocks' parts
        flag[1] = last;
      }
      __syncthreads();
      if (flag[1]) {
        // the last to arrive: all parts, in order, eight at a time (their
        // loads go out together; an online softmax over the groups of eight)
        const int parts = c_hi - c_lo + 1;
        for (int i = threadIdx.x; i < rows * C::CH; i += kWarps * 32) {
          const int r = i / C::CH, c = i % C::CH;
          float M = -INFINITY, L = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int p0 = 0; p0 < parts; p0 += kMergeAhead) {
            float ls[kMergeAhead];
            float4 x[kMergeAhead], y[kMergeAhead];
#pragma unroll
            for (int p = 0; p < kMergeAhead; ++p) {
              ls[p] = -INFINITY;
              if (p0 + p < parts) {
                const int64_t at = static_cast<int64_t>(slot_of(c_lo + p0 + p)) * 16 + r;
                const float4* src = reinterpret_cast<const float4*>(a.dec_o + at * D + 8 * c);
                ls[p] = __ldcg(a.dec_lse + at);
                x[p] = __ldcg(src);
                y[p] = __ldcg(src + 1);
              }
            }
            float m = M;
#pragma unroll
            for (int p = 0; p < kMergeAhead; ++p) m = fmaxf(m, ls[p]);
            const float sub = m == -INFINITY ? 0.f : m;
            const float old = expf(M - sub);
            M = m;
            L *= old;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] *= old;
#pragma unroll
            for (int p = 0; p < kMergeAhead; ++p) {
              const float f = expf(ls[p] - sub);
              L += f;
              if (p0 + p < parts) {   // (a weight of zero too: a non-finite V that the row sees is not lost)
                acc[0] += f * x[p].x; acc[1] += f * x[p].y; acc[2] += f * x[p].z; acc[3] += f * x[p].w;
                acc[4] += f * y[p].x; acc[5] += f * y[p].y; acc[6] += f * y[p].z; acc[7] += f * y[p].w;
              }
            }
          }
          const float inv = L == 0.f ? 0.f : 1.f / L;
          const int64_t row = (static_cast<int64_t>(cur.row0) + r / g) * a.hq + cur.kvh * g + r % g;
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + row * D + 8 * c) =
              make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv),
                         pack_bf16(acc[4] * inv, acc[5] * inv), pack_bf16(acc[6] * inv, acc[7] * inv));
          if (c == 0 && a.lse) a.lse[row] = L == 0.f ? -INFINITY : (M == -INFINITY ? 0.f : M) + logf(L);
        }
      }
    }
    __syncthreads();   // the merge memory, and the notes, are reused
    if (odd) {
      for (int i = threadIdx.x; i < 3 * D; i += kWarps * 32) bad[i] = INT32_MAX;
      if (threadIdx.x == 0) flag[0] = 0;
      __syncthreads();
    }
    if (it != steps - 1) {
      cur.step(a, max_kv);
      begin();
    }
  }
  // Every copy has been waited for; after a wait that ran out, once more.
  if (flag[2]) {
    int zero = 0;
    for (int it = max(0, issued - kStages); it < issued; ++it)
      mbar_wait(&full[it % kStages], (it / kStages) & 1, &zero, a.wait_limit_ns);
  }
}

template <int D, bool FOLD>
int launch(const AttendArgs& a, cudaStream_t s) {
  constexpr int smem = DecCfg<D>::SMEM;
  static_assert(smem <= 232448, "shared memory of one block");
  const int rc = allow_smem<attend_decode_kernel<D, FOLD>>(smem);
  if (rc != PA_OK) return rc;
  // (an empty cache has no page to read: every box is out of range, and the
  // maps are made over q only to have an address)
  const int64_t rows = a.n_slots > 0 ? a.n_slots : 1;
  const int box = a.page_size < kKT ? a.page_size : kKT;
  CUtensorMap mk, mv;
  if (!rows_map(&mk, a.n_slots > 0 ? a.k : a.q, rows, a.hkv, D, a.ldk, 1, box) ||
      !rows_map(&mv, a.n_slots > 0 ? a.v : a.q, rows, a.hkv, D, a.ldv, 1, box))
    return PA_ERR_CUDA;
  return launch_overlapped(attend_decode_kernel<D, FOLD>, dim3(a.decode_ctas), kWarps * 32, smem, s, mk, mv, a, box,
                           static_cast<int>(rows));
}

}  // namespace

int launch_attend_decode(const AttendArgs& a, cudaStream_t s) {
  // a warp has a quarter of a request's keys at most
  const bool fold = static_cast<int64_t>(a.max_pages) * a.page_size / kWarps > kFoldKeys;
  if (a.d == 128) return fold ? launch<128, true>(a, s) : launch<128, false>(a, s);
  return fold ? launch<64, true>(a, s) : launch<64, false>(a, s);
}

}  // namespace pa
