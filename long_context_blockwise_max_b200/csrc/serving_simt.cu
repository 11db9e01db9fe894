// Attention of packed rows or of rows over pages on the fp32 units: the path
// of fp32 inputs (every product and sum in fp32).
//
// Block = one piece: up to ROWS (token, query head) rows of one kv head
// against its key tiles, 64 keys at a time through shared memory (16-byte
// asynchronous copies, the next tile's under way during the current one), 256
// threads as 16 x 16: a thread has ROWS / 16 rows x 4 keys of the scores and
// the same rows x D / 16 columns of o.  Online softmax in log2 units, the
// running maximum and sum of a row kept by the 16 threads that share it.
// With 64 rows the fp32 FMAs and the shared-memory wavefronts that feed them
// (about 0.9 of a cycle per FMA cycle) are nearly even, and neither is hidden
// in full: one 2048-token prompt, 4 / 2 heads of 64, takes 84 us of the call's
// 89 (FMA pipe 52 %, LSU 64 % busy), one of 8192 tokens, 8 / 2 heads, 1.80 ms =
// 38 TFLOP/s.  Threads with 8 rows read less, but only half as many fit the
// registers: the same time.  With 16 rows (few new tokens) the reads bound it.
#include "serving.h"

namespace pa {

namespace {

constexpr int kKeys = 64;

template <int D, int ROWS>
struct SimtCfg {
  static constexpr int LDK = D + 4;              // 16 keys of a load fall on different banks
  static constexpr int LDP = kKeys + 4;
  static constexpr int STAGE = kKeys * (LDK + D);   // K, then V
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = OFF_Q + ROWS * D;
  static constexpr int OFF_P = OFF_KV + 2 * STAGE;
  static constexpr int FLOATS = OFF_P + ROWS * LDP;
  static constexpr int SMEM = FLOATS * 4 + 2 * kKeys * 8;
};

// two fp32 FMAs in one instruction (half the issue slots)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
        "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}

__device__ __forceinline__ void copy16(float* dst, const float* src, bool valid) {
  const int n = valid ? 16 : 0;   // 0: fill the 16 bytes with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(n)
               : "memory");
}

template <int D, int ROWS>
__global__ void __launch_bounds__(256, 2) attend_simt_kernel(AttendArgs a) {
  using C = SimtCfg<D, ROWS>;
  constexpr int R = ROWS / 16, CV = D / 64;      // rows, float4 columns of a thread
  extern __shared__ __align__(16) float sm[];
  float* sq = sm + C::OFF_Q;
  float* sp = sm + C::OFF_P;
  int64_t* slot = reinterpret_cast<int64_t*>(sm + C::FLOATS);   // [2][keys] rows of a tile's keys, -1: none
  grid_dep_wait();
  grid_dep_launch();
  int at, kvh;
  if (blockIdx.x >= static_cast<unsigned>(a.head->n_pieces) * static_cast<unsigned>(a.hkv)) return;
  piece_at(a, blockIdx.x, &at, &kvh);
  const Piece pc = a.pieces[at];
  const int g = a.hq / a.hkv;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int n_rows = min(a.tile_tokens, pc.q_len - pc.tok0) * g;
  const float scale = static_cast<float>(kLog2e / sqrt(static_cast<double>(D)));
  const float* Q = static_cast<const float*>(a.q);
  const float* K = static_cast<const float*>(a.k) + kvh * D;
  const float* V = static_cast<const float*>(a.v) + kvh * D;
  const int64_t key_lo = static_cast<int64_t>(pc.kt0) * kPlanTile;
  const int64_t key_hi = min(static_cast<int64_t>(pc.kt1) * kPlanTile,
                             keys_seen(pc.kv_len, pc.q_len, min(pc.q_len, pc.tok0 + a.tile_tokens)));
  // rows of the tile that starts at key c0, by the first threads
  auto look_up = [&](int64_t c0, int s) {
    if (tid < kKeys) {
      const int64_t key = c0 + tid;
      slot[s * kKeys + tid] = key >= key_hi ? -1 : a.block_table ? key_slot(a, pc.b, key) : pc.row0 + key;
    }
  };
  auto fetch = [&](int s) {
    float* k = sm + C::OFF_KV + s * C::STAGE;
    float* v = k + kKeys * C::LDK;
#pragma unroll
    for (int e = tid; e < kKeys * (D / 4); e += 256) {
      const int key = e / (D / 4), m = (e % (D / 4)) * 4;
      const int64_t row = slot[s * kKeys + key];
      const bool valid = row >= 0;
      copy16(k + key * C::LDK + m, valid ? K + row * a.ldk + m : Q, valid);
      copy16(v + key * D + m, valid ? V + row * a.ldv + m : Q, valid);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  look_up(key_lo, 0);
  look_up(key_lo + kKeys, 1);
  for (int e = tid; e < ROWS * (D / 4); e += 256) {
    const int r = e / (D / 4), m = (e % (D / 4)) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < n_rows) {
      const int64_t row = static_cast<int64_t>(pc.row0) + pc.tok0 + r / g;
      x = *reinterpret_cast<const float4*>(Q + row * a.ldq + (kvh * g + r % g) * D + m);
    }
    *reinterpret_cast<float4*>(sq + r * D + m) = x;
  }
  __syncthreads();
  fetch(0);
  int64_t lim[R];                                // last visible key of each row
  float m_run[R], l_run[R];
  float2 acc[R][2 * CV];                         // columns 64 j + 4 tx .. + 3 of each row
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = ty * R + i;
    lim[i] = r < n_rows ? static_cast<int64_t>(pc.kv_len) - pc.q_len + pc.tok0 + r / g : -1;
    m_run[i] = -INFINITY;
    l_run[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 2 * CV; ++j) acc[i][j] = make_float2(0.f, 0.f);
  }
  const int64_t lim_first = static_cast<int64_t>(pc.kv_len) - pc.q_len + pc.tok0;
  int st = 0;
  for (int64_t c0 = key_lo; c0 < key_hi; c0 += kKeys, st ^= 1) {
    // the next tile into the other stage (its last reader passed the barrier
    // at the end of the round before)
    fetch(st ^ 1);
    asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    __syncthreads();
    look_up(c0 + 2 * kKeys, st);
    const float* sk = sm + C::OFF_KV + st * C::STAGE;
    const float* sv = sk + kKeys * C::LDK;
    // scores of rows ty * R + i and keys tx + 16 * j
    // (even and odd columns summed apart, two FMAs to an instruction)
    float2 s2[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int m = 0; m < D; m += 4) {
      float4 q4[R], k4[4];
#pragma unroll
      for (int i = 0; i < R; ++i) q4[i] = *reinterpret_cast<const float4*>(sq + (ty * R + i) * D + m);
#pragma unroll
      for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * C::LDK + m);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s2[i][j] = fma2(make_float2(q4[i].x, q4[i].y), make_float2(k4[j].x, k4[j].y), s2[i][j]);
          s2[i][j] = fma2(make_float2(q4[i].z, q4[i].w), make_float2(k4[j].z, k4[j].w), s2[i][j]);
        }
    }
    float s[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
    // (before the stores below: a tile that every row sees in full needs no mask)
    const bool whole = c0 + kKeys - 1 <= lim_first;
    float alpha[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float mt = m_run[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = whole || c0 + tx + 16 * j <= lim[i] ? s[i][j] * scale : -INFINITY;
        mt = fmaxf(mt, s[i][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float sub = mt == -INFINITY ? 0.f : mt;   // a row without a visible key so far
      alpha[i] = fast_exp2(m_run[i] - sub);
      m_run[i] = mt;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = fast_exp2(s[i][j] - sub);
        sum += p;
        sp[(ty * R + i) * C::LDP + tx + 16 * j] = p;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l_run[i] = l_run[i] * alpha[i] + sum;
    }
    __syncwarp();   // a row's 16 threads are in one warp
    // each tile is summed by itself and then added: over thousands of keys the
    // rounding of one long chain of sums would be several times larger
    float2 part[R][2 * CV];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 2 * CV; ++j) part[i][j] = make_float2(0.f, 0.f);
    bool plain = whole;
    if (!whole) {
      // Some row does not see some key: there a masked key must add nothing
      // even if its V is not finite.  With finite V its zero probability does.
      bool odd = false;
#pragma unroll 4
      for (int e = tid; e < kKeys * (D / 4); e += 256) {
        const float4 x = reinterpret_cast<const float4*>(sv)[e];
        odd |= !(fabsf(x.x) < INFINITY) || !(fabsf(x.y) < INFINITY) || !(fabsf(x.z) < INFINITY) ||
               !(fabsf(x.w) < INFINITY);
      }
      plain = !__syncthreads_or(odd);
    }
    if (plain) {
#pragma unroll 2
      for (int key = 0; key < kKeys; key += 4) {
        float p[R][4];
#pragma unroll
        for (int i = 0; i < R; ++i)
          *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(sp + (ty * R + i) * C::LDP + key);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < CV; ++j) {
            const float4 v4 = *reinterpret_cast<const float4*>(sv + (key + k) * D + 64 * j + 4 * tx);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const float2 pp = make_float2(p[i][k], p[i][k]);
              part[i][2 * j] = fma2(pp, make_float2(v4.x, v4.y), part[i][2 * j]);
              part[i][2 * j + 1] = fma2(pp, make_float2(v4.z, v4.w), part[i][2 * j + 1]);
            }
          }
      }
    } else {
      // its product is skipped
#pragma unroll 1
      for (int key = 0; key < kKeys; ++key) {
#pragma unroll
        for (int j = 0; j < CV; ++j) {
          const float4 v4 = *reinterpret_cast<const float4*>(sv + key * D + 64 * j + 4 * tx);
#pragma unroll
          for (int i = 0; i < R; ++i)
            if (c0 + key <= lim[i]) {
              const float p = sp[(ty * R + i) * C::LDP + key];
              const float2 pp = make_float2(p, p);
              part[i][2 * j] = fma2(pp, make_float2(v4.x, v4.y), part[i][2 * j]);
              part[i][2 * j + 1] = fma2(pp, make_float2(v4.z, v4.w), part[i][2 * j + 1]);
            }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 2 * CV; ++j) acc[i][j] = fma2(acc[i][j], make_float2(alpha[i], alpha[i]), part[i][j]);
    __syncthreads();   // the stage and its slots are refilled
  }
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = ty * R + i;
    if (r >= n_rows) continue;
    const bool empty = l_run[i] == 0.f;   // no visible key
    const float inv = empty ? 0.f : 1.f / l_run[i];
    const float lse = empty ? -INFINITY : (m_run[i] + log2f(l_run[i])) * kLn2f;
    const int64_t part = (static_cast<int64_t>(pc.part) * a.hkv + kvh) * a.tile_rows + r;
    const int64_t row = (static_cast<int64_t>(pc.row0) + pc.tok0 + r / g) * a.hq + kvh * g + r % g;
    float* dst = pc.part >= 0 ? a.part_o + part * D : static_cast<float*>(a.o) + row * D;
#pragma unroll
    for (int j = 0; j < CV; ++j)
      *reinterpret_cast<float4*>(dst + 64 * j + 4 * tx) =
          make_float4(acc[i][2 * j].x * inv, acc[i][2 * j].y * inv, acc[i][2 * j + 1].x * inv,
                      acc[i][2 * j + 1].y * inv);
    if (tx == 0) {
      if (pc.part >= 0) a.part_lse[part] = lse;
      else if (a.lse) a.lse[row] = lse;
    }
  }
}

template <int D, int ROWS>
int launch(const AttendArgs& a, cudaStream_t s) {
  constexpr int smem = SimtCfg<D, ROWS>::SMEM;
  const int rc = allow_smem<attend_simt_kernel<D, ROWS>>(smem);
  if (rc != PA_OK) return rc;
  return launch_overlapped(attend_simt_kernel<D, ROWS>, dim3(tile_blocks(a)), 256, smem, s, a);
}

}  // namespace

// by shared memory (228 KB per SM) and registers (128 a thread)
int simt_blocks_per_sm(const AttendArgs& a) {
  const int smem = a.tile_rows == 16 ? (a.d == 128 ? SimtCfg<128, 16>::SMEM : SimtCfg<64, 16>::SMEM)
                                     : (a.d == 128 ? SimtCfg<128, 64>::SMEM : SimtCfg<64, 64>::SMEM);
  const int n = 228 * 1024 / (smem + 1024);
  return n < 2 ? n : 2;
}

int launch_attend_simt(const AttendArgs& a, cudaStream_t s) {
  if (a.tile_rows == 16) return a.d == 128 ? launch<128, 16>(a, s) : launch<64, 16>(a, s);
  return a.d == 128 ? launch<128, 64>(a, s) : launch<64, 64>(a, s);
}

}  // namespace pa
