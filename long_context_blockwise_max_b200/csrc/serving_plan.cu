// Work plan of an attention call over requests of different lengths, and
// the merge of rows whose keys were cut into pieces.
//
// The lengths are on the device, so the plan is made there, by one block,
// in the call itself: a list of pieces for the tile kernels (one per group
// of rows, the deepest first, so that the short ones fill the end of the
// launch), or, when that ends sooner, the same rows with their keys cut into
// about equal pieces; and the ranges of the decode kernel's blocks.  The kernels
// behind it are launched for the most pieces the arguments allow (the tile kernel
// of bf16 for a block per SM at most), and blocks without one return at once.
#include <type_traits>

#include "serving.h"

namespace pa {

namespace {

constexpr int kBuckets = 256;
// Cutting keys is looked at while the rows give less than three waves of
// blocks (prompts: from there on no row group is deeper than a block's share of
// the work) or less than 16 (paged rows: one long cache among short ones would
// be alone at the end.  512 tokens over 128K keys beside 64 x 128 over 1K: 1960 us
// whole, 1076 us cut; looking in vain costs 3 us).
constexpr int kPromptWaves = 3, kPagedWaves = 16;
// From three waves on, a cut has to promise a tenth: what it costs there is
// underrated.  512 tokens over 8K / 32K / 128K keys beside m x 128 over 1K, whole / cut, and
// the promise: m = 40 193 / 213 (5 %), 538 / 424 (30 %), 1967 / 1212 us (74 %);
// m = 64 237 / 272 (1 %), 537 / 476 (15 %), 1970 / 1262 (72 %); m = 140 439 / 457 (0),
// 638 / 720 (3 %), 2042 / 1537 (52 %).  (Beyond 16 waves it is not looked at: m = 200
// 642 / 647, 1031 / 898, 2462 / 1749.)
constexpr float kCutMargin = 0.9f;
constexpr int kCuts = 32;
constexpr int kMaxCut = 64;
constexpr int kMaxCutItems = 1024;
// key tiles of 2.1 us per block.  32 requests, four of them tokens behind up to
// 27 keys: 108 us with the decode kernel at work, 97 us without.  (The border lies
// low: beside five chunks of 256 over 8000 keys, 4 tokens over 1000, 2.8 tiles, take
// 285 / 265 us with and without, and 8 of them, 5.6 tiles, still 294 / 264.)
constexpr int kFewTiles = 3;
// ... and, where the chunks' pieces fit one wave of blocks, as long as blocks stay
// for the parts that their keys are cut into: this many key tiles per block at most
// may move from the few tokens' blocks to the others.  Chunks of 256 over 8000 keys,
// 32 / 8 heads, with tokens over 64 keys, decode kernel / tiles: one chunk with 2 or 8
// tokens (moves 2, 10) 65 / 61, 67 / 87 us; two with 2 or 8 (3, 21) 109 / 101, 110 / 113;
// three with 2 or 4 (5, 11) 148 / 145, 149 / 145; four with 2 or 4 (7, 15) 161 / 157,
// 159 / 190 us.
constexpr int kFewMoved = 9;
// K and V of this many bytes stay in L2 (126 MB) beside q and o, and pieces are taken
// over all heads in order of depth (24 prompts of 1 to 4096 tokens: 162 us, by heads
// 175).  Beyond, a head's pieces share its keys in L2 (8 x 4096 tokens, 134 MB: 1168 us by
// heads, 1247 over all of them; at 50 to 100 MB both within 2 %), unless they are so
// uneven that the last head's deepest piece would end alone: with at most two waves
// per head, and the deepest at least kUneven times the average.  32 mixed requests
// over up to 8K keys (128 MB) 97 us over all heads, 111 by heads; 2048 tokens each over
// 64K / 1 .. 64K / 4 keys 4.15 to 4.26 / 4.34 to 4.37 ms; but 8 x 2048 over 32K 9.0 to 9.3 /
// 8.14 ms, 4 x 2048 over 32K 4.23 to 4.30 / 4.03, and 16384 over 32K 6.2 / 6.1.
constexpr double kL2Keys = 100e6;
constexpr float kUneven = 1.5f;

struct Lens {
  int64_t row0, q, kv;
  int rows;      // packed (token, head) rows per kv head
};

__device__ __forceinline__ Lens lens_of(const AttendArgs& a, int b, int64_t max_kv, bool record) {
  Lens r;
  const int64_t lo = a.cu_q[b], hi = a.cu_q[b + 1];
  r.row0 = lo;
  r.q = hi - lo;
  r.kv = a.kv_len ? a.kv_len[b] : r.q;
  const bool bad = lo < 0 || hi < lo || hi > a.N || r.kv < 0 || r.kv > max_kv || (a.kv_len && r.q > a.max_q);
  if (bad) {
    if (record) set_status(a.status, PA_ERR_INVALID, b);
    r.q = 0;
    r.kv = 0;
  }
  const int64_t rows = r.q * (a.hq / a.hkv);
  r.rows = static_cast<int>(rows < INT32_MAX ? rows : INT32_MAX);
  return r;
}

__device__ __forceinline__ int depth_of(const Lens& r, int tok0, int tokens) {
  const int64_t end = min(r.q, static_cast<int64_t>(tok0) + tokens);
  return static_cast<int>((keys_seen(r.kv, r.q, end) + kPlanTile - 1) / kPlanTile);
}

__device__ __forceinline__ void put_piece(const AttendArgs& a, int at, int b, const Lens& r, int tok0, int kt0,
                                          int kt1, int part) {
  int4* dst = reinterpret_cast<int4*>(a.pieces + at);
  dst[0] = make_int4(b, tok0, kt0, kt1);
  dst[1] = make_int4(part, static_cast<int>(r.row0), static_cast<int>(r.q), static_cast<int>(r.kv));
}

// One block.  Latency-bound (loads of the lengths, one scan, bisections in
// shared memory): its time is on the critical path of every call, 2 to 3 us for
// generated tokens, 5 to 9 with cuts to weigh.
__global__ void __launch_bounds__(1024) attend_plan_kernel(AttendArgs a, int64_t max_kv) {
  grid_dep_wait();     // the lengths, and the workspace's last use
  grid_dep_launch();
  extern __shared__ __align__(16) uint8_t raw[];
  int64_t* units = reinterpret_cast<int64_t*>(raw);               // [B + 1] decode key groups before request b
  int32_t* items = reinterpret_cast<int32_t*>(units + a.B + 1);   // [B + 1] row groups before request b
  __shared__ int64_t tmp[2][64];
  __shared__ int hist[kBuckets];
  __shared__ int depth[kMaxCutItems], part_of[kMaxCutItems], first_piece[kMaxCutItems + 1];
  __shared__ int deepest, n_merge;
  // deepest chunk, deepest request of few rows, key tiles of those; pieces of the
  // chunks, their key tiles, requests of few rows
  __shared__ int few[6];
  __shared__ unsigned key_tiles;
  __shared__ unsigned long long piece_tiles;   // of all pieces, about
  __shared__ int cost_pieces[kCuts], cost_cuts[kCuts], cost_load[kCuts], best;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  if (tid < static_cast<int>(kStatusBytes / 4)) reinterpret_cast<int32_t*>(a.status)[tid] = 0;
  for (int c = tid; c < a.decode_ctas; c += threads) a.done[c] = 0;
  if (tid < kBuckets) hist[tid] = 0;
  if (tid == 0) {
    units[0] = 0;
    items[0] = 0;
    deepest = 0;
    n_merge = 0;
    key_tiles = 0;
    piece_tiles = 0;
  }
  if (tid < kCuts) cost_pieces[tid] = cost_cuts[tid] = cost_load[tid] = 0;
  if (tid < 6) few[tid] = 0;
  __syncthreads();
  // Few generated tokens with short caches beside chunks: the decode kernel
  // takes 8 us whatever it has to do, and 2 us for nothing.  They are the tile
  // kernel's when its blocks need less for them (kFewTiles key tiles each), no
  // cache is longer than the chunks' longest, and they take no blocks that the
  // chunks' keys need (kFewMoved).  (Sums are kept below 2^30 by clamps that only
  // calls of many waves reach.)
  int small_rows = a.small_rows;
  if (a.tiles && small_rows > 0) {
    constexpr int kMost = 1 << 20;
    int cost = 0, deep_small = 0, deep = 0, pieces = 0, tiles = 0, tokens = 0;
    for (int b = tid; b < a.B; b += threads) {
      const Lens r = lens_of(a, b, max_kv, false);
      if (r.q <= 0) continue;
      const int d = static_cast<int>((r.kv + kPlanTile - 1) / kPlanTile);
      if (r.rows > small_rows) {
        const int64_t n = (static_cast<uint32_t>(r.q) + a.tile_tokens - 1) / static_cast<uint32_t>(a.tile_tokens);
        deep = max(deep, d);
        pieces = static_cast<int>(min(pieces + n, static_cast<int64_t>(kMost)));
        tiles = static_cast<int>(min(tiles + n * d, static_cast<int64_t>(kMost)));
      } else {
        deep_small = max(deep_small, d);
        cost = min(cost + d + static_cast<int>(a.piece_cost), kMost);
        ++tokens;
      }
    }
    deep = __reduce_max_sync(0xffffffffu, deep);
    deep_small = __reduce_max_sync(0xffffffffu, deep_small);
    cost = __reduce_add_sync(0xffffffffu, cost);
    pieces = __reduce_add_sync(0xffffffffu, pieces);
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    if (lane == 0) {
      atomicMax(&few[0], deep);
      atomicMax(&few[1], deep_small);
      atomicAdd(&few[2], min(cost, kMost));
      atomicAdd(&few[3], min(pieces, kMost));
      atomicAdd(&few[4], min(tiles, kMost));
      atomicAdd(&few[5], tokens);
    }
    __syncthreads();
    if (few[1] <= few[0] && static_cast<int64_t>(few[2]) * a.hkv <= kFewTiles * a.slots) {
      const int64_t h = a.hkv, blocks = few[3] * h, taken = few[5] * h, left = a.slots - taken;
      if (blocks > a.slots || (left > 0 && few[4] * h * taken <= kFewMoved * a.slots * left)) small_rows = 0;
    }
  }
  int64_t item_base = 0, unit_base = 0;
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int b = b0 + tid;
    int64_t ni = 0, nu = 0;
    int depth_b = 0;
    unsigned tiles_b = 0;
    if (b < a.B) {
      const Lens r = lens_of(a, b, max_kv, true);
      if (r.q > 0) {
        if (r.rows <= small_rows) {
          const int64_t groups = (r.kv + kPlanTile - 1) / kPlanTile;
          nu = (groups > 0 ? groups : 1) * a.hkv;
        } else {
          ni = (static_cast<uint32_t>(r.q) + a.tile_tokens - 1) / static_cast<uint32_t>(a.tile_tokens);
          depth_b = static_cast<int>((r.kv + kPlanTile - 1) / kPlanTile);
          // (its average piece sees the keys before half of its tokens)
          const int64_t t = ni * (keys_seen(r.kv, r.q, r.q / 2) + kPlanTile - 1) / kPlanTile;
          tiles_b = static_cast<unsigned>(min(t, static_cast<int64_t>(1 << 26)));
        }
      }
    }
    depth_b = max(depth_b, 0);
    const int warp_deepest = __reduce_max_sync(0xffffffffu, depth_b);
    const unsigned warp_tiles = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(depth_b));
    const unsigned warp_piece_tiles = __reduce_add_sync(0xffffffffu, tiles_b);
    if (lane == 0 && warp_deepest > 0) {
      atomicMax(&deepest, warp_deepest);
      atomicAdd(&key_tiles, warp_tiles);
      atomicAdd(&piece_tiles, static_cast<unsigned long long>(warp_piece_tiles));
    }
    int64_t i_all, u_all;
    block_incl_scan2<int64_t>(ni, nu, tmp[(b0 / threads) & 1], &i_all, &u_all);
    if (b < a.B) {
      const int64_t x = item_base + ni;
      items[b + 1] = static_cast<int32_t>(x < INT32_MAX ? x : INT32_MAX);
      units[b + 1] = unit_base + nu;
    }
    item_base += i_all;
    unit_base += u_all;
  }
  __syncthreads();
  // ---- decode: equal ranges of key groups, one per block ----------------
  if (a.decode_ctas > 0) {
    const int64_t each = unit_base / a.decode_ctas, more = unit_base % a.decode_ctas;
    for (int c = tid; c < a.decode_ctas; c += threads) {
      const int64_t u0 = c * each + (c < more ? c : more);
      int4 x = make_int4(0, 0, 0, 1), y = make_int4(0, 0, 0, static_cast<int>(each + (c < more)));
      if (u0 < unit_base) {
        const int b = upper_index(units, a.B + 1, u0);
        const Lens r = lens_of(a, b, max_kv, false);
        const int groups = static_cast<int>((units[b + 1] - units[b]) / a.hkv);
        const int64_t rem = u0 - units[b];
        x = make_int4(b, static_cast<int>(rem / groups), static_cast<int>(rem % groups), groups);
        y.x = static_cast<int>(r.kv);
        y.y = static_cast<int>(r.q);
        y.z = static_cast<int>(r.row0);
      }
      int4* dst = reinterpret_cast<int4*>(a.starts + c);
      dst[0] = x;
      dst[1] = y;
      *reinterpret_cast<longlong2*>(dst + 2) = make_longlong2(u0, each);
      dst[3] = make_int4(static_cast<int>(more), 0, 0, 0);
    }
  }
  // ---- tiles --------------------------------------------------------------
  int n_pieces = 0;
  if (a.tiles) {
    // (offsets that fall and rise again count rows twice: what is above the
    // most that N rows can make is dropped, and cutting adds at most part_cap)
    const int64_t most = a.piece_cap - a.part_cap;
    const int n = static_cast<int>(item_base < most ? item_base : most);
    if (item_base > most && tid == 0) set_status(a.status, PA_ERR_INVALID, a.B);
    const int64_t blocks = static_cast<int64_t>(n) * a.hkv;
    bool cut = a.part_cap > 0 && n > 0 && n <= kMaxCutItems && deepest > 1;
    int parts = 1;
    if (cut) {
      for (int i = tid; i < n; i += threads) {
        const int b = upper_index(items, a.B + 1, i);
        depth[i] = depth_of(lens_of(a, b, max_kv, false), (i - items[b]) * a.tile_tokens, a.tile_tokens);
      }
      __syncthreads();
      // the number of cuts of the deepest rows that ends first: blocks run in
      // waves of one per slot, or, past one wave, fill the slots evenly with
      // half a piece of slack (less with many waves: the shortest are last); a
      // cut adds the merge of its partial results.
      // One lane per number, the rows spread over the warps.
      const int cuts = lane < 20 ? lane + 1 : min(kMaxCut, 20 + (lane - 19) * 4);   // 1 .. 20, then every fourth
      const int c = (deepest + cuts - 1) / cuts;
      int np = 0, nc = 0, load = 0;
      const float inv = 1.f / c;
      for (int i = warp; i < n; i += threads / 32) {
        const int d = depth[i], x = d + c - 1;
        int p = static_cast<int>(x * inv);   // x / c, put right by at most one
        p += (p + 1) * c <= x;
        p -= p * c > x;
        p = max(p, 1);
        np += p;
        nc += p > 1 ? p : 0;
        load += d;
      }
      atomicAdd(&cost_pieces[lane], np);
      atomicAdd(&cost_cuts[lane], nc);
      atomicAdd(&cost_load[lane], load);
      __syncthreads();
      if (warp == 0) {
        const float piece = a.piece_cost + c;   // the longest piece
        float cost = piece;
        if (static_cast<int64_t>(cost_pieces[lane]) * a.hkv > a.slots)
          cost = fmaxf(cost, (cost_load[lane] + a.piece_cost * cost_pieces[lane]) * a.hkv / a.slots +
                                 0.5f * piece * fminf(1.f, 3.f * a.slots / blocks));
        if (cuts > 1) cost += a.merge_cost * (1.f + cuts / 24.f);
        else if (blocks >= static_cast<int64_t>(kPromptWaves) * a.slots) cost *= kCutMargin;
        if (cost_cuts[lane] > a.part_cap || cuts > deepest) cost = INFINITY;
        const unsigned least = __reduce_min_sync(0xffffffffu, __float_as_uint(cost));
        const unsigned who = __ballot_sync(0xffffffffu, __float_as_uint(cost) == least);
        if (lane == __ffs(who) - 1) best = cuts;
      }
      __syncthreads();
      parts = best;
      cut = parts > 1;
    }
    if (cut) {
      // pieces and partial results by prefix sums over the rows, then one
      // thread per piece
      const int chunk = (deepest + parts - 1) / parts;
      int n_parts = 0;
      for (int i0 = 0; i0 < n; i0 += threads) {
        const int i = i0 + tid;
        int64_t p = 0;
        if (i < n) p = depth[i] > chunk ? (depth[i] + chunk - 1) / chunk : 1;
        int64_t at = p, slot = p > 1 ? p : 0, all, slots;
        __syncthreads();
        block_incl_scan2<int64_t>(at, slot, tmp[0], &all, &slots);
        if (i < n) {
          first_piece[i + 1] = n_pieces + static_cast<int>(at);
          if (p > 1) {
            const int first = n_parts + static_cast<int>(slot - p);
            part_of[i] = first;
            const int b = upper_index(items, a.B + 1, i);
            const Lens r = lens_of(a, b, max_kv, false);
            const int tok0 = (i - items[b]) * a.tile_tokens;
            a.items[atomicAdd(&n_merge, 1)] = {
                static_cast<int32_t>(r.row0) + tok0,
                static_cast<int32_t>(min(static_cast<int64_t>(a.tile_tokens), r.q - tok0)), first,
                static_cast<int32_t>(p)};
          } else {
            part_of[i] = -1;
          }
        }
        n_pieces += static_cast<int>(all);
        n_parts += static_cast<int>(slots);
      }
      if (tid == 0) first_piece[0] = 0;
      __syncthreads();
      // the longest first, by a counting sort (no piece is longer than `chunk`)
      const bool sort = static_cast<int64_t>(n_pieces) * a.hkv > a.slots;
      auto bucket = [&](int d) {
        return kBuckets - 1 - static_cast<int>(static_cast<int64_t>(d) * (kBuckets - 1) / chunk);
      };
      auto piece_len = [&](int x, int& i, int& kt0) {
        i = upper_index(first_piece, n + 1, x);
        const int p = first_piece[i + 1] - first_piece[i], k = x - first_piece[i];
        const int lo = depth[i] / p, more = depth[i] % p;   // the first `more` pieces have a tile more
        kt0 = k * lo + min(k, more);
        return lo + (k < more);
      };
      if (sort) {
        for (int x = tid; x < n_pieces; x += threads) {
          int i, kt0;
          atomicAdd(&hist[bucket(piece_len(x, i, kt0))], 1);
        }
        __syncthreads();
        const int64_t h = tid < kBuckets ? hist[tid] : 0;
        int64_t at = h, none = 0, all, none_all;
        block_incl_scan2<int64_t>(at, none, tmp[1], &all, &none_all);
        if (tid < kBuckets) hist[tid] = static_cast<int>(at - h);
        __syncthreads();
      }
      for (int x = tid; x < n_pieces; x += threads) {
        int i, kt0;
        const int len = piece_len(x, i, kt0);
        const int b = upper_index(items, a.B + 1, i);
        put_piece(a, sort ? atomicAdd(&hist[bucket(len)], 1) : x, b, lens_of(a, b, max_kv, false),
                  (i - items[b]) * a.tile_tokens, kt0, kt0 + len,
                  part_of[i] < 0 ? -1 : part_of[i] + x - first_piece[i]);
      }
    } else {
      // deepest first: a counting sort by depth (the order inside a bucket is
      // free; it changes no result).  One wave needs no order.
      const bool sort = blocks > a.slots;
      auto bucket = [&](int d) {
        return deepest > 0 ? kBuckets - 1 - static_cast<int>(static_cast<int64_t>(d) * (kBuckets - 1) / deepest) : 0;
      };
      if (sort) {
        for (int i = tid; i < n; i += threads) {
          const int b = upper_index(items, a.B + 1, i);
          atomicAdd(&hist[bucket(depth_of(lens_of(a, b, max_kv, false), (i - items[b]) * a.tile_tokens,
                                          a.tile_tokens))], 1);
        }
        __syncthreads();
        const int64_t h = tid < kBuckets ? hist[tid] : 0;
        int64_t at = h, none = 0, all, none_all;
        block_incl_scan2<int64_t>(at, none, tmp[0], &all, &none_all);
        if (tid < kBuckets) hist[tid] = static_cast<int>(at - h);
        __syncthreads();
      }
      for (int i = tid; i < n; i += threads) {
        const int b = upper_index(items, a.B + 1, i);
        const Lens r = lens_of(a, b, max_kv, false);
        const int tok0 = (i - items[b]) * a.tile_tokens;
        const int d = depth_of(r, tok0, a.tile_tokens);
        put_piece(a, sort ? atomicAdd(&hist[bucket(d)], 1) : i, b, r, tok0, 0, d, -1);
      }
      n_pieces = n;
    }
    __syncthreads();
  }
  if (tid == 0) {
    a.head->n_pieces = n_pieces;
    a.head->n_items = n_merge;
    a.head->abort = 0;
    a.head->next = 0;
    const double kv_bytes = static_cast<double>(key_tiles) * kPlanTile * a.hkv * a.d * (a.dtype == PA_BF16 ? 4 : 8);
    const bool uneven = static_cast<float>(deepest) * item_base >= kUneven * static_cast<float>(piece_tiles);
    a.head->heads_inner = kv_bytes <= kL2Keys || (n_pieces <= 2 * a.slots && uneven);
  }
}

// Rows cut into pieces: lse = ln sum_p exp(lse_p), o = sum_p exp(lse_p - lse) o_p,
// in piece order.  One warp per row, the rows of all items in one sequence.
// Bound by the latency of its loads: the parts' lse are loaded together, and
// eight of their rows at a time, the first eight without waiting for the
// weights; the grid is one wave (a second one's start costs more than its work).
// A 64-token query of 32 heads in 18 pieces (19 MB): 6 to 9 us.
template <typename OT, int D>
__global__ void __launch_bounds__(256, 4) attend_merge_kernel(AttendArgs a) {
  constexpr int VPL = D / 32, U = 8;   // elements of a lane, parts in flight (a divisor of 32)
  using Vec = std::conditional_t<VPL == 4, float4, float2>;
  grid_dep_wait();
  const int g = a.hq / a.hkv, lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(a.hkv) * a.tile_rows;   // rows from one partial result to the next
  const int64_t total = a.head->n_items * step;
  for (int64_t x = blockIdx.x * 8 + (threadIdx.x >> 5); x < total; x += static_cast<int64_t>(gridDim.x) * 8) {
    const int r = static_cast<int>(x % a.tile_rows);
    const int64_t y = x / a.tile_rows;
    const int kvh = static_cast<int>(y % a.hkv);
    const MergeItem it = a.items[y / a.hkv];
    if (r >= it.n_tok * g) continue;
    const int64_t base = (static_cast<int64_t>(it.part0) * a.hkv + kvh) * a.tile_rows + r;
    const float* ls = a.part_lse + base;
    const Vec* src = reinterpret_cast<const Vec*>(a.part_o + base * D) + lane;
    float m = -INFINITY;
#pragma unroll 1
    for (int p = lane; p < it.n_parts; p += 32) m = fmaxf(m, ls[p * step]);
    float v[U][VPL];
    auto load = [&](int k, int p) {
      const Vec x = src[p * step * (D / VPL)];
      v[k][0] = x.x;
      v[k][1] = x.y;
      if constexpr (VPL == 4) {
        v[k][2] = x.z;
        v[k][3] = x.w;
      }
    };
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (k < it.n_parts) load(k, k);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float sub = m == -INFINITY ? 0.f : m;   // a NaN stays one
    float z = 0.f, w = 0.f, acc[VPL] = {};
#pragma unroll 1
    for (int p = 0; p < it.n_parts; p += U) {
      if ((p & 31) == 0) {
        w = p + lane < it.n_parts ? expf(ls[(p + lane) * step] - sub) : 0.f;
        z += w;
      }
      if (p > 0) {
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (p + k < it.n_parts) load(k, p + k);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        // (a weight of zero is multiplied too: a non-finite V that the row sees
        // leaves its column non-finite however little its key weighs)
        const float wk = __shfl_sync(0xffffffffu, w, (p + k) & 31);
        if (p + k < it.n_parts) {
#pragma unroll
          for (int i = 0; i < VPL; ++i) acc[i] += wk * v[k][i];
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float inv = z == 0.f ? 0.f : 1.f / z;
    const int64_t row = static_cast<int64_t>(it.row0) + r / g;
    const int head = kvh * g + r % g;
    OT* dst = static_cast<OT*>(a.o) + (row * a.hq + head) * D + lane * VPL;
#pragma unroll
    for (int e = 0; e < VPL; ++e) dst[e] = from_f32<OT>(acc[e] * inv);
    if (lane == 0 && a.lse) a.lse[row * a.hq + head] = z == 0.f ? -INFINITY : sub + logf(z);
  }
}

template <typename OT>
int merge(const AttendArgs& a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.item_cap) * a.hkv * a.tile_rows;
  const int64_t want = (rows + 7) / 8;
  const dim3 grid(static_cast<unsigned>(want < 4 * kSms ? want : 4 * kSms));
  return launch_overlapped(a.d == 128 ? attend_merge_kernel<OT, 128> : attend_merge_kernel<OT, 64>, grid, 256, 0, s, a);
}

}  // namespace

// few requests and rows: the fewer warps at its barriers, the sooner it ends
static int plan_threads(const AttendArgs& a) { return a.B <= 256 && a.piece_cap <= 1024 ? 256 : 1024; }

size_t plan_attend(AttendArgs& a, int64_t max_kv, void* ws) {
  const int g = a.hq / a.hkv;
  if (a.dtype == PA_BF16) {
    a.tile_rows = 256;                // two tiles of 128 rows
    a.tile_tokens = 2 * (128 / g);
    a.slots = kSms;
    // in key tiles of 2.1 us: a piece's set-up and output, the merge's launch
    a.piece_cost = 5.f;
    a.merge_cost = 3.f;
  } else {
    // fp32 rows per block: 16 when no request has more, 64 otherwise
    a.tile_rows = a.max_q > 0 && static_cast<int64_t>(a.max_q) * g <= 16 ? 16 : 64;
    a.tile_tokens = a.tile_rows / g;
    a.slots = simt_blocks_per_sm(a) * kSms;
    // in key tiles of about 10 us with 64 rows, 3 us with 16
    a.piece_cost = a.tile_rows == 16 ? 1.f : 0.3f;
    a.merge_cost = a.tile_rows == 16 ? 2.f : 0.6f;
  }
  // Rows per kv head up to which a request is the decode kernel's, in calls
  // that may have such a request: a token has no more rows than that, and either
  // every request is that short or N < B * max_q says that some has fewer than
  // max_q tokens.  (N counts padding rows too: a batch padded to B * max_q rows is
  // the tile kernel's as a whole.)
  a.small_rows = 0;
  if (a.dtype == PA_BF16 && a.max_q > 0 && g <= kDecodeRows &&
      (static_cast<int64_t>(a.max_q) * g <= kDecodeRows || a.N < static_cast<int64_t>(a.B) * a.max_q))
    a.small_rows = kDecodeRows;
  a.decode_ctas = a.small_rows > 0 ? kSms : 0;
  a.tiles = a.small_rows == 0 || static_cast<int64_t>(a.max_q) * g > a.small_rows;
  const int64_t full = a.tiles ? a.N / a.tile_tokens : 0;
  const int64_t groups = a.tiles ? full + (a.B < a.N ? a.B : a.N) : 0;   // sum over requests of ceil(q / tile_tokens)
  const int64_t deep = (max_kv + kPlanTile - 1) / kPlanTile;
  a.part_cap = 0;
  a.item_cap = 0;
  const int64_t cuts = 2 * a.slots / a.hkv;   // partial results per kv head: two waves of blocks
  if (a.tiles && full * a.hkv < (a.max_q > 0 ? kPagedWaves : kPromptWaves) * a.slots && cuts >= 2 && deep > 1) {
    const int64_t most = groups * deep;
    a.part_cap = static_cast<int>(most < cuts ? most : cuts);
    a.item_cap = static_cast<int>(groups < a.part_cap ? groups : a.part_cap);   // rows that are cut
  }
  a.piece_cap = static_cast<int>(groups + a.part_cap);
  char* w = static_cast<char*>(ws);
  size_t off = 0;
  auto take = [&](auto*& p, size_t count) {
    using T = std::remove_reference_t<decltype(*p)>;
    if (w != nullptr) p = reinterpret_cast<T*>(w + off);
    off += align_up(sizeof(T) * count);
  };
  take(a.status, 1);
  take(a.head, 1);
  take(a.pieces, a.piece_cap);
  take(a.items, a.item_cap);
  take(a.starts, a.decode_ctas);
  take(a.done, a.decode_ctas);
  const size_t parts = static_cast<size_t>(a.part_cap) * a.hkv * a.tile_rows;
  take(a.part_lse, parts);
  take(a.part_o, parts * a.d);
  const bool folds = a.tiles && a.dtype == PA_BF16 && deep > kFoldTiles;
  if (folds) take(a.fold, static_cast<size_t>(a.slots) * 2 * a.tile_rows * (a.d + 4));
  take(a.dec_lse, static_cast<size_t>(a.decode_ctas) * 2 * 16);
  take(a.dec_o, static_cast<size_t>(a.decode_ctas) * 2 * 16 * a.d);
  return off;
}

int launch_attend(const AttendArgs& a, cudaStream_t s) {
  const int64_t max_kv = a.block_table ? static_cast<int64_t>(a.max_pages) * a.page_size : a.N;
  const size_t smem = (sizeof(int64_t) + sizeof(int32_t)) * (static_cast<size_t>(a.B) + 1);
  if (smem > 32 * 1024) {   // beside 14 KB of static arrays
    const int rc = allow_smem<attend_plan_kernel>(12 * (kMaxRequests + 1));
    if (rc != PA_OK) return rc;
  }
  int rc = launch_overlapped(attend_plan_kernel, dim3(1), plan_threads(a), smem, s, a, max_kv);
  if (rc != PA_OK) return rc;
  profile_begin(s);
  if (a.decode_ctas > 0) rc = launch_attend_decode(a, s);
  if (rc == PA_OK && a.tiles) rc = a.dtype == PA_BF16 ? launch_attend_tc(a, s) : launch_attend_simt(a, s);
  profile_end(s);
  if (rc == PA_OK && a.part_cap > 0) rc = a.dtype == PA_F32 ? merge<float>(a, s) : merge<__nv_bfloat16>(a, s);
  return rc;
}

}  // namespace pa
