// few.cu -- a whole mixture-of-experts layer for a few tokens in one kernel:
//
//   y[t] = sum_j weight[t, j] * (silu(g) * u) @ W2[e],   [g | u] = x[t] @ W1[e],
//   e = expert_ids[t, j]
//
// Decoding reads every weight of the chosen experts once and multiplies it
// with one to a few dozen rows, so the bound is the stream of the weights from
// HBM and everything else must hide behind it.
//
// Split.  The weights of the active experts are cut into units of 128 columns
// x 128 bytes of contraction (16 KB).  As many column tiles as fill whole waves
// of CTAs go one to a CTA; the contraction of the tiles left over is cut into
// slices (at most 16) so that every SM streams nearly the same number of
// bytes whatever the routing.  CTAs that run side by side read neighbouring
// tiles at the same depth, which for [G, K, N] weights is neighbouring memory
// (a copy-only version of this stream ran 41 us for 235 MB in this order and
// 55 us with contiguous unit ranges per CTA).  A sliced tile gets one fp32
// partial sum per slice, added in slice order, so the result does not depend
// on timing.
//
// Tile.  The weights are the 128-row operand of tcgen05.mma and stay in the
// layout they have in memory (MN-major for [G, K, N], K-major for [G, N, K]):
// TMA brings them to shared memory and no register ever holds one.  The
// expert's rows are the MMA's columns.
//
// Activations stay bf16 in precision although the MMA multiplies E4M3: a bf16
// value has 8 significant bits, so scaled by a power of two (one per row, that
// puts the row's largest magnitude into [128, 256)) it is hi + lo / 16 with two
// E4M3 values of 4 significant bits each, exactly for values down to 2^-13 of
// the row's largest and within 2^-21 of that largest below.  hi and lo are
// separate MMA columns, joined and unscaled once per tile.  (A scale per block
// of 128 instead would need every block's accumulator read and scaled on its
// own: that epilogue took 500 to 1000 cycles a unit and was the bound.)  bf16
// weights multiply the bf16 rows as they are.
//
// The layer is one cooperative launch: gate|up product, grid barrier, SwiGLU
// of the summed partials (rounded to bf16, as the separate calls round it),
// grid barrier, down product, grid barrier, weighted sum.  The producer starts
// the down product's first copies before the barriers, so HBM keeps working
// across them.  Measured (us): one token, two of 8 experts, K = 4096, F = 14336
// E4M3: 70 to 74, of which 53.7 is the weights at the copy rate; 16 tokens, 8 of
// 256 experts each, K = 7168, F = 2048: 645 to 705 from box to box (684 for the
// expected experts at the copy rate); the smallest layers 16 (set-up 2.4, a
// barrier 1.2, two chains of load, multiply and sum).
//
// Warps (512 threads, one CTA per SM): 0-1 TMA producers, 2-3 MMA issuers (2
// owns the TMEM), 4-11 activation loaders, 12-15 epilogue (TMEM lanes 32 (w %
// 4) ..).  Producers and issuers take alternate units: one thread's wait and
// issue per unit bounds the stream below HBM (copies alone, 235 MB: 57 and 51
// us with one producer, 41 with two; a third gains nothing here).  Each issuer
// sums its units of a tile in an accumulator of its own; the epilogue adds the
// two.  A loader warp prepares every eighth unit on its own, so that eight
// units' loads are in flight: under the weight stream one takes 1000 to 2000
// cycles, a unit's share of HBM 670.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "few.h"
#include "internal.h"
#include "ptx.cuh"

namespace gmm {
namespace {

constexpr int kFewThreads = 512;
constexpr int kFewMaxSlices = 16;
// The tokens' largest magnitudes: every CTA finds all of them on its own, 15
// warps taking pieces of 1024 values, or each row is one warp's of the grid and
// the results are shared through memory and one more barrier.  On its own a warp
// reads T pieces / 15 and shared it reads one row's pieces; sharing costs the
// barrier, about two pieces: shared where (T - 15) pieces > 30.  Measured, own
// against shared (us): K = 7168 (7 pieces), F = 2048, two of 32 experts, 2 tokens
// 37.2 / 39.6, 8 102.4 / 103.7, 16 152.4 / 152.2, 24 156.8 / 154.7, 64 257 / 248;
// K = 1024, F = 256, 30 tokens 23.8 / 24.2, 48 30.3 / 30.3, 64 31.4 / 31.1, 128
// 40.1 / 38.5.
constexpr int kFewOwnWarps = 15, kFewSharePieces = 30;
constexpr int kFewOwnTokens = kFewOwnWarps + kFewSharePieces;  // rows of one piece; longer ones fewer
constexpr int kUnitBytes = 16384;  // 128 columns x 128 bytes of contraction
constexpr int kProdWarps = 2;      // warps 0-1
constexpr int kMmaWarp0 = 2, kMmaWarps = 2;
constexpr int kLoadWarp0 = 4, kLoadWarps = 8;
constexpr int kFewEpiWarp0 = 12, kFewEpiWarps = 4;

// Rows of a group: an expert with more takes several groups, each of which
// reads its weights (a variant of 8 rows with 10 stages ran no faster for 1 to
// 8 tokens: 71.4 against 70.7 us for one, 199.9 against 199.2 for eight of the
// Mixtral-like layer).
constexpr int kRows = 32;
constexpr int kSt = 8, kBufs = 2;             // stages; tile accumulators in flight
constexpr int kBBytes = 2 * kRows * 128;      // a stage's rows: hi and lo
constexpr int kBufCols = 2 * kRows;           // TMEM columns of one issuer's accumulator
constexpr int kTmem = kBufs * kMmaWarps * kBufCols;
static_assert((kTmem & (kTmem - 1)) == 0 && kTmem >= 32 && kTmem <= 512, "TMEM columns: a power of two");

// a / b for 0 <= a < 2^24, b > 0: the set-up and the tile switches divide by
// sizes known only at run time, and the code of exact integer divisions cost
// more (cold instruction fetches) than they compute
__device__ __forceinline__ int few_div(int a, int b) {
  int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));  // off by one at most
  const int r = a - q * b;
  q += r >= b ? 1 : 0;
  return r < 0 ? q - 1 : q;
}

// One of the two products: `tiles` column tiles per group, kb contraction
// blocks.  The tiles of all groups are numbered; the first waves * gridDim.x go
// whole to CTA (number % gridDim.x), the `left` others as `slices` slices of
// their contraction, item (slice, tile) to CTA (item number % gridDim.x).
struct Product {
  int tiles, kb, waves, left, slices;
  int n, items;  // this CTA's units, and the items (tiles or slices) they belong to
  // by one warp, all lanes with the same result
  __device__ __forceinline__ void plan(int ngroups, int tiles_, int kb_, int lane) {
    tiles = tiles_;
    kb = kb_;
    const int grid = gridDim.x, total = ngroups * tiles;
    waves = few_div(total, grid);
    left = total - waves * grid;
    // slices that make the CTA with the most units have the fewest (of those
    // the smallest count): one candidate per lane
    const int c = min(lane + 1, kFewMaxSlices);
    unsigned cost = static_cast<unsigned>(few_div(left * c + grid - 1, grid)) * few_div(kb + c - 1, c) * 32u + c;
    if (c > kb) cost = 0xffffffffu;
    slices = static_cast<int>(__reduce_min_sync(0xffffffffu, cost) & 31u);
    // the CTA's slice items, one per lane (at most 16: left < grid)
    const int j = lane * grid + blockIdx.x;
    int len = 0;
    if (j < left * slices) {
      const int i = few_div(j, left);
      len = slice_begin(i + 1) - slice_begin(i);
    }
    n = waves * kb + __reduce_add_sync(0xffffffffu, len);
    items = waves + __popc(__ballot_sync(0xffffffffu, len > 0));
  }
  __device__ __forceinline__ int slice_begin(int i) const { return few_div(i * kb, slices); }
};

// Position in this CTA's units of a product.
struct Cursor {
  int item;              // waves first, then the CTA's slice items
  int group, tile;       // column tile `tile` of group `group`
  int kblk, kend;        // contraction block, end of the item's
  int left_tile, slice;  // number among the tiles left over (-1: a whole tile)
  __device__ __forceinline__ void open(const Product &p) {
    int gt = item * gridDim.x + blockIdx.x, k0 = 0;
    kend = p.kb;
    slice = 0;
    left_tile = -1;
    if (item >= p.waves) {
      const int j = gt - p.waves * gridDim.x;
      slice = few_div(j, p.left);
      left_tile = j - slice * p.left;
      gt = p.waves * gridDim.x + left_tile;
      k0 = p.slice_begin(slice);
      kend = p.slice_begin(slice + 1);
    }
    group = few_div(gt, p.tiles);
    tile = gt - group * p.tiles;
    kblk += k0;
  }
  __device__ __forceinline__ void next(const Product &p, int by = 1) {
    kblk += by;
    while (kblk >= kend) {
      kblk -= kend;
      ++item;
      open(p);
    }
  }
  // to unit `u` of the CTA (u < p.n)
  __device__ __forceinline__ void seek(const Product &p, int u) {
    item = -1;
    kend = 0;
    kblk = u;
    next(p, 0);
  }
};

// shared memory behind the stages
struct FewTail {
  // stage s: weights landed; weights landed and rows written; MMAs done
  uint64_t full_a[kSt], full[kSt], done[kSt];
  // accumulator b: sums of issuer i complete
  uint64_t tfull[kBufs][kMmaWarps];
  uint64_t drain[kMmaWarps];
  uint64_t tempty[kBufs];  // accumulator b: read (the only barrier with more than one arrival)
  int last[kSt];       // the stage's newest copy (unit), -1: none
  uint32_t tmem_slot;
  int abort_flag, no_abort;
  uint32_t gave_up;  // GMM_DEV_TIMEOUT of a wait of this CTA
  Product prod[2];
  int scan[kFewThreads / 32];        // rows and groups of each warp's experts
  uint32_t big[kFewOwnTokens];       // largest magnitude of each token's row (bf16 bits)
  float up[kFewMaxPairs];            // power of two that scales each pair's row (E4M3)
  int cnt[kMaxGroups];               // rows per expert, then group offset
  uint16_t first[kMaxGroups];        // first entry of the expert in rows[]
  uint16_t rows[kFewMaxPairs];       // pairs sorted by expert
  uint16_t pos[kFewMaxPairs];        // rank of each pair within its expert
  uint16_t token[kFewMaxPairs];      // token of each pair
  int16_t pair_group[kFewMaxPairs];  // group of each pair, -1: none
  uint16_t g_expert[kFewMaxPairs], g_first[kFewMaxPairs], g_count[kFewMaxPairs];
  int ids[kFewMaxPairs];
};

constexpr size_t kFewSmem = 1024 + static_cast<size_t>(kSt) * (kUnitBytes + kBBytes) + sizeof(FewTail);
static_assert(kFewSmem <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
}

// two E4M3 codes -> their values
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

// Power of two that puts a row's largest magnitude (bf16 bits) into [128, 256);
// at most 2^126, so that its inverse stays normal.  1 for a row with a value
// that is not finite (its results are NaN whatever the scale).
__device__ __forceinline__ float row_scale_up(uint32_t largest) {
  const int e = largest == 0 || largest >= 0x7f80u ? 0 : min(134 - static_cast<int>(largest >> 7), 126);
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

__device__ __forceinline__ float inverse_of_power(float up) {
  return __uint_as_float(0x7f000000u - __float_as_uint(up));  // 2^-e of 2^e
}

// the larger magnitudes of two pairs of bf16 values (as bits)
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t v) { return __vmaxu2(m, v & 0x7fff7fffu); }

// Four bf16 values, scaled, as E4M3 hi and lo codes.  A value that is not
// finite becomes NaN.
__device__ __forceinline__ void split_e4m3(const uint2 &raw, float up, uint32_t &hi, uint32_t &lo) {
  const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&raw);
  const float2 p0 = __bfloat1622float2(b[0]), p1 = __bfloat1622float2(b[1]);
  float v[4] = {p0.x, p0.y, p1.x, p1.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] *= up;
    if (!(fabsf(v[i]) <= 3.0e38f)) v[i] = __uint_as_float(0x7fffffffu);
  }
  const uint16_t h0 = cvt_e4m3x2(v[0], v[1]), h1 = cvt_e4m3x2(v[2], v[3]);
  const float2 f0 = e4m3x2_to_f32(h0), f1 = e4m3x2_to_f32(h1);
  const uint16_t l0 = cvt_e4m3x2((v[0] - f0.x) * 16.0f, (v[1] - f0.y) * 16.0f);
  const uint16_t l1 = cvt_e4m3x2((v[2] - f1.x) * 16.0f, (v[3] - f1.y) * 16.0f);
  hi = h0 | (static_cast<uint32_t>(h1) << 16);
  lo = l0 | (static_cast<uint32_t>(l1) << 16);
}

__device__ __forceinline__ float4 add4(const float4 &a, const float4 &b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

__device__ __forceinline__ float few_silu(float x) { return x / (1.0f + expf(-x)); }

template <int kElem, bool kMN>
__global__ void __launch_bounds__(kFewThreads, 1)
    moe_few_kernel(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2,
                   const FewParams p) {
  constexpr int kBKe = 128 / kElem;  // contraction elements per unit

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sA = smem, *sB = smem + kSt * kUnitBytes;
  FewTail &t = *reinterpret_cast<FewTail *>(sB + kSt * kBBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cooperative_groups::grid_group grid = cooperative_groups::this_grid();

  // ------------------------------------------------ set-up and row grouping
  for (int i = tid; i < p.pairs; i += kFewThreads) {
    t.ids[i] = p.ids[i];
    t.token[i] = static_cast<uint16_t>(i / p.k);
  }
  for (int i = tid; i < p.G; i += kFewThreads) t.cnt[i] = 0;
  if (kElem == 1 && blockIdx.x == 0)
    for (int i = tid; i < p.pairs; i += kFewThreads) p.largest[p.T + i] = 0;  // of h, set after the first product
  constexpr int kBars = 3 * kSt + kBufs * kMmaWarps + kMmaWarps;
  if (tid < kBars + kBufs) mbar_init(&t.full_a[0] + tid, tid < kBars ? 1 : kFewEpiWarps);
  if (tid < kSt) t.last[tid] = -1;
  if (tid < kFewOwnTokens) t.big[tid] = 0;
  if (tid == 0) {
    t.abort_flag = 0;
    t.no_abort = 0;
    t.gave_up = 0;
    if (blockIdx.x == 0) *p.status = 0;
  }
  fence_barrier_init();
  if (warp == 1 && lane == 0) {
    tma_prefetch_desc(&tm1);
    tma_prefetch_desc(&tm2);
  }
  if (warp == kMmaWarp0) {
    tmem_alloc(&t.tmem_slot, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = t.tmem_slot;
  // largest magnitude of each token's row: in every CTA for a few tokens, shared
  // through memory and one more barrier for more
  const int pieces = (p.kb1 * 128 + 1023) >> 10;  // of a row (E4M3: kb1 blocks of 128)
  const bool share = kElem == 1 && (p.T - kFewOwnWarps) * pieces > kFewSharePieces;
  if (warp == 0) {
    // rank of every pair within its expert, in pair order
    for (int base = 0; base < p.pairs; base += 32) {
      const int q = base + lane;
      const int id = q < p.pairs ? t.ids[q] : -1;
      const bool valid = id >= 0 && id < p.G;
      const uint32_t same = __match_any_sync(0xffffffffu, valid ? id : -1 - lane);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int c = valid ? t.cnt[id] : 0;
      __syncwarp();
      if (q < p.pairs) t.pos[q] = static_cast<uint16_t>(c + before);
      if (valid && before == 0) t.cnt[id] = c + __popc(same);
      __syncwarp();
    }
  } else if (kElem == 1) {
    // one warp per piece of 1024 values of a token's row (shared: per row)
    const int span = share ? pieces : 1;
    const int w0 = share ? blockIdx.x * kFewOwnWarps + warp - 1 : warp - 1;
    const int step = share ? gridDim.x * kFewOwnWarps : kFewOwnWarps;
    for (int i = w0; i < (share ? p.T : p.T * pieces); i += step) {
      const int tok = share ? i : few_div(i, pieces), first = share ? 0 : i - tok * pieces;
      const __nv_bfloat16 *row = p.x + static_cast<int64_t>(tok) * (p.kb1 * 128);
      uint32_t m = 0;
      for (int at = first * 1024; at < (first + span) * 1024; at += 1024) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = at + (e * 32 + lane) * 8;
          v[e] = c < p.kb1 * 128 ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          m = max_abs2(max_abs2(max_abs2(max_abs2(m, v[e].x), v[e].y), v[e].z), v[e].w);
      }
      m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
      if (lane == 0) {
        if (share) p.largest[tok] = m;
        else atomicMax(&t.big[tok], m);
      }
    }
  }
  __syncthreads();
  // rows and groups of the experts, in expert order: two experts a thread
  int c[2], n[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    c[i] = 2 * tid + i < p.G ? t.cnt[2 * tid + i] : 0;
    n[i] = (c[i] + kRows - 1) / kRows;
  }
  const int own = (c[0] + c[1]) | ((n[0] + n[1]) << 16);  // both sums in one word (each below 2^15)
  int upto = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) t.scan[warp] = upto;
  if (kElem == 1 && !share && tid < p.T) t.up[tid] = row_scale_up(t.big[tid]);
  __syncthreads();
  const int other = lane < kFewThreads / 32 ? t.scan[lane] : 0;
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? other : 0) + upto - own;
  const int ngroups = __reduce_add_sync(0xffffffffu, other) >> 16;
  if (own) {
    int r = before & 0xffff, g = before >> 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * tid + i;
      if (!c[i]) continue;
      t.first[e] = static_cast<uint16_t>(r);
      t.cnt[e] = g;
      for (int k = 0; k < n[i]; ++k, ++g) {
        t.g_expert[g] = static_cast<uint16_t>(e);
        t.g_first[g] = static_cast<uint16_t>(r + k * kRows);
        t.g_count[g] = static_cast<uint16_t>(min(kRows, c[i] - k * kRows));
      }
      r += c[i];
    }
  }
  if (warp == kFewThreads / 32 - 1 || warp == kFewThreads / 32 - 2) {
    const int ph = warp & 1;
    Product a;
    a.plan(ngroups, ph ? p.tiles2 : p.tiles1, ph ? p.kb2 : p.kb1, lane);
    if (lane == 0) t.prod[ph] = a;
  }
  __syncthreads();
  for (int q = tid; q < p.pairs; q += kFewThreads) {
    const int id = t.ids[q];
    const bool valid = id >= 0 && id < p.G;
    if (valid) t.rows[t.first[id] + t.pos[q]] = static_cast<uint16_t>(q);
    t.pair_group[q] = static_cast<int16_t>(valid ? t.cnt[id] + t.pos[q] / kRows : -1);
  }
  __syncthreads();
  if (share) {
    grid.sync();
    for (int i = tid; i < p.T; i += kFewThreads) t.up[i] = row_scale_up(__ldcg(p.largest + i));
    __syncthreads();
  }

  // A wait that gives up is kept in shared memory and reported when the CTA
  // leaves: no grid barrier lies between CTA 0's reset of the status word and
  // the first waits, so a report from here could be reset again.
  const WaitCtl ctl{p.wait_limit_ns, &t.abort_flag, &t.gave_up};
  // a CTA leaves only when its own copies and MMAs have landed, however short the caller's limit
  const WaitCtl ctl_drain{max(p.wait_limit_ns, static_cast<uint64_t>(1000000000)), &t.no_abort, &t.gave_up};
  const Product prod1 = t.prod[0], prod2 = t.prod[1];
  const int n1 = prod1.n, n2 = prod2.n;
  // E4M3 weights use hi and lo columns, bf16 one column a row
  auto mma_cols = [&](int count) { return kElem == 1 ? 2 * ((count + 7) & ~7) : ((count + 15) & ~15); };

  // Units are numbered over both products: 0 .. n1 - 1 of the first, n1 ..
  // n1 + n2 - 1 of the second; unit u uses stage u % kSt.  A role that gave up
  // a wait stops for good (ok = false) but still joins every barrier below.
  bool ok = true;
  int it = 0;            // producers: next unit of this warp; epilogue: next unit
  int items = 0;         // items before the current product's (accumulator item g uses buffer g % kBufs)
  uint32_t tphase = 0;   // epilogue: parity of each accumulator's next use
  if (warp < kProdWarps) it = warp;
  const uint64_t policy = l2_policy_evict_first();  // the weights are read once

  // producer: the warp's copies of product `ph` up to unit `stop`
  auto produce = [&](int ph, const Product &pr, int begin, int stop) {
    const CUtensorMap *tm = ph ? &tm2 : &tm1;
    if (!ok || it >= stop) return;
    Cursor c{};
    c.seek(pr, it - begin);
    for (;;) {
      const int s = it % kSt;
      if (!mbar_wait(&t.done[s], ((it / kSt) & 1) ^ 1, ctl)) {
        ok = false;
        return;
      }
      mbar_arrive_expect_tx(&t.full_a[s], kUnitBytes);
      t.last[s] = it;
      const int e = t.g_expert[c.group];
      uint8_t *dst = sA + s * kUnitBytes;
      if constexpr (kMN) {
        const int y = e * (pr.kb * kBKe) + c.kblk * kBKe;
#pragma unroll
        for (int h = 0; h < kElem; ++h)
          tma_load_2d_hint(dst + h * (kUnitBytes / kElem), tm, c.tile * 128 + h * kBKe, y, &t.full_a[s], policy);
      } else {
        tma_load_2d_hint(dst, tm, c.kblk * kBKe, e * (pr.tiles * 128) + c.tile * 128, &t.full_a[s], policy);
      }
      it += kProdWarps;
      if (it >= stop) return;
      c.next(pr, kProdWarps);
    }
  };

  for (int ph = 0; ph < 2; ++ph) {
    const Product pr = ph ? prod2 : prod1;
    const int begin = ph ? n1 : 0, end = begin + pr.n;
    if (warp < kProdWarps) {
      if (lane == 0) {
        if (ph == 0) {
          produce(0, prod1, 0, n1);
          // the second product's first stages are started before the barriers
          produce(1, prod2, n1, min(n1 + kSt, n1 + n2));
        } else {
          produce(1, prod2, n1, n1 + n2);
        }
      }
      __syncwarp();
    } else if (warp < kMmaWarp0 + kMmaWarps) {
      if (lane == 0) {
        const int mw = warp - kMmaWarp0;
        int u = begin + (mw - begin % kMmaWarps + kMmaWarps) % kMmaWarps;
        Cursor c{};
        if (ok && u < end) c.seek(pr, u - begin);
        const uint64_t a_desc = kMN ? smem_desc_sw128(smem_u32(sA), kUnitBytes / kElem, 1024)
                                    : smem_desc_sw128(smem_u32(sA), 16, 1024);
        const uint64_t b_desc = smem_desc_sw128(smem_u32(sB), 16, 1024);
        constexpr int kAStep = (kMN ? (32 / kElem) * 128 : 32) >> 4;  // descriptor units (16 bytes) per MMA
        int open = -1;  // the item this issuer is summing
        uint32_t idesc = 0, d = 0;
        for (; ok && u < end;) {
          const int s = u % kSt;
          bool first = c.item != open;
          if (first) {
            open = c.item;
            const int g = items + open, buf = g % kBufs;
            idesc = instr_desc_mn(kElem == 2, kMN, false, static_cast<uint32_t>(mma_cols(t.g_count[c.group])), 128u);
            d = tbase + (buf * kMmaWarps + mw) * kBufCols;
            if (!mbar_wait(&t.tempty[buf], ((g / kBufs) & 1) ^ 1, ctl)) {
              ok = false;
              break;
            }
          }
          // the loader has seen the weights land
          if (!mbar_wait(&t.full[s], (u / kSt) & 1, ctl)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = a_desc + s * (kUnitBytes >> 4), bd = b_desc + s * (kBBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            tc_mma<kElem == 2>(d, ad + kk * kAStep, bd + kk * 2, idesc, first ? 0u : 1u);
            first = false;
          }
          tc_commit(&t.done[s]);
          if (c.kblk + kMmaWarps >= c.kend) tc_commit(&t.tfull[(items + open) % kBufs][mw]);
          u += kMmaWarps;
          if (u < end) c.next(pr, kMmaWarps);
        }
      }
      __syncwarp();
    } else if (warp < kFewEpiWarp0) {
      // ------------------------------------------------- activation loader
      const int lw = warp - kLoadWarp0;
      const __nv_bfloat16 *src = ph ? p.h : p.x;
      const int64_t ld = static_cast<int64_t>(pr.kb) * kBKe;
      // eight rows of a unit: lane's 4 (E4M3) or 2 (bf16) values of each block
      uint2 raw[8];
      Cursor c{};
      auto fetch = [&](uint2 (&r)[8], int r0) {
        const int n = t.g_count[c.group] - r0, f = t.g_first[c.group] + r0;
        const __nv_bfloat16 *base = src + static_cast<int64_t>(c.kblk) * kBKe + lane * (kBKe / 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i < n) {
            const int q = t.rows[f + i];
            const __nv_bfloat16 *a = base + (ph ? q : static_cast<int>(t.token[q])) * ld;
            if constexpr (kElem == 1) r[i] = __ldcg(reinterpret_cast<const uint2 *>(a));
            else r[i].x = __ldcg(reinterpret_cast<const uint32_t *>(a));
          }
        }
      };
      int u = begin + (lw - begin % kLoadWarps + kLoadWarps) % kLoadWarps;  // this warp's units: u % 8 == lw
      if (u < end) {
        c.seek(pr, u - begin);
        fetch(raw, 0);
      }
      for (; ok && u < end; u += kLoadWarps) {
        const int s = u % kSt;
        bool got = mbar_wait(&t.done[s], ((u / kSt) & 1) ^ 1, ctl);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        const int cnt = t.g_count[c.group], lo_row = (cnt + 7) & ~7, f = t.g_first[c.group];
        uint8_t *b = sB + s * kBBytes;
#pragma unroll 1  // 32 rows unrolled overran the instruction cache
        for (int r0 = 0; r0 < cnt; r0 += 8) {
          uint2 next[8];
          if (r0 + 8 < cnt) fetch(next, r0 + 8);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (r0 + i < cnt) {
              const uint32_t at = static_cast<uint32_t>((r0 + i) * 128 + ((lane * 4) ^ (i << 4)));
              if constexpr (kElem == 1) {
                uint32_t hi, lo;
                const int q = t.rows[f + r0 + i];
                split_e4m3(raw[i], t.up[ph ? q : static_cast<int>(t.token[q])], hi, lo);
                *reinterpret_cast<uint32_t *>(b + at) = hi;
                *reinterpret_cast<uint32_t *>(b + lo_row * 128 + at) = lo;
              } else {
                *reinterpret_cast<uint32_t *>(b + at) = raw[i].x;
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) raw[i] = next[i];
        }
        fence_async_smem();
        __syncwarp();
        // the next unit's rows are on their way while the weights land
        if (u + kLoadWarps < end) {
          c.next(pr, kLoadWarps);
          fetch(raw, 0);
        }
        if (lane == 0 && (got = mbar_wait(&t.full_a[s], (u / kSt) & 1, ctl))) mbar_arrive(&t.full[s]);
        ok = __shfl_sync(0xffffffffu, got ? 1 : 0, 0);
      }
    } else {
      // ---------------------------------------------------------- epilogue
      const int q4 = warp & 3;
      const uint32_t tl = tbase + (static_cast<uint32_t>(q4 * 32) << 16);
      const int64_t cols = static_cast<int64_t>(pr.tiles) * 128;
      // one pass per item: the issuers' sums of the whole (sliced) contraction
      Cursor c{};
      it = begin;
      if (it < end) c.seek(pr, 0);
      while (ok && it < end) {
        const int len = c.kend - c.kblk, buf = (items + c.item) % kBufs;
        bool got = true;
        for (int m = 0; m < kMmaWarps; ++m) {
          // issuer m has units of the item unless it is one unit of the other's
          if (len > 1 || it % kMmaWarps == m) {
            if (got) got = mbar_wait(&t.tfull[buf][m], (tphase >> (buf * kMmaWarps + m)) & 1, ctl);
            tphase ^= 1u << (buf * kMmaWarps + m);
          }
        }
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int cnt = t.g_count[c.group], lo_col = (cnt + 7) & ~7, f = t.g_first[c.group];
        const int in_tile = q4 * 32 + lane;
        // slice 0 to [pair][column], the others to
        // [slice - 1][tile left over][row][128]
        float *dst = p.partial + c.tile * 128 + in_tile;
        float *more = p.extra + static_cast<int64_t>((c.slice - 1) * pr.left + c.left_tile) * kRows * 128 + in_tile;
#pragma unroll 1
        for (int r = 0; r < cnt; r += 8) {
          float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
          for (int m = 0; m < kMmaWarps; ++m) {
            if (len > 1 || it % kMmaWarps == m) {
              const uint32_t at = tl + (buf * kMmaWarps + m) * kBufCols + r;
              uint32_t a[8], b[8];
              tmem_ld8(at, a);
              if constexpr (kElem == 1) tmem_ld8(at + lo_col, b);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                v[i] += kElem == 1 ? __fmaf_rn(__uint_as_float(b[i]), 0.0625f, __uint_as_float(a[i]))
                                   : __uint_as_float(a[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (r + i < cnt) {
              const int q = t.rows[f + r + i];
              if constexpr (kElem == 1) v[i] *= inverse_of_power(t.up[ph ? q : static_cast<int>(t.token[q])]);
              if (c.slice == 0) dst[q * cols] = v[i];
              else more[(r + i) * 128] = v[i];
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&t.tempty[buf]);
        it += len;
        if (it < end) c.next(pr, len);
      }
    }
    items += pr.items;
    grid.sync();

    // one warp sums the slices of 128 columns (a tile) of one pair, four
    // columns a lane
    const int64_t cols = static_cast<int64_t>(pr.tiles) * 128;
    // slice `sl` of the tile (NULL: the tile has no such slice)
    auto part_of = [&](int pair, int tile, int sl) -> const float * {
      if (sl == 0) return p.partial + pair * cols + tile * 128;
      const int lt = t.pair_group[pair] * pr.tiles + tile - pr.waves * static_cast<int>(gridDim.x);
      if (lt < 0) return nullptr;
      return p.extra + (static_cast<int64_t>((sl - 1) * pr.left + lt) * kRows + t.pos[pair] % kRows) * 128;
    };
    auto load4 = [&](const float *src) -> float4 {
      return src ? __ldcg(reinterpret_cast<const float4 *>(src) + lane) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    auto tile4 = [&](int pair, int tile) -> float4 {
      float4 a = load4(part_of(pair, tile, 0));
      if (const float *src = pr.slices > 1 ? part_of(pair, tile, 1) : nullptr) {
        const int64_t step = static_cast<int64_t>(pr.left) * kRows * 128;
#pragma unroll 4
        for (int i = 1; i < pr.slices; ++i, src += step) a = add4(a, load4(src));
      }
      return a;
    };
    // With few (pair, tile) items each takes a whole CTA, the warps one slice
    // each, joined in shared memory in a fixed order (the rows' stages, idle
    // now): one warp's loop over up to 16 slices of several terms leaves their
    // latencies, 3 to 5 us, on a few SMs (one Mixtral-like token 74.5 us by
    // warps, 71.2 so).  With more than two a CTA, a warp takes each (the same
    // within 1 % up to 32 tokens).
    float4 *part = reinterpret_cast<float4 *>(sB);
    static_assert(kSt * kBBytes >= kFewThreads * 16, "one float4 a thread");
    const int nwarps = gridDim.x * (kFewThreads / 32), w0 = warp * gridDim.x + blockIdx.x;
    if (ph == 0) {
      const int F = p.F, ft = F / 128;
      // silu(g) * u of one pair's 128 columns (four a lane), g and u without
      // their channel scales
      auto activate = [&](int pair, int tile, float4 g, float4 u) {
        const int col = tile * 128 + lane * 4;
        if constexpr (kElem == 1) {
          const float *sc = p.s1 + static_cast<int64_t>(t.ids[pair]) * 2 * F + col;
          const float4 sg = *reinterpret_cast<const float4 *>(sc), su = *reinterpret_cast<const float4 *>(sc + F);
          g = make_float4(g.x * sg.x, g.y * sg.y, g.z * sg.z, g.w * sg.w);
          u = make_float4(u.x * su.x, u.y * su.y, u.z * su.z, u.w * su.w);
        }
        // one rounding to bf16: the down product's operand type
        const __nv_bfloat162 o[2] = {__floats2bfloat162_rn(few_silu(g.x) * u.x, few_silu(g.y) * u.y),
                                     __floats2bfloat162_rn(few_silu(g.z) * u.z, few_silu(g.w) * u.w)};
        const uint2 v = *reinterpret_cast<const uint2 *>(o);
        *reinterpret_cast<uint2 *>(p.h + static_cast<int64_t>(pair) * F + col) = v;
        if constexpr (kElem == 1) {
          // the row's largest, of the rounded values (a maximum: any order)
          uint32_t m = max_abs2(v.x & 0x7fff7fffu, v.y);
          m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
          if (lane == 0) atomicMax(p.largest + p.T + pair, m);
        }
      };
      if (p.pairs * ft <= 2 * static_cast<int>(gridDim.x)) {
        for (int i = blockIdx.x; i < p.pairs * ft; i += gridDim.x) {
          const int pair = few_div(i, ft), tile = i - pair * ft;
          if (t.pair_group[pair] < 0) continue;
          // warps 0-7: gate slices in turn, 8-15: up slices
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int sl = warp % 8; sl < pr.slices; sl += 8)
            v = add4(v, load4(part_of(pair, tile + (warp / 8) * ft, sl)));
          part[warp * 32 + lane] = v;
          __syncthreads();
          if (warp == 0) {
            float4 u = part[8 * 32 + lane];
#pragma unroll
            for (int w = 1; w < 8; ++w) {
              v = add4(v, part[w * 32 + lane]);
              u = add4(u, part[(8 + w) * 32 + lane]);
            }
            activate(pair, tile, v, u);
          }
          __syncthreads();
        }
      } else {
        for (int i = w0; i < p.pairs * ft; i += nwarps) {
          const int pair = few_div(i, ft), tile = i - pair * ft;
          if (t.pair_group[pair] < 0) continue;
          activate(pair, tile, tile4(pair, tile), tile4(pair, ft + tile));
        }
      }
      grid.sync();
      if constexpr (kElem == 1) {
        for (int q = tid; q < p.pairs; q += kFewThreads) t.up[q] = row_scale_up(__ldcg(p.largest + p.T + q));
        __syncthreads();
      }
    } else {
      const int N = p.N, nt = N / 128;
      auto store4 = [&](int tok, int col, const float4 &y) {
        if (p.y_f32) {
          *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + static_cast<int64_t>(tok) * N + col) = y;
        } else {
          __nv_bfloat162 o[2] = {__floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
          *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.y) + static_cast<int64_t>(tok) * N + col) =
              *reinterpret_cast<uint2 *>(o);
        }
      };
      auto weigh4 = [&](int pair, int col, float4 v) -> float4 {
        if constexpr (kElem == 1) {
          const float4 s = *reinterpret_cast<const float4 *>(p.s2 + static_cast<int64_t>(t.ids[pair]) * N + col);
          v = make_float4(v.x * s.x, v.y * s.y, v.z * s.z, v.w * s.w);
        }
        const float w = p.weights[pair];
        return make_float4(w * v.x, w * v.y, w * v.z, w * v.w);
      };
      if (p.T * nt <= 2 * static_cast<int>(gridDim.x)) {
        constexpr int kWarps = kFewThreads / 32;
        for (int i = blockIdx.x; i < p.T * nt; i += gridDim.x) {
          const int tok = few_div(i, nt), tile = i - tok * nt, col = tile * 128 + lane * 4;
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int c = warp; c < p.k * pr.slices; c += kWarps) {
            const int j = few_div(c, pr.slices), sl = c - j * pr.slices, pair = tok * p.k + j;
            if (t.pair_group[pair] < 0) continue;
            y = add4(y, weigh4(pair, col, load4(part_of(pair, tile, sl))));
          }
          part[warp * 32 + lane] = y;
          __syncthreads();
          if (warp == 0) {
#pragma unroll
            for (int w = 1; w < kWarps; ++w) y = add4(y, part[w * 32 + lane]);
            store4(tok, col, y);
          }
          __syncthreads();
        }
      } else {
        for (int i = w0; i < p.T * nt; i += nwarps) {
          const int tok = few_div(i, nt), tile = i - tok * nt, col = tile * 128 + lane * 4;
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
          for (int j = 0; j < p.k; ++j) {
            const int pair = tok * p.k + j;
            if (t.pair_group[pair] < 0) continue;
            y = add4(y, weigh4(pair, col, tile4(pair, tile)));
          }
          store4(tok, col, y);
        }
      }
    }
  }

  // every copy and MMA has ended before the CTA leaves
  if (warp >= kMmaWarp0 && warp < kMmaWarp0 + kMmaWarps) {
    if (lane == 0) {
      tc_commit(&t.drain[warp - kMmaWarp0]);
      mbar_wait(&t.drain[warp - kMmaWarp0], 0, ctl_drain);
    }
    __syncwarp();
  }
  __syncthreads();
  if (tid == 0)
    for (int s = 0; s < kSt; ++s)
      if (t.last[s] >= 0) mbar_wait(&t.full_a[s], (t.last[s] / kSt) & 1, ctl_drain);
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && t.gave_up) atomicOr(p.status, t.gave_up);  // after the reset: the products' grid barriers lie between
  if (warp == kMmaWarp0) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmem);
  }
}

template <int kElem, bool kMN>
cudaError_t launch_few_inst(const CUtensorMap &tm1, const CUtensorMap &tm2, const FewParams &p, cudaStream_t st) {
  auto kern = moe_few_kernel<kElem, kMN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kFewSmem));
  if (e != cudaSuccess) return e;
  // no more CTAs than units: the barriers of a small layer span fewer SMs
  const int64_t units = static_cast<int64_t>(p.pairs) * max(p.tiles1 * p.kb1, p.tiles2 * p.kb2);
  const int grid = static_cast<int>(units < num_sms() ? units : num_sms());
  void *args[] = {const_cast<CUtensorMap *>(&tm1), const_cast<CUtensorMap *>(&tm2), const_cast<FewParams *>(&p)};
  e = cudaLaunchCooperativeKernel(reinterpret_cast<const void *>(kern), dim3(grid), dim3(kFewThreads), args, kFewSmem,
                                  st);
  if (e != cudaSuccess) cudaGetLastError();  // reported by the return value
  return e;
}

}  // namespace

size_t few_extra_floats() {
  // tiles left over (fewer than CTAs) x (slices - 1) x rows of a group x 128
  return static_cast<size_t>(num_sms()) * (kFewMaxSlices - 1) * kRows * 128;
}

cudaError_t launch_moe_few(int elem, bool mn_major, const CUtensorMap &tm1, const CUtensorMap &tm2,
                           const FewParams &p, cudaStream_t st) {
  if (elem == 1)
    return mn_major ? launch_few_inst<1, true>(tm1, tm2, p, st) : launch_few_inst<1, false>(tm1, tm2, p, st);
  return mn_major ? launch_few_inst<2, true>(tm1, tm2, p, st) : launch_few_inst<2, false>(tm1, tm2, p, st);
}

}  // namespace gmm
