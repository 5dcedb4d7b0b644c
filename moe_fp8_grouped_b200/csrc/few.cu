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
// x 128 bytes of contraction (16 KB).  The units of both products are numbered
// (expert, column tile, contraction block) and every CTA takes one contiguous
// range of equal length, so all SMs stream the same number of bytes whatever
// the routing.  A column tile whose units fall into several ranges gets one
// fp32 partial sum from each CTA; the partials are added in CTA order, so the
// result does not depend on timing.
//
// Tile.  The weights are the 128-row operand of tcgen05.mma and stay in the
// layout they have in memory (MN-major for [G, K, N], K-major for [G, N, K]):
// TMA brings them to shared memory and no register ever holds one.  The
// expert's rows (at most kRows a group; an expert with more gets several
// groups) are the MMA's columns.
//
// Activations stay bf16 in precision although the MMA multiplies E4M3: a bf16
// value has 8 significant bits, so scaled by a power of two (one per row and
// block of 128, from the block's largest magnitude, put into [128, 256)) it is
// hi + lo / 16 with two E4M3 values of 4 significant bits each, exactly for
// values down to 2^-13 of the block's largest and within 2^-22 of that largest
// below.  hi and lo are separate MMA columns and are joined, unscaled and
// summed in fp32 by the epilogue, one block at a time.  bf16 weights multiply
// the bf16 rows as they are.
//
// The layer is one cooperative launch: gate|up product, grid barrier, SwiGLU
// of the summed partials (rounded to bf16, as the separate calls round it),
// grid barrier, down product, grid barrier, weighted sum.  The producer starts
// the down product's first copies before the barriers, so HBM keeps working
// across them.
//
// Warps (320 threads, one CTA per SM): 0 TMA producer, 1 MMA issuer and TMEM
// owner, 2-5 activation loaders, 6-9 epilogue (TMEM lanes 32 (w % 4) ..).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "few.h"
#include "internal.h"
#include "ptx.cuh"

namespace gmm {
namespace {

constexpr int kFewThreads = 320;
constexpr int kUnitBytes = 16384;  // 128 columns x 128 bytes of contraction
constexpr int kLoadWarp0 = 2, kLoadWarps = 4;
constexpr int kFewEpiWarp0 = 6, kFewEpiWarps = 4;

// rows of a group, stages and TMEM buffers of the two variants
template <int kRows>
struct FewCfg;
template <>
struct FewCfg<8> {
  static constexpr int kStages = 11, kBufs = 8, kAhead = 4;
};
template <>
struct FewCfg<32> {
  static constexpr int kStages = 8, kBufs = 4, kAhead = 2;
};

template <int kRows>
constexpr int few_b_bytes() { return 2 * kRows * 128; }  // hi rows and lo rows

// shared memory behind the stages
template <int kRows>
struct FewTail {
  using C = FewCfg<kRows>;
  static constexpr int kRing = C::kStages + C::kBufs;
  uint64_t full_a[C::kStages], full_b[C::kStages], empty[C::kStages];
  uint64_t tfull[C::kBufs], tempty[C::kBufs];
  uint64_t sfull[kRing];
  uint64_t drain;
  uint32_t tmem_slot;
  int abort_flag, no_abort, ngroups;
  float inv_scale[kRing][kRows];
  int cnt[kMaxGroups];               // rows per expert, then group offset
  uint16_t first[kMaxGroups];        // first entry of the expert in rows[]
  uint16_t rows[kFewMaxPairs];       // pairs sorted by expert
  uint16_t pos[kFewMaxPairs];        // rank of each pair within its expert
  int16_t pair_group[kFewMaxPairs];  // group of each pair, -1: none
  uint16_t g_expert[kFewMaxPairs], g_first[kFewMaxPairs], g_count[kFewMaxPairs];
  int ids[kFewMaxPairs];
};

template <int kRows>
constexpr size_t few_smem_bytes() {
  return 1024 + static_cast<size_t>(FewCfg<kRows>::kStages) * (kUnitBytes + few_b_bytes<kRows>()) +
         sizeof(FewTail<kRows>);
}

// One of the two products as a list of units, and this CTA's range of it.
struct Product {
  int tiles, kb;           // column tiles of 128, contraction blocks
  uint64_t total, lo, hi;  // units; this CTA's [lo, hi)
  uint32_t grid;           // CTAs that have units
  __device__ __forceinline__ void init(int ngroups, int tiles_, int kb_) {
    tiles = tiles_;
    kb = kb_;
    total = static_cast<uint64_t>(ngroups) * tiles * kb;
    // CTAs with work: with fewer units than CTAs the first `total` take one
    // each, so that the CTAs of a tile are always consecutive
    grid = static_cast<uint32_t>(min(static_cast<uint64_t>(gridDim.x), total));
    lo = hi = 0;
    if (blockIdx.x < grid) {
      lo = total * blockIdx.x / grid;
      hi = total * (blockIdx.x + 1) / grid;
    }
  }
  // the CTA whose range holds unit u: the largest c with total * c / grid <= u
  __device__ __forceinline__ uint32_t cta_of(uint64_t u) const {
    return static_cast<uint32_t>(((u + 1) * grid - 1) / total);
  }
};

// Position in a product's unit list, advanced one unit at a time.
struct Cursor {
  int group, tile, kblk;
  __device__ __forceinline__ void seek(const Product &p, uint64_t u) {
    kblk = static_cast<int>(u % p.kb);
    const uint64_t gt = u / p.kb;
    tile = static_cast<int>(gt % p.tiles);
    group = static_cast<int>(gt / p.tiles);
  }
  __device__ __forceinline__ void next(const Product &p) {
    if (++kblk == p.kb) {
      kblk = 0;
      if (++tile == p.tiles) {
        tile = 0;
        ++group;
      }
    }
  }
};

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

// Four bf16 values of a row's 128-block (the warp's lanes hold the block) as
// E4M3 hi and lo codes; returns the factor that undoes the scaling.  A value
// that is not finite becomes NaN.
__device__ __forceinline__ float split_e4m3(const uint2 &raw, uint32_t &hi, uint32_t &lo) {
  const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&raw);
  const float2 p0 = __bfloat1622float2(b[0]), p1 = __bfloat1622float2(b[1]);
  float v[4] = {p0.x, p0.y, p1.x, p1.y};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
    if (a >= 0x7f800000u) v[i] = __uint_as_float(0x7fffffffu);
    else m = max(m, a);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  // 2^s with largest * 2^s in [128, 256); s <= 126 so that 2^-s stays normal
  const int s = m == 0 ? 0 : min(134 - static_cast<int>(m >> 23), 126);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + s) << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] *= up;
  const uint16_t h0 = cvt_e4m3x2(v[0], v[1]), h1 = cvt_e4m3x2(v[2], v[3]);
  const float2 f0 = e4m3x2_to_f32(h0), f1 = e4m3x2_to_f32(h1);
  const uint16_t l0 = cvt_e4m3x2((v[0] - f0.x) * 16.0f, (v[1] - f0.y) * 16.0f);
  const uint16_t l1 = cvt_e4m3x2((v[2] - f1.x) * 16.0f, (v[3] - f1.y) * 16.0f);
  hi = h0 | (static_cast<uint32_t>(h1) << 16);
  lo = l0 | (static_cast<uint32_t>(l1) << 16);
  return __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
}

__device__ __forceinline__ float few_silu(float x) { return x / (1.0f + expf(-x)); }

template <int kElem, bool kMN, int kRows>
__global__ void __launch_bounds__(kFewThreads, 1)
    moe_few_kernel(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2,
                   const FewParams p) {
  using C = FewCfg<kRows>;
  using Tail = FewTail<kRows>;
  constexpr int kSt = C::kStages, kBufs = C::kBufs, kRing = Tail::kRing;
  constexpr int kBBytes = few_b_bytes<kRows>();
  constexpr int kBKe = 128 / kElem;  // contraction elements per unit
  constexpr int kBufCols = 2 * kRows;
  constexpr int kTmem = kBufs * kBufCols < 32 ? 32 : kBufs * kBufCols;
  constexpr int kRowsPerWarp = kRows / kLoadWarps;
  static_assert((kTmem & (kTmem - 1)) == 0 && kTmem <= 512, "TMEM columns: a power of two");

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sA = smem, *sB = smem + kSt * kUnitBytes;
  Tail &t = *reinterpret_cast<Tail *>(sB + kSt * kBBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cooperative_groups::grid_group grid = cooperative_groups::this_grid();

  // ------------------------------------------------ set-up and row grouping
  for (int i = tid; i < p.pairs; i += kFewThreads) t.ids[i] = p.ids[i];
  for (int i = tid; i < p.G; i += kFewThreads) t.cnt[i] = 0;
  if (tid == 0) {
    for (int i = 0; i < kSt; ++i) {
      mbar_init(&t.full_a[i], 1);
      mbar_init(&t.full_b[i], kLoadWarps);
      mbar_init(&t.empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&t.tfull[i], 1);
      mbar_init(&t.tempty[i], kFewEpiWarps);
    }
    for (int i = 0; i < kRing; ++i) mbar_init(&t.sfull[i], kLoadWarps);
    mbar_init(&t.drain, 1);
    t.abort_flag = 0;
    t.no_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm1);
    tma_prefetch_desc(&tm2);
    if (blockIdx.x == 0) *p.status = 0;
  }
  if (warp == 1) {
    tmem_alloc(&t.tmem_slot, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = t.tmem_slot;
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
    // rows and groups of the experts, in expert order
    int row0 = 0, grp0 = 0;
    for (int base = 0; base < p.G; base += 32) {
      const int e = base + lane;
      const int c = e < p.G ? t.cnt[e] : 0;
      const int n = (c + kRows - 1) / kRows;
      int both = c | (n << 16);  // both prefixes in one scan (each below 2^15)
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, both, d);
        if (lane >= d) both += o;
      }
      const int last = __shfl_sync(0xffffffffu, both, 31);
      const int r = row0 + (both & 0xffff) - c, g = grp0 + (both >> 16) - n;
      if (e < p.G) {
        t.first[e] = static_cast<uint16_t>(r);
        t.cnt[e] = g;
      }
      for (int i = 0; i < n; ++i) {
        t.g_expert[g + i] = static_cast<uint16_t>(e);
        t.g_first[g + i] = static_cast<uint16_t>(r + i * kRows);
        t.g_count[g + i] = static_cast<uint16_t>(min(kRows, c - i * kRows));
      }
      row0 += last & 0xffff;
      grp0 += last >> 16;
    }
    if (lane == 0) t.ngroups = grp0;
  }
  __syncthreads();
  for (int q = tid; q < p.pairs; q += kFewThreads) {
    const int id = t.ids[q];
    const bool valid = id >= 0 && id < p.G;
    if (valid) t.rows[t.first[id] + t.pos[q]] = static_cast<uint16_t>(q);
    t.pair_group[q] = static_cast<int16_t>(valid ? t.cnt[id] + t.pos[q] / kRows : -1);
  }
  __syncthreads();

  const WaitCtl ctl{p.wait_limit_ns, &t.abort_flag, p.status};
  const WaitCtl ctl_drain{p.wait_limit_ns, &t.no_abort, p.status};
  Product prod[2];
  prod[0].init(t.ngroups, p.tiles1, p.kb1);
  prod[1].init(t.ngroups, p.tiles2, p.kb2);
  const int n1 = static_cast<int>(prod[0].hi - prod[0].lo), n2 = static_cast<int>(prod[1].hi - prod[1].lo);
  // products with block scales (E4M3) use hi and lo columns, bf16 one column a row
  auto mma_cols = [&](int count) { return kElem == 1 ? 2 * ((count + 7) & ~7) : ((count + 15) & ~15); };

  // per-role position over both products: units it = 0 .. n1 - 1 belong to the
  // first product, n1 .. n1 + n2 - 1 to the second; a role that gave up a
  // wait stops for good (ok = false) but still joins every barrier below
  int it = 0;
  bool ok = true;

  // producer: copies until `stop`
  Cursor pc;
  auto produce = [&](int stop) {
    for (; ok && it < stop; ++it) {
      const int ph = it >= n1;
      const Product &pr = prod[ph];
      if (it == 0 || it == n1) pc.seek(pr, pr.lo);
      const int s = it % kSt;
      if (!mbar_wait(&t.empty[s], ((it / kSt) & 1) ^ 1, ctl)) {
        ok = false;
        break;
      }
      mbar_arrive_expect_tx(&t.full_a[s], kUnitBytes);
      const int e = t.g_expert[pc.group];
      const CUtensorMap *tm = ph ? &tm2 : &tm1;
      uint8_t *dst = sA + s * kUnitBytes;
      if constexpr (kMN) {
        const int y = e * (pr.kb * kBKe) + pc.kblk * kBKe;
#pragma unroll
        for (int h = 0; h < kElem; ++h)
          tma_load_2d(dst + h * (kUnitBytes / kElem), tm, pc.tile * 128 + h * kBKe, y, &t.full_a[s]);
      } else {
        tma_load_2d(dst, tm, pc.kblk * kBKe, e * (pr.tiles * 128) + pc.tile * 128, &t.full_a[s]);
      }
      pc.next(pr);
    }
  };

  for (int ph = 0; ph < 2; ++ph) {
    const Product &pr = prod[ph];
    const int end = ph ? n1 + n2 : n1;
    if (warp == 0) {
      // the second product's first stages are started before the barriers
      if (lane == 0) produce(ph ? end : min(n1 + kSt, n1 + n2));
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) {
        Cursor c;
        if (it < end) c.seek(pr, pr.lo);
        for (; ok && it < end; ++it, c.next(pr)) {
          const int s = it % kSt, buf = it % kBufs;
          if (!mbar_wait(&t.tempty[buf], ((it / kBufs) & 1) ^ 1, ctl) ||
              !mbar_wait(&t.full_a[s], (it / kSt) & 1, ctl) || !mbar_wait(&t.full_b[s], (it / kSt) & 1, ctl)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t idesc =
              instr_desc_mn(kElem == 2, kMN, false, static_cast<uint32_t>(mma_cols(t.g_count[c.group])), 128u);
          const uint32_t a0 = smem_u32(sA + s * kUnitBytes), b0 = smem_u32(sB + s * kBBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t ad = kMN ? smem_desc_sw128(a0 + kk * (32 / kElem) * 128, kUnitBytes / kElem, 1024)
                                    : smem_desc_sw128(a0 + kk * 32, 16, 1024);
            tc_mma<kElem == 2>(tbase + buf * kBufCols, ad, smem_desc_sw128(b0 + kk * 32, 16, 1024), idesc,
                               kk ? 1u : 0u);
          }
          tc_commit(&t.empty[s]);
          tc_commit(&t.tfull[buf]);
        }
      }
      __syncwarp();
    } else if (warp < kFewEpiWarp0) {
      // ------------------------------------------------- activation loader
      const int lw = warp - kLoadWarp0;
      const __nv_bfloat16 *src = ph ? p.h : p.x;
      const int64_t ld = static_cast<int64_t>(pr.kb) * kBKe;
      // lane's values of a row's block: 4 (E4M3) or 2 (bf16)
      uint2 ahead[C::kAhead][kRowsPerWarp];
      auto fetch = [&](const Cursor &c, uint2 (&r)[kRowsPerWarp]) {
        const int n = t.g_count[c.group], f = t.g_first[c.group];
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i) {
          const int row = lw + kLoadWarps * i;
          if (row < n) {
            const int q = t.rows[f + row];
            const __nv_bfloat16 *a =
                src + (ph ? q : q / p.k) * ld + static_cast<int64_t>(c.kblk) * kBKe + lane * (kBKe / 32);
            if constexpr (kElem == 1) r[i] = __ldcg(reinterpret_cast<const uint2 *>(a));
            else r[i].x = __ldcg(reinterpret_cast<const uint32_t *>(a));
          }
        }
      };
      const int n = end - it;
      Cursor c, f;
      if (n > 0) {
        c.seek(pr, pr.lo);
        f.seek(pr, pr.lo);
      }
      int fetched = 0;
#pragma unroll
      for (int d = 0; d < C::kAhead; ++d)
        if (fetched < n) {
          fetch(f, ahead[d]);
          f.next(pr);
          ++fetched;
        }
      for (int done = 0; ok && done < n;) {
#pragma unroll
        for (int d = 0; d < C::kAhead; ++d) {
          if (done >= n || !ok) continue;
          const int s = it % kSt, slot = it % kRing;
          bool got = mbar_wait(&t.empty[s], ((it / kSt) & 1) ^ 1, ctl);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            continue;
          }
          const int cnt = t.g_count[c.group], lo_row = (cnt + 7) & ~7;
          uint8_t *b = sB + s * kBBytes;
#pragma unroll
          for (int i = 0; i < kRowsPerWarp; ++i) {
            const int row = lw + kLoadWarps * i;
            if (row < cnt) {
              const uint32_t at = static_cast<uint32_t>(row * 128 + ((lane * 4) ^ ((row & 7) << 4)));
              if constexpr (kElem == 1) {
                uint32_t hi, lo;
                const float inv = split_e4m3(ahead[d][i], hi, lo);
                *reinterpret_cast<uint32_t *>(b + at) = hi;
                *reinterpret_cast<uint32_t *>(b + lo_row * 128 + at) = lo;
                if (lane == 0) t.inv_scale[slot][row] = inv;
              } else {
                *reinterpret_cast<uint32_t *>(b + at) = ahead[d][i].x;
              }
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&t.full_b[s]);
            mbar_arrive(&t.sfull[slot]);
          }
          if (fetched < n) {
            fetch(f, ahead[d]);
            f.next(pr);
            ++fetched;
          }
          c.next(pr);
          ++done;
          ++it;
        }
      }
    } else {
      // ---------------------------------------------------------- epilogue
      const int q4 = warp & 3;
      const uint32_t tl = tbase + (static_cast<uint32_t>(q4 * 32) << 16);
      const int64_t cols = static_cast<int64_t>(pr.tiles) * 128;
      float acc[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) acc[i] = 0.0f;
      Cursor c;
      if (it < end) c.seek(pr, pr.lo);
      for (; it < end; ++it) {
        const int buf = it % kBufs, slot = it % kRing;
        bool got = mbar_wait(&t.tfull[buf], (it / kBufs) & 1, ctl);
        if (got) got = mbar_wait(&t.sfull[slot], (it / kRing) & 1, ctl);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int cnt = t.g_count[c.group], lo_col = (cnt + 7) & ~7;
#pragma unroll
        for (int r = 0; r < kRows; r += 8) {
          if (r < cnt) {
            uint32_t a[8];
            tmem_ld8(tl + buf * kBufCols + r, a);
            if constexpr (kElem == 1) {
              uint32_t b[8];
              tmem_ld8(tl + buf * kBufCols + lo_col + r, b);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                acc[r + i] = __fmaf_rn(__fmaf_rn(__uint_as_float(b[i]), 0.0625f, __uint_as_float(a[i])),
                                       t.inv_scale[slot][r + i], acc[r + i]);
            } else {
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) acc[r + i] += __uint_as_float(a[i]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&t.tempty[buf]);
        if (c.kblk == pr.kb - 1 || it == end - 1) {
          // this CTA's partial sum of the tile: [slot][pair][column]
          const uint64_t u0 = (static_cast<uint64_t>(c.group) * pr.tiles + c.tile) * pr.kb;
          const uint32_t part = blockIdx.x - pr.cta_of(u0);
          const int f = t.g_first[c.group];
          float *dst = p.partial + static_cast<int64_t>(part) * p.pairs * cols + c.tile * 128 + q4 * 32 + lane;
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            if (r < cnt) dst[t.rows[f + r] * cols] = acc[r];
            acc[r] = 0.0f;
          }
        }
        c.next(pr);
      }
    }
    grid.sync();

    // sum of a tile's partials for one pair and four columns
    const int64_t cols = static_cast<int64_t>(pr.tiles) * 128;
    auto total4 = [&](int pair, int col) -> float4 {
      const uint64_t u0 = (static_cast<uint64_t>(t.pair_group[pair]) * pr.tiles + col / 128) * pr.kb;
      const uint32_t parts = pr.cta_of(u0 + pr.kb - 1) - pr.cta_of(u0) + 1;
      const float *src = p.partial + pair * cols + col;
      float4 a = __ldcg(reinterpret_cast<const float4 *>(src));
      for (uint32_t i = 1; i < parts; ++i) {
        const float4 b = __ldcg(reinterpret_cast<const float4 *>(src + i * p.pairs * cols));
        a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
      }
      return a;
    };
    const int64_t nthreads = static_cast<int64_t>(gridDim.x) * kFewThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kFewThreads + tid;
    if (ph == 0) {
      const int F = p.F;
      for (int64_t i = first; i < static_cast<int64_t>(p.pairs) * (F / 4); i += nthreads) {
        const int pair = static_cast<int>(i / (F / 4)), col = static_cast<int>(i % (F / 4)) * 4;
        const int id = t.ids[pair];
        if (t.pair_group[pair] < 0) continue;
        float4 g = total4(pair, col), u = total4(pair, F + col);
        if constexpr (kElem == 1) {
          const float *sc = p.s1 + static_cast<int64_t>(id) * 2 * F + col;
          const float4 sg = *reinterpret_cast<const float4 *>(sc), su = *reinterpret_cast<const float4 *>(sc + F);
          g = make_float4(g.x * sg.x, g.y * sg.y, g.z * sg.z, g.w * sg.w);
          u = make_float4(u.x * su.x, u.y * su.y, u.z * su.z, u.w * su.w);
        }
        // one rounding to bf16: the down product's operand type
        __nv_bfloat162 o[2] = {__floats2bfloat162_rn(few_silu(g.x) * u.x, few_silu(g.y) * u.y),
                               __floats2bfloat162_rn(few_silu(g.z) * u.z, few_silu(g.w) * u.w)};
        *reinterpret_cast<uint2 *>(p.h + static_cast<int64_t>(pair) * F + col) = *reinterpret_cast<uint2 *>(o);
      }
      grid.sync();
    } else {
      const int N = p.N;
      for (int64_t i = first; i < static_cast<int64_t>(p.T) * (N / 4); i += nthreads) {
        const int tok = static_cast<int>(i / (N / 4)), col = static_cast<int>(i % (N / 4)) * 4;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int j = 0; j < p.k; ++j) {
          const int pair = tok * p.k + j;
          if (t.pair_group[pair] < 0) continue;
          float4 v = total4(pair, col);
          if constexpr (kElem == 1) {
            const float4 s = *reinterpret_cast<const float4 *>(p.s2 + static_cast<int64_t>(t.ids[pair]) * N + col);
            v = make_float4(v.x * s.x, v.y * s.y, v.z * s.z, v.w * s.w);
          }
          const float w = p.weights[pair];
          y = make_float4(fmaf(w, v.x, y.x), fmaf(w, v.y, y.y), fmaf(w, v.z, y.z), fmaf(w, v.w, y.w));
        }
        if (p.y_f32) {
          *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + static_cast<int64_t>(tok) * N + col) = y;
        } else {
          __nv_bfloat162 o[2] = {__floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
          *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.y) + static_cast<int64_t>(tok) * N + col) =
              *reinterpret_cast<uint2 *>(o);
        }
      }
    }
  }

  // every copy and MMA has ended before the CTA leaves
  if (warp == 0 && lane == 0)
    for (int i = it > kSt ? it - kSt : 0; i < it; ++i) mbar_wait(&t.full_a[i % kSt], (i / kSt) & 1, ctl_drain);
  if (warp == 1) {
    if (lane == 0) {
      tc_commit(&t.drain);
      mbar_wait(&t.drain, 0, ctl_drain);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmem);
  }
}

template <int kElem, bool kMN, int kRows>
cudaError_t launch_few_inst(const CUtensorMap &tm1, const CUtensorMap &tm2, const FewParams &p, cudaStream_t st) {
  auto kern = moe_few_kernel<kElem, kMN, kRows>;
  constexpr size_t smem = few_smem_bytes<kRows>();
  static_assert(smem <= 232448, "shared memory of one CTA");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  void *args[] = {const_cast<CUtensorMap *>(&tm1), const_cast<CUtensorMap *>(&tm2), const_cast<FewParams *>(&p)};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void *>(kern), dim3(num_sms()), dim3(kFewThreads), args,
                                     smem, st);
}

template <int kElem, bool kMN>
cudaError_t launch_few_rows(const CUtensorMap &tm1, const CUtensorMap &tm2, const FewParams &p, cudaStream_t st) {
  return p.T <= 8 ? launch_few_inst<kElem, kMN, 8>(tm1, tm2, p, st)
                  : launch_few_inst<kElem, kMN, 32>(tm1, tm2, p, st);
}

}  // namespace

int few_parts(int64_t tiles, int64_t kb) {
  // fewest units: one group.  A CTA's range then holds at least `len` units,
  // so a tile's kb units lie in at most (kb - 1) / len + 2 ranges
  const int64_t len = tiles * kb / num_sms();
  if (len == 0) return static_cast<int>(kb);
  const int64_t parts = (kb - 1) / len + 2;
  return static_cast<int>(parts < kb ? parts : kb);
}

cudaError_t launch_moe_few(int elem, bool mn_major, const CUtensorMap &tm1, const CUtensorMap &tm2,
                           const FewParams &p, cudaStream_t st) {
  if (elem == 1) return mn_major ? launch_few_rows<1, true>(tm1, tm2, p, st) : launch_few_rows<1, false>(tm1, tm2, p, st);
  return mn_major ? launch_few_rows<2, true>(tm1, tm2, p, st) : launch_few_rows<2, false>(tm1, tm2, p, st);
}

}  // namespace gmm
