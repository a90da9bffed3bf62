// paged_decode.cuh -- attention of few rows (generated or drafted tokens) over a paged cache.
//
// The cache is read once and little is computed on it, so this kernel is bound by DRAM.  One
// CTA of eight warps per SM, and every warp a worker of its own: it has its share of the key tiles,
// keeps its ring of three tiles (8 KB of K and V each: 192 KB in flight per SM; TMA boxes of
// one page, zero fill for pages that are missing) full across units, and holds 8 or 16 rows'
// running maxima, sums and accumulators.  Nothing is exchanged between warps, so a change of unit
// costs one warp's latency under the seven others' loads (with the CTA as the worker and the
// warps joined at the end of each unit it cost 4 us of the SM).
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, by mma.sync m16n8k16 with the
// cache as the 16-row operand and the rows as the 8 columns: a group of up to 8 heads wastes
// nothing (as the 16-row operand it would waste half of every product and of the softmax; a tcgen05 tile
// of 128 rows nearly all).  P goes from the one accumulator layout to the other operand's by
// transposing its 8 x 8 blocks (movmatrix).  The running maximum is raised lazily, by more than 8
// in base 2, so that a tile usually needs no reduction across lanes and no rescaling.
//
// BF16 cache: operands by ldmatrix from the 128-byte-swizzled tiles, P rounded to BF16.
// E4M3 cache: K and V are converted to FP16, which holds E4M3 exactly; Q is scaled per row by
// a power of two into FP16 (11 bits: exact for BF16's 8 down to 2^-17 of the row's largest value, off by
// 2^-25 of that at most below) and P is rounded to FP16.  The order of the head dimension in the first product and of the
// output columns in the second is free, so each lane takes contiguous bytes of K rows (16) and
// V rows (D / 8) and no byte is shuffled across lanes.
#pragma once

#include <cuda_fp16.h>

#include "paged_common.cuh"

namespace mxq {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecStages = 3;  // of each warp
constexpr int kDecStageBytes = 8192;
constexpr int kDecMinTiles = 2;  // 777 keys x 8 heads: 13.6 us, with 4 14.7, with 1 20.3, with 8 16.1

// Workers of `ctas` CTAs, and whether every key head has one: shares are of one head's line, so with fewer
// workers than heads nobody would have any (1024 heads of 64 on a partition of fewer than 128 SMs).
__host__ __device__ constexpr int dec_workers(int ctas) { return ctas * kDecWarps; }
__host__ __device__ constexpr bool dec_covers(int ctas, int heads) { return dec_workers(ctas) >= heads; }

template <int D, bool kFp8>
struct DecShape {
  static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
  static constexpr int kTileBytes = kDecStageBytes / 2;  // K or V
  static constexpr int kKeys = kTileBytes / kRowBytes;
  static constexpr int kBoxRowBytes = kRowBytes > 128 ? 128 : kRowBytes;  // one TMA box's row
  static constexpr int kHalves = kRowBytes / kBoxRowBytes;
  static constexpr int kSmemBytes = 1024 + kDecWarps * kDecStages * kDecStageBytes;
  static_assert(kKeys >= 16 && kKeys / 8 * 2 <= 32, "a lane for each copy");
};

__device__ __forceinline__ void tma_load_5d(void* smem_dst, const CUtensorMap* m, int32_t c0, int32_t c1, int32_t c2,
                                            int32_t c3, int32_t c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <bool kHalf>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The 8 x 8 block of 16-bit values of which each lane holds two of a row, transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// E4M3 pairs (bits 0-15, 16-31) -> FP16 pairs, exactly.
__device__ __forceinline__ uint2 e4m3x4_to_f16(uint32_t w) {
  uint2 h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(h.x), "=r"(h.y)
      : "r"(w));
  return h;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// kNt: blocks of eight rows of a unit.
template <int D, bool kFp8, int kNt>
__global__ void __launch_bounds__(kDecThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const PagedParams p) {
  using S = DecShape<D, kFp8>;
  constexpr int kKeys = S::kKeys;
  constexpr int kMt = kKeys / 16;  // blocks of 16 keys
  constexpr int kKs = D / 16;      // steps of the first product, blocks of 16 output columns
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ ShareScratch scratch;
  __shared__ uint64_t full_bars[kDecWarps][kDecStages];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    for (int s = 0; s < kDecWarps * kDecStages; ++s) mbar_init(&full_bars[0][0] + s, 1);
    fence_mbar_init();
  }
  griddep_launch_dependents();
  griddep_wait();
  const Share sh = find_share<kKeys, kDecThreads, kDecWarps, kDecMinTiles, 0, true>(p, scratch);  // has the block's barriers
  const int worker = blockIdx.x * kDecWarps + warp;
  if (lane == 0) p.part_units[worker] = make_int4(0, 0, 0, 0);
  if (sh.count == 0) return;
  uint8_t* ring = smem + warp * kDecStages * kDecStageBytes;
  uint64_t* full = full_bars[warp];

  // Copies run kDecStages tiles ahead of the tile at hand.  Lane i has copy i of a tile: a box of K,
  // or of V.  The SM's copy engine takes some 20 ns a copy, so a box holds all of a token's bytes:
  // its 128-byte pieces follow one another, each of page_box rows.
  const int nbox = kKeys / p.page_box, box_shift = 31 - __clz(p.page_box);
  const int box = lane & (nbox - 1);
  const bool is_v = lane >= nbox, copies = lane < nbox * 2;
  const int piece_stride = p.page_box * 128;
  auto key_offset = [&](int key) {  // of its first piece, in a tile
    return (key >> box_shift) * p.page_box * S::kRowBytes + (key & (p.page_box - 1)) * S::kBoxRowBytes;
  };
  Unit lu = sh.u;
  int ltile = sh.offset;
  int64_t lleft = sh.count;
  int batch_at = 0, batch_b = -1, entries = -1;  // block-table entries [batch_at, +32) of sequence batch_b
  uint32_t boxes[kDecStages] = {};               // per stage: boxes whose page is there
  auto copy_next = [&](int stage) {
    if (lleft == 0) return;
    const int key0 = (lu.kt0 + ltile) * kKeys;
    const int first = key0 / p.page_size, box_key = key0 + box * p.page_box, entry = box_key / p.page_size;
    if (batch_b != lu.b || first < batch_at || first + nbox > batch_at + 32) {
      batch_b = lu.b;
      batch_at = first;
      entries = first + lane < p.table_stride ? p.block_table[lu.b * p.table_stride + first + lane] : -1;
    }
    const int page = __shfl_sync(0xffffffffu, entries, min(entry - batch_at, 31));
    const bool need = box_key < lu.hi && box_key + p.page_box > lu.lo;
    const bool there = need && page >= 0 && page < p.num_pages;
    const uint32_t mask = __ballot_sync(0xffffffffu, lane < nbox && there);
#pragma unroll
    for (int s = 0; s < kDecStages; ++s)
      if (s == stage) boxes[s] = mask;
    if (lane == 0) mbar_arrive_expect_tx(&full[stage], kDecStageBytes);
    __syncwarp();
    if (copies) {
      uint8_t* dst = ring + stage * kDecStageBytes + (is_v ? S::kTileBytes : 0) + box * p.page_box * S::kRowBytes;
      tma_load_5d(dst, is_v ? &tmap_v : &tmap_k, 0, there ? box_key - entry * p.page_size : 0, 0, lu.hk,
                  there ? page : -1, &full[stage]);  // page out of range: the box is filled with zeros
    }
    --lleft;
    if (++ltile == lu.nt && lleft > 0) {
      next_unit<kKeys, true>(p, lu);
      ltile = 0;
      // its queries, which are wanted when it begins
      if (lane < lu.rows)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + row_offset<D>(p, lu.s.q0, lu.hk, lu.r0 + lane, p.ldq)));
    }
  };
  for (int s = 0; s < kDecStages; ++s) copy_next(s);

  // Fragments: lane (r, c) has row r (of eight) of a block as an operand, and rows 2 c, 2 c + 1 in
  // accumulators.
  const int r = lane >> 2, c = lane & 3;
  int k_off[kMt], v_off[kMt];  // of this lane's rows for ldmatrix, BF16 (row & 7 = lane & 7 in both)
#pragma unroll
  for (int mt = 0; mt < kMt; ++mt) {
    k_off[mt] = key_offset(16 * mt + (lane & 15));
    v_off[mt] = key_offset(16 * mt + (lane & 7) + ((lane >> 4) << 3));
  }
  Unit u = sh.u;
  int tile = sh.offset, begun = tile;  // the tile at which this worker began the unit
  int64_t left = sh.count, at = sh.begin;
  int st = 0;
  uint32_t phase = 0;
  bool ok = true;
  while (ok && left > 0) {
    const int n = static_cast<int>(min(left, static_cast<int64_t>(min(u.nt - tile, kRunKeys / kKeys))));
    uint32_t qb[kKs][kNt][2];
    float t_scale[kNt][2];
    int klo[kNt][2], khi[kNt][2];  // the keys that rows 8 t + 2 c, + 1 attend
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
      const uint16_t* src = p.q + row_offset<D>(p, u.s.q0, u.hk, u.r0 + min(8 * t + r, u.rows - 1), p.ldq);
      if constexpr (kFp8) {
        uint2 raw[kKs];
        float big = 0.f;
#pragma unroll
        for (int s = 0; s < kKs; ++s) raw[s] = *reinterpret_cast<const uint2*>(src + (s >> 2) * 64 + 16 * c + 4 * (s & 3));
#pragma unroll
        for (int s = 0; s < kKs; ++s) {
          const uint32_t w[2] = {raw[s].x, raw[s].y};
#pragma unroll
          for (int k = 0; k < 2; ++k)
            big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^-e with the row's largest value in [1, 2) 2^e (or [2, 4) 2^126); Inf and subnormals as they are
        const int e = min(static_cast<int>(__float_as_uint(big) >> 23) - 127, 126);
        const bool fits = e >= -126 && big != INFINITY;
        const float down = fits ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 1.f;
        const float up =
            fits ? nonzero_scale(p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23)) : p.scale_log2;
#pragma unroll
        for (int s = 0; s < kKs; ++s) {
          const uint32_t w[2] = {raw[s].x, raw[s].y};
#pragma unroll
          for (int k = 0; k < 2; ++k)
            qb[s][t][k] = pack_f16x2(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) t_scale[t][i] = __shfl_sync(0xffffffffu, up, 4 * (2 * c + i));
      } else {
#pragma unroll
        for (int s = 0; s < kKs; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k) qb[s][t][k] = *reinterpret_cast<const uint32_t*>(src + 16 * s + 8 * k + 2 * c);
        t_scale[t][0] = t_scale[t][1] = p.scale_log2;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = (u.r0 + min(8 * t + 2 * c + i, u.rows - 1)) / p.G;
        const int2 kr = key_range(p, u.s, tok, tok);
        klo[t][i] = kr.x;
        khi[t][i] = kr.y;
      }
    }
    // keys that every row of the tile attends
    const int all_lo = key_range(p, u.s, u.i1, u.i1).x, all_hi = key_range(p, u.s, u.i0, u.i0).y;
    const uint32_t all_boxes = (1u << nbox) - 1u;

    float o[kKs][kNt][4] = {};
    float m[kNt][2], l[kNt][2];
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
    for (int k = 0; k < n; ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait(&full[st], phase));
      if (!ok) break;
      const int key0 = (u.kt0 + tile + k) * kKeys;
      uint32_t there = boxes[0];
#pragma unroll
      for (int s = 1; s < kDecStages; ++s)
        if (s == st) there = boxes[s];
      uint8_t* kt = ring + st * kDecStageBytes;
      uint8_t* vt = kt + S::kTileBytes;
      const uint32_t ks = smem_u32(kt), vs = smem_u32(vt);
      if (key0 < u.lo || key0 + kKeys > u.hi) {
        // values of keys that no row of the unit attends may be anything: 0 x NaN is NaN
        for (int i = lane; i < kKeys * (S::kRowBytes / 16); i += 32) {
          const int key = i / (S::kRowBytes / 16);
          if (key0 + key < u.lo || key0 + key >= u.hi) {
            const int ch = i % (S::kRowBytes / 16);
            *reinterpret_cast<uint4*>(vt + key_offset(key) + (ch >> 3) * piece_stride + (ch & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
        }
        __syncwarp();
      }
      // S^T = K Q^T
      float sc[kMt][kNt][4];
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
#pragma unroll
        for (int t = 0; t < kNt; ++t) sc[mt][t][0] = sc[mt][t][1] = sc[mt][t][2] = sc[mt][t][3] = 0.f;
        if constexpr (kFp8) {
          const int key = 16 * mt + r;  // and + 8, with the same swizzle in either layout
          const int sw = D == 128 ? (key & 7) : ((key >> 1) & 3);
#pragma unroll
          for (int g = 0; g < D / 64; ++g) {
            uint4 w[2];
            w[0] = *reinterpret_cast<const uint4*>(kt + key * D + (((4 * g + c) ^ sw) << 4));
            w[1] = *reinterpret_cast<const uint4*>(kt + (key + 8) * D + (((4 * g + c) ^ sw) << 4));
            const uint32_t x[2][4] = {{w[0].x, w[0].y, w[0].z, w[0].w}, {w[1].x, w[1].y, w[1].z, w[1].w}};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const uint2 lo = e4m3x4_to_f16(x[0][s]), hi = e4m3x4_to_f16(x[1][s]);
              const uint32_t a[4] = {lo.x, hi.x, lo.y, hi.y};
#pragma unroll
              for (int t = 0; t < kNt; ++t) mma_16816<true>(sc[mt][t], a, qb[4 * g + s][t][0], qb[4 * g + s][t][1]);
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < kKs; ++s) {
            const int ch = 2 * s + (lane >> 4);
            uint32_t a[4];
            ldmatrix_x4(ks + k_off[mt] + (ch >> 3) * piece_stride + (((ch & 7) ^ (lane & 7)) << 4), a);
#pragma unroll
            for (int t = 0; t < kNt; ++t) mma_16816<false>(sc[mt][t], a, qb[s][t][0], qb[s][t][1]);
          }
        }
      }
      // online softmax, base 2
      const bool masked = key0 < all_lo || key0 + kKeys > all_hi || there != all_boxes;
      if (masked) {
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int t = 0; t < kNt; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = 16 * mt + r + 8 * (i >> 1);
              const bool on = key0 + key >= klo[t][i & 1] && key0 + key < khi[t][i & 1] &&
                              ((there >> (key >> box_shift)) & 1u);
              if (!on) sc[mt][t][i] = -INFINITY;
            }
      }
      float mx[kNt][2];
      bool raise = false;
#pragma unroll
      for (int t = 0; t < kNt; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = fmaxf(sc[0][t][i], sc[0][t][i + 2]);
#pragma unroll
          for (int mt = 1; mt < kMt; ++mt) x = fmaxf(x, fmaxf(sc[mt][t][i], sc[mt][t][i + 2]));
          mx[t][i] = x * t_scale[t][i];
          raise |= !(mx[t][i] <= m[t][i] + 8.f);  // 2^(t - m) would pass 2^8
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int t = 0; t < kNt; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x = fmaxf(mx[t][i], m[t][i]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float f = x == -INFINITY ? 1.f : ex2(m[t][i] - x);
            m[t][i] = x;
            l[t][i] *= f;
#pragma unroll
            for (int s = 0; s < kKs; ++s) {
              o[s][t][i] *= f;
              o[s][t][i + 2] *= f;
            }
          }
      }
      // P rounded to the cache's operand type (BF16: 2^-8, FP16: 2^-11 relative at most, random over
      // keys; FP16 also 2^-32 of the largest weight), transposed
      uint32_t pb[kMt][kNt][2];
#pragma unroll
      for (int t = 0; t < kNt; ++t) {
        const float b0 = weight_base<kFp8>(m[t][0]), b1 = weight_base<kFp8>(m[t][1]);
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float e0 = ex2(fmaf(sc[mt][t][2 * h], t_scale[t][0], b0));
            const float e1 = ex2(fmaf(sc[mt][t][2 * h + 1], t_scale[t][1], b1));
            l[t][0] += e0;
            l[t][1] += e1;
            pb[mt][t][h] = movmatrix_trans(kFp8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1));
          }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        if constexpr (kFp8) {
          constexpr int kW = D / 32;  // words per lane and key
          uint32_t x[4][kW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 16 * mt + 2 * c + (i & 1) + 8 * (i >> 1);
            if constexpr (D == 128) {
              *reinterpret_cast<uint4*>(x[i]) = *reinterpret_cast<const uint4*>(vt + key * D + ((r ^ (key & 7)) << 4));
            } else {
              *reinterpret_cast<uint2*>(x[i]) = *reinterpret_cast<const uint2*>(
                  vt + key * D + (((r >> 1) ^ ((key >> 1) & 3)) << 4) + 8 * (r & 1));
            }
          }
          // bytes b of a lane's columns: block b / 2, its row r (b even) or r + 8
#pragma unroll
          for (int w = 0; w < kW; ++w) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint2 lo = e4m3x4_to_f16(__byte_perm(x[0][w], x[1][w], h ? 0x7362 : 0x5140));
              const uint2 hi = e4m3x4_to_f16(__byte_perm(x[2][w], x[3][w], h ? 0x7362 : 0x5140));
              const uint32_t a[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
              for (int t = 0; t < kNt; ++t) mma_16816<true>(o[2 * w + h][t], a, pb[mt][t][0], pb[mt][t][1]);
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < kKs; ++s) {
            const int ch = 2 * s + ((lane >> 3) & 1);
            uint32_t a[4];
            ldmatrix_x4_trans(vs + v_off[mt] + (ch >> 3) * piece_stride + (((ch & 7) ^ (lane & 7)) << 4), a);
#pragma unroll
            for (int t = 0; t < kNt; ++t) mma_16816<false>(o[s][t], a, pb[mt][t][0], pb[mt][t][1]);
          }
        }
      }
      fence_proxy_async_smem();  // zeros written above come before the next copy into the stage
      __syncwarp();
      copy_next(st);
      if (++st == kDecStages) {
        st = 0;
        phase ^= 1;
      }
    }
    if (!ok) break;

    // O / l to BF16, or this part of the unit to the workspace.
    const bool whole = begun == 0 && tile + n == u.nt;
    const int64_t slot = 2 * static_cast<int64_t>(worker) + (begun == 0 ? 1 : 0);
    // columns of o[s][t]: E4M3 r D / 8 + 2 s (accumulators 0, 1) and the next (2, 3); BF16 16 s + r and + 8
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 4);
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 8);
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 16);
        const int row = 8 * t + 2 * c + i;
        if (tile > begun) {
          if (row < u.rows) {
            const RunJoin join = join_run(p.part_ml[slot * p.tile_rows + row], m[t][i], l[t][i]);
            const float* src = p.part_o + (slot * p.tile_rows + row) * D + (kFp8 ? r * (D / 8) : r);
#pragma unroll
            for (int s = 0; s < kKs; ++s) {
              o[s][t][i] = fmaf(o[s][t][i], join.own, src[kFp8 ? 2 * s : 16 * s] * join.before);
              o[s][t][i + 2] = fmaf(o[s][t][i + 2], join.own, src[kFp8 ? 2 * s + 1 : 16 * s + 8] * join.before);
            }
          }
          __syncwarp();  // a row's maximum and sum are read by eight lanes, one of which writes them below
        }
        if (whole) {
          const float inv = l[t][i] == 0.f ? 0.f : p.v_scale / l[t][i];
#pragma unroll
          for (int s = 0; s < kKs; ++s) {
            o[s][t][i] *= inv;
            o[s][t][i + 2] *= inv;
          }
        } else if (row < u.rows) {
          float* dst = p.part_o + (slot * p.tile_rows + row) * D;
          if constexpr (kFp8) {
#pragma unroll
            for (int s = 0; s < kKs; s += 2)
              *reinterpret_cast<float4*>(dst + r * (D / 8) + 2 * s) =
                  make_float4(o[s][t][i], o[s][t][i + 2], o[s + 1][t][i], o[s + 1][t][i + 2]);
          } else {
#pragma unroll
            for (int s = 0; s < kKs; ++s) {
              dst[16 * s + r] = o[s][t][i];
              dst[16 * s + 8 + r] = o[s][t][i + 2];
            }
          }
          if (r == 0) p.part_ml[slot * p.tile_rows + row] = make_float2(m[t][i], l[t][i]);
        }
        if (kFp8 && whole && row < u.rows) {
          uint16_t* dst = p.out + row_offset<D>(p, u.s.q0, u.hk, u.r0 + row, p.ldo) + r * (D / 8);
#pragma unroll
          for (int s = 0; s < kKs; s += 4)
            *reinterpret_cast<uint4*>(dst + 2 * s) =
                make_uint4(pack_bf16x2(o[s][t][i], o[s][t][i + 2]), pack_bf16x2(o[s + 1][t][i], o[s + 1][t][i + 2]),
                           pack_bf16x2(o[s + 2][t][i], o[s + 2][t][i + 2]),
                           pack_bf16x2(o[s + 3][t][i], o[s + 3][t][i + 2]));
        }
      }
      if (!kFp8 && whole) {
        // transposed back: lane (r, c) has columns 2 c, 2 c + 1 of row r
        uint16_t* dst = p.out + row_offset<D>(p, u.s.q0, u.hk, u.r0 + min(8 * t + r, u.rows - 1), p.ldo) + 2 * c;
#pragma unroll
        for (int s = 0; s < kKs; ++s) {
          const uint32_t lo = movmatrix_trans(pack_bf16x2(o[s][t][0], o[s][t][1]));
          const uint32_t hi = movmatrix_trans(pack_bf16x2(o[s][t][2], o[s][t][3]));
          if (8 * t + r < u.rows) {
            *reinterpret_cast<uint32_t*>(dst + 16 * s) = lo;
            *reinterpret_cast<uint32_t*>(dst + 16 * s + 8) = hi;
          }
        }
      }
    }
    if (lane == 0 && left == n && begun == 0 && tile + n < u.nt) p.part_units[worker] = part_unit(sh, u, at - tile, true);
    left -= n;
    at += n;
    tile += n;
    if (tile == u.nt) {
      tile = begun = 0;
      if (left > 0) next_unit<kKeys, true>(p, u);
    }
  }
  if (!ok) {
    // a timeout: wait for the copies in flight
    for (int s = 0; s < kDecStages; ++s) mbar_wait_drain(&full[(st + s) % kDecStages], st + s < kDecStages ? phase : phase ^ 1);
  }
}

}  // namespace mxq
