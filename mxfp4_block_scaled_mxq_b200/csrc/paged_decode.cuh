// paged_decode.cuh -- attention of few rows (generated or drafted tokens) over a paged cache.
//
// The cache is read once and little is computed on it, so this kernel is bound by DRAM.  One
// CTA per SM: producer warps keep a ring of key tiles (K and V of kKeys keys, TMA boxes of one
// page each, zero fill for pages that are missing) full in shared memory, up to 180 KB in
// flight, across units; eight consumer warps take the tiles in turn.  Four producer warps, since
// one needs about 1000 cycles for a tile's pages and copies and 16 KB a tile have to come every 700.  A warp holds 16 rows
// and its own running maximum, sum and accumulator, so nothing is exchanged per tile: scores
// by mma.sync m16n8k16 (the rows are too few for a tcgen05 tile of 128), one online-softmax
// step in base 2, then P V with P in registers.  At the end of a unit the eight warps' states
// are joined through shared memory.
//
// BF16 cache: operands by ldmatrix from the 128-byte-swizzled tiles, P rounded to BF16.
// E4M3 cache: K and V are converted to FP16, which holds E4M3 exactly; Q is scaled per row by
// a power of two into FP16 (11 bits, exact for BF16's 8 down to 2^-14 of the row's largest
// value) and P is rounded to FP16.  The order of the head dimension in the
// first product and of the output columns in the second is free, so each lane takes
// contiguous bytes of K rows (16) and V rows (D / 8) and no byte is shuffled across lanes.
#pragma once

#include <cuda_fp16.h>

#include "paged_common.cuh"

namespace mxq {

constexpr int kDecRows = 16;
constexpr int kDecWarps = 8;
constexpr int kDecProducers = 4;
constexpr int kDecThreads = 32 * (kDecWarps + kDecProducers);
constexpr int kDecMaxStages = 24;
constexpr int kDecMinTiles = 4;

template <int D, bool kFp8>
struct DecShape {
  static constexpr int kKeys = kFp8 ? 64 : 32;
  static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
  static constexpr int kTileBytes = kKeys * kRowBytes;  // K or V
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kBoxRowBytes = kRowBytes > 128 ? 128 : kRowBytes;  // one TMA box's row
  static constexpr int kHalves = kRowBytes / kBoxRowBytes;
  static constexpr int kMergeBytes = kDecWarps / 2 * kDecRows * D * 4;
  static constexpr int kMlBytes = 2 * kDecWarps * kDecRows * 8;
  static constexpr int kFixed = 1024 + kMergeBytes + kMlBytes + kDecMaxStages * 20 + 512;
  static constexpr int kFit = (225 * 1024 - kFixed) / kStageBytes;
  // A stage is always filled by the same producer warp and read by the same consumer warp, each in
  // order: a warp that met the stage of another could be two rounds from it, where a barrier's
  // parity says nothing.
  static constexpr int kStages = (kFit < kDecMaxStages ? kFit : kDecMaxStages) / kDecWarps * kDecWarps;
  static constexpr int kOwnStages = kStages / kDecProducers;
  static_assert(kStages >= kDecWarps && kDecWarps % kDecProducers == 0, "stages");
  static constexpr int kSmemBytes = kFixed + kStages * kStageBytes;
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

__device__ __forceinline__ void bar_consumers() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kDecWarps) : "memory");
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kDecThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const PagedParams p) {
  using S = DecShape<D, kFp8>;
  constexpr int kKeys = S::kKeys;
  constexpr int kNt = kKeys / 8;   // score tiles of 8 keys
  constexpr int kKs = D / 16;      // steps of the first product
  constexpr int kOt = D / 8;       // output tiles of 8 columns
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  float* merge = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes);
  float2* ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(merge) + S::kMergeBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ml) + S::kMlBytes);
  uint64_t* empty = full + kDecMaxStages;
  uint32_t* boxes = reinterpret_cast<uint32_t*>(empty + kDecMaxStages);  // per stage: boxes that hold a page
  __shared__ ShareScratch scratch;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    fence_mbar_init();
  }
  griddep_launch_dependents();
  griddep_wait();
  const Share sh = find_share<kKeys, kDecThreads, kDecMinTiles>(p, scratch);  // has the block's barriers
  if (tid == 0 && sh.count == 0) p.part_units[blockIdx.x] = make_int4(0, 0, 0, 0);
  __syncthreads();
  if (sh.count == 0) return;

  if (warp >= kDecWarps) {
    // ------------------------------------------------------------------ producers
    Unit u = sh.u;
    int tile = sh.tile;
    const int nbox = kKeys / p.page_box;
    int own = 0;                  // this warp's next stage among its own
    int turn = warp - kDecWarps;  // tiles until its next one
    uint32_t phase = 0;
    bool ok = true;
    int64_t left = sh.count;
    uint32_t issued = 0, issued_phase = 0;
    int batch_at = -1, batch_b = -1, entries = -1;  // block-table entries [batch_at, +32) of sequence batch_b
    while (ok && left > 0) {
      const int n = static_cast<int>(min(left, static_cast<int64_t>(u.nt - tile)));
      const int32_t* table = p.block_table + static_cast<int64_t>(u.b) * p.table_stride;
      int k = turn;
      for (; k < n; k += kDecProducers) {
        const int stage = (warp - kDecWarps) * S::kOwnStages + own;
        const int key0 = (u.kt0 + tile + k) * kKeys;
        // pages of the tile's boxes: lane i < nbox has box i
        const int box_key = key0 + lane * p.page_box;
        const int first = key0 / p.page_size, entry = box_key / p.page_size;
        if (batch_b != u.b || first < batch_at || first + nbox > batch_at + 32) {
          batch_b = u.b;
          batch_at = first;
          entries = first + lane < p.table_stride ? table[first + lane] : -1;
        }
        const int page = __shfl_sync(0xffffffffu, entries, min(entry - batch_at, 31));
        const bool need = lane < nbox && box_key < u.hi && box_key + p.page_box > u.lo;
        const bool there = need && page >= 0 && page < p.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, there);
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1));
        if (!ok) break;
        issued |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (lane == 0) {
          boxes[stage] = mask;
          mbar_arrive_expect_tx(&full[stage], S::kStageBytes);
        }
        __syncwarp();
        if (lane < nbox) {
          const int pg = there ? page : -1;  // out of range: the box is filled with zeros
          const int in_page = there ? box_key - entry * p.page_size : 0;
          uint8_t* dst = ring + stage * S::kStageBytes + lane * p.page_box * S::kBoxRowBytes;
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h) {
            tma_load_5d(dst + h * kKeys * 128, &tmap_k, 0, in_page, h, u.hk, pg, &full[stage]);
            tma_load_5d(dst + S::kTileBytes + h * kKeys * 128, &tmap_v, 0, in_page, h, u.hk, pg, &full[stage]);
          }
        }
        if (++own == S::kOwnStages) {
          own = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      turn = k - n;
      left -= n;
      tile = 0;
      if (left > 0) next_unit<kKeys>(p, u);
    }
    if (!ok) {
      for (int s = 0; s < S::kStages; ++s)
        if (issued & (1u << s)) mbar_wait_drain(&full[s], (issued_phase >> s) & 1u);
    }
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int r = lane >> 2, c = lane & 3;  // rows r and r + 8; column pair c
  Unit u = sh.u;
  int tile = sh.tile;
  int64_t left = sh.count, at = sh.begin;
  int turn = 0;      // tiles handed out so far, modulo the warps
  int producer = 0;  // of the next tile, and which of its stages
  int own = 0;
  uint32_t phase = 0;
  int parity = 0;
  bool ok = true;  // after a timeout the warps still meet at every barrier below
  while (left > 0) {
    const int n = static_cast<int>(min(left, static_cast<int64_t>(u.nt - tile)));
    // Q fragments of rows r, r + 8, and the keys they attend
    uint32_t qa[kKs][4];
    float t_scale[2];
    int klo[2], khi[2];
    {
      const uint16_t* src[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = u.r0 + min(r + 8 * i, u.rows - 1);
        src[i] = p.q + row_offset<D>(p, u.s.q0, u.hk, row, p.ldq);
        const int2 kr = key_range(p, u.s, row / p.G, row / p.G);
        klo[i] = kr.x;
        khi[i] = kr.y;
        t_scale[i] = p.scale_log2;
      }
      if constexpr (kFp8) {
        uint2 raw[2][kKs];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int s = 0; s < kKs; ++s)
            raw[i][s] = *reinterpret_cast<const uint2*>(src[i] + (s >> 2) * 64 + 16 * c + 4 * (s & 3));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float big = 0.f;
#pragma unroll
          for (int s = 0; s < kKs; ++s) {
            const uint32_t w[2] = {raw[i][s].x, raw[i][s].y};
#pragma unroll
            for (int k = 0; k < 2; ++k)
              big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
          }
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          // 2^-e with the row's largest value in [1, 2) 2^e; rows outside |e| <= 100 are left as they are
          const int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;
          const bool fits = e >= -100 && e <= 100;
          const float down = fits ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 1.f;
          t_scale[i] = fits ? p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : p.scale_log2;
#pragma unroll
          for (int s = 0; s < kKs; ++s) {
            const uint32_t w[2] = {raw[i][s].x, raw[i][s].y};
#pragma unroll
            for (int k = 0; k < 2; ++k)
              qa[s][i + 2 * k] = pack_f16x2(__uint_as_float(w[k] << 16) * down,
                                            __uint_as_float(w[k] & 0xffff0000u) * down);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < kKs; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            qa[s][i] = *reinterpret_cast<const uint32_t*>(src[i] + 16 * s + 2 * c);
            qa[s][i + 2] = *reinterpret_cast<const uint32_t*>(src[i] + 16 * s + 8 + 2 * c);
          }
      }
    }
    // keys that every row of the tile attends
    const int all_lo = key_range(p, u.s, u.i1, u.i1).x, all_hi = key_range(p, u.s, u.i0, u.i0).y;
    const uint32_t all_boxes = (kKeys / p.page_box) == 32 ? 0xffffffffu : (1u << (kKeys / p.page_box)) - 1u;

    float o[kOt][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (int k = 0; k < n; ++k) {
      const bool mine = turn == warp;
      turn = turn + 1 == kDecWarps ? 0 : turn + 1;
      const int st = producer * S::kOwnStages + own;
      const uint32_t ph = phase;
      if (++producer == kDecProducers) {
        producer = 0;
        if (++own == S::kOwnStages) {
          own = 0;
          phase ^= 1;
        }
      }
      if (!mine || !ok) continue;
      ok = __all_sync(0xffffffffu, mbar_wait(&full[st], ph));
      if (!ok) continue;  // timed out: the status word is set and every other wait gives up too
      const int key0 = (u.kt0 + tile + k) * kKeys;
      const uint32_t there = boxes[st];
      uint8_t* kt = ring + st * S::kStageBytes;
      uint8_t* vt = kt + S::kTileBytes;
      const uint32_t ks = smem_u32(kt), vs = smem_u32(vt);
      if (key0 < u.lo || key0 + kKeys > u.hi) {
        // values of keys that no row of the unit attends may be anything: 0 x NaN is NaN
        for (int i = lane; i < kKeys * (S::kRowBytes / 16); i += 32) {
          const int key = i / (S::kRowBytes / 16);
          if (key0 + key < u.lo || key0 + key >= u.hi) {
            const int ch = i % (S::kRowBytes / 16);
            *reinterpret_cast<uint4*>(vt + (ch >> 3) * kKeys * 128 + key * S::kBoxRowBytes + (ch & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
        }
        __syncwarp();
      }
      // S = Q K^T
      float sc[kNt][4];
#pragma unroll
      for (int t = 0; t < kNt; ++t) {
        sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
        if constexpr (kFp8) {
          const int key = 8 * t + r;
#pragma unroll
          for (int g = 0; g < D / 64; ++g) {
            const int sw = D == 128 ? (key & 7) : ((key >> 1) & 3);
            const uint4 w = *reinterpret_cast<const uint4*>(kt + key * D + (((4 * g + c) ^ sw) << 4));
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const uint2 b = e4m3x4_to_f16(x[s]);
              mma_16816<true>(sc[t], qa[4 * g + s], b.x, b.y);
            }
          }
        } else {
          const int key = 8 * t + (lane & 7);
#pragma unroll
          for (int s = 0; s < kKs; s += 2) {
            const int ch = 2 * s + (lane >> 3);
            uint32_t b[4];
            ldmatrix_x4(ks + (ch >> 3) * kKeys * 128 + key * 128 + (((ch & 7) ^ (key & 7)) << 4), b);
            mma_16816<false>(sc[t], qa[s], b[0], b[1]);
            mma_16816<false>(sc[t], qa[s + 1], b[2], b[3]);
          }
        }
      }
      const bool masked = key0 < all_lo || key0 + kKeys > all_hi || there != all_boxes;
#pragma unroll
      for (int t = 0; t < kNt; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[t][i] *= t_scale[i >> 1];
      if (masked) {
#pragma unroll
        for (int t = 0; t < kNt; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 8 * t + 2 * c + (i & 1);
            const bool on = key0 + key >= klo[i >> 1] && key0 + key < khi[i >> 1] &&
                            ((there >> (key / p.page_box)) & 1u);
            if (!on) sc[t][i] = -INFINITY;
          }
      }
      // online softmax, base 2
      float base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = m[i];
#pragma unroll
        for (int t = 0; t < kNt; ++t) mx = fmaxf(mx, fmaxf(sc[t][2 * i], sc[t][2 * i + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        base[i] = mx == -INFINITY ? 0.f : mx;
        const float f = ex2(m[i] - base[i]);
        m[i] = mx;
        l[i] *= f;
#pragma unroll
        for (int t = 0; t < kOt; ++t) {
          o[t][2 * i] *= f;
          o[t][2 * i + 1] *= f;
        }
      }
      uint32_t pa[kNt / 2][4];
#pragma unroll
      for (int t = 0; t < kNt; ++t) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = ex2(sc[t][i] - base[i >> 1]);
        l[0] += e[0] + e[1];
        l[1] += e[2] + e[3];
        // rounding P to the cache's operand type (BF16: 2^-8, FP16: 2^-11 relative, random over keys)
        pa[t >> 1][(t & 1) * 2] = kFp8 ? pack_f16x2(e[0], e[1]) : pack_bf16x2(e[0], e[1]);
        pa[t >> 1][(t & 1) * 2 + 1] = kFp8 ? pack_f16x2(e[2], e[3]) : pack_bf16x2(e[2], e[3]);
      }
      // O += P V
#pragma unroll
      for (int s = 0; s < kNt / 2; ++s) {
        if constexpr (kFp8) {
          constexpr int kW = D / 32;  // words per lane and key
          uint32_t x[4][kW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 16 * s + 2 * c + (i & 1) + 8 * (i >> 1);
            if constexpr (D == 128) {
              *reinterpret_cast<uint4*>(x[i]) = *reinterpret_cast<const uint4*>(vt + key * D + ((r ^ (key & 7)) << 4));
            } else {
              *reinterpret_cast<uint2*>(x[i]) = *reinterpret_cast<const uint2*>(
                  vt + key * D + (((r >> 1) ^ ((key >> 1) & 3)) << 4) + 8 * (r & 1));
            }
          }
#pragma unroll
          for (int w = 0; w < kW; ++w) {
            const uint2 a0 = e4m3x4_to_f16(__byte_perm(x[0][w], x[1][w], 0x5140));
            const uint2 a1 = e4m3x4_to_f16(__byte_perm(x[0][w], x[1][w], 0x7362));
            const uint2 b0 = e4m3x4_to_f16(__byte_perm(x[2][w], x[3][w], 0x5140));
            const uint2 b1 = e4m3x4_to_f16(__byte_perm(x[2][w], x[3][w], 0x7362));
            mma_16816<true>(o[4 * w], pa[s], a0.x, b0.x);
            mma_16816<true>(o[4 * w + 1], pa[s], a0.y, b0.y);
            mma_16816<true>(o[4 * w + 2], pa[s], a1.x, b1.x);
            mma_16816<true>(o[4 * w + 3], pa[s], a1.y, b1.y);
          }
        } else {
          const int key = 16 * s + (lane & 15);
#pragma unroll
          for (int t = 0; t < kOt; t += 2) {
            const int ch = t + (lane >> 4);
            uint32_t b[4];
            ldmatrix_x4_trans(vs + (ch >> 3) * kKeys * 128 + key * 128 + (((ch & 7) ^ (key & 7)) << 4), b);
            mma_16816<false>(o[t], pa[s], b[0], b[1]);
            mma_16816<false>(o[t + 1], pa[s], b[2], b[3]);
          }
        }
      }
      fence_proxy_async_smem();  // zeros written above come before the next copy into the stage
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    // Join the warps: row maxima and sums, then accumulators scaled to the common maximum.
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (c == 0) ml[(parity * kDecWarps + warp) * kDecRows + r + 8 * i] = make_float2(m[i], l[i]);
    }
    bar_consumers();
    const float2* mls = ml + parity * kDecWarps * kDecRows;
    parity ^= 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) top = fmaxf(top, mls[w * kDecRows + r + 8 * i].x);
      const float f = ex2(m[i] - (top == -INFINITY ? 0.f : top));
#pragma unroll
      for (int t = 0; t < kOt; ++t) {
        o[t][2 * i] *= f;
        o[t][2 * i + 1] *= f;
      }
    }
    auto column = [&](int t, int e) { return kFp8 ? (2 * c + e) * kOt + t : 8 * t + 2 * c + e; };
    float* buf = merge + (warp & (kDecWarps / 2 - 1)) * kDecRows * D;
    if (warp >= kDecWarps / 2) {
#pragma unroll
      for (int t = 0; t < kOt; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) buf[(r + 8 * (i >> 1)) * D + column(t, i & 1)] = o[t][i];
    }
    bar_consumers();
    if (warp < kDecWarps / 2) {
#pragma unroll
      for (int t = 0; t < kOt; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) buf[(r + 8 * (i >> 1)) * D + column(t, i & 1)] += o[t][i];
    }
    bar_consumers();
    const bool whole = tile == 0 && n == u.nt;
    if (tid < kDecRows * D / 8) {
      const int row = tid / (D / 8), col = (tid % (D / 8)) * 8;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) top = fmaxf(top, mls[w * kDecRows + row].x);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float2 x = mls[w * kDecRows + row];
        sum += x.y * ex2(x.x - (top == -INFINITY ? 0.f : top));
      }
      float acc[8] = {};
#pragma unroll
      for (int w = 0; w < kDecWarps / 2; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += merge[(w * kDecRows + row) * D + col + i];
      if (row < u.rows) {
        if (whole) {
          const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] *= inv;
          *reinterpret_cast<uint4*>(p.out + row_offset<D>(p, u.s.q0, u.hk, u.r0 + row, p.ldo) + col) =
              make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                         pack_bf16x2(acc[6], acc[7]));
        } else {
          const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (tile == 0 ? 1 : 0);
          float4* dst = reinterpret_cast<float4*>(p.part_o) + (slot * (D / 4) + col / 4) * kDecRows + row;
          dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
          dst[kDecRows] = make_float4(acc[4], acc[5], acc[6], acc[7]);
          if (col == 0) p.part_ml[slot * kDecRows + row] = make_float2(top, sum);
        }
      }
    }
    if (tid == 0 && left == n) {
      int parts = 0;
      if (tile == 0 && n < u.nt) parts = owner(sh, at + u.nt - 1) - static_cast<int>(blockIdx.x) + 1;
      p.part_units[blockIdx.x] = make_int4(static_cast<int>(u.s.q0), u.rt, u.rows, u.hk * 4096 + parts);
    }
    left -= n;
    at += n;
    tile = 0;
    if (left > 0) next_unit<kKeys>(p, u);
  }
}

}  // namespace mxq
