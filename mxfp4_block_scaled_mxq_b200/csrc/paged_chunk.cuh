// paged_chunk.cuh -- attention of many rows (chunks of new tokens) over a paged cache, on tcgen05.
//
// A unit is up to 256 rows (two halves of 128 TMEM lanes; whole tokens, so 128 / G * G rows of
// each half are used) of one key head, against 128 keys per tile.  Roles:
//   warps 0..7   softmax, a warpgroup per half, one row per thread: scores from TMEM, 2^x against the
//                running maximum (which is raised lazily, by more than 8 in base 2, and then the
//                accumulator is rescaled in TMEM and the weights taken again), P back to TMEM over
//                the scores, row sums in FP32; at the end O / l to BF16, or the FP32 part to the
//                workspace.  (Two threads per row, with an exchange of their maxima, took 364 us
//                where this took 321: 1560 x 9360 rows x keys, 40 heads.)
//   warp 8       takes the CTA's share apart into segments of units, and these into runs, for the others (through shared
//                memory: carried by every thread, a unit's bounds cost the softmax registers); TMA:
//                Q of the unit once, then K and V tiles in turn, a box per page (zero fill for pages
//                that are missing or that no row reaches), into rings.
//   warp 9       MMA: S = Q K^T (128 x 128 x d) and O += P V (P from TMEM, V as the MN-major
//                operand) of the two halves in turn, so that one half's products run under the
//                other half's softmax; P V begins when three quarters of P are there.
//   warps 12..15 E4M3 cache only: V tiles to FP16 (which holds E4M3 exactly), Q to two E4M3 terms.
// E4M3 cache: K is used as it is, by kind::f8f6f4 at twice the rate, with every Q row scaled by a
// power of two and split into two E4M3 terms: four bits each of BF16's eight, in steps of 2^-9 at least where
// the row's largest value is in [2^7, 2^8).  So the split is exact down to 2^-9 of the largest value and off by
// 2^-17 of that at most below; rows whose largest is under 2^-119 count as zeros.  P and V are FP16.
// BF16 cache: everything is BF16.
// The scores and the accumulator of both halves fill TMEM, so a half's next scores wait for its
// P V: its softmax and its products alternate, and their latencies bound the kernel.  Per key tile
// 1.83 us with both halves (d = 128, BF16: 1.36 PFLOP/s; E4M3 2.17 us) against 1.63 (1.84) with one, and
// some 5 (7) us per unit for its first scores and its output, which nothing overlaps.
//
// Every wait is bounded (ptx.cuh); on a timeout the kernel records MXQ_ERR_TIMEOUT, drains
// its own copies and MMAs, releases TMEM and returns.
#pragma once

#include "attention.cuh"
#include "paged_common.cuh"
#include "paged_decode.cuh"

namespace mxq {

constexpr int kChunkKeys = 128;
constexpr int kChunkHalf = 128;  // TMEM lanes of a half
constexpr int kChunkRows = 2 * kChunkHalf;
constexpr int kChunkSoftWarps = 8;
constexpr int kChunkProducer = 8, kChunkMma = 9, kChunkConv = 12;  // warps
constexpr int kChunkConvWarps = 4;
constexpr int kChunkMasks = 8;  // tiles whose page masks are kept: more than the rings are ahead
constexpr int kChunkMinPlaces = 2;
constexpr int kChunkRun = kRunKeys / kChunkKeys;  // tiles
constexpr int kChunkEarly = 6;  // of a tile's eight 16-key steps: P V begins when these are there

template <int D, bool kFp8>
struct ChunkShape {
  static constexpr int kThreads = kFp8 ? 512 : 384;
  // What a unit costs beside its key tiles, in key tiles.  With 0, 1, 2, 3, 4, 6: chunks of 500 to
  // 2048 tokens behind up to 8192 (BF16, 32 / 8 heads) 290, 274, 267, 261, 259, 265 us; a 6001-token prompt
  // (E4M3, 40 / 8 heads), whose first units are short, 575, 522, 479, 441, 437, 445 us.  d = 64, a
  // 6000-token prompt, 32 / 8 heads, with 1 to 5: BF16 260, 252, 259, 262, 268 us, E4M3 305, 281, 285, 288,
  // 293 us (eight of 700 tokens, 16 / 16 heads: 73, 70, 68, 67, 65 us).
  static constexpr int kUnitCost = (kFp8 ? 4 : 3) - (D == 64 ? 1 : 0);
  // registers a thread: at launch, softmax warps, the other warps.  Some values of the softmax and of the converter
  // are kept on the stack for all that (bytes stored / loaded: BF16 96 / 128, d = 64 56 / 76; E4M3 400 / 472,
  // 332 / 404; 2 to 3 % of the L1's cycles in a 6001-token E4M3 prompt).
  static constexpr int kLaunchRegs = kFp8 ? 128 : 168;
  static constexpr int kSoftRegs = kFp8 ? 168 : 216;
  static constexpr int kCtrlRegs = kFp8 ? 88 : 72;
  static_assert(256 * kSoftRegs + (kThreads - 256) * kCtrlRegs <= kThreads * kLaunchRegs, "register split");
  static constexpr int kPieces = D / 64;                    // 128-byte pieces of a 16-bit row
  static constexpr int kPieceBytes = 128 * 128;             // 128 rows of one piece
  static constexpr int kQHalfBytes = kPieces * kPieceBytes;  // a half's Q: 16 bits, or two E4M3 terms
  static constexpr int kVBytes = kPieces * kPieceBytes;     // a V tile as operand
  static constexpr int kKBytes = kFp8 ? kChunkKeys * D : kVBytes;
  static constexpr int kRawBytes = kFp8 ? kChunkKeys * D : 0;  // a V tile as copied
  static constexpr int kKSlots = 3, kVSlots = 2, kRawSlots = kFp8 ? 2 : 0;
  // E4M3: the two terms take the place of the BF16 rows where a row stays in its own bytes
  // (d = 128: 256 = 2 x 128), else a place of their own
  static constexpr bool kSplitApart = kFp8 && D == 64;
  static constexpr int kOffQ = kSplitApart ? 2 * kQHalfBytes : 0;  // Q as operand
  static constexpr int kOffK = 2 * kQHalfBytes + kOffQ;
  static constexpr int kOffV = kOffK + kKSlots * kKBytes;
  static constexpr int kOffRaw = kOffV + kVSlots * kVBytes;
  static constexpr int kOffQScale = kOffRaw + kRawSlots * kRawBytes;
  static constexpr int kOffBar = kOffQScale + (kFp8 ? 2 * kChunkRows * 4 : 0);
  static constexpr int kSmemBytes = 1024 + kOffBar + 512;
  static_assert(kSmemBytes <= 232448 - 1024, "shared memory");
};

// A segment of a unit, or a run of it, as the producer hands it on.
struct ChunkUnit {
  int tiles;  // 0: no more
  int key0;   // of the first tile
  int lo, hi, rows, i0, i1, hk;
  Sequence s;
  int whole, slot;  // the unit is complete with this; else which of the CTA's two slots its part goes to
  int joined;       // there is a part of it in the slot already
};

constexpr uint32_t kChunkTmemCols = 512;
constexpr uint32_t kChunkColS = 0;    // two halves x 128 columns of scores (P in the first 64 of each)
constexpr uint32_t kChunkColO = 256;  // two halves x 128 columns of the accumulator

// Descriptors, D FP32: kind::f16 with A and B both BF16 or both FP16 (kind::f8f6f4 with both
// E4M3 is all zero in those fields, as FP16 is); M 128, N n; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t chunk_idesc(int n, bool b_mn, bool bf16) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kChunkHalf >> 4) << 24);
}

template <bool kFp8>
__device__ __forceinline__ void tc_mma_qk(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  if constexpr (kFp8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A from TMEM.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// max(a, b, c), NaN if any of them is.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// O <- O x own + before x scale for this thread's row of the accumulator; `before`: its part of the run before,
// [d / 4][row][4].  Ahead of the unit's output rather than in it: nearly all units have one run, and take one branch.
template <int D>
__device__ __forceinline__ void join_accumulator(uint32_t taddr, const float* before, float own, float scale, bool live) {
#pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    uint32_t v[16];
    __syncwarp();
    tmem_ld16(taddr + 16 * c, v);
    tmem_ld_wait();
    if (live) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = __float_as_uint(
            fmaf(__uint_as_float(v[i]), own, before[((4 * c + i / 4) * kChunkRows) * 4 + i % 4] * scale));
    }
    __syncwarp();
    tmem_st16(taddr + 16 * c, v);
  }
  tmem_st_wait();
}

template <int D, bool kFp8>
__global__ void __launch_bounds__((ChunkShape<D, kFp8>::kThreads), 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const PagedParams p) {
  using S = ChunkShape<D, kFp8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* q_scale = reinterpret_cast<float*>(smem + S::kOffQScale);  // [unit parity][row], E4M3
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* q_ready = q_full + 1;  // E4M3: Q is split
  uint64_t* q_empty = q_ready + 1;
  uint64_t* s_full = q_empty + 1;  // [2]
  uint64_t* p_full = s_full + 2;   // [2] three quarters of P
  uint64_t* p_rest = p_full + 2;   // [2]
  uint64_t* o_done = p_rest + 2;   // [2]
  uint64_t* drain = o_done + 2;
  uint64_t* unit_full = drain + 1;  // [2]
  uint64_t* unit_empty = unit_full + 2;
  uint64_t* k_full = unit_empty + 2;
  uint64_t* k_empty = k_full + S::kKSlots;
  uint64_t* v_full = k_empty + S::kKSlots;
  uint64_t* v_empty = v_full + S::kVSlots;
  uint64_t* raw_full = v_empty + S::kVSlots;
  uint64_t* raw_empty = raw_full + S::kRawSlots;
  uint32_t* masks = reinterpret_cast<uint32_t*>(raw_empty + S::kRawSlots);  // [kChunkMasks]
  uint32_t* tmem_slot = masks + kChunkMasks;
  __shared__ ShareScratch scratch;
  __shared__ ChunkUnit chunk_units[2];
  auto k_at = [&](int s) { return smem + S::kOffK + s * S::kKBytes; };
  auto v_at = [&](int s) { return smem + S::kOffV + s * S::kVBytes; };
  auto raw_at = [&](int s) { return smem + S::kOffRaw + s * S::kRawBytes; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    mbar_init(q_full, 1);
    mbar_init(q_ready, kChunkConvWarps);
    mbar_init(q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], kChunkSoftWarps / 2);  // one arrival per softmax warp of the half
      mbar_init(&p_rest[t], kChunkSoftWarps / 2);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(drain, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&unit_full[s], 1);
      mbar_init(&unit_empty[s], kChunkSoftWarps + 1 + (kFp8 ? kChunkConvWarps : 0));
    }
    for (int s = 0; s < S::kKSlots; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < S::kVSlots; ++s) {
      mbar_init(&v_full[s], kFp8 ? kChunkConvWarps : 1);  // the converter's warps, or the copy
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < S::kRawSlots; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kChunkConvWarps);
    }
    fence_mbar_init();
  }
  if (warp == kChunkMma) {
    tmem_alloc(tmem_slot, kChunkTmemCols);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  griddep_wait();
  const Share sh = find_share<kChunkKeys, S::kThreads, 1, kChunkMinPlaces, S::kUnitCost, false>(p, scratch);
  if (tid == 0) p.part_units[blockIdx.x] = make_int4(0, 0, 0, 0);  // nothing to join, also after a timeout
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int half_rows = p.tile_rows >> 1;

  if (warp >= kChunkSoftWarps) {
    setmaxnreg_dec<S::kCtrlRegs>();
    if (warp == kChunkProducer) {
      // ------------------------------------------------------------------ TMA producer
      Unit u = sh.u;
      int offset = sh.offset, begun = max(offset - S::kUnitCost, 0);  // the tile at which the CTA began the unit
      int64_t left = sh.count, unit_at = sh.begin - sh.offset;
      const int nbox = kChunkKeys / p.page_box, box_shift = 31 - __clz(p.page_box);
      // rings: 0 K, 1 V (as copied)
      constexpr int kRing1 = kFp8 ? S::kRawSlots : S::kVSlots;
      uint64_t* full1 = kFp8 ? raw_full : v_full;
      uint64_t* empty1 = kFp8 ? raw_empty : v_empty;
      int slot[2] = {0, 0};
      uint32_t phase[2] = {0, 0}, issued[2] = {0, 0}, issued_phase[2] = {0, 0};
      uint32_t units = 0, tiles = 0;
      bool ok = true;
      int batch_at = 0, batch_b = -1, entries = -1;  // block-table entries [batch_at, +32) of sequence batch_b
      while (ok && left > 0) {
        const int tile = max(offset - S::kUnitCost, 0);
        const int end = static_cast<int>(min(left + offset, static_cast<int64_t>(S::kUnitCost + min(u.nt, tile + kChunkRun))));
        const int n = max(end - S::kUnitCost, 0) - tile;
        left -= end - offset;
        if (n == 0) break;  // the share ends before the unit's first key tile
        ok = __all_sync(0xffffffffu, mbar_wait(&unit_empty[units & 1], ((units >> 1) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          ChunkUnit& c = chunk_units[units & 1];
          c.tiles = n;
          c.key0 = (u.kt0 + tile) * kChunkKeys;
          c.lo = u.lo;
          c.hi = u.hi;
          c.rows = u.rows;
          c.i0 = u.i0;
          c.i1 = u.i1;
          c.hk = u.hk;
          c.s = u.s;
          c.whole = begun == 0 && tile + n == u.nt;
          c.slot = begun == 0 ? 1 : 0;
          c.joined = tile > begun;
          mbar_arrive(&unit_full[units & 1]);
          if (left == 0) p.part_units[blockIdx.x] = part_unit(sh, u, unit_at + S::kUnitCost, begun == 0 && tile + n < u.nt);
        }
        // Q: to L2 while the unit before still has its place (1560 tokens over 9360 keys 324 -> 319 us)
        const int halves = u.rows > half_rows ? 2 : 1;
        if (lane == 0 && units > 0)
          for (int t = 0; t < halves; ++t)
            for (int c = 0; c < S::kPieces; ++c)
              tma_prefetch_4d(&tmap_q, 0, c, u.hk * p.G, static_cast<int>(u.s.q0) + u.i0 + t * (half_rows / p.G));
        __syncwarp();
        ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (units & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, halves * S::kPieces * half_rows * 128);
          for (int t = 0; t < halves; ++t)
            for (int c = 0; c < S::kPieces; ++c)
              tma_load_4d(smem + t * S::kQHalfBytes + c * S::kPieceBytes, &tmap_q, 0, c, u.hk * p.G,
                          static_cast<int>(u.s.q0) + u.i0 + t * (half_rows / p.G), q_full);
        }
        __syncwarp();
        ++units;
        for (int k = 0; k < n; ++k, ++tiles) {
          const int key0 = (u.kt0 + tile + k) * kChunkKeys;
          const int first = key0 / p.page_size, box_key = key0 + lane * p.page_box, entry = box_key / p.page_size;
          if (batch_b != u.b || first < batch_at || first + nbox > batch_at + 32) {
            batch_b = u.b;
            batch_at = first;
            entries = first + lane < p.table_stride ? p.block_table[u.b * p.table_stride + first + lane] : -1;
          }
          const int page = __shfl_sync(0xffffffffu, entries, min(entry - batch_at, 31));
          const bool need = lane < nbox && box_key < u.hi && box_key + p.page_box > u.lo;
          const bool there = need && page >= 0 && page < p.num_pages;
          // the tile's groups of eight keys (boxes hold whole ones) whose page is there
          const uint32_t mask = __ballot_sync(0xffffffffu, there);
          const uint32_t groups =
              __ballot_sync(0xffffffffu, lane < 16 && ((mask >> ((lane * 8) >> box_shift)) & 1u));
          const int pg = there ? page : -1;  // out of range: the box is filled with zeros
          const int in_page = there ? box_key - entry * p.page_size : 0;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            uint64_t* full = v ? full1 : k_full;
            uint64_t* empty = v ? empty1 : k_empty;
            const int s = slot[v];
            ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], phase[v] ^ 1));
            if (!ok) break;
            issued[v] |= 1u << s;
            issued_phase[v] = (issued_phase[v] & ~(1u << s)) | (phase[v] << s);
            if (lane == 0) {
              if (v == 0) masks[tiles & (kChunkMasks - 1)] = groups;
              mbar_arrive_expect_tx(&full[s], v ? (kFp8 ? S::kRawBytes : S::kVBytes) : S::kKBytes);
            }
            __syncwarp();
            if (lane < nbox) {
              const CUtensorMap* m = v ? &tmap_v : &tmap_k;
              uint8_t* dst = v ? (kFp8 ? raw_at(s) : v_at(s)) : k_at(s);
              if constexpr (kFp8) {
                tma_load_5d(dst + lane * p.page_box * D, m, 0, in_page, 0, u.hk, pg, &full[s]);
              } else {
#pragma unroll
                for (int c = 0; c < S::kPieces; ++c)
                  tma_load_5d(dst + c * S::kPieceBytes + lane * p.page_box * 128, m, 0, in_page, c, u.hk, pg, &full[s]);
              }
            }
            if (++slot[v] == (v ? kRing1 : S::kKSlots)) {
              slot[v] = 0;
              phase[v] ^= 1;
            }
          }
          if (!ok) break;
        }
        if (!ok) break;
        offset = end;
        if (end == S::kUnitCost + u.nt) {
          unit_at += end;
          offset = begun = 0;
          if (left > 0) next_unit<kChunkKeys, false>(p, u);
        }
      }
      if (ok && __all_sync(0xffffffffu, mbar_wait(&unit_empty[units & 1], ((units >> 1) & 1) ^ 1)) && lane == 0) {
        chunk_units[units & 1].tiles = 0;
        mbar_arrive(&unit_full[units & 1]);
      }
      if (!ok) {
        if (units) mbar_wait_drain(q_full, (units - 1) & 1);
        for (int s = 0; s < S::kKSlots; ++s)
          if (issued[0] & (1u << s)) mbar_wait_drain(&k_full[s], (issued_phase[0] >> s) & 1u);
        for (int s = 0; s < kRing1; ++s)
          if (issued[1] & (1u << s)) mbar_wait_drain(&full1[s], (issued_phase[1] >> s) & 1u);
      }
    } else if (warp == kChunkMma) {
      // ------------------------------------------------------------------ MMA issuer
      if (elect_one()) {
        uint32_t units = 0, it[2] = {0, 0};  // tiles issued per half
        int k_slot = 0, v_slot = 0;
        uint32_t k_phase = 0, v_phase = 0;
        bool ok = true;
        // descriptors: start addresses (16-byte units) are added to these; E4M3 rows of 64 bytes
        // (d = 64) have the 64-byte swizzle
        constexpr uint32_t kLayout = kFp8 && D == 64 ? 4 : 2, kSbo = kFp8 && D == 64 ? 512 : 1024;
        const uint64_t q_desc = smem_desc(smem_u32(smem + S::kOffQ), 16, kSbo, kLayout);
        const uint64_t k_desc = smem_desc(smem_u32(smem + S::kOffK), 16, kSbo, kLayout);
        const uint64_t v_desc = smem_desc(smem_u32(smem + S::kOffV), S::kPieceBytes, 1024, 2);
        auto issue_qk = [&](int t, int at) {
          const uint64_t a = q_desc + t * (S::kQHalfBytes >> 4), b = k_desc + at * (S::kKBytes >> 4);
          const uint32_t d = tmem + kChunkColS + 128 * t;
          if constexpr (kFp8) {
            constexpr int kSteps = D / 32;  // of 32 values; then the second terms of Q
#pragma unroll
            for (int kk = 0; kk < 2 * kSteps; ++kk)
              tc_mma_qk<true>(d, a + ((kk / kSteps * kChunkHalf * D + kk % kSteps * 32) >> 4), b + (kk % kSteps * 32 >> 4),
                              chunk_idesc(kChunkKeys, false, false), kk != 0);
          } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * S::kPieceBytes + (kk & 3) * 32) >> 4;
              tc_mma_qk<false>(d, a + off, b + off, chunk_idesc(kChunkKeys, false, true), kk != 0);
            }
          }
          tc_commit(&s_full[t]);
        };
        // O += P V for the tile's 16-key steps [0, 6), then the rest
        auto issue_pv = [&](int t, int at, bool rest, bool first) {
          const uint64_t b = v_desc + at * (S::kVBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kChunkKeys / 16; ++kk)
            if ((kk >= kChunkEarly) == rest)
              tc_mma_f16_ts(tmem + kChunkColO + 128 * t, tmem + kChunkColS + 128 * t + kk * 8, b + kk * (2048 >> 4),
                            chunk_idesc(D, true, !kFp8), !(first && kk == 0));
        };
        for (;;) {
          ok = mbar_wait(&unit_full[units & 1], (units >> 1) & 1);
          if (!ok) break;
          const int n = chunk_units[units & 1].tiles;
          if (n == 0) break;
          const int halves = chunk_units[units & 1].rows > half_rows ? 2 : 1;
          mbar_arrive(&unit_empty[units & 1]);
          ok = mbar_wait(kFp8 ? q_ready : q_full, units & 1) && mbar_wait(&k_full[k_slot], k_phase);
          if (!ok) break;
          tc_fence_after();
          for (int t = 0; t < halves; ++t) issue_qk(t, k_slot);
          tc_commit(&k_empty[k_slot]);
          if (n == 1) tc_commit(q_empty);
          for (int k = 0; k < n; ++k) {
            const bool more = k + 1 < n;
            if (++k_slot == S::kKSlots) {
              k_slot = 0;
              k_phase ^= 1;
            }
            ok = mbar_wait(&v_full[v_slot], v_phase) && (!more || mbar_wait(&k_full[k_slot], k_phase));
            if (!ok) break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (t >= halves) break;
              ok = mbar_spin(&p_full[t], it[t] & 1);
              if (!ok) break;
              tc_fence_after();
              issue_pv(t, v_slot, false, k == 0);
              ok = mbar_spin(&p_rest[t], it[t] & 1);
              if (!ok) break;
              ++it[t];
              tc_fence_after();
              issue_pv(t, v_slot, true, false);
              tc_commit(&o_done[t]);
              if (more) issue_qk(t, k_slot);
            }
            if (!ok) break;
            tc_commit(&v_empty[v_slot]);
            if (more) tc_commit(&k_empty[k_slot]);
            if (k + 2 == n) tc_commit(q_empty);
            if (++v_slot == S::kVSlots) {
              v_slot = 0;
              v_phase ^= 1;
            }
          }
          if (!ok) break;
          ++units;
        }
        if (!ok) {
          tc_commit(drain);
          mbar_wait_drain(drain, 0);
        }
      }
    } else if (kFp8 && warp >= kChunkConv) {
      // ------------------------------------------------------------------ converter of V
      if constexpr (kFp8) {
        constexpr int kThreadsC = 32 * kChunkConvWarps;
        constexpr int kChunks = D / 16;  // 16-value chunks of a row
        constexpr int kBatch = 4;        // chunks of a thread in flight
        const int ct = tid - 32 * kChunkConv;
        const int ch = ct % kChunks, key_in = ct / kChunks;
        uint32_t raw_phase = 0, v_phase = 1, units = 0;
        int rs = 0, vs = 0;
        for (bool ok = true; ok; ++units) {
          const ChunkUnit& u = chunk_units[units & 1];
          ok = __all_sync(0xffffffffu, mbar_wait(&unit_full[units & 1], (units >> 1) & 1));
          if (!ok) break;
          const int n = u.tiles;
          if (n == 0) break;
          // Q, under the last tile and the end of the unit before: 2^(7 - e) x row with the row's largest
          // value in [1, 2) 2^e, as two E4M3 terms (below 2^-119 zeros; a row with Inf gets a NaN scale, since
          // E4M3 has none).  The scales' slot was read by the softmax two units ago.
          ok = __all_sync(0xffffffffu, mbar_wait(q_full, units & 1));
          if (!ok) break;
#pragma unroll 1
          for (int t = 0; t < (u.rows > half_rows ? 2 : 1); ++t) {
            const int r = ct;  // a thread per row
            const uint8_t* src = smem + t * S::kQHalfBytes + r * 128;
            auto piece = [&](int i) {
              return *reinterpret_cast<const uint4*>(src + (i >> 3) * S::kPieceBytes + (((i & 7) ^ (r & 7)) << 4));
            };
            float big = 0.f;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
              const uint4 w = piece(i);
              const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                big = fmaxf(big, fmaxf(fabsf(__uint_as_float(x[j] << 16)), fabsf(__uint_as_float(x[j] & 0xffff0000u))));
            }
            const int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;
            const bool fits = e >= -119 && e <= 127;
            const float down = fits ? __uint_as_float(static_cast<uint32_t>(134 - e) << 23) : 1.f;
            q_scale[(units & 1) * kChunkRows + t * kChunkHalf + r] =
                fits ? __uint_as_float(static_cast<uint32_t>(120 + e) << 23) : e == 128 ? NAN : 1.f;
            // Rows of D bytes; the first terms' tile, then the second terms'.  In place (d = 128) these go
            // over the row's two pieces: what would go over values not yet read is held back.
            const int sw = D == 128 ? (r & 7) : ((r >> 1) & 3);
            uint8_t* dst = smem + S::kOffQ + t * S::kQHalfBytes + r * D;
            uint4 first[D / 16], held[D == 128 ? 4 : 1];
            auto split = [&](int j) {  // values [16 j, +16): their first terms stay, the second come back
              uint32_t hi[4], lo[4];
              const uint4 w2[2] = {piece(2 * j), piece(2 * j + 1)};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4& ww = w2[k >> 1];
                const uint32_t x0 = k & 1 ? ww.z : ww.x, x1 = k & 1 ? ww.w : ww.y;
                const float f[4] = {__uint_as_float(x0 << 16) * down, __uint_as_float(x0 & 0xffff0000u) * down,
                                    __uint_as_float(x1 << 16) * down, __uint_as_float(x1 & 0xffff0000u) * down};
                hi[k] = e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16);
                const uint2 b = e4m3x4_to_f16(hi[k]);
                const float2 b0 = __half22float2(*reinterpret_cast<const __half2*>(&b.x));
                const float2 b1 = __half22float2(*reinterpret_cast<const __half2*>(&b.y));
                lo[k] = e4m3x2(f[0] - b0.x, f[1] - b0.y) | (e4m3x2(f[2] - b1.x, f[3] - b1.y) << 16);
              }
              first[j] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              return make_uint4(lo[0], lo[1], lo[2], lo[3]);
            };
            auto write = [&](int j, int term, const uint4& w) {
              *reinterpret_cast<uint4*>(dst + term * kChunkHalf * D + ((j ^ sw) << 4)) = w;
            };
            if constexpr (D == 128) {
#pragma unroll
              for (int j = 4; j < 8; ++j) held[j - 4] = split(j);
#pragma unroll
              for (int j = 4; j < 8; ++j) write(j, 1, held[j - 4]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) write(j, 1, split(j));
#pragma unroll
            for (int j = 0; j < D / 16; ++j) write(j, 0, first[j]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_ready);
          for (int k = 0; k < n; ++k) {
            ok = __all_sync(0xffffffffu, mbar_wait(&raw_full[rs], raw_phase) && mbar_wait(&v_empty[vs], v_phase));
            if (!ok) break;
            const int key0 = u.key0 + k * kChunkKeys;
            const bool edge = key0 < u.lo || key0 + kChunkKeys > u.hi;
            const uint8_t* src = raw_at(rs);
            uint8_t* dst = v_at(vs) + (ch >> 2) * S::kPieceBytes;
            const int flip = D == 128 ? ch >> 2 : 0;  // the two pieces' chunks in turn: no bank conflict
            const int c0 = 2 * (ch & 3);
            constexpr int kStep = kThreadsC / kChunks;  // keys per pass
#pragma unroll 1
            for (int i = key_in; i < kChunkKeys; i += kBatch * kStep) {
              uint4 w[kBatch];
#pragma unroll
              for (int j = 0; j < kBatch; ++j) {
                const int key = i + j * kStep, sw = D == 128 ? (key & 7) : ((key >> 1) & 3);
                w[j] = *reinterpret_cast<const uint4*>(src + key * D + ((ch ^ sw) << 4));
                // values of keys that no row of the unit attends may be anything: 0 x NaN is NaN
                if (edge && (key0 + key < u.lo || key0 + key >= u.hi)) w[j] = make_uint4(0, 0, 0, 0);
              }
#pragma unroll
              for (int j = 0; j < kBatch; ++j) {
                const int key = i + j * kStep;
                const uint2 a = e4m3x4_to_f16(w[j].x), b = e4m3x4_to_f16(w[j].y), c = e4m3x4_to_f16(w[j].z),
                            d = e4m3x4_to_f16(w[j].w);
                const uint4 x0 = make_uint4(a.x, a.y, b.x, b.y), x1 = make_uint4(c.x, c.y, d.x, d.y);
                *reinterpret_cast<uint4*>(dst + key * 128 + (((c0 + flip) ^ (key & 7)) << 4)) = flip ? x1 : x0;
                *reinterpret_cast<uint4*>(dst + key * 128 + (((c0 + 1 - flip) ^ (key & 7)) << 4)) = flip ? x0 : x1;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&v_full[vs]);
              mbar_arrive(&raw_empty[rs]);
            }
            if (++rs == S::kRawSlots) {
              rs = 0;
              raw_phase ^= 1;
            }
            if (++vs == S::kVSlots) {
              vs = 0;
              v_phase ^= 1;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&unit_empty[units & 1]);
        }
      }
    }
  } else {
    // -------------------------------------------------------------------- softmax
    setmaxnreg_inc<S::kSoftRegs>();
    const int t = warp >> 2;               // half
    const int r = (warp & 3) * 32 + lane;  // TMEM lane: row of the half
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + kChunkColS + 128 * t, tO = tmem + lane_off + kChunkColO + 128 * t;
    const int row = t * half_rows + r;  // of a unit, whose first row is a token's first
    const int row_tok = row / p.G, row_head = row - row_tok * p.G;
    uint32_t it = 0, units = 0;
    uint32_t g = 0;  // tiles of all units so far
    bool ok = true;
    for (;; ++units) {
      ok = __all_sync(0xffffffffu, mbar_wait(&unit_full[units & 1], (units >> 1) & 1));
      if (!ok) break;
      const ChunkUnit& u = chunk_units[units & 1];
      const int n = u.tiles;
      if (n == 0) break;
      const bool live = r < half_rows && row < u.rows;
      float scale = p.scale_log2;
      // Rows that are not there have the scores of whatever their place in shared memory or in Q holds; with a
      // maximum that nothing passes these never make the others wait (8 x 130 rows over 60000 keys, E4M3,
      // beside rows of NaN that were raised at every tile: 114 us, so 92).
      float m = live ? -INFINITY : INFINITY, l = 0.f;
      if (t == 0 || u.rows > half_rows) {
        const int tok = min(u.i0 + row_tok, u.i1);
        const int2 kr = key_range(p, u.s, tok, tok);
        int key0 = u.key0;
        for (int k = 0; k < n; ++k, ++it, key0 += kChunkKeys) {
          ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], it & 1));
          if (!ok) break;
          tc_fence_after();
          float s[128];
          auto load = [&](int c) { tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c])); };
          if (kFp8 && k == 0) scale = nonzero_scale(scale * q_scale[(units & 1) * kChunkRows + t * kChunkHalf + r]);
          auto mask = [&](int c, uint32_t there) {
            // bit i of on: key 32 c + i is attended
            const int lo = min(max(kr.x - key0 - 32 * c, 0), 32), hi = min(max(kr.y - key0 - 32 * c, 0), 32);
            uint32_t on = hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
            const uint32_t b = there >> (4 * c);  // a group's bit to its eight keys
            on &= ((b & 1u) | ((b & 2u) << 7) | ((b & 4u) << 14) | ((b & 8u) << 21)) * 255u;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((on >> i) & 1u)) s[32 * c + i] = -INFINITY;
          };
          load(0);
          load(1);
          load(2);
          load(3);
          const uint32_t there = masks[(g + k) & (kChunkMasks - 1)];
          const bool masked =
              __any_sync(0xffffffffu, key0 < kr.x || key0 + kChunkKeys > kr.y || there != 0xffffu);
          tmem_ld_wait();
          auto arrive = [&](uint64_t* bar) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
          };
          // The weights of scores [64 h, +64), in place, for the maximum m as it is.
          const float2 sc2 = make_float2(scale, scale);
          auto weights = [&](int h) {
            const float base = weight_base<kFp8>(m);
            const float2 nb2 = make_float2(base, base);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int j = 64 * h + 2 * i;
              const float2 x = __ffma2_rn(make_float2(s[j], s[j + 1]), sc2, nb2);
              s[j] = ex2(x.x);
              s[j + 1] = ex2(x.y);
            }
          };
          // P rounded to the operand type (BF16: 2^-8 relative at most, FP16: 2^-11, and 2^-32 of the
          // largest weight), random over the keys, over columns whose scores have been read: 16 weights, 8 columns.
          auto store = [&](int c) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int j = 16 * c + 2 * i;
              w[i] = kFp8 ? pack_f16x2(s[j], s[j + 1]) : pack_bf16x2(s[j], s[j + 1]);
            }
            tmem_st8(tS + 8 * c, w);
          };
          // The maximum of the tile goes beside the first half's weights, which are taken with the
          // maximum so far: it seldom has to be raised (by more than 8), and then they are taken again.
          auto tile_pass = [&](bool with_mask) {
            if (with_mask) {
              mask(0, there);
              mask(1, there);
              mask(2, there);
              mask(3, there);
            }
            float m4[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              m4[q] = fmax3_nan(s[q], s[q + 4], s[q + 4]);
#pragma unroll
              for (int i = 8 + q; i < 128; i += 8) m4[q] = fmax3_nan(m4[q], s[i], s[i + 4]);
            }
            weights(0);
            float mx = fmax3_nan(fmax3_nan(m4[0], m4[1], m4[2]), m4[3], m4[3]) * scale;
            if (mx == INFINITY) mx = NAN;
            // raised when it would let 2^(t - m) pass 2^8; not for NaN (the weights, the row's sum and its
            // result are NaN either way), nor for a row that is not there
            const bool raise = mx > m + 8.f;
            if (__any_sync(0xffffffffu, raise)) {
              const float f = raise ? ex2(m - mx) : 1.f;
              if (__any_sync(0xffffffffu, raise && m != -INFINITY)) {
                ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (it - 1) & 1));
                if (!ok) return;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                  uint32_t v[32];
                  tmem_ld32(tO + 32 * c, v);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                  tmem_st32(tO + 32 * c, v);
                }
              }
              if (raise) {
                l *= f;
                m = mx;
              }
              load(0);
              load(1);
              tmem_ld_wait();
              if (with_mask) {
                mask(0, there);
                mask(1, there);
              }
              weights(0);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) store(c);
            weights(1);
#pragma unroll
            for (int c = 4; c < 8; ++c) {
              if (c == kChunkEarly) arrive(&p_full[t]);
              store(c);
            }
          };
          if (masked && !kFp8 && t == 0 && (key0 < u.lo || key0 + kChunkKeys > u.hi)) {
            // values of keys that no row of the unit attends may be anything: 0 x NaN is NaN
            const uint32_t i = g + k;
            const int sl = static_cast<int>(i % S::kVSlots);
            ok = __all_sync(0xffffffffu, mbar_wait(&v_full[sl], (i / S::kVSlots) & 1));
            if (!ok) break;
            if (key0 + r < u.lo || key0 + r >= u.hi) {
#pragma unroll
              for (int c = 0; c < S::kPieces; ++c)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  *reinterpret_cast<uint4*>(v_at(sl) + c * S::kPieceBytes + r * 128 + q * 16) =
                      make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          // One copy of the code for BF16, where a small call's time is reading it (18 -> 16 us with 64
          // rows of 64 keys, 1 % more with 1560 over 9360); with fewer registers two (451 -> 431 us, a
          // 6001-token prompt).
          if (kFp8 && !masked) tile_pass(false);
          else tile_pass(masked);
          if (!ok) break;
          arrive(&p_rest[t]);
          // the row sum, while the tensor core has P
          float2 sum[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            sum[q] = make_float2(s[2 * q], s[2 * q + 1]);
#pragma unroll
            for (int i = 8 + 2 * q; i < 128; i += 8) sum[q] = __fadd2_rn(sum[q], make_float2(s[i], s[i + 1]));
          }
          sum[0] = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
          l += sum[0].x + sum[0].y;
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (it - 1) & 1));
        if (ok) {
          tc_fence_after();
          const bool whole = u.whole != 0;
          const int64_t part_slot = 2 * static_cast<int64_t>(blockIdx.x) + u.slot;
          if (u.joined) {
            RunJoin join = {1.f, 0.f};
            if (live) join = join_run(p.part_ml[part_slot * kChunkRows + row], m, l);
            join_accumulator<D>(tO, p.part_o + (part_slot * (D / 4) * kChunkRows + row) * 4, join.own, join.before, live);
          }
          const float inv = l == 0.f ? 0.f : p.v_scale / l;
          uint16_t* dst = p.out + (u.s.q0 + u.i0 + row_tok) * p.ldo + static_cast<int64_t>(u.hk * p.G + row_head) * D;
          // parts: [four columns][row], so that a warp's stores are consecutive
          float4* part = reinterpret_cast<float4*>(p.part_o) + part_slot * (D / 4) * kChunkRows + row;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            __syncwarp();  // rows that are not there have skipped the stores below
            tmem_ld32(tO + 32 * c, v);
            tmem_ld_wait();
            if (live && whole) {
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                w[i] = pack_bf16x2(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
              if (p.out32) {
                st_global_v8(dst + 32 * c, w);
                st_global_v8(dst + 32 * c + 16, w + 8);
              } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  *reinterpret_cast<uint4*>(dst + 32 * c + 8 * q) =
                      make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
              }
            } else if (live) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                part[(8 * c + q) * kChunkRows] =
                    make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                                __uint_as_float(v[4 * q + 3]));
            }
          }
          if (live && !whole) p.part_ml[part_slot * kChunkRows + row] = make_float2(m, l);
          __syncwarp();
          tc_fence_before();
        }
      }
      if (!ok) break;
      g += n;
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_empty[units & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kChunkMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kChunkTmemCols);
  }
}

}  // namespace mxq
