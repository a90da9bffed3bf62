// paged_chunk.cuh -- attention of many rows (chunks of new tokens) over a paged cache, on tcgen05.
//
// A unit is up to 256 rows (two halves of 128 TMEM lanes; whole tokens, so 128 / G * G rows of
// each half are used) of one key head, against 128 keys per tile.  Roles:
//   warps 0..7   softmax, a warpgroup per half, one row per thread: scores from TMEM, the running
//                maximum (raised lazily, by more than 8 in base 2, then the accumulator is rescaled
//                in TMEM), 2^x, P back to TMEM over the scores, row sums in FP32; at the end
//                O / l to BF16, or the FP32 part to the workspace.
//   warp 8       TMA: Q of the unit once, then K and V tiles in turn, a box per page (zero fill
//                for pages that are missing or that no row reaches), into a ring.
//   warp 9       MMA: S = Q K^T (128 x 128 x d) and O += P V (P from TMEM, V as the MN-major
//                operand) of the two halves in turn, so that one half's products run under the
//                other half's softmax.
//   warps 10..15 E4M3 cache only: raw tiles to FP16 (which holds E4M3 exactly) in the operand
//                layout, and Q to FP16, scaled per row by a power of two as in the few-row kernel.
// Operands and P are BF16, or FP16 with an E4M3 cache.  Bound by the softmax's instructions and
// the tensor cores, close together.
//
// Every wait is bounded (ptx.cuh); on a timeout the kernel records MXQ_ERR_TIMEOUT, drains
// its own copies and MMAs, releases TMEM and returns.
#pragma once

#include "paged_common.cuh"
#include "attention.cuh"
#include "paged_decode.cuh"

namespace mxq {

constexpr int kChunkKeys = 128;
constexpr int kChunkHalf = 128;  // TMEM lanes of a half
constexpr int kChunkRows = 2 * kChunkHalf;
constexpr int kChunkSoftWarps = 8;
constexpr int kChunkMasks = 8;  // tiles whose page masks are kept: more than the ring is ahead
constexpr int kChunkMinTiles = 2;
constexpr int kChunkEarly = 6;     // of a tile's eight 16-key steps: P V begins when these are there
constexpr int kChunkProducer = 8, kChunkMma = 9, kChunkConv = 10;  // warps
constexpr int kChunkConvWarps = 6;

template <int D, bool kFp8>
struct ChunkShape {
  static constexpr int kThreads = kFp8 ? 512 : 384;
  // registers a thread: at launch, softmax warps, the other warps
  static constexpr int kLaunchRegs = kFp8 ? 128 : 168;
  static constexpr int kSoftRegs = kFp8 ? 168 : 208;
  static constexpr int kCtrlRegs = kFp8 ? 88 : 80;
  static_assert(256 * kSoftRegs + (kThreads - 256) * kCtrlRegs <= kThreads * kLaunchRegs, "register split");
  static constexpr int kPieces = D / 64;                        // 128-byte pieces of a BF16 row
  static constexpr int kPieceBytes = 128 * 128;                 // 128 rows of one piece
  static constexpr int kQBytes = 2 * kPieces * kPieceBytes;
  static constexpr int kTileBytes = kPieces * kPieceBytes;      // K or V, BF16
  static constexpr int kSlots = D == 128 ? (kFp8 ? 4 : 5) : 8;
  static constexpr int kRawKeys = 64;  // a raw slot: half a tile
  static constexpr int kRawBytes = kFp8 ? kRawKeys * D : 0;
  static constexpr int kRawSlots = kFp8 ? (D == 128 ? 3 : 6) : 0;
  static constexpr int kOffTiles = kQBytes;
  static constexpr int kOffRaw = kOffTiles + kSlots * kTileBytes;
  static constexpr int kOffQScale = kOffRaw + kRawSlots * kRawBytes;  // float [2][256], E4M3 only
  static constexpr int kOffBar = kOffQScale + (kFp8 ? 2048 : 0);
  static constexpr int kSmemBytes = 1024 + kOffBar + 512;
  static_assert(kSmemBytes <= 232448 - 512, "shared memory");
};

constexpr uint32_t kChunkTmemCols = 512;
constexpr uint32_t kChunkColS = 0;    // two halves x 128 columns of scores (P in the first 64 of each)
constexpr uint32_t kChunkColO = 256;  // two halves x 128 columns of the accumulator

// kind::f16 descriptors: D FP32, A and B both BF16 or both FP16; M 128, N n; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t chunk_idesc(int n, bool b_mn, bool bf16) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kChunkHalf >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_f16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
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

template <int D, bool kFp8>
__global__ void __launch_bounds__((ChunkShape<D, kFp8>::kThreads), 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const PagedParams p) {
  using S = ChunkShape<D, kFp8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* q_ready = q_full + 1;    // E4M3 only: Q is FP16
  uint64_t* q_empty = q_ready + 1;
  uint64_t* s_full = q_empty + 1;    // [2]
  uint64_t* p_full = s_full + 2;     // [2]
  uint64_t* p_rest = p_full + 2;     // [2]
  uint64_t* o_done = p_rest + 2;     // [2]
  uint64_t* drain = o_done + 2;
  uint64_t* kv_full = drain + 1;     // [kSlots]
  uint64_t* kv_empty = kv_full + S::kSlots;
  uint64_t* raw_full = kv_empty + S::kSlots;  // [kRawSlots]
  uint64_t* raw_empty = raw_full + S::kRawSlots;
  uint32_t* masks = reinterpret_cast<uint32_t*>(raw_empty + S::kRawSlots);  // [kChunkMasks]
  uint32_t* tmem_slot = masks + kChunkMasks;
  float* q_scale = reinterpret_cast<float*>(smem + S::kOffQScale);
  __shared__ ShareScratch scratch;
  auto slot_at = [&](int s) { return smem + S::kOffTiles + s * S::kTileBytes; };
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
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(&kv_full[s], kFp8 ? 2 * kChunkConvWarps : 1);  // the converter's warps, or the copy
      mbar_init(&kv_empty[s], 1);
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
  const Share sh = find_share<kChunkKeys, S::kThreads, 1, kChunkMinTiles, false>(p, scratch);
  if (tid == 0 && sh.count == 0) p.part_units[blockIdx.x] = make_int4(0, 0, 0, 0);
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
      int tile = sh.tile;
      int64_t left = sh.count;
      const int nbox = kChunkKeys / p.page_box, box_shift = 31 - __clz(p.page_box);
      constexpr int kRing = kFp8 ? S::kRawSlots : S::kSlots;
      uint64_t* full = kFp8 ? raw_full : kv_full;
      uint64_t* empty = kFp8 ? raw_empty : kv_empty;
      int slot = 0, units = 0, tiles = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      int64_t batch_at = -1;  // block-table entries [batch_at, +32) of sequence batch_b in the lanes
      int batch_b = -1, entries = -1;
      while (ok && left > 0) {
        const int n = static_cast<int>(min(left, static_cast<int64_t>(u.nt - tile)));
        const int64_t row = static_cast<int64_t>(u.b) * p.table_stride;
        if (!__all_sync(0xffffffffu, mbar_wait(q_empty, (units & 1) ^ 1))) {
          ok = false;
          break;
        }
        const int halves = u.rows > half_rows ? 2 : 1;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, halves * S::kPieces * half_rows * 128);
          for (int t = 0; t < halves; ++t)
            for (int c = 0; c < S::kPieces; ++c)
              tma_load_4d(sQ + (t * S::kPieces + c) * S::kPieceBytes, &tmap_q, 0, c, u.hk * p.G,
                          static_cast<int>(u.s.q0) + u.i0 + t * (half_rows / p.G), q_full);
        }
        __syncwarp();
        ++units;
        for (int k = 0; k < n; ++k, ++tiles) {
          const int key0 = (u.kt0 + tile + k) * kChunkKeys;
          const int box_key = key0 + lane * p.page_box;
          const int64_t entry = box_key / p.page_size;
          const int64_t first = key0 / p.page_size;
          if (batch_b != u.b || batch_at < 0 || first < batch_at || first + nbox > batch_at + 32) {
            batch_b = u.b;
            batch_at = first;
            const int64_t e = first + lane;
            entries = e < p.table_stride ? p.block_table[row + e] : -1;
          }
          const int page = __shfl_sync(0xffffffffu, entries, static_cast<int>(min(entry - batch_at, int64_t(31))));
          const bool need = lane < nbox && box_key < u.hi && box_key + p.page_box > u.lo;
          const bool there = need && page >= 0 && page < p.num_pages;
          // the tile's groups of eight keys (boxes hold whole ones) whose page is there
          const uint32_t mask = __ballot_sync(0xffffffffu, there);
          const uint32_t groups =
              __ballot_sync(0xffffffffu, lane < 16 && ((mask >> ((lane * 8) >> box_shift)) & 1u));
          const int pg = there ? page : -1;  // out of range: the box is filled with zeros
          const int in_page = there ? box_key - static_cast<int>(entry) * p.page_size : 0;
          constexpr int kCopies = kFp8 ? 4 : 2;  // K, V; E4M3: half tiles (page_box divides them)
#pragma unroll
          for (int v = 0; v < kCopies; ++v) {
            if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], phase ^ 1))) {
              ok = false;
              break;
            }
            issued |= 1u << slot;
            issued_phase = (issued_phase & ~(1u << slot)) | (phase << slot);
            if (lane == 0) {
              if (v == 0) masks[tiles & (kChunkMasks - 1)] = groups;
              mbar_arrive_expect_tx(&full[slot], kFp8 ? S::kRawBytes : S::kTileBytes);
            }
            __syncwarp();
            if constexpr (kFp8) {
              const int in_half = lane * p.page_box - (v & 1) * S::kRawKeys;
              if (in_half >= 0 && in_half < S::kRawKeys)
                tma_load_5d(raw_at(slot) + in_half * D, v >> 1 ? &tmap_v : &tmap_k, 0, in_page, 0, u.hk, pg, &full[slot]);
            } else if (lane < nbox) {
#pragma unroll
              for (int c = 0; c < S::kPieces; ++c)
                tma_load_5d(slot_at(slot) + c * S::kPieceBytes + lane * p.page_box * 128, v ? &tmap_v : &tmap_k, 0,
                            in_page, c, u.hk, pg, &full[slot]);
            }
            if (++slot == kRing) {
              slot = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
        }
        if (!ok) break;
        left -= n;
        tile = 0;
        if (left > 0) next_unit<kChunkKeys, false>(p, u);
      }
      if (!ok) {
        if (units) mbar_wait_drain(q_full, (units - 1) & 1);
        for (int s = 0; s < kRing; ++s)
          if (issued & (1u << s)) mbar_wait_drain(&full[s], (issued_phase >> s) & 1u);
      }
    } else if (warp == kChunkMma) {
      // ------------------------------------------------------------------ MMA issuer
      if (elect_one()) {
        Unit u = sh.u;
        int tile = sh.tile;
        int64_t left = sh.count;
        uint32_t units = 0, it[2] = {0, 0};  // tiles issued per half
        int slot = 0;                        // the ring's next tile (K, V, K, V, ...)
        uint32_t phase = 0;
        bool ok = true;
        // descriptors: start addresses (16-byte units) are added to these
        const uint64_t q_desc = smem_desc(smem_u32(sQ), 16, 1024, 2);
        const uint64_t k_desc = smem_desc(smem_u32(smem + S::kOffTiles), 16, 1024, 2);
        const uint64_t v_desc = smem_desc(smem_u32(smem + S::kOffTiles), S::kPieceBytes, 1024, 2);
        auto ring_next = [&](int& at) {  // the next tile's slot, once it is full
          at = slot;
          const bool full = mbar_wait(&kv_full[slot], phase);
          if (++slot == S::kSlots) {
            slot = 0;
            phase ^= 1;
          }
          return full;
        };
        auto issue_qk = [&](int t, int at) {
          const uint64_t a = q_desc + t * (S::kPieces * S::kPieceBytes >> 4), b = k_desc + at * (S::kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * S::kPieceBytes + (kk & 3) * 32) >> 4;
            tc_mma_f16(tmem + kChunkColS + 128 * t, a + off, b + off, chunk_idesc(kChunkKeys, false, !kFp8), kk != 0);
          }
          tc_commit(&s_full[t]);
        };
        auto issue_pv = [&](int t, int at, bool first, int from, int to) {
          const uint64_t b = v_desc + at * (S::kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kChunkKeys / 16; ++kk)
            if (kk >= from && kk < to)
              tc_mma_f16_ts(tmem + kChunkColO + 128 * t, tmem + kChunkColS + 128 * t + kk * 8, b + kk * (2048 >> 4),
                            chunk_idesc(D, true, !kFp8), !(first && kk == 0));
        };
        while (ok && left > 0) {
          const int n = static_cast<int>(min(left, static_cast<int64_t>(u.nt - tile)));
          const int halves = u.rows > half_rows ? 2 : 1;
          int ks, vs, next = 0;
          if (!mbar_wait(kFp8 ? q_ready : q_full, units & 1) || !ring_next(ks)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int t = 0; t < halves; ++t) issue_qk(t, ks);
          tc_commit(&kv_empty[ks]);
          if (n == 1) tc_commit(q_empty);
          for (int k = 0; k < n; ++k) {
            const bool more = k + 1 < n;
            if (!ring_next(vs) || (more && !ring_next(next))) {
              ok = false;
              break;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (t >= halves) break;
              ok = mbar_spin(&p_full[t], it[t] & 1);
              if (!ok) break;
              tc_fence_after();
              issue_pv(t, vs, k == 0, 0, kChunkEarly);
              ok = mbar_spin(&p_rest[t], it[t] & 1);
              if (!ok) break;
              ++it[t];
              tc_fence_after();
              issue_pv(t, vs, false, kChunkEarly, kChunkKeys / 16);
              tc_commit(&o_done[t]);
              if (more) issue_qk(t, next);
            }
            if (!ok) break;
            tc_commit(&kv_empty[vs]);
            if (more) tc_commit(&kv_empty[next]);
            if (k + 2 == n) tc_commit(q_empty);
          }
          if (!ok) break;
          ++units;
          left -= n;
          tile = 0;
          if (left > 0) next_unit<kChunkKeys, false>(p, u);
        }
        if (!ok) {
          tc_commit(drain);
          mbar_wait_drain(drain, 0);
        }
      }
    } else if (kFp8 && warp >= kChunkConv) {
      // ------------------------------------------------------------------ converter
      if constexpr (kFp8) {
        constexpr int kThreadsC = 32 * kChunkConvWarps;
        constexpr int kChunks = D / 16;  // 16-value chunks of a row
        const int ct = tid - 32 * kChunkConv;
        Unit u = sh.u;
        int tile = sh.tile;
        int64_t left = sh.count;
        uint32_t units = 0, raw_phase = 0, slot_phase = 1;
        int rs = 0, ss = 0;
        bool ok = true;
        while (ok && left > 0) {
          const int n = static_cast<int>(min(left, static_cast<int64_t>(u.nt - tile)));
          // Q: 2^-e x row with the row's largest value in [1, 2) 2^e (rows with |e| > 100 as they are);
          // exact for BF16's 8 bits down to 2^-14 of that value
          ok = __all_sync(0xffffffffu, mbar_wait(q_full, units & 1));
          if (!ok) break;
          for (int i = ct; i < min(u.rows, kChunkRows); i += kThreadsC) {
            const int t = i >= half_rows, r = i - t * half_rows;
            uint8_t* row = sQ + t * S::kPieces * S::kPieceBytes + r * 128;
            float big = 0.f;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
              const uint4 w = *reinterpret_cast<const uint4*>(row + (c >> 3) * S::kPieceBytes + (((c & 7) ^ (r & 7)) << 4));
              const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                big = fmaxf(big, fmaxf(fabsf(__uint_as_float(x[j] << 16)), fabsf(__uint_as_float(x[j] & 0xffff0000u))));
            }
            const int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;
            const bool fits = e >= -100 && e <= 100;
            const float down = fits ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 1.f;
            q_scale[(units & 1) * kChunkRows + t * kChunkHalf + r] =
                fits ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : 1.f;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
              uint4* at = reinterpret_cast<uint4*>(row + (c >> 3) * S::kPieceBytes + (((c & 7) ^ (r & 7)) << 4));
              const uint4 w = *at;
              const uint32_t x[4] = {w.x, w.y, w.z, w.w};
              uint32_t h[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                h[j] = pack_f16x2(__uint_as_float(x[j] << 16) * down, __uint_as_float(x[j] & 0xffff0000u) * down);
              *at = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_ready);
          ++units;
          for (int k = 0; k < 4 * n; ++k) {  // half tiles: K, K, V, V
            ok = __all_sync(0xffffffffu, mbar_wait(&raw_full[rs], raw_phase) && mbar_wait(&kv_empty[ss], slot_phase));
            if (!ok) break;
            const int half0 = (k & 1) * S::kRawKeys;
            const int key0 = (u.kt0 + tile + (k >> 2)) * kChunkKeys + half0;
            const bool edge = (k & 2) && (key0 < u.lo || key0 + S::kRawKeys > u.hi);
            const uint8_t* src = raw_at(rs);
            uint8_t* dst = slot_at(ss) + half0 * 128;
            constexpr int kSteps = (S::kRawKeys * kChunks + kThreadsC - 1) / kThreadsC;
            uint4 w[kSteps];
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              const int i = ct + j * kThreadsC, ch = i % kChunks, key = i / kChunks;
              const int sw = D == 128 ? (key & 7) : ((key >> 1) & 3);
              if (key < S::kRawKeys) w[j] = *reinterpret_cast<const uint4*>(src + key * D + ((ch ^ sw) << 4));
              // values of keys that no row of the unit attends may be anything: 0 x NaN is NaN
              if (edge && (key0 + key < u.lo || key0 + key >= u.hi)) w[j] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              const int i = ct + j * kThreadsC, ch = i % kChunks, key = i / kChunks;
              if (key >= S::kRawKeys) break;
              const uint2 a = e4m3x4_to_f16(w[j].x), b = e4m3x4_to_f16(w[j].y), c = e4m3x4_to_f16(w[j].z),
                          d = e4m3x4_to_f16(w[j].w);
              const uint4 v0 = make_uint4(a.x, a.y, b.x, b.y), v1 = make_uint4(c.x, c.y, d.x, d.y);
              const int flip = D == 128 ? ch >> 2 : 0;  // the two pieces' chunks in turn: no bank conflict
              const int c0 = 2 * (ch & 3);
              uint8_t* to = dst + (ch >> 2) * S::kPieceBytes + key * 128;
              *reinterpret_cast<uint4*>(to + (((c0 + flip) ^ (key & 7)) << 4)) = flip ? v1 : v0;
              *reinterpret_cast<uint4*>(to + (((c0 + 1 - flip) ^ (key & 7)) << 4)) = flip ? v0 : v1;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&kv_full[ss]);
              mbar_arrive(&raw_empty[rs]);
            }
            if (++rs == S::kRawSlots) {
              rs = 0;
              raw_phase ^= 1;
            }
            if ((k & 1) && ++ss == S::kSlots) {
              ss = 0;
              slot_phase ^= 1;
            }
          }
          left -= n;
          tile = 0;
          if (ok && left > 0) next_unit<kChunkKeys, false>(p, u);
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
    Unit u = sh.u;
    int tile = sh.tile;
    int64_t left = sh.count, at = sh.begin;
    uint32_t it = 0, units = 0;
    uint32_t g = 0;  // tiles of all units so far
    bool ok = true;
    while (ok && left > 0) {
      const int n = static_cast<int>(min(left, static_cast<int64_t>(u.nt - tile)));
      const int row = t * half_rows + r;  // of the unit
      const bool live = r < half_rows && row < u.rows;
      float m = -INFINITY, l = 0.f;
      if (t == 0 || u.rows > half_rows) {
        const int tok = (u.r0 + min(row, u.rows - 1)) / p.G;
        const int2 kr = key_range(p, u.s, tok, tok);
        float scale = p.scale_log2;
        for (int k = 0; k < n; ++k, ++it) {
          const int key0 = (u.kt0 + tile + k) * kChunkKeys;
          ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], it & 1));
          if (!ok) break;
          tc_fence_after();
          float s[128];
          auto load = [&](int c) { tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c])); };
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
          if (kFp8 && k == 0) scale = p.scale_log2 * q_scale[(units & 1) * kChunkRows + t * kChunkHalf + r];
          const uint32_t there = masks[(g + k) & (kChunkMasks - 1)];
          const bool masked =
              __any_sync(0xffffffffu, key0 < kr.x || key0 + kChunkKeys > kr.y || there != 0xffffu);
          tmem_ld_wait();
          load(2);
          load(3);
          auto arrive = [&](uint64_t* bar) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
          };
          // The weights of scores [64 h, +64), in place, for the maximum m as it is.
          const float2 sc2 = make_float2(scale, scale);
          auto weights = [&](int h) {
            const float base = m == -INFINITY ? 0.f : -m;
            const float2 nb2 = make_float2(base, base);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int j = 64 * h + 2 * i;
              const float2 x = __ffma2_rn(make_float2(s[j], s[j + 1]), sc2, nb2);
              s[j] = ex2(x.x);
              s[j + 1] = ex2(x.y);
            }
          };
          // P rounded to the operand type (BF16: 2^-8 relative at most, FP16: 2^-11), random over the
          // keys, over columns whose scores have been read: 16 weights, 8 columns.
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
            }
            float m4[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              m4[q] = fmax3_nan(s[q], s[q + 4], s[q + 4]);
#pragma unroll
              for (int i = 8 + q; i < 64; i += 8) m4[q] = fmax3_nan(m4[q], s[i], s[i + 4]);
            }
            weights(0);
            tmem_ld_wait();
            if (with_mask) {
              mask(2, there);
              mask(3, there);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int i = 64 + q; i < 128; i += 8) m4[q] = fmax3_nan(m4[q], s[i], s[i + 4]);
            float mx = fmax3_nan(fmax3_nan(m4[0], m4[1], m4[2]), m4[3], m4[3]) * scale;
            if (mx == INFINITY) mx = NAN;
            // raised when it would let P pass 2^8 (and when a score is NaN: then the row's maximum, sum
            // and result are)
            const bool raise = !(mx <= m + 8.f);
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
          if (masked) {
            if (!kFp8 && t == 0 && (key0 < u.lo || key0 + kChunkKeys > u.hi)) {
              // values of keys that no row of the unit attends may be anything: 0 x NaN is NaN
              const uint32_t i = 2 * (g + k) + 1;
              const int sl = static_cast<int>(i % S::kSlots);
              ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[sl], (i / S::kSlots) & 1));
              if (!ok) break;
              if (key0 + r < u.lo || key0 + r >= u.hi) {
#pragma unroll
                for (int c = 0; c < S::kPieces; ++c)
#pragma unroll
                  for (int q = 0; q < 8; ++q)
                    *reinterpret_cast<uint4*>(slot_at(sl) + c * S::kPieceBytes + r * 128 + q * 16) =
                        make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
            }
            tile_pass(true);
          } else {
            tile_pass(false);
          }
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
          const bool whole = tile == 0 && n == u.nt;
          const float inv = l == 0.f ? 0.f : p.v_scale / l;
          const int64_t part_slot = 2 * static_cast<int64_t>(blockIdx.x) + (tile == 0 ? 1 : 0);
          uint16_t* dst = p.out + row_offset<D>(p, u.s.q0, u.hk, u.r0 + (live ? row : 0), p.ldo);
          // parts: [four columns][row], so that a warp's stores are consecutive
          float4* part = reinterpret_cast<float4*>(p.part_o) + part_slot * (D / 4) * kChunkRows + row;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(tO + 32 * c, v);
            tmem_ld_wait();
            if (!live) continue;
            if (whole) {
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
            } else {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                part[(8 * c + q) * kChunkRows] =
                    make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                                __uint_as_float(v[4 * q + 3]));
            }
          }
          if (live && !whole) p.part_ml[part_slot * kChunkRows + row] = make_float2(m, l);
          tc_fence_before();
        }
      }
      if (tid == 0 && left == n)
        p.part_units[blockIdx.x] = part_unit(sh, u, at, tile == 0 && n < u.nt);
      g += n;
      ++units;
      left -= n;
      at += n;
      tile = 0;
      if (ok && left > 0) next_unit<kChunkKeys, false>(p, u);
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
