// paged_chunk.cuh -- attention of many rows (chunks of new tokens) over a paged cache, on tcgen05.
//
// A unit is up to 256 rows (two halves of 128 TMEM lanes; whole tokens, so 128 / G * G rows of
// each half are used) of one key head, against 128 keys per tile.  Roles:
//   warps 0..7   softmax, a warpgroup per half, one row per thread: scores from TMEM, running
//                maximum (raised lazily, by more than 8 in base 2, then the accumulator is rescaled
//                in TMEM), 2^x, row sum in FP32, P in BF16 back to TMEM over the scores;
//                at the end O / l to BF16, or the FP32 part to the workspace.
//   warp 8       TMA: Q of the unit once, then K and V tiles in turn, a box per page (zero fill
//                for pages that are missing or that no row reaches), into a ring.
//   warp 9       MMA: S = Q K^T (128 x 128 x d) and O += P V (P from TMEM, V as the MN-major
//                operand) of the two halves in turn, so that one half's products run under the
//                other half's softmax.
//   warps 12..15 E4M3 cache only: raw tiles to BF16 (exactly) into the operand layout.
// Bound by the tensor cores and, close behind, by the 2^x of the softmax.
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
constexpr int kChunkSoftThreads = 256;
constexpr int kChunkMasks = 8;  // tiles whose page masks are kept: more than the ring is ahead
constexpr int kChunkMinTiles = 2;

template <int D, bool kFp8>
struct ChunkShape {
  static constexpr int kThreads = kFp8 ? 512 : 384;
  // registers: the launch's share, and what each warpgroup takes of it (softmax twice)
  static constexpr int kLaunchRegs = kFp8 ? 128 : 168;
  static constexpr int kSoftRegs = kFp8 ? 152 : 200;
  static constexpr int kCtrlRegs = kFp8 ? 104 : 96;
  static constexpr int kConvRegs = 104;
  static_assert(256 * kSoftRegs + 128 * kCtrlRegs + (kFp8 ? 128 * kConvRegs : 0) <= kThreads * kLaunchRegs,
                "register split");
  static constexpr int kPieces = D / 64;                        // 128-byte pieces of a BF16 row
  static constexpr int kPieceBytes = 128 * 128;                 // 128 rows of one piece
  static constexpr int kQBytes = 2 * kPieces * kPieceBytes;
  static constexpr int kTileBytes = kPieces * kPieceBytes;      // K or V, BF16
  static constexpr int kSlots = kFp8 ? 4 : (D == 128 ? 5 : 8);
  static constexpr int kRawBytes = kFp8 ? kChunkKeys * D : 0;
  static constexpr int kRawSlots = kFp8 ? (D == 128 ? 2 : 4) : 0;
  static constexpr int kOffTiles = kQBytes;
  static constexpr int kOffRaw = kOffTiles + kSlots * kTileBytes;
  static constexpr int kOffBar = kOffRaw + kRawSlots * kRawBytes;
  static constexpr int kSmemBytes = 1024 + kOffBar + 512;
  static_assert(kSmemBytes <= 232448 - 512, "shared memory");
};

constexpr uint32_t kChunkTmemCols = 512;
constexpr uint32_t kChunkColS = 0;    // two halves x 128 columns of scores (P in the first 64 of each)
constexpr uint32_t kChunkColO = 256;  // two halves x 128 columns of the accumulator

// kind::f16 descriptors: D FP32, A and B BF16; M 128, N n; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t chunk_idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
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

// Four E4M3 values -> four BF16 values, exactly.
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t w) {
  const uint2 h = e4m3x4_to_f16(w);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
  return make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y));
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
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;    // [2]
  uint64_t* p_full = s_full + 2;     // [2]
  uint64_t* o_done = p_full + 2;     // [2]
  uint64_t* drain = o_done + 2;
  uint64_t* kv_full = drain + 1;     // [kSlots]
  uint64_t* kv_empty = kv_full + S::kSlots;
  uint64_t* raw_full = kv_empty + S::kSlots;  // [kRawSlots]
  uint64_t* raw_empty = raw_full + S::kRawSlots;
  uint32_t* masks = reinterpret_cast<uint32_t*>(raw_empty + S::kRawSlots);  // [kChunkMasks]
  uint32_t* tmem_slot = masks + kChunkMasks;
  __shared__ ShareScratch scratch;
  auto slot_at = [&](int s) { return smem + S::kOffTiles + s * S::kTileBytes; };
  auto raw_at = [&](int s) { return smem + S::kOffRaw + s * S::kRawBytes; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);  // one arrival per softmax warp of the half
      mbar_init(&o_done[t], 1);
    }
    mbar_init(drain, 1);
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(&kv_full[s], kFp8 ? 4 : 1);  // the converter's warps, or the copy
      mbar_init(&kv_empty[s], 1);
    }
    for (int s = 0; s < S::kRawSlots; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, kChunkTmemCols);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  griddep_wait();
  const Share sh = find_share<kChunkKeys, S::kThreads, kChunkMinTiles>(p, scratch);
  if (tid == 0 && sh.count == 0) p.part_units[blockIdx.x] = make_int4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int half_rows = p.tile_rows >> 1;

  if (warp >= 8 && warp < 12) {
    setmaxnreg_dec<S::kCtrlRegs>();
    if (warp == 8) {
      // ------------------------------------------------------------------ TMA producer
      Unit u = sh.u;
      int tile = sh.tile;
      int64_t left = sh.count;
      const int nbox = kChunkKeys / p.page_box;
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
          const uint32_t mask = __ballot_sync(0xffffffffu, there);
          const int pg = there ? page : -1;  // out of range: the box is filled with zeros
          const int in_page = there ? box_key - static_cast<int>(entry) * p.page_size : 0;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], phase ^ 1))) {
              ok = false;
              break;
            }
            issued |= 1u << slot;
            issued_phase = (issued_phase & ~(1u << slot)) | (phase << slot);
            if (lane == 0) {
              if (v == 0) masks[tiles & (kChunkMasks - 1)] = mask;
              mbar_arrive_expect_tx(&full[slot], kFp8 ? S::kRawBytes : S::kTileBytes);
            }
            __syncwarp();
            if (lane < nbox) {
              const CUtensorMap* m = v ? &tmap_v : &tmap_k;
              if constexpr (kFp8) {
                tma_load_5d(raw_at(slot) + lane * p.page_box * D, m, 0, in_page, 0, u.hk, pg, &full[slot]);
              } else {
#pragma unroll
                for (int c = 0; c < S::kPieces; ++c)
                  tma_load_5d(slot_at(slot) + c * S::kPieceBytes + lane * p.page_box * 128, m, 0, in_page, c, u.hk, pg,
                              &full[slot]);
              }
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
        if (left > 0) next_unit<kChunkKeys>(p, u);
      }
      if (!ok) {
        if (units) mbar_wait_drain(q_full, (units - 1) & 1);
        for (int s = 0; s < kRing; ++s)
          if (issued & (1u << s)) mbar_wait_drain(&full[s], (issued_phase >> s) & 1u);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------------ MMA issuer
      if (elect_one()) {
        Unit u = sh.u;
        int tile = sh.tile;
        int64_t left = sh.count;
        int units = 0;
        uint32_t it[2] = {0, 0};  // tiles issued per half
        int64_t seq = 0;          // tiles consumed from the ring (K, V, K, V, ...)
        bool ok = true;
        auto ring_slot = [&](int64_t i) { return static_cast<int>(i % S::kSlots); };
        auto ring_wait = [&](int64_t i) { return mbar_wait(&kv_full[ring_slot(i)], (i / S::kSlots) & 1); };
        auto issue_qk = [&](int t, int64_t i) {
          const uint32_t a = smem_u32(sQ) + t * S::kPieces * S::kPieceBytes, b = smem_u32(slot_at(ring_slot(i)));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * S::kPieceBytes + (kk & 3) * 32;
            tc_mma_f16(tmem + kChunkColS + 128 * t, smem_desc(a + off, 16, 1024, 2), smem_desc(b + off, 16, 1024, 2),
                       chunk_idesc(kChunkKeys, false), kk != 0);
          }
          tc_commit(&s_full[t]);
        };
        auto issue_pv = [&](int t, int64_t i, bool first) {
          const uint32_t b = smem_u32(slot_at(ring_slot(i)));
#pragma unroll
          for (int kk = 0; kk < kChunkKeys / 16; ++kk)
            tc_mma_f16_ts(tmem + kChunkColO + 128 * t, tmem + kChunkColS + 128 * t + kk * 8,
                          smem_desc(b + kk * 2048, S::kPieceBytes, 1024, 2), chunk_idesc(D, true), !(first && kk == 0));
          tc_commit(&o_done[t]);
        };
        while (ok && left > 0) {
          const int n = static_cast<int>(min(left, static_cast<int64_t>(u.nt - tile)));
          const int halves = u.rows > half_rows ? 2 : 1;
          if (!mbar_wait(q_full, units & 1) || !ring_wait(seq)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int t = 0; t < halves; ++t) issue_qk(t, seq);
          tc_commit(&kv_empty[ring_slot(seq)]);
          if (n == 1) tc_commit(q_empty);
          for (int k = 0; k < n; ++k) {
            const bool more = k + 1 < n;
            if (!ring_wait(seq + 1) || (more && !ring_wait(seq + 2))) {
              ok = false;
              break;
            }
            tc_fence_after();
            for (int t = 0; t < halves; ++t) {
              if (!mbar_wait(&p_full[t], it[t] & 1)) {
                ok = false;
                break;
              }
              ++it[t];
              tc_fence_after();
              issue_pv(t, seq + 1, k == 0);
              if (more) issue_qk(t, seq + 2);
            }
            if (!ok) break;
            tc_commit(&kv_empty[ring_slot(seq + 1)]);
            if (more) tc_commit(&kv_empty[ring_slot(seq + 2)]);
            if (k + 2 == n) tc_commit(q_empty);
            seq += 2;
          }
          if (!ok) break;
          ++units;
          left -= n;
          tile = 0;
          if (left > 0) next_unit<kChunkKeys>(p, u);
        }
        if (!ok) {
          tc_commit(drain);
          mbar_wait_drain(drain, 0);
        }
      }
    }
  } else if (kFp8 && warp >= 12) {
    // -------------------------------------------------------------------- converter
    setmaxnreg_dec<S::kConvRegs>();
    if constexpr (kFp8) {
      constexpr int kChunks = D / 16;             // 16-value chunks of a row
      constexpr int kKeysPerStep = 128 / kChunks;  // keys per pass of the warpgroup
      const int ct = tid - 384;
      const int ch = ct % kChunks, kb = ct / kChunks;
      Unit u = sh.u;
      int tile = sh.tile;
      int64_t left = sh.count, seq = 0;
      bool ok = true;
      while (ok && left > 0) {
        const int n = static_cast<int>(min(left, static_cast<int64_t>(u.nt - tile)));
        for (int k = 0; ok && k < 2 * n; ++k, ++seq) {
          const int rs = static_cast<int>(seq % S::kRawSlots), ss = static_cast<int>(seq % S::kSlots);
          ok = __all_sync(0xffffffffu, mbar_wait(&raw_full[rs], (seq / S::kRawSlots) & 1) &&
                                           mbar_wait(&kv_empty[ss], ((seq / S::kSlots) & 1) ^ 1));
          if (!ok) break;
          const int key0 = (u.kt0 + tile + (k >> 1)) * kChunkKeys;
          const bool edge = (k & 1) && (key0 < u.lo || key0 + kChunkKeys > u.hi);
          const uint8_t* src = raw_at(rs);
          uint8_t* dst = slot_at(ss) + (ch >> 2) * S::kPieceBytes;
          const int flip = D == 128 ? ch >> 2 : 0;  // the two pieces' chunks in turn: no bank conflict
#pragma unroll 4
          for (int i = 0; i < 128 / kKeysPerStep; ++i) {
            const int key = kb + i * kKeysPerStep;
            const int sw = D == 128 ? (key & 7) : ((key >> 1) & 3);
            uint4 w = *reinterpret_cast<const uint4*>(src + key * D + ((ch ^ sw) << 4));
            // values of keys that no row of the unit attends may be anything: 0 x NaN is NaN
            if (edge && (key0 + key < u.lo || key0 + key >= u.hi)) w = make_uint4(0, 0, 0, 0);
            const uint2 a = e4m3x4_to_bf16(w.x), b = e4m3x4_to_bf16(w.y), c = e4m3x4_to_bf16(w.z), d = e4m3x4_to_bf16(w.w);
            const uint4 v0 = make_uint4(a.x, a.y, b.x, b.y), v1 = make_uint4(c.x, c.y, d.x, d.y);
            const int c0 = 2 * (ch & 3);
            *reinterpret_cast<uint4*>(dst + key * 128 + (((c0 + flip) ^ (key & 7)) << 4)) = flip ? v1 : v0;
            *reinterpret_cast<uint4*>(dst + key * 128 + (((c0 + 1 - flip) ^ (key & 7)) << 4)) = flip ? v0 : v1;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&kv_full[ss]);
            mbar_arrive(&raw_empty[rs]);
          }
        }
        left -= n;
        tile = 0;
        if (ok && left > 0) next_unit<kChunkKeys>(p, u);
      }
    }
  } else {
    // -------------------------------------------------------------------- softmax
    setmaxnreg_inc<S::kSoftRegs>();
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // TMEM lane: row of the half
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + kChunkColS + 128 * t, tO = tmem + lane_off + kChunkColO + 128 * t;
    const int box_shift = 31 - __clz(p.page_box);
    const uint32_t all_boxes = (1u << (kChunkKeys / p.page_box)) - 1u;
    Unit u = sh.u;
    int tile = sh.tile;
    int64_t left = sh.count, at = sh.begin;
    uint32_t it = 0;
    int64_t g = 0;  // tiles of all units so far
    bool ok = true;
    while (ok && left > 0) {
      const int n = static_cast<int>(min(left, static_cast<int64_t>(u.nt - tile)));
      const int row = t * half_rows + r;  // of the unit
      const bool live = r < half_rows && row < u.rows;
      float m = -INFINITY, l = 0.f;
      if (t == 0 || u.rows > half_rows) {
        const int tok = (u.r0 + min(row, u.rows - 1)) / p.G;
        const int2 kr = key_range(p, u.s, tok, tok);
        for (int k = 0; k < n; ++k, ++it) {
          const int key0 = (u.kt0 + tile + k) * kChunkKeys;
          if (!__all_sync(0xffffffffu, mbar_wait(&s_full[t], it & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t there = masks[(g + k) & (kChunkMasks - 1)];
          const bool masked =
              __any_sync(0xffffffffu, key0 < kr.x || key0 + kChunkKeys > kr.y || there != all_boxes);
          const int lo = kr.x - key0, hi = kr.y - key0;
          // The scores are read twice, 32 columns at a time with the next 32 on their way: TMEM
          // has the bandwidth, and 128 live values a thread would not leave registers for it.
          auto over_scores = [&](auto&& use) {
            float v[2][32];
            tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(v[0]));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              tmem_ld_wait();
              if (c < 3) tmem_ld32(tS + 32 * (c + 1), *reinterpret_cast<uint32_t(*)[32]>(v[(c + 1) & 1]));
              float(&s)[32] = v[c & 1];
              if (masked) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (32 * c + i < lo || 32 * c + i >= hi || !((there >> ((32 * c + i) >> box_shift)) & 1u))
                    s[i] = -INFINITY;
              }
              use(c, s);
            }
          };
          if (!kFp8 && t == 0 && (key0 < u.lo || key0 + kChunkKeys > u.hi)) {
            // values of keys that no row of the unit attends may be anything: 0 x NaN is NaN
            const int64_t i = 2 * (g + k) + 1;
            const int sl = static_cast<int>(i % S::kSlots);
            if (!__all_sync(0xffffffffu, mbar_wait(&kv_full[sl], (i / S::kSlots) & 1))) {
              ok = false;
              break;
            }
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
          float mx = -INFINITY;
          over_scores([&](int, const float(&s)[32]) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx = fmax3(mx, s[i], s[i + 1]);
          });
          mx *= p.scale_log2;
          // the maximum is raised when it would let P pass 2^8; rows without keys so far have none
          const bool raise = mx > m + 8.f || (m == -INFINITY && mx > -INFINITY);
          const float f = raise ? ex2(m - mx) : 1.f;
          if (__any_sync(0xffffffffu, raise && m > -INFINITY)) {
            if (!__all_sync(0xffffffffu, mbar_wait(&o_done[t], (it - 1) & 1))) {
              ok = false;
              break;
            }
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
          const float base = m == -INFINITY ? 0.f : -m;
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nb2 = make_float2(base, base);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          over_scores([&](int c, const float(&s)[32]) {
            uint32_t w[16];  // over columns whose scores have been read
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), sc2, nb2);
              const float2 e = make_float2(ex2(x.x), ex2(x.y));
              sum[i & 1] = __fadd2_rn(sum[i & 1], e);
              // P rounded to the operand type: 2^-8 relative at most, random over the keys
              w[i] = pack_bf16x2(e.x, e.y);
            }
            tmem_st16(tS + 16 * c, w);
          });
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[t]);
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (it - 1) & 1));
        if (ok) {
          tc_fence_after();
          const bool whole = tile == 0 && n == u.nt;
          const float inv = l == 0.f ? 0.f : p.v_scale / l;
          const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (tile == 0 ? 1 : 0)) * kChunkRows + row;
          uint16_t* dst = p.out + row_offset<D>(p, u.s.q0, u.hk, u.r0 + (live ? row : 0), p.ldo);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(tO + 32 * c, v);
            tmem_ld_wait();
            if (!live) continue;
            if (whole) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  w[i] = pack_bf16x2(__uint_as_float(v[8 * q + 2 * i]) * inv, __uint_as_float(v[8 * q + 2 * i + 1]) * inv);
                *reinterpret_cast<uint4*>(dst + 32 * c + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(p.part_o + slot * D + 32 * c + 4 * q) =
                    make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
          }
          if (live && !whole) p.part_ml[slot] = make_float2(m, l);
          tc_fence_before();
        }
      }
      if (tid == 0 && left == n) {
        int parts = 0;
        if (tile == 0 && n < u.nt) parts = owner(sh, at + u.nt - 1) - static_cast<int>(blockIdx.x) + 1;
        p.part_units[blockIdx.x] = make_int4(static_cast<int>(u.s.q0), u.rt, u.rows, u.hk * 4096 + parts);
      }
      g += n;
      left -= n;
      at += n;
      tile = 0;
      if (ok && left > 0) next_unit<kChunkKeys>(p, u);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kChunkTmemCols);
  }
}

}  // namespace mxq
