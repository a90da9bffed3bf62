// rope_cache.cuh -- what lies between a QKV projection and the attention: the RMS norm of
// queries and keys, their position rotation, and the append of keys and values to a paged cache.
//
// For a vector x of n values (one head, n = d, or one row of all heads, n = H d):
//   y = w * x / sqrt(mean(x^2) + eps)                             (FP32; w = 1 without weights)
// and for i < rot / 2 of each head, with (c, s) = table[position]:
//   (y_a, y_b) <- (y_a c_i - y_b s_i, y_b c_i + y_a s_i)
// where (a, b) = (i, i + rot / 2) (halves) or (2 i, 2 i + 1) (pairs); values from `rot` on pass.
// The result is rounded once: to BF16, or to the E4M3 cache as E4M3_RNE_satfinite(fl32(y *
// fl32(1 / scale))), the static FP8 quantiser's arithmetic.
//
// Bound by DRAM: 2 bytes read and 2 (or 1) written per value.  A CTA takes every gridDim.x-th token.
// Its first warp finds the tokens' positions and places, 32 at a time, and keeps a ring of
// tokens full in shared memory: one bulk copy each for the Q, K and V row and the rotation table's
// row (some 50 KB have to be on their way per SM; loads into registers left half of that).  The other
// warps read a token's heads from there.  A lane owns 16 values of one head, two 16-byte chunks
// chosen so that both members of every rotated pair are its own (`rot / 2` apart for halves), as
// u[8] and v[8], the pairs' first and second members, on which the packed FP32 operations work.
// cos and sin then depend on the lane alone, the rotation needs no shuffle, and a head's sum of
// squares takes log2(lanes per head) of them.  Instructions are the next bound: some 110 per 16
// values.
#pragma once

#include "gemm_common.cuh"
#include "quantize.cuh"

namespace mxq {

// Threads that compute (and a warp that copies).  Four CTAs per SM at 64 registers, with nothing kept
// on the stack: the cosines stay in registers over a token's heads, the sines are read from shared
// memory again for each (both in registers: 278 us for 32760 x 80 heads with a norm over the row, a
// third of the loads being of spilled registers; so 255 us; both read again 260).  Fewer threads with
// more registers are slower (three CTAs at 80 registers 311 us with all in registers).
constexpr int kRopeMaxThreads = 224;
constexpr int kRopeCtas = 4;
constexpr int kRopeMaxStages = 16;

struct RopeOperand {
  const uint16_t* x;       // [T][ld] BF16; null: operand absent (heads = 0)
  const uint16_t* weight;  // BF16 [d] or [heads * d]; null: no norm
  int64_t ld;
  uint16_t* out;  // [T][ldo] BF16 (queries, and keys outside the cache)
  int64_t ldo;
  int heads;
};

struct RopeParams {
  RopeOperand q, k;
  const uint16_t* v;  // append only: [T][ldv]
  int64_t ldv;
  const float* table;  // [table_rows][rot]: rot / 2 cosines, then rot / 2 sines; null: no rotation
  int64_t table_rows;
  const int32_t* positions;  // null: the row index (or the cache position when appending)
  int64_t T;
  float eps, inv_d, inv_q, inv_k;  // 1 / d, 1 / (heads d)
  int d, rot, lanes;  // lanes: threads per head, the power of two >= d / 16
  bool row_norm;
  int seg_heads;      // heads (of Q, K, V in a row) per blockIdx.y; with row_norm 0: all, or Q, K, V apart (-1)
  int stages, stage_bytes;

  __device__ __forceinline__ uint32_t stage_bytes_of(int heads) const {
    return static_cast<uint32_t>(heads * d * 2 + (table ? rot * 4 : 0));
  }
};

struct AppendParams {
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* block_table;
  void* k_cache;
  void* v_cache;
  int64_t stride_page, stride_token, stride_head;  // elements
  int64_t table_stride;                            // block_table entries per sequence
  int batch, num_pages, page_size;
  float k_inv_scale, v_inv_scale;  // fl32(1 / scale), FP8 only
};

// The sequence whose rows [cu[b], cu[b + 1]) hold row t, or -1 (a row behind the last sequence).
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ cu, int batch, int64_t t) {
  int lo = 0, hi = batch;  // cu[lo] <= t < cu[hi], if any
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return cu[lo] <= t && t < cu[lo + 1] ? lo : -1;
}

// Untiled bulk copy global -> shared, completion counted on `bar` (both addresses 16-byte
// aligned, bytes a multiple of 16).
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem_dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Two chunks of eight BF16 values as pair members: halves, u from the one and v from the other;
// pairs, u the even and v the odd values.
template <bool kPairs>
__device__ __forceinline__ void unpack_members(const uint4& a, const uint4& b, float (&u)[8], float (&v)[8]) {
  const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float lo = __uint_as_float(x[i] << 16), hi = __uint_as_float(x[i] & 0xffff0000u);
    if constexpr (kPairs) {
      u[i] = lo;
      v[i] = hi;
    } else {
      float(&w)[8] = i < 4 ? u : v;
      w[2 * (i & 3)] = lo;
      w[2 * (i & 3) + 1] = hi;
    }
  }
}

// Value i of a chunk pair's chunk (0 or 1), back from the members.
template <bool kPairs>
__device__ __forceinline__ float member(const float (&u)[8], const float (&v)[8], int chunk, int i) {
  if constexpr (kPairs) return i & 1 ? v[4 * chunk + (i >> 1)] : u[4 * chunk + (i >> 1)];
  else return chunk ? v[i] : u[i];
}

__device__ __forceinline__ float2 pair_of(const float (&x)[8], int i) { return make_float2(x[i], x[i + 1]); }
__device__ __forceinline__ void set_pair(float (&x)[8], int i, float2 y) {
  x[i] = y.x;
  x[i + 1] = y.y;
}

__device__ __forceinline__ float sum_squares(const float (&u)[8], const float (&v)[8]) {
  float2 ss = __fmul2_rn(pair_of(u, 0), pair_of(u, 0)), tt = __fmul2_rn(pair_of(v, 0), pair_of(v, 0));
#pragma unroll
  for (int i = 2; i < 8; i += 2) {
    ss = __ffma2_rn(pair_of(u, i), pair_of(u, i), ss);
    tt = __ffma2_rn(pair_of(v, i), pair_of(v, i), tt);
  }
  ss = __fadd2_rn(ss, tt);
  return ss.x + ss.y;
}

template <bool kPairs>
__device__ __forceinline__ uint4 pack_bf16(const float (&u)[8], const float (&v)[8], int chunk) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_bf16x2(member<kPairs>(u, v, chunk, 2 * i), member<kPairs>(u, v, chunk, 2 * i + 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool kPairs>
__device__ __forceinline__ uint2 pack_e4m3(const float (&u)[8], const float (&v)[8], int chunk, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3x2(__fmul_rn(member<kPairs>(u, v, chunk, 2 * i), inv), __fmul_rn(member<kPairs>(u, v, chunk, 2 * i + 1), inv));
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// kCache: 0 queries and keys to BF16 rows, 1 keys and values to a BF16 cache, 2 to an E4M3 cache.
template <int kCache, bool kPairs>
__global__ void __launch_bounds__(kRopeMaxThreads + 32, kRopeCtas) rope_cache_kernel(const RopeParams p, const AppendParams a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kRopeMaxStages], empty[kRopeMaxStages], sums;
  __shared__ int64_t s_slot[kRopeMaxStages];
  __shared__ int s_token[kRopeMaxStages];  // -1: no more
  static_assert(kRopeMaxThreads <= 16 * 32, "a lane per warp's sum");
  __shared__ float s_sum[2][2][kRopeMaxThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warps = static_cast<int>(blockDim.x >> 5) - 1;  // that compute
  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], static_cast<uint32_t>(warps));
    }
    mbar_init(&sums, static_cast<uint32_t>(warps));
    fence_mbar_init();
  }
  griddep_launch_dependents();
  __syncthreads();
  griddep_wait();

  // this block's heads [h0, h1) of the row Q, K, V
  const int heads_qk = p.q.heads + p.k.heads;
  const int heads = heads_qk + (kCache != 0 ? p.k.heads : 0);
  int h0 = 0, h1 = heads;
  if (p.seg_heads > 0) {
    h0 = blockIdx.y * p.seg_heads;
    h1 = min(h0 + p.seg_heads, heads);
  } else if (p.seg_heads < 0) {
    const int first = p.q.heads ? 0 : 1;  // without Q: K, V
    const int o = first + static_cast<int>(blockIdx.y);
    h0 = o == 0 ? 0 : o == 1 ? p.q.heads : heads_qk;
    h1 = o == 0 ? p.q.heads : o == 1 ? heads_qk : heads;
  }

  if (tid < 32) {
    // ------------------------------------------------------------------ copies
    const int qn = max(min(h1, p.q.heads) - h0, 0), kn = max(min(h1, heads_qk) - max(h0, p.q.heads), 0);
    const int vn = h1 - h0 - qn - kn, row = p.d * 2;
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_phase = 0;
    bool ok = true;
    for (int64_t base = blockIdx.x; ok && base < p.T; base += 32 * static_cast<int64_t>(gridDim.x)) {
      const int64_t t = base + lane * static_cast<int64_t>(gridDim.x);
      // position and place of this lane's token
      int64_t pos = t, slot = -1;
      bool on = t < p.T;
      if (on) {
        if constexpr (kCache == 0) {
          if (p.positions) pos = p.positions[t];
        } else {
          const int b = find_sequence(a.cu_q, a.batch, t);
          on = b >= 0;
          if (on) {
            const int64_t first = a.cu_q[b];
            pos = static_cast<int64_t>(a.kv_len[b]) - (a.cu_q[b + 1] - first) + (t - first);
            const int64_t entry = pos < 0 ? a.table_stride : pos / a.page_size;
            on = entry < a.table_stride;  // else no place in the sequence's pages
            if (on) {
              const int page = a.block_table[b * a.table_stride + entry];
              if (page >= 0 && page < a.num_pages)
                slot = page * a.stride_page + (pos - entry * a.page_size) * a.stride_token;
            }
          }
        }
        on = on && !(p.table && (pos < 0 || pos >= p.table_rows));
      }
      for (unsigned left = __ballot_sync(0xffffffffu, on); left; left &= left - 1) {
        const int l = __ffs(left) - 1;
        const int64_t tt = __shfl_sync(0xffffffffu, t, l), tpos = __shfl_sync(0xffffffffu, pos, l);
        const int64_t tslot = __shfl_sync(0xffffffffu, slot, l);
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1));
        if (!ok) break;
        issued |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (lane == 0) {
          s_token[stage] = static_cast<int>(tt);
          s_slot[stage] = tslot;
          mbar_arrive_expect_tx(&full[stage], p.stage_bytes_of(h1 - h0));
        }
        __syncwarp();
        uint8_t* dst = ring + stage * p.stage_bytes;
        if (lane == 0 && qn) bulk_load(dst, p.q.x + tt * p.q.ld + h0 * p.d, qn * row, &full[stage]);
        if (lane == 1 && kn)
          bulk_load(dst + qn * row, p.k.x + tt * p.k.ld + max(h0 - p.q.heads, 0) * p.d, kn * row, &full[stage]);
        if (lane == 2 && vn)
          bulk_load(dst + (qn + kn) * row, p.v + tt * p.ldv + max(h0 - heads_qk, 0) * p.d, vn * row, &full[stage]);
        if (lane == 3 && p.table) bulk_load(dst + (h1 - h0) * row, p.table + tpos * p.rot, p.rot * 4, &full[stage]);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (ok && __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1))) {
      if (lane == 0) {
        s_token[stage] = -1;
        mbar_arrive(&full[stage]);
      }
    } else {
      for (int s = 0; s < p.stages; ++s)
        if (issued & (1u << s)) mbar_wait_drain(&full[s], (issued_phase >> s) & 1u);
    }
    return;
  }

  // -------------------------------------------------------------------- norm and rotation
  const int ct = tid - 32, cwarp = ct >> 5;
  const int j = ct & (p.lanes - 1);  // this lane's place in its head
  const int groups = warps * 32 / p.lanes, g0 = ct / p.lanes;
  const int head_lanes = p.d >> 4, rot_lanes = p.rot >> 4;
  const bool live = j < head_lanes;
  // the lane's two chunks of eight values; whether they rotate (halves: both or none)
  int c0 = j, c1 = j + head_lanes;
  if (!kPairs) {
    c1 = j + rot_lanes;
    if (j >= rot_lanes) {
      c0 = rot_lanes + j;
      c1 = head_lanes + j;
    }
  }
  const bool rot0 = p.table && (kPairs ? 8 * c0 < p.rot : j < rot_lanes);
  const bool rot1 = p.table && (kPairs ? 8 * c1 < p.rot : j < rot_lanes);
  int stage = 0, parity = 0;
  uint32_t phase = 0;
  for (;;) {
    if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase))) break;
    const int t = s_token[stage];
    if (t < 0) break;
    const int64_t slot = s_slot[stage];
    const uint8_t* src = ring + stage * p.stage_bytes;
    auto head = [&](int h) { return reinterpret_cast<const uint4*>(src + (h - h0) * p.d * 2); };

    // One norm over the row: the sums of squares of all heads first.
    float root[2] = {0.f, 0.f};
    if (p.row_norm) {
      for (int h = h0 + g0; h < min(h1, heads_qk); h += groups) {
        if (!live) continue;
        float u[8], v[8];
        unpack_members<kPairs>(head(h)[c0], head(h)[c1], u, v);
        const float ss = sum_squares(u, v);
        if (h < p.q.heads) root[0] += ss;
        else root[1] += ss;
      }
      // Q's sum in the lower half of the warp, K's in the upper
      float x = lane < 16 ? root[0] : root[1];
      x += __shfl_xor_sync(0xffffffffu, lane < 16 ? root[1] : root[0], 16);
#pragma unroll
      for (int m = 8; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
      if ((lane & 15) == 0) s_sum[parity][lane >> 4][cwarp] = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sums);
      if (!__all_sync(0xffffffffu, mbar_wait(&sums, parity))) break;
      x = (lane & 15) < warps ? s_sum[parity][lane >> 4][lane & 15] : 0.f;
#pragma unroll
      for (int m = 8; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
      x = rsqrtf(fmaf(x, lane < 16 ? p.inv_q : p.inv_k, p.eps));
      root[0] = __shfl_sync(0xffffffffu, x, 0);
      root[1] = __shfl_sync(0xffffffffu, x, 16);
      parity ^= 1;  // the next token's sums go elsewhere: these may still be read
    }

    float cs[8];
    if (rot0 || rot1) {
      const float4* row = reinterpret_cast<const float4*>(src + (h1 - h0) * p.d * 2);
      // pairs: four of a chunk; halves: eight of the lane
      const int a0 = kPairs ? c0 : 2 * j, a1 = kPairs ? c1 : 2 * j + 1;
      if (rot0) {
        *reinterpret_cast<float4*>(cs) = row[a0];
      }
      if (rot1) {
        *reinterpret_cast<float4*>(cs + 4) = row[a1];
      }
    }
    // A warp's groups take the same number of steps (the shuffles below are warp-wide).
    for (int base = h0; base < h1; base += groups) {
      const int h = base + g0;
      const bool on = live && h < h1;
      const bool is_v = kCache != 0 && h >= heads_qk;
      const bool is_q = h < p.q.heads;
      const int hh = is_q ? h : is_v ? h - heads_qk : h - p.q.heads;
      float u[8], v[8];
      float r = is_q ? root[0] : root[1];
      if (on) {
        unpack_members<kPairs>(head(h)[c0], head(h)[c1], u, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = v[i] = 0.f;
      }
      if (!p.row_norm) {
        float ss = sum_squares(u, v);
        for (int m = p.lanes >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
      }
      if (!on) continue;
      if (!is_v) {
        const uint16_t* weight = is_q ? p.q.weight : p.k.weight;
        if (weight) {
          const uint4* wt = reinterpret_cast<const uint4*>(weight + (p.row_norm ? hh * p.d : 0));
          float wu[8], wv[8];
          unpack_members<kPairs>(__ldg(wt + c0), __ldg(wt + c1), wu, wv);
          const float2 r2 = make_float2(r, r);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            set_pair(u, i, __fmul2_rn(__fmul2_rn(pair_of(u, i), r2), pair_of(wu, i)));
            set_pair(v, i, __fmul2_rn(__fmul2_rn(pair_of(v, i), r2), pair_of(wv, i)));
          }
        }
        // (read here: the registers do not hold them over the heads)
        const float4* sines = reinterpret_cast<const float4*>(src + (h1 - h0) * p.d * 2) + (p.rot >> 3);
        float sn[8];
        if (rot0) *reinterpret_cast<float4*>(sn) = sines[kPairs ? c0 : 2 * j];
        if (rot1) *reinterpret_cast<float4*>(sn + 4) = sines[kPairs ? c1 : 2 * j + 1];
        auto rotate = [&](int i) {
          const float2 c = pair_of(cs, i), sp = pair_of(sn, i), sm = make_float2(-sp.x, -sp.y);
          const float2 x = pair_of(u, i), y = pair_of(v, i);
          set_pair(u, i, __ffma2_rn(y, sm, __fmul2_rn(x, c)));
          set_pair(v, i, __ffma2_rn(x, sp, __fmul2_rn(y, c)));
        };
        if (rot0) {
          rotate(0);
          rotate(2);
        }
        if (rot1) {
          rotate(4);
          rotate(6);
        }
      }
      if (kCache == 0 || is_q) {
        const RopeOperand& o = is_q ? p.q : p.k;
        uint4* out = reinterpret_cast<uint4*>(o.out + t * o.ldo + hh * p.d);
        out[c0] = pack_bf16<kPairs>(u, v, 0);
        out[c1] = pack_bf16<kPairs>(u, v, 1);
      } else if (slot >= 0) {
        const int64_t at = slot + hh * a.stride_head;
        if constexpr (kCache == 1) {
          uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.v_cache : a.k_cache) + at);
          out[c0] = pack_bf16<kPairs>(u, v, 0);
          out[c1] = pack_bf16<kPairs>(u, v, 1);
        } else {
          uint2* out = reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + at);
          const float inv = is_v ? a.v_inv_scale : a.k_inv_scale;
          out[c0] = pack_e4m3<kPairs>(u, v, 0, inv);
          out[c1] = pack_e4m3<kPairs>(u, v, 1, inv);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[stage]);
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
}

}  // namespace mxq
