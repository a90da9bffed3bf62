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
// One CTA per token.  A lane owns 16 values of one head, chosen so that both members of every
// rotated pair are its own: two 16-byte chunks, `rot / 2` apart (halves) or adjacent (pairs and
// the values that pass).  cos and sin then depend on the lane alone and stay in registers over
// the token's heads, the rotation needs no shuffle, and a head's sum of squares takes
// log2(lanes per head) of them.  Bound by DRAM: 2 bytes read and 2 (or 1) written per value.
#pragma once

#include "gemm_common.cuh"
#include "quantize.cuh"

namespace mxq {

constexpr int kRopeMaxThreads = 512;

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
  float eps;
  int d, rot, lanes;  // lanes: threads per head, the power of two >= d / 16
  bool pairs, row_norm;
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

// The sequence whose rows [cu[b], cu[b + 1]) hold row t, or -1 (a row behind the last sequence):
// a 32-way search by one warp, two rounds for up to 1024 sequences.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ cu, int batch, int64_t t, int lane) {
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, i < n && cu[lo + i] <= t);
    const int h = le ? 31 - __clz(le) : 0;
    lo += h * step;
    n = min(step, n - h * step);
  }
  return cu[lo] <= t && t < cu[lo + 1] ? lo : -1;
}

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8_bf16(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ uint2 pack8_e4m3(const float* f, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = e4m3x2(__fmul_rn(f[2 * i], inv), __fmul_rn(f[2 * i + 1], inv));
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// kCache: 0 queries and keys to BF16 rows, 1 keys and values to a BF16 cache, 2 to an E4M3 cache.
template <int kCache>
__global__ void __launch_bounds__(kRopeMaxThreads) rope_cache_kernel(const RopeParams p, const AppendParams a) {
  __shared__ float s_sum[2][kRopeMaxThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int j = threadIdx.x & (p.lanes - 1);  // this lane's place in its head
  const int groups = blockDim.x / p.lanes;
  const bool live = 16 * j < p.d;
  const int rot_lanes = p.rot >> 4;
  // first and second chunk of eight values within the head
  int c0 = 2 * j, c1 = 2 * j + 1;
  if (!p.pairs && j < rot_lanes) {
    c0 = j;
    c1 = j + rot_lanes;
  }

  // Position of the token, and its place in the cache.
  int64_t pos = p.positions ? p.positions[t] : t;
  int64_t slot = -1;  // element offset of the token in the cache
  if constexpr (kCache != 0) {
    const int b = find_sequence(a.cu_q, a.batch, t, lane);
    if (b < 0) return;
    const int64_t first = a.cu_q[b];
    pos = static_cast<int64_t>(a.kv_len[b]) - (a.cu_q[b + 1] - first) + (t - first);
    const int64_t entry = pos < 0 ? a.table_stride : pos / a.page_size;
    if (entry >= a.table_stride) return;  // no place in the sequence's pages
    const int page = a.block_table[b * a.table_stride + entry];
    if (page >= 0 && page < a.num_pages)
      slot = page * a.stride_page + (pos - entry * a.page_size) * a.stride_token;
  }
  if (p.table && (pos < 0 || pos >= p.table_rows)) return;

  float cs[8], sn[8];
  const bool rotate = p.table && j < rot_lanes;
  if (rotate) {
    const float* row = p.table + pos * p.rot + 8 * j;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<float4*>(cs + 4 * i) = __ldg(reinterpret_cast<const float4*>(row) + i);
      *reinterpret_cast<float4*>(sn + 4 * i) = __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1)) + i);
    }
  }

  const int heads_qk = p.q.heads + p.k.heads;
  const int heads = heads_qk + (kCache != 0 ? p.k.heads : 0);
  const int g0 = threadIdx.x / p.lanes;

  // One norm over the row: the sums of squares first (the second read comes from L1 / L2).
  float row_ss[2] = {0.f, 0.f};
  if (p.row_norm) {
    for (int h = g0; h < heads_qk; h += groups) {
      const bool is_q = h < p.q.heads;
      const RopeOperand& o = is_q ? p.q : p.k;
      if (!live || !o.weight) continue;
      const uint16_t* x = o.x + t * o.ld + static_cast<int64_t>(is_q ? h : h - p.q.heads) * p.d;
      float f[16];
      unpack8(*reinterpret_cast<const uint4*>(x + 8 * c0), f);
      unpack8(*reinterpret_cast<const uint4*>(x + 8 * c1), f + 8);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
      if (is_q) row_ss[0] += ss;
      else row_ss[1] += ss;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) row_ss[i] += __shfl_xor_sync(0xffffffffu, row_ss[i], m);
      if (lane == 0) s_sum[i][threadIdx.x >> 5] = row_ss[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      row_ss[i] = 0.f;
      for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) row_ss[i] += s_sum[i][w];
    }
  }

  // A warp's groups take the same number of steps (the shuffles below are warp-wide).
  for (int base = 0; base < heads; base += groups) {
    const int h = base + g0;
    const bool on = live && h < heads;
    const bool is_v = kCache != 0 && h >= heads_qk;
    const bool is_q = h < p.q.heads;
    const RopeOperand& o = is_q ? p.q : p.k;
    const int hh = is_q ? h : is_v ? h - heads_qk : h - p.q.heads;
    float f[16];
    if (on) {
      const uint16_t* x = (is_v ? p.v + t * p.ldv : o.x + t * o.ld) + static_cast<int64_t>(hh) * p.d;
      unpack8(*reinterpret_cast<const uint4*>(x + 8 * c0), f);
      unpack8(*reinterpret_cast<const uint4*>(x + 8 * c1), f + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
    if (!p.row_norm) {
      for (int m = p.lanes >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    }
    if (!on) continue;
    if (!is_v) {
      if (o.weight) {
        const float mean = p.row_norm ? (is_q ? row_ss[0] : row_ss[1]) / static_cast<float>(o.heads * p.d)
                                      : ss / static_cast<float>(p.d);
        const float r = 1.0f / sqrtf(mean + p.eps);
        const uint16_t* wt = o.weight + (p.row_norm ? hh * p.d : 0);
        float w[16];
        unpack8(__ldg(reinterpret_cast<const uint4*>(wt + 8 * c0)), w);
        unpack8(__ldg(reinterpret_cast<const uint4*>(wt + 8 * c1)), w + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = f[i] * r * w[i];
      }
      if (rotate) {
        if (p.pairs) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float u = f[2 * i], v = f[2 * i + 1];
            f[2 * i] = u * cs[i] - v * sn[i];
            f[2 * i + 1] = v * cs[i] + u * sn[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float u = f[i], v = f[8 + i];
            f[i] = u * cs[i] - v * sn[i];
            f[8 + i] = v * cs[i] + u * sn[i];
          }
        }
      }
    }
    if (kCache == 0 || is_q) {
      uint16_t* out = o.out + t * o.ldo + static_cast<int64_t>(hh) * p.d;
      *reinterpret_cast<uint4*>(out + 8 * c0) = pack8_bf16(f);
      *reinterpret_cast<uint4*>(out + 8 * c1) = pack8_bf16(f + 8);
    } else if (slot >= 0) {
      const int64_t at = slot + hh * a.stride_head;
      if constexpr (kCache == 1) {
        uint16_t* out = static_cast<uint16_t*>(is_v ? a.v_cache : a.k_cache) + at;
        *reinterpret_cast<uint4*>(out + 8 * c0) = pack8_bf16(f);
        *reinterpret_cast<uint4*>(out + 8 * c1) = pack8_bf16(f + 8);
      } else {
        uint8_t* out = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + at;
        const float inv = is_v ? a.v_inv_scale : a.k_inv_scale;
        *reinterpret_cast<uint2*>(out + 8 * c0) = pack8_e4m3(f, inv);
        *reinterpret_cast<uint2*>(out + 8 * c1) = pack8_e4m3(f + 8, inv);
      }
    }
  }
}

}  // namespace mxq
