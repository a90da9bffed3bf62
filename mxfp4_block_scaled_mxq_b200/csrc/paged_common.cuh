// paged_common.cuh -- what the paged attention kernels share: the batch's metadata, the
// division of its work over the CTAs, and the kernel that joins split rows.
//
//   O_i = v_scale * sum_j 2^(t_ij - m_i) V_j / sum_j 2^(t_ij - m_i),
//   t_ij = scale * log2(e) * k_scale * (q_i . K_j),  m_i = max_j t_ij,
// over the keys j that row i attends: j < kv_len, with causal also j <= p_i, with a window also
// j > p_i - window, p_i = kv_len - q_len + i; a row without keys is 0.
//
// Work.  The query heads of one key head share its keys, so a row is (token, head of the group)
// and a unit is (sequence, key head, row tile) with the key tiles its rows reach.  All units'
// key tiles in a line, every CTA takes an equal, contiguous share of it: the load is even
// whatever the lengths, nothing is planned on the host, and only the first and the last
// segment of a CTA can be a part of a unit.  Such a part goes to the workspace as an
// unnormalised FP32 accumulator with its row maxima and sums (two slots per CTA, so the
// workspace does not grow with the lengths), and the joining kernel adds the parts of each unit
// in the order of the keys.
#pragma once

#include "gemm_common.cuh"

namespace mxq {

struct PagedParams {
  const uint16_t* q;  // [T][ldq] BF16, head h in columns [h d, (h + 1) d)
  uint16_t* out;      // [T][ldo]
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* block_table;
  float* part_o;     // [2 ctas][d / 4][rows][4]
  float2* part_ml;   // [2 ctas][rows]: (row maximum, row sum)
  int4* part_units;  // [ctas]: the unit that CTA c begins and does not finish: (the sequence's first
                     // row of Q, row tile, rows in it, key head * 4096 + parts); parts 0: none
  int64_t ldq, ldo, T, table_stride;
  int batch, num_pages, page_size;
  int Hk, G;
  int tile_rows;       // rows (token, head of the group) in a row tile
  int causal, window;  // window 0: none
  int out32;           // rows of `out` are 32-byte aligned
  int page_box;        // keys per TMA box: gcd(page size, key tile)
  int ctas;            // that share the work (the partial slots' count is twice that)
  float scale_log2;    // scale * log2(e) * k_scale
  float v_scale;
};

// One sequence: its rows of Q, its length, clamped to what Q and the block table hold.
struct Sequence {
  int64_t q0;
  int n, len;
};

__device__ __forceinline__ Sequence load_sequence(const PagedParams& p, int b) {
  Sequence s;
  const int64_t a = p.cu_q[b], e = p.cu_q[b + 1];
  s.q0 = min(max(a, int64_t(0)), p.T);
  s.n = static_cast<int>(min(max(e, s.q0), p.T) - s.q0);
  s.len = static_cast<int>(min(static_cast<int64_t>(max(p.kv_len[b], 0)), p.table_stride * p.page_size));  // <= 2^30
  return s;
}

// Keys [lo, hi) that the tokens [i0, i1] of a sequence reach together.
__device__ __forceinline__ int2 key_range(const PagedParams& p, const Sequence& s, int i0, int i1) {
  int lo = 0, hi = s.len;
  if (p.causal) {
    const int p0 = s.len - s.n;
    hi = min(hi, p0 + i1 + 1);
    if (p.window) lo = max(0, p0 + i0 - p.window + 1);
  }
  return make_int2(min(lo, max(hi, 0)), max(hi, 0));
}

// A unit: `rows` rows from r0 (row r: token r / G, head r % G of the group) of tokens [i0, i1],
// and the key tiles [kt0, kt0 + nt) that cover their keys [lo, hi); at least one key tile, since
// a row without keys is written too.
struct Unit {
  int b, hk, rt;
  Sequence s;
  int r0, rows, i0, i1;
  int lo, hi;
  int kt0, nt;
};

__device__ __forceinline__ int row_tiles(const PagedParams& p, const Sequence& s) {
  return (s.n * p.G + p.tile_rows - 1) / p.tile_rows;  // n * G < 2^30
}

template <int kKeys>
__device__ __forceinline__ void set_unit(const PagedParams& p, Unit& u) {
  u.r0 = u.rt * p.tile_rows;
  u.rows = min(p.tile_rows, u.s.n * p.G - u.r0);
  u.i0 = u.r0 / p.G;
  u.i1 = (u.r0 + u.rows - 1) / p.G;
  const int2 r = key_range(p, u.s, u.i0, u.i1);
  u.lo = r.x;
  u.hi = r.y;
  u.kt0 = r.x / kKeys;
  u.nt = max(1, (r.y + kKeys - 1) / kKeys - u.kt0);
}

template <int kKeys>
__device__ __forceinline__ int unit_tiles(const PagedParams& p, const Sequence& s, int rt) {
  Unit u;
  u.rt = rt;
  u.s = s;
  set_unit<kKeys>(p, u);
  return u.nt;
}

// The next unit in the line (row tiles within key heads within sequences).
template <int kKeys>
__device__ __forceinline__ void next_unit(const PagedParams& p, Unit& u) {
  if (u.rt + 1 < row_tiles(p, u.s)) {
    ++u.rt;
  } else {
    u.rt = 0;
    if (++u.hk == p.Hk) {
      u.hk = 0;
      do {
        ++u.b;
        if (u.b >= p.batch) return;  // only past the last share
        u.s = load_sequence(p, u.b);
      } while (u.s.n == 0);
    }
  }
  set_unit<kKeys>(p, u);
}

// This CTA's share of the line: where it begins, and how many key tiles it has.
struct Share {
  Unit u;
  int tile;              // first key tile within the unit
  int64_t begin, count;  // key tiles: the first one's place in the line, how many
  int64_t total;         // the line's length
  int shares;            // CTAs that have one
};

struct ShareScratch {
  int64_t warp_sum[32];
  int64_t weight, rest;
  int b;
};

// Called by all kThreads threads.  Sequences are weighed in parallel, by a warp each when
// there are few of them (a long chunk has many row tiles), by a thread each otherwise.  A
// share has at least about kMinTiles key tiles: fewer CTAs take part in a small call.
template <int kKeys, int kThreads, int kMinTiles>
__device__ __forceinline__ Share find_share(const PagedParams& p, ShareScratch& sc) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps <= 32, "scratch");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool by_warp = p.batch <= kWarps;
  const int per_round = by_warp ? kWarps : kThreads;
  auto weigh = [&](int b) -> int64_t {  // by_warp: the same value in lane 0 only, 0 elsewhere
    int64_t w = 0;
    if (b < p.batch) {
      const Sequence s = load_sequence(p, b);
      const int tiles = row_tiles(p, s);
      for (int rt = by_warp ? lane : 0; rt < tiles; rt += by_warp ? 32 : 1)
        w += unit_tiles<kKeys>(p, s, rt);
      w *= p.Hk;
    }
    if (by_warp) {
      for (int m = 16; m > 0; m >>= 1) w += __shfl_xor_sync(0xffffffffu, w, m);
      if (lane) w = 0;
    }
    return w;
  };
  if (tid == 0) sc.b = -1;
  int64_t total = 0, mine = 0;
  const int rounds = (p.batch + per_round - 1) / per_round;
  // the total, then (with the weights still in hand when one round holds them all) the search
  for (int r = 0; r < rounds; ++r) {
    mine = weigh(r * per_round + (by_warp ? warp : tid));
    int64_t w = mine;
    for (int m = 16; m > 0; m >>= 1) w += __shfl_xor_sync(0xffffffffu, w, m);
    __syncthreads();
    if (lane == 0) sc.warp_sum[warp] = w;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) total += sc.warp_sum[i];
  }
  const int64_t c = blockIdx.x;
  const int64_t shares = min(static_cast<int64_t>(p.ctas), (total + kMinTiles - 1) / kMinTiles);
  const int64_t begin = c < shares ? total * c / shares : total;
  const int64_t end = c < shares ? total * (c + 1) / shares : total;
  int64_t before = 0;
  for (int r = 0; r < rounds; ++r) {
    const int b = r * per_round + (by_warp ? warp : tid);
    if (rounds > 1) mine = weigh(b);
    int64_t incl = mine;
    for (int m = 1; m < 32; m <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += o;
    }
    if (rounds > 1) {
      __syncthreads();
      if (lane == 31) sc.warp_sum[warp] = incl;
      __syncthreads();
    }  // one round: the first loop's sums are these
    int64_t base = before;
    for (int i = 0; i < warp; ++i) base += sc.warp_sum[i];
    const int64_t lo = base + incl - mine;
    if (mine > 0 && lo <= begin && begin < lo + mine) {
      sc.b = b;
      sc.rest = begin - lo;
      sc.weight = mine;
    }
    for (int i = 0; i < kWarps; ++i) before += sc.warp_sum[i];
  }
  __syncthreads();
  Share sh;
  sh.begin = begin;
  sh.count = sc.b < 0 ? 0 : end - begin;
  sh.total = total;
  sh.shares = static_cast<int>(shares);
  sh.tile = 0;
  sh.u.b = sc.b;
  if (sh.count > 0) {
    sh.u.s = load_sequence(p, sh.u.b);
    const int64_t per_head = sc.weight / p.Hk;
    int64_t rest = sc.rest;
    sh.u.hk = static_cast<int>(rest / per_head);
    rest -= sh.u.hk * per_head;
    // the row tile: 32 at a time, each warp for itself
    const int tiles = row_tiles(p, sh.u.s);
    for (int rt0 = 0;; rt0 += 32) {
      const int w = rt0 + lane < tiles ? unit_tiles<kKeys>(p, sh.u.s, rt0 + lane) : 0;
      int incl = w;
      for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m) incl += o;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, w > 0 && rest < incl);
      if (hit || rt0 + 32 >= tiles) {
        const int l = hit ? __ffs(hit) - 1 : 0;
        sh.u.rt = rt0 + l;
        sh.tile = static_cast<int>(rest - __shfl_sync(0xffffffffu, incl - w, l));
        break;
      }
      rest -= __shfl_sync(0xffffffffu, incl, 31);
    }
    set_unit<kKeys>(p, sh.u);
  }
  return sh;
}

// The CTA that has the key tile at place x of the line.
__device__ __forceinline__ int owner(const Share& sh, int64_t x) {
  return static_cast<int>(((x + 1) * sh.shares - 1) / sh.total);
}

// Row r (from the sequence's first) of key head hk in a [T][ld] matrix of heads of D columns.
template <int D>
__device__ __forceinline__ int64_t row_offset(const PagedParams& p, int64_t q0, int hk, int r, int64_t ld) {
  const int i = r / p.G;
  return (q0 + i) * ld + static_cast<int64_t>(hk * p.G + r - i * p.G) * D;
}

// Joins the parts of the unit that CTA blockIdx.x began: its last slot, then the first slots
// of the CTAs after it.  A block has 8 rows x 16 groups of D / 16 columns: the parts' loads are
// consecutive over the rows, the result's over the columns.
template <int D, int kRows>
__global__ void __launch_bounds__(128) paged_join_kernel(const PagedParams p) {
  constexpr int kGroup = D / 16;   // columns of a thread
  constexpr int kVec = kGroup / 4;
  griddep_wait();
  const int c = blockIdx.x;
  const int4 un = p.part_units[c];
  const int parts = un.w & 4095;
  const int r = blockIdx.y * 8 + (threadIdx.x & 7), group = threadIdx.x >> 3;
  if (parts == 0 || r >= un.z) return;
  auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)); };
  float m = -INFINITY;
  for (int i = 0; i < parts; ++i) m = fmaxf(m, p.part_ml[slot(i) * kRows + r].x);
  const float base = m == -INFINITY ? 0.f : m;
  float acc[kGroup] = {}, l = 0.f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float2 ml = p.part_ml[slot(i) * kRows + r];
    const float f = exp2f(ml.x - base);
    l = fmaf(ml.y, f, l);
    const float4* o = reinterpret_cast<const float4*>(p.part_o) + (slot(i) * (D / 4) + group * kVec) * kRows + r;
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const float4 v = o[k * kRows];
      acc[4 * k] = fmaf(v.x, f, acc[4 * k]);
      acc[4 * k + 1] = fmaf(v.y, f, acc[4 * k + 1]);
      acc[4 * k + 2] = fmaf(v.z, f, acc[4 * k + 2]);
      acc[4 * k + 3] = fmaf(v.w, f, acc[4 * k + 3]);
    }
  }
  const float inv = l == 0.f ? 0.f : p.v_scale / l;
  uint16_t* dst = p.out + row_offset<D>(p, un.x, un.w >> 12, un.y * p.tile_rows + r, p.ldo) + group * kGroup;
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    *reinterpret_cast<uint2*>(dst + 4 * k) = make_uint2(pack_bf16x2(acc[4 * k] * inv, acc[4 * k + 1] * inv),
                                                        pack_bf16x2(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv));
}

}  // namespace mxq
