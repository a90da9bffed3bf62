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
// key tiles (and, in the many-row kernel, some places for what a unit costs beside them) in a line,
// every worker (a CTA, or a warp in the few-row kernel) takes an equal, contiguous share of it: the
// load is even whatever the lengths, nothing is planned on the host, and only the first and the
// last segment of a share can be a part of a unit.  Such a part goes to the workspace as an
// unnormalised FP32 accumulator with its row maxima and sums (two slots per worker, so the
// workspace does not grow with the lengths), and the joining kernel adds the parts of each unit in
// an order that the lengths fix.
//
// kPerHead (the few-row kernel, which has over a thousand workers): the line is one key head's, and
// workers g, g + 1, ... take the same share of heads g mod Hk, so that the heads of a token are
// read side by side at the same time (E4M3, d = 128, [page][token][head][d]: 128-byte pieces of
// 1 KB rows).  Else the line goes over all key heads.
#pragma once

#include "gemm_common.cuh"

namespace mxq {

struct PagedParams {
  const uint16_t* q;  // [T][ldq] BF16, head h in columns [h d, (h + 1) d)
  uint16_t* out;      // [T][ldo]
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* block_table;
  float* part_o;     // [2 workers][rows x d]
  float2* part_ml;   // [2 workers][rows]: (row maximum, row sum)
  int4* part_units;  // [workers]: the unit that a worker begins and does not finish: (the sequence's first
                     // row of Q, row tile, rows in it, key head * 4096 + parts); parts 0: none
  int64_t ldq, ldo, T, table_stride;
  int batch, num_pages, page_size;
  int Hk, G;
  int tile_rows;       // rows (token, head of the group) in a row tile
  int causal, window;  // window 0: none
  int out32;           // rows of `out` are 32-byte aligned
  int page_box;        // keys per TMA box: gcd(page size, key tile)
  int workers;         // that may share the work
  float scale_log2;    // scale * log2(e) * k_scale
  float v_scale;
};

// A score's scale, held off zero (NaN stays): a masked score of -inf must not become NaN.  2^-126 times
// a score below 2^100 is zero to 2^-26.
__device__ __host__ __forceinline__ float nonzero_scale(float x) { return x < 0x1p-126f ? 0x1p-126f : x; }

// The weights 2^(t - m) of an E4M3 cache are rounded to FP16: 2^-11 relative, but 2^-25 absolute below its normal
// range, where small ones vanish from the product and not from the row sum (one strong key over a flat
// tail loses the tail).  So they are taken as 2^(t - m + 7), in sums and parts alike, which cancels in O / l: the
// running maximum is at most 8 behind, so that they reach 2^15 (FP16 holds up to 2^16), and a weight is off by
// 2^-32 of the largest at most.  BF16 has FP32's exponents and needs no shift.
template <bool kFp8>
__device__ __forceinline__ float weight_base(float m) {  // added to t
  return m == -INFINITY ? 0.f : (kFp8 ? 7.f : 0.f) - m;
}

// Keys that are added up in one accumulator.  The tensor core's FP32 sums are cut, not rounded: a step of 16
// keys loses some 1.6e-7 of the sum so far, always toward zero (positive values, 2^20 keys: 0.5 %, 2^22: 2.6 %).
// So a worker's part of a unit is taken in runs of at most this many keys (0.03 %), each joined to the ones before
// in the worker's place in the workspace, in rounded FP32.
constexpr int kRunKeys = 65536;

// What joins a run (m, l, O) to the part before it, of maximum ml.x and sum ml.y: O <- O x own + part x before.
struct RunJoin {
  float own, before;
};

__device__ __forceinline__ RunJoin join_run(float2 ml, float& m, float& l) {
  const float top = fmaxf(m, ml.x), base = top == -INFINITY ? 0.f : top;
  const RunJoin j = {exp2f(m - base), exp2f(ml.x - base)};
  l = fmaf(l, j.own, ml.y * j.before);
  m = top;
  return j;
}

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

template <int kKeys, int kUnitCost>
__device__ __forceinline__ int unit_weight(const PagedParams& p, const Sequence& s, int rt) {
  Unit u;
  u.rt = rt;
  u.s = s;
  set_unit<kKeys>(p, u);
  return kUnitCost + u.nt;
}

// The next unit in the line (row tiles within key heads within sequences).
template <int kKeys, bool kPerHead>
__device__ __forceinline__ void next_unit(const PagedParams& p, Unit& u) {
  if (u.rt + 1 < row_tiles(p, u.s)) {
    ++u.rt;
  } else {
    u.rt = 0;
    if (kPerHead || ++u.hk == p.Hk) {
      if (!kPerHead) u.hk = 0;
      do {
        ++u.b;
        if (u.b >= p.batch) return;  // only past the last share
        u.s = load_sequence(p, u.b);
      } while (u.s.n == 0);
    }
  }
  set_unit<kKeys>(p, u);
}

// A worker's share of the line: the places [begin, begin + count).  A unit has kUnitCost places for
// what is spent on it once (nobody's work when a border falls among them), then one per key tile.
struct Share {
  Unit u;
  int offset;  // of the first place within the unit
  int64_t begin, count;
  int64_t total;         // the line's length
  int shares;            // into which it is divided
  int index;             // which of them this is
};

constexpr int kMaxWorkers = 16;  // of one CTA

struct ShareScratch {
  int64_t warp_sum[32];
  int64_t begin[kMaxWorkers], end[kMaxWorkers];
  int64_t weight[kMaxWorkers], rest[kMaxWorkers];
  int b[kMaxWorkers], index[kMaxWorkers];
};

// The share of this thread's worker: the CTA has kWorkers, one for each of its first kWorkers
// warps (or one for all of them).  Called by all kThreads threads.  Sequences are weighed in
// parallel, by a warp each when there are few of them (a long chunk has many row tiles), by a
// thread each otherwise.  A share has at least about kMinPlaces: fewer workers take part in a small
// call.
template <int kKeys, int kThreads, int kWorkers, int kMinPlaces, int kUnitCost, bool kPerHead>
__device__ __forceinline__ Share find_share(const PagedParams& p, ShareScratch& sc) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps <= 32 && kWorkers <= kMaxWorkers && kWorkers <= kWarps, "scratch");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool by_warp = p.batch <= kWarps;
  const int per_round = by_warp ? kWarps : kThreads;
  auto weigh = [&](int b) -> int64_t {  // by_warp: in lane 0 only, 0 elsewhere
    int64_t w = 0;
    if (b < p.batch) {
      const Sequence s = load_sequence(p, b);
      const int tiles = row_tiles(p, s);
      for (int rt = by_warp ? lane : 0; rt < tiles; rt += by_warp ? 32 : 1)
        w += unit_weight<kKeys, kUnitCost>(p, s, rt);
      if (!kPerHead) w *= p.Hk;
    }
    if (by_warp) {
      for (int m = 16; m > 0; m >>= 1) w += __shfl_xor_sync(0xffffffffu, w, m);
      if (lane) w = 0;
    }
    return w;
  };
  int64_t total = 0, mine = 0;
  const int rounds = (p.batch + per_round - 1) / per_round;
  // the total, then (with the weights still in hand when one round holds them all) the search
  for (int r = 0; r < rounds; ++r) {
    mine = weigh(r * per_round + (by_warp ? warp : tid));
    int64_t w = mine;
    for (int m = 16; m > 0; m >>= 1) w += __shfl_xor_sync(0xffffffffu, w, m);
    __syncthreads();
    if (lane == 0) sc.warp_sum[warp] = w;
    if (tid < kWorkers) sc.b[tid] = -1;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) total += sc.warp_sum[i];
  }
  int64_t shares =
      min(static_cast<int64_t>(kPerHead ? p.workers / p.Hk : p.workers), (total + kMinPlaces - 1) / kMinPlaces);
  // One key tile more in every share costs what some 16 parts more cost in the join: a few long units
  // have about four times the square root of their tiles in parts (one token, BF16, 20000 keys of one key head:
  // 20 to 22 us, with all workers 25; 100000: 33 to 36, 38; with the factor 2: 25 and 45).  The workers that
  // take part are those of the first CTAs, so these times hold the bandwidth of few SMs as well.
  if (kPerHead) {
    const float units = fmaxf(static_cast<float>(p.batch), static_cast<float>(p.T * p.G / p.tile_rows));
    shares = min(shares, static_cast<int64_t>(4.f * sqrtf(static_cast<float>(total) * units)) + 1);
  }
  if (tid < kWorkers) {
    const int g = blockIdx.x * kWorkers + tid;
    const int64_t c = kPerHead ? g / p.Hk : g;
    sc.index[tid] = static_cast<int>(c);
    sc.begin[tid] = c < shares ? total * c / shares : total;
    sc.end[tid] = c < shares ? total * (c + 1) / shares : total;
  }
  __syncthreads();
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
    int64_t lo = before + incl - mine;
    for (int i = 0; i < warp; ++i) lo += sc.warp_sum[i];
    if (mine > 0) {
      for (int w = 0; w < kWorkers; ++w) {
        const int64_t begin = sc.begin[w];
        if (begin >= lo && begin < lo + mine) {
          sc.b[w] = b;
          sc.rest[w] = begin - lo;
          sc.weight[w] = mine;
        }
      }
    }
    for (int i = 0; i < kWarps; ++i) before += sc.warp_sum[i];
  }
  __syncthreads();
  const int worker = kWorkers == 1 ? 0 : min(warp, kWorkers - 1);
  Share sh;
  sh.begin = sc.begin[worker];
  sh.count = sc.b[worker] < 0 ? 0 : sc.end[worker] - sh.begin;
  sh.index = sc.index[worker];
  sh.total = total;
  sh.shares = static_cast<int>(shares);
  sh.offset = 0;
  sh.u.b = sc.b[worker];
  if (sh.count > 0) {
    sh.u.s = load_sequence(p, sh.u.b);
    int64_t rest = sc.rest[worker];
    if (kPerHead) {
      sh.u.hk = static_cast<int>(blockIdx.x * kWorkers + worker) % p.Hk;
    } else {
      const int64_t per_head = sc.weight[worker] / p.Hk;
      sh.u.hk = static_cast<int>(rest / per_head);
      rest -= sh.u.hk * per_head;
    }
    // the row tile: 32 at a time, each warp for itself
    const int tiles = row_tiles(p, sh.u.s);
    for (int rt0 = 0;; rt0 += 32) {
      const int w = rt0 + lane < tiles ? unit_weight<kKeys, kUnitCost>(p, sh.u.s, rt0 + lane) : 0;
      int incl = w;
      for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m) incl += o;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, w > 0 && rest < incl);
      if (hit || rt0 + 32 >= tiles) {
        const int l = hit ? __ffs(hit) - 1 : 0;
        sh.u.rt = rt0 + l;
        sh.offset = static_cast<int>(rest - __shfl_sync(0xffffffffu, incl - w, l));
        break;
      }
      rest -= __shfl_sync(0xffffffffu, incl, 31);
    }
    set_unit<kKeys>(p, sh.u);
  }
  return sh;
}

// The share that has place x of the line.
__device__ __forceinline__ int owner(const Share& sh, int64_t x) {
  return static_cast<int>(((x + 1) * sh.shares - 1) / sh.total);
}

// Row r (from the sequence's first) of key head hk in a [T][ld] matrix of heads of D columns.
template <int D>
__device__ __forceinline__ int64_t row_offset(const PagedParams& p, int64_t q0, int hk, int r, int64_t ld) {
  const int i = r / p.G;
  return (q0 + i) * ld + static_cast<int64_t>(hk * p.G + r - i * p.G) * D;
}

// What a worker leaves for the joining kernel: parts 0 unless it began the unit and did not
// finish it.  `at`: the place in the line of the unit's first key tile.
__device__ __forceinline__ int4 part_unit(const Share& sh, const Unit& u, int64_t at, bool begun_only) {
  const int parts = begun_only ? owner(sh, at + u.nt - 1) - sh.index + 1 : 0;
  return make_int4(static_cast<int>(u.s.q0), u.rt, u.rows, u.hk * 4096 + parts);
}

// The maximum of two row maxima, or NaN if one is.
__device__ __forceinline__ float max_or_nan(float a, float b) { return a != a || a >= b ? a : b; }

// Joins the parts of the units that the kWorkers workers of CTA blockIdx.x began: the worker's last
// slot, then the first slots of the workers of the next shares of its head.  gridDim.y
// blocks take the pairs of a worker and a row in turn: a warp each where the unit has up to
// kJoinWarpParts parts, else a block (a unit that spans the whole machine has over a thousand; 20000
// keys of one key head, eight rows, parts by all workers: 24 us with its rows in different blocks, 128 in one;
// 20 to 22 with the parts of find_share).
constexpr int kJoinWarpParts = 32;

template <int D, int kWorkers>
__global__ void __launch_bounds__(256) paged_join_few_kernel(const PagedParams p) {
  constexpr int kGroups = D / 4, kSlices = 256 / kGroups;
  __shared__ float s_m[8], s_l[kSlices];
  __shared__ float4 s_o[kSlices][kGroups];
  __shared__ int4 s_units[kWorkers];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, group = threadIdx.x % kGroups, slice = threadIdx.x / kGroups;
  if (threadIdx.x < kWorkers) s_units[threadIdx.x] = p.part_units[blockIdx.x * kWorkers + threadIdx.x];
  __syncthreads();
  // Units of few parts: a warp each, D / 32 columns a lane.
  const int pairs = kWorkers * p.tile_rows;  // of a worker and a row
  for (int q = blockIdx.y * 8 + (threadIdx.x >> 5); q < pairs; q += 8 * gridDim.y) {
    constexpr int kCols = D / 32, kAhead = 4;
    const int w = q % kWorkers, r = q / kWorkers, c = blockIdx.x * kWorkers + w;
    const int4 un = s_units[w];
    const int parts = un.w & 4095;
    if (parts > 0 && parts <= kJoinWarpParts && r < un.z) {
      auto row_of = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i * p.Hk)) * p.tile_rows + r; };
      auto value = [&](int i, float (&v)[kCols]) {
        const float* o = p.part_o + row_of(i) * D + lane * kCols;
        if constexpr (kCols == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(o);
        else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(o);
      };
      float ahead[kAhead][kCols];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < parts) value(i, ahead[i]);
      const float2 mine = lane < parts ? p.part_ml[row_of(lane)] : make_float2(-INFINITY, 0.f);
      float m = mine.x;
      for (int k = 16; k > 0; k >>= 1) m = max_or_nan(m, __shfl_xor_sync(0xffffffffu, m, k));
      const float f = exp2f(mine.x - (m == -INFINITY ? 0.f : m));
      float l = mine.y * f;
      for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
      float acc[kCols] = {};
      auto add = [&](int i, const float (&v)[kCols]) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] = fmaf(v[k], fi, acc[k]);
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < parts) add(i, ahead[i]);
#pragma unroll 4
      for (int i = kAhead; i < parts; ++i) {
        float v[kCols];
        value(i, v);
        add(i, v);
      }
      const float inv = l == 0.f ? 0.f : p.v_scale / l;
      uint32_t h[kCols / 2];
#pragma unroll
      for (int k = 0; k < kCols / 2; ++k) h[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
      uint16_t* dst = p.out + row_offset<D>(p, un.x, un.w >> 12, un.y * p.tile_rows + r, p.ldo) + lane * kCols;
      if constexpr (kCols == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
      else *reinterpret_cast<uint32_t*>(dst) = h[0];
    }
  }
  // The others: the whole block, slices of the parts side by side; the rows of a unit, and the
  // units of a row, are in different blocks.
  for (int q = blockIdx.y; q < pairs; q += gridDim.y) {
    const int r = q / kWorkers, w = (q + r) % kWorkers, c = blockIdx.x * kWorkers + w;
    const int4 un = s_units[w];
    const int parts = un.w & 4095;
    if (parts <= kJoinWarpParts || r >= un.z) continue;
    auto row_of = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i * p.Hk)) * p.tile_rows + r; };
    float m = -INFINITY;
    for (int i = threadIdx.x; i < parts; i += 256) m = max_or_nan(m, p.part_ml[row_of(i)].x);
    for (int k = 16; k > 0; k >>= 1) m = max_or_nan(m, __shfl_xor_sync(0xffffffffu, m, k));
    if (lane == 0) s_m[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int i = 0; i < 8; ++i) m = max_or_nan(m, s_m[i]);
    const float base = m == -INFINITY ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int i = slice; i < parts; i += kSlices) {
      const float2 ml = p.part_ml[row_of(i)];
      const float f = exp2f(ml.x - base);
      l = fmaf(ml.y, f, l);
      const float4 v = reinterpret_cast<const float4*>(p.part_o)[row_of(i) * kGroups + group];
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
    }
    s_o[slice][group] = acc;
    if (group == 0) s_l[slice] = l;
    __syncthreads();
    if (slice == 0) {
      for (int i = 1; i < kSlices; ++i) {
        const float4 v = s_o[i][group];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
        l += s_l[i];
      }
      const float inv = l == 0.f ? 0.f : p.v_scale / l;
      uint16_t* dst = p.out + row_offset<D>(p, un.x, un.w >> 12, un.y * p.tile_rows + r, p.ldo) + 4 * group;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    }
    __syncthreads();
  }
}

// The same for the unit that worker blockIdx.x began, many rows: a block has 8 rows at a time and
// all groups of four columns; parts are [d / 4][row][4], the layout in which the thread per row that
// wrote them stored consecutively.  A warp finds the factors of a row's parts, a lane each, while
// the first values are on their way.
template <int D, int kRows, int kMaxParts>
__global__ void __launch_bounds__(2 * D) paged_join_many_kernel(const PagedParams p) {
  constexpr int kWarps = 2 * D / 32, kAhead = 4;
  __shared__ float s_f[kMaxParts][8], s_inv[8];
  griddep_wait();  // no early launch of what follows: a 6001-token E4M3 prompt after itself took 470 us, not 430
  const int c = blockIdx.x, lane = threadIdx.x & 31, group = threadIdx.x >> 3;
  const int4 un = p.part_units[c];
  const int parts = un.w & 4095;
  if (parts == 0) return;
  auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)); };
  for (int r0 = blockIdx.y * 8; r0 < un.z; r0 += 8 * gridDim.y) {
    const int r = r0 + (threadIdx.x & 7);  // below kRows; from un.z on not kept
    auto value = [&](int i) {
      return reinterpret_cast<const float4*>(p.part_o)[(slot(i) * (D / 4) + group) * kRows + r];
    };
    float4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < parts && r < un.z) ahead[i] = value(i);
    for (int row = threadIdx.x >> 5; row < min(8, un.z - r0); row += kWarps) {
      constexpr int kMine = (kMaxParts + 31) / 32;
      float2 ml[kMine];
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        ml[k] = lane + 32 * k < parts ? p.part_ml[slot(lane + 32 * k) * kRows + r0 + row] : make_float2(-INFINITY, 0.f);
        m = max_or_nan(m, ml[k].x);
      }
      for (int k = 16; k > 0; k >>= 1) m = max_or_nan(m, __shfl_xor_sync(0xffffffffu, m, k));
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const float f = exp2f(ml[k].x - base);
        l = fmaf(ml[k].y, f, l);
        if (lane + 32 * k < parts) s_f[lane + 32 * k][row] = f;
      }
      for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
      if (lane == 0) s_inv[row] = l == 0.f ? 0.f : p.v_scale / l;
    }
    __syncthreads();
    if (r < un.z) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](int i, const float4& v) {
        const float f = s_f[i][threadIdx.x & 7];
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < parts) add(i, ahead[i]);
#pragma unroll 8
      for (int i = kAhead; i < parts; ++i) add(i, value(i));
      const float inv = s_inv[threadIdx.x & 7];
      uint16_t* dst = p.out + row_offset<D>(p, un.x, un.w >> 12, un.y * p.tile_rows + r, p.ldo) + 4 * group;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    }
    __syncthreads();
  }
}

}  // namespace mxq
