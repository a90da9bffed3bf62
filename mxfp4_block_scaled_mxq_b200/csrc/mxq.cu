// mxq.cu -- libmxq: the C ABI of include/mxq.h (host-side validation, TMA tensor-map
// encoding and launches) over the sm_100a kernels in quantize.cuh, gemm_pair.cuh and gemm_swap.cuh.
// One translation unit, so the library's device status word exists exactly once.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "mxq.h"
#include "gemm_common.cuh"
#include "gemm_pair.cuh"
#include "gemm_swap.cuh"
#include "policy.cuh"
#include "attention.cuh"
#include "paged_chunk.cuh"
#include "paged_decode.cuh"
#include "quantize.cuh"
#include "rope_cache.cuh"

// Scratch of mxq_linear_w4a4_static: the quantised activations of one call, per device.
constexpr int64_t kStaticScratchBytes = MXQ_STATIC_SCRATCH_BYTES;
static __device__ __align__(256) uint8_t g_linear_scratch[kStaticScratchBytes];

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

constexpr int kMaxDevices = 64;

// Per-device facts, looked up once per device.
struct DeviceInfo {
  bool ok = false;
  int index = -1;
  int sm_count = 0;
};

DeviceInfo device_info(int dev) {
  static DeviceInfo info[kMaxDevices];
  static std::once_flag once[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return {};
  std::call_once(once[dev], [dev] {
    cudaDeviceProp p;
    if (cudaGetDeviceProperties(&p, dev) != cudaSuccess) return;
    info[dev].ok = (p.major == 10 && p.minor == 0);
    info[dev].index = dev;
    info[dev].sm_count = p.multiProcessorCount;
  });
  return info[dev];
}

mxq_status current_device(DeviceInfo* out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return MXQ_ERR_CUDA;
  *out = device_info(dev);
  if (!out->ok) return MXQ_ERR_UNSUPPORTED;
  return MXQ_OK;
}

// One-time set-up per device.  Kernel attributes (the opt-in shared memory size), the
// occupancy they allow and symbol addresses belong to one device's context, so every device
// runs `setup` (with that device current) before its first launch.  Only a successful set-up
// is remembered: a failed one returns false and runs again on the next call.
class PerDevice {
 public:
  template <typename Setup>
  bool ensure(int dev, Setup&& setup) {
    if (dev < 0 || dev >= kMaxDevices) return false;
    if (done_[dev].load(std::memory_order_acquire)) return true;
    std::lock_guard<std::mutex> lock(mu_);
    if (!done_[dev].load(std::memory_order_relaxed) && setup()) done_[dev].store(true, std::memory_order_release);
    return done_[dev].load(std::memory_order_relaxed);
  }

 private:
  std::mutex mu_;
  std::atomic<bool> done_[kMaxDevices] = {};
};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

mxq_status launch_status() {
  return cudaGetLastError() == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

// Launch with programmatic stream serialisation: the kernel may start while the kernel
// before it in the stream (normally the activation quantiser, which lets dependents start)
// finishes; the kernel executes griddepcontrol.wait before it reads any input.
template <typename... KArgs, typename... Args>
mxq_status launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, int smem, cudaStream_t stream,
                            Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

// 2-D tensor map over a row-major [rows][cols] matrix.
bool make_tmap_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t cols, uint64_t rows,
                  uint64_t row_stride_bytes, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle sw) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {row_stride_bytes};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 4-D tensor map over a swizzled scale-factor buffer of `rows` rows and K columns:
// (byte in 128-byte chunk, chunk in atom, atom along K, 128-row tile); a box of
// {128, 4, atoms, row_tiles} lands as contiguous 512-byte atoms, [row tile][atom].
bool make_tmap_sf(CUtensorMap* m, const void* base, int64_t rows, int64_t K, uint32_t atoms, uint32_t row_tiles) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const uint64_t atoms_per_row_tile = static_cast<uint64_t>(K) / 128;
  const cuuint64_t dims[4] = {128, 4, atoms_per_row_tile, static_cast<cuuint64_t>((rows + 127) / 128)};
  const cuuint64_t strides[3] = {128, 512, atoms_per_row_tile * 512};
  const cuuint32_t box[4] = {128, 4, atoms, row_tiles};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Two-CTA path (one 256 x 192 tile per CTA pair), persistent over as many pairs as
// can be resident at once.
template <bool kW4A8>
mxq_status launch_gemm_pair(const DeviceInfo& dev, const void* a, const void* a_sf, const void* b, const void* b_sf,
                            int64_t M, int64_t N, int64_t K, float alpha, const void* bias, void* d, int64_t ldd,
                            cudaStream_t stream) {
  using S = mxq::PairShape<kW4A8>;
  auto kernel = mxq::mx_gemm_pair_kernel<kW4A8>;
  static PerDevice setup;
  static int max_clusters_of[kMaxDevices];
  const bool ready = setup.ensure(dev.index, [&] {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes) != cudaSuccess)
      return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(mxq::kGemmThreads, 1, 1);
    cfg.dynamicSmemBytes = S::kSmemBytes;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return false;
    max_clusters_of[dev.index] = n;
    return true;
  });
  if (!ready) return MXQ_ERR_CUDA;
  const int max_clusters = max_clusters_of[dev.index];

  CUtensorMap ta, tb, tsa, tsb;
  bool ok;
  if (kW4A8) {
    ok = make_tmap_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K, M, K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_tmap_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, b, K, N, K / 2, 128, S::kBRows,
                      CU_TENSOR_MAP_SWIZZLE_128B);
    tsa = tb;  // unused: E4M3 activations carry unit scales
  } else {
    ok = make_tmap_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K / 2, M, K / 2, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_tmap_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, b, K / 2, N, K / 2, 128, S::kBRows,
                      CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_tmap_sf(&tsa, a_sf, M, K, S::kAtoms, 1);
  }
  ok = ok && make_tmap_sf(&tsb, b_sf, N, K, S::kAtoms, 2);
  if (!ok) return MXQ_ERR_CUDA;
  const int64_t tiles = ((M + 255) / 256) * ((N + mxq::kBN - 1) / mxq::kBN);
  const int clusters = static_cast<int>(tiles < max_clusters ? tiles : max_clusters);
  // 32-byte output stores need 32-byte aligned rows
  const int d_vec32 = (ldd % 16 == 0 && aligned(d, 32)) ? 1 : 0;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(2 * clusters), 1, 1), dim3(mxq::kGemmThreads, 1, 1),
                          S::kSmemBytes, stream, ta, tb, tsa, tsb, static_cast<__nv_bfloat16*>(d), ldd, d_vec32,
                          static_cast<const __nv_bfloat16*>(bias), static_cast<int>(M), static_cast<int>(N),
                          static_cast<int>(K), alpha);
}

// Device address of g_linear_scratch on the current device `dev`, looked up once per device
// (a failed lookup is retried on the next call).
void* static_scratch(int dev) {
  static PerDevice setup;
  static void* addr[kMaxDevices];
  const bool ready = setup.ensure(dev, [dev] {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_linear_scratch) != cudaSuccess || !p) return false;
    addr[dev] = p;
    return true;
  });
  return ready ? addr[dev] : nullptr;
}

// Workspace of the quantized linear layer: the quantised activations (codes, then scales).
struct LinearWorkspace {
  int64_t codes = 0, sf = 0, bytes = 0;
};

LinearWorkspace linear_workspace(int64_t M, int64_t K) {
  auto up = [](int64_t v) { return (v + 1023) / 1024 * 1024; };
  LinearWorkspace w;
  w.codes = 0;
  w.sf = up(M * (K / 2));
  w.bytes = w.sf + up((M + 127) / 128 * 128 * ((K / 32 + 3) / 4 * 4));
  return w;
}

// Few tokens (M <= 128): D^T = W X^T with the weights on the MMA's 128-row side; one
// kernel instance per token tile width Mt (the tokens rounded up to 16).
template <bool kW4A8, int Mt>
mxq_status launch_gemm_swap_mt(const DeviceInfo& dev, const CUtensorMap& tw, const CUtensorMap& tt,
                               const CUtensorMap& tsw, const CUtensorMap& tst, int64_t M, int64_t N, int64_t K,
                               float alpha, const void* bias, void* d, int64_t ldd, cudaStream_t stream) {
  using S = mxq::SwapShape<kW4A8>;
  auto kernel = mxq::mx_gemm_swap_kernel<kW4A8, Mt>;
  constexpr int kMaxSmem = 232448;  // opt-in shared memory per CTA on sm_100
  static PerDevice setup;
  if (!setup.ensure(dev.index, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) == cudaSuccess;
      }))
    return MXQ_ERR_CUDA;
  int stages = (kMaxSmem - S::kFixedBytes - S::out_bytes(Mt)) / S::stage_bytes(Mt);
  stages = stages > mxq::kSwapMaxStages ? mxq::kSwapMaxStages : stages;
  const int smem = S::kFixedBytes + S::out_bytes(Mt) + stages * S::stage_bytes(Mt);
  // D [M][N] BF16 written as [Mt][128] boxes (row stride ldd * 2 bytes: ldd % 8 == 0)
  CUtensorMap td;
  if (!make_tmap_2d(&td, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d, N, M, ldd * 2, 128, Mt, CU_TENSOR_MAP_SWIZZLE_NONE))
    return MXQ_ERR_CUDA;
  const int64_t tiles = (N + 127) / 128;
  const int grid = static_cast<int>(tiles < dev.sm_count ? tiles : dev.sm_count);
  return launch_dependent(kernel, dim3(static_cast<unsigned>(grid), 1, 1), dim3(mxq::kSwapThreads, 1, 1), smem,
                          stream, tw, tt, tsw, tst, td, static_cast<const __nv_bfloat16*>(bias), static_cast<int>(M),
                          static_cast<int>(N), static_cast<int>(K), alpha, stages);
}

template <bool kW4A8>
mxq_status launch_gemm_swap(const DeviceInfo& dev, const void* a, const void* a_sf, const void* b, const void* b_sf,
                            int64_t M, int64_t N, int64_t K, float alpha, const void* bias, void* d, int64_t ldd,
                            cudaStream_t stream) {
  using S = mxq::SwapShape<kW4A8>;
  const int Mt = static_cast<int>((M + 15) / 16 * 16);
  CUtensorMap tw, tt, tsw, tst;
  bool ok;
  if (kW4A8) {
    ok = make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, b, K, N, K / 2, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_tmap_2d(&tt, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K, M, K, 128, Mt, CU_TENSOR_MAP_SWIZZLE_128B);
    tst = tw;  // unused: E4M3 tokens carry unit scales
  } else {
    ok = make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, b, K / 2, N, K / 2, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_tmap_2d(&tt, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K / 2, M, K / 2, 128, Mt, CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_tmap_sf(&tst, a_sf, M, K, S::kAtoms, 1);
  }
  ok = ok && make_tmap_sf(&tsw, b_sf, N, K, S::kAtoms, 1);
  if (!ok) return MXQ_ERR_CUDA;
  switch (Mt) {
#define MXQ_SWAP_CASE(T) \
  case T: return launch_gemm_swap_mt<kW4A8, T>(dev, tw, tt, tsw, tst, M, N, K, alpha, bias, d, ldd, stream);
    MXQ_SWAP_CASE(16) MXQ_SWAP_CASE(32) MXQ_SWAP_CASE(48) MXQ_SWAP_CASE(64)
    MXQ_SWAP_CASE(80) MXQ_SWAP_CASE(96) MXQ_SWAP_CASE(112) MXQ_SWAP_CASE(128)
#undef MXQ_SWAP_CASE
    default: return MXQ_ERR_SHAPE;
  }
}

template <bool kW4A8>
mxq_status launch_gemm(const void* a, const void* a_sf, const void* b, const void* b_sf, int64_t M, int64_t N,
                       int64_t K, float alpha, const void* bias, void* d, int64_t ldd, cudaStream_t stream) {
  DeviceInfo dev;
  mxq_status st = current_device(&dev);
  if (st != MXQ_OK) return st;
  if (M > mxq::kBM) return launch_gemm_pair<kW4A8>(dev, a, a_sf, b, b_sf, M, N, K, alpha, bias, d, ldd, stream);
  return launch_gemm_swap<kW4A8>(dev, a, a_sf, b, b_sf, M, N, K, alpha, bias, d, ldd, stream);
}

mxq_status check_gemm_shapes(const void* a, const void* b, const void* b_sf, const void* d, int64_t M, int64_t N,
                             int64_t K, int64_t ldd, const void* bias) {
  if (!a || !b || !b_sf || !d) return MXQ_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || K < 128 || K % 128 != 0) return MXQ_ERR_SHAPE;
  if (M > (int64_t(1) << 30) || N > (int64_t(1) << 30) || K > (int64_t(1) << 22)) return MXQ_ERR_SHAPE;
  const int64_t tiles = ((M + mxq::kBM - 1) / mxq::kBM) * ((N + mxq::kBN - 1) / mxq::kBN);
  if (tiles > INT32_MAX) return MXQ_ERR_SHAPE;  // tile indices are 32-bit in the kernel
  if (ldd < N || ldd % 8 != 0) return MXQ_ERR_ALIGN;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(b_sf, 16) || !aligned(d, 16)) return MXQ_ERR_ALIGN;
  if (bias && !aligned(bias, 16)) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

mxq_status launch_mxfp4(bool weight, const void* x, int64_t rows, int64_t K, int64_t ld, mxq_scale_rule rule,
                        int hadamard, void* codes, void* sf, cudaStream_t stream) {
  // grid.x: 128-column tiles (K <= 2^22 keeps it <= 32768), grid.y: 128-row tiles.
  const dim3 grid(static_cast<unsigned>((K + 127) / 128), static_cast<unsigned>((rows + 127) / 128));
  const auto* xp = static_cast<const uint16_t*>(x);
  auto* cp = static_cast<uint8_t*>(codes);
  auto* sp = static_cast<uint8_t*>(sf);
  const bool uos = rule == MXQ_SCALE_UOS;
  const int sel = (hadamard ? 2 : 0) | (uos ? 1 : 0);
  if (weight) {
    switch (sel) {
      case 0: mxq::pack_weight_mxfp4_kernel<false, false><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ld, cp, sp); break;
      case 1: mxq::pack_weight_mxfp4_kernel<false, true><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ld, cp, sp); break;
      case 2: mxq::pack_weight_mxfp4_kernel<true, false><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ld, cp, sp); break;
      default: mxq::pack_weight_mxfp4_kernel<true, true><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ld, cp, sp); break;
    }
  } else {
    switch (sel) {
      case 0: mxq::quantize_act_mxfp4_kernel<false, false><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ld, cp, sp); break;
      case 1: mxq::quantize_act_mxfp4_kernel<false, true><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ld, cp, sp); break;
      case 2: mxq::quantize_act_mxfp4_kernel<true, false><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ld, cp, sp); break;
      default: mxq::quantize_act_mxfp4_kernel<true, true><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ld, cp, sp); break;
    }
  }
  return launch_status();
}

mxq_status check_quant_args(const void* x, int64_t rows, int64_t K, int64_t ld, mxq_scale_rule rule, int hadamard,
                            const void* q, const void* sf) {
  if (!x || !q || !sf) return MXQ_ERR_INVALID_ARG;
  if (rule != MXQ_SCALE_OCP && rule != MXQ_SCALE_UOS) return MXQ_ERR_INVALID_ARG;
  // rows <= 65535 * 128 keeps grid.y within its limit
  if (rows < 1 || rows > int64_t(65535) * 128 || K < 32 || K % 32 != 0 || K > (int64_t(1) << 22)) return MXQ_ERR_SHAPE;
  if (hadamard && K % 128 != 0) return MXQ_ERR_SHAPE;
  // 16 BF16 values per load: 16-byte aligned rows (32-byte loads where rows allow them)
  if (ld < K || ld % 8 != 0) return MXQ_ERR_ALIGN;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 16)) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

// ----------------------------------------------------------------------------- paged cache
// Norm, rotation and operand checks shared by mxq_qk_norm_rope and mxq_kv_append.
mxq_status check_norm_rope(const mxq_norm_rope* c, int64_t d) {
  if (!c) return MXQ_ERR_INVALID_ARG;
  if (c->span != MXQ_NORM_HEAD && c->span != MXQ_NORM_ROW) return MXQ_ERR_INVALID_ARG;
  if (c->style != MXQ_ROPE_HALVES && c->style != MXQ_ROPE_PAIRS) return MXQ_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f) || !std::isfinite(c->eps)) return MXQ_ERR_INVALID_ARG;
  if ((c->table != nullptr) != (c->rot > 0)) return MXQ_ERR_INVALID_ARG;
  if (d < 16 || d > 256 || d % 16 != 0 || c->rot < 0 || c->rot > d || c->rot % 16 != 0) return MXQ_ERR_SHAPE;
  if (c->table && (c->table_rows < 1 || c->table_rows > (int64_t(1) << 31))) return MXQ_ERR_SHAPE;
  if (!aligned(c->q_weight, 16) || !aligned(c->k_weight, 16) || !aligned(c->table, 16)) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

// A [T][ld] BF16 operand of `heads` heads; null pointers are the caller's to allow.
mxq_status check_heads(const void* x, int64_t heads, int64_t d, int64_t ld) {
  if (heads < 1 || heads * d > (int64_t(1) << 16)) return MXQ_ERR_SHAPE;
  if (ld < heads * d || ld % 8 != 0 || !aligned(x, 16)) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

mxq_status check_paged(const mxq_paged_kv* c, const mxq_paged_batch* b) {
  if (!c || !b || !c->k || !c->v || !b->cu_q || !b->kv_len || !b->block_table) return MXQ_ERR_INVALID_ARG;
  if (c->fmt != MXQ_KV_BF16 && c->fmt != MXQ_KV_FP8_E4M3) return MXQ_ERR_INVALID_ARG;
  const float scales[2] = {c->k_scale, c->v_scale};
  for (float s : scales)
    if (!(s > 0.f) || !std::isfinite(s) || !std::isfinite(1.0f / s)) return MXQ_ERR_INVALID_ARG;
  if (c->fmt == MXQ_KV_BF16 && (c->k_scale != 1.f || c->v_scale != 1.f)) return MXQ_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_pages > (int64_t(1) << 30)) return MXQ_ERR_SHAPE;
  if (c->page_size < 8 || c->page_size % 8 != 0 || c->page_size > (int64_t(1) << 20)) return MXQ_ERR_SHAPE;
  if (c->heads < 1 || c->d < 16 || c->d > 256 || c->d % 16 != 0 || c->heads * c->d > (int64_t(1) << 16))
    return MXQ_ERR_SHAPE;
  if (b->batch < 1 || b->batch > (int64_t(1) << 20)) return MXQ_ERR_SHAPE;
  if (b->max_pages < 1 || b->max_pages > (int64_t(1) << 30) || b->max_pages * c->page_size > (int64_t(1) << 30))
    return MXQ_ERR_SHAPE;
  const int64_t size = c->fmt == MXQ_KV_BF16 ? 2 : 1;
  const int64_t strides[3] = {c->stride_page, c->stride_token, c->stride_head};
  for (int64_t s : strides)
    if (s < c->d || s * size % 16 != 0 || s * size >= (int64_t(1) << 40)) return MXQ_ERR_ALIGN;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(b->cu_q, 4) || !aligned(b->kv_len, 4) ||
      !aligned(b->block_table, 4))
    return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

mxq::RopeParams rope_params(const mxq_norm_rope* c, int64_t T, int64_t d) {
  mxq::RopeParams p = {};
  p.table = c->table;
  p.table_rows = c->table_rows;
  p.T = T;
  p.eps = c->eps;
  p.d = static_cast<int>(d);
  p.rot = static_cast<int>(c->rot);
  p.lanes = 1;
  while (16 * p.lanes < d) p.lanes *= 2;
  p.inv_d = 1.0f / static_cast<float>(d);
  p.row_norm = c->span == MXQ_NORM_ROW;
  return p;
}

mxq::RopeOperand rope_operand(const void* x, const void* weight, int64_t ld, void* out, int64_t ldo, int64_t heads) {
  mxq::RopeOperand o = {};
  if (!x) return o;
  o.x = static_cast<const uint16_t*>(x);
  o.weight = static_cast<const uint16_t*>(weight);
  o.ld = ld;
  o.out = static_cast<uint16_t*>(out);
  o.ldo = ldo;
  o.heads = static_cast<int>(heads);
  return o;
}

template <int kCache, bool kPairs>
mxq_status launch_rope_cache_as(const DeviceInfo& dev, mxq::RopeParams p, const mxq::AppendParams& a,
                             cudaStream_t stream) {
  constexpr int kMaxSmem = 224 * 1024;  // of an SM, less what its blocks have statically and as a reserve
  auto kernel = mxq::rope_cache_kernel<kCache, kPairs>;
  static PerDevice setup;
  if (!setup.ensure(dev.index, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) == cudaSuccess;
      }))
    return MXQ_ERR_CUDA;
  const int k_heads = p.k.heads * (kCache ? 2 : 1);
  const int heads = p.q.heads + k_heads;
  const int table = p.table ? p.rot * 4 : 0;
  // Heads per block: all of a token's, or as many as leave each of four CTAs room for one token; a norm over
  // the row keeps each operand whole (at most 128 KB: heads * d <= 2^16).  Rows of 28 to 56 KB have one
  // stage, and the other CTAs' copies run meanwhile (8192 tokens of 64 + 64 + 64 heads of 128 appended, BF16: 141 us,
  // 0.89 of the measured copy).
  int seg = heads, blocks_y = 1;
  const int fit = std::max(1, (kMaxSmem / 4 - table) / (p.d * 2));
  if (heads > fit) {
    if (p.row_norm) {
      seg = std::max(p.q.heads, p.k.heads);
      blocks_y = (p.q.heads ? 1 : 0) + (p.k.heads ? (kCache ? 2 : 1) : 0);
      p.seg_heads = -1;
    } else {
      blocks_y = (heads + fit - 1) / fit;
      seg = (heads + blocks_y - 1) / blocks_y;
      p.seg_heads = seg;
    }
  }
  p.stage_bytes = seg * p.d * 2 + table;
  const int lanes = seg * p.lanes;
  const int passes = (lanes + mxq::kRopeMaxThreads - 1) / mxq::kRopeMaxThreads;
  const int threads = std::min(mxq::kRopeMaxThreads, ((seg + passes - 1) / passes * p.lanes + 31) / 32 * 32);
  // short rows need more CTAs per SM, for the threads
  const int per_sm = std::min(8, std::max(mxq::kRopeCtas, 1024 / (threads + 32)));
  p.stages = std::min(mxq::kRopeMaxStages, std::max(1, (kMaxSmem / per_sm - 1024) / p.stage_bytes));
  const int64_t grid = std::min<int64_t>(p.T, std::max(1, per_sm * dev.sm_count / blocks_y));
  return launch_dependent(kernel, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(blocks_y)),
                          dim3(static_cast<unsigned>(threads + 32)), p.stages * p.stage_bytes, stream, p, a);
}

template <int kCache>
mxq_status launch_rope_cache(const DeviceInfo& dev, const mxq_norm_rope* cfg, mxq::RopeParams p,
                             const mxq::AppendParams& a, cudaStream_t stream) {
  p.inv_q = p.q.heads ? 1.0f / static_cast<float>(p.q.heads * p.d) : 0.f;
  p.inv_k = p.k.heads ? 1.0f / static_cast<float>(p.k.heads * p.d) : 0.f;
  return cfg->style == MXQ_ROPE_PAIRS ? launch_rope_cache_as<kCache, true>(dev, p, a, stream)
                                      : launch_rope_cache_as<kCache, false>(dev, p, a, stream);
}

// 5-D tensor map over a paged cache: (128-byte piece of a head, token, piece, head, page).
// A box: box_tokens tokens of one head of one page, one piece or (whole) all.
bool make_tmap_cache(CUtensorMap* m, const mxq_paged_kv* c, const void* base, int box_tokens, bool whole) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const bool fp8 = c->fmt == MXQ_KV_FP8_E4M3;
  const uint64_t size = fp8 ? 1 : 2;
  const uint64_t row = static_cast<uint64_t>(c->d) * size, piece = row > 128 ? 128 : row;
  const cuuint64_t dims[5] = {piece / size, static_cast<cuuint64_t>(c->page_size), row / piece,
                              static_cast<cuuint64_t>(c->heads), static_cast<cuuint64_t>(c->num_pages)};
  const cuuint64_t strides[4] = {c->stride_token * size, piece, c->stride_head * size, c->stride_page * size};
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(piece / size), static_cast<cuuint32_t>(box_tokens),
                             whole ? static_cast<cuuint32_t>(row / piece) : 1, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            piece == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace of the paged attention: the parts of units that several CTAs share.
struct PagedWorkspace {
  int64_t o = 0, ml = 0, units = 0, bytes = 0;
};

constexpr int kPagedMaxCtas = 160;  // at least the SMs of any sm_100 device
static_assert(mxq::dec_workers(kPagedMaxCtas) < 4096, "a unit's parts are counted in 12 bits");

PagedWorkspace paged_workspace(int tile_rows, int64_t d) {
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  const int64_t workers = kPagedMaxCtas * (tile_rows == mxq::kChunkRows ? 1 : mxq::kDecWarps);
  PagedWorkspace w;
  w.ml = up(2 * workers * tile_rows * d * 4);
  w.units = w.ml + up(2 * workers * tile_rows * 8);
  w.bytes = w.units + up(workers * 16);
  return w;
}

// Which kernel, by the rows that share a key head: the few-row one streams the cache once per row tile of
// 8 or 16 rows, the other computes 256 whether they are there or not.  24 sequences of 4000 keys,
// 8 key heads, d = 128, BF16 (E4M3): 16 rows 84 (64) us against 92 (103) us, 32 rows 99 (92) against 93
// (103); four sequences of 1000 keys: 16 rows 26 (22) us against 18 (21), 32 rows 26 (23) against 18
// (21).  By the mean over the sequences, since the lengths are on the device: every kernel is right
// for any, but in a mixed call some sequences have the slower one (tokens of 2000 keys beside a chunk behind
// 2000, 32 / 8 heads, one call against two: 255 + one of 512, few-row kernel, BF16 355 against 332 + 43 us, E4M3
// 323 against 173 + 52; 63 + one of 2048, many-row kernel, 254 against 94 + 126, 293 against 57 + 145).
int paged_tile_rows(int64_t T, int64_t batch, int64_t G) {
  const int64_t rows = (T * G + batch - 1) / batch;
  if (rows <= 8) return 8;
  return rows <= 16 || G > mxq::kChunkHalf ? 16 : mxq::kChunkRows;
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <int D, bool kFp8, int kNt>
mxq_status launch_paged_decode(const DeviceInfo& dev, const mxq_paged_kv* c, mxq::PagedParams p,
                               cudaStream_t stream) {
  using S = mxq::DecShape<D, kFp8>;
  const int ctas = std::min(dev.sm_count, kPagedMaxCtas);
  if (!mxq::dec_covers(ctas, p.Hk)) return MXQ_ERR_UNSUPPORTED;
  auto kernel = mxq::paged_decode_kernel<D, kFp8, kNt>;
  static PerDevice setup;
  if (!setup.ensure(dev.index, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes) == cudaSuccess;
      }))
    return MXQ_ERR_CUDA;
  p.workers = mxq::dec_workers(ctas);
  p.page_box = gcd(p.page_size, S::kKeys);
  CUtensorMap tk, tv;
  if (!make_tmap_cache(&tk, c, c->k, p.page_box, true) || !make_tmap_cache(&tv, c, c->v, p.page_box, true))
    return MXQ_ERR_CUDA;
  mxq_status st = launch_dependent(kernel, dim3(static_cast<unsigned>(ctas)), dim3(mxq::kDecThreads), S::kSmemBytes,
                                   stream, tk, tv, p);
  if (st != MXQ_OK) return st;
  // Few sequences begin in few CTAs, whose units need more blocks (8000 keys of one sequence, 32 / 8 heads:
  // 27 us with 8, 22 with 16); for many, more blocks only take longer to start (64 of 1000 keys: 52, 53).
  const unsigned join_blocks = p.batch <= 8 ? 16 : 8;
  return launch_dependent(mxq::paged_join_few_kernel<D, mxq::kDecWarps>, dim3(static_cast<unsigned>(ctas), join_blocks),
                          dim3(256), 0, stream, p);
}

// Q as (128-byte piece, piece, head, token): a box is one piece of the G heads of whole tokens.
bool make_tmap_q(CUtensorMap* m, const mxq::PagedParams& p, int64_t d, int tokens) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(d / 64), static_cast<cuuint64_t>(p.Hk) * p.G,
                              static_cast<cuuint64_t>(p.T)};
  const cuuint64_t strides[3] = {128, static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(p.ldq) * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(p.q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kFp8>
mxq_status launch_paged_chunk(const DeviceInfo& dev, const mxq_paged_kv* c, mxq::PagedParams p, cudaStream_t stream) {
  using S = mxq::ChunkShape<D, kFp8>;
  auto kernel = mxq::paged_chunk_kernel<D, kFp8>;
  static PerDevice setup;
  if (!setup.ensure(dev.index, [&] {
        // the register split must be covered by what the kernel is launched with: setmaxnreg waits otherwise
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, kernel) == cudaSuccess && a.numRegs == S::kLaunchRegs &&
               cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes) == cudaSuccess;
      }))
    return MXQ_ERR_CUDA;
  p.workers = std::min(dev.sm_count, kPagedMaxCtas);
  const int tokens = mxq::kChunkHalf / p.G;  // whole tokens of a half
  p.tile_rows = 2 * tokens * p.G;
  p.page_box = gcd(p.page_size, mxq::kChunkKeys);
  CUtensorMap tq, tk, tv;
  if (!make_tmap_q(&tq, p, D, tokens) || !make_tmap_cache(&tk, c, c->k, p.page_box, false) ||
      !make_tmap_cache(&tv, c, c->v, p.page_box, false))
    return MXQ_ERR_CUDA;
  mxq_status st = launch_dependent(kernel, dim3(static_cast<unsigned>(p.workers)), dim3(S::kThreads), S::kSmemBytes,
                                   stream, tq, tk, tv, p);
  if (st != MXQ_OK) return st;
  return launch_dependent(mxq::paged_join_many_kernel<D, mxq::kChunkRows, kPagedMaxCtas>,
                          dim3(static_cast<unsigned>(p.workers), 16), dim3(2 * D), 0, stream, p);
}

template <int D, bool kFp8>
mxq_status launch_paged(const DeviceInfo& dev, const mxq_paged_kv* c, const mxq::PagedParams& p, cudaStream_t stream) {
  if (p.tile_rows == mxq::kChunkRows) return launch_paged_chunk<D, kFp8>(dev, c, p, stream);
  return p.tile_rows == 8 ? launch_paged_decode<D, kFp8, 1>(dev, c, p, stream)
                          : launch_paged_decode<D, kFp8, 2>(dev, c, p, stream);
}

}  // namespace

extern "C" {

const char* mxq_status_string(mxq_status s) {
  switch (s) {
    case MXQ_OK: return "MXQ_OK";
    case MXQ_ERR_INVALID_ARG: return "MXQ_ERR_INVALID_ARG";
    case MXQ_ERR_SHAPE: return "MXQ_ERR_SHAPE";
    case MXQ_ERR_ALIGN: return "MXQ_ERR_ALIGN";
    case MXQ_ERR_UNSUPPORTED: return "MXQ_ERR_UNSUPPORTED";
    case MXQ_ERR_CUDA: return "MXQ_ERR_CUDA";
    case MXQ_ERR_TIMEOUT: return "MXQ_ERR_TIMEOUT";
  }
  return "MXQ_ERR_UNKNOWN";
}

int64_t mxq_sf_bytes(int64_t rows, int64_t K) {
  if (rows < 1 || K < 32 || K % 32 != 0) return -1;
  return (rows + 127) / 128 * 128 * ((K / 32 + 3) / 4 * 4);
}

mxq_status mxq_quantize_act(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, mxq_act_format fmt,
                            mxq_scale_rule rule, int hadamard128, float act_scale, void* q_out, void* sf_out,
                            mxq_stream_t stream) {
  if (fmt == MXQ_ACT_FP8_E4M3) {
    if (!x_bf16 || !q_out || sf_out) return MXQ_ERR_INVALID_ARG;
    if (rule != MXQ_SCALE_OCP || hadamard128) return MXQ_ERR_INVALID_ARG;
    if (!(act_scale > 0.f) || !std::isfinite(act_scale)) return MXQ_ERR_INVALID_ARG;
    if (M < 1 || M > (int64_t(1) << 31) || K < 32 || K % 32 != 0 || K > (int64_t(1) << 22)) return MXQ_ERR_SHAPE;
    if (ldx < K || ldx % 8 != 0) return MXQ_ERR_ALIGN;
    if (!aligned(x_bf16, 16) || !aligned(q_out, 16)) return MXQ_ERR_ALIGN;
    const float inv = 1.0f / act_scale;  // fl32(1 / s), IEEE division on the host
    if (!std::isfinite(inv)) return MXQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    mxq_status st = current_device(&dev);
    if (st != MXQ_OK) return st;
    // grid.x: groups of 64 chunk columns (K <= 2^22: at most 4096); grid.y: groups of
    // kFp8Rows rows, at most 65535 (the kernel strides over the rest)
    const int64_t gx = (K / 16 + 63) / 64;
    const int64_t gy = std::min<int64_t>((M + mxq::kFp8Rows - 1) / mxq::kFp8Rows, 65535);
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
    mxq::quantize_act_fp8_kernel<<<grid, mxq::kQuantThreads, 0, stream>>>(
        static_cast<const uint16_t*>(x_bf16), M, K, ldx, inv, static_cast<uint8_t*>(q_out));
    return launch_status();
  }
  if (fmt != MXQ_ACT_MXFP4) return MXQ_ERR_INVALID_ARG;
  mxq_status st = check_quant_args(x_bf16, M, K, ldx, rule, hadamard128, q_out, sf_out);
  if (st != MXQ_OK) return st;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != MXQ_OK) return st;
  return launch_mxfp4(false, x_bf16, M, K, ldx, rule, hadamard128, q_out, sf_out, stream);
}

mxq_status mxq_pack_weight(const void* w_bf16, int64_t N, int64_t K, int64_t ldw, mxq_scale_rule rule,
                           int hadamard128, void* codes_out, void* sf_out, mxq_stream_t stream) {
  mxq_status st = check_quant_args(w_bf16, N, K, ldw, rule, hadamard128, codes_out, sf_out);
  if (st != MXQ_OK) return st;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != MXQ_OK) return st;
  return launch_mxfp4(true, w_bf16, N, K, ldw, rule, hadamard128, codes_out, sf_out, stream);
}

mxq_status mxq_gemm_w4a4(const void* a_codes, const void* a_sf, const void* b_codes, const void* b_sf, int64_t M,
                         int64_t N, int64_t K, float alpha, const void* bias_bf16, void* d_bf16, int64_t ldd,
                         mxq_stream_t stream) {
  if (!a_sf) return MXQ_ERR_INVALID_ARG;
  if (!std::isfinite(alpha)) return MXQ_ERR_INVALID_ARG;
  mxq_status st = check_gemm_shapes(a_codes, b_codes, b_sf, d_bf16, M, N, K, ldd, bias_bf16);
  if (st != MXQ_OK) return st;
  if (!aligned(a_sf, 16)) return MXQ_ERR_ALIGN;
  return launch_gemm<false>(a_codes, a_sf, b_codes, b_sf, M, N, K, alpha, bias_bf16, d_bf16, ldd, stream);
}

mxq_status mxq_gemm_w4a8(const void* a_e4m3, float act_scale, const void* b_codes, const void* b_sf, int64_t M,
                         int64_t N, int64_t K, const void* bias_bf16, void* d_bf16, int64_t ldd,
                         mxq_stream_t stream) {
  if (!(act_scale > 0.f) || !std::isfinite(act_scale)) return MXQ_ERR_INVALID_ARG;
  mxq_status st = check_gemm_shapes(a_e4m3, b_codes, b_sf, d_bf16, M, N, K, ldd, bias_bf16);
  if (st != MXQ_OK) return st;
  if (!aligned(b_codes, 32)) return MXQ_ERR_ALIGN;  // 16U4_ALIGN16B tensor maps need 32-byte bases
  return launch_gemm<true>(a_e4m3, nullptr, b_codes, b_sf, M, N, K, act_scale, bias_bf16, d_bf16, ldd, stream);
}

mxq_status mxq_dequant_mxfp4(const void* codes, const void* sf, int64_t rows, int64_t K, void* out_bf16,
                             int64_t ldo, mxq_stream_t stream) {
  if (!codes || !sf || !out_bf16) return MXQ_ERR_INVALID_ARG;
  if (rows < 1 || rows > (int64_t(1) << 31) || K < 32 || K % 32 != 0 || K > (int64_t(1) << 22)) return MXQ_ERR_SHAPE;
  if (ldo < K || ldo % 8 != 0) return MXQ_ERR_ALIGN;
  if (!aligned(codes, 16) || !aligned(out_bf16, 16)) return MXQ_ERR_ALIGN;
  DeviceInfo dev;
  mxq_status st = current_device(&dev);
  if (st != MXQ_OK) return st;
  const int64_t units = rows * (K / 16);
  const int64_t per_block = int64_t(mxq::kQuantThreads) * mxq::kDequantUnroll;
  int64_t blocks = (units + per_block - 1) / per_block;
  // Grid-stride: exactly the CTAs that fit at once, so none starts late (a second, partial
  // round of a latency-bound kernel costs as much as a full one).
  static PerDevice setup;
  static int resident_of[kMaxDevices];
  setup.ensure(dev.index, [&] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, mxq::dequant_mxfp4_kernel, mxq::kQuantThreads, 0) !=
            cudaSuccess || n < 1)
      return false;
    resident_of[dev.index] = n;
    return true;
  });
  const int resident = resident_of[dev.index] > 0 ? resident_of[dev.index] : 1;
  const int64_t cap = static_cast<int64_t>(dev.sm_count) * resident;
  if (blocks > cap) blocks = cap;
  mxq::dequant_mxfp4_kernel<<<static_cast<unsigned>(blocks), mxq::kQuantThreads, 0, stream>>>(
      static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(sf), rows, K,
      static_cast<uint16_t*>(out_bf16), ldo);
  return launch_status();
}

mxq_status mxq_qdq_act(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, mxq_act_format fmt,
                       mxq_scale_rule rule, int hadamard128, float act_scale, void* out_bf16, int64_t ldo,
                       mxq_stream_t stream) {
  if (!x_bf16 || !out_bf16) return MXQ_ERR_INVALID_ARG;
  if (fmt != MXQ_ACT_MXFP4 && fmt != MXQ_ACT_FP8_E4M3) return MXQ_ERR_INVALID_ARG;
  if (rule != MXQ_SCALE_OCP && rule != MXQ_SCALE_UOS) return MXQ_ERR_INVALID_ARG;
  float inv = 0.f;
  if (fmt == MXQ_ACT_FP8_E4M3) {
    if (rule != MXQ_SCALE_OCP || hadamard128) return MXQ_ERR_INVALID_ARG;
    if (!(act_scale > 0.f) || !std::isfinite(act_scale)) return MXQ_ERR_INVALID_ARG;
    inv = 1.0f / act_scale;  // fl32(1 / s), as in the quantiser
    if (!std::isfinite(inv)) return MXQ_ERR_INVALID_ARG;
  }
  const int64_t max_rows = fmt == MXQ_ACT_FP8_E4M3 ? (int64_t(1) << 31) : int64_t(65535) * 128;
  if (M < 1 || M > max_rows || K < 32 || K % 32 != 0 || K > (int64_t(1) << 22)) return MXQ_ERR_SHAPE;
  if (hadamard128 && K % 128 != 0) return MXQ_ERR_SHAPE;
  if (ldx < K || ldx % 8 != 0 || ldo < K || ldo % 8 != 0) return MXQ_ERR_ALIGN;
  if (!aligned(x_bf16, 16) || !aligned(out_bf16, 16)) return MXQ_ERR_ALIGN;
  DeviceInfo dev;
  mxq_status st = current_device(&dev);
  if (st != MXQ_OK) return st;
  const auto* xp = static_cast<const uint16_t*>(x_bf16);
  auto* op = static_cast<uint16_t*>(out_bf16);
  if (fmt == MXQ_ACT_FP8_E4M3) {
    const int64_t chunks = M * (K / 16);
    int64_t blocks = (chunks + mxq::kQuantThreads - 1) / mxq::kQuantThreads;
    const int64_t cap = static_cast<int64_t>(dev.sm_count) * 16;
    if (blocks > cap) blocks = cap;
    mxq::qdq_act_fp8_kernel<<<static_cast<unsigned>(blocks), mxq::kQuantThreads, 0, stream>>>(xp, M, K, ldx, inv,
                                                                                             act_scale, op, ldo);
    return launch_status();
  }
  const dim3 grid(static_cast<unsigned>((K + 127) / 128), static_cast<unsigned>((M + 127) / 128));
  const int sel = (hadamard128 ? 2 : 0) | (rule == MXQ_SCALE_UOS ? 1 : 0);
  switch (sel) {
    case 0: mxq::qdq_act_mxfp4_kernel<false, false><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, M, K, ldx, op, ldo); break;
    case 1: mxq::qdq_act_mxfp4_kernel<false, true><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, M, K, ldx, op, ldo); break;
    case 2: mxq::qdq_act_mxfp4_kernel<true, false><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, M, K, ldx, op, ldo); break;
    default: mxq::qdq_act_mxfp4_kernel<true, true><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, M, K, ldx, op, ldo); break;
  }
  return launch_status();
}

mxq_status mxq_channel_absmax(const void* x_bf16, int64_t rows, int64_t K, int64_t ldx, int hadamard128,
                              int accumulate, float* amax_out, mxq_stream_t stream) {
  if (!amax_out) return MXQ_ERR_INVALID_ARG;
  // same tiling and limits as the quantiser (the scale pointers are not used)
  mxq_status st = check_quant_args(x_bf16, rows, K, ldx, MXQ_SCALE_OCP, hadamard128, amax_out, amax_out);
  if (st != MXQ_OK) return st;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != MXQ_OK) return st;
  if (!accumulate && cudaMemsetAsync(amax_out, 0, static_cast<size_t>(K) * sizeof(float), stream) != cudaSuccess)
    return MXQ_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>((K + 127) / 128), static_cast<unsigned>((rows + 127) / 128));
  const auto* xp = static_cast<const uint16_t*>(x_bf16);
  if (hadamard128)
    mxq::channel_absmax_kernel<true><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ldx, amax_out);
  else
    mxq::channel_absmax_kernel<false><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ldx, amax_out);
  return launch_status();
}

mxq_status mxq_smooth_factors(const float* amax_x, const float* amax_w, int64_t K, float alpha, float* lambda_out,
                              float* inv_lambda_out, mxq_stream_t stream) {
  if (!amax_x || !amax_w || !lambda_out || !inv_lambda_out) return MXQ_ERR_INVALID_ARG;
  if (!(alpha >= 0.f && alpha <= 1.f)) return MXQ_ERR_INVALID_ARG;
  if (K < 1 || K > (int64_t(1) << 22)) return MXQ_ERR_SHAPE;
  DeviceInfo dev;
  mxq_status st = current_device(&dev);
  if (st != MXQ_OK) return st;
  const unsigned blocks = static_cast<unsigned>((K + 255) / 256);
  mxq::smooth_factors_kernel<<<blocks, 256, 0, stream>>>(amax_x, amax_w, K, alpha, lambda_out, inv_lambda_out);
  return launch_status();
}

mxq_status mxq_quantize_smooth(const void* x_bf16, int64_t rows, int64_t K, int64_t ldx, mxq_scale_rule rule,
                               int hadamard128, const float* chan_scale, void* codes_out, void* sf_out,
                               mxq_stream_t stream) {
  if (!chan_scale) return MXQ_ERR_INVALID_ARG;
  mxq_status st = check_quant_args(x_bf16, rows, K, ldx, rule, hadamard128, codes_out, sf_out);
  if (st != MXQ_OK) return st;
  if (!aligned(chan_scale, 16)) return MXQ_ERR_ALIGN;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != MXQ_OK) return st;
  const dim3 grid(static_cast<unsigned>((K + 127) / 128), static_cast<unsigned>((rows + 127) / 128));
  const auto* xp = static_cast<const uint16_t*>(x_bf16);
  auto* cp = static_cast<uint8_t*>(codes_out);
  auto* sp = static_cast<uint8_t*>(sf_out);
  const int sel = (hadamard128 ? 2 : 0) | (rule == MXQ_SCALE_UOS ? 1 : 0);
  switch (sel) {
    case 0: mxq::quantize_smooth_mxfp4_kernel<false, false><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ldx, chan_scale, cp, sp); break;
    case 1: mxq::quantize_smooth_mxfp4_kernel<false, true><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ldx, chan_scale, cp, sp); break;
    case 2: mxq::quantize_smooth_mxfp4_kernel<true, false><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ldx, chan_scale, cp, sp); break;
    default: mxq::quantize_smooth_mxfp4_kernel<true, true><<<grid, mxq::kQuantThreads, 0, stream>>>(xp, rows, K, ldx, chan_scale, cp, sp); break;
  }
  return launch_status();
}

mxq_status mxq_sqnr_accumulate(const void* y_bf16, int64_t ldy, const void* ref_bf16, int64_t ldr, int64_t M,
                               int64_t N, int accumulate, double* acc, mxq_stream_t stream) {
  if (!y_bf16 || !ref_bf16 || !acc) return MXQ_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || M > (int64_t(1) << 31) || N > (int64_t(1) << 31)) return MXQ_ERR_SHAPE;
  if (ldy < N || ldr < N || ldy % 8 != 0 || ldr % 8 != 0) return MXQ_ERR_ALIGN;
  if (!aligned(y_bf16, 16) || !aligned(ref_bf16, 16) || !aligned(acc, 8)) return MXQ_ERR_ALIGN;
  DeviceInfo dev;
  mxq_status st = current_device(&dev);
  if (st != MXQ_OK) return st;
  if (!accumulate && cudaMemsetAsync(acc, 0, 2 * sizeof(double), stream) != cudaSuccess) return MXQ_ERR_CUDA;
  const int64_t chunks = M * ((N + 7) / 8);
  int64_t blocks = (chunks + mxq::kSqnrThreads - 1) / mxq::kSqnrThreads;
  const int64_t cap = static_cast<int64_t>(dev.sm_count) * 8;
  if (blocks > cap) blocks = cap;
  mxq::sqnr_sums_kernel<<<static_cast<unsigned>(blocks), mxq::kSqnrThreads, 0, stream>>>(
      static_cast<const uint16_t*>(y_bf16), ldy, static_cast<const uint16_t*>(ref_bf16), ldr, M, N, acc);
  return launch_status();
}

double mxq_sqnr_db(double signal, double noise) {
  if (!(noise > 0.0)) return HUGE_VAL;
  if (!(signal > 0.0)) return -HUGE_VAL;
  return 10.0 * std::log10(signal / noise);
}

mxq_precision mxq_select_precision(double sqnr_plain_db, double sqnr_transform_db, double high_db,
                                   double low_db) {
  if (sqnr_plain_db >= high_db) return MXQ_PREC_W4A4;
  if (sqnr_transform_db >= high_db) return MXQ_PREC_W4A4_TRANSFORM;
  if ((sqnr_plain_db > sqnr_transform_db ? sqnr_plain_db : sqnr_transform_db) >= low_db) return MXQ_PREC_W4A8;
  return MXQ_PREC_BF16;
}

void mxq_attn_code_poly(float coeffs[4]) {
  if (!coeffs) return;
  coeffs[0] = 1.0f;
  coeffs[1] = mxq::kCodeA1;
  coeffs[2] = mxq::kCodeA2;
  coeffs[3] = mxq::kCodeA3;
}

int64_t mxq_attn_padded_keys(int64_t S_kv) {
  if (S_kv < 1 || S_kv > (int64_t(1) << 23)) return -1;
  return (S_kv + mxq::kAttnBN - 1) / mxq::kAttnBN * mxq::kAttnBN;
}

mxq_status mxq_quantize_vt(const void* v_bf16, int64_t S, int64_t HD, int64_t ldv, mxq_scale_rule rule,
                           void* codes_out, void* sf_out, mxq_stream_t stream) {
  if (!v_bf16 || !codes_out || !sf_out) return MXQ_ERR_INVALID_ARG;
  if (rule != MXQ_SCALE_OCP && rule != MXQ_SCALE_UOS) return MXQ_ERR_INVALID_ARG;
  const int64_t Sp = mxq_attn_padded_keys(S);
  if (Sp < 0 || HD < 128 || HD % 128 != 0 || HD > (int64_t(1) << 16)) return MXQ_ERR_SHAPE;
  if (ldv < HD || ldv % 8 != 0) return MXQ_ERR_ALIGN;
  if (!aligned(v_bf16, 16) || !aligned(codes_out, 16)) return MXQ_ERR_ALIGN;
  DeviceInfo dev;
  mxq_status st = current_device(&dev);
  if (st != MXQ_OK) return st;
  const dim3 grid(static_cast<unsigned>(HD / 128), static_cast<unsigned>(Sp / 128));
  const auto* vp = static_cast<const uint16_t*>(v_bf16);
  auto* cp = static_cast<uint8_t*>(codes_out);
  auto* sp = static_cast<uint8_t*>(sf_out);
  if (rule == MXQ_SCALE_UOS)
    mxq::quantize_vt_kernel<true><<<grid, 256, 0, stream>>>(vp, S, ldv, Sp, cp, sp);
  else
    mxq::quantize_vt_kernel<false><<<grid, 256, 0, stream>>>(vp, S, ldv, Sp, cp, sp);
  return launch_status();
}

mxq_status mxq_attention_mxfp4(const void* q_codes, const void* q_sf, const void* k_codes, const void* k_sf,
                               const void* vt_codes, const void* vt_sf, int64_t S_q, int64_t S_kv, int64_t H,
                               int64_t d, mxq_scale_rule rule, void* out_bf16, int64_t ldo, mxq_stream_t stream) {
  if (!q_codes || !q_sf || !k_codes || !k_sf || !vt_codes || !vt_sf || !out_bf16) return MXQ_ERR_INVALID_ARG;
  if (rule != MXQ_SCALE_OCP && rule != MXQ_SCALE_UOS) return MXQ_ERR_INVALID_ARG;
  if (d != mxq::kAttnD) return MXQ_ERR_UNSUPPORTED;
  const int64_t Sp = mxq_attn_padded_keys(S_kv);
  if (Sp < 0 || S_q < 1 || S_q > (int64_t(65535) * mxq::kAttnBM) || H < 1 || H > 65535 || H * d > (int64_t(1) << 16))
    return MXQ_ERR_SHAPE;
  const int64_t HD = H * d;
  if (ldo < HD || ldo % 8 != 0) return MXQ_ERR_ALIGN;
  if (!aligned(q_codes, 16) || !aligned(k_codes, 16) || !aligned(vt_codes, 16) || !aligned(q_sf, 16) ||
      !aligned(k_sf, 16) || !aligned(vt_sf, 16) || !aligned(out_bf16, 16))
    return MXQ_ERR_ALIGN;
  DeviceInfo dev;
  mxq_status st = current_device(&dev);
  if (st != MXQ_OK) return st;

  CUtensorMap tq, tsq, tk, tsk, tv, tsv;
  const bool ok =
      make_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, q_codes, HD / 2, S_q, HD / 2, 64, mxq::kAttnBM,
                   CU_TENSOR_MAP_SWIZZLE_64B) &&
      make_tmap_sf(&tsq, q_sf, S_q, HD, 1, 1) &&
      make_tmap_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, k_codes, HD / 2, S_kv, HD / 2, 64, mxq::kAttnBN,
                   CU_TENSOR_MAP_SWIZZLE_64B) &&
      make_tmap_sf(&tsk, k_sf, S_kv, HD, 1, 2) &&
      make_tmap_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, vt_codes, Sp / 2, HD, Sp / 2, 128, mxq::kAttnD,
                   CU_TENSOR_MAP_SWIZZLE_128B) &&
      make_tmap_sf(&tsv, vt_sf, HD, Sp, 2, 1);
  if (!ok) return MXQ_ERR_CUDA;

  mxq::AttnParams prm;
  prm.t_scale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
  prm.Sq = static_cast<int>(S_q);
  prm.Skv = static_cast<int>(S_kv);
  prm.num_tiles = static_cast<int>(Sp / mxq::kAttnBN);

  auto kernel = rule == MXQ_SCALE_UOS ? mxq::mx_attention_kernel<true> : mxq::mx_attention_kernel<false>;
  static PerDevice setup;
  if (!setup.ensure(dev.index, [] {
        return cudaFuncSetAttribute(mxq::mx_attention_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    mxq::kAttnSmemBytes) == cudaSuccess &&
               cudaFuncSetAttribute(mxq::mx_attention_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    mxq::kAttnSmemBytes) == cudaSuccess;
      }))
    return MXQ_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>((S_q + mxq::kAttnBM - 1) / mxq::kAttnBM), static_cast<unsigned>(H));
  kernel<<<grid, mxq::kAttnThreads, mxq::kAttnSmemBytes, stream>>>(tq, tsq, tk, tsk, tv, tsv,
                                                                   static_cast<__nv_bfloat16*>(out_bf16), ldo, prm);
  return launch_status();
}

int64_t mxq_linear_workspace_bytes(int64_t M, int64_t K) {
  if (M < 1 || M > (int64_t(1) << 30) || K < 128 || K % 128 != 0 || K > (int64_t(1) << 22)) return -1;
  return linear_workspace(M, K).bytes;
}

mxq_status mxq_linear_w4a4(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, mxq_scale_rule rule,
                           const void* w_codes, const void* w_sf, int64_t N, float alpha, const void* bias_bf16,
                           void* workspace, int64_t workspace_bytes, void* d_bf16, int64_t ldd, mxq_stream_t stream) {
  if (!x_bf16 || !workspace) return MXQ_ERR_INVALID_ARG;
  if (rule != MXQ_SCALE_OCP && rule != MXQ_SCALE_UOS) return MXQ_ERR_INVALID_ARG;
  if (!std::isfinite(alpha)) return MXQ_ERR_INVALID_ARG;
  const int64_t need = mxq_linear_workspace_bytes(M, K);
  if (need < 0 || M > int64_t(65535) * 128) return MXQ_ERR_SHAPE;
  if (workspace_bytes < need) return MXQ_ERR_INVALID_ARG;
  if (ldx < K || ldx % 8 != 0 || !aligned(x_bf16, 16) || !aligned(workspace, 16)) return MXQ_ERR_ALIGN;
  const LinearWorkspace ws = linear_workspace(M, K);
  auto* base = static_cast<uint8_t*>(workspace);
  void* a_codes = base + ws.codes;
  void* a_sf = base + ws.sf;
  mxq_status st = check_gemm_shapes(a_codes, w_codes, w_sf, d_bf16, M, N, K, ldd, bias_bf16);
  if (st != MXQ_OK) return st;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != MXQ_OK) return st;
  st = launch_mxfp4(false, x_bf16, M, K, ldx, rule, 0, a_codes, a_sf, stream);
  if (st != MXQ_OK) return st;
  return launch_gemm<false>(a_codes, a_sf, w_codes, w_sf, M, N, K, alpha, bias_bf16, d_bf16, ldd, stream);
}

mxq_status mxq_linear_w4a4_static(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, mxq_scale_rule rule,
                                  const void* w_codes, const void* w_sf, int64_t N, float alpha,
                                  const void* bias_bf16, void* d_bf16, int64_t ldd, mxq_stream_t stream) {
  const int64_t need = mxq_linear_workspace_bytes(M, K);
  if (need < 0 || need > kStaticScratchBytes) return MXQ_ERR_SHAPE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return MXQ_ERR_CUDA;
  void* scratch = static_scratch(dev);
  if (!scratch) return MXQ_ERR_CUDA;
  // Nothing in the scratch has to start at zero: the quantiser writes every byte the GEMM
  // reads (codes of all M rows, whole scale atoms including their padding).
  return mxq_linear_w4a4(x_bf16, M, K, ldx, rule, w_codes, w_sf, N, alpha, bias_bf16, scratch, kStaticScratchBytes,
                         d_bf16, ldd, stream);
}

mxq_status mxq_qk_norm_rope(const mxq_norm_rope* cfg, int64_t T, int64_t d, const void* q_bf16, int64_t Hq,
                            int64_t ldq, void* q_out, int64_t ldqo, const void* k_bf16, int64_t Hk, int64_t ldk,
                            void* k_out, int64_t ldko, const int32_t* positions, mxq_stream_t stream) {
  mxq_status st = check_norm_rope(cfg, d);
  if (st != MXQ_OK) return st;
  if ((!q_bf16 && !k_bf16) || (q_bf16 && !q_out) || (k_bf16 && !k_out)) return MXQ_ERR_INVALID_ARG;
  if (T < 1 || T > INT32_MAX) return MXQ_ERR_SHAPE;
  if (q_bf16 && ((st = check_heads(q_bf16, Hq, d, ldq)) != MXQ_OK || (st = check_heads(q_out, Hq, d, ldqo)) != MXQ_OK))
    return st;
  if (k_bf16 && ((st = check_heads(k_bf16, Hk, d, ldk)) != MXQ_OK || (st = check_heads(k_out, Hk, d, ldko)) != MXQ_OK))
    return st;
  if (!aligned(positions, 4)) return MXQ_ERR_ALIGN;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != MXQ_OK) return st;
  mxq::RopeParams p = rope_params(cfg, T, d);
  p.q = rope_operand(q_bf16, cfg->q_weight, ldq, q_out, ldqo, Hq);
  p.k = rope_operand(k_bf16, cfg->k_weight, ldk, k_out, ldko, Hk);
  p.positions = positions;
  return launch_rope_cache<0>(dev, cfg, p, mxq::AppendParams{}, stream);
}

mxq_status mxq_kv_append(const mxq_norm_rope* cfg, const mxq_paged_kv* cache, const mxq_paged_batch* batch, int64_t T,
                         const void* k_bf16, int64_t ldk, const void* v_bf16, int64_t ldv, const void* q_bf16,
                         int64_t Hq, int64_t ldq, void* q_out, int64_t ldqo, mxq_stream_t stream) {
  mxq_status st = check_paged(cache, batch);
  if (st != MXQ_OK) return st;
  const int64_t d = cache->d;
  if ((st = check_norm_rope(cfg, d)) != MXQ_OK) return st;
  if (!k_bf16 || !v_bf16 || (q_bf16 && !q_out)) return MXQ_ERR_INVALID_ARG;
  if (T < 1 || T > INT32_MAX) return MXQ_ERR_SHAPE;
  if ((st = check_heads(k_bf16, cache->heads, d, ldk)) != MXQ_OK || (st = check_heads(v_bf16, cache->heads, d, ldv)) != MXQ_OK)
    return st;
  if (q_bf16 && ((st = check_heads(q_bf16, Hq, d, ldq)) != MXQ_OK || (st = check_heads(q_out, Hq, d, ldqo)) != MXQ_OK))
    return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != MXQ_OK) return st;
  mxq::RopeParams p = rope_params(cfg, T, d);
  p.q = rope_operand(q_bf16, cfg->q_weight, ldq, q_out, ldqo, Hq);
  p.k = rope_operand(k_bf16, cfg->k_weight, ldk, nullptr, 0, cache->heads);
  p.v = static_cast<const uint16_t*>(v_bf16);
  p.ldv = ldv;
  mxq::AppendParams a = {};
  a.cu_q = batch->cu_q;
  a.kv_len = batch->kv_len;
  a.block_table = batch->block_table;
  a.table_stride = batch->max_pages;
  a.batch = static_cast<int>(batch->batch);
  a.k_cache = cache->k;
  a.v_cache = cache->v;
  a.stride_page = cache->stride_page;
  a.stride_token = cache->stride_token;
  a.stride_head = cache->stride_head;
  a.num_pages = static_cast<int>(cache->num_pages);
  a.page_size = static_cast<int>(cache->page_size);
  a.k_inv_scale = 1.0f / cache->k_scale;
  a.v_inv_scale = 1.0f / cache->v_scale;
  return cache->fmt == MXQ_KV_BF16 ? launch_rope_cache<1>(dev, cfg, p, a, stream) : launch_rope_cache<2>(dev, cfg, p, a, stream);
}

int64_t mxq_attention_paged_workspace_bytes(int64_t T, int64_t batch, int64_t Hq, int64_t Hk, int64_t d) {
  if (T < 1 || batch < 1 || Hk < 1 || Hq < Hk || Hq % Hk != 0 || (d != 64 && d != 128)) return -1;
  return paged_workspace(paged_tile_rows(T, batch, Hq / Hk), d).bytes;
}

mxq_status mxq_attention_paged(const void* q_bf16, int64_t T, int64_t Hq, int64_t ldq, const mxq_paged_kv* cache,
                               const mxq_paged_batch* batch, int causal, int64_t window, float scale, void* workspace,
                               int64_t workspace_bytes, void* out_bf16, int64_t ldo, mxq_stream_t stream) {
  mxq_status st = check_paged(cache, batch);
  if (st != MXQ_OK) return st;
  if (!q_bf16 || !out_bf16 || !workspace) return MXQ_ERR_INVALID_ARG;
  if (!(scale >= 0.f) || !std::isfinite(scale) || window < 0 || (window > 0 && !causal)) return MXQ_ERR_INVALID_ARG;
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * cache->k_scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return MXQ_ERR_INVALID_ARG;
  const int64_t d = cache->d, Hk = cache->heads;
  if (d != 64 && d != 128) return MXQ_ERR_UNSUPPORTED;
  if (T < 1 || Hq < 1 || Hq % Hk != 0 || T * Hq > (int64_t(1) << 30) || T > (int64_t(1) << 30)) return MXQ_ERR_SHAPE;
  if (window > (int64_t(1) << 30)) return MXQ_ERR_SHAPE;
  if ((st = check_heads(q_bf16, Hq, d, ldq)) != MXQ_OK || (st = check_heads(out_bf16, Hq, d, ldo)) != MXQ_OK) return st;
  if (!aligned(workspace, 256)) return MXQ_ERR_ALIGN;
  if (workspace_bytes < mxq_attention_paged_workspace_bytes(T, batch->batch, Hq, Hk, d)) return MXQ_ERR_INVALID_ARG;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != MXQ_OK) return st;

  const int tile_rows = paged_tile_rows(T, batch->batch, Hq / Hk);
  const PagedWorkspace ws = paged_workspace(tile_rows, d);
  auto* base = static_cast<uint8_t*>(workspace);
  mxq::PagedParams p = {};
  p.q = static_cast<const uint16_t*>(q_bf16);
  p.out = static_cast<uint16_t*>(out_bf16);
  p.cu_q = batch->cu_q;
  p.kv_len = batch->kv_len;
  p.block_table = batch->block_table;
  p.part_o = reinterpret_cast<float*>(base);
  p.part_ml = reinterpret_cast<float2*>(base + ws.ml);
  p.part_units = reinterpret_cast<int4*>(base + ws.units);
  p.ldq = ldq;
  p.ldo = ldo;
  p.T = T;
  p.table_stride = batch->max_pages;
  p.batch = static_cast<int>(batch->batch);
  p.num_pages = static_cast<int>(cache->num_pages);
  p.page_size = static_cast<int>(cache->page_size);
  p.Hk = static_cast<int>(Hk);
  p.G = static_cast<int>(Hq / Hk);
  p.out32 = ldo % 16 == 0 && aligned(out_bf16, 32);  // and d % 16 == 0
  p.causal = causal != 0;
  p.window = static_cast<int>(window);
  p.tile_rows = tile_rows;
  p.scale_log2 = mxq::nonzero_scale(scale_log2);
  p.v_scale = cache->v_scale;
  const bool fp8 = cache->fmt == MXQ_KV_FP8_E4M3;
  if (d == 128)
    return fp8 ? launch_paged<128, true>(dev, cache, p, stream) : launch_paged<128, false>(dev, cache, p, stream);
  return fp8 ? launch_paged<64, true>(dev, cache, p, stream) : launch_paged<64, false>(dev, cache, p, stream);
}

mxq_status mxq_selftest_wait_timeout(mxq_stream_t stream) {
  DeviceInfo dev;
  const mxq_status st = current_device(&dev);
  if (st != MXQ_OK) return st;
  mxq::selftest_wait_timeout_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>();
  return launch_status();
}

mxq_status mxq_debug_poll(void) {
  if (cudaDeviceSynchronize() != cudaSuccess) return MXQ_ERR_CUDA;
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, mxq::g_status, sizeof v) != cudaSuccess) return MXQ_ERR_CUDA;
  if (v != 0) {
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(mxq::g_status, &zero, sizeof zero) != cudaSuccess) return MXQ_ERR_CUDA;
    return static_cast<mxq_status>(v);
  }
  return MXQ_OK;
}

}  // extern "C"
