// dq_handle.h -- the handle behind dqgemm_handle and the host helpers that the
// library's translation units share.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstdlib>
#include <mutex>

#include "dqgemm.h"

struct dqgemm_s {
  int fmt = 0, K = 0, N = 0;
  int k_stages = 0, n_tiles = 0;
  int device = 0, num_sms = 0;
  uint8_t* wchunks = nullptr;       // pre-tiled weight
  size_t wchunk_bytes = 0;
  float* col_scale = nullptr;       // [N] for FP8 formats
  __nv_bfloat16* bias = nullptr;    // [N] or null
  int* status = nullptr;            // status word as the device addresses it
  int* status_host = nullptr;       //   ... and as the host reads it (mapped pinned memory)
  float sigma = 1.f, s_x = 1.f;
  int mx_bias = 126;
  long long weight_bytes = 0;       // canonical packed + scale bytes
  // co-resident clusters per (BN index, cluster size), 0 = unknown (calls from
  // several threads may ask at once: each finds the same)
  std::atomic<int> max_clusters[4][9] = {};
  // FP4 x FP4: the activation workspace (codes, scale words, the NVFP4 amax
  // partials, ticket and g_x), grown on demand and reused by every call
  uint8_t* ws = nullptr;
  size_t ws_bytes = 0;
  unsigned long long timeout_ns = 0;  // limit of the kernels' pipeline waits
  // activation tensor maps already encoded, by (x, M, tile rows, e4m3 input):
  // encoding one costs host time on every call, and layers see the same
  // few activation buffers again and again
  struct MapEntry {
    const void* x = nullptr;
    int M = 0, bn = 0;
    bool xq = false, x3d = false;
    CUtensorMap map;
  };
  static constexpr int kMaps = 8;
  MapEntry maps[kMaps];
  int next_map = 0;
  // block-scaled FP8 (fmt == FMT_FP8B): wchunks holds the canonical codes
  // [E * N, K], col_scale the block scales [E][N / 128][K / 128] (rounded up)
  int E = 1;
  bool experts = false;             // made by dqgemm_create_experts: calls take offsets
  CUtensorMap wmap, wmap64;         // boxes of 128 k x 128 (64) rows of the codes
  std::mutex maps_mu;               // run entry points may be called from several threads
};

namespace dq {

// the handle's fmt of a block-scaled FP8 layer (the public DQ_FP8_BLOCK128;
// 8 and 9 name kernel variants here)
constexpr int FMT_FP8B = 10;

// block-scaled FP8 (dq_block_api.cu); arguments checked by the callers where
// a comment says so
dqgemm_status block_create(dqgemm_handle* out, bool experts, int E, int K, int N, const void* packed_w, const void* scales,
                           const void* bias);
dqgemm_status block_run_x(dqgemm_handle h, const void* x, int M, void* y, void* stream);
dqgemm_status block_dequantize(dqgemm_handle h, void* w_bf16, void* stream);
void block_fill_plan(dqgemm_handle h, int M, dqgemm_plan* plan);
dqgemm_status block_pack_host(const float* W, int K, int N, void* packed, void* scales);      // W finite
dqgemm_status block_pack_device(const float* W, int K, int N, void* packed, void* scales, cudaStream_t s);

constexpr unsigned long long kDefaultTimeoutNs = 2000000000ull;   // 2 s

inline unsigned long long timeout_ns() {
  static unsigned long long t = [] {
    const char* e = std::getenv("DQGEMM_TIMEOUT_MS");
    return e ? (unsigned long long)std::strtoull(e, nullptr, 10) * 1000000ull : kDefaultTimeoutNs;
  }();
  return t;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool is_device_ptr(const void* p) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// e4m3 activations [M, K] (u8, K % 16 == 0): box of 128 k x bn rows, the
// tensor core's 128-byte-swizzled K-major image
inline bool make_q_map(CUtensorMap* map, const void* q, int M, int K, int bn) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)M};
  const cuuint64_t strides[1] = {(cuuint64_t)K};
  const cuuint32_t box[2] = {128, (cuuint32_t)bn};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool pdl_enabled() {
  static bool on = [] {
    const char* e = std::getenv("DQGEMM_PDL");
    return !(e && e[0] == '0');
  }();
  return on;
}

// a small kernel in the programmatic-dependent-launch chain of the GEMMs
// (its first instruction waits for the previous grid)
template <typename... KArgs, typename... Args>
cudaError_t launch_chained(void (*kern)(KArgs...), int grid, int block, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  int na = 0;
  if (pdl_enabled()) {
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    na = 1;
  }
  cfg.attrs = a;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

inline dqgemm_status cuda_err(cudaError_t e) { return e == cudaSuccess ? DQ_OK : DQ_ERR_CUDA; }

}  // namespace dq
