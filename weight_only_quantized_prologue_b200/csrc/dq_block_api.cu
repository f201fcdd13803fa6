// dq_block_api.cu -- block-scaled FP8 layers and experts: handles, launch plan
// and the entry points of include/dqgemm.h that only they have.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "dq_block.cuh"
#include "dq_handle.h"

using namespace dq;

namespace {

constexpr int QB = 128;   // elements per scale

int blocks(int n) { return (n + QB - 1) / QB; }

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
struct BlockPlan {
  bool pair;       // block_pair_kernel, else block_skinny_kernel
  int bn;          // rows per tile
  int m_tiles, n_tiles;
  int split;
  int grid;        // CTAs
};

template <int BN, bool G, bool X>
cudaError_t skinny_attr() {
  cudaError_t e = cudaFuncSetAttribute(block_skinny_kernel<BN, G, X>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       SkinnyCfg<BN, X>::SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(block_skinny_kernel<BN, G, X>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared);
  return e;
}

template <bool G>
cudaError_t pair_attr() {
  cudaError_t e = cudaFuncSetAttribute(block_pair_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, PairCfg::SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(block_pair_kernel<G>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared);
  return e;
}

cudaError_t set_attrs() {
  cudaError_t e = cudaSuccess;
  for (cudaError_t r :
       {skinny_attr<16, false, false>(), skinny_attr<32, false, false>(), skinny_attr<64, false, false>(),
        skinny_attr<128, false, false>(), skinny_attr<16, true, false>(), skinny_attr<32, true, false>(),
        skinny_attr<64, true, false>(), skinny_attr<16, false, true>(),
        skinny_attr<16, true, true>(), pair_attr<false>(), pair_attr<true>()})
    if (e == cudaSuccess) e = r;
  return e;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

int force_split() {
  static const int s = [] {
    const char* e = std::getenv("DQGEMM_SPLIT");
    return e ? std::atoi(e) : 0;
  }();
  return s;
}

// Whether a call on bf16 activations quantizes them in the product itself, one
// launch instead of two.  A layer: up to 8 rows, which the quantizing warps hold
// in registers at once.  It saves a launch and the caller's temporary, not time
// on the GPU.  Weights from HBM, us, one launch / quantizer and product:
//                               1 row       8 rows      9 rows      16 rows
//   4096 x 14336, GPU only   14.4 / 13.3  14.7 / 13.7  18.8 / 13.8  19.5 / 13.9
//   4096 x 4096, GPU only     8.3 /  8.3   8.5 /  8.5   9.6 /  8.5   9.8 /  8.7
//   4096 x 4096, from Python  8.4 / 11.6   8.5 / 11.7   9.6 / 11.7   9.7 / 11.7
//   2048 x 2048, from Python  7.4 / 11.6   7.2 / 11.7   7.4 / 11.6   7.6 / 11.5
// Experts, whose CTAs go through several tiles: 16 rows and at most 16 blocks a
// CTA (7 rows, 5 of 8 of 1024 x 768: 6.0 / 6.3 us on the GPU; 16 rows, 12 of 32
// of 4096 x 2048, 64 blocks a CTA: 26.6 / 24.4).
bool quantizes(const dqgemm_s* h, int M) {
  if (!h->experts) return M <= 8;
  return M <= 16 && h->k_stages * ceil_div((long long)std::min(h->E, M) * h->n_tiles, h->num_sms) <= 16;
}

template <int BN>
int skinny_clusters(int split) {
  using C = SkinnyCfg<BN, false>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = split;
  a[0].val.clusterDim.y = 1;
  a[0].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, block_skinny_kernel<BN, false, false>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return n;
}

// how many clusters of `split` CTAs run at once (they have to lie in one GPC
// each, so not as many as the SMs would hold); asked once per handle
int cluster_capacity(dqgemm_s* h, int bn, int split) {
  std::atomic<int>& known = h->max_clusters[bn == 16 ? 0 : bn == 32 ? 1 : bn == 64 ? 2 : 3][split];
  int c = known.load(std::memory_order_relaxed);
  if (c == 0) {
    const int n = bn == 16 ? skinny_clusters<16>(split) : bn == 32 ? skinny_clusters<32>(split)
                : bn == 64 ? skinny_clusters<64>(split) : skinny_clusters<128>(split);
    c = n > 0 ? n : -1;
    known.store(c, std::memory_order_relaxed);
  }
  return c;
}

// The split of K: the largest power of two S <= 8, S <= kb, whose T clusters of
// S CTAs all run at once (1 x 2048 x 2048, T = 16: S = 8 would take two turns,
// 9.9 us against 4.6 at S = 4).
int pick_split(dqgemm_s* h, long long T, int bn) {
  int s = 1;
  if (force_split() > 0) {
    while (2 * s <= std::min({force_split(), 8, h->k_stages})) s *= 2;
    return s;
  }
  for (int c = 2; c <= 8 && c <= h->k_stages && T * c <= h->num_sms; c *= 2)
    if (cluster_capacity(h, bn, c) >= T) s = c;
  return s;
}

// Above 64 rows: 128 x 128 tiles by single CTAs or 256 x 256 by pairs, whichever
// takes less by this fit, in ns, of both kernels' times: rounds of tiles, each so
// much per block of K and so much per tile (its output), a split's meeting.
// Measured with weights from HBM at K = 512, 1152 and 4096, N = 1024, 2048,
// 4096, 5000, 8192 and 14336 and 17 counts of rows from 65 to 2048: the choice is
// the faster kernel or within 7 %, 0.2 % on average.  A bias costs a pair's tile
// half a us more (1040 x 5000, 777 rows: 15.7 / 16.2).  Some of it (us, single / pair):
//   rows                  65          256          512          777         1024         2048
//   512 x 2048     6.4 / 6.3    7.4 / 6.3    7.9 / 6.3    6.7 / 6.4    6.9 / 6.4   10.8 / 7.0
//   1152 x 5000    8.9 / 8.7    8.8 / 8.7   14.5 / 9.3  15.0 / 14.6  20.4 / 14.7  32.4 / 20.7
//   4096 x 4096  10.9 / 18.8  14.7 / 19.0  20.4 / 19.4  37.2 / 20.1  37.2 / 20.3  71.4 / 35.9
//   4096 x 14336 20.4 / 21.7  38.6 / 22.1  71.8 / 37.6  106.0 / 68.1  122.6 / 68.6  224.0 / 120.3
BlockPlan dense_plan(dqgemm_s* h, int M) {
  BlockPlan pl{};
  pl.bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  if (M > 64) {
    const long long t1 = ceil_div(M, 128) * h->n_tiles, t2 = ceil_div(M, 256) * ceil_div(h->N, 256);
    const int s = pick_split(h, t1, 128);
    const long long c1 = ceil_div(t1 * s, h->num_sms) * (470 * ceil_div(h->k_stages, s) + 1850) + (s > 1 ? 2000 : 250);
    const long long c2 = ceil_div(t2, h->num_sms / 2) * (460 * h->k_stages + 1900 + (h->bias ? 500 : 0));
    if (c2 <= c1) {
      pl.pair = true;
      pl.bn = 256;
    }
  }
  pl.m_tiles = (int)ceil_div(M, pl.bn);
  pl.n_tiles = (int)ceil_div(h->N, pl.pair ? 256 : 128);
  const long long T = (long long)pl.m_tiles * pl.n_tiles;
  if (pl.pair) {
    pl.split = 1;
    pl.grid = 2 * (int)std::min<long long>(T, h->num_sms / 2);
  } else {
    pl.split = pick_split(h, T, pl.bn);
    pl.grid = (int)(pl.split > 1 ? T * pl.split : std::min<long long>(T, h->num_sms));
  }
  return pl;
}

// The rows of each expert are known on the device only; the tile is picked by
// their mean over all experts.  Measured with 32 experts of 4096 x 2048 and rows
// that fall on them at random (us; 64 experts of 2048 x 1536 cross at the same places):
//   rows an expert   4     8    16    24    32    48    64    80    96   128   192
//   16-row tiles    45.2  46.3  47.7  63.9  83
//   32-row tiles    45.3  46.4  46.9  49.3  51.8  65.5  77.6
//   64-row tiles    48.3  49.6  50.7  52.7  54.9  58.8  71.9  80.5  88.7   106   137
//   256-row (pair)  69.6  73.2  76.1  79.5  83.1  79.5  80.0  80.5  82.7  82.3  86.8
// Rows that gather on few of many experts would want larger tiles than their
// mean says: 512 rows on one of 32 experts take 19.5 us with the 32-row tiles
// of a mean of 16 (64-row tiles 14.7), 2048 rows on two of 128 60 us (pairs 22.9).
BlockPlan grouped_plan(const dqgemm_s* h, int M) {
  BlockPlan pl{};
  const long long mean = ceil_div(M, h->E);
  pl.pair = mean > 80;
  pl.bn = pl.pair ? 256 : M <= 16 || mean <= 4 ? 16 : mean <= 32 ? 32 : 64;
  pl.n_tiles = (int)ceil_div(h->N, pl.pair ? 256 : 128);
  pl.m_tiles = 0;
  pl.split = 1;
  // at most one partial row tile per expert with rows
  const long long T = (M / pl.bn + std::min(h->E, M)) * (long long)pl.n_tiles;
  pl.grid = pl.pair ? 2 * (int)std::min<long long>(T, h->num_sms / 2)
                    : (int)std::min<long long>(T, h->num_sms);
  return pl;
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------

// the map of the codes q [M, K] in boxes of 128 k x `rows` rows, encoded once
// for a buffer that comes again
bool codes_map(dqgemm_s* h, const void* q, int M, int rows, CUtensorMap* tm) {
  std::lock_guard<std::mutex> lock(h->maps_mu);
  for (const auto& e : h->maps) {
    if (e.x == q && e.M == M && e.bn == rows) {
      *tm = e.map;
      return true;
    }
  }
  if (!make_q_map(tm, q, M, h->K, rows)) return false;
  auto& e = h->maps[h->next_map];
  h->next_map = (h->next_map + 1) % dqgemm_s::kMaps;
  e.x = q;
  e.M = M;
  e.bn = rows;
  e.xq = true;
  e.map = *tm;
  return true;
}

template <typename K>
cudaError_t launch(K kern, int grid, int threads, int smem, int cluster, const CUtensorMap& tw, const CUtensorMap& tx,
                   const BlockParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute a[2];
  int na = 0;
  if (pdl_enabled()) {
    a[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  if (cluster > 1) {
    a[na].id = cudaLaunchAttributeClusterDimension;
    a[na].val.clusterDim.x = cluster;
    a[na].val.clusterDim.y = 1;
    a[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = a;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, kern, tw, tx, p);
}

template <int BN, bool G, bool X>
cudaError_t launch_skinny(const BlockPlan& pl, const CUtensorMap& tw, const CUtensorMap& tx, const BlockParams& p,
                          cudaStream_t s) {
  using C = SkinnyCfg<BN, X>;
  return launch(block_skinny_kernel<BN, G, X>, pl.grid, C::THREADS, C::SMEM, pl.split, tw, tx, p, s);
}

template <bool G>
cudaError_t launch_plan(const BlockPlan& pl, const CUtensorMap& tw, const CUtensorMap& tx, const BlockParams& p,
                        cudaStream_t s) {
  // (the pair kernel's cluster size is a property of the kernel)
  if (pl.pair) return launch(block_pair_kernel<G>, pl.grid, PairCfg::THREADS, PairCfg::SMEM, 1, tw, tx, p, s);
  if (p.x) return launch_skinny<16, G, true>(pl, tw, tx, p, s);
  switch (pl.bn) {
    case 16: return launch_skinny<16, G, false>(pl, tw, tx, p, s);
    case 32: return launch_skinny<32, G, false>(pl, tw, tx, p, s);
    case 64: return launch_skinny<64, G, false>(pl, tw, tx, p, s);
    default:
      if constexpr (G) return cudaErrorInvalidValue;   // (never planned)
      else return launch_skinny<128, G, false>(pl, tw, tx, p, s);
  }
}

// Codes q and scales sx, or (where quantizes()) bf16 x; arguments checked
// by the callers.
dqgemm_status run_block(dqgemm_handle h, const BlockPlan& pl, const void* q, const float* sx, const void* x, int M,
                        const int* offsets, void* y, void* stream) {
  if ((M / pl.bn + (long long)std::max(h->E, 1)) * pl.n_tiles > 0x7FFFFFFFll) return DQ_ERR_UNSUPPORTED;
  const CUtensorMap& tw = pl.pair ? h->wmap64 : h->wmap;
  CUtensorMap tx;
  if (!x && !codes_map(h, q, M, pl.pair ? 128 : pl.bn, &tx)) return DQ_ERR_CUDA;
  BlockParams p{};
  p.sx = sx;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.sw = h->col_scale;
  p.bias = h->bias;
  p.y = static_cast<__nv_bfloat16*>(y);
  p.offsets = offsets;
  p.status = h->status;
  p.M = M;
  p.N = h->N;
  p.K = h->K;
  p.E = h->E;
  p.kb = h->k_stages;
  p.nb = h->n_tiles;
  p.n_tiles = pl.n_tiles;
  p.m_tiles = pl.m_tiles;
  p.split = pl.split;
  p.vec_y = h->N % 8 == 0 && aligned16(y);
  p.timeout_ns = h->timeout_ns;
  p.drain_ns = std::max(timeout_ns(), kDefaultTimeoutNs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // (a call on bf16 x uses no map of the codes: any map fills the parameter)
  return cuda_err(offsets ? launch_plan<true>(pl, tw, x ? tw : tx, p, s) : launch_plan<false>(pl, tw, x ? tw : tx, p, s));
}

long long x_workspace(const dqgemm_s* h, int M) {
  return quantizes(h, M) ? 0 : ((long long)M * h->K + 255) / 256 * 256 + (long long)M * h->k_stages * 4;
}

// x bf16: in one launch where the product quantizes it itself, else quantized
// into the workspace `ws` (codes, then scales) first
dqgemm_status run_x(dqgemm_handle h, const void* x, int M, const int* offsets, void* y, void* ws, void* stream) {
  const BlockPlan pl = offsets ? grouped_plan(h, M) : dense_plan(h, M);
  if (quantizes(h, M)) return run_block(h, pl, nullptr, nullptr, x, M, offsets, y, stream);
  float* sx = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + ((size_t)M * h->K + 255) / 256 * 256);
  const dqgemm_status st = dqgemm_quantize_act_fp8_block(DQ_BF16, x, h->K, M, h->K, ws, sx, stream);
  return st == DQ_OK ? run_block(h, pl, ws, sx, nullptr, M, offsets, y, stream) : st;
}

}  // namespace

namespace dq {

dqgemm_status block_create(dqgemm_handle* out, bool experts, int E, int K, int N, const void* packed_w, const void* scales,
                           const void* bias) {
  // (out set to null and the shape checked by the callers)
  if (!packed_w || !scales) return DQ_ERR_INVALID_ARG;
  if (!aligned16(packed_w) || !aligned16(scales) || (bias && !aligned16(bias))) return DQ_ERR_ALIGNMENT;
  if (!is_device_ptr(packed_w) || !is_device_ptr(scales) || (bias && !is_device_ptr(bias))) return DQ_ERR_INVALID_ARG;
  if ((long long)E * N > 0x7FFFFFFFll - 256) return DQ_ERR_UNSUPPORTED;   // (a row index of the weight's tensor map)
  dqgemm_s* h = new (std::nothrow) dqgemm_s();
  if (!h) return DQ_ERR_ALLOC;
  h->fmt = FMT_FP8B;
  h->K = K;
  h->N = N;
  h->E = E;
  h->experts = experts;
  h->k_stages = blocks(K);
  h->n_tiles = blocks(N);
  h->timeout_ns = timeout_ns();
  cudaGetDevice(&h->device);
  cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  const size_t rows = (size_t)E * N, wb = rows * K, ns = (size_t)E * h->n_tiles * h->k_stages;
  h->wchunk_bytes = wb;
  h->weight_bytes = (long long)(wb + ns * 4);
  cudaError_t e = cudaMalloc(&h->wchunks, wb);
  if (e == cudaSuccess) e = cudaMalloc(&h->col_scale, ns * 4);
  if (e == cudaSuccess && bias) e = cudaMalloc(&h->bias, rows * 2);
  if (e == cudaSuccess) e = cudaHostAlloc(&h->status_host, sizeof(int), cudaHostAllocMapped | cudaHostAllocPortable);
  if (e != cudaSuccess) {
    cudaGetLastError();
    dqgemm_destroy(h);
    return DQ_ERR_ALLOC;
  }
  *h->status_host = 0;
  e = cudaHostGetDevicePointer(reinterpret_cast<void**>(&h->status), h->status_host, 0);
  // (the buffers may still be being written, on whatever stream)
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(h->wchunks, packed_w, wb, cudaMemcpyDeviceToDevice);
  if (e == cudaSuccess) e = cudaMemcpy(h->col_scale, scales, ns * 4, cudaMemcpyDeviceToDevice);
  if (e == cudaSuccess && bias) e = cudaMemcpy(h->bias, bias, rows * 2, cudaMemcpyDeviceToDevice);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  // codes and scales outside the format are noted in the status word
  if (e == cudaSuccess) {
    check_fp8_block_kernel<<<h->num_sms * 4, 256>>>(h->wchunks, wb, h->col_scale, ns, h->status);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = set_attrs();
  if (e != cudaSuccess || !make_q_map(&h->wmap, h->wchunks, (int)rows, K, 128) ||
      !make_q_map(&h->wmap64, h->wchunks, (int)rows, K, 64)) {
    dqgemm_destroy(h);
    return DQ_ERR_CUDA;
  }
  if (*h->status_host != 0) {
    dqgemm_destroy(h);
    return DQ_ERR_INVALID_ARG;
  }
  *out = h;
  return DQ_OK;
}

// dqgemm_run: the workspace, where one is needed, is the handle's
dqgemm_status block_run_x(dqgemm_handle h, const void* x, int M, void* y, void* stream) {
  if (!aligned16(x) || !aligned16(y)) return DQ_ERR_ALIGNMENT;
  const size_t total = (size_t)x_workspace(h, M);
  if (total > 0) {
    std::lock_guard<std::mutex> lock(h->maps_mu);
    if (h->ws_bytes < total) {
      // grow: calls already launched may still read the old workspace
      if (cudaDeviceSynchronize() != cudaSuccess) return DQ_ERR_CUDA;
      cudaFree(h->ws);
      h->ws = nullptr;
      h->ws_bytes = 0;
      if (cudaMalloc(&h->ws, total) != cudaSuccess) {
        cudaGetLastError();
        h->ws = nullptr;
        return DQ_ERR_ALLOC;
      }
      h->ws_bytes = total;
    }
  }
  return run_x(h, x, M, nullptr, y, h->ws, stream);
}

dqgemm_status block_dequantize(dqgemm_handle h, void* w_bf16, void* stream) {
  dequant_fp8_block_kernel<<<h->num_sms * 8, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      h->wchunks, h->col_scale, (size_t)h->E * h->N, h->N, h->K, static_cast<__nv_bfloat16*>(w_bf16));
  return cuda_err(cudaGetLastError());
}

void block_fill_plan(dqgemm_handle h, int M, dqgemm_plan* pl) {
  std::memset(pl, 0, sizeof(*pl));
  const BlockPlan b = h->experts ? grouped_plan(h, M) : dense_plan(h, M);
  pl->bn = b.bn;
  pl->m_tiles = (int)ceil_div(M, b.bn);
  pl->n_tiles = b.n_tiles;
  pl->k_stages = h->k_stages;
  pl->grid = b.grid;
  pl->max_segments = b.split;
  pl->stages = pl->x_stages = b.pair ? PairCfg::ST
                              : b.bn == 16 ? SkinnyCfg<16, true>::ST
                              : b.bn == 32 ? SkinnyCfg<32, false>::ST
                              : b.bn == 64 ? SkinnyCfg<64, false>::ST
                                           : SkinnyCfg<128, false>::ST;
  pl->smem_bytes = b.pair ? PairCfg::SMEM
                   : b.bn == 16 ? SkinnyCfg<16, true>::SMEM
                   : b.bn == 32 ? SkinnyCfg<32, false>::SMEM
                   : b.bn == 64 ? SkinnyCfg<64, false>::SMEM
                                : SkinnyCfg<128, false>::SMEM;
  pl->workspace_bytes = x_workspace(h, M);
  pl->weight_bytes = h->weight_bytes;
  const long long T = (long long)pl->m_tiles * b.n_tiles;
  const long long at_once = b.pair ? b.grid / 2 : b.grid;
  pl->max_cta_stages = b.split > 1 ? (int)ceil_div(h->k_stages, b.split) : (int)ceil_div(T, at_once) * h->k_stages;
}

dqgemm_status block_pack_host(const float* W, int K, int N, void* packed, void* scales) {
  uint8_t* P = static_cast<uint8_t*>(packed);
  float* S = static_cast<float*>(scales);
  for (int i = 0; i < blocks(N); ++i)
    for (int j = 0; j < blocks(K); ++j) {
      const int n1 = std::min(N, (i + 1) * QB), k1 = std::min(K, (j + 1) * QB);
      float a = 0.f;
      for (int n = i * QB; n < n1; ++n)
        for (int k = j * QB; k < k1; ++k) a = std::max(a, std::fabs(W[(size_t)n * K + k]));
      const float s = fdiv(a, 448.f);
      S[(size_t)i * blocks(K) + j] = s;
      for (int n = i * QB; n < n1; ++n)
        for (int k = j * QB; k < k1; ++k)
          P[(size_t)n * K + k] = s > 0.f ? e4m3_encode_sat(fdiv(W[(size_t)n * K + k], s)) : 0;
    }
  return DQ_OK;
}

dqgemm_status block_pack_device(const float* W, int K, int N, void* packed, void* scales, cudaStream_t s) {
  if (blocks(N) > 65535) return DQ_ERR_UNSUPPORTED;   // a grid row per block of channels
  pack_fp8_block_kernel<<<dim3(blocks(K), blocks(N)), 256, 0, s>>>(W, N, K, static_cast<uint8_t*>(packed),
                                                                   static_cast<float*>(scales));
  return cuda_err(cudaGetLastError());
}

}  // namespace dq

extern "C" {

dqgemm_status dqgemm_create_experts(dqgemm_handle* out, dqgemm_format fmt, int E, int K, int N, const void* packed_w,
                                    const void* scales, const void* bias) {
  if (!out) return DQ_ERR_INVALID_ARG;
  *out = nullptr;
  if (E < 1 || K < 1 || N < 1 || (int)fmt < 0 || (int)fmt > (int)DQ_FP8_BLOCK128) return DQ_ERR_INVALID_ARG;
  if (fmt != DQ_FP8_BLOCK128 || E > MAX_EXPERTS) return DQ_ERR_UNSUPPORTED;
  if (K % 16) return DQ_ERR_INVALID_ARG;
  return block_create(out, true, E, K, N, packed_w, scales, bias);
}

dqgemm_status dqgemm_run_fp8_block_quantized(dqgemm_handle h, const void* q, const float* scales, int M, void* y,
                                             void* stream) {
  if (!h || !q || !scales || !y || M < 1) return DQ_ERR_INVALID_ARG;
  if (h->fmt != FMT_FP8B || h->experts) return DQ_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(y) || reinterpret_cast<uintptr_t>(scales) % 4) return DQ_ERR_ALIGNMENT;
  return run_block(h, dense_plan(h, M), q, scales, nullptr, M, nullptr, y, stream);
}

dqgemm_status dqgemm_run_experts_quantized(dqgemm_handle h, const void* q, const float* scales, int M, const int* offsets,
                                           void* y, void* stream) {
  if (!h || !q || !scales || !offsets || !y || M < 1) return DQ_ERR_INVALID_ARG;
  if (h->fmt != FMT_FP8B || !h->experts) return DQ_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(y) || reinterpret_cast<uintptr_t>(scales) % 4 ||
      reinterpret_cast<uintptr_t>(offsets) % 4)
    return DQ_ERR_ALIGNMENT;
  return run_block(h, grouped_plan(h, M), q, scales, nullptr, M, offsets, y, stream);
}

dqgemm_status dqgemm_run_fp8_block(dqgemm_handle h, const void* x, int M, const int* offsets, void* y, void* workspace,
                                   long long workspace_bytes, void* stream) {
  if (!h || !x || !y || M < 1) return DQ_ERR_INVALID_ARG;
  if (h->fmt != FMT_FP8B || (offsets != nullptr) != h->experts) return DQ_ERR_UNSUPPORTED;
  const long long need = x_workspace(h, M);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || (need > 0 && !aligned16(workspace)) || reinterpret_cast<uintptr_t>(offsets) % 4)
    return DQ_ERR_ALIGNMENT;
  return run_x(h, x, M, offsets, y, workspace, stream);
}

}  // extern "C"
