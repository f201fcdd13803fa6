// dq_rows_api.cu -- the row operators of include/dqgemm.h: dqgemm_rmsnorm,
// dqgemm_silu_mul, dqgemm_quantize_act_fp8_block.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "dq_handle.h"
#include "dq_rows.cuh"

using namespace dq;

namespace {

size_t type_bytes(int t) { return t == ROW_FP32 ? 4 : 2; }

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

size_t out_bytes(int out) { return out == OUT_FP32 ? 4 : out <= OUT_FP16 ? 2 : 1; }

// Natural alignment of every buffer; *al: how whole vectors of 16 elements can
// be moved (see load16).
dqgemm_status check_rows(const RowArgs& a, int type, int out, int halves, int* al) {
  if (type < ROW_BF16 || type > ROW_FP32 || out < OUT_BF16 || out > OUT_STATIC) return DQ_ERR_INVALID_ARG;
  if (!a.x || !a.out || a.M < 1 || a.K < 1 || a.K > (1 << 28) || a.ldx < (long long)halves * a.K)
    return DQ_ERR_INVALID_ARG;
  if (out == OUT_BLOCK && !a.scales) return DQ_ERR_INVALID_ARG;
  if (out == OUT_STATIC && !(std::isfinite(a.s_out) && a.s_out > 0.f)) return DQ_ERR_INVALID_ARG;
  const size_t tb = type_bytes(type), ob = out_bytes(out);
  if (!aligned_to(a.x, tb) || !aligned_to(a.out, ob) || (out == OUT_BLOCK && !aligned_to(a.scales, 4)) ||
      (a.res && (!aligned_to(a.res, tb) || !aligned_to(a.res_out, tb))) || (a.w && !aligned_to(a.w, type_bytes(a.w_type))))
    return DQ_ERR_ALIGNMENT;
  const auto fits = [&](int elems, size_t bytes) {
    return a.K % elems == 0 && aligned_to(a.x, bytes) && (a.ldx * (long long)tb) % (long long)bytes == 0 &&
           aligned_to(a.out, ob == 1 ? bytes / 2 : bytes) &&
           (!a.res || (aligned_to(a.res, bytes) && aligned_to(a.res_out, bytes))) && (!a.w || aligned_to(a.w, bytes));
  };
  *al = fits(16, 32) ? 2 : fits(8, 16) ? 1 : 0;
  return DQ_OK;
}

// multiprocessors of the current device
int sm_count() {
  static std::atomic<int> counts[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int n = counts[dev].load(std::memory_order_relaxed);
  if (n == 0) {   // (every thread finds the same)
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    counts[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// CTAs of a kernel that are resident at once, on all multiprocessors: what a
// launch over many rows starts, since each goes on to the next rows itself
template <typename K>
long long resident_ctas(K kern, int threads, std::atomic<int> (&cache)[33]) {
  std::atomic<int>& known = cache[threads / 32];   // (every thread finds the same)
  int n = known.load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 0) != cudaSuccess) cudaGetLastError();
    n = std::max(1, n);
    known.store(n, std::memory_order_relaxed);
  }
  return (long long)n * sm_count();
}

template <typename... KArgs, typename... Args>
dqgemm_status launch_rows(void (*kern)(KArgs...), dim3 grid, dim3 block, void* stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cuda_err(cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...));
}

template <typename T, int NV, int OUT, int AL, int MT>
dqgemm_status norm_grid(const RowArgs& a, long long need, dim3 block, void* stream) {
  static std::atomic<int> cache[33] = {};
  const long long most = resident_ctas(rmsnorm_kernel<T, NV, OUT, AL, MT>, (int)(block.x * block.y), cache);
  return launch_rows(rmsnorm_kernel<T, NV, OUT, AL, MT>, dim3((unsigned)std::min(need, most)), block, stream, a);
}

template <typename T, int OUT, int AL>
dqgemm_status norm_launch(const RowArgs& a, void* stream) {
  // threads a row: one vector each up to 512 of them (K = 8192: 82.8 us for
  // 8192 rows, with two each on half the threads 88.0), then two; rows past
  // K = 16384 are read twice.  Rows that start anywhere: one each up to 1024
  // (4096 x 12001 in bf16: 116 us, with two each 158).
  constexpr int single = AL == 0 ? 1024 : 512;
  const int vecs = (a.K + 15) / 16, per = vecs <= single ? 1 : 2;
  const int tpr = std::min(single, ((vecs + per - 1) / per + 31) / 32 * 32);
  const int rows = std::max(1, 128 / tpr);
  const dim3 block(tpr, rows);
  const long long need = (a.M + (long long)rows - 1) / rows;
  if (vecs > 1024) return norm_grid<T, 0, OUT, AL, single>(a, need, block, stream);
  if (tpr <= 256 && per == 1) return norm_grid<T, 1, OUT, AL, 256>(a, need, block, stream);
  if constexpr (AL == 0) {
    return tpr <= 384   ? norm_grid<T, 1, OUT, AL, 384>(a, need, block, stream)
           : tpr <= 768 ? norm_grid<T, 1, OUT, AL, 768>(a, need, block, stream)
                        : norm_grid<T, 1, OUT, AL, 1024>(a, need, block, stream);
  } else {
    return per == 1 ? norm_grid<T, 1, OUT, AL, 512>(a, need, block, stream) : norm_grid<T, 2, OUT, AL, 512>(a, need, block, stream);
  }
}

template <typename T, bool GATE, int OUT, int AL>
dqgemm_status plain_launch(const RowArgs& a, void* stream) {
  const int parts = (a.K + 511) / 512;
  const long long items = (long long)parts * a.M;
  // (few warps: one a CTA, so that they spread over the multiprocessors)
  const int per = (int)std::max<long long>(1, std::min<long long>(8, items / sm_count()));
  static std::atomic<int> cache[33] = {};
  const int ctas = (int)std::min((items + per - 1) / per, resident_ctas(rows_kernel<T, GATE, OUT, AL>, 32 * per, cache));
  return launch_rows(rows_kernel<T, GATE, OUT, AL>, dim3(ctas), dim3(32 * per), stream, a, parts);
}

// OP 0: rmsnorm, 1: gated SiLU, 2: plain (block-quantized output only)
template <int OP, typename T, int OUT>
dqgemm_status go(const RowArgs& a, int al, void* stream) {
  if constexpr (OP == 0)
    return al == 2   ? norm_launch<T, OUT, 2>(a, stream)
           : al == 1 ? norm_launch<T, OUT, 1>(a, stream)
                     : norm_launch<T, OUT, 0>(a, stream);
  else
    return al == 2   ? plain_launch<T, OP == 1, OUT, 2>(a, stream)
           : al == 1 ? plain_launch<T, OP == 1, OUT, 1>(a, stream)
                     : plain_launch<T, OP == 1, OUT, 0>(a, stream);
}

template <int OP, typename T>
dqgemm_status go_out(const RowArgs& a, int out, int al, void* stream) {
  if constexpr (OP == 2) {
    return go<OP, T, OUT_BLOCK>(a, al, stream);
  } else {
    switch (out) {
      case OUT_BF16: return go<OP, T, OUT_BF16>(a, al, stream);
      case OUT_FP16: return go<OP, T, OUT_FP16>(a, al, stream);
      case OUT_FP32: return go<OP, T, OUT_FP32>(a, al, stream);
      case OUT_BLOCK: return go<OP, T, OUT_BLOCK>(a, al, stream);
      default: return go<OP, T, OUT_STATIC>(a, al, stream);
    }
  }
}

template <int OP>
dqgemm_status run_rows(RowArgs& a, int type, int out, float s_out, void* stream) {
  a.s_out = out == OUT_STATIC ? s_out : 1.f;
  int al = 0;
  const dqgemm_status st = check_rows(a, type, out, OP == 1 ? 2 : 1, &al);
  if (st != DQ_OK) return st;
  const long long tb = (long long)type_bytes(type);
  a.x_bytes = ((a.M - 1) * a.ldx + (OP == 1 ? 2 : 1) * (long long)a.K) * tb;
  a.row_bytes = (long long)a.M * a.K * tb;
  volatile float one = 1.f;
  volatile float r = one / a.s_out;   // an fp32 division
  a.r_out = r;
  switch (type) {
    case ROW_BF16: return go_out<OP, __nv_bfloat16>(a, out, al, stream);
    case ROW_FP16: return go_out<OP, __half>(a, out, al, stream);
    default: return go_out<OP, float>(a, out, al, stream);
  }
}

}  // namespace

extern "C" {

dqgemm_status dqgemm_rmsnorm(dqgemm_dtype type, const void* x, long long ldx, const void* residual,
                             void* residual_out, dqgemm_dtype weight_type, const void* weight, float eps, int M, int K,
                             dqgemm_out out_kind, float s_out, void* out, float* scales, void* stream) {
  if ((residual == nullptr) != (residual_out == nullptr)) return DQ_ERR_INVALID_ARG;
  if (residual_out && residual_out == out) return DQ_ERR_INVALID_ARG;
  if ((int)weight_type < ROW_BF16 || (int)weight_type > ROW_FP32) return DQ_ERR_INVALID_ARG;
  if (!(std::isfinite(eps) && eps >= 0.f)) return DQ_ERR_INVALID_ARG;
  RowArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.res = residual;
  a.res_out = residual_out;
  a.w = weight;
  a.w_type = (int)weight_type;
  a.eps = eps;
  a.M = M;
  a.K = K;
  a.out = out;
  a.scales = scales;
  return run_rows<0>(a, (int)type, (int)out_kind, s_out, stream);
}

dqgemm_status dqgemm_silu_mul(dqgemm_dtype type, const void* x, long long ldx, int M, int K, dqgemm_out out_kind,
                              float s_out, void* out, float* scales, void* stream) {
  RowArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.M = M;
  a.K = K;
  a.out = out;
  a.scales = scales;
  return run_rows<1>(a, (int)type, (int)out_kind, s_out, stream);
}

dqgemm_status dqgemm_quantize_act_fp8_block(dqgemm_dtype type, const void* x, long long ldx, int M, int K, void* q,
                                            float* scales, void* stream) {
  RowArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.M = M;
  a.K = K;
  a.out = q;
  a.scales = scales;
  return run_rows<2>(a, (int)type, OUT_BLOCK, 1.f, stream);
}

}  // extern "C"
