// dq_block.cuh -- products in e4m3 with a scale per 128 x 128 block of the
// weight and per 128 activations of a row, dense or grouped by expert:
//
//   y[m, n] = sum_b sx[m, b] * sw[n / 128, b] * (sum_{k in block b} qx[m, k] qw[n, k])  + bias[n]
//
// The tensor core sums the 128 products of a block into a TMEM buffer of its
// own (fp32); the epilogue warps multiply that partial by the block's two
// scales and add it to their fp32 accumulators in registers while the next
// block's MMAs run into another buffer.  Weights stay row-major [N, K]: TMA
// writes the tensor core's swizzled image, so nothing is laid out again.
//
// Two kernels:
//   block_skinny_kernel  y^T = W x^T: 128 weight rows are the MMA's M, BN
//       activation rows its N (16..128).  Bound by the weight's bytes.  With
//       few tiles the K range is split over a thread-block cluster, whose
//       partials meet in distributed shared memory in rank order.
//   block_pair_kernel    256 rows x 256 channels by a pair of CTAs
//       (cta_group::2): each CTA holds 128 activation rows and half of the
//       weight rows, so a product of 128 k costs each SM 32 KB of loads where
//       a single CTA's 128 x 256 tile costs 48.  The two halves of 128
//       channels are separate chains (MMA thread, partial buffers, epilogue
//       warps), so one half's MMAs run while the other's partial is read.
//
// Grouped calls (E > 0 experts): rows offsets[e] .. offsets[e + 1] belong to
// expert e.  The offsets are read on the device; each CTA counts the tiles
// of every expert itself.  Offsets outside [0, M] are clamped, so no value in
// them makes an access leave the buffers.
#pragma once

#include "dq_codec.h"
#include "dq_common.cuh"
#include "dq_rows.cuh"

namespace dq {

constexpr int MAX_EXPERTS = 1024;

struct BlockParams {
  const float* sx;             // [M, kb]
  const __nv_bfloat16* x;      // activations that the kernel quantizes itself [M, K]
  const float* sw;             // [E][nb][kb]
  const __nv_bfloat16* bias;   // [E][N] or null
  __nv_bfloat16* y;            // [M, N]
  const int* offsets;          // grouped: device [E + 1]
  int* status;
  int M, N, K, E;
  int kb, nb;                  // blocks along K and N
  int n_tiles, m_tiles;        // (m_tiles: dense)
  int split;
  int vec_y;                   // y rows are 16-byte aligned
  unsigned long long timeout_ns, drain_ns;
};

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
struct BlockTile {
  int e, n0;         // expert, first channel
  int m0, m_end;     // first row, end of the expert's rows
};

__device__ __forceinline__ void expert_rows(const BlockParams& p, int e, int& a, int& b) {
  a = max(0, min(p.M, p.offsets[e]));
  b = max(a, min(p.M, p.offsets[e + 1]));
}

// start[e]: row tiles of the experts before e, start[E]: all of them.  The
// whole CTA calls this (it ends with a barrier).
template <int TM>
__device__ __forceinline__ void count_tiles(const BlockParams& p, int* start) {
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    int a, b;
    expert_rows(p, e, a, b);
    start[e + 1] = (b - a + TM - 1) / TM;
  }
  if (threadIdx.x == 0) start[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + (int)threadIdx.x;
      int v = e < p.E ? start[e + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if ((int)threadIdx.x >= o) v += u;
      }
      if (e < p.E) start[e + 1] = base + v;
      base += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
  }
  __syncthreads();
}

// tile t, rows fastest: neighbouring CTAs share a weight tile
template <int TM, int TN, bool GROUPED>
__device__ __forceinline__ BlockTile block_tile(const BlockParams& p, const int* start, int t) {
  BlockTile r;
  if constexpr (GROUPED) {
    const int u = t / p.n_tiles;   // start[e] <= u < start[e + 1]
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= u) lo = mid;
      else hi = mid;
    }
    const int mt = start[lo + 1] - start[lo], local = t - start[lo] * p.n_tiles;
    const int nt = local / mt;
    int a, b;
    expert_rows(p, lo, a, b);
    r.e = lo;
    r.n0 = nt * TN;
    r.m0 = a + (local - nt * mt) * TM;
    r.m_end = b;
  } else {
    const int nt = t / p.m_tiles;
    r.e = 0;
    r.n0 = nt * TN;
    r.m0 = (t - nt * p.m_tiles) * TM;
    r.m_end = p.M;
  }
  return r;
}

// One lane of a converged warp, the same each time.  The MMAs and copies are
// issued under this and not under a test of the lane: they take their
// descriptors from uniform registers, and the compiler knows of elect.sync
// that one thread runs (of lane == 0 it does not, and wraps each instruction
// in a loop over the active lanes).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ---------------------------------------------------------------------------
// bounded waits without a clock on the common path: the limit is looked at
// only after a round of tries (reading the global timer first costs every
// wait that does not succeed at once several hundred cycles, which the MMA
// thread and the epilogue pay for each block of K).  try_wait suspends the
// thread for a short time of the hardware's choosing.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool block_wait(uint64_t* bar, uint32_t parity, const WaitCtl ctl) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (int round = 0;; ++round) {
    if (round > 0 || ctl.timeout_ns < 1000u) {
      if (t0 == 0) t0 = globaltimer_ns();
      if (wait_give_up(ctl, t0)) return false;
    }
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
  }
}
// whether three barriers have all completed their phases, looked at together
__device__ __forceinline__ bool mbar_try_wait3(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, uint64_t* c, uint32_t pc) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q, r;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 r, [%5], %6;\n\t"
      "and.pred p, p, q;\n\t"
      "and.pred p, p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb), "r"(smem_u32(c)), "r"(pc)
      : "memory");
  return ok != 0;
}
// the whole warp on two barriers at once: every lane observes the phases itself
__device__ __forceinline__ bool block_wait_warp2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, const WaitCtl ctl) {
  uint64_t t0 = 0;
  for (int i = ctl.timeout_ns < 1000u ? 63 : 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
        "and.pred p, p, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb)
        : "memory");
    if (__all_sync(0xFFFFFFFFu, ok != 0u)) return true;
    if ((i & 63) == 63) {
      if (t0 == 0) t0 = globaltimer_ns();
      if (__any_sync(0xFFFFFFFFu, wait_give_up(ctl, t0))) return false;
    }
  }
}
// ... and on one
__device__ __forceinline__ bool block_wait_warp(uint64_t* bar, uint32_t parity, const WaitCtl ctl) {
  uint64_t t0 = 0;
  for (int i = ctl.timeout_ns < 1000u ? 63 : 0;; ++i) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    if ((i & 63) == 63) {
      if (t0 == 0) t0 = globaltimer_ns();
      if (__any_sync(0xFFFFFFFFu, wait_give_up(ctl, t0))) return false;
    }
  }
}

// ---------------------------------------------------------------------------
// tensor memory reads whose wait carries the registers, so that no use of
// them can be scheduled before it
// ---------------------------------------------------------------------------
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, float (&v)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "8, 16 or 32 columns");
  if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr)
                 : "memory");
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
  }
}
template <int N>
__device__ __forceinline__ void tmem_wait_regs(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
               :
               : "memory");
  if constexpr (N > 8)
    asm volatile("" : "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
  if constexpr (N > 16) {
    asm volatile("" : "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]));
    asm volatile("" : "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
  }
}

// distributed shared memory: cluster CTA `rank`'s copy of a local address
__device__ __forceinline__ float4 ld_dsmem_f4(uint32_t local, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\t"
      "mapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(local), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// four consecutive blocks' scales of one row (0 past `end`)
__device__ __forceinline__ void load_scales(const float* row, bool live, int b, int end, float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = live && b + i < end ? row[b + i] : 0.f;
}

// ---------------------------------------------------------------------------
// skinny: 128 channels x BN rows per CTA
// warps: 0 weight copies, 1 MMA, 2 activation copies, 3 scales, 4..11
// epilogue; with bf16 activations (XBF) 12..19 quantize them instead of 2 and 3
//
// The combined scales sx * sw of each block of K go through a ring of their
// own, [SR][BN].  It needs no barrier against reuse: who writes entry i + SR
// has seen the MMAs of block i + SR - ST done, hence those of block i + PB,
// which were issued after the epilogue had finished with block i.  The MMAs
// of a block wait for its scales too (through full_x): nobody falls a whole
// phase of a barrier behind, where a parity would be taken for the next.
// ---------------------------------------------------------------------------
template <int BN, bool XBF>
struct SkinnyCfg {
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int X_BYTES = BN * 128;
  static constexpr int STAGE = W_BYTES + X_BYTES;          // both multiples of 1024
  // One CTA an SM with the whole ring: 144 KB of weights in flight.  (Two an SM
  // with five stages each: 1 x 4096 x 14336 13.7 us against 11.9, 32 rows 14.7
  // against 12.1; and of grouped tiles T, 148 CTAs take ceil(T / 148) rounds,
  // 296 twice ceil(T / 296), never fewer.)
  static constexpr int ST = BN <= 32 ? 9 : BN == 64 ? 8 : 6;
  static constexpr int PB = 4;                             // partial buffers
  static constexpr int SR = ST + PB;                       // scale entries
  static constexpr int TMEM_COLS = PB * BN < 32 ? 32 : PB * BN;
  static constexpr int HALF = BN / 2;                      // columns per epilogue thread
  static constexpr int BAR_OFF = ST * STAGE;
  static constexpr int BAR_BYTES = 448;
  static constexpr int SC_OFF = BAR_OFF + BAR_BYTES;
  static constexpr int SC_BYTES = SR * BN * 4;
  static constexpr int TAB_OFF = SC_OFF + SC_BYTES;        // grouped: tile counts
  static constexpr int TAB_BYTES = (MAX_EXPERTS + 1) * 4;
  static constexpr int SMEM = TAB_OFF + TAB_BYTES + 1024;
  // quantizing warps (1 x 4096 x 14336: 8 of them 13.5 us, 4 14.4, codes 11.9)
  static constexpr int QW = 8;
  static constexpr int THREADS = 384 + (XBF ? 32 * QW : 0);
  static_assert(X_BYTES % 1024 == 0, "swizzle atoms");
  static_assert(!XBF || BN == 16, "the quantizing warps keep up with a few rows only");
  static_assert(BN * 128 * 4 <= ST * STAGE, "the reduction reuses the ring");
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(TMEM_COLS <= 512, "tensor memory");
};

// One block of K of a tile's rows: 16 lanes a row, 8 elements a lane, two rows
// an instruction.  Codes into the tensor core's swizzled rows, combined scales
// into `sc`.  The same arithmetic as the row quantizer's.  Rows past m_end are
// left out: what their columns hold is not stored.  The first eight rows come
// in `first`, fetched by load_rows8 while the warp's last block was quantized.
__device__ __forceinline__ void load_rows8(const __nv_bfloat16* x, int K, int m0, int r0, int rows, int b, int lane,
                                           uint4 (&u)[4]) {
  const int k = b * 128 + (lane & 15) * 8, half = lane >> 4;
  const __nv_bfloat16* src = x + (size_t)(m0 + half) * K + k;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = r0 + 2 * i + half < rows && k < K ? *reinterpret_cast<const uint4*>(src + (size_t)(r0 + 2 * i) * K)
                                             : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void quantize_stage(const uint4 (&first)[4], const __nv_bfloat16* x, int K, int m0, int rows, int b,
                                               float sw, uint8_t* xs, float* sc, int lane) {
  const int half = lane >> 4;
  uint4 u[4] = {first[0], first[1], first[2], first[3]};
  for (int r0 = 0; r0 < rows; r0 += 8) {
    // four row pairs at once: maxima and quotients of one overlap the others'
    if (r0 > 0) load_rows8(x, K, m0, r0, rows, b, lane, u);
    // the maxima as bf16 bits, two pairs of rows in a word
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = __vmaxu2(__vmaxu2(u[i].x & 0x7FFF7FFFu, u[i].y & 0x7FFF7FFFu),
                                  __vmaxu2(u[i].z & 0x7FFF7FFFu, u[i].w & 0x7FFF7FFFu));
      m[i] = max(w & 0xFFFFu, w >> 16);
    }
    uint32_t m01 = m[0] | (m[1] << 16), m23 = m[2] | (m[3] << 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) {
      m01 = __vmaxu2(m01, __shfl_xor_sync(0xFFFFFFFFu, m01, o));
      m23 = __vmaxu2(m23, __shfl_xor_sync(0xFFFFFFFFu, m23, o));
    }
    m[0] = m01 << 16;
    m[1] = m01 & 0xFFFF0000u;
    m[2] = m23 << 16;
    m[3] = m23 & 0xFFFF0000u;
    BlockScale bs[4];
    bool fast = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bs[i] = block_scale_of(m[i]);
      fast = fast && bs[i].fast;
    }
    fast = __all_sync(0xFFFFFFFFu, fast);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 2 * i + half;   // (below the tile's 16: the rows that fill the last eight hold zeros)
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      F2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
      uint2 c;
      if (fast) {
        c = codes8_fast(v, bs[i].s, bs[i].r);
      } else {
        bs[i].s = __fdiv_rn(__uint_as_float(m[i]), 448.f);
        c = codes8_any(v, bs[i].s);
      }
      if ((lane & 15) == 0) sc[r] = bs[i].s * sw;
      *reinterpret_cast<uint2*>(xs + r * 128 + ((((lane & 15) >> 1) ^ (r & 7)) << 4) + (lane & 1) * 8) = c;
    }
  }
}

template <int BN, bool GROUPED, bool XBF>
__global__ void __launch_bounds__(SkinnyCfg<BN, XBF>::THREADS, 1)
    block_skinny_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                        const BlockParams p) {
  using C = SkinnyCfg<BN, XBF>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_w = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* full_x = full_w + C::ST;
  uint64_t* empty = full_x + C::ST;          // stage read by the MMAs
  uint64_t* acc_full = empty + C::ST;        // [PB]
  uint64_t* acc_empty = acc_full + C::PB;    // [PB]
  uint64_t* sc_full = acc_empty + C::PB;     // [SR] scales written
  uint64_t* drain = sc_full + C::SR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* bad = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);   // an epilogue warp gave up
  static_assert((3 * C::ST + 2 * C::PB + C::SR + 1) * 8 + 12 <= C::BAR_BYTES, "barriers");
  float* scales = reinterpret_cast<float*>(smem + C::SC_OFF);
  int* start = reinterpret_cast<int*>(smem + C::TAB_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto ctl = [&] { return WaitCtl{abort_flag, p.status, p.timeout_ns}; };
  const auto ctl_drain = [&] { return WaitCtl{nullptr, p.status, p.drain_ns}; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(&full_w[s], 1);
      mbar_init(&full_x[s], XBF ? 1 : 2);   // a quantizing warp, or copies and scales
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::PB; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);
    }
    for (int b = 0; b < C::SR; ++b) mbar_init(&sc_full[b], 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *bad = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(tmem_slot, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();

  int tiles;
  if constexpr (GROUPED) {
    pdl_wait();   // the offsets may be the previous grid's output
    count_tiles<BN>(p, start);
    tiles = start[p.E] * p.n_tiles;
  } else {
    tiles = p.n_tiles * p.m_tiles;
  }
  // split-K: cluster c computes tile c, rank q its blocks [q kb / S, (q + 1) kb / S)
  const int S = GROUPED ? 1 : p.split;
  const int rank = S > 1 ? (int)cluster_rank() : 0;
  const int t0 = S > 1 ? (int)blockIdx.x / S : (int)blockIdx.x;
  const int step = S > 1 ? tiles : (int)gridDim.x;
  const int b0 = rank * p.kb / S, b1 = (rank + 1) * p.kb / S;

  if (warp == 0) {
    // ------------------------------------------------------------ weight copies (ahead of the previous grid's end)
    if (elect_one()) {
      int it = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = t0; ok && t < tiles; t += step) {
        const BlockTile tl = block_tile<BN, 128, GROUPED>(p, start, t);
        for (int b = b0; b < b1; ++b, ++it) {
          if (it >= C::ST && !block_wait(&empty[s], ph ^ 1, ctl())) { ok = false; break; }
          mbar_arrive_expect_tx(&full_w[s], C::W_BYTES);
          tma_load_2d(smem + s * C::STAGE, &tmap_w, b * 128, tl.e * p.N + tl.n0, &full_w[s]);
          if (++s == C::ST) { s = 0; ph ^= 1; }
        }
      }
      for (int i = it > C::ST ? it - C::ST : 0; i < it; ++i) block_wait(&full_w[i % C::ST], (i / C::ST) & 1, ctl_drain());
    }
    __syncwarp();
  } else if (!XBF && warp == 2) {
    // ------------------------------------------------------------ activation copies
    if (elect_one()) {
      if constexpr (!GROUPED) pdl_wait();
      int it = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = t0; ok && t < tiles; t += step) {
        const BlockTile tl = block_tile<BN, 128, GROUPED>(p, start, t);
        for (int b = b0; b < b1; ++b, ++it) {
          if (it >= C::ST && !block_wait(&empty[s], ph ^ 1, ctl())) { ok = false; break; }
          mbar_arrive_expect_tx(&full_x[s], C::X_BYTES);
          tma_load_2d(smem + s * C::STAGE + C::W_BYTES, &tmap_x, b * 128, tl.m0, &full_x[s]);
          if (++s == C::ST) { s = 0; ph ^= 1; }
        }
      }
      for (int i = it > C::ST ? it - C::ST : 0; i < it; ++i) block_wait(&full_x[i % C::ST], (i / C::ST) & 1, ctl_drain());
    }
    __syncwarp();
  } else if (!XBF && warp == 3) {
    // ------------------------------------------------------------ scales, fetched four blocks ahead
    if constexpr (!GROUPED) pdl_wait();
    constexpr int CPL = (BN + 31) / 32;                 // rows per lane
    int it = 0, s = 0, e = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int t = t0; ok && t < tiles; t += step) {
      const BlockTile tl = block_tile<BN, 128, GROUPED>(p, start, t);
      const float* sw = p.sw + ((size_t)tl.e * p.nb + (tl.n0 >> 7)) * p.kb;
      const float* sx[CPL];
      bool live[CPL];
      float nx[CPL][4], nw[4];
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        const int m = tl.m0 + lane + 32 * j;
        live[j] = lane + 32 * j < BN && m < tl.m_end;
        sx[j] = p.sx + (size_t)(live[j] ? m : 0) * p.kb;
        load_scales(sx[j], live[j], b0, b1, nx[j]);
      }
      load_scales(sw, true, b0, b1, nw);
      for (int bg = b0; ok && bg < b1; bg += 4) {
        float c[CPL][4];
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) c[j][i] = nx[j][i] * nw[i];
          load_scales(sx[j], live[j], bg + 4, b1, nx[j]);
        }
        load_scales(sw, true, bg + 4, b1, nw);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (bg + i >= b1) break;
          if (it >= C::ST && !block_wait_warp(&empty[s], ph ^ 1, ctl())) { ok = false; break; }
#pragma unroll
          for (int j = 0; j < CPL; ++j)
            if (lane + 32 * j < BN) scales[e * BN + lane + 32 * j] = c[j][i];
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full_x[s]);
            mbar_arrive(&sc_full[e]);
          }
          ++it;
          if (++s == C::ST) { s = 0; ph ^= 1; }
          if (++e == C::SR) e = 0;
        }
      }
    }
  } else if (XBF && warp >= 12) {
    // ------------------------------------------------------------ quantizer: QW warps take the blocks in turn
    if constexpr (!GROUPED) pdl_wait();
    const int w = warp - 12;
    int it = 0;
    bool ok = true;
    for (int t = t0; ok && t < tiles; t += step) {
      const BlockTile tl = block_tile<BN, 128, GROUPED>(p, start, t);
      const float* sw = p.sw + ((size_t)tl.e * p.nb + (tl.n0 >> 7)) * p.kb;
      const int rows = min(BN, tl.m_end - tl.m0);
      uint4 u[4], next[4];
      float su = 0.f, snext = 0.f;
      bool have = false;
      for (int b = b0; b < b1; ++b, ++it) {
        if (it % C::QW != w) continue;
        if (!have) {
          load_rows8(p.x, p.K, tl.m0, 0, rows, b, lane, next);
          snext = sw[b];
          have = true;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = next[i];
        su = snext;
        if (b + C::QW < b1) {
          load_rows8(p.x, p.K, tl.m0, 0, rows, b + C::QW, lane, next);
          snext = sw[b + C::QW];
        }
        const int s = it % C::ST, e = it % C::SR;
        if (it >= C::ST && !block_wait_warp(&empty[s], (uint32_t)(it / C::ST + 1) & 1u, ctl())) { ok = false; break; }
        quantize_stage(u, p.x, p.K, tl.m0, rows, b, su, smem + s * C::STAGE + C::W_BYTES, scales + e * BN, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full_x[s]);
          mbar_arrive(&sc_full[e]);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (elect_one()) {
      int s = 0, pb = 0;
      uint32_t ph = 0, pph = 0;
      bool ok = true, issued = false;
      for (int t = t0; ok && t < tiles; t += step) {
        for (int b = b0; b < b1; ++b) {
          if (!mbar_try_wait3(&full_w[s], ph, &full_x[s], ph, &acc_empty[pb], pph ^ 1) &&
              (!block_wait(&full_w[s], ph, ctl()) || !block_wait(&full_x[s], ph, ctl()) ||
               !block_wait(&acc_empty[pb], pph ^ 1, ctl()))) { ok = false; break; }
          tc_fence_after();
          const uint32_t wb = smem_u32(smem + s * C::STAGE), xb = wb + C::W_BYTES;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8_ss(tmem + pb * BN, sdesc_sw128(wb + kk * 32), sdesc_sw128(xb + kk * 32), idesc_e4m3(BN), kk > 0 ? 1u : 0u);
          issued = true;
          tc_commit(&empty[s]);
          tc_commit(&acc_full[pb]);
          if (++s == C::ST) { s = 0; ph ^= 1; }
          if (++pb == C::PB) { pb = 0; pph ^= 1; }
        }
      }
      if (issued) {
        tc_commit(drain);
        block_wait(drain, 0, ctl_drain());
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ scaling, sum and output
    if constexpr (!GROUPED) pdl_wait();
    const int qd = warp & 3, h = (warp - 4) >> 2;
    const int r = qd * 32 + lane;                       // channel within the tile
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
    constexpr int LD = C::HALF < 32 ? C::HALF : 32;
    int pb = 0, e = 0;
    uint32_t pph = 0, eph = 0;
    bool ok = true;
    for (int t = t0; ok && t < tiles; t += step) {
      const BlockTile tl = block_tile<BN, 128, GROUPED>(p, start, t);
      float acc[C::HALF];
#pragma unroll
      for (int i = 0; i < C::HALF; ++i) acc[i] = 0.f;
      for (int b = b0; b < b1; ++b) {
        if (!block_wait_warp2(&sc_full[e], eph, &acc_full[pb], pph, ctl())) { ok = false; break; }
        tc_fence_after();
        const float* f = scales + e * BN + h * C::HALF;
#pragma unroll
        for (int c0 = 0; c0 < C::HALF; c0 += LD) {
          float v[LD];
          tmem_ld_n<LD>(tmem + lane_base + pb * BN + h * C::HALF + c0, v);
          tmem_wait_regs<LD>(v);
#pragma unroll
          for (int c = 0; c < LD; c += 4) {
            const float4 q = *reinterpret_cast<const float4*>(f + c0 + c);
            acc[c0 + c] = fmaf(v[c], q.x, acc[c0 + c]);
            acc[c0 + c + 1] = fmaf(v[c + 1], q.y, acc[c0 + c + 1]);
            acc[c0 + c + 2] = fmaf(v[c + 2], q.z, acc[c0 + c + 2]);
            acc[c0 + c + 3] = fmaf(v[c + 3], q.w, acc[c0 + c + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[pb]);
        if (++pb == C::PB) { pb = 0; pph ^= 1; }
        if (++e == C::SR) { e = 0; eph ^= 1; }
      }
      if (!ok) break;
      if (S == 1) {
        const int n = tl.n0 + r;
        if (n < p.N) {
          const float bias = p.bias ? __bfloat162float(p.bias[(size_t)tl.e * p.N + n]) : 0.f;
#pragma unroll
          for (int i = 0; i < C::HALF; ++i) {
            const int m = tl.m0 + h * C::HALF + i;
            if (m < tl.m_end) p.y[(size_t)m * p.N + n] = __float2bfloat16_rn(acc[i] + bias);
          }
        }
      } else {
        // every MMA of this CTA has completed: the ring is free for the partial [column][channel]
        float* red = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int i = 0; i < C::HALF; ++i) red[(h * C::HALF + i) * 128 + r] = acc[i];
      }
    }
    if (!ok) {
      *abort_flag = 1;
      *bad = 1;
    }
    __syncwarp();
  }

  if (S > 1) {
    __syncwarp();
    cluster_sync();   // every partial (or its absence) is in its CTA's shared memory
    if (warp >= 4 && warp < 12) {
      const BlockTile tl = block_tile<BN, 128, GROUPED>(p, start, t0);
      const int cols = BN / S;                        // S is a power of two <= 8 <= BN
      bool good = true;
      for (int q = 0; q < S; ++q) good = good && ld_dsmem_u32(dsmem_addr(const_cast<uint32_t*>(bad), q)) == 0u;
      if (good) {
        // four channels of a column at a time, every rank's partials on their
        // way before the first is added (one by one 128 x 4096 x 4096 took
        // 14.1 us)
        const uint32_t base = smem_u32(smem);
        for (int i = threadIdx.x - 128; i < cols * 32; i += 256) {
          const int c = rank * cols + (i >> 5), r = (i & 31) * 4;
          float4 v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < S) v[q] = ld_dsmem_f4(base + (uint32_t)(c * 128 + r) * 4, q);
#pragma unroll
          for (int q = 1; q < 8; ++q) {
            if (q < S) {
              v[0].x += v[q].x;
              v[0].y += v[q].y;
              v[0].z += v[q].z;
              v[0].w += v[q].w;
            }
          }
          const int n = tl.n0 + r, m = tl.m0 + c;
          if (m < tl.m_end) {
            const float o[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
            __nv_bfloat16* y = p.y + (size_t)m * p.N + n;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (n + j < p.N) y[j] = __float2bfloat16_rn(o[j] + (p.bias ? __bfloat162float(p.bias[n + j]) : 0.f));
          }
        }
      }
    }
    __syncwarp();
    cluster_sync();   // no CTA leaves while its shared memory is read
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, C::TMEM_COLS);
}

// ---------------------------------------------------------------------------
// pair: 256 rows x 256 channels by two CTAs
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {   // one warp of each CTA
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (256 rows over the pair) (+)= A . B^T, each CTA holding half of A's and of B's rows
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrive on the barrier of both CTAs when the MMAs issued so far are done
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// Between the two CTAs.  `addr`: a barrier of either, as the cluster addresses
// it.  An arrival orders nothing by itself (relaxed), and need not:
//  - on acc_empty it follows tcgen05.wait::ld and tcgen05.fence::before_thread_sync,
//    and the MMA thread's wait is followed by tcgen05.fence::after_thread_sync:
//    the pair of fences orders tensor memory across any wait of their scope;
//  - on full it only announces bytes.  What the MMAs read is published by the
//    copies themselves, whose completion on the barrier is a release at cluster
//    scope, and the MMA thread's wait there acquires at cluster scope.
// (With a release on every arrival of the epilogue the large product took 1187 us, not 888.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(addr), "r"(bytes)
               : "memory");
}
// a tile into this CTA's shared memory, its bytes counted on a barrier of either CTA
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Waits on barriers that the other CTA completes: their scope is the cluster.
// ACQUIRE false: for tensor memory, with a tcgen05 fence behind the wait.
template <bool ACQUIRE>
__device__ __forceinline__ bool mbar_try_wait_pair(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (ACQUIRE)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  return ok != 0;
}
// as block_wait
template <bool ACQUIRE>
__device__ __forceinline__ bool block_wait_pair(uint64_t* bar, uint32_t parity, const WaitCtl ctl) {
  if (mbar_try_wait_pair<ACQUIRE>(bar, parity)) return true;
  uint64_t t0 = 0;
  for (int round = 0;; ++round) {
    if (round > 0 || ctl.timeout_ns < 1000u) {
      if (t0 == 0) t0 = globaltimer_ns();
      if (wait_give_up(ctl, t0)) return false;
    }
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait_pair<ACQUIRE>(bar, parity)) return true;
  }
}
// as block_wait_warp, for tensor memory
__device__ __forceinline__ bool block_wait_warp_pair(uint64_t* bar, uint32_t parity, const WaitCtl ctl) {
  uint64_t t0 = 0;
  for (int i = ctl.timeout_ns < 1000u ? 63 : 0;; ++i) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait_pair<false>(bar, parity))) return true;
    if ((i & 63) == 63) {
      if (t0 == 0) t0 = globaltimer_ns();
      if (__any_sync(0xFFFFFFFFu, wait_give_up(ctl, t0))) return false;
    }
  }
}
// the stage's copies have landed and the buffer has been read, looked at together
__device__ __forceinline__ bool pair_ready(uint64_t* full, uint32_t pf, uint64_t* acc_empty, uint32_t pe) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(full)), "r"(pf), "r"(smem_u32(acc_empty)), "r"(pe)
      : "memory");
  return ok != 0;
}

// shared -> global, complete in the issuing thread's bulk group
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile(
      "cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\t"
      "cp.async.bulk.commit_group;" ::"l"(dst),
      "r"(smem_u32(src)), "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// a look at a barrier whose answer is used later (as mbar_try_wait_pair<false>)
__device__ __forceinline__ uint32_t mbar_peek(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok;
}

struct PairCfg {
  static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int ST = 4;
  static constexpr int PB = 2;                  // partial buffers of 2 x 128 columns: all of TMEM
  static constexpr int TMEM_COLS = 512;
  static constexpr int BAR_OFF = ST * STAGE;
  static constexpr int BAR_BYTES = 256;
  // output staging: a row of 128 bf16 per epilogue thread, rows 272 bytes
  // apart (16-byte pieces of 8 neighbouring rows then lie in different banks)
  static constexpr int OUT_PITCH = 272;
  static constexpr int OUT_OFF = BAR_OFF + BAR_BYTES;
  static constexpr int OUT_BYTES = 256 * OUT_PITCH;
  static constexpr int TAB_OFF = OUT_OFF + OUT_BYTES;
  static constexpr int SMEM = TAB_OFF + (MAX_EXPERTS + 1) * 4 + 1024;
  static constexpr int THREADS = 384;   // 4 warps of copies and MMAs, 8 of sums
  // M = 256, N = 256, e4m3 x e4m3 -> f32
  static constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
  // registers: 128 threads at 64 (fewer spill), 256 at 208, out of the launch's 384 x 168
  static constexpr int REGS_LOW = 64, REGS_HIGH = 208;
  static_assert(128 * REGS_LOW + 256 * REGS_HIGH <= 384 * 168, "register split");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <bool GROUPED>
__global__ void __launch_bounds__(384, 1) __cluster_dims__(2, 1, 1)
    block_pair_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                      const BlockParams p) {
  using C = PairCfg;
  extern __shared__ uint8_t smem_raw[];
  // (the same offset in both CTAs: the dynamic base is the same)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);   // leader: both CTAs' copies of a stage have landed
  uint64_t* empty = full + C::ST;            // both: the pair's MMAs have read the stage
  uint64_t* acc_full = empty + C::ST;        // both
  uint64_t* acc_empty = acc_full + 2 * C::PB;    // leader: the 8 + 8 epilogue warps have read a buffer
  uint64_t* drain = acc_empty + 2 * C::PB;       // both: every MMA of a half is done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // how this CTA ended, and how the other did: stages filled << 3 | MMAs issued in half h << (1 + h) | a wait gave up
  volatile uint32_t* ended = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);
  volatile uint32_t* other_ended = reinterpret_cast<volatile uint32_t*>(tmem_slot + 3);
  volatile uint32_t* issued_flag = reinterpret_cast<volatile uint32_t*>(tmem_slot + 4);   // [2]
  static_assert((2 * C::ST + 4 * C::PB + 2) * 8 + 24 <= C::BAR_BYTES, "barriers");
  int* start = reinterpret_cast<int*>(smem + C::TAB_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();   // 0: the leader, which issues the MMAs
  const auto ctl = [&] { return WaitCtl{abort_flag, p.status, p.timeout_ns}; };
  const auto ctl_drain = [&] { return WaitCtl{nullptr, p.status, p.drain_ns}; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(&full[s], 2);   // each CTA announces its own bytes
      mbar_init(&empty[s], 2);
    }
    for (int b = 0; b < 2 * C::PB; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);   // 4 warps of each CTA
    }
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
    *abort_flag = 0;
    *ended = 0;
    issued_flag[0] = issued_flag[1] = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the other CTA's barriers are initialized
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();

  int tiles;
  if constexpr (GROUPED) {
    pdl_wait();
    count_tiles<256>(p, start);
    tiles = start[p.E] * p.n_tiles;
  } else {
    tiles = p.n_tiles * p.m_tiles;
  }
  const int t0 = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_LOW));
    if (warp == 0) {
      // ---------------------------------------------------------- copies
      if (elect_one()) {
        if constexpr (!GROUPED) pdl_wait();
        const uint32_t full_addr = dsmem_addr(full, 0);
        int it = 0, s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int t = t0; ok && t < tiles; t += step) {
          const BlockTile tl = block_tile<256, 256, GROUPED>(p, start, t);
          for (int b = 0; b < p.kb; ++b, ++it) {
            if (it >= C::ST && !block_wait_pair<true>(&empty[s], ph ^ 1, ctl())) { ok = false; break; }
            const uint32_t bar = full_addr + s * 8;
            mbar_arrive_expect_tx_cluster(bar, C::STAGE);
            tma_load_2d_pair(smem + s * C::STAGE, &tmap_x, b * 128, tl.m0 + rank * 128, bar);
            tma_load_2d_pair(smem + s * C::STAGE + C::A_BYTES, &tmap_w, b * 128, tl.e * p.N + tl.n0 + rank * 64, bar);
            tma_load_2d_pair(smem + s * C::STAGE + C::A_BYTES + 8192, &tmap_w, b * 128, tl.e * p.N + tl.n0 + 128 + rank * 64, bar);
            if (++s == C::ST) { s = 0; ph ^= 1; }
          }
        }
        *ended = (uint32_t)it << 3;
        // the leader's last signals have arrived before this CTA can leave
        for (int i = it > C::ST ? it - C::ST : 0; ok && i < it; ++i)
          ok = block_wait_pair<true>(&empty[i % C::ST], (i / C::ST) & 1, ctl());
      }
    } else if ((warp == 1 || warp == 3) && rank == 0) {
      // ---------------------------------------------------------- MMA
      if (elect_one()) {
        const int h = warp == 1 ? 0 : 1;
        int s = 0, pb = 0;
        uint32_t ph = 0, pph = 0;
        bool ok = true, issued = false;
        for (int t = t0; ok && t < tiles; t += step) {
          for (int b = 0; b < p.kb; ++b) {
            // (one after the other the two looks cost two latencies)
            if (!pair_ready(&full[s], ph, &acc_empty[h * 2 + pb], pph ^ 1) &&
                (!block_wait_pair<true>(&full[s], ph, ctl()) ||
                 !block_wait_pair<false>(&acc_empty[h * 2 + pb], pph ^ 1, ctl()))) { ok = false; break; }
            tc_fence_after();
            const uint32_t ab = smem_u32(smem + s * C::STAGE), bb = ab + C::A_BYTES + h * 8192;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8_pair(tmem + pb * 256 + h * 128, sdesc_sw128(ab + kk * 32), sdesc_sw128(bb + kk * 32), C::IDESC, kk > 0 ? 1u : 0u);
            issued = true;
            tc_commit_pair(&empty[s]);
            tc_commit_pair(&acc_full[h * 2 + pb]);
            if (++s == C::ST) { s = 0; ph ^= 1; }
            if (++pb == C::PB) { pb = 0; pph ^= 1; }
          }
        }
        if (issued) {
          issued_flag[h] = 1u;
          tc_commit_pair(drain + h);
          block_wait(drain + h, 0, ctl_drain());
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scaling, sum and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_HIGH));
    if constexpr (!GROUPED) pdl_wait();
    const int qd = warp & 3, h = (warp - 4) >> 2;   // 32 rows x half h of the tile's columns
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
    uint32_t ready = 0;   // the next block's partial was complete when last looked at
    const uint32_t empty_addr = dsmem_addr(acc_empty, 0);
    int pb = 0;
    uint32_t pph = 0;
    bool ok = true;
    for (int t = t0; ok && t < tiles; t += step) {
      const float *sxr, *sw;
      bool live, live_n;   // this row and half exist
      {
        const BlockTile tl = block_tile<256, 256, GROUPED>(p, start, t);
        const int m = tl.m0 + rank * 128 + qd * 32 + lane, n0 = tl.n0 + h * 128;
        live = m < tl.m_end;
        live_n = n0 < p.N;
        sxr = p.sx + (size_t)(live ? m : 0) * p.kb;
        sw = p.sw + ((size_t)tl.e * p.nb + (live_n ? n0 >> 7 : 0)) * p.kb;
      }
      // (the next block's scales are fetched while this one is summed: mostly
      // from L1, a row's 32 consecutive blocks share a line)
      float nx = live ? sxr[0] : 0.f, nw = live_n ? sw[0] : 0.f;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      for (int b = 0; b < p.kb; ++b) {
        const float s1 = nx * nw;
        if (b + 1 < p.kb) {
          if (live) nx = sxr[b + 1];
          if (live_n) nw = sw[b + 1];
        }
        if (!__all_sync(0xFFFFFFFFu, ready) && !block_wait_warp_pair(&acc_full[h * 2 + pb], pph, ctl())) { ok = false; break; }
        tc_fence_after();
        const uint32_t ta = tmem + lane_base + pb * 256 + h * 128;
        uint64_t* next_bar = &acc_full[h * 2 + (pb ^ 1)];
        const uint32_t next_par = pb ? pph ^ 1 : pph;
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 16) {
          float v[16];
          tmem_ld_n<16>(ta + c0, v);
          tmem_wait_regs<16>(v);
          if (c0 + 16 == 128) {   // the buffer is free as soon as the last columns have arrived
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(empty_addr + (h * 2 + pb) * 8);
            ready = mbar_peek(next_bar, next_par);   // (its answer arrives during the last sums)
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) acc[c0 + c] = fmaf(v[c], s1, acc[c0 + c]);
        }
        if (++pb == C::PB) { pb = 0; pph ^= 1; }
      }
      if (!ok) break;
      // Out through shared memory: each thread leaves its row there and hands
      // it to the copy engine, which writes it while the next tile is summed
      // (stores from the registers touch 32 rows an instruction: 5000 cycles
      // a tile against 32 x 512 of MMAs).
      if (live_n) {
        // (where the tile lies is found again: kept over the sums it would cost
        // registers that they have not)
        const BlockTile tl = block_tile<256, 256, GROUPED>(p, start, t);
        const int m = tl.m0 + rank * 128 + qd * 32 + lane, n0 = tl.n0 + h * 128;
        const __nv_bfloat16* bias = p.bias ? p.bias + (size_t)tl.e * p.N + n0 : nullptr;
        const int nn = min(128, p.N - n0);
        uint8_t* mine = smem + C::OUT_OFF + (threadIdx.x - 128) * C::OUT_PITCH;
        bulk_wait_read();   // this thread's last row has left
        if (bias && nn == 128 && (reinterpret_cast<uintptr_t>(bias) & 15) == 0) {   // (one by one: 1.9 us a tile)
#pragma unroll
          for (int c = 0; c < 128; c += 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(bias + c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              acc[c + 2 * k] += __uint_as_float(w[k] << 16);
              acc[c + 2 * k + 1] += __uint_as_float(w[k] & 0xFFFF0000u);
            }
          }
        } else if (bias) {
#pragma unroll
          for (int c = 0; c < 128; ++c) acc[c] += c < nn ? __bfloat162float(bias[c]) : 0.f;
        }
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 v2 = __floats2bfloat162_rn(acc[c + 2 * k], acc[c + 2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&v2);
          }
          sts128(mine + c * 2, make_uint4(w[0], w[1], w[2], w[3]));
        }
        if (p.vec_y) {   // (N a multiple of 8: whole 16-byte pieces)
          fence_proxy_async_smem();
          if (live) bulk_s2g(p.y + (size_t)m * p.N + n0, mine, (uint32_t)nn * 2);
        } else {
          __syncwarp();
          const int mw = m - lane, rows = min(32, tl.m_end - mw);
          for (int r = 0; r < rows; ++r)
            for (int c = lane; c < nn; c += 32)
              p.y[(size_t)(mw + r) * p.N + n0 + c] =
                  *reinterpret_cast<const __nv_bfloat16*>(mine + (r - lane) * C::OUT_PITCH + c * 2);
          __syncwarp();
        }
      }
    }
    bulk_wait_all();
    if (!ok) *abort_flag = 1;
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t e = *ended | issued_flag[0] << 1 | issued_flag[1] << 2 | (*abort_flag ? 1u : 0u);
    *ended = e;
    st_dsmem_u32(dsmem_addr(const_cast<uint32_t*>(other_ended), rank ^ 1), e);
  }
  __syncwarp();
  // both CTAs are done with each other's barriers, shared and tensor memory
  // (where no wait gave up: every copy was waited for by an MMA, every MMA by
  // an epilogue warp)
  cluster_sync();
  const uint32_t mine = *ended, other = *other_ended;
  const bool gave_up = (mine | other) & 1u;
  if (warp == 0 && elect_one()) {
    if (gave_up) {
      // Copies and MMAs of either CTA may still run: they end before this CTA's
      // shared memory is given back.  A CTA has filled at most ST stages more
      // than the other; for those the other arrives too, with no bytes, so
      // that each phase the leader waits for here completes.
      const int a = (int)(mine >> 3), b = (int)(other >> 3), last = max(a, b);
      for (int i = a; i < b; ++i) mbar_arrive_cluster(dsmem_addr(full, 0) + (i % C::ST) * 8);
      for (int i = last > C::ST ? last - C::ST : 0; rank == 0 && i < last; ++i)
        block_wait_pair<true>(&full[i % C::ST], (i / C::ST) & 1, ctl_drain());
    }
    // the leader's last signal of each half (the leader has waited for its own)
    for (int h = 0; rank == 1 && h < 2; ++h)
      if (other >> (1 + h) & 1u) block_wait_pair<true>(drain + h, 0, ctl_drain());
  }
  __syncwarp();
  if (gave_up) cluster_sync();
  tc_fence_after();
  if (warp == 0) tmem_dealloc_pair(tmem, C::TMEM_COLS);
}

// ---------------------------------------------------------------------------
// weight packing, checking and (debug) dequantization
// ---------------------------------------------------------------------------

// one CTA of 256 threads per 128 x 128 block of W fp32 [N, K]
__global__ void __launch_bounds__(256) pack_fp8_block_kernel(const float* W, int N, int K, uint8_t* codes, float* scales) {
  const int bn = blockIdx.y, bk = blockIdx.x;
  const int rows = min(128, N - bn * 128), cols = min(128, K - bk * 128);
  const float* w = W + (size_t)bn * 128 * K + bk * 128;
  uint8_t* c = codes + (size_t)bn * 128 * K + bk * 128;
  const int col = threadIdx.x & 127, r0 = threadIdx.x >> 7;
  float a = 0.f;
  if (col < cols)
    for (int r = r0; r < rows; r += 2) a = fmaxf(a, fabsf(w[(size_t)r * K + col]));
#pragma unroll
  for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  __shared__ float wmax[8];
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, wmax[i]);
  const float s = fdiv(a, 448.f);
  if (threadIdx.x == 0) scales[(size_t)bn * gridDim.x + bk] = s;
  if (col < cols)
    for (int r = r0; r < rows; r += 2)
      c[(size_t)r * K + col] = s > 0.f ? e4m3_encode_sat(fdiv(w[(size_t)r * K + col], s)) : 0;
}

// *flag becomes nonzero for a NaN code or a scale that is negative, infinite or NaN
__global__ void check_fp8_block_kernel(const uint8_t* codes, size_t count, const float* scales, size_t ns, int* flag) {
  int bad = 0;
  const size_t i0 = blockIdx.x * (size_t)blockDim.x + threadIdx.x, step = (size_t)gridDim.x * blockDim.x;
  for (size_t i = i0; i < count / 16; i += step) {
    const uint4 v = reinterpret_cast<const uint4*>(codes)[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)   // a byte of 0x7F or 0xFF: its low 7 bits all set
      bad |= ((((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u) ? 1 : 0;
  }
  for (size_t i = i0; i < ns; i += step) bad |= (scales[i] >= 0.f && scales[i] <= 3.402823466e38f) ? 0 : 2;
  if (bad) *reinterpret_cast<volatile int*>(flag) = bad;   // (any writer's value refuses the weight)
}

__global__ void dequant_fp8_block_kernel(const uint8_t* codes, const float* scales, size_t rows, int N, int K,
                                         __nv_bfloat16* out) {
  const int kb = (K + 127) / 128, nb = (N + 127) / 128;
  for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < rows * K; i += (size_t)gridDim.x * blockDim.x) {
    const size_t row = i / K;
    const int k = (int)(i - row * K), e = (int)(row / N), n = (int)(row - (size_t)e * N);
    const float s = scales[((size_t)e * nb + n / 128) * kb + k / 128];
    out[i] = __float2bfloat16_rn(__fmul_rn(e4m3_decode(codes[i]), s));
  }
}

}  // namespace dq
