// Linear layer out = residual + act(x w^T + bias) and its gradients on the 5th-generation tensor
// cores (bf16 operands, fp32 accumulation in tensor memory).
//
// One kernel serves the three products, since each operand tile may be K-major (the reduction runs
// along its rows) or MN-major (the reduction runs down its columns), which the shared-memory
// descriptors express without a transpose:
//   out [M, N] = x [M, K] . w [N, K]^T    both K-major
//   dx  [M, K] = dz [M, N] . w [N, K]     dz K-major, w MN-major
//   dw  [N, K] = dz [M, N]^T . x [M, K]   both MN-major
//
// Bound by the tensor pipe for many rows. A persistent CTA per SM walks output tiles; one warp issues
// TMA loads into a ring of 64-deep slices, one issues the MMAs, eight turn accumulators into
// outputs. The accumulator is double-buffered in tensor memory, so the epilogue of one tile (bias,
// activation, residual, rounding, and a TMA store per warp out of swizzled shared memory) runs
// under the products of the next. Large products run on pairs of SMs: a 256 x 256 (or 256 x 128)
// tile, of which each CTA loads its 128 rows of A and its half of B's rows, and one thread issues the
// MMAs for both. That halves what shared memory takes in per product for B (33272 x 4096 -> 16384 in bursts of
// five calls: 2.99 to 3.04 ms, 1.47 to 1.49 PFLOP/s, and 3.07 to 3.09 with bias and gelu; 3.47 and 3.53 in calls on
// end, under the power cap; tiles of 128 x 256 on single SMs, bursts: 3.07 and 3.09). Few tiles go to single SMs,
// 128 x 128 or 128 x 64 each, to fill more of them; with a long reduction and a workspace, the tiles past the last
// whole turn of the SMs go in pieces of the reduction, which a second kernel adds (200 x 4096 -> 4096, weights from
// DRAM: 33 us whole, 19 us).
//
// With up to kFewRows rows the layer is bound by reading w once. There the product is taken
// transposed: 128 rows of w are the M side of the MMA and the tokens its N side, so the ring holds
// almost nothing but w. The reduction is split over the CTAs of a cluster to have enough loads in
// flight, and the cluster adds its fp32 partial tiles over distributed shared memory in rank order,
// so no workspace and no atomics are needed and the bits do not depend on timing.
//
// Every wait is bounded: on expiry the CTA records the timeout in the caller's workspace (where one
// is given), lets its copies and MMAs in flight end, frees its tensor memory and returns. What it could not
// compute it stores as NaN, also in what other CTAs add to theirs, so that the data tell without a workspace.
#include <cmath>
#include <type_traits>

#include "chained.cuh"
#include "device_common.cuh"
#include "launchers.h"

namespace sol {

namespace {

constexpr int BM = 128;            // output rows per tile
constexpr int BK = 64;             // reduction depth per slice: one 128-byte swizzle row of bf16
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kEpiWarps;
constexpr int kEpiBuf = 32 * 64;   // one warp's staging buffer: 32 rows x 32 bf16 columns
// A piece of a split tile has at least so many slices; the pieces cost their fp32 tiles through memory and a
// second kernel.
constexpr int kPieceSlices = 16;
constexpr double kPieceCycles = 9000.0;
// Output rows walked together, column by column: at least 2048, so that a wave of tiles is about square
// and its tiles share operands as they stream by; with a short reduction as many as keep their part
// of A in L2 while B passes (at K = 4096, 4096 rows instead of 2048: 3085 against 3140 us, gelu included).
constexpr int kGroupRows = 2048;
constexpr double kGroupBytes = 33554432.0;

// CG: CTAs of a tile, 1 or 2 (a cluster); each has 128 of its rows and TN / CG of B's rows.
template <int CG, int TN>
struct GemmCfg {
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_ROWS = TN / CG;
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = 196608 / STAGE;  // 6 or 8 slices of 32 or 24 KB
  static constexpr int OFF_EPI = NS * STAGE;
  static constexpr int OFF_BAR = OFF_EPI + kEpiWarps * 2 * kEpiBuf;
  static constexpr int OFF_COUNT = OFF_BAR + 16 * NS + 48 + 16 * kEpiWarps;  // behind the barriers
  static constexpr int SMEM = OFF_BAR + 384 + 1024;  // + alignment of the ring to 1024 bytes
  static_assert(OFF_COUNT + 16 <= OFF_BAR + 384, "barriers and flags");
  static constexpr int TMEM_COLS = 2 * TN;
};

struct GemmParams {
  int Mo, No, nk;  // output rows and columns, reduction slices
  int tiles_m, tiles_n;
  int group;             // row tiles walked together
  int whole, split;      // units from `whole` on are pieces of the last tiles, `split` of each
  float* part;           // their fp32 accumulators, or null
  const float* bias;               // [No] or null
  int act;
  int has_residual, store_z;
  int drop;      // DROP_*: a copy left out, for the tests of expired waits
  uint64_t wait_limit_ns;
  uint32_t* ws;  // error words, or null
};

// ---- activations and their slopes, two values at a time ------------------------------------------------
__device__ __forceinline__ f2 dup2(float v) { return pack2(v, v); }
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ f2 ex2_2(f2 x) {
  const float2 v = unpack2(x);
  return pack2(ex2_approx(v.x), ex2_approx(v.y));
}
__device__ __forceinline__ f2 rcp_2(f2 x) {
  const float2 v = unpack2(x);
  return pack2(rcp_approx(v.x), rcp_approx(v.y));
}
// 1 / (1 + 2^x): both ends are right without a branch, 2^x = inf gives 0.
__device__ __forceinline__ f2 sigmoid_ex2(f2 x) { return rcp_2(add2(ex2_2(x), dup2(1.0f))); }

// The normal distribution's Phi(z), with e = exp(-z^2 / 2), which its density shares. From erfc(x) =
// (a1 t + .. + a5 t^5) exp(-x^2), t = 1 / (1 + 0.3275911 x), x >= 0, of Abramowitz and Stegun, 7.1.26
// (after Hastings), off by at most 1.5e-7: half of that here, a bf16 step of values near 1 is 2e-3.
__device__ __forceinline__ f2 normal_cdf(f2 z, f2& e) {
  e = ex2_2(mul2(mul2(z, z), dup2(-0.72134752044448170f)));
  const float2 v = unpack2(z);
  const f2 t = rcp_2(fma2(pack2(fabsf(v.x), fabsf(v.y)), dup2(0.3275911f * 0.70710678118654752f), dup2(1.0f)));
  f2 q = fma2(t, dup2(0.5f * 1.061405429f), dup2(0.5f * -1.453152027f));
  q = fma2(q, t, dup2(0.5f * 1.421413741f));
  q = fma2(q, t, dup2(0.5f * -0.284496736f));
  q = fma2(q, t, dup2(0.5f * 0.254829592f));
  const float2 h = unpack2(mul2(mul2(q, t), e));  // the tail beyond |z|
  return pack2(v.x < 0.f ? h.x : 1.0f - h.x, v.y < 0.f ? h.y : 1.0f - h.y);
}
// -2 log2(e) sqrt(2 / pi) (z + 0.044715 z^3): the tanh form of gelu is z times the sigmoid of it
__device__ __forceinline__ f2 gelu_tanh_arg(f2 z, f2 z2) {
  return mul2(z, fma2(z2, dup2(-2.3022082f * 0.044715f), dup2(-2.3022082f)));
}

template <int ACT>
__device__ __forceinline__ f2 activate(f2 z) {
  if constexpr (ACT == ACT_GELU) {
    f2 e;
    return mul2(z, normal_cdf(z, e));
  } else if constexpr (ACT == ACT_GELU_TANH) {
    return mul2(z, sigmoid_ex2(gelu_tanh_arg(z, mul2(z, z))));
  } else if constexpr (ACT == ACT_SILU) {
    return mul2(z, sigmoid_ex2(mul2(z, dup2(-1.4426950408889634f))));
  } else {
    return z;
  }
}
template <int ACT>
__device__ __forceinline__ f2 activation_slope(f2 z) {
  if constexpr (ACT == ACT_GELU) {
    f2 e;
    const f2 c = normal_cdf(z, e);
    return fma2(mul2(z, dup2(0.39894228040143268f)), e, c);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    // s + z s (1 - s) 2 sqrt(2 / pi) (1 + 3 0.044715 z^2). Beyond |z| = 100, s is 0 or 1 and its product with 1 - s 0:
    // the cubic stays finite there, so that the slope does, up to the largest z
    const float2 q = unpack2(mul2(z, z));
    const f2 z2 = pack2(fminf(q.x, 1e4f), fminf(q.y, 1e4f)), s = sigmoid_ex2(gelu_tanh_arg(z, z2));
    const f2 g = mul2(z, mul2(s, fma2(s, dup2(-1.0f), dup2(1.0f))));
    return fma2(g, fma2(z2, dup2(1.5957691216057308f * 3.0f * 0.044715f), dup2(1.5957691216057308f)), s);
  } else if constexpr (ACT == ACT_SILU) {
    const f2 s = sigmoid_ex2(mul2(z, dup2(-1.4426950408889634f)));
    return mul2(s, fma2(z, fma2(s, dup2(-1.0f), dup2(1.0f)), dup2(1.0f)));
  } else {
    return dup2(1.0f);
  }
}
// f(its constant) for the activation of a call
template <typename F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  switch (act) {
    case ACT_GELU: f(std::integral_constant<int, ACT_GELU>{}); break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>{}); break;
    case ACT_SILU: f(std::integral_constant<int, ACT_SILU>{}); break;
    default: break;
  }
}

// ---- small PTX helpers of this file -----------------------------------------------------------------
// CG = 2: the barrier may lie in the other CTA of the pair.
template <int CG = 1>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, uint32_t bar, int x, int y) {
  if constexpr (CG == 1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
               ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
// The address of this CTA's shared memory `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}

// The tcgen05 operations that differ for a pair of CTAs.
template <int CG>
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  if constexpr (CG == 1) {
    tmem_alloc(dst_smem, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  if constexpr (CG == 1) tmem_dealloc(taddr, ncols);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
template <int CG>
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 1) {
    mma_bf16_ss(d_tmem, a_desc, b_desc, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// Arrive on `bar`, of a pair in both CTAs, when the operations issued so far have completed.
template <int CG>
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  if constexpr (CG == 1) {
    tc_commit(bar);
  } else {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(bar), "h"(static_cast<uint16_t>(3))
                 : "memory");
  }
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Two counts to the other CTA of the pair: 8 bytes to `dst`, reported to `bar`, both as they lie in this CTA.
__device__ __forceinline__ void send_counts(uint32_t dst, uint32_t bar, uint32_t to, uint32_t a, uint32_t b) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];"
               ::"r"(in_cta(dst, to)), "l"(static_cast<uint64_t>(b) << 32 | a), "r"(in_cta(bar, to))
               : "memory");
}
// All threads of the CTA, or of the pair.
template <int CG>
__device__ __forceinline__ void pair_sync() {
  if constexpr (CG == 1) __syncthreads();
  else cluster_arrive_wait();
}

// Records an expired wait: stops the CTA's other roles and, where there is a workspace, tells the host.
__device__ __forceinline__ void report(volatile int* abort_flag, uint32_t* ws, uint32_t where) {
  if (ws != nullptr) raise_timeout(abort_flag, ws, where);
  else *abort_flag = 1;
}

constexpr uint32_t instr_desc(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16_f32(M, N, b_mn) | (a_mn ? 1u << 15 : 0u);
}

// For the tests of expired waits: the slice of an operand whose copy this CTA leaves out, if any.
__device__ __forceinline__ uint32_t left_out(int drop) {
  return drop == (blockIdx.x == 0 ? DROP_OPERAND : blockIdx.x == 1 ? DROP_OPERAND_SECOND : -1) ? 1u : ~0u;
}

// Before a CTA's shared memory is released: every commit to its barriers has arrived. Commits to different
// barriers arrive in no stated order, so the last phase of each is waited for: `slices` commits went around
// the ring, `accs` to the accumulators' barriers, one to `bar_last`.
template <int NS>
__device__ __forceinline__ void settle(uint32_t bar_empty, uint32_t slices, uint32_t bar_acc, uint32_t accs, uint32_t bar_last,
                                       uint64_t limit) {
  for (uint32_t i = slices > NS ? slices - NS : 0; i < slices; ++i)
    mbar_wait(bar_empty + 8 * (i % NS), (i / NS) & 1u, nullptr, limit);
  for (uint32_t i = accs > 2 ? accs - 2 : 0; i < accs; ++i) mbar_wait(bar_acc + 8 * (i & 1u), (i >> 1) & 1u, nullptr, limit);
  mbar_wait(bar_last, 0, nullptr, limit);
}

// One 64-deep slice of an operand: `rows` rows along its M or N side, starting at r0, reduction from
// k0. K-major: one box of 64 x rows. MN-major: boxes of 64 (M or N) x 64 (reduction), 8 KB each.
template <int CG, bool MN>
__device__ __forceinline__ void load_operand(uint32_t dst, const void* tmap, uint32_t bar, int r0, int rows, int k0) {
  if constexpr (!MN) {
    tma_load_2d<CG>(dst, tmap, bar, k0, r0);
  } else {
    for (int i = 0; i < rows / 64; ++i) tma_load_2d<CG>(dst + i * 8192, tmap, bar, r0 + 64 * i, k0);
  }
}
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
  return MN ? smem_desc_sw128(saddr, 8192, 1024) : smem_desc_sw128(saddr, 16, 1024);
}
// descriptor step of 16 reduction elements: 32 bytes along a row, or 16 rows of 128 bytes
template <bool MN>
constexpr uint32_t kDescStep = MN ? 2048 >> 4 : 32 >> 4;

// A unit of work: a tile, or one of `split` pieces of the reduction of one of the last tiles, which
// would otherwise leave most SMs idle while they take a whole turn.
struct Unit {
  int tm, tn, k_lo, k_hi;
};
__device__ __forceinline__ int unit_count(const GemmParams& p) {
  return p.whole + (p.tiles_m * p.tiles_n - p.whole) * p.split;
}
__device__ __forceinline__ Unit unit_of(const GemmParams& p, int u) {
  Unit w;
  int t = u;
  w.k_lo = 0;
  w.k_hi = p.nk;
  if (u >= p.whole) {
    const int v = u - p.whole, piece = v % p.split;
    t = p.whole + v / p.split;
    w.k_lo = static_cast<int>(static_cast<long long>(p.nk) * piece / p.split);
    w.k_hi = static_cast<int>(static_cast<long long>(p.nk) * (piece + 1) / p.split);
  }
  const int per_group = p.group * p.tiles_n;
  const int g = t / per_group, in = t - g * per_group;
  const int rows = min(p.group, p.tiles_m - g * p.group);
  w.tm = g * p.group + in % rows;
  w.tn = in / rows;
  return w;
}

// Where unit `u`, a piece, keeps the 32 x 32 sums of CTA `rank`, TMEM lanes 32 q.. and columns c..: 8 x 32 vectors.
template <int CG, int TN>
__device__ __forceinline__ float4* piece_chunk(const GemmParams& p, int u, uint32_t rank, int q, int c) {
  return reinterpret_cast<float4*>(p.part) + (((static_cast<size_t>(u - p.whole) * CG + rank) * 4 + q) * (TN / 32) + c / 32) * 256;
}

// ---- many rows ------------------------------------------------------------------------------------
template <int CG, int TN, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    sol_linear_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_z,
                      const __grid_constant__ CUtensorMap map_res,
                      const __grid_constant__ GemmParams p) {
  using C = GemmCfg<CG, TN>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;  // the same offset in both CTAs of a pair
  uint8_t* smem = smem_raw + (sb - raw);
  const uint32_t bars = sb + C::OFF_BAR;
  const uint32_t bar_full = bars, bar_empty = bars + 8 * C::NS, bar_acc = bars + 16 * C::NS,
                 bar_free = bar_acc + 16, bar_drain = bar_free + 16, bar_res = bar_drain + 8,
                 bar_count = bar_res + 16 * kEpiWarps;
  volatile uint32_t* s_count = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_COUNT);  // from the other CTA of a pair
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::OFF_COUNT + 8);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_COUNT + 12);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CG == 1 ? 0u : cluster_rank();  // rank 0 issues the MMAs of a pair
  if (tid == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bar_full + 8 * s, 1);   // of a pair only rank 0's, for the bytes of both
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar_acc + 8 * a, 1);
      mbar_init(bar_free + 8 * a, CG * kEpiWarps);  // of a pair only rank 0's
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_count, 1);
    for (int i = 0; i < 2 * kEpiWarps; ++i) mbar_init(bar_res + 8 * i, 1);
    fence_mbar_init();
    *s_abort = 0;
  }
  if (warp == 1) pair_tmem_alloc<CG>(smem_u32(s_tmem), C::TMEM_COLS);
  tc_fence_before();
  if constexpr (CG == 2) __syncthreads();
  pair_sync<CG>();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  chained_wait();
  const int units = unit_count(p), first = blockIdx.x / CG, step = gridDim.x / CG;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&map_a);
      tma_prefetch_desc(&map_b);
      const uint32_t full0 = CG == 1 ? bar_full : in_cta(bar_full, 0);
      const uint32_t gone = left_out(p.drop);
      uint32_t g = 0;  // slices loaded so far
      int w = WAIT_OK;
      for (int t = first; t < units && w == WAIT_OK; t += step) {
        const Unit un = unit_of(p, t);
        const int row0 = (un.tm * CG + static_cast<int>(rank)) * BM, col0 = un.tn * TN + static_cast<int>(rank) * C::B_ROWS;
        for (int k = un.k_lo; k < un.k_hi; ++k, ++g) {
          const uint32_t s = g % C::NS;
          if (g >= C::NS) {
            w = mbar_wait(bar_empty + 8 * s, (g / C::NS - 1u) & 1u, s_abort, p.wait_limit_ns);
            if (w != WAIT_OK) break;
          }
          // rank 1's bytes may land first: its slice is free, so the barrier is already in this phase
          if (rank == 0) mbar_arrive_expect_tx(bar_full + 8 * s, CG * C::STAGE);
          const uint32_t dst = sb + s * C::STAGE;
          load_operand<CG, A_MN>(dst, &map_a, full0 + 8 * s, row0, BM, k * BK);
          if (g == gone) continue;
          load_operand<CG, B_MN>(dst + C::A_BYTES, &map_b, full0 + 8 * s, col0, C::B_ROWS, k * BK);
        }
      }
      if (w == WAIT_TIMEOUT) report(s_abort, p.ws, WHERE_PRODUCER);
      // No copy and no commit may be on its way here when shared memory is released. Copies are seen on rank 0's
      // full barriers only, commits in each CTA for itself, so of a pair rank 1 tells rank 0 how many slices it
      // has loaded, and rank 0's MMA thread tells rank 1 how many commits it has issued.
      bool told = false;
      if constexpr (CG == 2) {
        if (rank == 1) send_counts(sb + C::OFF_COUNT, bar_count, 0, g, 0);
        mbar_arrive_expect_tx(bar_count, 8);
        told = mbar_wait(bar_count, 0, nullptr, 2 * p.wait_limit_ns) == WAIT_OK;
      }
      if (rank == 0) {
        uint32_t last = g;
        // after an abort rank 1 may be ahead: slices that this CTA has not announced, with rank 1's bytes alone
        for (; told && last < s_count[0]; ++last) mbar_arrive_expect_tx(bar_full + 8 * (last % C::NS), C::STAGE);
        for (uint32_t i = last > C::NS ? last - C::NS : 0; i < last; ++i)
          mbar_wait(bar_full + 8 * (i % C::NS), (i / C::NS) & 1u, nullptr, p.wait_limit_ns);
      } else {
        settle<C::NS>(bar_empty, told ? s_count[0] : 0u, bar_acc, told ? s_count[1] : 0u, bar_drain, p.wait_limit_ns);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = instr_desc(CG * BM, TN, A_MN, B_MN);
      const uint64_t da0 = operand_desc<A_MN>(sb), db0 = operand_desc<B_MN>(sb + C::A_BYTES);
      uint32_t g = 0, it = 0, done = 0;  // slices and tiles committed
      int w = WAIT_OK;
      for (int t = first; t < units && w == WAIT_OK; t += step, ++it) {
        const Unit un = unit_of(p, t);
        const uint32_t acc = it & 1u;
        if (it >= 2) {
          w = mbar_wait(bar_free + 8 * acc, (it / 2 - 1u) & 1u, s_abort, p.wait_limit_ns);
          if (w != WAIT_OK) break;
          tc_fence_after();
        }
        for (int k = un.k_lo; k < un.k_hi; ++k, ++g) {
          const uint32_t s = g % C::NS;
          w = mbar_wait(bar_full + 8 * s, (g / C::NS) & 1u, s_abort, p.wait_limit_ns);
          if (w != WAIT_OK) break;
          tc_fence_after();
          const uint64_t da = da0 + ((s * C::STAGE) >> 4), db = db0 + ((s * C::STAGE) >> 4);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            pair_mma<CG>(tmem + acc * TN, da + kk * kDescStep<A_MN>, db + kk * kDescStep<B_MN>, idesc,
                         (k > un.k_lo || kk > 0) ? 1u : 0u);
          pair_commit<CG>(bar_empty + 8 * s);
        }
        if (w == WAIT_OK) {
          pair_commit<CG>(bar_acc + 8 * acc);
          ++done;
        }
      }
      if (w == WAIT_TIMEOUT) report(s_abort, p.ws, WHERE_MMA);
      pair_commit<CG>(bar_drain);  // no MMA may be in flight when tensor memory is freed
      if constexpr (CG == 2) send_counts(sb + C::OFF_COUNT, bar_count, 1, g, done);
      settle<C::NS>(bar_empty, g, bar_acc, done, bar_drain, p.wait_limit_ns);
    }
    __syncwarp();
  } else {
    const int ew = warp - 2, q = warp & 3, side = ew >> 2;  // TMEM lanes 32 q.., column half
    const int c_lo = side * (TN / 2);
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t buf0 = sb + C::OFF_EPI + ew * 2 * kEpiBuf;
    const uint32_t swz = (lane >> 1) & 3;  // 64-byte swizzle: 16-byte chunk c of row r sits at c ^ ((r / 2) % 4)
    const uint32_t free0 = CG == 1 ? bar_free : in_cta(bar_free, 0);
    const uint32_t bar_mine = bar_res + 16 * ew;
    uint32_t it = 0, chunks = 0, asked = 0;  // chunks stored; residual chunks asked for
    bool alive = true;  // no wait has expired
    int t = first, undone = c_lo;  // the unit at hand; after an abort the first column of it that has not left
    for (; t < units; t += step, ++it) {
      const Unit un = unit_of(p, t);
      const int tm = un.tm, tn = un.tn;
      const uint32_t acc = it & 1u;
      const int row0 = (tm * CG + static_cast<int>(rank)) * BM + q * 32;
      // The residual's values of a chunk come by TMA, one chunk ahead, into the buffer from which the chunk
      // will be stored: rows read by their own lanes (16 bytes of 32 rows at a time) held the whole
      // epilogue back.
      auto ask = [&](int col, int pending) {  // pending: stores after the last one out of this buffer
        const uint32_t i = asked & 1u;
        if (lane == 0) {
          if (pending == 0) bulk_wait_read<0>();
          else bulk_wait_read<1>();
          mbar_arrive_expect_tx(bar_mine + 8 * i, kEpiBuf);
          if (p.drop != DROP_RESIDUAL || asked != (TN > 64 ? 1u : 0u) || blockIdx.x != 0 || ew != 0)
            tma_load_2d(buf0 + i * kEpiBuf, &map_res, bar_mine + 8 * i, col, row0);
        }
        ++asked;
      };
      const bool with_res = p.has_residual && t < p.whole;  // past the last row too: zeros, so that every chunk counts alike
      if (with_res && tn * TN + c_lo < p.No) ask(tn * TN + c_lo, 1);
      float4 bias[8];  // of a chunk, read ahead as well
      auto read_bias = [&](int c) {
#pragma unroll
        for (int j = 0; j < 8; ++j)  // No is a multiple of 8
          if (c < c_lo + TN / 2 && tn * TN + c + 4 * j < p.No)
            bias[j] = __ldg(reinterpret_cast<const float4*>(p.bias + tn * TN + c + 4 * j));
      };
#pragma unroll
      for (int j = 0; j < 8; ++j) bias[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.bias != nullptr) read_bias(c_lo);
      const int w = mbar_wait(bar_acc + 8 * acc, (it / 2) & 1u, s_abort, p.wait_limit_ns);
      if (w == WAIT_TIMEOUT) report(s_abort, p.ws, WHERE_SOFTMAX);
      if (__any_sync(0xffffffffu, w != WAIT_OK)) {
        alive = false;
        break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int c = c_lo; c < c_lo + TN / 2; c += 32) {
        const int col0 = tn * TN + c;
        if (col0 >= p.No) break;  // uniform: the rest of the tile is past the last column
        uint32_t r[32];
        tmem_ld_x32(tmem + lane_base + acc * TN + c, r);
        if (t >= p.whole) {  // a piece: its sums as they are, 16 bytes per lane side by side, for the kernel that adds them
          float4* to = piece_chunk<CG, TN>(p, t, rank, q, c) + lane;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            to[32 * j] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]),
                                     __uint_as_float(r[4 * j + 3]));
          continue;
        }
        f2 v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = pack2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        const uint32_t buf = buf0 + (chunks & 1u) * kEpiBuf;
        bool fresh = true;  // nothing of this chunk has left through its buffer yet
        auto emit = [&](const CUtensorMap* map) {
          if (lane == 0) {
            if (!fresh) bulk_wait_read<0>();
            else if (!with_res) bulk_wait_read<1>();  // the store before the last one has left this buffer
          }
          fresh = false;
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t pk[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = unpack2(v[4 * i + j]);
              pk[j] = pack_bf16x2(f.x, f.y);
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 64 + ((i ^ swz) << 4)), "r"(pk[0]),
                         "r"(pk[1]), "r"(pk[2]), "r"(pk[3])
                         : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < p.Mo) tma_store_2d(map, buf, col0, row0);  // rows and columns past the end are not written
            bulk_commit();
          }
        };
        if (p.bias != nullptr) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[2 * j] = add2(v[2 * j], pack2(bias[j].x, bias[j].y));
            v[2 * j + 1] = add2(v[2 * j + 1], pack2(bias[j].z, bias[j].w));
          }
          read_bias(c + 32);
        }
        uint4 res[4];
        if (with_res) {
          if (c + 32 < c_lo + TN / 2 && col0 + 32 < p.No) ask(col0 + 32, 0);
          const uint32_t i = chunks & 1u;
          const int rw = mbar_wait(bar_mine + 8 * i, (chunks >> 1) & 1u, s_abort, p.wait_limit_ns);
          if (rw == WAIT_TIMEOUT) report(s_abort, p.ws, WHERE_SOFTMAX);
          if (__any_sync(0xffffffffu, rw != WAIT_OK)) {  // the buffer does not hold the residual
            alive = false;
            undone = c;
            break;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(res[j].x), "=r"(res[j].y), "=r"(res[j].z), "=r"(res[j].w)
                         : "r"(buf + lane * 64 + ((j ^ swz) << 4))
                         : "memory");
        }
        if (p.store_z) emit(&map_z);
        with_activation(p.act, [&](auto kind) {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = activate<decltype(kind)::value>(v[j]);
        });
        if (with_res) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t wv[4] = {res[i].x, res[i].y, res[i].z, res[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[4 * i + j] = add2(v[4 * i + j], pack2(__uint_as_float(wv[j] << 16), __uint_as_float(wv[j] & 0xffff0000u)));
          }
        }
        emit(&map_out);
        ++chunks;
      }
      if (!alive) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 1) mbar_arrive(bar_free + 8 * acc);
        else mbar_arrive_cluster(free0 + 8 * acc);
      }
    }
    if (!alive) {
      // a copy of the residual's must not outlive its buffer
      if (p.has_residual) {
        for (uint32_t n = chunks; n != asked; ++n) mbar_wait(bar_mine + 8 * (n & 1u), (n >> 1) & 1u, nullptr, p.wait_limit_ns);
      }
      // NaN to all that is left of this warp's outputs, or pieces
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
      for (int j = 0; j < 4; ++j)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(buf0 + lane * 64 + 16 * j), "r"(0x7fff7fffu) : "memory");
      fence_proxy_async_smem();
      __syncwarp();
      for (; t < units; t += step, undone = c_lo) {
        const Unit un = unit_of(p, t);
        const int row0 = (un.tm * CG + static_cast<int>(rank)) * BM + q * 32;
        for (int c = undone; c < c_lo + TN / 2 && un.tn * TN + c < p.No; c += 32) {
          if (t >= p.whole) {
            float4* to = piece_chunk<CG, TN>(p, t, rank, q, c) + lane;
            const float n = __uint_as_float(0x7fffffffu);
            for (int j = 0; j < 8; ++j) to[32 * j] = make_float4(n, n, n, n);
          } else if (lane == 0 && row0 < p.Mo) {
            tma_store_2d(&map_out, buf0, un.tn * TN + c, row0);
            if (p.store_z) tma_store_2d(&map_z, buf0, un.tn * TN + c, row0);
            bulk_commit();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  if constexpr (CG == 2) __syncthreads();
  pair_sync<CG>();
  tc_fence_after();
  if (warp == 1) pair_tmem_dealloc<CG>(tmem, C::TMEM_COLS);
}

// The pieces of the last tiles added, in order, with the epilogue of the others: one warp per 32 x 32
// outputs, a row of 32 to each lane.
struct PieceArgs {
  __nv_bfloat16* out;
  __nv_bfloat16* z;               // or null
  const __nv_bfloat16* residual;  // or null
};
template <int CG, int TN>
__global__ void __launch_bounds__(256) sol_linear_pieces_kernel(const __grid_constant__ GemmParams p, const PieceArgs a) {
  chained_wait();
  const int lane = threadIdx.x & 31, i = blockIdx.x * 8 + (threadIdx.x >> 5);
  constexpr int kChunks = CG * 4 * (TN / 32);
  const int tile = i / kChunks, in = i - tile * kChunks;
  if (tile >= p.tiles_m * p.tiles_n - p.whole) return;
  const Unit un = unit_of(p, p.whole + tile * p.split);
  const int row = un.tm * CG * BM + in / (TN / 32) * 32 + lane, col0 = un.tn * TN + in % (TN / 32) * 32;
  float4 s[8];
  const float4* from = reinterpret_cast<const float4*>(p.part) + (static_cast<size_t>(tile) * p.split * kChunks + in) * 256 + lane;
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = __ldcs(from + 32 * j);
  for (int piece = 1; piece < p.split; ++piece) {
    from += static_cast<size_t>(kChunks) * 256;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 a = __ldcs(from + 32 * j);
      s[j].x += a.x;
      s[j].y += a.y;
      s[j].z += a.z;
      s[j].w += a.w;
    }
  }
  if (row >= p.Mo) return;
  const size_t o = static_cast<size_t>(row) * p.No + col0;
  f2 v[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[2 * j] = pack2(s[j].x, s[j].y);
    v[2 * j + 1] = pack2(s[j].z, s[j].w);
    if (p.bias != nullptr && col0 + 4 * j < p.No) {  // No is a multiple of 8
      const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + col0 + 4 * j));
      v[2 * j] = add2(v[2 * j], pack2(b.x, b.y));
      v[2 * j + 1] = add2(v[2 * j + 1], pack2(b.z, b.w));
    }
  }
  auto put = [&](__nv_bfloat16* to) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2(v[4 * j + k]);
        w[k] = pack_bf16x2(f.x, f.y);
      }
      if (col0 + 8 * j < p.No) *reinterpret_cast<uint4*>(to + o + 8 * j) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  if (a.z != nullptr) put(a.z);
  with_activation(p.act, [&](auto kind) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = activate<decltype(kind)::value>(v[j]);
  });
  if (a.residual != nullptr) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (col0 + 8 * j >= p.No) break;
      const uint4 r = *reinterpret_cast<const uint4*>(a.residual + o + 8 * j);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[4 * j + k] = add2(v[4 * j + k], pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u)));
    }
  }
  put(a.out);
}

// ---- few rows --------------------------------------------------------------------------------------
constexpr int kFewThreads = 192;

template <int TT>
struct FewCfg {
  static constexpr int A_BYTES = BM * BK * 2;  // 128 rows of w
  static constexpr int B_BYTES = TT * BK * 2;  // TT tokens
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = 3;  // few, so that several CTAs share an SM and one loads while another finishes
  static constexpr int PART = TT * BM * 4;     // fp32 partial tile [token][row of w], over the ring once it is done
  static constexpr int RING = NS * STAGE > PART ? NS * STAGE : PART;
  static constexpr int OFF_BAR = RING;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;
  static constexpr int TMEM_COLS = TT < 32 ? 32 : TT;
};

struct FewParams {
  int M, N, nk;
  int split;  // CTAs of a cluster, each with its share of the reduction
  const float* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* out;
  __nv_bfloat16* z;
  int act;
  int drop;
  uint64_t wait_limit_ns;
  uint32_t* ws;
};

template <int TT>
__global__ void __launch_bounds__(kFewThreads)
    sol_linear_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                          const __grid_constant__ FewParams p) {
  using C = FewCfg<TT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sb - raw);
  const uint32_t bar_full = sb + C::OFF_BAR, bar_empty = bar_full + 8 * C::NS, bar_acc = bar_empty + 8 * C::NS;
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 16 * C::NS + 8);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 16 * C::NS + 12);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int n0 = blockIdx.x / p.split * BM;
  const int k_lo = static_cast<int>(static_cast<long long>(p.nk) * rank / p.split);
  const int k_hi = static_cast<int>(static_cast<long long>(p.nk) * (rank + 1) / p.split);  // split <= nk: at least one slice
  if (tid == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_acc, 1);
    fence_mbar_init();
    *s_abort = 0;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  chained_wait();

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t gone = left_out(p.drop);
      uint32_t g = 0;
      int w = WAIT_OK;
      for (int k = k_lo; k < k_hi; ++k, ++g) {
        const uint32_t s = g % C::NS;
        if (g >= C::NS) {
          w = mbar_wait(bar_empty + 8 * s, (g / C::NS - 1u) & 1u, s_abort, p.wait_limit_ns);
          if (w != WAIT_OK) break;
        }
        mbar_arrive_expect_tx(bar_full + 8 * s, C::STAGE);
        tma_load_2d(sb + s * C::STAGE, &map_w, bar_full + 8 * s, k * BK, n0);
        if (g == gone) continue;
        tma_load_2d(sb + s * C::STAGE + C::A_BYTES, &map_x, bar_full + 8 * s, k * BK, 0);
      }
      if (w == WAIT_TIMEOUT) report(s_abort, p.ws, WHERE_PRODUCER);
      for (uint32_t i = g > C::NS ? g - C::NS : 0; i < g; ++i)
        mbar_wait(bar_full + 8 * (i % C::NS), (i / C::NS) & 1u, nullptr, p.wait_limit_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = instr_desc(BM, TT, false, false);
      const uint64_t da0 = operand_desc<false>(sb), db0 = operand_desc<false>(sb + C::A_BYTES);
      uint32_t g = 0;
      int w = WAIT_OK;
      for (int k = k_lo; k < k_hi; ++k, ++g) {
        const uint32_t s = g % C::NS;
        w = mbar_wait(bar_full + 8 * s, (g / C::NS) & 1u, s_abort, p.wait_limit_ns);
        if (w != WAIT_OK) break;
        tc_fence_after();
        const uint64_t da = da0 + ((s * C::STAGE) >> 4), db = db0 + ((s * C::STAGE) >> 4);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_bf16_ss(tmem, da + kk * kDescStep<false>, db + kk * kDescStep<false>, idesc, (g > 0 || kk > 0) ? 1u : 0u);
        tc_commit(bar_empty + 8 * s);
      }
      if (w == WAIT_TIMEOUT) report(s_abort, p.ws, WHERE_MMA);
      tc_commit(bar_acc);  // also after an abort: the MMAs in flight end before tensor memory is freed
      settle<C::NS>(bar_empty, g, bar_acc, 0, bar_acc, p.wait_limit_ns);
    }
    __syncwarp();
  } else {
    const int w = mbar_wait(bar_acc, 0, nullptr, p.wait_limit_ns);
    if (w == WAIT_TIMEOUT) report(s_abort, p.ws, WHERE_SOFTMAX);
    if (!__any_sync(0xffffffffu, w != WAIT_OK)) {
      tc_fence_after();
      // every slice has been read by the MMAs, so the partial tile may take the ring's place
      const int q = warp & 3, n = q * 32 + lane;
      float* part = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int c = 0; c < TT; c += 16) {
        if (c >= p.M) break;
        uint32_t r[16];
        tmem_ld_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, r);
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * BM + n] = __uint_as_float(r[j]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
  if (*s_abort != 0) {  // the partial tile is incomplete: NaN, which the sums over the cluster keep
    const float n = __uint_as_float(0x7fffffffu);
    for (int e = tid; e < p.M * (BM / 4); e += kFewThreads) reinterpret_cast<float4*>(smem)[e] = make_float4(n, n, n, n);
    __syncthreads();
  }
  if (p.split > 1) cluster_arrive_wait();
  // each CTA of the cluster finishes an equal share of the M x 128 values, four at a time (128 / 4 is a
  // multiple of split)
  {
    const int share = p.M * (BM / 4) / p.split;
    for (int e = rank * share + tid; e < (rank + 1) * share; e += kFewThreads) {
      const int m = e / (BM / 4), n = n0 + 4 * (e & (BM / 4 - 1));
      if (n >= p.N) continue;  // N is a multiple of 8
      f2 v[2];
      if (p.split == 1) {
        const float4 f = reinterpret_cast<const float4*>(smem)[e];
        v[0] = pack2(f.x, f.y);
        v[1] = pack2(f.z, f.w);
      } else {
        v[0] = v[1] = dup2(0.f);
        for (int r = 0; r < p.split; ++r) {
          const float4 f = ld_cluster_f32x4(sb + 16 * e, r);
          v[0] = add2(v[0], pack2(f.x, f.y));
          v[1] = add2(v[1], pack2(f.z, f.w));
        }
      }
      if (p.bias != nullptr) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p.bias + n));
        v[0] = add2(v[0], pack2(f.x, f.y));
        v[1] = add2(v[1], pack2(f.z, f.w));
      }
      const size_t o = static_cast<size_t>(m) * p.N + n;
      auto put = [&](__nv_bfloat16* to) {
        const float2 lo = unpack2(v[0]), hi = unpack2(v[1]);
        *reinterpret_cast<uint2*>(to + o) = make_uint2(pack_bf16x2(lo.x, lo.y), pack_bf16x2(hi.x, hi.y));
      };
      if (p.z != nullptr) put(p.z);
      with_activation(p.act, [&](auto kind) {
        v[0] = activate<decltype(kind)::value>(v[0]);
        v[1] = activate<decltype(kind)::value>(v[1]);
      });
      if (p.residual != nullptr) {
        const uint2 r = *reinterpret_cast<const uint2*>(p.residual + o);
        v[0] = add2(v[0], pack2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u)));
        v[1] = add2(v[1], pack2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u)));
      }
      put(p.out);
    }
  }
  if (p.split > 1) cluster_arrive_wait();  // no CTA leaves while another reads its partial tile
}

// ---- gradient of the activation and of the bias --------------------------------------------------------
// dz = dy act'(z) in bf16 (the operand of the two products that follow; the rounding is theirs), and
// per block of rows the fp32 column sums of the unrounded dz, added by a second kernel in a fixed
// order. HBM-bound (8192 x 4096 with gelu: 41 us, 4.9 TB/s): 32 threads side by side cover 256 columns with 16-byte vectors, 8 rows at a time.
constexpr int kDzCols = 256, kDzRows = 8;

__device__ __forceinline__ void widen_bf16(const uint4& v, f2 (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
}

struct DzParams {
  const __nv_bfloat16* dy;
  const __nv_bfloat16* z;   // null: dz = dy
  __nv_bfloat16* dz;        // null where dz = dy
  float* part;              // [chunks, N] or null
  int M, N, rows;           // rows per block
};

template <int ACT>
__global__ void __launch_bounds__(kDzCols / 8 * kDzRows) sol_linear_dz_kernel(const __grid_constant__ DzParams p) {
  __shared__ float s[kDzRows][kDzCols + 8];
  chained_wait();
  const int lane = threadIdx.x, ty = threadIdx.y;
  const int c = blockIdx.x * kDzCols + lane * 8;
  const int r_lo = blockIdx.y * p.rows, r_hi = min(r_lo + p.rows, p.M);
  f2 a[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) a[k] = dup2(0.f);
  if (c < p.N) {
#pragma unroll 4
    for (int r = r_lo + ty; r < r_hi; r += kDzRows) {
      const size_t o = static_cast<size_t>(r) * p.N + c;
      const uint4 g = __ldg(reinterpret_cast<const uint4*>(p.dy + o));
      f2 v[4];
      widen_bf16(g, v);
      if constexpr (ACT != ACT_NONE) {
        f2 zz[4];
        widen_bf16(__ldg(reinterpret_cast<const uint4*>(p.z + o)), zz);
        uint32_t pk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = mul2(v[k], activation_slope<ACT>(zz[k]));
          const float2 f = unpack2(v[k]);
          pk[k] = pack_bf16x2(f.x, f.y);
        }
        *reinterpret_cast<uint4*>(p.dz + o) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] = add2(a[k], v[k]);
    }
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) *reinterpret_cast<float2*>(&s[ty][lane * 8 + 2 * k]) = unpack2(a[k]);
  __syncthreads();
  const int i = ty * 32 + lane, col = blockIdx.x * kDzCols + i;  // 256 threads: one column each
  if (col < p.N) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kDzRows; ++k) t += s[k][i];
    p.part[static_cast<size_t>(blockIdx.y) * p.N + col] = t;
  }
}

__global__ void __launch_bounds__(512) sol_linear_db_kernel(const float* __restrict__ part, float* __restrict__ db, int N,
                                                            int chunks) {
  __shared__ float s[16][33];
  chained_wait();
  const int col = blockIdx.x * 32 + threadIdx.x;
  float a = 0.f;
  if (col < N) {
#pragma unroll 4
    for (int i = threadIdx.y; i < chunks; i += 16) a += part[static_cast<size_t>(i) * N + col];
  }
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && col < N) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][threadIdx.x];
    db[col] = t;
  }
}

template <int CG, int TN, bool A_MN, bool B_MN>
cudaError_t launch_gemm_t(const GemmArgs& a, GemmParams p, cudaStream_t stream) {
  using C = GemmCfg<CG, TN>;
  p.tiles_m = (a.Mo + CG * BM - 1) / (CG * BM);
  p.tiles_n = (a.No + TN - 1) / TN;
  const cudaError_t e = allow_smem<sol_linear_kernel<CG, TN, A_MN, B_MN>>(C::SMEM);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
  const int units = a.num_sms / CG;
  const double rows = kGroupBytes / (2.0 * a.Ko);
  p.group = static_cast<int>(rows > kGroupRows ? rows < 1e6 ? rows : 1e6 : kGroupRows) / (CG * BM);
  if (p.group > p.tiles_m) p.group = p.tiles_m;
  const int rest = static_cast<int>(tiles % units);
  p.split = a.tile.split;
  p.whole = static_cast<int>(tiles) - (p.split > 1 ? rest : 0);
  const long long work = p.whole + static_cast<long long>(rest) * (p.split > 1 ? p.split : 0);
  const cudaError_t le = launch_chained(sol_linear_kernel<CG, TN, A_MN, B_MN>, dim3(CG * static_cast<int>(work < units ? work : units)),
                                        dim3(kGemmThreads), C::SMEM, stream, CG, a.maps[0], a.maps[1], a.maps[2], a.maps[3],
                                        a.maps[4], p);
  if (le != cudaSuccess || p.split == 1) return le;
  const PieceArgs pieces = {static_cast<__nv_bfloat16*>(a.out), static_cast<__nv_bfloat16*>(a.z),
                            static_cast<const __nv_bfloat16*>(a.residual)};
  return launch_chained(sol_linear_pieces_kernel<CG, TN>, dim3(rest * CG * 4 * (TN / 32) / 8), dim3(256), 0, stream, 1, p, pieces);
}

template <bool A_MN, bool B_MN>
cudaError_t launch_gemm_n(const GemmArgs& a, const GemmParams& p, cudaStream_t stream) {
  if (a.tile.ctas == 2)
    return a.tile.n == 256 ? launch_gemm_t<2, 256, A_MN, B_MN>(a, p, stream) : launch_gemm_t<2, 128, A_MN, B_MN>(a, p, stream);
  return a.tile.n == 128 ? launch_gemm_t<1, 128, A_MN, B_MN>(a, p, stream) : launch_gemm_t<1, 64, A_MN, B_MN>(a, p, stream);
}

template <int TT>
cudaError_t launch_few_t(const FewArgs& a, const FewParams& p, cudaStream_t stream) {
  using C = FewCfg<TT>;
  const cudaError_t e = allow_smem<sol_linear_few_kernel<TT>>(C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_chained(sol_linear_few_kernel<TT>, dim3((a.N + BM - 1) / BM * p.split), dim3(kFewThreads), C::SMEM, stream, p.split,
                        a.maps[0], a.maps[1], p);
}

}  // namespace

GemmTile linear_tile(int Mo, int No, int Ko, bool splittable, int num_sms) {
  // SM cycles until the last one is done, from measured products: a slice (64 deep) takes about as long on
  // the smaller tiles, which wait for their operands, as the 512 MMA cycles of the largest; the last
  // epilogue is not overlapped. (8191 x 768 -> 768 takes 15.5, 18.3, 17.1 and 27.6 us in this order,
  // 1000 x 768 -> 768 9.5, 8.6, 7.2 and 7.1 us.)
  const struct { int ctas, n; double slice, last; } options[] = {
      {2, 256, 600.0, 6500.0}, {2, 128, 510.0, 6000.0}, {1, 128, 545.0, 4000.0}, {1, 64, 487.0, 3200.0}};
  const int nk = (Ko + BK - 1) / BK;
  GemmTile best = {};
  double least = 0.0;
  for (const auto& o : options) {
    const int units = num_sms / o.ctas;
    const long long tiles = static_cast<long long>(std::ceil(Mo / (128.0 * o.ctas))) * ((No + o.n - 1) / o.n);
    const int rest = static_cast<int>(tiles % units);
    for (int split = 1; split == 1 || (splittable && rest > 0 && rest * split <= units && nk / split >= kPieceSlices); ++split) {
      const double turns = static_cast<double>(tiles / units) * nk + (rest > 0 ? std::ceil(nk / static_cast<double>(split)) : 0.0);
      double t = turns * o.slice + o.last;
      if (split > 1) t = 1.03 * (t + kPieceCycles);  // not for a few percent
      if (least == 0.0 || t < least) {
        least = t;
        best = {o.ctas, o.n, split};
      }
    }
  }
  return best;
}

size_t linear_part_bytes(int num_sms) { return static_cast<size_t>(num_sms) * 128 * 256 * 4; }

int linear_few_tile(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

int linear_dz_chunks(int M, int N) {
  const int cols = (N + kDzCols - 1) / kDzCols;
  const int most = (M + 4 * kDzRows - 1) / (4 * kDzRows);  // at least four rows per thread
  const int want = (kDzBlocks + cols - 1) / cols;
  const int rows = (M + (most < want ? most : want) - 1) / (most < want ? most : want);
  return (M + rows - 1) / rows;
}

cudaError_t launch_linear_gemm(const GemmArgs& a, cudaStream_t stream) {
  GemmParams p = {};
  p.Mo = a.Mo;
  p.No = a.No;
  p.nk = (a.Ko + BK - 1) / BK;
  p.bias = a.bias;
  p.has_residual = a.residual != nullptr;
  p.act = a.act;
  p.store_z = a.z != nullptr;
  p.part = a.part;
  p.drop = a.drop;
  p.wait_limit_ns = a.wait_limit_ns;
  p.ws = a.ws;
  if (a.a_mn) return launch_gemm_n<true, true>(a, p, stream);
  return a.b_mn ? launch_gemm_n<false, true>(a, p, stream) : launch_gemm_n<false, false>(a, p, stream);
}

cudaError_t launch_linear_few(const FewArgs& a, cudaStream_t stream) {
  FewParams p = {};
  p.M = a.M;
  p.N = a.N;
  p.nk = (a.K + BK - 1) / BK;
  p.bias = a.bias;
  p.residual = static_cast<const __nv_bfloat16*>(a.residual);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.z = static_cast<__nv_bfloat16*>(a.z);
  p.act = a.act;
  p.drop = a.drop;
  p.wait_limit_ns = a.wait_limit_ns;
  p.ws = a.ws;
  // the reduction over 1, 2, 4 or 8 CTAs: as many as are resident at once, each with two slices at least
  // (2 x 5120 -> 30720: 50.9 us over 1, 49.9 over 2, 51.9 over 4; 16 x 4096 -> 4096: 25.4, 16.5, 12.0 and 11.1 over 1, 2, 4, 8)
  const int resident = a.num_sms * (a.M <= 16 ? 4 : a.M <= 64 ? 3 : 2);
  const int tiles = (a.N + BM - 1) / BM;
  p.split = 1;
  while (p.split < 8 && tiles * 2 * p.split <= resident && p.nk / (2 * p.split) >= 2) p.split *= 2;
  switch (linear_few_tile(a.M)) {
    case 16: return launch_few_t<16>(a, p, stream);
    case 32: return launch_few_t<32>(a, p, stream);
    case 64: return launch_few_t<64>(a, p, stream);
    default: return launch_few_t<128>(a, p, stream);
  }
}

cudaError_t launch_linear_dz(const void* dy, const void* z, int act, int M, int N, void* dz, float* part, float* db,
                             cudaStream_t stream) {
  DzParams p;
  p.dy = static_cast<const __nv_bfloat16*>(dy);
  p.z = static_cast<const __nv_bfloat16*>(z);
  p.dz = static_cast<__nv_bfloat16*>(dz);
  p.part = part;
  p.M = M;
  p.N = N;
  const int chunks = linear_dz_chunks(M, N);
  p.rows = (M + chunks - 1) / chunks;
  const dim3 grid((N + kDzCols - 1) / kDzCols, chunks), block(kDzCols / 8, kDzRows);
  cudaError_t e;
  switch (act) {
    case ACT_GELU: e = launch_chained(sol_linear_dz_kernel<ACT_GELU>, grid, block, 0, stream, 1, p); break;
    case ACT_GELU_TANH: e = launch_chained(sol_linear_dz_kernel<ACT_GELU_TANH>, grid, block, 0, stream, 1, p); break;
    case ACT_SILU: e = launch_chained(sol_linear_dz_kernel<ACT_SILU>, grid, block, 0, stream, 1, p); break;
    default: e = launch_chained(sol_linear_dz_kernel<ACT_NONE>, grid, block, 0, stream, 1, p); break;
  }
  if (e != cudaSuccess || part == nullptr) return e;
  return launch_chained(sol_linear_db_kernel, dim3((N + 31) / 32), dim3(32, 16), 0, stream, 1, part, db, N, chunks);
}

}  // namespace sol
