// Gated residual and norm, the step between two halves of a transformer block, and its gradients:
//   u  = y, or norm_post(y) * post_gain          (a norm behind the branch)
//   x' = res_scale * x + gate[b] * u             (the residual stream)
//   h  = norm(x') * gain * (1 + scale[b]) + shift[b]
// with norm either layer, (v - mean) / sqrt(var + eps), or rms, v / sqrt(mean v^2 + eps), over the
// C channels of a row. Every vector (gate, gains, scale, shift) may be absent.
//
// HBM-bound: x and y are read once, x' and h written once; a row stays in registers between. A
// thread owns the same E channels of every row of its batch entry, in 16-byte vectors, with the
// vectors' products (gate post_gain and gain (1 + scale)) formed once, and keeps the next rows on
// their way with asynchronous copies into a ring in shared memory that belongs to the thread alone:
// no barrier and no wait on another thread, and enough bytes in flight while rows are reduced. Rows
// whose length or address does not allow 16-byte accesses are read value by value. Rows are reduced
// by warp shuffles and, where a row spans several warps, one shared-memory exchange per statistic.
// Variance is taken about the mean in a second reduction over the registers, not as a difference of
// moments, so a large common offset costs no digits. All arithmetic is fp32, two channels per
// instruction; only the stored rows are rounded.
#include <cmath>
#include <type_traits>

#include "chained.cuh"
#include "device_common.cuh"
#include "launchers.h"

namespace sol {

namespace {

constexpr int kMaxWarps = 32;  // of a row
constexpr int kSlot = 512;     // 16 bytes of each of a warp's threads
constexpr int kMaxRows = 16;   // of several warps in a block: 15 named barriers
constexpr int kSmemMax = 227 * 1024 - 10240;  // of a block's dynamic shared memory, beside the exchange buffers

// ---- element access ------------------------------------------------------------------------------------
// A 16-byte vector (V = 8 bf16 or 4 fp32) as V / 2 pairs, and back.
template <int V>
__device__ __forceinline__ void widen(const uint4& v, f2* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (V == 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) x[k] = pack2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
  }
}
template <int V>
__device__ __forceinline__ uint4 narrow(const f2* x) {
  uint32_t w[4];
  if constexpr (V == 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 t = unpack2(x[k]);
      w[k] = pack_bf16x2(t.x, t.y);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 t = unpack2(x[k]);
      w[2 * k] = __float_as_uint(t.x);
      w[2 * k + 1] = __float_as_uint(t.y);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// The E channels of a row that a thread owns, E / V vectors of V consecutive ones (V = 8 or 4: 16
// bytes; V = 1: single values), and its part of shared memory: 16-byte slots, a warp's side by side.
// A warp's channels lie together, so that a thread's vectors and slots are at fixed distances: rows
// are addressed by the byte offset of the thread's first channel, which the loops carry along, and
// everything else is an immediate (address arithmetic was a third of the instructions before).
// FULL: every vector of the warp lies within the row, and a row has whole warps.
template <typename T, int V, int E, bool FULL>
struct Lane {
  enum : int { NV = E / V, P = E / 2 };  // vectors, pairs
  static constexpr bool kFull = FULL;
  static constexpr int kMost = V == 1 ? kMaxWarps : 16;  // warps of a row: single values may be 8 to a thread
  int first, side, C;  // first channel; threads side by side (32, or a shorter row's)
  uint32_t smem;

  __device__ __forceinline__ Lane(int tpr, int t, int C, uint32_t smem)
      : first(t / 32 * 32 * E + t % 32 * V), side(tpr < 32 ? tpr : 32), C(C), smem(smem) {}
  __device__ __forceinline__ int chan(int j) const { return first + j * (FULL ? 32 : side) * V; }
  __device__ __forceinline__ bool on(int j) const { return FULL || chan(j) < C; }
  __device__ __forceinline__ uint32_t slot(int i) const { return smem + static_cast<uint32_t>(i) * kSlot; }
  __device__ __forceinline__ const T* at(const void* base, size_t o, int j) const {
    return reinterpret_cast<const T*>(static_cast<const char*>(base) + o + j * (FULL ? 32 : side) * V * static_cast<int>(sizeof(T)));
  }
  __device__ __forceinline__ T* at(void* base, size_t o, int j) const {
    return reinterpret_cast<T*>(static_cast<char*>(base) + o + j * (FULL ? 32 : side) * V * static_cast<int>(sizeof(T)));
  }

  // a row from global memory
  __device__ __forceinline__ void load(const void* base, size_t o, f2 (&x)[P]) const {
    if constexpr (V > 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on(j)) widen<V>(__ldg(reinterpret_cast<const uint4*>(at(base, o, j))), &x[j * V / 2]);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        x[i] = pack2(on(2 * i) ? static_cast<float>(*at(base, o, 2 * i)) : 0.f,
                     on(2 * i + 1) ? static_cast<float>(*at(base, o, 2 * i + 1)) : 0.f);
    }
  }
  __device__ __forceinline__ void store(void* base, size_t o, const f2 (&x)[P]) const {
    if constexpr (V > 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on(j)) *reinterpret_cast<uint4*>(at(base, o, j)) = narrow<V>(&x[j * V / 2]);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 v = unpack2(x[i]);
        if (on(2 * i)) put(at(base, o, 2 * i), v.x);
        if (on(2 * i + 1)) put(at(base, o, 2 * i + 1), v.y);
      }
    }
  }
  static __device__ __forceinline__ void put(T* p, float v) {
    if constexpr (sizeof(T) == 2) *p = __float2bfloat16_rn(v);
    else *p = v;
  }
  // a row on its way to the slots from i on, and out of slots at an address
  __device__ __forceinline__ void fetch(const void* base, size_t o, uint32_t to) const {
    if constexpr (V > 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on(j)) cp_async16(to + j * kSlot, at(base, o, j));
    }
  }
  __device__ __forceinline__ void take(uint32_t from, f2 (&x)[P]) const {
    if constexpr (V > 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on(j)) widen<V>(lds128(from + j * kSlot), &x[j * V / 2]);
    }
  }
  // an fp32 vector (16-byte aligned where V > 1); channels past C and an absent vector read as `absent`
  __device__ __forceinline__ void param(const float* p, float absent, f2 (&x)[P]) const {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = pack2(absent, absent);
    if (p == nullptr) return;
    if constexpr (V > 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!on(j)) continue;
#pragma unroll
        for (int k = 0; k < V; k += 4) widen<4>(__ldg(reinterpret_cast<const uint4*>(p + chan(j) + k)), &x[(j * V + k) / 2]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        x[i] = pack2(on(2 * i) ? __ldg(p + chan(2 * i)) : absent, on(2 * i + 1) ? __ldg(p + chan(2 * i + 1)) : absent);
    }
  }
  // zeros in the channels past C
  __device__ __forceinline__ void mask(f2 (&x)[P]) const {
    if constexpr (!FULL) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 v = unpack2(x[i]);
        x[i] = pack2(on(2 * i / V) ? v.x : 0.f, on((2 * i + 1) / V) ? v.y : 0.f);
      }
    }
  }
};

// One row spread over `tpr` consecutive threads, a power of two up to 32 or a multiple of 32, of a
// block that holds blockDim.x / tpr rows. The exchange buffer alternates between its two halves, so
// one barrier per reduction is enough: a half is written again only behind the barrier of the
// reduction in between. Each row of a block has a barrier of its own.
struct RowGroup {
  float* buf;  // the row's [2][2][kMaxWarps]: half, value, warp (zero past nwarps)
  int nwarps, width, lane, warp, phase, sub, tpr;
};

// s_buf: [kMaxRows][2][2][kMaxWarps], zeroed here; the caller meets at a barrier before the first sum.
__device__ __forceinline__ RowGroup row_group(float* s_buf, int tpr) {
  RowGroup g;
  g.lane = threadIdx.x & 31;
  g.nwarps = tpr > 32 ? tpr >> 5 : 1;
  g.width = tpr > 32 ? 32 : tpr;
  g.sub = threadIdx.x / tpr;
  g.warp = (threadIdx.x >> 5) - (tpr > 32 ? g.sub * g.nwarps : 0);  // within the row, where it has several
  g.buf = s_buf + (tpr > 32 ? g.sub : 0) * 4 * kMaxWarps;
  g.phase = 0;
  g.tpr = tpr;
  for (int i = threadIdx.x; i < kMaxRows * 4 * kMaxWarps; i += blockDim.x) s_buf[i] = 0.f;
  return g;
}

// Sums of N values over a row, the same for all its threads. Each thread adds the warps' sums itself:
// a few 16-byte broadcasts take a third of the latency of five more shuffles.
// WARPS: a row has whole warps; MOST: how many at most.
template <bool WARPS, int MOST, int N>
__device__ __forceinline__ void row_sum(RowGroup& g, float (&v)[N]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (WARPS || o < g.width) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  }
  if (g.nwarps == 1) return;
  float* b = g.buf + g.phase * (2 * kMaxWarps);
  g.phase ^= 1;
  if (g.lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i * kMaxWarps + g.warp] = v[i];
  }
  named_barrier_sync(1 + g.sub, g.tpr);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float4* q = reinterpret_cast<const float4*>(b + i * kMaxWarps);
    const float4 a = q[0], c = q[1];
    float s = ((a.x + a.y) + (a.z + a.w)) + ((c.x + c.y) + (c.z + c.w));
    if (g.nwarps > 8) {
      const float4 d = q[2], e = q[3];
      s += ((d.x + d.y) + (d.z + d.w)) + ((e.x + e.y) + (e.z + e.w));
    }
    if constexpr (MOST > 16) {
      for (int k = 4; 4 * k < g.nwarps; ++k) s += (q[k].x + q[k].y) + (q[k].z + q[k].w);
    }
    v[i] = s;
  }
}

// The row's values, centred for a layer norm; returns 1 / sqrt(mean square + eps), by which they are
// still to be multiplied. Channels past C hold zeros before and after.
template <typename L>
__device__ __forceinline__ float centre(const L& l, RowGroup& g, f2 (&x)[L::P], int kind, float inv_c, float eps) {
  if (kind == NORM_LAYER) {
    f2 s = x[0];
#pragma unroll
    for (int i = 1; i < L::P; ++i) s = add2(s, x[i]);
    float v[1] = {sum2(s)};
    row_sum<L::kFull, L::kMost>(g, v);
    const f2 m = pack2(-v[0] * inv_c, -v[0] * inv_c);
#pragma unroll
    for (int i = 0; i < L::P; ++i) x[i] = add2(x[i], m);
    l.mask(x);
  }
  f2 q = mul2(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < L::P; ++i) q = fma2(x[i], x[i], q);
  float v[1] = {sum2(q)};
  row_sum<L::kFull, L::kMost>(g, v);
  return 1.0f / sqrtf(fmaf(v[0], inv_c, eps));
}
template <int P>
__device__ __forceinline__ void scale_by(f2 (&x)[P], float r) {
  const f2 rr = pack2(r, r);
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = mul2(x[i], rr);
}

// Gradient of a row from the gradient w of its normalised values n, added to `to`:
// to + r (w - [mean w] - n mean(w n)). Channels past C hold zeros before and after.
template <typename L>
__device__ __forceinline__ void normalise_back(const L& l, RowGroup& g, f2 (&w)[L::P], const f2 (&n)[L::P], float r, int kind,
                                               float inv_c) {
  f2 s = mul2(w[0], n[0]);
#pragma unroll
  for (int i = 1; i < L::P; ++i) s = fma2(w[i], n[i], s);
  f2 m = pack2(0.f, 0.f);
  float a;
  if (kind == NORM_LAYER) {
    m = w[0];
#pragma unroll
    for (int i = 1; i < L::P; ++i) m = add2(m, w[i]);
    float v[2] = {sum2(s), sum2(m)};
    row_sum<L::kFull, L::kMost>(g, v);
    a = -v[0] * inv_c * r;
    m = pack2(-v[1] * inv_c, -v[1] * inv_c);
  } else {
    float v[1] = {sum2(s)};
    row_sum<L::kFull, L::kMost>(g, v);
    a = -v[0] * inv_c * r;
  }
  const f2 rr = pack2(r, r), aa = pack2(a, a);
  // w - mean before the multiplication by r: a large common part of w leaves without rounding with it
#pragma unroll
  for (int i = 0; i < L::P; ++i) w[i] = fma2(n[i], aa, mul2(kind == NORM_LAYER ? add2(w[i], m) : w[i], rr));
  l.mask(w);
}

// ---- forward ---------------------------------------------------------------------------------------
// A block's groups of tpr threads take rows of one batch entry, so they share the vectors' products in
// shared memory: A = gate post_gain, S = gain (1 + scale), H = shift. (In registers they left room
// for half as many threads and spilled: 874 us at 75600 x 5120 bf16; read per row from L1, 793 us; this
// form 479 to 517 us on different GPUs, 6.0 to 6.5 TB/s.)
// RING: the next row is on its way while one is reduced; else direct loads.
template <typename T, int V, int E, bool RING, bool FULL, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) sol_residual_norm_kernel(const __grid_constant__ NormArgs p, int tpr, int chunks) {
  using L = Lane<T, V, E, FULL>;
  constexpr int kParam = E / 4;  // slots of a product
  extern __shared__ uint4 s_mem[];  // per warp of a row products [3][kParam], per warp of the block ring [2][2][NV], in slots
  __shared__ float s_buf[kMaxRows * 4 * kMaxWarps];
  RowGroup g = row_group(s_buf, tpr);
  const int rpb = blockDim.x / tpr, t = threadIdx.x - g.sub * tpr;
  const uint32_t prod = smem_u32(s_mem) + (t / 32 * 3 * kParam * kSlot + t % 32 * 16);
  const uint32_t ring = smem_u32(s_mem) + ((tpr + 31) / 32 * 3 * kParam + threadIdx.x / 32 * 4 * L::NV) * kSlot + threadIdx.x % 32 * 16;
  const L l(tpr, t, p.C, ring);
  const int b = blockIdx.x / chunks, chunk = blockIdx.x - b * chunks;
  const float inv_c = 1.0f / static_cast<float>(p.C);
  const bool has_y = p.y != nullptr;
  constexpr uint32_t slot_bytes = 2 * L::NV * kSlot;
  const int stride = chunks * rpb;  // a block's last rows may be past the end
  const size_t step = static_cast<size_t>(stride) * p.C * sizeof(T);
  int row = chunk * rpb + g.sub;
  size_t o = (static_cast<size_t>(b) * p.T + row) * p.C * sizeof(T) + static_cast<size_t>(l.chan(0)) * sizeof(T);
  auto fetch = [&](int r, size_t from, uint32_t to) {
    if (r < p.T) {
      l.fetch(p.x, from, to);
      if (has_y) l.fetch(p.y, from, to + L::NV * kSlot);
    }
    cp_async_commit();
  };
  chained_wait();
  if constexpr (RING) fetch(row, o, ring);
  if (g.sub == 0) {
    f2 u[L::P], v[L::P];
    auto put = [&](int at) {
#pragma unroll
      for (int i = 0; i < kParam; ++i) sts128(prod + (at * kParam + i) * kSlot, narrow<4>(&v[2 * i]));
    };
    l.param(p.gate != nullptr ? p.gate + b * p.gate_stride : nullptr, 1.f, v);
    l.param(p.post_gain, 1.f, u);
#pragma unroll
    for (int i = 0; i < L::P; ++i) v[i] = mul2(v[i], u[i]);
    put(0);
    l.param(p.scale != nullptr ? p.scale + b * p.scale_stride : nullptr, 0.f, v);
    l.param(p.gain, 1.f, u);
#pragma unroll
    for (int i = 0; i < L::P; ++i) v[i] = fma2(v[i], u[i], u[i]);
    put(1);
    l.param(p.shift != nullptr ? p.shift + b * p.shift_stride : nullptr, 0.f, v);
    put(2);
  }
  __syncthreads();
  auto product = [&](int at, int i, f2 (&m)[2]) { widen<4>(lds128(prod + (at * kParam + i) * kSlot), m); };
  const f2 res = pack2(p.res_scale, p.res_scale);
  uint32_t now = ring, next = ring + slot_bytes;
  // a row of several warps stops by itself; rows that share a warp stop with the block's first
  for (int lead = FULL ? row : chunk * rpb; lead < p.T; lead += stride, row += stride, o += step) {
    const bool go = FULL || row < p.T;
    f2 x[L::P], y[L::P];
    if constexpr (!FULL) {
#pragma unroll
      for (int k = 0; k < L::P; ++k) x[k] = y[k] = pack2(0.f, 0.f);
    }
    if constexpr (RING) {
      fetch(row + stride, o + step, next);
      cp_async_wait<1>();
    }
    if (has_y) {
      if (go) {
        if constexpr (RING) l.take(now + L::NV * kSlot, y);
        else l.load(p.y, o, y);
      }
      if (p.post_norm != NORM_NONE) scale_by(y, centre(l, g, y, p.post_norm, inv_c, p.eps));
#pragma unroll
      for (int i = 0; i < kParam; ++i) {
        f2 m[2];
        product(0, i, m);
        y[2 * i] = mul2(y[2 * i], m[0]);
        y[2 * i + 1] = mul2(y[2 * i + 1], m[1]);
      }
    }
    if (go) {
      if constexpr (RING) l.take(now, x);
      else l.load(p.x, o, x);
    }
    if (has_y) {
#pragma unroll
      for (int k = 0; k < L::P; ++k) x[k] = fma2(res, x[k], y[k]);
      if (go) l.store(p.x_out, o, x);
    }
    const float r = centre(l, g, x, p.norm, inv_c, p.eps);
    const f2 rr = pack2(r, r);
#pragma unroll
    for (int i = 0; i < kParam; ++i) {
      f2 m[2], h[2];
      product(1, i, m);
      product(2, i, h);
      x[2 * i] = fma2(mul2(x[2 * i], rr), m[0], h[0]);
      x[2 * i + 1] = fma2(mul2(x[2 * i + 1], rr), m[1], h[1]);
    }
    if (go) l.store(p.h, o, x);
    const uint32_t free = now;
    now = next;
    next = free;
  }
  if constexpr (RING) cp_async_wait<0>();
}

// ---- backward --------------------------------------------------------------------------------------
// Per row (n, ny the normalised x' and y; ny = y without a norm behind the branch):
//   w = dh gain (1 + scale);  D = dx_out + norm'(w);  dx = res_scale D;  du = gate D
//   dy = norm_post'(du post_gain), or du
// and over the rows of a batch entry, per channel: P = sum dh n, S = sum dh, Q = sum D ny. From them
//   dscale = gain P, dshift = S, dgate = post_gain Q, dgain = sum_b (1 + scale) P, dpost_gain = sum_b gate Q.
// x' and its statistics are formed again from x and y, so the forward pass keeps nothing. P, S and
// Q stay in registers over a block's rows, are added over the rows that a block holds side by side,
// go to the workspace once per block, and a second kernel adds the blocks in a fixed order: no
// atomics, the same bits every time. With three sums, n, ny and w in registers the vectors' products
// have no room there; they lie in the thread's slots of shared memory. 2 x 33272 x 4096 bf16 with both norms:
// 659 to 694 us on different GPUs, 4.7 to 5.0 TB/s; with 128 registers, 16 warps per SM have to cover a row's four
// reductions, one behind the other. (mean(w n) = r mean(w x') does not have to wait for r: its sum could share the
// exchange of the squares, which is not done here.)
template <typename T, int V, int E, bool RING, bool FULL, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) sol_residual_norm_bwd_kernel(const __grid_constant__ NormBwdArgs p, int tpr) {
  using L = Lane<T, V, E, FULL>;
  extern __shared__ uint4 s_ring[];
  __shared__ float s_buf[kMaxRows * 4 * kMaxWarps];
  RowGroup g = row_group(s_buf, tpr);
  const NormArgs& f = p.fwd;
  const int rpb = blockDim.x / tpr;
  const int b = blockIdx.x / p.chunks, chunk = blockIdx.x - b * p.chunks;
  const float inv_c = 1.0f / static_cast<float>(p.C);
  const bool has_y = f.y != nullptr, has_d = p.dx_out != nullptr;
  // slots: gain (1 + scale), gate post_gain, then the ring: x, dh, and y and dx_out where they are
  constexpr int kParam = E / 4;
  const int t = static_cast<int>(threadIdx.x) - g.sub * tpr;
  const uint32_t mem = smem_u32(s_ring) + threadIdx.x / 32 * (2 * kParam + (RING ? 8 * L::NV : 0)) * kSlot + threadIdx.x % 32 * 16;
  const L l(tpr, t, p.C, mem);
  const uint32_t ring = l.slot(2 * kParam);
  constexpr uint32_t slot_bytes = 4 * L::NV * kSlot;
  const int stride = p.chunks * rpb;
  const size_t step = static_cast<size_t>(stride) * p.C * sizeof(T);
  int row = chunk * rpb + g.sub;
  size_t o = (static_cast<size_t>(b) * f.T + row) * p.C * sizeof(T) + static_cast<size_t>(l.chan(0)) * sizeof(T);
  auto fetch = [&](const auto& l, int r, size_t from, uint32_t to) {
    if (r < f.T) {
      l.fetch(f.x, from, to);
      l.fetch(p.dh, from, to + L::NV * kSlot);
      if (has_y) l.fetch(f.y, from, to + 2 * L::NV * kSlot);
      if (has_d) l.fetch(p.dx_out, from, to + 3 * L::NV * kSlot);  // only with y
    }
    cp_async_commit();
  };
  chained_wait();
  if constexpr (RING) fetch(l, row, o, ring);
  f2 aP[L::P], aS[L::P], aQ[L::P];
  {
    f2 u[L::P], v[L::P];
    l.param(f.scale != nullptr ? f.scale + static_cast<size_t>(b) * f.scale_stride : nullptr, 0.f, v);
    l.param(f.gain, 1.f, u);
#pragma unroll
    for (int i = 0; i < L::P; ++i) v[i] = fma2(v[i], u[i], u[i]);
#pragma unroll
    for (int i = 0; i < kParam; ++i) sts128(l.slot(i), narrow<4>(&v[2 * i]));
    l.param(f.gate != nullptr ? f.gate + static_cast<size_t>(b) * f.gate_stride : nullptr, 1.f, v);
    l.param(f.post_gain, 1.f, u);
#pragma unroll
    for (int i = 0; i < L::P; ++i) v[i] = mul2(v[i], u[i]);
#pragma unroll
    for (int i = 0; i < kParam; ++i) sts128(l.slot(kParam + i), narrow<4>(&v[2 * i]));
  }
#pragma unroll
  for (int i = 0; i < L::P; ++i) aP[i] = aS[i] = aQ[i] = pack2(0.f, 0.f);
  // v times the vector in the slots from `at` on
  auto times = [&](const f2 (&v)[L::P], int at, f2 (&out)[L::P]) {
#pragma unroll
    for (int i = 0; i < kParam; ++i) {
      f2 m[2];
      widen<4>(lds128(l.slot(at + i)), m);
      out[2 * i] = mul2(v[2 * i], m[0]);
      out[2 * i + 1] = mul2(v[2 * i + 1], m[1]);
    }
  };
  const f2 res = pack2(f.res_scale, f.res_scale);
  __syncthreads();  // the exchange buffer is zeroed
  uint32_t now = ring, next = ring + slot_bytes;
  auto rows = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    const Lane<T, V, E, kWhole> l(tpr, t, p.C, mem);
    for (int lead = kWhole || tpr >= 32 ? row : chunk * rpb; lead < f.T; lead += stride, row += stride, o += step) {
      const bool live = kWhole || row < f.T;
      f2 x[L::P], y[L::P], w[L::P];
      if constexpr (!kWhole) {
#pragma unroll
        for (int k = 0; k < L::P; ++k) x[k] = y[k] = w[k] = pack2(0.f, 0.f);
      }
      if constexpr (RING) {
        fetch(l, row + stride, o + step, next);
        cp_async_wait<1>();
      }
      auto read = [&](int tensor, const void* from, f2 (&v)[L::P]) {
        if constexpr (RING) l.take(now + tensor * L::NV * kSlot, v);
        else l.load(from, o, v);
      };
      if (live) read(0, f.x, x);
      float ry = 0.f;
      if (has_y) {
        if (live) read(2, f.y, y);
        if (f.post_norm != NORM_NONE) {
          ry = centre(l, g, y, f.post_norm, inv_c, f.eps);
          scale_by(y, ry);
        }
        times(y, kParam, w);
#pragma unroll
        for (int k = 0; k < L::P; ++k) x[k] = fma2(res, x[k], w[k]);
      }
      const float r = centre(l, g, x, f.norm, inv_c, f.eps);
      scale_by(x, r);
      if constexpr (!kWhole) {
#pragma unroll
        for (int k = 0; k < L::P; ++k) w[k] = pack2(0.f, 0.f);
      }
      if (live) read(1, p.dh, w);
#pragma unroll
      for (int k = 0; k < L::P; ++k) {
        aP[k] = fma2(w[k], x[k], aP[k]);
        aS[k] = add2(aS[k], w[k]);
      }
      times(w, 0, w);
      normalise_back(l, g, w, x, r, f.norm, inv_c);
      if (has_d && live) {
        f2 d[L::P];
        if constexpr (!kWhole) {
#pragma unroll
          for (int k = 0; k < L::P; ++k) d[k] = pack2(0.f, 0.f);
        }
        read(3, p.dx_out, d);
#pragma unroll
        for (int k = 0; k < L::P; ++k) w[k] = add2(w[k], d[k]);
      }
      if (has_y) {
#pragma unroll
        for (int k = 0; k < L::P; ++k) x[k] = mul2(w[k], res);
        if (live) l.store(p.dx, o, x);
#pragma unroll
        for (int k = 0; k < L::P; ++k) aQ[k] = fma2(w[k], y[k], aQ[k]);
        times(w, kParam, w);
        if (f.post_norm != NORM_NONE) normalise_back(l, g, w, y, ry, f.post_norm, inv_c);
        if (live) l.store(p.dy, o, w);
      } else if (live) {
        l.store(p.dx, o, w);
      }
      const uint32_t free = now;
      now = next;
      next = free;
    }
  };
  if (FULL || (tpr >= 32 && (t / 32 + 1) * 32 * E <= p.C)) rows(std::true_type{});
  else if constexpr (!FULL) rows(std::false_type{});
  if constexpr (RING) cp_async_wait<0>();
  if (p.part == nullptr) return;
  // a row past the end added zeros only; rows side by side: first those of a warp, then warp by warp
  for (int q = tpr; q < 32; q <<= 1) {
#pragma unroll
    for (int i = 0; i < L::P; ++i) {
      aP[i] = add2(aP[i], __shfl_xor_sync(0xffffffffu, aP[i], q));
      aS[i] = add2(aS[i], __shfl_xor_sync(0xffffffffu, aS[i], q));
      aQ[i] = add2(aQ[i], __shfl_xor_sync(0xffffffffu, aQ[i], q));
    }
  }
  const int held = tpr < 32 ? blockDim.x / 32 : rpb, mine = tpr < 32 ? g.warp : g.sub;  // sums to add
  const bool writer = tpr >= 32 || g.lane < tpr;
  float* s_sum = reinterpret_cast<float*>(s_ring);  // [3][C], over the slots
  float* part = p.part + static_cast<size_t>(blockIdx.x) * 3 * p.C;
  for (int s = 0; s < held; ++s) {
    if (held > 1) __syncthreads();
    if (s != mine || !writer) continue;
#pragma unroll
    for (int i = 0; i < L::P; ++i) {
      const f2 sums[3] = {aP[i], aS[i], aQ[i]};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = 2 * i + k;
        if (!l.on(e / V)) continue;
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const float2 pair = unpack2(sums[q]);
          float v = k == 0 ? pair.x : pair.y;
          const int to = q * p.C + l.chan(e / V) + e % V;
          if (s > 0) v += s_sum[to];
          if (s == held - 1) part[to] = v;
          else s_sum[to] = v;
        }
      }
    }
  }
}

constexpr int kSumCols = 32, kSumRows = 32;

// Sums over `n` rows of one column, by the kSumRows threads of a block column; all of them return it.
template <typename F>
__device__ __forceinline__ float column_sum(F&& get, int n) {
  __shared__ float s[kSumRows][kSumCols + 1];
  float a = 0.f;
#pragma unroll 8
  for (int i = threadIdx.y; i < n; i += kSumRows) a += get(i);
  __syncthreads();
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kSumRows; ++i) t += s[i][threadIdx.x];
  return t;
}

// The gradients of one batch entry's vectors from the partial sums, blockIdx.z of P, S and Q; where shared
// gains have several batch entries to add, the entry's P and Q replace its first slot for the next kernel.
// Latency is what counts, so the three sums and the slots go to as many threads as there are.
__global__ void __launch_bounds__(kSumCols* kSumRows) sol_residual_norm_sum_kernel(const __grid_constant__ NormBwdArgs p,
                                                                                  int slots) {
  chained_wait();
  const int b = blockIdx.y, which = blockIdx.z, cc = blockIdx.x * kSumCols + threadIdx.x;
  const bool on = cc < p.C;
  const int c = on ? cc : 0;
  const NormArgs& f = p.fwd;
  float* part = p.part + static_cast<size_t>(b) * slots * 3 * p.C + static_cast<size_t>(which) * p.C;
  const size_t step = 3 * static_cast<size_t>(p.C), at = static_cast<size_t>(b) * p.C + c;
  const bool first = threadIdx.y == 0 && on;
  float* own = which == 0 ? p.dscale : which == 1 ? p.dshift : p.dgate;
  float* shared = which == 0 ? p.dgain : which == 2 ? p.dpost_gain : nullptr;
  if (own == nullptr && shared == nullptr) return;
  const float v = column_sum([&](int i) { return part[i * step + c]; }, slots);
  if (!first) return;
  if (own != nullptr) {
    const float* gain = which == 0 ? f.gain : which == 2 ? f.post_gain : nullptr;
    own[at] = gain != nullptr ? gain[c] * v : v;
  }
  if (shared != nullptr) {
    float one = v;
    if (which == 0 && f.scale != nullptr) one = v * (1.0f + f.scale[static_cast<size_t>(b) * f.scale_stride + c]);
    if (which == 2 && f.gate != nullptr) one = v * f.gate[static_cast<size_t>(b) * f.gate_stride + c];
    if (f.B == 1) shared[c] = one;
    else part[c] = one;
  }
}

// The shared gains' gradients: the batch entries' shares added.
__global__ void __launch_bounds__(kSumCols* kSumRows) sol_residual_norm_sum_b_kernel(const __grid_constant__ NormBwdArgs p,
                                                                                    int slots) {
  chained_wait();
  const int cc = blockIdx.x * kSumCols + threadIdx.x;
  const bool on = cc < p.C;
  const int c = on ? cc : 0;
  const size_t step = static_cast<size_t>(slots) * 3 * p.C;
  const bool first = threadIdx.y == 0 && on;
  if (p.dgain != nullptr) {
    const float s = column_sum([&](int i) { return p.part[i * step + c]; }, p.fwd.B);
    if (first) p.dgain[c] = s;
  }
  if (p.dpost_gain != nullptr) {
    const float s = column_sum([&](int i) { return p.part[i * step + 2 * static_cast<size_t>(p.C) + c]; }, p.fwd.B);
    if (first) p.dpost_gain[c] = s;
  }
}

// How a row is laid over threads, `elems` channels each.
struct Shape {
  int elems, tpr, rpb, threads;
};
Shape shape_of(int C, int elems) {
  Shape s;
  s.elems = elems;
  const int n = (C + elems - 1) / elems;
  if (n >= 32) {
    s.tpr = (n + 31) / 32 * 32;
  } else {
    s.tpr = 1;
    while (s.tpr < n) s.tpr *= 2;
  }
  s.rpb = s.tpr >= 256 ? 1 : 256 / s.tpr;
  s.threads = s.tpr * s.rpb;
  return s;
}
// 16 channels halve the shuffles per value (gradient of 20000 x 5120 bf16: 318 us in ten warps per SM, 321
// in twenty with 8); 8 pad short rows less, and leave the gradient's single values room for an
// address and a test each (20000 x 5119: 854 us, 1465 with 16 that spill).
int fwd_elems(int C) {
  const Shape a = shape_of(C, 16), b = shape_of(C, 8);
  return C > 2048 || 16 * a.tpr <= 8 * b.tpr ? 16 : 8;
}
int bwd_elems(int C, bool vec) { return !vec && C <= 6144 ? 8 : fwd_elems(C); }
size_t row_bytes(const Shape& s, int bytes) { return static_cast<size_t>(s.threads) * s.elems * bytes; }

template <typename T, int V, int E, bool RING, bool FULL, int MAXT>
cudaError_t launch_fwd_k(const NormArgs& a, Shape s, int num_sms, cudaStream_t stream) {
  // rows side by side in a block: as many as share an SM, unless the batch entries have fewer
  const long long share = (static_cast<long long>(a.B) * a.T + num_sms - 1) / num_sms;
  const size_t row = RING ? static_cast<size_t>(s.tpr) * E * sizeof(T) * 4 : 0;  // two rows of x and y
  const size_t products = static_cast<size_t>(s.tpr < 32 ? 32 : s.tpr) * E * 12;
  const int unit = s.tpr < 32 ? 32 / s.tpr : 1;  // whole warps
  long long rows = MAXT / s.tpr;
  if (s.tpr > 32 && rows > 15) rows = 15;  // each with a named barrier
  if (rows > a.T) rows = a.T;
  if (rows > share) rows = share;
  rows = (rows + unit - 1) / unit * unit;
  if constexpr (RING) {
    const long long fit = static_cast<long long>((kSmemMax - products) / row) / unit * unit;
    if (rows > fit) rows = fit;
  }
  s.rpb = static_cast<int>(rows);
  s.threads = s.tpr * s.rpb;
  const size_t smem = products + row * s.rpb;
  const long long per_sm = static_cast<long long>(MAXT / s.threads) < 1 ? 1 : MAXT / s.threads;
  long long chunks = per_sm * num_sms / a.B, most = (a.T + s.rpb - 1) / s.rpb;
  if (chunks > most) chunks = most;
  if (chunks < 1) chunks = 1;
  const cudaError_t e = allow_smem<sol_residual_norm_kernel<T, V, E, RING, FULL, MAXT>>(kSmemMax);
  if (e != cudaSuccess) return e;
  return launch_chained(sol_residual_norm_kernel<T, V, E, RING, FULL, MAXT>, dim3(static_cast<unsigned>(a.B * chunks)),
                        dim3(s.threads), smem, stream, 1, a, s.tpr, static_cast<int>(chunks));
}
template <typename T, int V, bool FULL>
cudaError_t launch_fwd(const NormArgs& a, const Shape& s, int num_sms, cudaStream_t stream) {
  if constexpr (V == 1) {
    return s.elems == 8 ? launch_fwd_k<T, V, 8, false, FULL, 1024>(a, s, num_sms, stream)
                        : launch_fwd_k<T, V, 16, false, FULL, 1024>(a, s, num_sms, stream);
  } else {
    // two rows in the ring; fp32 rows of more than 7680 channels leave it no room and are read directly
    if constexpr (sizeof(T) == 4) {
      if (static_cast<size_t>(s.tpr) * s.elems * 28 > kSmemMax) return launch_fwd_k<T, V, 16, false, FULL, 1024>(a, s, num_sms, stream);
    }
    return s.elems == 8 ? launch_fwd_k<T, V, 8, true, FULL, 1024>(a, s, num_sms, stream)
                        : launch_fwd_k<T, V, 16, true, FULL, 1024>(a, s, num_sms, stream);
  }
}

template <typename T, int V, int E, bool RING, bool FULL, int MAXT, int MINB>
cudaError_t launch_bwd_k(const NormBwdArgs& a, const Shape& s, cudaStream_t stream) {
  size_t smem = row_bytes(s, 8 + (RING ? 8 : 0) * static_cast<int>(sizeof(T)));
  if (s.rpb > 1 && smem < 12u * a.C) smem = 12u * a.C;  // the sums of a block's rows take the slots' place
  const cudaError_t e = allow_smem<sol_residual_norm_bwd_kernel<T, V, E, RING, FULL, MAXT, MINB>>(kSmemMax);
  if (e != cudaSuccess) return e;
  return launch_chained(sol_residual_norm_bwd_kernel<T, V, E, RING, FULL, MAXT, MINB>, dim3(a.fwd.B * a.chunks), dim3(s.threads),
                        smem, stream, 1, a, s.tpr);
}
template <typename T, int V, int E, bool RING, bool FULL>
cudaError_t launch_bwd_t(const NormBwdArgs& a, const Shape& s, cudaStream_t stream) {
  // 8 channels a thread in more than 256 threads, and 16 without the ring in fewer, do not come up (bwd_elems)
  if constexpr (E == 16) {
    if constexpr (RING) {
      if (s.threads <= 256) return launch_bwd_k<T, V, E, RING, FULL, 256, 2>(a, s, stream);
    }
    return launch_bwd_k<T, V, E, RING, FULL, 512, 1>(a, s, stream);
  } else {
    if constexpr (V == 1) {
      if (s.threads > 256) return launch_bwd_k<T, V, E, RING, FULL, 768, 1>(a, s, stream);
    }
    return launch_bwd_k<T, V, E, RING, FULL, 256, 3>(a, s, stream);
  }
}
template <typename T, int V, bool FULL>
cudaError_t launch_bwd(const NormBwdArgs& a, const Shape& s, cudaStream_t stream) {
  if constexpr (V == 1) {
    return s.elems == 8 ? launch_bwd_t<T, V, 8, false, FULL>(a, s, stream) : launch_bwd_t<T, V, 16, false, FULL>(a, s, stream);
  } else {
    // two rows in the ring; fp32 rows of more than 5120 channels leave it no room and are read directly
    if constexpr (sizeof(T) == 4) {
      if (row_bytes(s, 40) > kSmemMax) return launch_bwd_t<T, V, 16, false, FULL>(a, s, stream);
    }
    return s.elems == 8 ? launch_bwd_t<T, V, 8, true, FULL>(a, s, stream) : launch_bwd_t<T, V, 16, true, FULL>(a, s, stream);
  }
}

}  // namespace

int norm_bwd_chunks(int B, int T, int C, bool vec) {
  // one to three blocks per SM, by their threads and registers; of fp32 rows the ring leaves room for fewer, and the
  // blocks take turns
  const Shape s = shape_of(C, bwd_elems(C, vec));
  const int most = (T + s.rpb - 1) / s.rpb;
  const int blocks = s.threads > 256 ? kNormBwdBlocks / 4 : s.elems == 16 ? kNormBwdBlocks / 2 : kNormBwdBlocks * 3 / 4;
  const int want = blocks / B > 1 ? blocks / B : 1;
  return most < want ? most : want;
}
size_t norm_bwd_part_floats(int B, int T, int C) {  // for either kind of access, which the sizes alone do not tell
  const int a = norm_bwd_chunks(B, T, C, true), b = norm_bwd_chunks(B, T, C, false);
  return static_cast<size_t>(B) * (a > b ? a : b) * 3 * C;
}

cudaError_t launch_residual_norm(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const Shape s = shape_of(a.C, fwd_elems(a.C));
  const bool full = a.C == s.tpr * s.elems && s.tpr >= 32;
  if (a.bf16) {
    if (!a.vec) return launch_fwd<__nv_bfloat16, 1, false>(a, s, num_sms, stream);
    return full ? launch_fwd<__nv_bfloat16, 8, true>(a, s, num_sms, stream) : launch_fwd<__nv_bfloat16, 8, false>(a, s, num_sms, stream);
  }
  if (!a.vec) return launch_fwd<float, 1, false>(a, s, num_sms, stream);
  return full ? launch_fwd<float, 4, true>(a, s, num_sms, stream) : launch_fwd<float, 4, false>(a, s, num_sms, stream);
}

cudaError_t launch_residual_norm_bwd(const NormBwdArgs& a, cudaStream_t stream) {
  const NormArgs& f = a.fwd;
  const Shape s = shape_of(a.C, bwd_elems(a.C, f.vec));
  const bool full = a.C == s.tpr * s.elems && s.tpr >= 32;
  cudaError_t e;
  if (f.bf16) {
    e = !f.vec ? launch_bwd<__nv_bfloat16, 1, false>(a, s, stream)
        : full ? launch_bwd<__nv_bfloat16, 8, true>(a, s, stream) : launch_bwd<__nv_bfloat16, 8, false>(a, s, stream);
  } else {
    e = !f.vec ? launch_bwd<float, 1, false>(a, s, stream)
        : full ? launch_bwd<float, 4, true>(a, s, stream) : launch_bwd<float, 4, false>(a, s, stream);
  }
  if (e != cudaSuccess || a.part == nullptr) return e;
  const int slots = a.chunks;
  const dim3 block(kSumCols, kSumRows);
  const unsigned cols = (a.C + kSumCols - 1) / kSumCols;
  if ((e = launch_chained(sol_residual_norm_sum_kernel, dim3(cols, f.B, 3), block, 0, stream, 1, a, slots)) != cudaSuccess) return e;
  if (f.B > 1 && (a.dgain != nullptr || a.dpost_gain != nullptr)) {
    e = launch_chained(sol_residual_norm_sum_b_kernel, dim3(cols), block, 0, stream, 1, a, slots);
  }
  return e;
}

}  // namespace sol
