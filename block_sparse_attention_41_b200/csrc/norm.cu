// Gated residual and norm, the step between two halves of a transformer block, and its gradients:
//   u  = y, or norm_post(y) * post_gain          (a norm behind the branch)
//   x' = res_scale * x + gate[b] * u             (the residual stream)
//   h  = norm(x') * gain * (1 + scale[b]) + shift[b]
// with norm either layer, (v - mean) / sqrt(var + eps), or rms, v / sqrt(mean v^2 + eps), over the
// C channels of a row. Every vector (gate, gains, scale, shift) may be absent.
//
// HBM-bound: x and y are read once, x' and h written once; a row stays in registers between. A
// thread owns the same 16 (backward: 8) channels of every row, in 16-byte vectors (or single values where C
// or an address does not allow those); rows are reduced by warp shuffles and, where a row spans
// several warps, one shared-memory exchange per statistic. Variance is taken about the mean in a
// second reduction over the registers, not as a difference of moments, so a large common offset
// costs no digits. All arithmetic is fp32; only the stored rows are rounded.
#include <cmath>

#include "device_common.cuh"
#include "launchers.h"

namespace sol {

namespace {

constexpr int kFwdElems = 16;  // channels per thread
constexpr int kBwdElems = 8;   // fewer than forward: the sums of three gradients stay in registers too
constexpr int kMaxWarps = 32;

// ---- element access: V consecutive values as fp32 ------------------------------------------------
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[V]) {
  if constexpr (V == 8) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  } else if constexpr (V == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else if constexpr (sizeof(T) == 2) {
    x[0] = __bfloat162float(*p);
  } else {
    x[0] = __ldg(p);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[V]) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else if constexpr (V == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else if constexpr (sizeof(T) == 2) {
    *p = __float2bfloat16_rn(x[0]);
  } else {
    *p = x[0];
  }
}
// V values of an fp32 vector (16-byte aligned where V > 1)
template <int V>
__device__ __forceinline__ void load_param(const float* p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = __ldg(p);
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + k));
      x[k] = v.x; x[k + 1] = v.y; x[k + 2] = v.z; x[k + 3] = v.w;
    }
  }
}

// One row spread over `tpr` consecutive threads (a multiple of 32) of a block that holds blockDim.x
// / tpr rows. The exchange buffer alternates between its two halves, so one barrier per reduction
// is enough: a half is written again only behind the barrier of the reduction in between.
struct RowGroup {
  float* buf;  // [2][kMaxWarps][2]
  int first_warp, nwarps, warp, lane, phase;
};

// Sums of N values over a row. Every thread of the block calls it the same number of times.
template <int N>
__device__ __forceinline__ void row_sum(RowGroup& g, float (&v)[N]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if (g.nwarps == 1) return;
  float* b = g.buf + g.phase * (kMaxWarps * 2);
  g.phase ^= 1;
  if (g.lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[g.warp * 2 + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = g.lane < g.nwarps ? b[(g.first_warp + g.lane) * 2 + i] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    v[i] = s;
  }
}

// The row's values, normalised in place; returns 1 / sqrt(mean square or variance + eps). Channels
// past C (on[j] false) hold zeros before and after.
template <int V, int NV>
__device__ __forceinline__ float normalise(RowGroup& g, float (&x)[NV][V], const bool (&on)[NV], int kind, float inv_c,
                                           float eps) {
  if (kind == NORM_LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < V; ++k) s[0] += x[j][k];
    row_sum(g, s);
    const float mean = s[0] * inv_c;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < V; ++k) x[j][k] = on[j] ? x[j][k] - mean : 0.f;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) q[0] = fmaf(x[j][k], x[j][k], q[0]);
  row_sum(g, q);
  const float r = 1.0f / sqrtf(fmaf(q[0], inv_c, eps));
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) x[j][k] *= r;
  return r;
}

// Gradient of a row from the gradient w of its normalised values n: r (w - [mean w] - n mean(w n)),
// in place in w.
template <int V, int NV>
__device__ __forceinline__ void normalise_back(RowGroup& g, float (&w)[NV][V], const float (&n)[NV][V], float r,
                                               int kind, float inv_c) {
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      s[0] = fmaf(w[j][k], n[j][k], s[0]);
      s[1] += w[j][k];
    }
  row_sum(g, s);
  const float a = s[0] * inv_c, m = kind == NORM_LAYER ? s[1] * inv_c : 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) w[j][k] = r * (w[j][k] - m - n[j][k] * a);
}

__device__ __forceinline__ RowGroup row_group(float* buf, int tpr) {
  RowGroup g;
  g.buf = buf;
  g.warp = threadIdx.x >> 5;
  g.lane = threadIdx.x & 31;
  g.nwarps = tpr >> 5;
  g.first_warp = g.warp / g.nwarps * g.nwarps;
  g.phase = 0;
  return g;
}

// ---- forward ---------------------------------------------------------------------------------------
template <typename T, int V, int E, int MAXT>
__global__ void __launch_bounds__(MAXT) sol_residual_norm_kernel(const __grid_constant__ NormArgs p, int tpr) {
  constexpr int NV = E / V;
  __shared__ float s_buf[2 * kMaxWarps * 2];
  RowGroup g = row_group(s_buf, tpr);
  const int rpb = blockDim.x / tpr, sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
  const long long rows = static_cast<long long>(p.B) * p.T;
  const float inv_c = 1.0f / static_cast<float>(p.C);
  bool on[NV];
  int c[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    c[j] = (j * tpr + t) * V;
    on[j] = c[j] < p.C;
  }
  for (long long r0 = static_cast<long long>(blockIdx.x) * rpb; r0 < rows; r0 += static_cast<long long>(gridDim.x) * rpb) {
    const long long row = r0 + sub;
    const bool live = row < rows;  // a block's last rows may be past the end; their threads still meet at the barriers
    const size_t base = live ? static_cast<size_t>(row) * p.C : 0;
    const int b = live ? static_cast<int>(row / p.T) : 0;
    float x[NV][V], y[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int k = 0; k < V; ++k) x[j][k] = y[j][k] = 0.f;
      if (live && on[j]) {
        load_vec<T, V>(static_cast<const T*>(p.x) + base + c[j], x[j]);
        if (p.y != nullptr) load_vec<T, V>(static_cast<const T*>(p.y) + base + c[j], y[j]);
      }
    }
    if (p.y != nullptr) {
      if (p.post_norm != NORM_NONE) normalise<V, NV>(g, y, on, p.post_norm, inv_c, p.eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!on[j]) continue;
        float w[V];
        if (p.post_gain != nullptr) {
          load_param<V>(p.post_gain + c[j], w);
#pragma unroll
          for (int k = 0; k < V; ++k) y[j][k] *= w[k];
        }
        if (p.gate != nullptr) {
          load_param<V>(p.gate + static_cast<size_t>(b) * p.gate_stride + c[j], w);
#pragma unroll
          for (int k = 0; k < V; ++k) y[j][k] *= w[k];
        }
#pragma unroll
        for (int k = 0; k < V; ++k) x[j][k] = fmaf(p.res_scale, x[j][k], y[j][k]);
        if (live) store_vec<T, V>(static_cast<T*>(p.x_out) + base + c[j], x[j]);
      }
    }
    normalise<V, NV>(g, x, on, p.norm, inv_c, p.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!on[j] || !live) continue;
      float w[V];
      if (p.gain != nullptr) {
        load_param<V>(p.gain + c[j], w);
#pragma unroll
        for (int k = 0; k < V; ++k) x[j][k] *= w[k];
      }
      if (p.scale != nullptr) {
        load_param<V>(p.scale + static_cast<size_t>(b) * p.scale_stride + c[j], w);
#pragma unroll
        for (int k = 0; k < V; ++k) x[j][k] = fmaf(x[j][k], w[k], x[j][k]);
      }
      if (p.shift != nullptr) {
        load_param<V>(p.shift + static_cast<size_t>(b) * p.shift_stride + c[j], w);
#pragma unroll
        for (int k = 0; k < V; ++k) x[j][k] += w[k];
      }
      store_vec<T, V>(static_cast<T*>(p.h) + base + c[j], x[j]);
    }
  }
}

// ---- backward --------------------------------------------------------------------------------------
// Per row (n, ny the normalised x' and y; ny = y without a norm behind the branch):
//   w = dh gain (1 + scale);  D = dx_out + norm'(w);  dx = res_scale D;  du = gate D
//   dy = norm_post'(du post_gain), or du
// and over the rows of a batch entry, per channel: P = sum dh n, S = sum dh, Q = sum D ny. From them
//   dscale = gain P, dshift = S, dgate = post_gain Q, dgain = sum_b (1 + scale) P, dpost_gain = sum_b gate Q.
// x' and its statistics are formed again from x and y, so the forward pass keeps nothing. P, S and
// Q stay in registers over a block's rows, go to the workspace once per block, and a second kernel
// adds the blocks in a fixed order: no atomics, the same bits every time.
template <typename T, int V, int E, int MAXT>
__global__ void __launch_bounds__(MAXT) sol_residual_norm_bwd_kernel(const __grid_constant__ NormBwdArgs p, int tpr) {
  constexpr int NV = E / V;
  __shared__ float s_buf[2 * kMaxWarps * 2];
  RowGroup g = row_group(s_buf, tpr);
  const int rpb = blockDim.x / tpr, sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
  const int b = blockIdx.x / p.chunks, chunk = blockIdx.x - b * p.chunks;
  const float inv_c = 1.0f / static_cast<float>(p.C);
  const NormArgs& f = p.fwd;
  bool on[NV];
  int c[NV];
  float aP[NV][V], aS[NV][V], aQ[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    c[j] = (j * tpr + t) * V;
    on[j] = c[j] < p.C;
#pragma unroll
    for (int k = 0; k < V; ++k) aP[j][k] = aS[j][k] = aQ[j][k] = 0.f;
  }
  for (int r0 = chunk * rpb; r0 < f.T; r0 += p.chunks * rpb) {
    const int row = r0 + sub;
    const bool live = row < f.T;
    const size_t base = (static_cast<size_t>(b) * f.T + (live ? row : 0)) * p.C;
    float x[NV][V], y[NV][V], w[NV][V], d[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int k = 0; k < V; ++k) x[j][k] = y[j][k] = w[j][k] = d[j][k] = 0.f;
      if (live && on[j]) {
        load_vec<T, V>(static_cast<const T*>(f.x) + base + c[j], x[j]);
        if (f.y != nullptr) load_vec<T, V>(static_cast<const T*>(f.y) + base + c[j], y[j]);
        load_vec<T, V>(static_cast<const T*>(p.dh) + base + c[j], w[j]);
        if (p.dx_out != nullptr) load_vec<T, V>(static_cast<const T*>(p.dx_out) + base + c[j], d[j]);
      }
    }
    float ry = 0.f;
    if (f.y != nullptr) {
      if (f.post_norm != NORM_NONE) ry = normalise<V, NV>(g, y, on, f.post_norm, inv_c, f.eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!on[j]) continue;
        float u[V], v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) u[k] = y[j][k];
        if (f.post_gain != nullptr) {
          load_param<V>(f.post_gain + c[j], v);
#pragma unroll
          for (int k = 0; k < V; ++k) u[k] *= v[k];
        }
        if (f.gate != nullptr) {
          load_param<V>(f.gate + static_cast<size_t>(b) * f.gate_stride + c[j], v);
#pragma unroll
          for (int k = 0; k < V; ++k) u[k] *= v[k];
        }
#pragma unroll
        for (int k = 0; k < V; ++k) x[j][k] = fmaf(f.res_scale, x[j][k], u[k]);
      }
    }
    const float r = normalise<V, NV>(g, x, on, f.norm, inv_c, f.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!on[j]) continue;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        aP[j][k] = fmaf(w[j][k], x[j][k], aP[j][k]);
        aS[j][k] += w[j][k];
      }
      float v[V];
      if (f.gain != nullptr) {
        load_param<V>(f.gain + c[j], v);
#pragma unroll
        for (int k = 0; k < V; ++k) w[j][k] *= v[k];
      }
      if (f.scale != nullptr) {
        load_param<V>(f.scale + static_cast<size_t>(b) * f.scale_stride + c[j], v);
#pragma unroll
        for (int k = 0; k < V; ++k) w[j][k] = fmaf(w[j][k], v[k], w[j][k]);
      }
    }
    normalise_back<V, NV>(g, w, x, r, f.norm, inv_c);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!on[j]) continue;
      float o[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        d[j][k] += w[j][k];
        o[k] = f.y != nullptr ? f.res_scale * d[j][k] : d[j][k];
      }
      if (live) store_vec<T, V>(static_cast<T*>(p.dx) + base + c[j], o);
    }
    if (f.y != nullptr) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!on[j]) continue;
        float v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) aQ[j][k] = fmaf(d[j][k], y[j][k], aQ[j][k]);
        if (f.gate != nullptr) {
          load_param<V>(f.gate + static_cast<size_t>(b) * f.gate_stride + c[j], v);
#pragma unroll
          for (int k = 0; k < V; ++k) d[j][k] *= v[k];
        }
        if (f.post_gain != nullptr) {
          load_param<V>(f.post_gain + c[j], v);
#pragma unroll
          for (int k = 0; k < V; ++k) d[j][k] *= v[k];
        }
      }
      if (f.post_norm != NORM_NONE) normalise_back<V, NV>(g, d, y, ry, f.post_norm, inv_c);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (live && on[j]) store_vec<T, V>(static_cast<T*>(p.dy) + base + c[j], d[j]);
    }
  }
  // a row past the end added zeros only
  if (p.part != nullptr) {
    float* part = p.part + static_cast<size_t>(blockIdx.x * rpb + sub) * 3 * p.C;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!on[j]) continue;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        part[c[j] + k] = aP[j][k];
        part[p.C + c[j] + k] = aS[j][k];
        if (f.y != nullptr) part[2 * static_cast<size_t>(p.C) + c[j] + k] = aQ[j][k];
      }
    }
  }
}

constexpr int kSumCols = 32, kSumRows = 16;

// Sums over `n` rows of one column, by the kSumRows threads of a block column; all of them return it.
template <typename F>
__device__ __forceinline__ float column_sum(F&& get, int n) {
  __shared__ float s[kSumRows][kSumCols + 1];
  float a = 0.f;
#pragma unroll 4
  for (int i = threadIdx.y; i < n; i += kSumRows) a += get(i);
  __syncthreads();
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kSumRows; ++i) t += s[i][threadIdx.x];
  return t;
}

// The gradients of one batch entry's vectors from the partial sums; where shared gains have several
// batch entries to add, the entry's P and Q replace its first slot for the next kernel.
__global__ void __launch_bounds__(kSumCols* kSumRows) sol_residual_norm_sum_kernel(const __grid_constant__ NormBwdArgs p,
                                                                                  int slots) {
  const int b = blockIdx.y, cc = blockIdx.x * kSumCols + threadIdx.x;
  const bool on = cc < p.C;
  const int c = on ? cc : 0;
  const NormArgs& f = p.fwd;
  float* part = p.part + static_cast<size_t>(b) * slots * 3 * p.C;
  const size_t step = 3 * static_cast<size_t>(p.C);
  const bool first = threadIdx.y == 0 && on;
  if (p.dscale != nullptr || p.dgain != nullptr) {
    const float P = column_sum([&](int i) { return part[i * step + c]; }, slots);
    if (first) {
      if (p.dscale != nullptr) p.dscale[static_cast<size_t>(b) * p.C + c] = f.gain != nullptr ? f.gain[c] * P : P;
      if (p.dgain != nullptr) {
        const float one = f.scale != nullptr ? P * (1.0f + f.scale[static_cast<size_t>(b) * f.scale_stride + c]) : P;
        if (f.B == 1) p.dgain[c] = one;
        else part[c] = one;
      }
    }
  }
  if (p.dshift != nullptr) {
    const float S = column_sum([&](int i) { return part[i * step + p.C + c]; }, slots);
    if (first) p.dshift[static_cast<size_t>(b) * p.C + c] = S;
  }
  if (p.dgate != nullptr || p.dpost_gain != nullptr) {
    const float Q = column_sum([&](int i) { return part[i * step + 2 * static_cast<size_t>(p.C) + c]; }, slots);
    if (first) {
      if (p.dgate != nullptr) p.dgate[static_cast<size_t>(b) * p.C + c] = f.post_gain != nullptr ? f.post_gain[c] * Q : Q;
      if (p.dpost_gain != nullptr) {
        const float one = f.gate != nullptr ? Q * f.gate[static_cast<size_t>(b) * f.gate_stride + c] : Q;
        if (f.B == 1) p.dpost_gain[c] = one;
        else part[2 * static_cast<size_t>(p.C) + c] = one;
      }
    }
  }
}

// The shared gains' gradients: the batch entries' shares added.
__global__ void __launch_bounds__(kSumCols* kSumRows) sol_residual_norm_sum_b_kernel(const __grid_constant__ NormBwdArgs p,
                                                                                    int slots) {
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

int threads_per_row(int C, int elems) { return (C + 32 * elems - 1) / (32 * elems) * 32; }
int rows_per_block(int tpr) { return tpr >= 256 ? 1 : 256 / tpr; }

template <typename T, int V>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t stream) {
  const int tpr = threads_per_row(a.C, kFwdElems), rpb = rows_per_block(tpr), nt = tpr * rpb;
  const long long blocks = (static_cast<long long>(a.B) * a.T + rpb - 1) / rpb;
  const int grid = static_cast<int>(blocks < 0x7fffffffll ? blocks : 0x7fffffffll);
  if (nt <= 256) sol_residual_norm_kernel<T, V, kFwdElems, 256><<<grid, nt, 0, stream>>>(a, tpr);
  else sol_residual_norm_kernel<T, V, kFwdElems, 512><<<grid, nt, 0, stream>>>(a, tpr);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_bwd(const NormBwdArgs& a, cudaStream_t stream) {
  const int tpr = threads_per_row(a.C, kBwdElems), rpb = rows_per_block(tpr), nt = tpr * rpb;
  const int grid = a.fwd.B * a.chunks;
  if (nt <= 256) sol_residual_norm_bwd_kernel<T, V, kBwdElems, 256><<<grid, nt, 0, stream>>>(a, tpr);
  else if (nt <= 512) sol_residual_norm_bwd_kernel<T, V, kBwdElems, 512><<<grid, nt, 0, stream>>>(a, tpr);
  else sol_residual_norm_bwd_kernel<T, V, kBwdElems, 1024><<<grid, nt, 0, stream>>>(a, tpr);
  return cudaGetLastError();
}

}  // namespace

int norm_bwd_chunks(int B, int T, int C) {
  const int rpb = rows_per_block(threads_per_row(C, kBwdElems));
  const int most = (T + rpb - 1) / rpb;
  const int want = kNormBwdBlocks / B > 1 ? kNormBwdBlocks / B : 1;
  return most < want ? most : want;
}
size_t norm_bwd_part_floats(int B, int T, int C) {
  return static_cast<size_t>(B) * norm_bwd_chunks(B, T, C) * rows_per_block(threads_per_row(C, kBwdElems)) * 3 * C;
}

cudaError_t launch_residual_norm(const NormArgs& a, cudaStream_t stream) {
  if (a.bf16) return a.vec ? launch_fwd<__nv_bfloat16, 8>(a, stream) : launch_fwd<__nv_bfloat16, 1>(a, stream);
  return a.vec ? launch_fwd<float, 4>(a, stream) : launch_fwd<float, 1>(a, stream);
}

cudaError_t launch_residual_norm_bwd(const NormBwdArgs& a, cudaStream_t stream) {
  const NormArgs& f = a.fwd;
  cudaError_t e;
  if (f.bf16) e = f.vec ? launch_bwd<__nv_bfloat16, 8>(a, stream) : launch_bwd<__nv_bfloat16, 1>(a, stream);
  else e = f.vec ? launch_bwd<float, 4>(a, stream) : launch_bwd<float, 1>(a, stream);
  if (e != cudaSuccess || a.part == nullptr) return e;
  const int slots = a.chunks * rows_per_block(threads_per_row(a.C, kBwdElems));
  const dim3 block(kSumCols, kSumRows);
  const unsigned cols = (a.C + kSumCols - 1) / kSumCols;
  sol_residual_norm_sum_kernel<<<dim3(cols, f.B), block, 0, stream>>>(a, slots);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (f.B > 1 && (a.dgain != nullptr || a.dpost_gain != nullptr)) {
    sol_residual_norm_sum_b_kernel<<<cols, block, 0, stream>>>(a, slots);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace sol
