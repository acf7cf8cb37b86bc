// Rotary positions of queries and keys, and the cosine and sine tables of the fused norm pass.
//
// A pair (a, b) of channels turns by angle(t, i) = pos[axis(i)][t] * inv_freq[i]:
//   (a, b) -> m (a cos - b sin, a sin + b cos)
// with m the factor of a stretched context; the inverse turns by -angle (the gradient of the first).
// Pairs are interleaved, (2i, 2i + 1), or halves, (i, i + rot / 2); channels from rot on pass through.
//
// Angles are formed in 64 bits: a position of 10^6 turns its fastest pair by 10^6 radians, where a
// 32-bit angle is off by 0.03. The angle over pi is reduced to [-1, 1] there and only the rest goes
// to 32 bits, so cosine and sine are good to about 2e-7 at every position.
//
// HBM-bound: every element is read and written once. A thread owns one 16-byte vector of columns (a
// vector of each half in the half layout) of one token, forms its cosines and sines once and then
// runs over heads with them, so their cost is shared by all heads of a token. Input and output have
// strides of their own: the same pass takes a token-major projection to head-major rows, or back.
#include <cmath>

#include "device_common.cuh"
#include "launchers.h"

namespace sol {

namespace {

constexpr int kThreads = 256;

// m cos, m sin of pair i at the given token (column of pos)
__device__ __forceinline__ void turn(const int* pos, int L, const double* inv_freq, const int (&end)[4], int i,
                                     float factor, float& c, float& s) {
  const int axis = (i >= end[0]) + (i >= end[1]) + (i >= end[2]);
  const double x = static_cast<double>(__ldg(pos + static_cast<size_t>(axis) * L)) * __ldg(inv_freq + i) *
                   0.31830988618379067154;  // angle / pi
  const double y = x - 2.0 * rint(0.5 * x);
  sincospif(static_cast<float>(y), &s, &c);
  c *= factor;
  s *= factor;
}

template <typename T, int V>
struct Vec {
  float x[V];
  __device__ __forceinline__ void load(const T* p) {
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
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] = static_cast<float>(p[k]);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else if constexpr (V == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < V; ++k) p[k] = __float2bfloat16_rn(x[k]);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) p[k] = x[k];
    }
  }
};

// V values moved as bits.
template <typename T, int V>
__device__ __forceinline__ void copy_vec(T* out, const T* in) {
  if constexpr (V * sizeof(T) == 16) {
    *reinterpret_cast<uint4*>(out) = __ldg(reinterpret_cast<const uint4*>(in));
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) out[k] = in[k];
  }
}

// Calls f(in, out) for heads [h0, h1) of the queries followed by the keys.
template <typename T, typename F>
__device__ __forceinline__ void for_heads(const RopeArgs& p, int b, int t, int h0, int h1, F&& f) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const RopeSide& r = p.side[s];
    const int shift = s == 0 ? 0 : p.side[0].heads;
    const int lo = max(h0 - shift, 0), hi = min(h1 - shift, r.heads);
    const T* in = static_cast<const T*>(r.in) + b * r.in_b + t * r.in_l;
    T* out = static_cast<T*>(r.out) + b * r.out_b + t * r.out_l;
    f(in, out, r.in_h, r.out_h, lo, hi);
  }
}

// Interleaved pairs: N columns of consecutive pairs per thread. V = N: one vector. V = 2 values is
// one pair read and written as scalars.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) sol_rope_interleaved_kernel(const __grid_constant__ RopeArgs p, int groups,
                                                                         int heads_per_block) {
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int t = static_cast<int>(i / groups), g = static_cast<int>(i - static_cast<long long>(t) * groups);
  if (t >= p.L) return;
  const int b = blockIdx.z, col = g * V;
  const int heads = p.side[0].heads + p.side[1].heads;
  const int h0 = blockIdx.y * heads_per_block, h1 = min(h0 + heads_per_block, heads);
  if (col >= p.rot) {  // the rest passes through as bits, infinities and NaN included
    for_heads<T>(p, b, t, h0, h1, [&](const T* in, T* out, long long ih, long long oh, int lo, int hi) {
#pragma unroll 4
      for (int h = lo; h < hi; ++h) copy_vec<T, V>(out + h * oh + col, in + h * ih + col);
    });
    return;
  }
  const int turned = min(V, p.rot - col);  // a vector across the border: its first values turn
  float c[V / 2], s[V / 2];
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    c[k] = 1.f;
    s[k] = 0.f;
    if (2 * k < turned) turn(p.pos + b * p.pos_b + t, p.L, p.inv_freq, p.end, col / 2 + k, p.factor, c[k], s[k]);
    if (p.inverse) s[k] = -s[k];
  }
  for_heads<T>(p, b, t, h0, h1, [&](const T* in, T* out, long long ih, long long oh, int lo, int hi) {
#pragma unroll 4
    for (int h = lo; h < hi; ++h) {
      Vec<T, V> v;
      v.load(in + h * ih + col);
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const float a = v.x[2 * k], q = v.x[2 * k + 1];
        v.x[2 * k] = fmaf(a, c[k], -q * s[k]);
        v.x[2 * k + 1] = fmaf(a, s[k], q * c[k]);
      }
      if (turned == V) {
        v.store(out + h * oh + col);
      } else {
        for (int k = 0; k < V; ++k) {
          T* o = out + h * oh + col + k;
          if (k >= turned) *o = in[h * ih + col + k];
          else if constexpr (sizeof(T) == 2) *o = __float2bfloat16_rn(v.x[k]);
          else *o = v.x[k];
        }
      }
    }
  });
}

// Half layout: V pairs per thread, (i, i + rot / 2); groups past those copy V channels of the rest.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) sol_rope_half_kernel(const __grid_constant__ RopeArgs p, int groups,
                                                                  int heads_per_block) {
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int t = static_cast<int>(i / groups), g = static_cast<int>(i - static_cast<long long>(t) * groups);
  if (t >= p.L) return;
  const int b = blockIdx.z, half = p.rot / 2;
  const int heads = p.side[0].heads + p.side[1].heads;
  const int h0 = blockIdx.y * heads_per_block, h1 = min(h0 + heads_per_block, heads);
  if (g * V >= half) {
    const int col = p.rot + g * V - half;
    for_heads<T>(p, b, t, h0, h1, [&](const T* in, T* out, long long ih, long long oh, int lo, int hi) {
#pragma unroll 4
      for (int h = lo; h < hi; ++h) copy_vec<T, V>(out + h * oh + col, in + h * ih + col);
    });
    return;
  }
  const int col = g * V;
  float c[V], s[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    turn(p.pos + b * p.pos_b + t, p.L, p.inv_freq, p.end, col + k, p.factor, c[k], s[k]);
    if (p.inverse) s[k] = -s[k];
  }
  for_heads<T>(p, b, t, h0, h1, [&](const T* in, T* out, long long ih, long long oh, int lo, int hi) {
#pragma unroll 4
    for (int h = lo; h < hi; ++h) {
      Vec<T, V> u, w;
      u.load(in + h * ih + col);
      w.load(in + h * ih + col + half);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float a = u.x[k], q = w.x[k];
        u.x[k] = fmaf(a, c[k], -q * s[k]);
        w.x[k] = fmaf(a, s[k], q * c[k]);
      }
      u.store(out + h * oh + col);
      w.store(out + h * oh + col + half);
    }
  });
}

template <typename T, int V>
cudaError_t launch_t(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int VI = V == 1 ? 2 : V;  // an interleaved group is at least one pair
  // V divides every width here (the caller's rule for vec); a scalar group is one pair or channel
  const int rest = a.copy_rest ? a.d - a.rot : 0;
  const int groups = a.half ? a.rot / 2 / V + rest / V : (a.rot + rest + VI - 1) / VI;
  const long long blocks = (static_cast<long long>(a.L) * groups + kThreads - 1) / kThreads;
  const int heads = a.side[0].heads + a.side[1].heads;
  // Heads of one token share their cosines: as many per block as leave four blocks per SM, but at
  // least four, the number of rows in flight per thread.
  long long split = 4ll * num_sms / (blocks * a.B);
  if (split < 1) split = 1;
  int hpb = static_cast<int>((heads + split - 1) / split);
  if (hpb < 4) hpb = heads < 4 ? heads : 4;
  const dim3 grid(static_cast<unsigned>(blocks), (heads + hpb - 1) / hpb, a.B);
  if (a.half) sol_rope_half_kernel<T, V><<<grid, kThreads, 0, stream>>>(a, groups, hpb);
  else sol_rope_interleaved_kernel<T, VI><<<grid, kThreads, 0, stream>>>(a, groups, hpb);
  return cudaGetLastError();
}

__global__ void __launch_bounds__(kThreads) sol_rope_tables_kernel(const __grid_constant__ RopeTableArgs p) {
  const int half = p.rot / 2;
  const long long n = static_cast<long long>(p.L) * half;
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= n) return;
  const int t = static_cast<int>(i / half), j = static_cast<int>(i - static_cast<long long>(t) * half);
  float c, s;
  turn(p.pos + t, p.L, p.inv_freq, p.end, j, p.factor, c, s);
  p.cos[i] = c;
  p.sin[i] = s;
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  if (a.bf16) return a.vec ? launch_t<__nv_bfloat16, 8>(a, num_sms, stream) : launch_t<__nv_bfloat16, 1>(a, num_sms, stream);
  return a.vec ? launch_t<float, 4>(a, num_sms, stream) : launch_t<float, 1>(a, num_sms, stream);
}

cudaError_t launch_rope_tables(const RopeTableArgs& a, cudaStream_t stream) {
  const long long n = static_cast<long long>(a.L) * (a.rot / 2);
  sol_rope_tables_kernel<<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace sol
