// Rotary positions of queries and keys, and the cosine and sine tables of the fused norm pass.
//
// A pair (a, b) of channels turns by angle(t, i) = pos[axis(i)][t] * inv_freq[i]:
//   (a, b) -> m (a cos - b sin, a sin + b cos)
// with m the factor of a stretched context; the inverse turns by -angle (the gradient of the first).
// Pairs are interleaved, (2i, 2i + 1), or halves, (i, i + rot / 2); channels from rot on pass through.
//
// A position of 10^6 turns its fastest pair by 10^6 radians, where a 32-bit angle is off by 0.03. So a
// pair's turn per position, modulo one, becomes a 64-bit fraction, and the angle is position times
// fraction in integers, where whole turns fall off by themselves; its top 32 bits are the angle to
// 2^-32 of a turn. Cosine and sine of what is left of it in the nearest quarter turn come from their
// Taylor series, good to about 1e-7 at every position. The 64-bit float work is one product per pair.
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

// Turn per position of a pair, modulo one, as a 64-bit fraction.
__device__ __forceinline__ unsigned long long turn_fraction(double inv_freq) {
  const double f = inv_freq * 0.15915494309189533577;  // over 2 pi
  return __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
}
// m cos, m sin at a position.
__device__ __forceinline__ void turn(int pos, unsigned long long fraction, float m, float& c, float& s) {
  const uint32_t lo = static_cast<uint32_t>(fraction), hi = static_cast<uint32_t>(fraction >> 32);
  uint32_t a = static_cast<uint32_t>(pos) * hi + __umulhi(static_cast<uint32_t>(pos), lo);
  if (pos < 0) a -= lo;  // the product of a negative position, as its low 32 bits are above 0
  const uint32_t quarter = (a + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int>(a - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi 2^-32: |x| <= pi / 4
  const float q = x * x;
  // degrees 9 and 10: the next terms are below 2e-9 and 2e-10 of the first
  float sn = fmaf(q, 2.7557319e-6f, -1.9841270e-4f);
  sn = fmaf(sn, q, 8.3333333e-3f);
  sn = fmaf(sn, q, -1.6666667e-1f);
  sn = fmaf(sn * q, x, x);
  float cs = fmaf(q, -2.7557319e-7f, 2.4801587e-5f);
  cs = fmaf(cs, q, -1.3888889e-3f);
  cs = fmaf(cs, q, 4.1666667e-2f);
  cs = fmaf(cs, q, -0.5f);
  cs = fmaf(cs, q, 1.0f);
  const float cc = (quarter & 1u) ? sn : cs, ss = (quarter & 1u) ? cs : sn;  // cos(x + pi/2) = -sin x, ..
  c = ((quarter + 1u) & 2u) ? -m * cc : m * cc;
  s = (quarter & 2u) ? -m * ss : m * ss;
}
__device__ __forceinline__ int axis_of(const int (&end)[4], int i) { return (i >= end[0]) + (i >= end[1]) + (i >= end[2]); }
__device__ __forceinline__ void turn_of(const RopeArgs& p, int b, int t, int i, float& c, float& s) {
  turn(__ldg(p.pos + b * p.pos_b + static_cast<size_t>(axis_of(p.end, i)) * p.L + t), turn_fraction(__ldg(p.inv_freq + i)),
       p.factor, c, s);
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
    if (2 * k < turned) turn_of(p, b, t, col / 2 + k, c[k], s[k]);
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
    turn_of(p, b, t, col + k, c[k], s[k]);
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

// Tables: V pairs of one token per thread and turn of the loop, the same pairs every time, so that
// their fractions stay in registers. Bound by the stores.
template <int V>
__global__ void __launch_bounds__(kThreads) sol_rope_tables_kernel(const __grid_constant__ RopeTableArgs p, int groups, int tokens) {
  const int half = p.rot / 2, g = threadIdx.x % groups;
  if (threadIdx.x >= groups * tokens) return;
  for (int j = g * V; j < half; j += groups * V) {
    unsigned long long f[V];
    const int* pos[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      f[k] = turn_fraction(__ldg(p.inv_freq + j + k));
      pos[k] = p.pos + static_cast<size_t>(axis_of(p.end, j + k)) * p.L;
    }
    const long long step = static_cast<long long>(gridDim.x) * tokens;
    for (long long t = static_cast<long long>(blockIdx.x) * tokens + threadIdx.x / groups; t < p.L; t += step) {
      float c[V], s[V];
#pragma unroll
      for (int k = 0; k < V; ++k) turn(__ldg(pos[k] + t), f[k], p.factor, c[k], s[k]);
      const size_t o = static_cast<size_t>(t) * half + j;
      if constexpr (V == 4) {
        *reinterpret_cast<float4*>(p.cos + o) = make_float4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<float4*>(p.sin + o) = make_float4(s[0], s[1], s[2], s[3]);
      } else {
        p.cos[o] = c[0];
        p.sin[o] = s[0];
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  if (a.bf16) return a.vec ? launch_t<__nv_bfloat16, 8>(a, num_sms, stream) : launch_t<__nv_bfloat16, 1>(a, num_sms, stream);
  return a.vec ? launch_t<float, 4>(a, num_sms, stream) : launch_t<float, 1>(a, num_sms, stream);
}

cudaError_t launch_rope_tables(const RopeTableArgs& a, int num_sms, cudaStream_t stream) {
  const int half = a.rot / 2;
  const bool vec = half % 4 == 0 && (reinterpret_cast<uintptr_t>(a.cos) & 15u) == 0 && (reinterpret_cast<uintptr_t>(a.sin) & 15u) == 0;
  const int per_token = vec ? half / 4 : half, groups = per_token < kThreads ? per_token : kThreads, tokens = kThreads / groups;
  const long long blocks = (static_cast<long long>(a.L) + tokens - 1) / tokens, most = 8ll * num_sms;
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  if (vec) sol_rope_tables_kernel<4><<<grid, kThreads, 0, stream>>>(a, groups, tokens);
  else sol_rope_tables_kernel<1><<<grid, kThreads, 0, stream>>>(a, groups, tokens);
  return cudaGetLastError();
}

}  // namespace sol
