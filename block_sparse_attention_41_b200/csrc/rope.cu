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
// Taylor series in fp32. What that costs, in units of u = 2^-24 with a factor of 1: 0.1 u for the angle cut to 2^-32
// of a turn (6 u more at the far end of 32-bit positions, for the rounding of the frequency over 2 pi in 64 bits), 1.7 u
// for its value in radians (converted, times a rounded constant, rounded: 3 u of at most pi / 4, times a slope of 0.71),
// 1.4 u for the polynomial and the multiplication by the factor: at most 4 u up to positions of 10^7. The 64-bit float work is one product per pair.
//
// HBM-bound: every element is read and written once. A thread owns one vector of columns of one token
// (one of each half in the half layout), of 16 bytes where lengths, strides and addresses allow. It forms
// its cosines and sines once and then runs over heads with them, so their cost is shared by all heads of
// a token. Input and output have strides of their own: the same pass takes a token-major projection to
// head-major rows, or back. 75600 tokens of 80 heads of 128 bf16: 488 us, 6.3 TB/s.
#include <cmath>

#include "chained.cuh"
#include "device_common.cuh"
#include "launchers.h"

namespace sol {

namespace {

constexpr int kThreads = 128;       // of a rotary block
constexpr int kTableThreads = 256;

// Turn per position of a pair, modulo one, as a 64-bit fraction: hi 2^32 + lo with a signed lo.
struct Fraction {
  int hi, lo;
};
__device__ __forceinline__ Fraction turn_fraction(double inv_freq) {
  const double f = inv_freq * 0.15915494309189533577;  // over 2 pi
  const unsigned long long u = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
  const int lo = static_cast<int>(static_cast<uint32_t>(u));
  return {static_cast<int>(static_cast<uint32_t>(u >> 32) + (lo < 0 ? 1u : 0u)), lo};
}
// The top 32 bits of a position's angle, in turns; wraps as turns do.
__device__ __forceinline__ uint32_t angle_of(int pos, const Fraction& f) {
  return static_cast<uint32_t>(pos) * static_cast<uint32_t>(f.hi) + static_cast<uint32_t>(__mulhi(pos, f.lo));
}
// m cos, m sin of two angles.
__device__ __forceinline__ void turn2(uint32_t a0, uint32_t a1, float m, float (&c)[2], float (&s)[2]) {
  const uint32_t a[2] = {a0, a1};
  uint32_t quarter[2];
  float r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    quarter[i] = a[i] + 0x20000000u;  // the nearest quarter turn, in its top two bits
    r[i] = static_cast<float>(static_cast<int>(a[i] - (quarter[i] & 0xc0000000u)));
  }
  auto two = [](float v) { return pack2(v, v); };
  const f2 x = mul2(pack2(r[0], r[1]), two(1.4629180792671596e-9f));  // 2 pi 2^-32: |x| <= pi / 4
  const f2 q = mul2(x, x);
  // degrees 9 and 10: the next terms are below 2e-9 and 2e-10 of the first
  f2 sn = fma2(q, two(2.7557319e-6f), two(-1.9841270e-4f));
  sn = fma2(sn, q, two(8.3333333e-3f));
  sn = fma2(sn, q, two(-1.6666667e-1f));
  sn = fma2(mul2(sn, q), x, x);
  f2 cs = fma2(q, two(-2.7557319e-7f), two(2.4801587e-5f));
  cs = fma2(cs, q, two(-1.3888889e-3f));
  cs = fma2(cs, q, two(4.1666667e-2f));
  cs = fma2(cs, q, two(-0.5f));
  cs = fma2(cs, q, two(1.0f));
  const float2 sv = unpack2(mul2(sn, two(m))), cv = unpack2(mul2(cs, two(m)));
  const float ss[2] = {sv.x, sv.y}, cc[2] = {cv.x, cv.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // cos(x + pi / 2) = -sin x, sin(x + pi / 2) = cos x, and their negatives
    const bool odd = (quarter[i] & 0x40000000u) != 0;
    const uint32_t neg_s = quarter[i] & 0x80000000u, neg_c = (quarter[i] + 0x40000000u) & 0x80000000u;
    c[i] = __uint_as_float(__float_as_uint(odd ? ss[i] : cc[i]) ^ neg_c);
    s[i] = __uint_as_float(__float_as_uint(odd ? cc[i] : ss[i]) ^ neg_s);
  }
}
__device__ __forceinline__ int axis_of(const int (&end)[4], int i) { return (i >= end[0]) + (i >= end[1]) + (i >= end[2]); }
// m cos, m sin of the pairs i .. i + N - 1 of a token, those past the last with cosine m and sine 0.
template <int N>
__device__ __forceinline__ void turns_of(const RopeArgs& p, int b, int t, int i, int last, float (&c)[N], float (&s)[N]) {
  uint32_t a[N + 1];
  a[N] = 0;
#pragma unroll
  for (int k = 0; k < N; ++k)
    a[k] = i + k < last ? angle_of(__ldg(p.pos + b * p.pos_b + static_cast<size_t>(axis_of(p.end, i + k)) * p.L + t),
                                   turn_fraction(__ldg(p.inv_freq + i + k)))
                        : 0u;
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    float cc[2], ss[2];
    turn2(a[k], a[k + 1], p.factor, cc, ss);
    c[k] = cc[0];
    s[k] = p.inverse ? -ss[0] : ss[0];
    if (k + 1 < N) {
      c[k + 1] = cc[1];
      s[k + 1] = p.inverse ? -ss[1] : ss[1];
    }
  }
}

// V values as 32-bit words, in one access of 4, 8 or 16 bytes (WIDE) or one by one.
template <typename T, int V>
using Words = uint32_t[V * sizeof(T) / 4 > 0 ? V * sizeof(T) / 4 : 1];
template <typename T, int V>
__device__ __forceinline__ void load_wide(const T* p, Words<T, V>& w) {
  if constexpr (V * sizeof(T) == 16) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (V * sizeof(T) == 8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_wide(T* p, const Words<T, V>& w) {
  if constexpr (V * sizeof(T) == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (V * sizeof(T) == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(p) = w[0];
}

// V values, as fp32 and as they were read: a store may keep those (infinities and NaN included).
template <typename T, int V, bool WIDE>
struct Vec {
  enum : int { kWords = V * static_cast<int>(sizeof(T)) / 4 };
  float x[V];
  Words<T, V> w;
  T one[WIDE ? 1 : V];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (WIDE) {
      load_wide<T, V>(p, w);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if constexpr (sizeof(T) == 4) x[k] = __uint_as_float(w[k]);
        else x[k] = __uint_as_float(k % 2 == 0 ? w[k / 2] << 16 : w[k / 2] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        one[k] = p[k];
        x[k] = static_cast<float>(one[k]);
      }
    }
  }
  __device__ __forceinline__ void store(T* p, bool as_read) const {
    if constexpr (WIDE) {
      Words<T, V> o;
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        if constexpr (sizeof(T) == 4) o[k] = __float_as_uint(x[k]);
        else o[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
        if (as_read) o[k] = w[k];
      }
      store_wide<T, V>(p, o);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        T o;
        if constexpr (sizeof(T) == 2) o = __float2bfloat16_rn(x[k]);
        else o = x[k];
        p[k] = as_read ? one[k] : o;
      }
    }
  }
};

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

// A pass with channels that only pass through has them in the same loop as the turned ones, where the
// store chooses: threads of a warp that took loops of their own would wait for one another. Without such
// channels the loop has no choice in it (75600 tokens of 80 heads of 128, bf16: 488 us, 567 with one: it
// kept the loads of several heads from going out together).

// Interleaved pairs: V columns of consecutive pairs per thread.
template <typename T, int V, bool WIDE>
__global__ void __launch_bounds__(kThreads, 8) sol_rope_interleaved_kernel(const __grid_constant__ RopeArgs p, int groups,
                                                                         int heads_per_block) {
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int t = static_cast<int>(i / groups), g = static_cast<int>(i - static_cast<long long>(t) * groups);
  if (t >= p.L) return;
  chained_wait();
  const int b = blockIdx.z, col = g * V;
  const int heads = p.side[0].heads + p.side[1].heads;
  const int h0 = blockIdx.y * heads_per_block, h1 = min(h0 + heads_per_block, heads);
  const bool keep = col >= p.rot;
  float c[V / 2], s[V / 2];
  turns_of<V / 2>(p, b, t, col / 2, p.rot / 2, c, s);
  auto run = [&](bool as_read) {
    for_heads<T>(p, b, t, h0, h1, [&](const T* in, T* out, long long ih, long long oh, int lo, int hi) {
#pragma unroll 4
      for (int h = lo; h < hi; ++h) {
        Vec<T, V, WIDE> v;
        v.load(in + h * ih + col);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
          const float a = v.x[2 * k], q = v.x[2 * k + 1];
          v.x[2 * k] = fmaf(a, c[k], -q * s[k]);
          v.x[2 * k + 1] = fmaf(a, s[k], q * c[k]);
        }
        v.store(out + h * oh + col, as_read);
      }
    });
  };
  if (groups * V == p.rot) run(false);
  else run(keep);
}

// Half layout: V pairs per thread, (i, i + rot / 2); groups past those pass two vectors of the rest through.
template <typename T, int V, bool WIDE>
__global__ void __launch_bounds__(kThreads, 8) sol_rope_half_kernel(const __grid_constant__ RopeArgs p, int groups,
                                                                  int heads_per_block) {
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int t = static_cast<int>(i / groups), g = static_cast<int>(i - static_cast<long long>(t) * groups);
  if (t >= p.L) return;
  chained_wait();
  const int b = blockIdx.z, half = p.rot / 2;
  const int heads = p.side[0].heads + p.side[1].heads;
  const int h0 = blockIdx.y * heads_per_block, h1 = min(h0 + heads_per_block, heads);
  const bool keep = g * V >= half;
  const int first = keep ? p.rot + 2 * (g * V - half) : g * V;
  const bool both = !keep || first + V < p.d;
  const int second = !keep ? first + half : both ? first + V : first;
  float c[V], s[V];
  turns_of<V>(p, b, t, g * V, half, c, s);
  auto run = [&](bool as_read, bool two) {
    for_heads<T>(p, b, t, h0, h1, [&](const T* in, T* out, long long ih, long long oh, int lo, int hi) {
#pragma unroll 4
      for (int h = lo; h < hi; ++h) {
        Vec<T, V, WIDE> u, w;
        u.load(in + h * ih + first);
        w.load(in + h * ih + second);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float a = u.x[k], q = w.x[k];
          u.x[k] = fmaf(a, c[k], -q * s[k]);
          w.x[k] = fmaf(a, s[k], q * c[k]);
        }
        u.store(out + h * oh + first, as_read);
        if (two) w.store(out + h * oh + second, as_read);
      }
    });
  };
  if (groups * V == half) run(false, true);
  else run(keep, both);
}

template <typename T, int V>
cudaError_t launch_t(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr bool WIDE = V * sizeof(T) >= 4 && V > 1;
  constexpr int VI = V == 1 ? 2 : V;  // an interleaved group is at least one pair
  // V divides every width here (the caller's rule); a group of single values is one pair or channel
  const int rest = a.copy_rest ? a.d - a.rot : 0;
  const int groups = a.half ? a.rot / 2 / V + (rest / V + 1) / 2 : (a.rot + rest) / VI;
  const long long blocks = (static_cast<long long>(a.L) * groups + kThreads - 1) / kThreads;
  const int heads = a.side[0].heads + a.side[1].heads;
  // Heads of one token share their cosines: as many per block as leave eight blocks per SM, but at
  // least four, the number of rows in flight per thread.
  long long split = 8ll * num_sms / (blocks * a.B);
  if (split < 1) split = 1;
  int hpb = static_cast<int>((heads + split - 1) / split);
  if (hpb < 4) hpb = heads < 4 ? heads : 4;
  const dim3 grid(static_cast<unsigned>(blocks), (heads + hpb - 1) / hpb, a.B);
  return launch_chained(a.half ? sol_rope_half_kernel<T, V, WIDE> : sol_rope_interleaved_kernel<T, VI, WIDE>, grid, dim3(kThreads), 0, stream, 1,
                        a, groups, hpb);
}

// Tables: V pairs of one token per thread and turn of the loop, the same pairs every time, so that
// their fractions stay in registers. Bound by the stores.
template <int V>
__global__ void __launch_bounds__(kTableThreads) sol_rope_tables_kernel(const __grid_constant__ RopeTableArgs p, int groups, int tokens,
                                                                    int share) {
  const int half = p.rot / 2, g = threadIdx.x % groups;
  chained_wait();
  if (threadIdx.x >= groups * tokens) return;
  // a block's tokens lie together: their positions share cache lines
  const long long from = static_cast<long long>(blockIdx.x) * share;
  const int t_end = static_cast<int>(from + share < p.L ? from + share : p.L);
  if (from + threadIdx.x / groups >= t_end) return;
  const int t_first = static_cast<int>(from) + threadIdx.x / groups;
  for (int j = g * V; j < half; j += groups * V) {
    Fraction f[V];
    const int* pos[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      f[k] = turn_fraction(__ldg(p.inv_freq + j + k));
      pos[k] = p.pos + static_cast<size_t>(axis_of(p.end, j + k)) * p.L;
    }
    const bool one_axis = pos[0] == pos[V - 1];
    int next[V];
    auto read = [&](int t) {
      if (t >= t_end) return;
      next[0] = __ldg(pos[0] + t);
#pragma unroll
      for (int k = 1; k < V; ++k) next[k] = one_axis ? next[0] : __ldg(pos[k] + t);
    };
    read(t_first);
    for (int t = t_first; t < t_end; t += tokens) {
      uint32_t a[V + 1];
      a[V] = 0;
#pragma unroll
      for (int k = 0; k < V; ++k) a[k] = angle_of(next[k], f[k]);
      read(t + tokens);
      float c[V + 1], s[V + 1];
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        float cc[2], ss[2];
        turn2(a[k], a[k + 1], p.factor, cc, ss);
        c[k] = cc[0];
        s[k] = ss[0];
        c[k + 1] = cc[1];
        s[k + 1] = ss[1];
      }
      const size_t o = static_cast<size_t>(t) * half + j;
      if constexpr (V == 4) {
        __stcs(reinterpret_cast<float4*>(p.cos + o), make_float4(c[0], c[1], c[2], c[3]));
        __stcs(reinterpret_cast<float4*>(p.sin + o), make_float4(s[0], s[1], s[2], s[3]));
      } else {
        p.cos[o] = c[0];
        p.sin[o] = s[0];
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  // the widest access that divides every length, stride and address (half layout, 40000 tokens of 32 heads of
  // 128: 278 us with 94 channels turned, pair by pair, 139 with 92, two pairs at a time, 114 with 88, four)
  if (a.bf16) {
    switch (a.width) {
      case 8: return launch_t<__nv_bfloat16, 8>(a, num_sms, stream);
      case 4: return launch_t<__nv_bfloat16, 4>(a, num_sms, stream);
      case 2: return launch_t<__nv_bfloat16, 2>(a, num_sms, stream);
      default: return launch_t<__nv_bfloat16, 1>(a, num_sms, stream);
    }
  }
  switch (a.width) {
    case 4: return launch_t<float, 4>(a, num_sms, stream);
    case 2: return launch_t<float, 2>(a, num_sms, stream);
    default: return launch_t<float, 1>(a, num_sms, stream);
  }
}

cudaError_t launch_rope_tables(const RopeTableArgs& a, int num_sms, cudaStream_t stream) {
  const int half = a.rot / 2;
  const bool vec = half % 4 == 0 && (reinterpret_cast<uintptr_t>(a.cos) & 15u) == 0 && (reinterpret_cast<uintptr_t>(a.sin) & 15u) == 0;
  const int per_token = vec ? half / 4 : half, groups = per_token < kTableThreads ? per_token : kTableThreads, tokens = kTableThreads / groups;
  // four blocks per SM, each with an equal run of whole turns
  const long long turns = (static_cast<long long>(a.L) + tokens - 1) / tokens, per = (turns + 4ll * num_sms - 1) / (4ll * num_sms);
  const unsigned grid = static_cast<unsigned>((turns + per - 1) / per);
  const int share = static_cast<int>(per * tokens);
  return launch_chained(vec ? sol_rope_tables_kernel<4> : sol_rope_tables_kernel<1>, dim3(grid), dim3(kTableThreads), 0, stream, 1, a,
                        groups, tokens, share);
}

}  // namespace sol
