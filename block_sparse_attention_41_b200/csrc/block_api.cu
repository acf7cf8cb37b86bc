// C ABI of the dense operators around the attention (declared in include/sol_attn.h): gated
// residual and norm, rotary positions. Arguments are checked on the host before anything is
// launched; nothing here allocates device memory.
#include <climits>
#include <cmath>

#include "api_common.h"
#include "launchers.h"
#include "sol_attn.h"

namespace {

using namespace sol::api;

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The forward's arguments, checked; the outputs are the caller's to check.
sol_status norm_args(const void* x, const void* y, const float* gate, int64_t gate_stride, const float* gain,
                     const float* scale, int64_t scale_stride, const float* shift, int64_t shift_stride,
                     const float* post_gain, sol_dtype dt, sol_norm norm, sol_norm post_norm, float res_scale, float eps,
                     int B, int T, int C, sol::NormArgs* a) {
  if (dt != SOL_F32 && dt != SOL_BF16) return fail(SOL_EINVAL, "unknown dtype %d", static_cast<int>(dt));
  if (!size_ok(B, 1 << 28) || !size_ok(T, 1 << 28) || !size_ok(C, 1 << 28))
    return fail(SOL_EINVAL, "sizes must be positive (B=%d T=%d C=%d)", B, T, C);
  if (norm != SOL_NORM_LAYER && norm != SOL_NORM_RMS) return fail(SOL_EINVAL, "norm must be layer or rms");
  if (post_norm != SOL_NORM_NONE && post_norm != SOL_NORM_LAYER && post_norm != SOL_NORM_RMS)
    return fail(SOL_EINVAL, "unknown post_norm %d", static_cast<int>(post_norm));
  if (!(eps > 0.f) || std::isinf(eps)) return fail(SOL_EINVAL, "eps=%g must be positive and finite", eps);
  if (!std::isfinite(res_scale)) return fail(SOL_EINVAL, "res_scale=%g must be finite", res_scale);
  if (x == nullptr) return fail(SOL_EINVAL, "x must be non-null");
  if (!aligned16(x) || !aligned16(y)) return fail(SOL_EINVAL, "x and y must be 16-byte aligned");
  if (y == nullptr && (gate != nullptr || post_gain != nullptr || post_norm != SOL_NORM_NONE || res_scale != 1.f))
    return fail(SOL_EINVAL, "gate, post_gain, post_norm and res_scale need y");
  if (post_gain != nullptr && post_norm == SOL_NORM_NONE) return fail(SOL_EINVAL, "post_gain needs post_norm");
  const struct { const float* p; int64_t stride; const char* name; } rows[] = {
      {gate, gate_stride, "gate"}, {scale, scale_stride, "scale"}, {shift, shift_stride, "shift"}};
  for (const auto& r : rows)
    if (r.p != nullptr && B > 1 && r.stride < 0) return fail(SOL_EINVAL, "%s's row stride must not be negative", r.name);
  const float* vecs[] = {gate, gain, scale, shift, post_gain};
  for (const float* v : vecs)
    if (!aligned_to(v, 4)) return fail(SOL_EINVAL, "vectors must be 4-byte aligned");
  if (C > sol::kNormMaxC) return fail(SOL_EUNSUPPORTED, "C=%d exceeds %d", C, sol::kNormMaxC);
  if (static_cast<long long>(B) * T >= (1ll << 31)) return fail(SOL_EUNSUPPORTED, "B*T must be < 2^31");
  a->x = x;
  a->y = y;
  a->gate = gate;
  a->gate_stride = gate_stride;
  a->gain = gain;
  a->scale = scale;
  a->scale_stride = scale_stride;
  a->shift = shift;
  a->shift_stride = shift_stride;
  a->post_gain = post_gain;
  a->x_out = nullptr;
  a->h = nullptr;
  a->B = B;
  a->T = T;
  a->C = C;
  a->norm = norm;
  a->post_norm = post_norm;
  a->res_scale = res_scale;
  a->eps = eps;
  a->bf16 = dt == SOL_BF16;
  // 16-byte accesses: whole vectors per row, and every fp32 vector's rows on 16-byte addresses
  a->vec = C % (a->bf16 ? 8 : 4) == 0;
  for (const float* v : vecs)
    if (!aligned16(v)) a->vec = false;
  for (const auto& r : rows)
    if (r.p != nullptr && B > 1 && r.stride % 4 != 0) a->vec = false;
  return SOL_OK;
}

// The sections of a rotary call as ends of each axis's pairs (unused ends: no pair is past them).
sol_status rope_sections(int rot, int axes, const int* sections, int (&end)[4]) {
  if (axes < 1 || axes > 4) return fail(SOL_EINVAL, "axes=%d must be 1 to 4", axes);
  if (rot < 2 || rot % 2 != 0) return fail(SOL_EINVAL, "rot=%d must be even and at least 2", rot);
  for (int& e : end) e = INT_MAX;
  if (sections == nullptr) {
    if (axes != 1) return fail(SOL_EINVAL, "sections must be given for more than one axis");
    return SOL_OK;
  }
  long long sum = 0;
  for (int i = 0; i < axes; ++i) {
    if (sections[i] < 0 || sections[i] > rot / 2) return fail(SOL_EINVAL, "sections[%d]=%d is out of range", i, sections[i]);
    sum += sections[i];
    if (i < axes - 1) end[i] = static_cast<int>(sum);
  }
  if (sum != rot / 2) return fail(SOL_EINVAL, "sections must add up to rot / 2 = %d (they give %lld)", rot / 2, sum);
  return SOL_OK;
}

}  // namespace

extern "C" {

sol_status sol_attn_residual_norm(const void* x, const void* y, const float* gate, int64_t gate_stride, const float* gain,
                                  const float* scale, int64_t scale_stride, const float* shift, int64_t shift_stride,
                                  const float* post_gain, sol_dtype dt, sol_norm norm, sol_norm post_norm,
                                  float res_scale, float eps, int B, int T, int C, void* x_out, void* h, void* stream) {
  clear_error();
  sol::NormArgs a;
  sol_status st = norm_args(x, y, gate, gate_stride, gain, scale, scale_stride, shift, shift_stride, post_gain, dt, norm,
                            post_norm, res_scale, eps, B, T, C, &a);
  if (st != SOL_OK) return st;
  if (h == nullptr || (y != nullptr) != (x_out != nullptr))
    return fail(SOL_EINVAL, "h must be non-null, and x_out given exactly where y is");
  if (!aligned16(h) || !aligned16(x_out)) return fail(SOL_EINVAL, "x_out and h must be 16-byte aligned");
  int sms = 0;
  if ((st = current_device(&sms)) != SOL_OK) return st;
  a.x_out = x_out;
  a.h = h;
  const cudaError_t e = sol::launch_residual_norm(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "residual norm launch");
  return SOL_OK;
}

size_t sol_attn_residual_norm_bwd_workspace_bytes(int B, int T, int C) {
  if (!size_ok(B, 1 << 28) || !size_ok(T, 1 << 28) || !size_ok(C, sol::kNormMaxC)) return 0;
  return (sol::norm_bwd_part_floats(B, T, C) * 4 + 255) / 256 * 256;
}

sol_status sol_attn_residual_norm_bwd(const void* dh, const void* dx_out, const void* x, const void* y, const float* gate,
                                      int64_t gate_stride, const float* gain, const float* scale, int64_t scale_stride,
                                      const float* post_gain, sol_dtype dt, sol_norm norm, sol_norm post_norm,
                                      float res_scale, float eps, int B, int T, int C, void* dx, void* dy, float* dgate,
                                      float* dgain, float* dscale, float* dshift, float* dpost_gain, void* workspace,
                                      size_t ws_bytes, void* stream) {
  clear_error();
  sol::NormBwdArgs a;
  sol_status st = norm_args(x, y, gate, gate_stride, gain, scale, scale_stride, nullptr, 0, post_gain, dt, norm, post_norm,
                            res_scale, eps, B, T, C, &a.fwd);
  if (st != SOL_OK) return st;
  if (dh == nullptr || dx == nullptr || (y != nullptr) != (dy != nullptr))
    return fail(SOL_EINVAL, "dh and dx must be non-null, and dy given exactly where y is");
  if (dx_out != nullptr && y == nullptr) return fail(SOL_EINVAL, "dx_out needs y: without a residual step there is no x_out");
  const void* ptrs[] = {dh, dx_out, dx, dy, workspace};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return fail(SOL_EINVAL, "device pointers must be 16-byte aligned");
  const struct { const float* want; const float* of; const char* name; } grads[] = {
      {dgate, gate, "gate"}, {dgain, gain, "gain"}, {dscale, scale, "scale"}, {dpost_gain, post_gain, "post_gain"}};
  bool any = dshift != nullptr;
  for (const auto& g : grads) {
    if (g.want != nullptr && g.of == nullptr) return fail(SOL_EINVAL, "the gradient of %s needs %s", g.name, g.name);
    if (!aligned_to(g.want, 4)) return fail(SOL_EINVAL, "gradients of vectors must be 4-byte aligned");
    any = any || g.want != nullptr;
  }
  if (!aligned_to(dshift, 4)) return fail(SOL_EINVAL, "gradients of vectors must be 4-byte aligned");
  if (B > 65535) return fail(SOL_EUNSUPPORTED, "B must be <= 65535");
  const size_t need = sol_attn_residual_norm_bwd_workspace_bytes(B, T, C);
  if (any && (workspace == nullptr || ws_bytes < need))
    return fail(SOL_EINVAL, "workspace too small (%zu < %zu bytes)", workspace == nullptr ? size_t(0) : ws_bytes, need);
  int sms = 0;
  if ((st = current_device(&sms)) != SOL_OK) return st;
  a.dh = dh;
  a.dx_out = dx_out;
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.dscale = dscale;
  a.dshift = dshift;
  a.dgain = dgain;
  a.dpost_gain = dpost_gain;
  a.part = any ? static_cast<float*>(workspace) : nullptr;
  a.C = C;
  a.chunks = sol::norm_bwd_chunks(B, T, C);
  const cudaError_t e = sol::launch_residual_norm_bwd(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "residual norm gradient launch");
  return SOL_OK;
}

sol_status sol_attn_rope_inv_freq(int rot, double base, int axes, const int* sections, sol_rope_scaling scaling,
                                  double factor, double original_length, double turns_low, double turns_high,
                                  double* inv_freq, float* attn_factor) {
  clear_error();
  int end[4];
  const sol_status st = rope_sections(rot, axes, sections, end);
  if (st != SOL_OK) return st;
  if (inv_freq == nullptr || attn_factor == nullptr) return fail(SOL_EINVAL, "inv_freq and attn_factor must be non-null");
  if (!(base > 1.0) || std::isinf(base)) return fail(SOL_EINVAL, "base=%g must be finite and above 1", base);
  if (scaling < SOL_ROPE_PLAIN || scaling > SOL_ROPE_YARN) return fail(SOL_EINVAL, "unknown scaling %d", static_cast<int>(scaling));
  if (scaling != SOL_ROPE_PLAIN && (!(factor >= 1.0) || std::isinf(factor)))
    return fail(SOL_EINVAL, "factor=%g must be finite and at least 1", factor);
  if (scaling == SOL_ROPE_YARN && (!(original_length > 0.0) || std::isinf(original_length) || !(turns_low < turns_high) ||
                                   !(turns_low >= 0.0) || std::isinf(turns_high)))
    return fail(SOL_EINVAL, "yarn needs original_length > 0 and 0 <= turns_low < turns_high");
  int at = 0;
  for (int a = 0; a < axes; ++a) {
    const int n = sections != nullptr ? sections[a] : rot / 2;
    double b = base;
    // a section of one pair has frequency 1 whatever the base
    if (scaling == SOL_ROPE_NTK && n > 1) b = base * std::pow(factor, static_cast<double>(n) / (n - 1));
    for (int j = 0; j < n; ++j) {
      double f = std::pow(b, -static_cast<double>(j) / n);
      if (scaling == SOL_ROPE_LINEAR) f /= factor;
      if (scaling == SOL_ROPE_YARN) {
        const double turns = original_length * f / 6.283185307179586476925;
        double keep = (turns - turns_low) / (turns_high - turns_low);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        f = f * keep + f / factor * (1.0 - keep);
      }
      inv_freq[at++] = f;
    }
  }
  *attn_factor = scaling == SOL_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  return SOL_OK;
}

sol_status sol_attn_rope_tables(const int32_t* pos, int axes, const int* sections, const double* inv_freq,
                                float attn_factor, int L, int rot, float* rope_cos, float* rope_sin, void* stream) {
  clear_error();
  sol::RopeTableArgs a;
  if (!size_ok(L, 1 << 28) || !size_ok(rot, 1 << 16)) return fail(SOL_EINVAL, "sizes must be positive (L=%d rot=%d)", L, rot);
  sol_status st = rope_sections(rot, axes, sections, a.end);
  if (st != SOL_OK) return st;
  if (!std::isfinite(attn_factor)) return fail(SOL_EINVAL, "attn_factor=%g must be finite", attn_factor);
  if (pos == nullptr || inv_freq == nullptr || rope_cos == nullptr || rope_sin == nullptr)
    return fail(SOL_EINVAL, "pos, inv_freq, rope_cos and rope_sin must be non-null");
  if (!aligned_to(pos, 4) || !aligned_to(inv_freq, 8) || !aligned_to(rope_cos, 4) || !aligned_to(rope_sin, 4))
    return fail(SOL_EINVAL, "device pointers must be aligned to their elements");
  int sms = 0;
  if ((st = current_device(&sms)) != SOL_OK) return st;
  a.pos = pos;
  a.inv_freq = inv_freq;
  a.L = L;
  a.rot = rot;
  a.axes = axes;
  a.factor = attn_factor;
  a.cos = rope_cos;
  a.sin = rope_sin;
  const cudaError_t e = sol::launch_rope_tables(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rotary table launch");
  return SOL_OK;
}

sol_status sol_attn_rope(const void* Q, const int64_t* q_strides, const void* K, const int64_t* k_strides, sol_dtype dt,
                         const int32_t* pos, int64_t pos_stride_b, int axes, const int* sections, const double* inv_freq,
                         float attn_factor, sol_rope_layout layout, int inverse, int B, int Hq, int Hk, int L, int d,
                         int rot, void* Q_out, const int64_t* q_out_strides, void* K_out, const int64_t* k_out_strides,
                         void* stream) {
  clear_error();
  if (dt != SOL_F32 && dt != SOL_BF16) return fail(SOL_EINVAL, "unknown dtype %d", static_cast<int>(dt));
  if (!size_ok(B, 1 << 28) || !size_ok(Hq, 1 << 28) || Hk < 0 || Hk > (1 << 28) || !size_ok(L, 1 << 28) || !size_ok(d, 1 << 28))
    return fail(SOL_EINVAL, "sizes must be positive (B=%d Hq=%d Hk=%d L=%d d=%d)", B, Hq, Hk, L, d);
  sol::RopeArgs a;
  sol_status st = rope_sections(rot, axes, sections, a.end);
  if (st != SOL_OK) return st;
  if (rot > d) return fail(SOL_EINVAL, "rot=%d must be at most d=%d", rot, d);
  if (layout != SOL_ROPE_INTERLEAVED && layout != SOL_ROPE_HALF) return fail(SOL_EINVAL, "unknown layout %d", static_cast<int>(layout));
  if (!std::isfinite(attn_factor)) return fail(SOL_EINVAL, "attn_factor=%g must be finite", attn_factor);
  if (Q == nullptr || Q_out == nullptr || q_strides == nullptr || q_out_strides == nullptr || pos == nullptr || inv_freq == nullptr)
    return fail(SOL_EINVAL, "Q, Q_out, their strides, pos and inv_freq must be non-null");
  if (Hk > 0 && (K == nullptr || K_out == nullptr || k_strides == nullptr || k_out_strides == nullptr))
    return fail(SOL_EINVAL, "K, K_out and their strides must be non-null for Hk > 0");
  const size_t es = dt == SOL_BF16 ? 2 : 4;
  if (!aligned_to(Q, es) || !aligned_to(Q_out, es) || (Hk > 0 && (!aligned_to(K, es) || !aligned_to(K_out, es))) ||
      !aligned_to(pos, 4) || !aligned_to(inv_freq, 8))
    return fail(SOL_EINVAL, "device pointers must be aligned to their elements");
  if (d > 512 || d % 2 != 0) return fail(SOL_EUNSUPPORTED, "rotary positions need an even d <= 512 (d=%d)", d);
  if (B > 65535 || static_cast<long long>(Hq) + Hk > 65535) return fail(SOL_EUNSUPPORTED, "B and Hq + Hk must be <= 65535");
  const int V = dt == SOL_BF16 ? 8 : 4;
  a.vec = layout == SOL_ROPE_HALF ? (rot / 2) % V == 0 && d % V == 0 : d % V == 0;
  a.copy_rest = false;
  for (int i = 0; i < 2; ++i) {
    sol::RopeSide& r = a.side[i];
    const int64_t* in = i == 0 ? q_strides : k_strides;
    const int64_t* out = i == 0 ? q_out_strides : k_out_strides;
    r.in = i == 0 ? Q : K;
    r.out = i == 0 ? Q_out : K_out;
    r.heads = i == 0 ? Hq : Hk;
    r.in_b = r.in_h = r.in_l = r.out_b = r.out_h = r.out_l = 0;
    if (r.heads == 0) continue;
    // a size of one has no stride
    const int sizes[3] = {B, r.heads, L};
    long long* dst[2][3] = {{&r.in_b, &r.in_h, &r.in_l}, {&r.out_b, &r.out_h, &r.out_l}};
    bool same = r.in == r.out;
    for (int k = 0; k < 3; ++k) {
      if (sizes[k] == 1) continue;
      if (in[k] < 0 || out[k] < d) return fail(SOL_EINVAL, "input strides must not be negative, output strides at least d");
      *dst[0][k] = in[k];
      *dst[1][k] = out[k];
      if (in[k] != out[k]) same = false;
      if (in[k] % V != 0 || out[k] % V != 0) a.vec = false;
    }
    if (r.in == r.out && !same) return fail(SOL_EINVAL, "in place, input and output must have the same strides");
    if (!same) a.copy_rest = true;
    if (!aligned16(r.in) || !aligned16(r.out)) a.vec = false;
  }
  int sms = 0;
  if ((st = current_device(&sms)) != SOL_OK) return st;
  a.pos = pos;
  a.pos_b = B > 1 ? pos_stride_b : 0;
  a.inv_freq = inv_freq;
  a.B = B;
  a.L = L;
  a.d = d;
  a.rot = rot;
  a.axes = axes;
  a.factor = attn_factor;
  a.half = layout == SOL_ROPE_HALF;
  a.inverse = inverse != 0;
  a.bf16 = dt == SOL_BF16;
  const cudaError_t e = sol::launch_rope(a, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rotary launch");
  return SOL_OK;
}

}  // extern "C"
