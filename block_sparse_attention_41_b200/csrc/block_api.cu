// C ABI of the dense operators around the attention (declared in include/sol_attn.h): gated
// residual and norm, rotary positions, linear layer. Arguments are checked on the host before anything is
// launched; nothing here allocates device memory.
#include <algorithm>
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

// Do the rows of d values of an output lie apart? Strides of sizes above one have to nest: from the shortest on,
// each is at least as long as everything within it.
bool rows_apart(const int (&sizes)[3], const int64_t* strides, int d) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int i, int j) { return strides[i] < strides[j]; });
  __int128 extent = d;
  for (int i : order) {
    if (sizes[i] == 1) continue;
    if (strides[i] < extent) return false;
    extent += static_cast<__int128>(strides[i]) * (sizes[i] - 1);
  }
  return true;
}

// Is one of the outputs given twice, or also as one of the inputs that other blocks still read? (Null: not there.
// The starts are compared: the same buffer given twice is what happens by mistake.)
template <size_t O, size_t I>
bool shares(const void* const (&outs)[O], const void* const (&ins)[I]) {
  for (size_t i = 0; i < O; ++i) {
    if (outs[i] == nullptr) continue;
    for (size_t j = 0; j < i; ++j)
      if (outs[i] == outs[j]) return true;
    for (const void* in : ins)
      if (outs[i] == in) return true;
  }
  return false;
}

// 2-D bf16 view [rows][inner] with boxes of box_inner x box_rows; what lies outside reads as zero and
// is not written.
sol_status make_map2d(CUtensorMap* m, const void* base, int inner, int rows, int box_inner, int box_rows,
                      CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return fail(SOL_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(inner) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SOL_ECUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
  return SOL_OK;
}

// An operand of a product with `rows` rows and `inner` columns in memory: K-major tiles of tile_rows
// rows x 64, or MN-major boxes of 64 x 64.
sol_status make_operand_map(CUtensorMap* m, const void* base, int rows, int inner, bool mn, int tile_rows) {
  return make_map2d(m, base, inner, rows, 64, mn ? 64 : tile_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// out [Mo, No] = A . B over Ko. A lies in memory as [Mo, Ko] or, a_mn, as
// [Ko, Mo]; B as [No, Ko] or, b_mn, as [Ko, No].
sol_status run_gemm(sol::GemmArgs& a, const void* A, const void* Bm, void* out, void* z, cudaStream_t stream) {
  a.tile = sol::linear_tile(a.Mo, a.No, a.Ko, a.part != nullptr, a.num_sms);
  a.out = out;
  a.z = z;
  sol_status st;
  if ((st = make_operand_map(&a.maps[0], A, a.a_mn ? a.Ko : a.Mo, a.a_mn ? a.Mo : a.Ko, a.a_mn, 128)) != SOL_OK) return st;
  if ((st = make_operand_map(&a.maps[1], Bm, a.b_mn ? a.Ko : a.No, a.b_mn ? a.No : a.Ko, a.b_mn, a.tile.n / a.tile.ctas)) != SOL_OK) return st;
  if ((st = make_map2d(&a.maps[2], out, a.No, a.Mo, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)) != SOL_OK) return st;
  a.maps[3] = a.maps[4] = a.maps[2];
  if (z != nullptr && (st = make_map2d(&a.maps[3], z, a.No, a.Mo, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)) != SOL_OK) return st;
  if (a.residual != nullptr &&
      (st = make_map2d(&a.maps[4], a.residual, a.No, a.Mo, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)) != SOL_OK)
    return st;
  a.drop = take_drop(true, &a.wait_limit_ns);
  const cudaError_t e = sol::launch_linear_gemm(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "linear layer launch");
  return SOL_OK;
}

sol_status linear_sizes(int M, int N, int K, sol_activation act) {
  if (act < SOL_ACT_NONE || act > SOL_ACT_SILU) return fail(SOL_EINVAL, "unknown activation %d", static_cast<int>(act));
  if (!size_ok(M, 1 << 28) || !size_ok(N, 1 << 28) || !size_ok(K, 1 << 28))
    return fail(SOL_EINVAL, "sizes must be positive (M=%d N=%d K=%d)", M, N, K);
  if (N % 8 != 0 || K % 8 != 0) return fail(SOL_EUNSUPPORTED, "the linear layer needs N and K in multiples of 8 (N=%d K=%d)", N, K);
  const long long m = (M + 127) / 128, n = (N + 63) / 64, k = (K + 63) / 64;
  if (m * n >= (1ll << 31) || ((M + 63ll) / 64) * k >= (1ll << 31) || n * k >= (1ll << 31))
    return fail(SOL_EUNSUPPORTED, "too many tiles (M=%d N=%d K=%d)", M, N, K);
  return SOL_OK;
}

constexpr int kMaxSms = 148;  // of a B200: the workspace's size is asked for without a device
constexpr size_t kErrorBytes = 256;  // the workspace's error words, as sol_attn_check_device_error reads them
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

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
  if (x_out == h) return fail(SOL_EINVAL, "x_out and h must be two buffers");
  if (!aligned16(h) || !aligned16(x_out)) return fail(SOL_EINVAL, "x_out and h must be 16-byte aligned");
  int sms = 0;
  if ((st = current_device(&sms)) != SOL_OK) return st;
  a.x_out = x_out;
  a.h = h;
  const cudaError_t e = sol::launch_residual_norm(a, sms, static_cast<cudaStream_t>(stream));
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
  if (dx == dy) return fail(SOL_EINVAL, "dx and dy must be two buffers");
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
  a.chunks = sol::norm_bwd_chunks(B, T, C, a.fwd.vec);
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
  a.factor = attn_factor;
  a.cos = rope_cos;
  a.sin = rope_sin;
  const cudaError_t e = sol::launch_rope_tables(a, sms, static_cast<cudaStream_t>(stream));
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
  if (Hk > 0 && (Q_out == K_out || Q_out == K || K_out == Q))
    return fail(SOL_EINVAL, "an output must be neither the other side's input nor its output");
  const size_t es = dt == SOL_BF16 ? 2 : 4;
  if (!aligned_to(Q, es) || !aligned_to(Q_out, es) || (Hk > 0 && (!aligned_to(K, es) || !aligned_to(K_out, es))) ||
      !aligned_to(pos, 4) || !aligned_to(inv_freq, 8))
    return fail(SOL_EINVAL, "device pointers must be aligned to their elements");
  if (d > 512 || d % 2 != 0) return fail(SOL_EUNSUPPORTED, "rotary positions need an even d <= 512 (d=%d)", d);
  if (B > 1 && pos_stride_b < 0) return fail(SOL_EINVAL, "pos_stride_b=%lld must not be negative", static_cast<long long>(pos_stride_b));
  if (B > 65535 || static_cast<long long>(Hq) + Hk > 65535) return fail(SOL_EUNSUPPORTED, "B and Hq + Hk must be <= 65535");
  const int esize = dt == SOL_BF16 ? 2 : 4;
  a.width = 16 / esize;
  auto narrow_to = [&a](long long n) {
    while (n % a.width != 0) a.width /= 2;
  };
  narrow_to(d);
  narrow_to(layout == SOL_ROPE_HALF ? rot / 2 : rot);
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
      narrow_to(in[k]);
      narrow_to(out[k]);
    }
    if (!rows_apart(sizes, out, d)) return fail(SOL_EINVAL, "rows of an output overlap: strides must nest");
    if (r.in == r.out && !same) return fail(SOL_EINVAL, "in place, input and output must have the same strides");
    if (!same) a.copy_rest = true;
    narrow_to(static_cast<long long>(reinterpret_cast<uintptr_t>(r.in) % 16) / esize);
    narrow_to(static_cast<long long>(reinterpret_cast<uintptr_t>(r.out) % 16) / esize);
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
  a.factor = attn_factor;
  a.half = layout == SOL_ROPE_HALF;
  a.inverse = inverse != 0;
  a.bf16 = dt == SOL_BF16;
  const cudaError_t e = sol::launch_rope(a, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rotary launch");
  return SOL_OK;
}

size_t sol_attn_linear_workspace_bytes(int M, int N, int K) {
  if (linear_sizes(M, N, K, SOL_ACT_NONE) != SOL_OK) {
    clear_error();
    return 0;
  }
  const bool split = M > sol::kFewRows && sol::linear_tile(M, N, K, true, kMaxSms).split > 1;
  return kErrorBytes + (split ? sol::linear_part_bytes(kMaxSms) : 0);
}

sol_status sol_attn_linear(const void* x, const void* w, const float* bias, const void* residual, sol_activation act, int M,
                           int N, int K, void* out, void* z, void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  sol_status st = linear_sizes(M, N, K, act);
  if (st != SOL_OK) return st;
  if (x == nullptr || w == nullptr || out == nullptr) return fail(SOL_EINVAL, "x, w and out must be non-null");
  const void* const outs[] = {out, z};
  const void* const ins[] = {x, w, workspace};
  if (shares(outs, ins) || (z != nullptr && z == residual))
    return fail(SOL_EINVAL, "out and z must be two buffers, neither of them x, w or the workspace, nor z the residual");
  const void* ptrs[] = {x, w, bias, residual, out, z, workspace};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return fail(SOL_EINVAL, "device pointers must be 16-byte aligned");
  if (workspace != nullptr && ws_bytes < kErrorBytes) return fail(SOL_EINVAL, "workspace too small (%zu < %zu bytes)", ws_bytes, kErrorBytes);
  int sms = 0;
  if ((st = current_device(&sms)) != SOL_OK) return st;
  if (M <= sol::kFewRows) {
    sol::FewArgs a;
    if ((st = make_operand_map(&a.maps[0], w, N, K, false, 128)) != SOL_OK) return st;
    if ((st = make_operand_map(&a.maps[1], x, M, K, false, sol::linear_few_tile(M))) != SOL_OK) return st;
    a.M = M;
    a.N = N;
    a.K = K;
    a.bias = bias;
    a.residual = residual;
    a.out = out;
    a.z = z;
    a.act = act;
    a.ws = static_cast<uint32_t*>(workspace);
    a.num_sms = sms;
    a.drop = take_drop(true, &a.wait_limit_ns);
    const cudaError_t e = sol::launch_linear_few(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "linear layer launch");
    return SOL_OK;
  }
  sol::GemmArgs a;
  a.Mo = M;
  a.No = N;
  a.Ko = K;
  a.a_mn = a.b_mn = false;
  a.bias = bias;
  a.residual = residual;
  a.act = act;
  a.part = workspace != nullptr && ws_bytes >= kErrorBytes + sol::linear_part_bytes(kMaxSms) && sms <= kMaxSms
               ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kErrorBytes)
               : nullptr;
  a.ws = static_cast<uint32_t*>(workspace);
  a.num_sms = sms;
  return run_gemm(a, x, w, out, z, static_cast<cudaStream_t>(stream));
}

size_t sol_attn_linear_bwd_workspace_bytes(int M, int N, sol_activation act) {
  if (!size_ok(M, 1 << 28) || !size_ok(N, 1 << 28) || act < SOL_ACT_NONE || act > SOL_ACT_SILU) return 0;
  return kErrorBytes + sol::linear_part_bytes(kMaxSms) + round256(static_cast<size_t>(sol::linear_dz_chunks(M, N)) * N * 4) +
         (act == SOL_ACT_NONE ? 0 : round256(static_cast<size_t>(M) * N * 2));
}

sol_status sol_attn_linear_bwd(const void* dy, const void* x, const void* w, const void* z, sol_activation act, int M, int N,
                               int K, void* dx, void* dw, float* db, void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  sol_status st = linear_sizes(M, N, K, act);
  if (st != SOL_OK) return st;
  if (dy == nullptr || workspace == nullptr) return fail(SOL_EINVAL, "dy and workspace must be non-null");
  if (dx == nullptr && dw == nullptr && db == nullptr) return fail(SOL_EINVAL, "no gradient is wanted: dx, dw and db are all null");
  if (dx != nullptr && w == nullptr) return fail(SOL_EINVAL, "dx needs w");
  if (dw != nullptr && x == nullptr) return fail(SOL_EINVAL, "dw needs x");
  if ((act != SOL_ACT_NONE) != (z != nullptr)) return fail(SOL_EINVAL, "z must be given exactly where there is an activation");
  const void* const outs[] = {dx, dw, db};
  const void* const ins[] = {dy, x, w, z, workspace};
  if (shares(outs, ins)) return fail(SOL_EINVAL, "dx, dw and db must be buffers of their own");
  const void* ptrs[] = {dy, x, w, z, dx, dw, workspace};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return fail(SOL_EINVAL, "device pointers must be 16-byte aligned");
  if (!aligned_to(db, 4)) return fail(SOL_EINVAL, "db must be 4-byte aligned");
  const size_t need = sol_attn_linear_bwd_workspace_bytes(M, N, act);
  if (ws_bytes < need) return fail(SOL_EINVAL, "workspace too small (%zu < %zu bytes)", ws_bytes, need);
  int sms = 0;
  if ((st = current_device(&sms)) != SOL_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* at = static_cast<uint8_t*>(workspace) + kErrorBytes;
  float* pieces = reinterpret_cast<float*>(at);
  at += sol::linear_part_bytes(kMaxSms);
  float* part = reinterpret_cast<float*>(at);
  void* dz = at + round256(static_cast<size_t>(sol::linear_dz_chunks(M, N)) * N * 4);
  if (act != SOL_ACT_NONE || db != nullptr) {
    const cudaError_t e = sol::launch_linear_dz(dy, z, act, M, N, dz, db != nullptr ? part : nullptr, db, s);
    if (e != cudaSuccess) return cuda_fail(e, "activation gradient launch");
  }
  const void* g = act != SOL_ACT_NONE ? dz : dy;
  sol::GemmArgs a;
  a.bias = nullptr;
  a.residual = nullptr;
  a.act = sol::ACT_NONE;
  a.part = sms <= kMaxSms ? pieces : nullptr;
  a.ws = static_cast<uint32_t*>(workspace);
  a.num_sms = sms;
  if (dx != nullptr) {
    a.Mo = M;
    a.No = K;
    a.Ko = N;
    a.a_mn = false;
    a.b_mn = true;
    if ((st = run_gemm(a, g, w, dx, nullptr, s)) != SOL_OK) return st;
  }
  if (dw != nullptr) {
    a.Mo = N;
    a.No = K;
    a.Ko = M;
    a.a_mn = a.b_mn = true;
    if ((st = run_gemm(a, g, x, dw, nullptr, s)) != SOL_OK) return st;
  }
  return SOL_OK;
}

}  // extern "C"
