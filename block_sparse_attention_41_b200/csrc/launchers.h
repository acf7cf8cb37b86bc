// Internal launcher interface between the C ABI (sol_attn_api.cu) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace sol {

// 8-bit QK^T operands of the forward (sol_attn_quantize_qk8): codes and per-tile scales
struct Qk8Operands {
  const int8_t* q8;        // [BH, L, d]
  const int8_t* k8;        // [BH, L, d], K - mu
  const int8_t* kb8;       // [BH, N_kb, d], k_bar - mu
  const float* q_scale;    // [BH, N_qb]
  const float* k_scale;    // [BH, N_kb]
  const float* kb_scale;   // [BH, ceil(N_kb / 128)]
};

// 8-bit PV operands of the forward (sol_attn_quantize_v8): E4M3 codes, transposed, and channel scales
struct Pv8Operands {
  const uint8_t* v8t;      // [BH, d, N_kb * 128]
  const uint8_t* vb8t;     // [BH, d, 128 * ceil(N_kb / 128)]
  const float* v_scale;    // [BH, d]
};

struct FwdArgs {
  const void* Q;
  const void* K;
  const void* V;
  const float* kbar;
  const float* vbar;
  const void* kbar_lp;
  const void* vbar_lp;
  const float* tau;  // host [H]
  bool bf16;
  int B, H, L, d, block;
  int n_force;
  void* O;
  uint8_t* kept_mask;
  float* density;
  uint32_t* ws;
  int num_sms;
  int drop_one_load;       // failure-detection test hook (bf16 path)
  uint32_t* route_bits;    // bf16 path: [B*H, N_qb, ceil(N_kb/32)] keep bits from launch_route, or null
                           // (the fused kernel then routes each unit itself)
  float* route_qbar;       // with route_bits: [B*H, N_qb, d] fp32 query-block means (workspace)
  uint64_t wait_limit_ns;  // bound on every on-device wait
  int k_keep = 0;          // routing pass: 0 = threshold max - tau; k > 0 = the k highest scores
  unsigned long long* cta_times = nullptr;  // measurement hook: [2 * cta_capacity] start/finish ns
  int cta_capacity = 0;
  const Qk8Operands* qk8 = nullptr;  // bf16 path: int8 Q, K and pooled keys for QK^T, or null
  const Pv8Operands* pv8 = nullptr;  // with qk8: E4M3 V and v_bar for PV (kind::f8f6f4), or null
  const float* qbar_in = nullptr;    // routing pass: fp32 [B*H, N_qb, d] query-block means given by the
                                     // caller (the QK-norm + RoPE pass); null = computed from Q
};

cudaError_t launch_pool(const void* K, const void* V, bool bf16, int BH, int L, int d, int block,
                        float* kbar, float* vbar, void* kbar_lp, void* vbar_lp, cudaStream_t stream);

struct RopePoolArgs {
  const void* Q;  // bf16 [BH, L, d]
  const void* K;
  const void* V;
  const float* gain_q;  // [d]
  const float* gain_k;  // [d]
  const float* cos;     // [L, d/2]
  const float* sin;     // [L, d/2]
  float eps;
  void* Qout;  // bf16 [BH, L, d]
  void* Kout;
  float* kbar;  // fp32 [BH, N_kb, d]
  float* vbar;
  void* kbar_lp;  // bf16 [BH, N_kb, d]
  void* vbar_lp;
  float* qbar = nullptr;  // out, optional: fp32 [BH, N_kb, d] means of the stored query rows per block
  int BH, L, d, block;
};

struct QuantArgs {
  const void* Q;       // bf16 [BH, L, d]
  const void* K;       // bf16 [BH, L, d]
  const float* kbar;   // fp32 [BH, N_kb, d] from the pooling pass
  float* mu;           // out: fp32 [BH, d] mean key
  int8_t* q8;          // out: int8 [BH, L, d]
  int8_t* k8;          // out: int8 [BH, L, d] codes of K - mu
  int8_t* kb8;         // out: int8 [BH, N_kb, d] codes of k_bar - mu
  float* q_scale;      // out: [BH, N_qb]
  float* k_scale;      // out: [BH, N_kb]
  float* kb_scale;     // out: [BH, ceil(N_kb / 128)]
  int BH, L, d;
};

// bf16, d in {64, 128}, blocks of 128: the mean key, then int8 codes and tile scales of Q, K - mu
// and k_bar - mu.
cudaError_t launch_quant_qk8(const QuantArgs& a, cudaStream_t stream);

// 8-bit PV values (d = 128): per-channel scales of V and the transposed E4M3 codes of V and v_bar.
struct QuantV8Args {
  const void* V;        // bf16 [BH, L, d]
  const float* vbar;    // fp32 [BH, N_kb, d] from the pooling pass
  uint8_t* v8t;         // out: E4M3 [BH, d, N_kb * 128], keys contiguous, zero past L
  uint8_t* vb8t;        // out: E4M3 [BH, d, 128 * ceil(N_kb / 128)], zero past N_kb
  float* v_scale;       // out: fp32 [BH, d] (also the amax accumulator while the pass runs)
  int BH, L, d;
};
cudaError_t launch_quant_v8(const QuantV8Args& a, cudaStream_t stream);

// bf16, d in {64, 128}: QK RMS norm + rotary embedding + K/V block pooling in one pass.
cudaError_t launch_qknorm_rope_pool(const RopePoolArgs& a, cudaStream_t stream);

// Gated residual and norm (sol_attn_residual_norm); null vectors are absent.
enum : int { NORM_NONE = 0, NORM_LAYER = 1, NORM_RMS = 2 };
constexpr int kNormMaxC = 8192;
struct NormArgs {
  const void* x;  // [B, T, C]
  const void* y;  // [B, T, C] or null: no residual step, x is normalised as it is
  const float* gate;  // rows of C, one per batch entry, gate_stride floats apart
  long long gate_stride;
  const float* gain;  // [C]
  const float* scale;
  long long scale_stride;
  const float* shift;
  long long shift_stride;
  const float* post_gain;  // [C]
  void* x_out;  // with y: [B, T, C]
  void* h;      // [B, T, C]
  int B, T, C;
  int norm, post_norm;
  float res_scale, eps;
  bool bf16;
  bool vec;  // rows and vectors allow 16-byte accesses
};
cudaError_t launch_residual_norm(const NormArgs& a, int num_sms, cudaStream_t stream);

// Its gradients. fwd.x_out, fwd.h and fwd.shift are not read.
struct NormBwdArgs {
  NormArgs fwd;
  const void* dh;      // [B, T, C]
  const void* dx_out;  // [B, T, C] or null
  void* dx;            // [B, T, C]
  void* dy;            // with y: [B, T, C]
  float* dgate;        // [B, C] or null, as the next two
  float* dscale;
  float* dshift;
  float* dgain;        // [C] or null
  float* dpost_gain;   // [C] or null
  float* part;         // workspace of norm_bwd_part_floats, or null where no vector's gradient is wanted
  int C, chunks;       // chunks = norm_bwd_chunks(B, T, C, fwd.vec)
};
constexpr int kNormBwdBlocks = 592;  // 4 per SM, of which 1 to 3 are taken over all batch entries
int norm_bwd_chunks(int B, int T, int C, bool vec);
size_t norm_bwd_part_floats(int B, int T, int C);
cudaError_t launch_residual_norm_bwd(const NormBwdArgs& a, cudaStream_t stream);

// Rotary positions (sol_attn_rope): rows of Q and K, each [B, heads, L, d] with its own strides.
struct RopeSide {
  const void* in;
  void* out;
  int heads;
  long long in_b, in_h, in_l;     // strides in elements; the d channels are contiguous
  long long out_b, out_h, out_l;
};
struct RopeArgs {
  RopeSide side[2];
  const int* pos;        // [axes, L], pos_b apart per batch entry
  long long pos_b;
  const double* inv_freq;  // [rot / 2]
  int B, L, d, rot;
  int end[4];            // pairs [end[a - 1], end[a]) turn by axis a
  float factor;
  bool half, inverse, bf16;
  int width;             // values per access: it divides every length, stride and address
  bool copy_rest;        // channels [rot, d) have to be written too
};
cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream);
struct RopeTableArgs {
  const int* pos;  // [axes, L]
  const double* inv_freq;
  int L, rot;
  int end[4];
  float factor;
  float* cos;  // [L, rot / 2]
  float* sin;
};
cudaError_t launch_rope_tables(const RopeTableArgs& a, int num_sms, cudaStream_t stream);

// Linear layer (sol_attn_linear) and its gradients: bf16 operands, fp32 accumulation.
// The copy that a launch leaves out (sol_attn_debug_drop_one_load): one of the attention, of the second operand's
// in the launch's first or second CTA, or of the residual's.
enum : int { DROP_ATTENTION = 1, DROP_OPERAND = 2, DROP_OPERAND_SECOND = 3, DROP_RESIDUAL = 4 };
enum : int { ACT_NONE = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_SILU = 3 };
constexpr int kFewRows = 128;  // up to here the forward takes the kernel for few rows
constexpr int kDzBlocks = 1184;  // blocks of the dz pass: 8 per SM
struct GemmTile {
  int ctas, n;  // a tile is 128 ctas x n outputs on a pair of SMs or one
  int split;    // pieces of the reduction of the last tiles, those past the last whole turn of the SMs
};
GemmTile linear_tile(int Mo, int No, int Ko, bool splittable, int num_sms);
size_t linear_part_bytes(int num_sms);           // accumulators of one tile per SM
int linear_few_tile(int M);                      // tokens per tile of the kernel for few rows
int linear_dz_chunks(int M, int N);              // row blocks of the dz pass, one partial column sum each
struct GemmArgs {
  CUtensorMap maps[5];  // A, B (boxes as launch_linear_gemm's tiles want them), out, z, residual
  int Mo, No, Ko;       // output rows, columns, reduction
  bool a_mn, b_mn;      // operand is MN-major: its memory rows run along M or N
  GemmTile tile;
  const float* bias;    // [No] or null
  const void* residual; // bf16 [Mo, No] or null
  int act;
  void* out;
  void* z;              // or null
  float* part;          // linear_part_bytes for the pieces of the last tiles, or null: none are split
  int drop;             // failure-detection test hook, as the limit of a device wait
  uint64_t wait_limit_ns;
  uint32_t* ws;         // error words or null
  int num_sms;
};
cudaError_t launch_linear_gemm(const GemmArgs& a, cudaStream_t stream);
struct FewArgs {
  CUtensorMap maps[2];  // w, x
  int M, N, K;
  const float* bias;
  const void* residual;
  void* out;
  void* z;  // or null
  int act;
  int drop;
  uint64_t wait_limit_ns;
  uint32_t* ws;
  int num_sms;
};
cudaError_t launch_linear_few(const FewArgs& a, cudaStream_t stream);
// dz = dy act'(z) (z null: dz = dy, not written) and, with part and db, the column sums of dz.
cudaError_t launch_linear_dz(const void* dy, const void* z, int act, int M, int N, void* dz, float* part, float* db,
                             cudaStream_t stream);

// bf16, d in {64, 128}, block 128: routing pass for every unit (q_bar kernel, then the routing
// kernel); writes a.route_qbar, a.route_bits, the optional mask and the per-head kept counts
// (ws + WS_COUNTS).
cudaError_t launch_route(const FwdArgs& a, cudaStream_t stream);

// bf16, d in {64, 128}, block 128: TMA + tcgen05 persistent kernel.
cudaError_t launch_fwd_tc(const FwdArgs& a, const CUtensorMap* maps /* Q, K, V, Kbar_lp, Vbar_lp */,
                          cudaStream_t stream);

// fp32, d in {32, 64, 128}, block in {32, 64, 128}: SIMT kernel.
cudaError_t launch_fwd_simt(const FwdArgs& a, cudaStream_t stream);

}  // namespace sol
