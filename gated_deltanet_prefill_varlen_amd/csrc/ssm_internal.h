// Internal interface between the C-ABI host layer and the launchers of the
// state space layers' kernels and the norm around them.  Every struct here is
// filled only after the host layer validated the call.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

// What a layer keeps: its geometry and constants.
struct SsmLayer {
  int32_t H, G, P, N;      // heads, groups of B and C, channels of a head, state columns
  int32_t conv_dim;        // H P + 2 G N: channels [x | B | C]
  int32_t softplus;        // the raw steps go through softplus
  int32_t dt_f32;          // raw steps are fp32 (else bf16)
  float dt_min, dt_max;
  const float* A;          // [H]
  const float* dt_bias;    // [H] or nullptr
  const float* D;          // [H] or nullptr
  const float* conv_w;     // [conv_dim, 4] or nullptr (rows are convolved already)
  const float* conv_bias;  // [conv_dim] or nullptr
};

struct SsmScanArgs {
  SsmLayer l;
  const int32_t* cu;       // device [n_seqs + 1]
  int32_t n_seqs, n_tokens;
  const uint16_t* x;       // [T, conv_dim] bf16, token stride x_stride
  const void* dt;          // [T, H], token stride dt_stride
  int64_t x_stride, dt_stride;
  const float* init;       // [n_seqs, H, P, N] or nullptr
  const int32_t* ckpt;     // [n_ckpt]
  int32_t n_ckpt;
  uint16_t* out;           // [T, H, P]
  float* final_state;      // or nullptr
  float* ckpt_buf;
  const uint16_t* conv_in; // [n_seqs, 3, conv_dim] or nullptr (zeros)
  uint16_t* conv_out;      // or nullptr; may equal conv_in
  uint16_t* conv_ckpt;     // [n_ckpt, 3, conv_dim] or nullptr
};

struct SsmDecodeArgs {
  SsmLayer l;
  int32_t batch, n_tok;
  const uint16_t* x;       // [batch * n_tok, conv_dim]
  const void* dt;
  int64_t x_stride, dt_stride;
  float* state;            // [pool, H, P, N]
  const int32_t* slot;     // [batch] or nullptr
  uint16_t* out;           // [batch * n_tok, H, P]
  float* snap;             // [batch, n_tok, H, P, N] or nullptr
  uint16_t* conv_state;    // [pool, 3, conv_dim], with l.conv_w
};

struct NormArgs {
  int32_t dim, groups, group_dim, scale_block;
  int32_t n_rows;
  int32_t x_f32, res_f32, gate_first, codes_i8;
  float eps, weight_offset;
  int32_t weight_dim;
  const void* x;
  const void* res;         // or nullptr
  const void* gate;        // or nullptr
  int64_t x_stride, res_stride, gate_stride;
  const float* w;          // [weight_dim] or nullptr (ones)
  void* out;               // [n_rows, dim] of x's type, or nullptr
  void* res_out;           // of the residual's type and stride, or nullptr
  uint8_t* codes;          // [n_rows, dim] or nullptr
  float* scales;           // [n_rows, dim / scale_block or 1]
};

hipError_t launch_ssm_scan(const SsmScanArgs& a, const int32_t* cu_host, const int32_t* ckpt_host, void* workspace,
                           hipStream_t stream);
int64_t ssm_scan_bytes(const SsmLayer& l, int32_t n_seqs, const int32_t* cu_host);
int64_t ssm_scan_groups(const SsmLayer& l, int32_t n_seqs, int64_t n_tokens);   // workgroups of its largest launch, at most
hipError_t launch_ssm_decode(const SsmDecodeArgs& a, hipStream_t stream);
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream);

}  // namespace gdn
