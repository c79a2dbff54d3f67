// Packed scan of the state space layers, token by token: a workgroup owns 32
// rows of one (prompt, head), as the decode step does.
#include <climits>

#include "ssm_device.h"

namespace gdn {
namespace {

constexpr int kRows = 32;

// Input of channel c at position p of prompt s (t0 = its first row; p < 0: its history).
__device__ __forceinline__ uint16_t raw_at(const SsmScanArgs& a, int s, int t0, int p, int c) {
  if (p >= 0) return a.x[(size_t)(t0 + p) * a.x_stride + c];
  return a.conv_in ? a.conv_in[((size_t)s * 3 + 3 + p) * a.l.conv_dim + c] : 0;
}

template <int N>
__global__ void __launch_bounds__(kRows * (N / 16)) ssm_scan_kernel(const SsmScanArgs a) {
  constexpr int LPR = N / 16, THREADS = kRows * LPR, NCH = kRows + 2 * N;
  const SsmLayer& l = a.l;
  const int s = blockIdx.x, h = blockIdx.y, P = l.P, row0 = blockIdx.z * kRows;
  const int tid = threadIdx.x, rg = tid / LPR, jl = tid % LPR;
  const int grp = h / (l.H / l.G), inner = l.H * P;
  const int t0 = a.cu[s], len = a.cu[s + 1] - t0;
  float S[16];
  const size_t at = ((size_t)h * P + row0 + rg) * N + 4 * jl, all = (size_t)l.H * P * N;
#pragma unroll
  for (int k = 0; k < 16; ++k) S[k] = a.init ? a.init[s * all + at + 4 * LPR * (k / 4) + k % 4] : 0.f;
  int ci = lower_bound_i32(a.ckpt, a.n_ckpt, t0 + 1);
  int next = ci < a.n_ckpt ? a.ckpt[ci] : INT_MAX;
  __shared__ float u[NCH];
  const float A = l.A[h], D = l.D ? l.D[h] : 0.f;
  auto store = [&](float* q) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 16; ++k) q[at + 4 * LPR * (k / 4) + k % 4] = S[k];
  };
  for (int p = 0; p < len; ++p) {
    const size_t t = t0 + p;
    __syncthreads();
    for (int e = tid; e < NCH; e += THREADS) {
      const int c = e < kRows ? h * P + row0 + e
                  : e < kRows + N ? inner + grp * N + e - kRows : inner + (l.G + grp) * N + e - kRows - N;
      if (l.conv_w) {
        const float4 w = reinterpret_cast<const float4*>(l.conv_w)[c];
        u[e] = conv4_bias_silu(l.conv_bias ? conv_tap(l.conv_bias[c]) : 0.f, conv_tap(w.x), conv_tap(w.y), conv_tap(w.z),
                               conv_tap(w.w), bf16_to_f32(raw_at(a, s, t0, p - 3, c)), bf16_to_f32(raw_at(a, s, t0, p - 2, c)),
                               bf16_to_f32(raw_at(a, s, t0, p - 1, c)), bf16_to_f32(raw_at(a, s, t0, p, c)));
      } else {
        u[e] = bf16_to_f32(raw_at(a, s, t0, p, c));
      }
    }
    const float dt = ssm_step(l, a.dt, t * a.dt_stride + h, h), alpha = expf(A * dt);
    __syncthreads();
    const float x = u[rg], dx = dt * x;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int n = 4 * LPR * (k / 4) + 4 * jl + k % 4;
      S[k] = fmaf(alpha, S[k], dx * u[kRows + n]);
      y = fmaf(S[k], u[kRows + N + n], y);
    }
    y = group_sum<LPR>(y);
    if (jl == 0) a.out[(t * l.H + h) * P + row0 + rg] = (uint16_t)f32_to_bf16(fmaf(D, x, y));
    if (t + 1 == (size_t)next) {
      store(a.ckpt_buf + (size_t)ci * all);
      ++ci;
      next = ci < a.n_ckpt ? a.ckpt[ci] : INT_MAX;
    }
  }
  if (a.final_state) store(a.final_state + s * all);
}

// The three inputs before each checkpoint (blockIdx.x < n_ck), or each
// prompt's last three; all reads before all writes of a thread's channels.
__global__ void __launch_bounds__(256) ssm_scan_window_kernel(const SsmScanArgs a, int n_ck) {
  const int c = blockIdx.y * 256 + threadIdx.x, dim = a.l.conv_dim;
  if (c >= dim) return;
  const int i = blockIdx.x;
  const int s = i < n_ck ? seq_of_token(a.cu, a.n_seqs, a.ckpt[i] - 1) : i - n_ck;
  const int t0 = a.cu[s], p = (i < n_ck ? a.ckpt[i] : a.cu[s + 1]) - t0;
  uint16_t* to = (i < n_ck ? a.conv_ckpt + (size_t)i * 3 * dim : a.conv_out + (size_t)s * 3 * dim) + c;
  uint16_t v[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) v[j] = raw_at(a, s, t0, p - 3 + j, c);
#pragma unroll
  for (int j = 0; j < 3; ++j) to[(size_t)j * dim] = v[j];
}

}  // namespace

int64_t ssm_scan_bytes(const SsmLayer&, int32_t, const int32_t*) { return 0; }

hipError_t launch_ssm_scan(const SsmScanArgs& a, void*, hipStream_t st) {
  const dim3 grid(a.n_seqs, a.l.H, a.l.P / kRows), blk(kRows * (a.l.N / 16));
  if (a.l.N == 32) hipLaunchKernelGGL((ssm_scan_kernel<32>), grid, blk, 0, st, a);
  else if (a.l.N == 64) hipLaunchKernelGGL((ssm_scan_kernel<64>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((ssm_scan_kernel<128>), grid, blk, 0, st, a);
  hipError_t e = hipGetLastError();
  const int gy = (a.l.conv_dim + 255) / 256;
  // the checkpoints' windows read conv_in, which the prompts' own may overwrite: before them
  if (e == hipSuccess && a.conv_ckpt && a.n_ckpt > 0) {
    hipLaunchKernelGGL(ssm_scan_window_kernel, dim3(a.n_ckpt, gy), dim3(256), 0, st, a, a.n_ckpt);
    e = hipGetLastError();
  }
  if (e == hipSuccess && a.conv_out) {
    hipLaunchKernelGGL(ssm_scan_window_kernel, dim3(a.n_seqs, gy), dim3(256), 0, st, a, 0);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace gdn
