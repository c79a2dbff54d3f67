// Decode step of the state space layers: n_tok tokens per sequence in place on
// a pool of fp32 states.
//
//   S <- exp(A dt) S + dt x B^T,   y = S C + D x
//
// What bounds it is the state: every (sequence, head) reads and writes P x N
// fp32 once per call, whatever n_tok is.  A workgroup owns 32 rows of one
// (sequence, head); a row's N columns lie on LPR = N / 16 lanes as four
// float4 each, so a load instruction reads whole 128-byte (N = 128) pieces of
// rows, and the sum S C of a row is a reduction over LPR lanes in a fixed
// order.  The convolved x (this workgroup's rows), B and C go through LDS,
// computed once per workgroup and token.  On one pool over and over: with four
// tokens computed at once 64 sequences of one token took 57.0 us for 46.5, with 64
// rows a workgroup 47.0; one sequence then took 6.5 us for 6.0, four tokens of one
// 11.8 for 10.5.
// 64 sequences, 268 MB from and to memory: 50 us with the windows' launch, 5.5 TB/s.
#include "cache_device.h"
#include "ssm_device.h"

namespace gdn {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 32;

template <int N, int P, bool CONV>
__global__ void __launch_bounds__(kRows * (N / 16)) ssm_decode_kernel(const SsmDecodeArgs a) {
  constexpr int LPR = N / 16, THREADS = kRows * LPR, NCH = kRows + 2 * N;
  const SsmLayer& l = a.l;
  const int b = blockIdx.x, h = blockIdx.y, row0 = blockIdx.z * kRows;
  const int tid = threadIdx.x, rg = tid / LPR, jl = tid % LPR;
  const int grp = h / (l.H / l.G), inner = l.H * P;
  const int r = a.slot ? a.slot[b] : b;

  // The row of the state is asked for before the token's inputs.  A layer's states
  // are met again only after all other layers' have passed, so they stay out of
  // the caches: 64 sequences on states that come from memory 57.6 -> 50.0 us, 256
  // 214 -> 184.  (One pool over and over, which no model does, would find half of
  // it in the last cache: 46.5 us for 49.0.)
  f32x4* const sp = reinterpret_cast<f32x4*>(a.state + (((size_t)r * l.H + h) * P + row0 + rg) * N + 4 * jl);
  f32x4 S[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) S[k] = __builtin_nontemporal_load(sp + LPR * k);

  __shared__ float u[NCH];   // the token's x of these rows, B, C
  const float A = l.A[h], D = l.D ? l.D[h] : 0.f;
  for (int n = 0; n < a.n_tok; ++n) {
    const size_t t = (size_t)b * a.n_tok + n;
    if (n > 0) __syncthreads();   // the previous token's values have been read
    for (int e = tid; e < NCH; e += THREADS) {
      const int c = e < kRows ? h * P + row0 + e
                  : e < kRows + N ? inner + grp * N + e - kRows : inner + (l.G + grp) * N + e - kRows - N;
      if constexpr (CONV) {
        // inputs n - 3 .. n: the tokens' own, before them the slot's window
        float xw[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int pp = n - 3 + p;
          xw[p] = bf16_to_f32(pp >= 0 ? a.x[((size_t)b * a.n_tok + pp) * a.x_stride + c]
                                      : a.conv_state[((size_t)r * 3 + 3 + pp) * l.conv_dim + c]);
        }
        const float4 w = reinterpret_cast<const float4*>(l.conv_w)[c];
        u[e] = conv4_bias_silu(l.conv_bias ? conv_tap(l.conv_bias[c]) : 0.f, conv_tap(w.x), conv_tap(w.y), conv_tap(w.z),
                               conv_tap(w.w), xw[0], xw[1], xw[2], xw[3]);
      } else {
        u[e] = bf16_to_f32(a.x[t * a.x_stride + c]);
      }
    }
    const float dt = ssm_step(l, a.dt, t * a.dt_stride + h, h), alpha = expf(A * dt);
    __syncthreads();
    const float x = u[rg], dx = dt * x;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = 4 * LPR * k + 4 * jl;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        S[k][i] = fmaf(alpha, S[k][i], dx * u[kRows + at + i]);
        y = fmaf(S[k][i], u[kRows + N + at + i], y);
      }
    }
    y = group_sum<LPR>(y);
    if (jl == 0) a.out[(t * l.H + h) * P + row0 + rg] = (uint16_t)pack_bf16(fmaf(D, x, y), 0.f);   // (keeps every NaN)
    if (a.snap) {
      // (through the caches: 23.0 us for 16 sequences of 4 tokens, past them 31.1)
      f32x4* q = reinterpret_cast<f32x4*>(a.snap + ((t * l.H + h) * P + row0 + rg) * N + 4 * jl);
#pragma unroll
      for (int k = 0; k < 4; ++k) q[LPR * k] = S[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) __builtin_nontemporal_store(S[k], sp + LPR * k);
}

// Each slot's window moves on by n_tok inputs: a launch of its own, since
// every head of a group reads the group's old window.  Four channels a
// thread, all reads before all writes.
__global__ void __launch_bounds__(256) ssm_window_kernel(const SsmDecodeArgs a) {
  const int b = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 4, dim = a.l.conv_dim;
  if (c >= dim) return;
  const int r = a.slot ? a.slot[b] : b;
  uint16_t* w = a.conv_state + (size_t)r * 3 * dim + c;
  uint2 v[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int p = a.n_tok - 3 + j;
    v[j] = *reinterpret_cast<const uint2*>(p >= 0 ? a.x + ((size_t)b * a.n_tok + p) * a.x_stride + c : w + (size_t)(3 + p) * dim);
  }
#pragma unroll
  for (int j = 0; j < 3; ++j) *reinterpret_cast<uint2*>(w + (size_t)j * dim) = v[j];
}

template <int N, int P>
hipError_t launch(const SsmDecodeArgs& a, hipStream_t st) {
  const dim3 grid(a.batch, a.l.H, P / kRows), blk(kRows * (N / 16));
  if (!a.l.conv_w) {
    hipLaunchKernelGGL((ssm_decode_kernel<N, P, false>), grid, blk, 0, st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((ssm_decode_kernel<N, P, true>), grid, blk, 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(ssm_window_kernel, dim3(a.batch, (a.l.conv_dim + 1023) / 1024), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <int N>
hipError_t launch_n(const SsmDecodeArgs& a, hipStream_t st) {
  return a.l.P == 32 ? launch<N, 32>(a, st) : a.l.P == 64 ? launch<N, 64>(a, st) : launch<N, 128>(a, st);
}

}  // namespace

hipError_t launch_ssm_decode(const SsmDecodeArgs& a, hipStream_t st) {
  return a.l.N == 32 ? launch_n<32>(a, st) : a.l.N == 64 ? launch_n<64>(a, st) : launch_n<128>(a, st);
}

}  // namespace gdn
