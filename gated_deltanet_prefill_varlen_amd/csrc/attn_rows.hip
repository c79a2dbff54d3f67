// Causal softmax attention over the paged 8-bit cache: one wave per (row,
// query head), 64 keys at a time.  A lane scores one key against the whole
// query (in LDS), the wave joins the 64 scores, and each lane then sums its
// own channels of the values.  fp32 throughout.
#include "cache_device.h"

namespace gdn {
namespace {

template <int D, bool I8>
__global__ void __launch_bounds__(64) attn_row_kernel(const AttnArgs a) {
  __shared__ float qs[D];
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x / a.Hq;
  const int h = (int)(blockIdx.x % a.Hq), hk = h / (a.Hq / a.c.Hkv);
  int s, i, n;
  if (a.n_tok) {
    s = (int)(row / a.n_tok);
    i = (int)(row % a.n_tok);
    n = a.n_tok;
  } else {
    if (row >= a.cu[a.n_seqs]) return;
    s = seq_of_token(a.cu, a.n_seqs, (int)row);
    i = (int)row - a.cu[s];
    n = a.cu[s + 1] - a.cu[s];
  }
  const int L = a.kv_len[s];
  uint16_t* const out = a.out + (row * a.Hq + h) * D;
  if (L < 0 || L > a.max_kv) {
    for (int c = lane; c < D; c += 64) out[c] = 0x7FC0;
    return;
  }
  for (int c = lane; c < D; c += 64) qs[c] = bf16_to_f32(a.q[row * a.q_stride + (int64_t)h * D + c]) * a.scale;
  __syncthreads();
  const int seen = max(0, L - n + i + 1);
  constexpr int C = D / 64;
  float o[C] = {};
  float m = -__builtin_inff(), l = 0.f;
  const int shift = a.c.page_shift, mask = (1 << shift) - 1;
  for (int j0 = 0; j0 < seen; j0 += 64) {
    const int j = j0 + lane;
    int page = -1;
    if (j < seen) page = a.table[(int64_t)s * a.max_pages + (j >> shift)];
    if (page >= a.c.n_pages) page = -1;
    float score = -__builtin_inff(), vs = 0.f;
    if (page >= 0) {
      const uint4* kp = reinterpret_cast<const uint4*>(a.c.k + page_base(a.c, page, hk) + (j & mask) * D);
      float sum = 0.f;
      for (int c = 0; c < D / 16; ++c) {
        const uint4 w = kp[c];
        float x[16];
        decode4<I8>(w.x, x);
        decode4<I8>(w.y, x + 4);
        decode4<I8>(w.z, x + 8);
        decode4<I8>(w.w, x + 12);
#pragma unroll
        for (int e = 0; e < 16; ++e) sum = fmaf(x[e], qs[16 * c + e], sum);
      }
      score = sum * a.c.ks[(int64_t)page * a.c.Hkv + hk];
      vs = a.c.vs[(int64_t)page * a.c.Hkv + hk];
    }
    float mx = score;
#pragma unroll
    for (int d = 32; d; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    const float m1 = fmaxf(m, mx);
    if (m1 == -__builtin_inff()) continue;   // nothing held yet
    const float p = page >= 0 ? expf(score - m1) : 0.f;
    const float again = expf(m - m1);
    float ps = p;
#pragma unroll
    for (int d = 32; d; d >>= 1) ps += __shfl_xor(ps, d);
    l = l * again + ps;
    m = m1;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= again;
    const float pv = page >= 0 ? p * vs : 0.f;
    for (int e = 0; e < 64 && j0 + e < seen; ++e) {
      const int pg = __shfl(page, e);
      if (pg < 0) continue;
      const float w = __shfl(pv, e);
      const int off = (j0 + e) & mask;
      const uint8_t* vp = a.c.v + page_base(a.c, pg, hk) + (off >> 4) * 16 * D + (off & 15);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[4];
        decode4<I8>(vp[(lane + 64 * c) * 16], f);
        o[c] = fmaf(w, f[0], o[c]);
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) out[lane + 64 * c] = (uint16_t)pack_bf16(seen > 0 && m > -__builtin_inff() ? o[c] * inv : 0.f, 0.f);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)((int64_t)a.n_tokens * a.Hq)), block(64);
  switch (a.c.dim) {
    case 64:
      if (a.c.i8) hipLaunchKernelGGL((attn_row_kernel<64, true>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((attn_row_kernel<64, false>), grid, block, 0, st, a);
      break;
    case 128:
      if (a.c.i8) hipLaunchKernelGGL((attn_row_kernel<128, true>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((attn_row_kernel<128, false>), grid, block, 0, st, a);
      break;
    default:
      if (a.c.i8) hipLaunchKernelGGL((attn_row_kernel<256, true>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((attn_row_kernel<256, false>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace gdn
