// Root-mean-square norm of rows, with the residual's addition before it, the
// gate silu(z) before or after it, and the result in 8-bit codes with scales:
//
//   r = x + residual,   v = r silu(z) (gate first) or r,
//   y = v / sqrt(mean over the group of v^2 + eps) * (weight + offset)
//       [* silu(z) (gate after)],
//   scale = max |y| of the block / largest code,  code = round(y / scale).
//
// Bound by memory: every input is read once and every output written once, a
// row staying in registers between its sums and its outputs.  A thread holds
// vectors of 8 channels: rows of up to 512 channels lie on a power of two of
// lanes of one wave (several rows a workgroup), wider ones on a workgroup.
// 32,768 rows of 4,096 with residual and codes (0.94 GB): 177 us, 5.3 TB/s; 8,192
// with a gate (0.2 GB): 31 us; 32 rows, bound by the way to memory and two
// barriers: 4.2 us.
// All sums are fp32 in an order that depends on the row's width alone, so a
// row's bits do not depend on the batch.  Rows need no alignment: an 8-channel
// vector is loaded as it lies, a last partial one channel by channel.
#include "cache_device.h"
#include "gdn_device.h"
#include "ssm_internal.h"

namespace gdn {
namespace {

typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2a1 __attribute__((ext_vector_type(2), aligned(1)));

// 8 consecutive elements as they lie in memory, bf16 or fp32.
template <bool F32> struct Raw8;
template <> struct Raw8<false> {
  u32x4a2 w;
  __device__ __forceinline__ void load(const void* p, int64_t at, int n) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    if (n == 8) { w = *reinterpret_cast<const u32x4a2*>(q); return; }
    w = u32x4a2{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) w[i / 2] |= (uint32_t)q[i] << (16 * (i % 2));
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  static __device__ __forceinline__ void store(void* p, int64_t at, int n, const float* f) {
    uint16_t* q = static_cast<uint16_t*>(p) + at;
    const u32x4a2 o{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
    if (n == 8) { *reinterpret_cast<u32x4a2*>(q) = o; return; }
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) q[i] = (uint16_t)(o[i / 2] >> (16 * (i % 2)));
  }
};
template <> struct Raw8<true> {
  f32x4a4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t at, int n) {
    const float* q = static_cast<const float*>(p) + at;
    if (n == 8) {
      a = *reinterpret_cast<const f32x4a4*>(q);
      b = *reinterpret_cast<const f32x4a4*>(q + 4);
      return;
    }
    a = b = f32x4a4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) { if (i < 4) a[i] = q[i]; else b[i - 4] = q[i]; }
  }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
  static __device__ __forceinline__ void store(void* p, int64_t at, int n, const float* f) {
    float* q = static_cast<float*>(p) + at;
    if (n == 8) {
      *reinterpret_cast<f32x4a4*>(q) = f32x4a4{f[0], f[1], f[2], f[3]};
      *reinterpret_cast<f32x4a4*>(q + 4) = f32x4a4{f[4], f[5], f[6], f[7]};
      return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) q[i] = f[i];
  }
};

__device__ __forceinline__ float silu(float z) {
  return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(kNegLog2e * z));
}

struct Add { __device__ __forceinline__ float operator()(float a, float b) const { return a + b; } };
struct Max { __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); } };

// Over aligned groups of `width` lanes (a power of two): every lane of a
// group ends with the same bits.
template <typename Op>
__device__ __forceinline__ float over_lanes(float x, int width, Op op) {
  if (width >= 2) x = op(x, dpp_f32<0xB1>(x));
  if (width >= 4) x = op(x, dpp_f32<0x4E>(x));
  if (width >= 8) x = op(x, dpp_f32<0x141>(x));
  if (width >= 16) x = op(x, dpp_f32<0x140>(x));
  if (width >= 32) x = op(x, __shfl_xor(x, 16));
  if (width >= 64) x = op(x, __shfl_xor(x, 32));
  return x;
}

// XF32: x, gate and out are fp32 (else bf16).  VPT vectors a thread; WAVE:
// rows of `lanes` lanes, VPT = 1; else a row a workgroup.
template <bool XF32, int VPT, int THREADS, bool WAVE>
__global__ void __launch_bounds__(THREADS) rms_norm_kernel(const NormArgs a, int lanes) {
  constexpr int WAVES = THREADS / 64;
  __shared__ float part[WAVE ? 1 : VPT * WAVES], tops[WAVES];
  const int tid = threadIdx.x, lane = WAVE ? tid & (lanes - 1) : tid;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * (THREADS / lanes) + tid / lanes : (int64_t)blockIdx.x;
  const bool real = !WAVE || row < a.n_rows;
  int n[VPT];          // channels of each vector
#pragma unroll
  for (int i = 0; i < VPT; ++i) n[i] = real ? min(8, max(0, a.dim - 8 * (lane + THREADS * i))) : 0;

  Raw8<XF32> x[VPT], z[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (n[i]) x[i].load(a.x, row * a.x_stride + 8 * (lane + THREADS * i), n[i]);
  if (a.gate) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (n[i]) z[i].load(a.gate, row * a.gate_stride + 8 * (lane + THREADS * i), n[i]);
  }
  // The weights are asked for ahead of the sums, but where they would take the
  // registers of two or four vectors (4,096 rows of 16,384: 108 us, ahead 138 us).
  Raw8<true> w[VPT];
  if (VPT == 1 && a.w) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (n[i]) {
        const int c = 8 * (lane + THREADS * i);
        w[i].load(a.w, a.weight_dim == a.dim ? c : c % a.weight_dim, n[i]);
      }
  }
  float v[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = n[i] ? x[i].get(e) : 0.f;
  auto add = [&](auto kind) __attribute__((always_inline)) {
    using R = decltype(kind);
    R r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (n[i]) r[i].load(a.res, row * a.res_stride + 8 * (lane + THREADS * i), n[i]);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (n[i]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] += r[i].get(e);
        if (a.res_out) R::store(a.res_out, row * a.res_stride + 8 * (lane + THREADS * i), n[i], v[i]);
      }
  };
  if (a.res) {
    if (a.res_f32) add(Raw8<true>{});
    else add(Raw8<false>{});
  }
  if (a.gate && a.gate_first) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n[i]) v[i][e] *= silu(z[i].get(e));
  }

  // sums of squares: of the lanes that share a vector's group inside a wave,
  // then of the waves' pieces (512 channels each) where a group is wider
  float ss[VPT];
  const int gl = WAVE || a.group_dim < 512 ? min(a.group_dim == a.dim && WAVE ? lanes : a.group_dim / 8, 64) : 64;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    ss[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss[i] = fmaf(v[i][e], v[i][e], ss[i]);
    ss[i] = over_lanes(ss[i], gl, Add{});
  }
  if (!WAVE && (a.group_dim > 512 || a.groups == 1)) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if ((tid & 63) == 0) part[i * WAVES + tid / 64] = ss[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int per = a.groups == 1 ? VPT * WAVES : a.group_dim / 512;
      const int first = a.groups == 1 ? 0 : (i * WAVES + tid / 64) / per * per;
      if (i > 0 && a.groups == 1) { ss[i] = ss[0]; continue; }
      if ((per & (per - 1)) == 0) {
        ss[i] = over_lanes(part[min(first + (tid & (per - 1)), VPT * WAVES - 1)], per, Add{});
      } else {
        ss[i] = 0.f;
        for (int k = 0; k < per && first + k < VPT * WAVES; ++k) ss[i] += part[first + k];
      }
    }
  }

  float top = 0.f;
  const float inv_n = 1.f / (float)a.group_dim;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const float rinv = 1.f / sqrtf(fmaf(ss[i], inv_n, a.eps));
    if (n[i]) {
      const int c = 8 * (lane + THREADS * i);
      if (VPT > 1 && a.w) w[i].load(a.w, a.weight_dim == a.dim ? c : c % a.weight_dim, n[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float y = v[i][e] * rinv;
        if (a.w) y *= w[i].get(e) + a.weight_offset;
        if (a.gate && !a.gate_first) y *= silu(z[i].get(e));
        v[i][e] = e < n[i] ? y : 0.f;
      }
    }
    if (a.out && n[i]) Raw8<XF32>::store(a.out, row * a.dim + 8 * (lane + THREADS * i), n[i], v[i]);
  }
  if (!a.codes) return;

  const float most = a.codes_i8 ? 127.f : 448.f;
  float m[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    m[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m[i] = fmaxf(m[i], finite_abs(v[i][e]));
    if (a.scale_block) m[i] = over_lanes(m[i], 16, Max{});
    else top = fmaxf(top, m[i]);
  }
  if (!a.scale_block) {
    top = over_lanes(top, WAVE ? lanes : 64, Max{});
    if constexpr (!WAVE) {
      if ((tid & 63) == 0) tops[tid / 64] = top;
      __syncthreads();
      top = over_lanes(tops[tid & (WAVES - 1)], WAVES, Max{});
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (!n[i]) continue;
    const int c = 8 * (lane + THREADS * i);
    const float amax = a.scale_block ? m[i] : top;
    const float scale = fmaxf(amax / most, kMinScale), inv = amax > kMinScale * most ? most / amax : 1.f / kMinScale;
    if (a.scale_block ? (lane & 15) == 0 : lane + i == 0)
      a.scales[a.scale_block ? row * (a.dim / 128) + c / 128 : row] = scale;
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {   // y / scale: the product with 1 / scale, its remainder put right
      const float c = v[i][e] * inv;
      q[e] = fmaf(fmaf(-c, scale, v[i][e]), inv, c);
      if (!(fabsf(c) < 0x1p60f)) q[e] = c;   // (infinities and NaN leave no remainder)
    }
    const u32x2a1 o = a.codes_i8 ? u32x2a1{encode4<true>(q), encode4<true>(q + 4)} : u32x2a1{encode4<false>(q), encode4<false>(q + 4)};
    uint8_t* p = a.codes + row * a.dim + c;
    if (n[i] == 8) *reinterpret_cast<u32x2a1*>(p) = o;
    else
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n[i]) p[e] = (uint8_t)(o[e / 4] >> (8 * (e % 4)));
  }
}

template <bool XF32, int VPT, int THREADS, bool WAVE>
hipError_t go(const NormArgs& a, int lanes, hipStream_t st) {
  const int per = WAVE ? THREADS / lanes : 1;
  hipLaunchKernelGGL((rms_norm_kernel<XF32, VPT, THREADS, WAVE>), dim3((a.n_rows + (int64_t)per - 1) / per), dim3(THREADS), 0,
                     st, a, lanes);
  return hipGetLastError();
}

template <bool XF32>
hipError_t launch(const NormArgs& a, hipStream_t st) {
  const int nv = (a.dim + 7) / 8;
  if (nv <= 64) {
    int lanes = 1;
    while (lanes < nv) lanes *= 2;
    return go<XF32, 1, 256, true>(a, lanes, st);
  }
  // One vector a thread up to 8,192 channels: against two and four on 256 threads
  // 5.7 -> 4.2 us for 32 rows of 4,096, 8.7 -> 5.2 us for 32 of 8,192, 219 -> 188 us
  // for 16,384 of 8,192.
  if (nv <= 256) return go<XF32, 1, 256, false>(a, 0, st);
  if (nv <= 512) return go<XF32, 1, 512, false>(a, 0, st);
  if (nv <= 1024) return go<XF32, 1, 1024, false>(a, 0, st);
  if (nv <= 2048) return go<XF32, 2, 1024, false>(a, 0, st);
  return go<XF32, 4, 1024, false>(a, 0, st);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t st) { return a.x_f32 ? launch<true>(a, st) : launch<false>(a, st); }

}  // namespace gdn
