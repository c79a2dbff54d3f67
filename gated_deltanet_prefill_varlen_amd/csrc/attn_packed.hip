// Causal attention of packed prompts over the paged 8-bit cache: many rows per
// prompt, so the matrix cores bound it.
//
// The rows of a prompt that share a kv head (tokens x Hq / Hkv heads) are
// packed and dealt out to workgroups of four waves, 32 MB rows a wave.  Every
// wave computes, for 64 keys at a time,
//   S^T = K Q^T and O^T += V^T P^T   (32x32x16 products; columns = query rows)
// from tiles that the workgroup stages in LDS as bf16: the 8-bit codes are
// converted once per workgroup, exactly, and a tile's operand is read once for
// all MB row blocks of a wave.
//
// A product's result holds in lane half h the rows 8 a + 4 h + b of a column
// (a, b = 0 .. 3), and its second operand wants there the contraction indices
// 8 h .. 8 h + 7 of a step of 16.  So score row 8 a + 4 h + b is made key
// 16 (a / 2) + 8 h + 4 (a % 2) + b of its 32, and the probabilities become the
// next product's operand without leaving their lane.  Register group a / 2 is
// then one 16-key piece of a page: its scales are the same for every lane.
//
// LDS rows are permuted in 16-byte chunks (chunk ^ row), so that the reads of
// eight lanes at one chunk of eight rows touch all banks.
#include <algorithm>

#include "attn_device.h"

namespace gdn {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 64;      // keys per step
constexpr float kLazy = 8.f;   // the running maximum follows once it lags by this many powers of two

__device__ __forceinline__ float max_halves(float x) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const uint32_t u = __float_as_uint(x);
  const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(u, u, false, false));
  return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}
__device__ __forceinline__ float add_halves(float x) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const uint32_t u = __float_as_uint(x);
  const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(u, u, false, false));
  return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// The permutation of a key row's chunks; the eight keys that eight lanes read
// together are 0 .. 3 and 8 .. 11 of 16, or the others.
template <int KC>
__device__ __forceinline__ int swizzle(int key) {
  return KC == 8 ? (key & 3) | ((key >> 1) & 4) : key & 15;
}

typedef const int32_t __attribute__((address_space(4)))* ConstI32;
typedef const float __attribute__((address_space(4)))* ConstF32;

// One 16-key piece of a tile: its page (-1: not held) and scales, uniform.
struct Piece {
  int page;
  float ks, vs;
};

template <int D, bool I8, int MB>
__global__ void __launch_bounds__(64 * kWaves, 1) attn_packed_kernel(const AttnArgs a, const int units) {
  constexpr int M = 32 * MB * kWaves;   // rows of a workgroup
  constexpr int KC = D / 8;             // 16-byte chunks of a key row
  constexpr int KS = D / 16;            // contraction steps of a score
  constexpr int OB = D / 32;            // 32-channel blocks of the output
  constexpr int NL = D / 64;            // 16-byte loads of codes per lane, keys and values each
  __shared__ __align__(16) uint16_t kl[2][kTile * D];   // [key][d]
  __shared__ __align__(16) uint16_t vl[2][D * kTile];   // [channel][key]

  const int hk = blockIdx.x % a.c.Hkv;
  const int unit = units - 1 - (int)(blockIdx.x / a.c.Hkv);   // late rows see most keys: first
  const int G = a.Hq / a.c.Hkv;
  // unit -> (prompt, its j-th tile of rows): prompt s has the units
  // cu[s] G / M + s on, at least as many as its tiles
  const ConstI32 cu = (ConstI32)a.cu;
  int lo = 0, hi = a.n_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int)((int64_t)cu[mid] * G / M) + mid <= unit) lo = mid; else hi = mid;
  }
  const int s = lo, i0 = cu[s], n = min(cu[s + 1], a.n_tokens) - i0;
  const int64_t first = (int64_t)(unit - (int)((int64_t)i0 * G / M) - s) * M;
  const int64_t rows = (int64_t)n * G;
  if (i0 < 0 || first < 0 || first >= rows) return;
  const int L = ((ConstI32)a.kv_len)[s];
  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  int64_t at[MB];   // this lane's query rows
  int last[MB];     // the last key each sees
  const int r0 = (int)first + wave * 32 * MB;
#pragma unroll
  for (int t = 0; t < MB; ++t) {
    const int r = min(r0 + 32 * t + c32, (int)rows - 1), i = r / G;
    at[t] = (int64_t)(i0 + i) * a.Hq + hk * G + (r - i * G);
    last[t] = L - n + i;
  }
  const bool bad = L < 0 || L > a.max_kv;
  // keys that the workgroup's last row sees, and the wave's first and last
  const int wg_last = (int)min(first + M, rows) - 1, w_last = min(r0 + 32 * MB, (int)rows) - 1;
  const int keys = bad ? 0 : max(0, min(L, L - n + wg_last / G + 1));
  const int w_keys = r0 < rows && !bad ? max(0, L - n + w_last / G + 1) : 0;
  const int w_free = L - n + r0 / G + 1;   // keys that all of the wave's rows see

  // queries: the factor's sign goes into them, so that it leaves maxima maxima
  bf16x8 q[MB][KS];
#pragma unroll
  for (int t = 0; t < MB; ++t) {
    const int64_t tok = at[t] / a.Hq, hd = at[t] % a.Hq;
    const uint16_t* p = a.q + tok * a.q_stride + hd * D + 8 * h;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      u32x4 w = *reinterpret_cast<const u32x4*>(p + 16 * k);
      if (a.scale < 0.f) w ^= 0x80008000u;
      q[t][k] = __builtin_bit_cast(bf16x8, w);
    }
  }
  const float log_scale = fabsf(a.scale) * kLog2e;

  f32x16 o[MB][OB];
  float m[MB], l[MB];
#pragma unroll
  for (int t = 0; t < MB; ++t) {
    m[t] = -__builtin_inff();
    l[t] = 0.f;
#pragma unroll
    for (int x = 0; x < OB; ++x)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[t][x][e] = 0.f;
  }

  const int shift = a.c.page_shift, pmask = (1 << shift) - 1;
  const ConstI32 table = (ConstI32)(a.table + (int64_t)s * a.max_pages);
  auto page_at = [&](int key) -> int {
    if (key >= keys) return -1;
    const int p = table[key >> shift];
    return p >= 0 && p < a.c.n_pages ? p : -1;
  };
  auto piece_at = [&](int key) -> Piece {
    Piece p;
    p.page = page_at(key);
    const int64_t e = (int64_t)max(p.page, 0) * a.c.Hkv + hk;
    // at least 2^-126: a product with a masked score stays -inf
    p.ks = p.page < 0 ? 1.f : fmaxf(((ConstF32)a.c.ks)[e] * log_scale, 0x1p-126f);
    p.vs = p.page < 0 ? 1.f : ((ConstF32)a.c.vs)[e];
    return p;
  };

  // staging: wave w brings the tile's 16-key piece w
  uint4 kr[NL], vr[NL];
  auto fetch = [&](int t0) {
    const int key = t0 + 16 * wave, page = page_at(key);
    const int64_t base = page_base(a.c, max(page, 0), hk) + (key & pmask) * D;
    const uint8_t* kp = a.c.k + base + lane * 16;
    const uint8_t* vp = a.c.v + base + lane * 16;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      kr[i] = *reinterpret_cast<const uint4*>(kp + i * 1024);
      vr[i] = *reinterpret_cast<const uint4*>(vp + i * 1024);
    }
    // codes behind the last key or of a page not held may be anything (NaN)
    const int left = page < 0 ? 0 : keys - key;
    if (left < 16) {
      uint32_t keep[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = left - 4 * j;
        keep[j] = c >= 4 ? 0xFFFFFFFFu : c <= 0 ? 0u : (1u << (8 * c)) - 1;
      }
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        vr[i].x &= keep[0];
        vr[i].y &= keep[1];
        vr[i].z &= keep[2];
        vr[i].w &= keep[3];
      }
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      // 16 codes of key 16 wave + e / D from channel e % D on
      const int e = i * 1024 + lane * 16, key = 16 * wave + e / D, ch = (e % D) / 8;
      bf16x8* row = reinterpret_cast<bf16x8*>(&kl[buf][key * D]);
      row[ch ^ swizzle<KC>(key)] = codes_to_operand<I8>(kr[i].x, kr[i].y);
      row[(ch + 1) ^ swizzle<KC>(key)] = codes_to_operand<I8>(kr[i].z, kr[i].w);
      // 16 keys of channel e / 16
      const int c = i * 64 + lane;
      bf16x8* col = reinterpret_cast<bf16x8*>(&vl[buf][c * kTile]);
      col[(2 * wave) ^ (c & 7)] = codes_to_operand<I8>(vr[i].x, vr[i].y);
      col[(2 * wave + 1) ^ (c & 7)] = codes_to_operand<I8>(vr[i].z, vr[i].w);
    }
  };

  const int krow = 16 * (c32 >> 4) + 8 * ((c32 >> 2) & 1) + 4 * ((c32 >> 3) & 1) + (c32 & 3);
  if (keys > 0) {
    fetch(0);
    stage(0);
  }
  __syncthreads();
  for (int t0 = 0, buf = 0; t0 < keys; t0 += kTile, buf ^= 1) {
    const bool more = t0 + kTile < keys;
    if (more) fetch(t0 + kTile);
    if (t0 < w_keys) {
      Piece pc[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) pc[u] = piece_at(t0 + 16 * u);
      f32x16 sc[MB][2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int t = 0; t < MB; ++t)
#pragma unroll
          for (int e = 0; e < 16; ++e) sc[t][b][e] = 0.f;
        const int key = 32 * b + krow;
        const bf16x8* row = reinterpret_cast<const bf16x8*>(&kl[buf][key * D]);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const bf16x8 kk = row[(2 * k + h) ^ swizzle<KC>(key)];
#pragma unroll
          for (int t = 0; t < MB; ++t) sc[t][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kk, q[t][k], sc[t][b], 0, 0, 0);
        }
      }
      const bool all = pc[0].page >= 0 && pc[1].page >= 0 && pc[2].page >= 0 && pc[3].page >= 0;
      if (!all || t0 + kTile > w_free) {
#pragma unroll
        for (int t = 0; t < MB; ++t)
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int key = t0 + 32 * b + 16 * (e >> 3) + 8 * h + (e & 7);
              if (pc[2 * b + (e >> 3)].page < 0 || key > last[t]) sc[t][b][e] = -__builtin_inff();
            }
      }
      bf16x8 p[MB][4];
#pragma unroll
      for (int t = 0; t < MB; ++t) {
        float mx = -__builtin_inff();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float x = sc[t][u >> 1][8 * (u & 1)];
#pragma unroll
          for (int e = 1; e < 8; ++e) x = fmaxf(x, sc[t][u >> 1][8 * (u & 1) + e]);
          mx = fmaxf(mx, x * pc[u].ks);
        }
        mx = max_halves(mx);
        if (__any(mx > m[t] + kLazy)) {
          const float m1 = mx > m[t] + kLazy ? mx : m[t];
          const float again = m1 == m[t] ? 1.f : exp2_fast(m[t] - m1);
          l[t] *= again;
#pragma unroll
          for (int x = 0; x < OB; ++x) o[t][x] *= again;
          m[t] = m1;
        }
        const float base = m[t] == -__builtin_inff() ? 0.f : m[t];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float e[8], sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = sc[t][u >> 1][8 * (u & 1) + i];
            e[i] = exp2_fast(fmaf(x, pc[u].ks, -base));
            sum += e[i];
          }
          l[t] += sum;
          u32x4 w;
          w.x = pack_bf16(e[0] * pc[u].vs, e[1] * pc[u].vs);
          w.y = pack_bf16(e[2] * pc[u].vs, e[3] * pc[u].vs);
          w.z = pack_bf16(e[4] * pc[u].vs, e[5] * pc[u].vs);
          w.w = pack_bf16(e[6] * pc[u].vs, e[7] * pc[u].vs);
          p[t][u] = __builtin_bit_cast(bf16x8, w);
        }
      }
#pragma unroll
      for (int x = 0; x < OB; ++x) {
        const int c = 32 * x + c32;
        const bf16x8* col = reinterpret_cast<const bf16x8*>(&vl[buf][c * kTile]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bf16x8 vv = col[(2 * u + h) ^ (c & 7)];
#pragma unroll
          for (int t = 0; t < MB; ++t) o[t][x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vv, p[t][u], o[t][x], 0, 0, 0);
        }
      }
    }
    if (more) stage(buf ^ 1);
    __syncthreads();
  }

#pragma unroll
  for (int t = 0; t < MB; ++t) {
    if (r0 + 32 * t + c32 >= rows) continue;
    const float sum = add_halves(l[t]);
    const float inv = bad ? __builtin_nanf("") : m[t] == -__builtin_inff() ? 0.f : 1.f / sum;
    uint16_t* out = a.out + at[t] * D + 4 * h;
#pragma unroll
    for (int x = 0; x < OB; ++x)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<uint2*>(out + 32 * x + 8 * g) =
            make_uint2(pack_bf16(o[t][x][4 * g] * inv, o[t][x][4 * g + 1] * inv),
                       pack_bf16(o[t][x][4 * g + 2] * inv, o[t][x][4 * g + 3] * inv));
  }
}

template <int D, bool I8>
hipError_t launch_d(const AttnArgs& a, hipStream_t st) {
  constexpr int MB = D == 256 ? 1 : 2;
  constexpr int M = 32 * MB * kWaves;
  const int64_t units = (int64_t)a.n_tokens * (a.Hq / a.c.Hkv) / M + a.n_seqs;
  hipLaunchKernelGGL((attn_packed_kernel<D, I8, MB>), dim3((uint32_t)(units * a.c.Hkv)), dim3(64 * kWaves), 0, st, a, (int)units);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_packed(const AttnArgs& a, hipStream_t st) {
  switch (a.c.dim) {
    case 64: return a.c.i8 ? launch_d<64, true>(a, st) : launch_d<64, false>(a, st);
    case 128: return a.c.i8 ? launch_d<128, true>(a, st) : launch_d<128, false>(a, st);
    default: return a.c.i8 ? launch_d<256, true>(a, st) : launch_d<256, false>(a, st);
  }
}

}  // namespace gdn
