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

// The same for a channel row of KT keys (128 or 64 bytes) of the value tile.
template <int KT>
__device__ __forceinline__ int swizzle_v(int c) {
  return KT == 64 ? c & 7 : (c >> 2) & 3;
}

// x + both bf16 of a dword.
__device__ __forceinline__ float add_pair(uint32_t two, float x) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), __builtin_bit_cast(bf16x2, 0x3F803F80u), x, false);
}

typedef const int32_t __attribute__((address_space(4)))* ConstI32;
typedef const float __attribute__((address_space(4)))* ConstF32;

// One 16-key piece of a tile: its page (-1: not held) and scales, uniform.
struct Piece {
  int page;
  float ks, vs;
};

// KT: keys per staged tile (64 or 32); a step of the loop takes 32 keys.
template <int D, bool I8, int MB, int KT>
__global__ void __launch_bounds__(64 * kWaves, 1) attn_packed_kernel(const AttnArgs a, const int units) {
  constexpr int M = 32 * MB * kWaves;   // rows of a workgroup
  constexpr int KC = D / 8;             // 16-byte chunks of a key row
  constexpr int KS = D / 16;            // contraction steps of a score
  constexpr int OB = D / 32;            // 32-channel blocks of the output
  constexpr int SUB = KT / 32;          // steps per tile
  constexpr int AHEAD = SUB == 2 ? 1 : 2;   // tiles staged ahead of the one in use
  constexpr int VRING = AHEAD + 2;
  constexpr int NP = KT / 16;           // 16-key pieces of a tile
  constexpr int NL = KT * D / (64 * kWaves * 16);   // 16-byte loads of codes per lane, keys and values each
  constexpr int PER = kWaves / NP;      // waves that share a piece
  __shared__ __align__(16) uint16_t kl[2][KT * D];       // [key][d]
  __shared__ __align__(16) uint16_t vl[VRING][D * KT];   // [channel][key]
  __shared__ uint32_t nan_keys[VRING][kWaves];           // keys of a tile with a NaN value, per staging wave

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
  // keys that the workgroup's last row sees, and that all of its rows and all
  // of the wave's rows see.  Waves whose rows see fewer keys keep step with the
  // others, their scores masked.
  const int wg_last = (int)min(first + M, rows) - 1;
  const int keys = bad ? 0 : max(0, min(L, L - n + wg_last / G + 1));
  const int wg_free = L - n + (int)first / G + 1, w_free = L - n + min(r0, (int)rows - 1) / G + 1;

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
    const int p = table[min(key, max(keys, 1) - 1) >> shift];   // no branch
    return key < keys && p >= 0 && p < a.c.n_pages ? p : -1;
  };
  auto piece_at = [&](int key) -> Piece {
    Piece p;
    p.page = page_at(key);
    const int64_t e = (int64_t)max(p.page, 0) * a.c.Hkv + hk;
    p.ks = ((ConstF32)a.c.ks)[e];
    p.vs = ((ConstF32)a.c.vs)[e];
    return p;
  };

  // ---- staging: a wave brings 1 / PER of one 16-key piece of a tile ----
  uint4 kr[NL], vr[NL];
  const int my_piece = wave / PER, my_part = wave % PER;
  int fetched = 0, page = -1;   // the tile in kr, vr and its page
  auto fetch = [&](int tile) {
    fetched = tile;
    const int key = tile * KT + 16 * my_piece;
    page = page_at(key);
    const int64_t base = page_base(a.c, max(page, 0), hk) + (key & pmask) * D + my_part * (NL * 1024) + lane * 16;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      kr[i] = *reinterpret_cast<const uint4*>(a.c.k + base + i * 1024);
      vr[i] = *reinterpret_cast<const uint4*>(a.c.v + base + i * 1024);
    }
  };
  // Values that not every row of the workgroup may see: what lies behind the
  // last key or in a page not held may be anything, and a NaN that a row does
  // not see would get into it as 0 * NaN.  The former become 0; so do NaN
  // values, whose keys then score NaN for the rows that see them.
  auto clean = [&]() {
    if ((fetched + 1) * KT <= wg_free && page >= 0) return;
    const int left = page < 0 ? 0 : keys - (fetched * KT + 16 * my_piece);
    uint32_t found = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      uint32_t w[4] = {vr[i].x, vr[i].y, vr[i].z, vr[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = left - 4 * j;
        w[j] &= c >= 4 ? 0xFFFFFFFFu : c <= 0 ? 0u : (1u << (8 * c)) - 1;
        if constexpr (!I8) {
          const uint32_t nan = (((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
          w[j] &= ~(nan * 0xFFu);
          found |= ((nan * 0x10204080u) >> 28) << (4 * j);   // the four flags side by side
        }
      }
      vr[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if constexpr (!I8) {
#pragma unroll
      for (int d = 32; d; d >>= 1) found |= __shfl_xor(found, d);
      if (lane == 0) nan_keys[fetched % VRING][wave] = found;
    }
  };
  auto stage = [&]() {
    uint16_t* const kd = kl[fetched & 1];
    uint16_t* const vd = vl[fetched % VRING];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      // 16 codes of one key
      const int e = my_part * (NL * 1024) + i * 1024 + lane * 16, key = 16 * my_piece + e / D, ch = (e % D) / 8;
      bf16x8* row = reinterpret_cast<bf16x8*>(kd + key * D);
      row[ch ^ swizzle<KC>(key)] = codes_to_operand<I8>(kr[i].x, kr[i].y);
      row[(ch + 1) ^ swizzle<KC>(key)] = codes_to_operand<I8>(kr[i].z, kr[i].w);
      // 16 keys of one channel
      const int c = e / 16;
      bf16x8* col = reinterpret_cast<bf16x8*>(vd + c * KT);
      col[(2 * my_piece) ^ swizzle_v<KT>(c)] = codes_to_operand<I8>(vr[i].x, vr[i].y);
      col[(2 * my_piece + 1) ^ swizzle_v<KT>(c)] = codes_to_operand<I8>(vr[i].z, vr[i].w);
    }
  };

  const int krow = 16 * (c32 >> 4) + 8 * ((c32 >> 2) & 1) + 4 * ((c32 >> 3) & 1) + (c32 & 3);
  // scores of step j (32 keys)
  auto qk = [&](int j, f32x16(&sc)[MB]) {
    const int key = 32 * (j % SUB) + krow;
    const bf16x8* row = reinterpret_cast<const bf16x8*>(kl[(j / SUB) & 1] + key * D);
#pragma unroll
    for (int t = 0; t < MB; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[t][e] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const bf16x8 kk = row[(2 * k + h) ^ swizzle<KC>(key)];
#pragma unroll
      for (int t = 0; t < MB; ++t) sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kk, q[t][k], sc[t], 0, 0, 0);
    }
  };
  // output blocks x0 .. x1 - 1 gain step j's probabilities times values
  auto pv = [&](int j, bf16x8(&p)[MB][2], int x0, int x1) {
    const uint16_t* const vd = vl[(j / SUB) % VRING];
#pragma unroll
    for (int x = x0; x < x1; ++x) {
      const int c = 32 * x + c32;
      const bf16x8* col = reinterpret_cast<const bf16x8*>(vd + c * KT);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bf16x8 vv = col[(4 * (j % SUB) + 2 * u + h) ^ swizzle_v<KT>(c)];
#pragma unroll
        for (int t = 0; t < MB; ++t) o[t][x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vv, p[t][u], o[t][x], 0, 0, 0);
      }
    }
  };

  const int steps = (keys + KT - 1) / KT * SUB;
  if (steps > 0) {
#pragma unroll
    for (int t = 0; t < AHEAD; ++t) {
      fetch(t);
      clean();
      stage();
    }
    fetch(AHEAD);
  }
  __syncthreads();

  Piece pc[2] = {piece_at(0), piece_at(16)};
  // Values are measured in units of the first page's scale, within limits that
  // keep zero pages and huge ones from pushing the others out of range.
  const float unit_log = fminf(fmaxf(__builtin_amdgcn_logf(pc[0].page >= 0 ? fmaxf(pc[0].vs, kMinScale) : 1.f), -30.f), 60.f);
  // A step finishes the scores of its 32 keys (formed a step before), and
  // between their exponentials forms the next step's scores and adds the step
  // before's probabilities times values.
  auto step = [&](int j, f32x16(&sc)[MB], f32x16(&next)[MB], bf16x8(&before)[MB][2], bf16x8(&p)[MB][2]) {
    const int key0 = 32 * j, jb = max(j - 1, 0);
    const bool put = j % SUB == 0;
    if (put) clean();
    {
      const bool held0 = pc[0].page >= 0, held1 = pc[1].page >= 0;
      if (key0 + 32 > w_free || !held0 || !held1) {
#pragma unroll
        for (int t = 0; t < MB; ++t)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (!(e < 8 ? held0 : held1) || key0 + 16 * (e >> 3) + 8 * h + (e & 7) > last[t]) sc[t][e] = -__builtin_inff();
      }
      if constexpr (!I8) {
        if ((j / SUB + 1) * KT > wg_free) {
          const uint32_t* const f = nan_keys[(j / SUB) % VRING];
          const int pa = 2 * (j % SUB);
          uint32_t nan[2] = {0, 0};
#pragma unroll
          for (int w = 0; w < PER; ++w) {
            nan[0] |= f[pa * PER + w];
            nan[1] |= f[(pa + 1) * PER + w];
          }
          if (nan[0] | nan[1]) {
#pragma unroll
            for (int t = 0; t < MB; ++t)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if ((nan[e >> 3] >> (8 * h + (e & 7)) & 1) && sc[t][e] != -__builtin_inff()) sc[t][e] = __builtin_nanf("");
          }
        }
      }
      // at least 2^-126: a product with a masked score stays -inf
      float ks[2], lv[2], iv[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool held = u ? held1 : held0;
        ks[u] = held ? fmaxf(pc[u].ks * log_scale, 0x1p-126f) : 1.f;
        const float vs = held ? fmaxf(pc[u].vs, kMinScale) : 1.f;
        lv[u] = __builtin_amdgcn_logf(vs) - unit_log;
        iv[u] = exp2_fast(-lv[u]);
      }
      pc[0] = piece_at(key0 + 32);
      pc[1] = piece_at(key0 + 48);
      float mx[MB];
      bool grow = false;
#pragma unroll
      for (int t = 0; t < MB; ++t) {
        float x[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          x[u] = sc[t][8 * u];
#pragma unroll
          for (int e = 1; e < 8; ++e) x[u] = fmaxf(x[u], sc[t][8 * u + e]);
        }
        mx[t] = max_halves(fmaxf(x[0] * ks[0], x[1] * ks[1]));
        grow |= mx[t] > m[t] + kLazy;
      }
      if (__any(grow)) {
        // the measure is a whole number, so the factor is a power of two and
        // exact, also for the probabilities that are still to be added
#pragma unroll
        for (int t = 0; t < MB; ++t) {
          const float m1 = mx[t] > m[t] + kLazy ? ceilf(mx[t]) : m[t];
          const float again = m1 == m[t] ? 1.f : exp2_fast(m[t] - m1);
          l[t] *= again;
#pragma unroll
          for (int x = 0; x < OB; ++x) {
            asm volatile("" : "+a"(o[t][x]));   // its registers are read here, not before the branch
            o[t][x] *= again;
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            u32x4 w = __builtin_bit_cast(u32x4, before[t][u]);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16(lo_bf16(w[i]) * again, hi_bf16(w[i]) * again);
            before[t][u] = __builtin_bit_cast(bf16x8, w);
          }
          m[t] = m1;
        }
      }
      qk(j + 1, next);
      pv(jb, before, 0, OB);
      if (put) stage();
#pragma unroll
      for (int t = 0; t < MB; ++t) {
        const float base = m[t] == -__builtin_inff() ? 0.f : m[t];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // p times its value's scale, a power of two, rounded to bf16 once;
          // the sum is of the rounded ones, so a row that one key takes is
          // that key's value exactly
          const float b = base - lv[u];
          u32x4 w;
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t two = pack_bf16(exp2_fast(fmaf(sc[t][8 * u + 2 * i], ks[u], -b)),
                                           exp2_fast(fmaf(sc[t][8 * u + 2 * i + 1], ks[u], -b)));
            w[i] = two;
            sum = add_pair(two, sum);
          }
          l[t] = fmaf(sum, iv[u], l[t]);
          asm volatile("" : "+v"(w));   // here, not at its use in the next step
          p[t][u] = __builtin_bit_cast(bf16x8, w);
        }
      }
    }
    if (put) {
      fetch(fetched + 1);
      __syncthreads();
    }
  };

  f32x16 sa[MB], sb[MB];
  bf16x8 pa[MB][2], pb[MB][2];
#pragma unroll
  for (int t = 0; t < MB; ++t) pa[t][0] = pa[t][1] = pb[t][0] = pb[t][1] = bf16x8{};
  if (steps > 0) qk(0, sa);
  for (int j = 0; j < steps; j += 2) {
    step(j, sa, sb, pb, pa);
    if (j + 1 < steps) step(j + 1, sb, sa, pa, pb);
  }
  if (steps > 0) {
    if (steps & 1) pv(steps - 1, pa, 0, OB);
    else pv(steps - 1, pb, 0, OB);
  }

#pragma unroll
  for (int t = 0; t < MB; ++t) {
    if (r0 + 32 * t + c32 >= rows) continue;
    const float sum = add_halves(l[t]);
    const float inv = bad ? __builtin_nanf("") : m[t] == -__builtin_inff() ? 0.f : exp2_fast(unit_log) / sum;
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
  constexpr int KT = D == 256 ? 32 : 64;
  hipLaunchKernelGGL((attn_packed_kernel<D, I8, MB, KT>), dim3((uint32_t)(units * a.c.Hkv)), dim3(64 * kWaves), 0, st, a, (int)units);
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
