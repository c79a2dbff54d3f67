// Causal attention of packed prompts over the paged 8-bit cache: many rows per
// prompt, so the matrix cores bound it.
//
// The rows of a prompt that share a kv head (tokens x Hq / Hkv heads) are
// packed and dealt out to workgroups of four waves, 32 MB rows a wave.  Every
// wave computes, for 32 keys at a time,
//   S^T = K Q^T and O^T += V^T P^T   (32x32x16 products; columns = query rows)
// from tiles of 64 keys that the workgroup stages in LDS as bf16: the 8-bit
// codes are converted once per workgroup, exactly, and a tile's operand is read
// once for all MB row blocks of a wave.
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
#include <type_traits>

#include "attn_device.h"

namespace gdn {
namespace {

constexpr int kWaves = 8;
constexpr int kTile = 64;      // keys staged at a time; a step takes 32
constexpr float kLazy = 8.f;   // the running maximum follows once it lags by this many powers of two

__device__ __forceinline__ uint2 both_halves(float x) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const uint32_t u = __float_as_uint(x);
  const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(u, u, false, false));
  return make_uint2(r.x, r.y);
}
__device__ __forceinline__ float max_halves(float x) {
  const uint2 r = both_halves(x);
  return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}
__device__ __forceinline__ float add_halves(float x) {
  const uint2 r = both_halves(x);
  return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// The permutation of a key row's chunks; the eight keys that eight lanes read
// together are 0 .. 3 and 8 .. 11 of 16, or the others.
template <int D>
__device__ __forceinline__ int swizzle(int key) {
  return D == 64 ? (key & 3) | ((key >> 1) & 4) : key & 15;
}

// x + both bf16 of a dword.
__device__ __forceinline__ float add_pair(uint32_t two, float x) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), __builtin_bit_cast(bf16x2, 0x3F803F80u), x, false);
}

typedef const int32_t __attribute__((address_space(4)))* ConstI32;
typedef const float __attribute__((address_space(4)))* ConstF32;

template <int D, bool I8, int MB>
__global__ void __launch_bounds__(64 * kWaves, 2) attn_packed_kernel(const AttnArgs a, const int units) {
  constexpr int M = 32 * MB * kWaves;   // rows of a workgroup
  constexpr int KS = D / 16;            // contraction steps of a score
  constexpr int OB = D / 32;            // 32-channel blocks of the output
  constexpr int NU = D / 64;            // units of 8 codes per lane and tile, keys and values each
  constexpr int KBYTES = kTile * D * 2; // a staged tile of keys [key][d], or of values [channel][key]
  __shared__ __align__(16) char lds[4 * KBYTES];        // keys of two tiles, values of two tiles
  __shared__ __align__(16) float4 pieces[4][4];         // of four tiles: each 16 keys' scales
  __shared__ uint32_t nan_keys[4][kWaves];              // of four tiles: keys with a NaN value
  char* const vlds = lds + 2 * KBYTES;

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

  // ---- staging: two waves bring a 16-key piece of a tile ----
  const int piece = wave >> 1, part = wave & 1;
  const int shift = a.c.page_shift, pmask = (1 << shift) - 1;
  const ConstI32 table = (ConstI32)(a.table + (int64_t)s * a.max_pages);
  uint2 kr[NU], vr[NU];
  int page = -1, key = 0;   // the wave's piece of the tile looked up last: its page (-1: none) and first key
  int64_t base = 0;         // its codes
  float ks = 0.f, vs = 0.f;
  auto look_up = [&](int tile) {
    key = tile * kTile + 16 * piece;
    const int p = table[min(key, max(keys, 1) - 1) >> shift];
    page = key < keys && p >= 0 && p < a.c.n_pages ? p : -1;
    const int64_t e = (int64_t)max(page, 0) * a.c.Hkv + hk;
    base = ((e << shift) + (key & pmask)) * D;
    ks = ((ConstF32)a.c.ks)[e];
    vs = ((ConstF32)a.c.vs)[e];
  };
  auto fetch = [&](const uint8_t* from, uint2(&r)[NU]) {
    const uint8_t* const p = from + base + part * 8 * D;
    if constexpr (NU == 1) {
      r[0] = *reinterpret_cast<const uint2*>(p + lane * 8);
    } else {
#pragma unroll
      for (int i = 0; i < NU / 2; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(p + i * 1024 + lane * 16);
        r[2 * i] = make_uint2(w.x, w.y);
        r[2 * i + 1] = make_uint2(w.z, w.w);
      }
    }
  };
  auto value_scale = [&]() { return page < 0 ? 1.f : fmaxf(vs, kMinScale); };
  // Values that not every row of the workgroup may see: what lies behind the
  // last key or in a page not held may be anything, and a NaN that a row does
  // not see would get into it as 0 * NaN.  The former become 0; so do NaN
  // values, whose keys then score NaN for the rows that see them.
  auto clean = [&](int tile) {
    if ((tile + 1) * kTile <= wg_free && page >= 0) return;
    uint32_t found = 0;
#pragma unroll
    for (int x = 0; x < NU; ++x) {
      const int second = NU == 1 ? lane & 1 : x & 1;   // which 8 of the 16 keys
      const int left = (page < 0 ? 0 : keys - key) - 8 * second;
      uint32_t w[2] = {vr[x].x, vr[x].y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = left - 4 * j;
        w[j] &= c >= 4 ? 0xFFFFFFFFu : c <= 0 ? 0u : (1u << (8 * c)) - 1;
        if constexpr (!I8) {
          const uint32_t nan = (((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
          w[j] &= ~(nan * 0xFFu);
          found |= ((nan * 0x10204080u) >> 28) << (8 * second + 4 * j);   // the four flags side by side
        }
      }
      vr[x] = make_uint2(w[0], w[1]);
    }
    if constexpr (!I8) {
#pragma unroll
      for (int d = 32; d; d >>= 1) found |= __shfl_xor(found, d);
      if (lane == 0) nan_keys[tile & 3][wave] = found;
    }
  };
  // The scales as the steps use them: the scores' factor (at least 2^-126: its
  // product with a masked score stays -inf), the values' as a power of two and
  // the inverse of that, which is 0 for a piece that is not held.  Values are
  // measured in units of the first page's scale, within limits that keep zero
  // pages and huge ones from pushing the others out of range.
  float unit_log = 0.f;
  auto put_scales = [&](int tile) {
    const float lv = __builtin_amdgcn_logf(value_scale()) - unit_log;
    if (lane == 0 && part == 0)
      pieces[tile & 3][piece] = page < 0 ? make_float4(1.f, 0.f, 0.f, 0.f)
                                        : make_float4(fmaxf(ks * log_scale, 0x1p-126f), lv, exp2_fast(-lv), 0.f);
  };
  // LDS addresses of a lane's units of a tile: 8 channels of a key, 8 keys of a channel
  constexpr int NA = NU == 1 ? 1 : 2;
  int kput[NA], vput[NA];
#pragma unroll
  for (int x = 0; x < NA; ++x) {
    const int e = part * 8 * D + (NU == 1 ? lane * 8 : lane * 16 + x * 8), k = 16 * piece + e / D, c = e / 16;
    kput[x] = k * D * 2 + (((e % D / 8) ^ swizzle<D>(k)) * 16);
    vput[x] = c * kTile * 2 + (((2 * piece + (e >> 3 & 1)) ^ (c & 7)) * 16);
  }
  // (units 2 and 3, D = 256: keys 4 on, channels 64 on)
  auto put_keys = [&](int buf, int x) {
    *reinterpret_cast<bf16x8*>(lds + ((kput[x % NA] ^ (x >= 2 ? 4 * 16 : 0)) + buf * KBYTES + (x >= 2 ? 4 * D * 2 : 0))) =
        codes_to_operand<I8>(kr[x].x, kr[x].y);
  };
  auto put_values = [&](int buf, int x) {
    *reinterpret_cast<bf16x8*>(vlds + (vput[x % NA] + buf * KBYTES + (x >= 2 ? 64 * kTile * 2 : 0))) =
        codes_to_operand<I8>(vr[x].x, vr[x].y);
  };

  // ---- operands: even ones 16 channels of 32 keys, odd ones 16 keys of 32 channels ----
  constexpr int OPS = 2 * KS, KA = KS < 8 ? KS : 8;
  const int krow = 16 * (c32 >> 4) + 8 * ((c32 >> 2) & 1) + 4 * ((c32 >> 3) & 1) + (c32 & 3);
  int kget[KA], vget[4];
#pragma unroll
  for (int k = 0; k < KA; ++k) kget[k] = krow * D * 2 + (((2 * k + h) ^ swizzle<D>(krow)) * 16);
#pragma unroll
  for (int u = 0; u < 4; ++u) vget[u] = c32 * kTile * 2 + (((2 * u + h) ^ (c32 & 7)) * 16);
  // jk, jv: steps modulo 4 of the keys and of the values
  auto operand = [&](int c, int jk, int jv) -> bf16x8 {
    if (c & 1) {
      const int x = c >> 2, u = (c >> 1) & 1;
      return *reinterpret_cast<const bf16x8*>(vlds + (vget[2 * (jv & 1) + u] + (jv >> 1) * KBYTES + x * 32 * kTile * 2));
    }
    const int k = c >> 1;
    return *reinterpret_cast<const bf16x8*>(lds + (kget[k % KA] + (jk >> 1) * KBYTES + (jk & 1) * 32 * D * 2 + k / KA * 256));
  };
  // products with operand c: next += keys x queries, or o += values x p
  auto product = [&](int c, bf16x8 x, f32x16(&next)[MB], bf16x8(&p)[MB][2]) {
#pragma unroll
    for (int t = 0; t < MB; ++t) {
      if (c & 1) o[t][c >> 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, p[t][(c >> 1) & 1], o[t][c >> 2], 0, 0, 0);
      else next[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, q[t][c >> 1], next[t], 0, 0, 0);
    }
  };

  const int steps = (keys + kTile - 1) / kTile * 2;
  if (steps > 0) {
    look_up(0);
    const int p0 = table[0];
    const float v0 = ((ConstF32)a.c.vs)[(int64_t)(p0 >= 0 && p0 < a.c.n_pages ? p0 : 0) * a.c.Hkv + hk];
    unit_log = fminf(fmaxf(__builtin_amdgcn_logf(p0 >= 0 && p0 < a.c.n_pages ? fmaxf(v0, kMinScale) : 1.f), -30.f), 60.f);
    fetch(a.c.k, kr);
    fetch(a.c.v, vr);
    clean(0);
    put_scales(0);
#pragma unroll
    for (int x = 0; x < NU; ++x) {
      put_keys(0, x);
      put_values(0, x);
      put_values(1, x);   // step 0 multiplies these by probabilities of 0: no NaN of old may be there
    }
    look_up(1);
    fetch(a.c.k, kr);
    fetch(a.c.v, vr);
  }
  __syncthreads();

  // A step turns the scores of its 32 keys (formed a step before) into
  // probabilities, and meanwhile forms the next step's scores and adds the
  // step before's probabilities times values.  One wave has a SIMD to itself
  // and issues one instruction at a time, so what counts is how few there are:
  // LDS addresses are fixed (four steps are laid out one after the other: two
  // tiles of two steps), the scales come from LDS, and products are dealt out
  // evenly between the vector instructions, each operand read LEAD products
  // before its use; the first EARLY of them run beside the maximum.
  // Even steps stage the next tile's keys, odd ones its values: a tile's last
  // reader is past the barrier (at the end of even steps) by then.
  constexpr int LEAD = 3, EARLY = OPS / 5, PAIRS = 8 * MB;
  auto step = [&](auto jc, int j, f32x16(&sc)[MB], f32x16(&next)[MB], bf16x8(&before)[MB][2], bf16x8(&p)[MB][2]) {
    constexpr int J = decltype(jc)::value, JK = (J + 1) & 3, JV = (J + 3) & 3;
    const int key0 = 32 * j, tile = j >> 1;
    if ((J & 1) == 0) clean(tile + 1);
    const float4 pc0 = pieces[tile & 3][2 * (J & 1)], pc1 = pieces[tile & 3][2 * (J & 1) + 1];
    bf16x8 x[OPS];
#pragma unroll
    for (int c = 0; c < LEAD; ++c) x[c] = operand(c, JK, JV);
    if (key0 + 32 > w_free || __any(fminf(pc0.z, pc1.z) == 0.f)) {
#pragma unroll
      for (int t = 0; t < MB; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if ((e < 8 ? pc0.z : pc1.z) == 0.f || key0 + 16 * (e >> 3) + 8 * h + (e & 7) > last[t]) sc[t][e] = -__builtin_inff();
      if constexpr (!I8) {
        if ((tile + 1) * kTile > wg_free) {
          const uint32_t* const f = nan_keys[tile & 3] + 4 * (J & 1);
          const uint32_t nan[2] = {f[0] | f[1], f[2] | f[3]};
          if (__any(nan[0] | nan[1])) {
#pragma unroll
            for (int t = 0; t < MB; ++t)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if ((nan[e >> 3] >> (8 * h + (e & 7)) & 1) && sc[t][e] != -__builtin_inff()) sc[t][e] = __builtin_nanf("");
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < MB; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) next[t][e] = 0.f;
#pragma unroll
    for (int c = 0; c < EARLY; ++c) {
      x[c + LEAD] = operand(c + LEAD, JK, JV);
      product(c, x[c], next, before);
    }
    float mx[MB];
    bool grow = false;
#pragma unroll
    for (int t = 0; t < MB; ++t) {
      float y[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        y[u] = sc[t][8 * u];
#pragma unroll
        for (int e = 1; e < 8; ++e) y[u] = fmaxf(y[u], sc[t][8 * u + e]);
      }
      mx[t] = max_halves(fmaxf(y[0] * pc0.x, y[1] * pc1.x));
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
        for (int b = 0; b < OB; ++b) {
          o[t][b] *= again;
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
    float off[MB][2], sum[MB][2];
#pragma unroll
    for (int t = 0; t < MB; ++t) {
      const float b = m[t] == -__builtin_inff() ? 0.f : m[t];
      off[t][0] = pc0.y - b;
      off[t][1] = pc1.y - b;
      sum[t][0] = sum[t][1] = 0.f;
    }
    u32x4 w[MB][2];
#pragma unroll
    for (int c = EARLY; c < OPS; ++c) {
      if (c + LEAD < OPS) x[c + LEAD] = operand(c + LEAD, JK, JV);
      product(c, x[c], next, before);
      // p times its value's scale, a power of two, rounded to bf16 once; the
      // sum is of the rounded ones, so a row that one key takes is that key's
      // value exactly
#pragma unroll
      for (int e = (c - EARLY) * PAIRS / (OPS - EARLY); e < (c - EARLY + 1) * PAIRS / (OPS - EARLY); ++e) {
        const int t = e / 8, u = (e / 4) & 1, i = e & 3;
        const float f = u ? pc1.x : pc0.x;
        uint32_t two = pack_bf16(exp2_fast(fmaf(sc[t][8 * u + 2 * i], f, off[t][u])),
                                 exp2_fast(fmaf(sc[t][8 * u + 2 * i + 1], f, off[t][u])));
        asm volatile("" : "+v"(two));   // formed here, not at its use in the next step
        w[t][u][i] = two;
        sum[t][u] = add_pair(two, sum[t][u]);
      }
#pragma unroll
      for (int e = (c - EARLY) * NU / (OPS - EARLY); e < (c - EARLY + 1) * NU / (OPS - EARLY); ++e) {
        if (J & 1) put_values((J >> 1) ^ 1, e);
        else put_keys((J >> 1) ^ 1, e);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int t = 0; t < MB; ++t) {
      l[t] = fmaf(sum[t][1], pc1.z, fmaf(sum[t][0], pc0.z, l[t]));
#pragma unroll
      for (int u = 0; u < 2; ++u) p[t][u] = __builtin_bit_cast(bf16x8, w[t][u]);
    }
    if (J & 1) {
      fetch(a.c.v, vr);      // of the tile looked up a step before
    } else {
      put_scales(tile + 1);
      look_up(tile + 2);
      fetch(a.c.k, kr);
      __syncthreads();
    }
  };

  f32x16 sa[MB], sb[MB];
  bf16x8 pa[MB][2], pb[MB][2];
#pragma unroll
  for (int t = 0; t < MB; ++t) {
    pa[t][0] = pa[t][1] = pb[t][0] = pb[t][1] = bf16x8{};
#pragma unroll
    for (int e = 0; e < 16; ++e) sa[t][e] = sb[t][e] = 0.f;
  }
  if (steps > 0) {
#pragma unroll
    for (int c = 0; c < OPS; c += 2) product(c, operand(c, 0, 0), sa, pa);
  }
  int j = 0;
  for (; j + 4 <= steps; j += 4) {   // (a way out of its middle would cost registers)
    step(std::integral_constant<int, 0>(), j, sa, sb, pb, pa);
    step(std::integral_constant<int, 1>(), j + 1, sb, sa, pa, pb);
    step(std::integral_constant<int, 2>(), j + 2, sa, sb, pb, pa);
    step(std::integral_constant<int, 3>(), j + 3, sb, sa, pa, pb);
  }
  if (steps & 2) {
    step(std::integral_constant<int, 0>(), j, sa, sb, pb, pa);
    step(std::integral_constant<int, 1>(), j + 1, sb, sa, pa, pb);
  }
  if (steps > 0) {   // the last step's probabilities
    const char* const tail = vlds + ((steps >> 1) - 1 & 1) * KBYTES;
#pragma unroll
    for (int c = 1; c < OPS; c += 2)
      product(c, *reinterpret_cast<const bf16x8*>(tail + vget[2 + ((c >> 1) & 1)] + (c >> 2) * 32 * kTile * 2), sa, pb);
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
  constexpr int MB = 1;
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
