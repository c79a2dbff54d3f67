// Causal attention of packed prompts over the paged 8-bit cache: many rows per
// prompt, work for the matrix cores.  (Prompts of few rows are left to the
// kernel of the decoding requests.)
//
// The rows of a prompt that share a kv head (tokens x Hq / Hkv heads) are
// packed and dealt out to workgroups of eight waves, 32 rows a wave.  Every
// wave computes, a tile of 64 (head_dim 256: 32) keys at a time,
//   S^T = K Q^T and O^T += V^T P^T   (32x32x16 products; columns = query rows)
// from tiles that the workgroup stages in LDS as bf16, so the 8-bit codes are
// converted once per workgroup, exactly.
//
// A product's result holds in lane half h the rows 8 a + 4 h + b of a column
// (a, b = 0 .. 3), and its second operand wants there the contraction indices
// 8 h .. 8 h + 7 of a step of 16.  So score row 8 a + 4 h + b is made key
// 16 (a / 2) + 8 h + 4 (a % 2) + b of its 32, and the probabilities become the
// next product's operand without leaving their lane.  Register group a / 2 is
// then one 16-key piece of a page: its scales are the same for every lane.
//
// Measured: 4 prompts of 8,192 tokens, 16 query heads on 4 kv heads of 128,
// int8: 1.13 ms, 976 TFLOP/s (a bf16 library product of 8,192^3 reaches 1,270 to
// 1,390).  Prompts of 4,096: heads of 64 570 TFLOP/s, of 128 785, of 256 825
// (int8) and 770 (e4m3); both spill a few registers.  No unit is near its
// limit there: of a SIMD's or CU's cycles, matrix cores are busy in 27, 41 and
// 40 % (heads of 64, 128, 256, int8), vector units in 52, 48 and 33 %, LDS in
// 26, 35 and 32 %.  Half steps (below) end at barriers, where each side waits
// for the slower one.
//
// LDS rows are permuted in 16-byte chunks, so that the reads of sixteen lanes
// at one chunk of sixteen rows touch all banks.
#include <algorithm>
#include <type_traits>

#include "attn_device.h"

namespace gdn {
namespace {

constexpr int kWaves = 8;
constexpr int kRows = 32 * kWaves;   // of a workgroup
constexpr float kLazy = 16.f;  // the running maximum follows once it lags by this many powers of two

// Values are measured in units of 2^-kUnit, so that a page of the smallest scale
// (2^-100) keeps probabilities down to 2^-50.  The sum of the probabilities is
// formed from their products with the scales, divided by the scale again.
// Beyond these limits the products could lose what the sum needs (they are down
// to 2^-74 by the measure and 2^-26 by a probability), or fp32 does not hold
// the inverse, and it is formed apart.
constexpr float kUnit = 24.f, kTiny = -26.f, kHuge = 126.f;

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

// The permutation of a key row's chunks (D = 64: two rows share the banks, and
// the sixteen keys read together are 0 .. 15 in the order of krow below).
template <int D>
__device__ __forceinline__ int swizzle_k(int key) {
  return D == 64 ? (key >> 1) & 7 : key & 15;
}
// The same for a channel's row of KT keys.
template <int KT>
__device__ __forceinline__ int swizzle_v(int c) {
  return KT == 64 ? (c >> 1) & 7 : (c >> 2) & 3;
}

// x + both bf16 of a dword.
__device__ __forceinline__ float add_pair(uint32_t two, float x) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), __builtin_bit_cast(bf16x2, 0x3F803F80u), x, false);
}

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

typedef const int32_t __attribute__((address_space(4)))* ConstI32;
typedef const float __attribute__((address_space(4)))* ConstF32;

// Workgroups start in order of their index.  A prompt's last rows see most keys
// and go first; up to 64 prompts are taken in the order of the keys that their
// first rows see, so that the short tiles fill the end (8 prompts of 17 to 2,048
// tokens on up to 4,096, two draws: 535 -> 507 us and 450 -> 452 us).  By the
// keys of each tile, across the prompts, the end is as even, but the prompts no
// longer share an L2 (507 and 462 us).  More prompts are taken in the pack's
// order: each is little beside the card's 256 workgroups.
__device__ __forceinline__ bool tile_of_rank(const AttnArgs& a, int G, int rank, int* prompt, int* first) {
  const int lane = threadIdx.x & 63, s = min(lane, a.n_seqs - 1);
  const int i0 = a.cu[s], n = lane < a.n_seqs && i0 >= 0 ? max(min(a.cu[s + 1], a.n_tokens) - i0, 0) : 0;
  const int tiles = n <= few_rows(a.c.dim) / G ? 0 : (int)(((int64_t)n * G + kRows - 1) / kRows);
  const int keys = max(a.kv_len[s] - n + min(n, kRows / G), 0);   // of the first tile, nearly
  int before = 0;   // tiles of the prompts that go first
  for (int j = 0; j < a.n_seqs; ++j) {
    const int k = __builtin_amdgcn_readlane(keys, j), t = __builtin_amdgcn_readlane(tiles, j);
    if (k > keys || (k == keys && j > s)) before += t;
  }
  const uint64_t mine = __ballot(rank >= before && rank < before + tiles);
  if (!mine) return false;
  *prompt = __builtin_ctzll(mine);
  *first = __builtin_amdgcn_readlane((before + tiles - 1 - rank) * kRows, *prompt);
  return true;
}

template <int D, bool I8>
__global__ void __launch_bounds__(64 * kWaves, 2) attn_packed_kernel(const AttnArgs a, const int units) {
  constexpr int KT = D == 256 ? 32 : 64;   // keys of a tile, and of a step
  constexpr int KB = KT / 32;              // blocks of 32 keys
  constexpr int NP = KT / 16;              // 16-key pieces, each in one page
  constexpr int KS = D / 16;               // contraction steps of a score
  constexpr int OB = D / 32;               // 32-channel blocks of the output
  constexpr int PARTS = kWaves / NP;       // waves that bring a piece
  constexpr int NU = KT * D / (64 * kWaves * 8);   // units of 8 codes per lane and tile, keys and values each
  constexpr int BYTES = KT * D * 2;        // a staged tile of keys [key][d], or of values [channel][key]
  __shared__ __align__(16) char lds[6 * BYTES];      // three tiles of keys, three of values
  __shared__ __align__(16) float4 pieces[4][NP];     // of four tiles: each piece's scales
  __shared__ uint32_t nan_keys[4][kWaves];           // of four tiles: keys with a NaN value
  char* const vlds = lds + 3 * BYTES;

  const int hk = blockIdx.x % a.c.Hkv;
  const int G = a.Hq / a.c.Hkv;
  const ConstI32 cu = (ConstI32)a.cu;
  int s = 0, first = 0;
  if (a.n_seqs <= 64) {
    if (!tile_of_rank(a, G, (int)(blockIdx.x / a.c.Hkv), &s, &first)) return;
  } else {
    // unit -> (prompt, its j-th tile of rows): prompt s has the units
    // cu[s] G / kRows + s on, at least as many as its tiles
    const int unit = units - 1 - (int)(blockIdx.x / a.c.Hkv);
    int hi = a.n_seqs;
    while (hi - s > 1) {
      const int mid = (s + hi) >> 1;
      if ((int)((int64_t)cu[mid] * G / kRows) + mid <= unit) s = mid; else hi = mid;
    }
    const int64_t at = (int64_t)(unit - (int)((int64_t)cu[s] * G / kRows) - s) * kRows;
    const int n = min(cu[s + 1], a.n_tokens) - cu[s];
    if (cu[s] < 0 || at < 0 || at >= (int64_t)n * G || n <= few_rows(D) / G) return;
    first = (int)at;
  }
  const int i0 = cu[s], n = min(cu[s + 1], a.n_tokens) - i0;
  const int64_t rows = (int64_t)n * G;
  const int L = ((ConstI32)a.kv_len)[s];
  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // this lane's query row and the last key it sees
  const int r0 = first + wave * 32;
  const int r = min(r0 + c32, (int)rows - 1), i = r / G, hq = hk * G + (r - i * G);
  const int last = L - n + i;
  const bool bad = L < 0 || L > a.max_kv;
  // keys that the workgroup's last row sees, and that all of its rows and all
  // of the wave's rows see.  Waves whose rows see fewer keys keep step with the
  // others, their scores masked.
  const int wg_last = (int)min((int64_t)first + kRows, rows) - 1;
  const int keys = bad ? 0 : max(0, min(L, L - n + wg_last / G + 1));
  const int wg_free = L - n + first / G + 1, w_free = L - n + min(r0, (int)rows - 1) / G + 1;

  // queries: the factor's sign goes into them, so that it leaves maxima maxima
  bf16x8 q[KS];
  const uint16_t* const qp = a.q + (int64_t)(i0 + i) * a.q_stride + hq * D + 8 * h;
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    u32x4 w = *reinterpret_cast<const u32x4*>(qp + 16 * k);
    if (a.scale < 0.f) w ^= 0x80008000u;
    q[k] = __builtin_bit_cast(bf16x8, w);
  }
  const float log_scale = uniform(fabsf(a.scale) * kLog2e);

  f32x16 o[OB];
  float m = -__builtin_inff(), l = 0.f;
#pragma unroll
  for (int x = 0; x < OB; ++x)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[x][e] = 0.f;

  // ---- staging: PARTS waves bring a 16-key piece of a tile ----
  const int piece = wave / PARTS, part = wave % PARTS;
  const int shift = a.c.page_shift, pmask = (1 << shift) - 1;
  const ConstI32 table = (ConstI32)(a.table + (int64_t)s * a.max_pages);
  // The piece of the tile looked up last: its first key, page (-1: none), codes
  // and scales.  A tile's entry of the table is asked for a tile ahead, and its
  // scales when the page is known, both early in a half step, so that the waits
  // at its end cover them.
  auto entry_of = [&](int tile) -> int { return table[min(tile * KT + 16 * piece, max(keys, 1) - 1) >> shift]; };
  int entry = 0, key = 0, page = -1;
  int64_t base = 0;
  float ks = 0.f, vs = 0.f;
  auto look_up = [&](int tile) {
    key = tile * KT + 16 * piece;
    page = key < keys && entry >= 0 && entry < a.c.n_pages ? entry : -1;
    entry = entry_of(tile + 1);
    const int64_t e = (int64_t)max(page, 0) * a.c.Hkv + hk;
    base = ((e << shift) + (key & pmask)) * D;
    ks = ((ConstF32)a.c.ks)[e];
    vs = ((ConstF32)a.c.vs)[e];
  };
  uint2 kr[NU], vr[NU];
  int v_key = 0, v_page = -1;   // of the values in vr
  auto fetch = [&](const uint8_t* from, uint2(&to)[NU]) {
    const uint8_t* const p = from + base + part * (16 * D / PARTS);
    if constexpr (NU == 1) {
      to[0] = *reinterpret_cast<const uint2*>(p + lane * 8);
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(p + lane * 16);
      to[0] = make_uint2(w.x, w.y);
      to[1] = make_uint2(w.z, w.w);
    }
  };
  auto fetch_values = [&]() {
    v_key = key;
    v_page = page;
    fetch(a.c.v, vr);
  };
  // Values that not every row of the workgroup may see: what lies behind the
  // last key or in a page not held may be anything, and a NaN that a row does
  // not see would get into it as 0 * NaN.  The former become 0; so do NaN
  // values, whose keys then score NaN for the rows that see them.
  auto clean = [&](int tile) {
    if ((tile + 1) * KT <= wg_free && v_page >= 0) return;
    uint32_t found = 0;
#pragma unroll
    for (int x = 0; x < NU; ++x) {
      const int second = NU == 1 ? lane & 1 : x & 1;   // which 8 of the 16 keys
      const int left = (v_page < 0 ? 0 : keys - v_key) - 8 * second;
      vr[x].x = without_nan<I8>(vr[x].x & first_bytes(left), 8 * second, &found);
      vr[x].y = without_nan<I8>(vr[x].y & first_bytes(left - 4), 8 * second + 4, &found);
    }
    if constexpr (!I8) {
#pragma unroll
      for (int d = 32; d; d >>= 1) found |= __shfl_xor(found, d);
      if (lane == 0) nan_keys[tile & 3][wave] = found;
    }
  };
  // The scales as the steps use them: the scores' factor (a number, at least
  // 2^-126: its product with a masked score stays -inf); the values' as a power
  // of two; the inverse of that, or 0 where the piece is not held or its
  // probabilities are summed apart; and the power of two by which the values'
  // is too large, or -1 where the piece is not held.
  auto put_scales = [&](int tile) {
    const float lv = __builtin_amdgcn_logf(page < 0 ? 1.f : fmaxf(vs, kMinScale)) + kUnit;
    if (lane == 0 && part == 0)
      pieces[tile & 3][piece] = page < 0 ? make_float4(1.f, 0.f, 0.f, -1.f)
                                         : make_float4(__builtin_amdgcn_fmed3f(ks * log_scale, 0x1p-126f, kMostFactor), lv,
                                                       lv < kTiny || lv > kHuge ? 0.f : exp2_fast(-lv),
                                                       fmaxf(lv - (kLarge - kLazy), 0.f));
  };
  // LDS addresses of a lane's units of a tile: 8 channels of a key, 8 keys of a channel
  // (of two units: in chunks that differ in their last bit)
  const int put_e = part * (16 * D / PARTS) + lane * NU * 8, put_k = 16 * piece + put_e / D, put_c = put_e / 16;
  const int kput = put_k * D * 2 + (((put_e % D / 8) ^ swizzle_k<D>(put_k)) * 16);
  const int vput = put_c * KT * 2 + (((2 * piece + (put_e >> 3 & 1)) ^ swizzle_v<KT>(put_c)) * 16);
  auto put_keys = [&](int buf, int x) {
    *reinterpret_cast<bf16x8*>(lds + ((kput ^ 16 * x) + buf * BYTES)) = codes_to_operand<I8>(kr[x].x, kr[x].y);
  };
  auto put_values = [&](int buf, int x) {
    *reinterpret_cast<bf16x8*>(vlds + ((vput ^ 16 * x) + buf * BYTES)) = codes_to_operand<I8>(vr[x].x, vr[x].y);
  };

  // ---- operands: even ones 16 channels of 32 keys, odd ones 16 keys of 32 channels ----
  constexpr int OPS = 2 * KB * KS, KA = KS < 8 ? KS : 8;
  static_assert(KB * KS == NP * OB, "as many operands of keys as of values");
  const int krow = 16 * (c32 >> 4) + 8 * ((c32 >> 2) & 1) + 4 * ((c32 >> 3) & 1) + (c32 & 3);
  // Heads of 256 leave no registers for the addresses of every chunk: those are
  // formed from the first one's, by its bits (the others keep them: a vector
  // instruction a product costs more).
  constexpr bool FORM = D == 256;
  int kget[FORM ? 1 : KA], vget[FORM ? 1 : NP];
#pragma unroll
  for (int k = 0; k < (FORM ? 1 : KA); ++k) kget[k] = krow * D * 2 + (((2 * k + h) ^ swizzle_k<D>(krow)) * 16);
#pragma unroll
  for (int u = 0; u < (FORM ? 1 : NP); ++u) vget[u] = c32 * KT * 2 + (((2 * u + h) ^ swizzle_v<KT>(c32)) * 16);
  auto v_at = [&](int u) -> int { return FORM ? vget[0] ^ 32 * u : vget[u]; };
  auto operand = [&](int c, int kbuf, int vbuf) -> bf16x8 {
    if (c & 1) {
      const int x = (c >> 1) / NP, u = (c >> 1) % NP;
      return *reinterpret_cast<const bf16x8*>(vlds + (v_at(u) + vbuf * BYTES + x * 32 * KT * 2));
    }
    const int b = (c >> 1) / KS, k = (c >> 1) % KS;
    return *reinterpret_cast<const bf16x8*>(lds + ((FORM ? kget[0] ^ 32 * (k % KA) : kget[k % KA]) + kbuf * BYTES + b * 32 * D * 2 + k / KA * 256));
  };

  // The waves of one SIMD take turns: while waves 0 - 3 form products, waves
  // 4 - 7 do everything else, and the other way round after a barrier, so the
  // matrix cores and the vector units of a SIMD both have work all the time.
  // (Products dealt out between the vector instructions of one wave overlap
  // worse: 190 ns for 8 products and 56 vector instructions of a SIMD's two
  // waves, against 147 ns in turns; the products alone take 136.)
  //
  // Step t of a wave: the scores of tile t and the products of step t - 1's
  // probabilities with its values, and between them tile t + 2's keys and tile
  // t + 1's values converted; a barrier; the probabilities; a barrier.  Waves
  // 0 - 3 do the first in half step 2 t, waves 4 - 7 in 2 t + 1.  Tile t's keys
  // are read in the half steps 2 t - 1 to 2 t + 1, its values in 2 t + 1 to
  // 2 t + 3 (the first LEAD operands a half step early), and are staged in
  // 2 t - 4 and 2 t - 3, and in 2 t - 2 and 2 t - 1: three buffers of each do.
  auto barrier = [&]() {
    __builtin_amdgcn_sched_barrier(0);   // the halves stay apart
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int LEAD = D == 256 ? 2 : 4;
  bf16x8 x[LEAD];     // the first operands of the next products
  bf16x8 p[NP];       // probabilities
  auto step = [&](auto jc, int tile) {
    constexpr int J = decltype(jc)::value, J1 = (J + 1) % 3, J2 = (J + 2) % 3;   // buffers of tiles t, t + 1 and t - 1 or t + 2
    const int key0 = KT * tile;
    if constexpr (FORM) asm volatile("" : "+v"(kget[0]), "+v"(vget[0]));   // in every step anew
    clean(tile + 1);
    f32x16 sc[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[b][e] = 0.f;
    {
      bf16x8 y[OPS];
#pragma unroll
      for (int c = 0; c < LEAD; ++c) y[c] = x[c];
#pragma unroll
      for (int c = 0; c < OPS; ++c) {
        if (c + LEAD < OPS) y[c + LEAD] = operand(c + LEAD, J, J2);
        const int i = c >> 1;
        if (c & 1) o[i / NP] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y[c], p[i % NP], o[i / NP], 0, 0, 0);
        else sc[i / KS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y[c], q[i % KS], sc[i / KS], 0, 0, 0);
        if (c >= OPS / 2) {   // in the second half: the codes have had time to come
#pragma unroll
          for (int e = (c - OPS / 2) * 2 * NU / (OPS / 2); e < (c + 1 - OPS / 2) * 2 * NU / (OPS / 2); ++e) {
            if (e < NU) put_keys(J2, e);
            else put_values(J1, e - NU);
          }
        }
        __builtin_amdgcn_sched_barrier(0);   // operands stay LEAD ahead
      }
    }
    float4 pc[NP];
#pragma unroll
    for (int u = 0; u < NP; ++u) pc[u] = pieces[tile & 3][u];
    barrier();

    put_scales(tile + 2);
    fetch_values();        // of tile t + 2
    look_up(tile + 3);
    fetch(a.c.k, kr);
    float least = pc[0].z;
#pragma unroll
    for (int u = 1; u < NP; ++u) least = fminf(least, pc[u].z);
    const bool odd = __any(least == 0.f);   // pieces not held, or summed apart
    // (e4m3: for every wave of the tiles that were cleaned, also where its rows
    // all see them: the marks stand for the NaN values taken out)
    if (key0 + KT > (I8 ? w_free : wg_free) || odd) {
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (pc[2 * b + (e >> 3)].w < 0.f || key0 + 32 * b + 16 * (e >> 3) + 8 * h + (e & 7) > last) sc[b][e] = -__builtin_inff();
      if constexpr (!I8) {
        if (key0 + KT > wg_free) {
          uint32_t nan[NP], any = 0;
#pragma unroll
          for (int u = 0; u < NP; ++u) {
            nan[u] = 0;
#pragma unroll
            for (int w = 0; w < PARTS; ++w) nan[u] |= nan_keys[tile & 3][u * PARTS + w];
            any |= nan[u];
            nan[u] >>= 8 * h;
          }
          if (__any(any)) {
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if ((nan[2 * b + (e >> 3)] >> (e & 7) & 1) && sc[b][e] != -__builtin_inff()) sc[b][e] = __builtin_nanf("");
          }
        }
      }
    }
    float mx = -__builtin_inff();
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      float y = sc[u >> 1][8 * (u & 1)];
#pragma unroll
      for (int e = 1; e < 8; ++e) y = fmaxf(y, sc[u >> 1][8 * (u & 1) + e]);
      mx = fmaxf(mx, fmaf(y, pc[u].x, pc[u].w));
    }
    mx = max_halves(mx);
    const bool grow = mx > m + kLazy;
    if (__any(grow)) {
      // the measure is a whole number, so the factor is a power of two and exact
      const float m1 = grow ? ceilf(mx) : m;
      const float again = grow ? exp2_fast(m - m1) : 1.f;
      l *= again;
#pragma unroll
      for (int b = 0; b < OB; ++b) o[b] *= again;
      m = m1;
    }
    const float less = m == -__builtin_inff() ? 0.f : m;
    if (odd) {
#pragma unroll
      for (int u = 0; u < NP; ++u)
        if (pc[u].z == 0.f && pc[u].w >= 0.f) {
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            l = add_pair(pack_bf16(exp2_fast(fmaf(sc[u >> 1][8 * (u & 1) + i], pc[u].x, -less)),
                                   exp2_fast(fmaf(sc[u >> 1][8 * (u & 1) + i + 1], pc[u].x, -less))), l);
        }
    }
    // p times its value's scale, a power of two, rounded to bf16 once; the sum
    // is of the rounded ones, so a row that one key takes is that key's value
    // exactly
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const float off = pc[u].y - less;
      float sum = 0.f;
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s0 = sc[u >> 1][8 * (u & 1) + 2 * i], s1 = sc[u >> 1][8 * (u & 1) + 2 * i + 1];
        w[i] = pack_bf16(exp2_fast(fmaf(s0, pc[u].x, off)), exp2_fast(fmaf(s1, pc[u].x, off)));
        sum = add_pair(w[i], sum);
      }
      l = fmaf(sum, pc[u].z, l);
      asm volatile("" : "+v"(w), "+v"(l));   // formed here, not beside the next products
      p[u] = __builtin_bit_cast(bf16x8, w);
      if (u == NP - 2) {
#pragma unroll
        for (int c = 0; c < LEAD; ++c) x[c] = operand(c, J1, J);
      }
    }
    barrier();
  };

  const int steps = (keys + KT - 1) / KT;
#pragma unroll
  for (int u = 0; u < NP; ++u) p[u] = bf16x8{};
  if (steps > 0) {
    entry = entry_of(0);
    look_up(0);
    fetch(a.c.k, kr);
    fetch_values();
    put_scales(0);
    clean(0);
#pragma unroll
    for (int x = 0; x < NU; ++x) {
      put_keys(0, x);
      put_values(0, x);
      put_values(2, x);   // step 0 multiplies these by probabilities of 0: no NaN of old may be there
    }
    look_up(1);
    fetch(a.c.k, kr);
    fetch_values();       // stay in vr for step 0
    put_scales(1);
#pragma unroll
    for (int x = 0; x < NU; ++x) put_keys(1, x);
    look_up(2);
    fetch(a.c.k, kr);     // stay in kr for step 0
    barrier();
    if (wave >= 4) barrier();
#pragma unroll
    for (int c = 0; c < LEAD; ++c) x[c] = operand(c, 0, 2);
    int t = 0;
    for (; t + 3 <= steps; t += 3) {   // (a way out of its middle would cost registers)
      step(std::integral_constant<int, 0>(), t);
      step(std::integral_constant<int, 1>(), t + 1);
      step(std::integral_constant<int, 2>(), t + 2);
    }
    if (t < steps) step(std::integral_constant<int, 0>(), t);
    if (t + 1 < steps) step(std::integral_constant<int, 1>(), t + 1);
    // the last step's probabilities
    const char* const tail = vlds + (steps - 1) % 3 * BYTES;
#pragma unroll
    for (int c = 0; c < NP * OB; ++c)
      o[c / NP] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          *reinterpret_cast<const bf16x8*>(tail + v_at(c % NP) + c / NP * 32 * KT * 2), p[c % NP], o[c / NP], 0, 0, 0);
    if (wave < 4) barrier();
  }

  // (the row formed again: it would cost registers all the way)
  const int lane1 = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  const int r1 = r0 + (lane1 & 31), i1 = r1 / G;
  if (r1 >= rows) return;
  const float sum = add_halves(l);
  const float inv = bad ? __builtin_nanf("") : m == -__builtin_inff() ? 0.f : exp2_fast(-kUnit) / sum;
  uint16_t* out = a.out + ((int64_t)(i0 + i1) * a.Hq + hk * G + (r1 - i1 * G)) * D + 4 * (lane1 >> 5);
#pragma unroll
  for (int x = 0; x < OB; ++x)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<uint2*>(out + 32 * x + 8 * g) =
          make_uint2(pack_bf16(o[x][4 * g] * inv, o[x][4 * g + 1] * inv),
                     pack_bf16(o[x][4 * g + 2] * inv, o[x][4 * g + 3] * inv));
}

template <int D, bool I8>
hipError_t launch_d(const AttnArgs& a, hipStream_t st) {
  const int64_t units = (int64_t)a.n_tokens * (a.Hq / a.c.Hkv) / kRows + a.n_seqs;
  hipLaunchKernelGGL((attn_packed_kernel<D, I8>), dim3((uint32_t)(units * a.c.Hkv)), dim3(64 * kWaves), 0, st, a, (int)units);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_packed(const AttnArgs& a, hipStream_t st) {
  if (a.few) {
    const hipError_t e = launch_attn_few(a, st);
    if (e != hipSuccess || !a.many) return e;
  }
  switch (a.c.dim) {
    case 64: return a.c.i8 ? launch_d<64, true>(a, st) : launch_d<64, false>(a, st);
    case 128: return a.c.i8 ? launch_d<128, true>(a, st) : launch_d<128, false>(a, st);
    default: return a.c.i8 ? launch_d<256, true>(a, st) : launch_d<256, false>(a, st);
  }
}

}  // namespace gdn
