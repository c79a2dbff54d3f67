// Decode attention over the paged 8-bit cache: few query rows per request, the
// whole cache read once, so HBM bounds it.
//
// The rows of a request that share a kv head (n_tok tokens x Hq / Hkv heads)
// are packed into tiles of 16.  A wave takes 64 keys at a time (or 32, with 8 a
// lane group below) straight from the pages into registers, with no LDS between:
//   S^T = K Q^T   (16x16x32 products, rows = keys, columns = query rows)
//   O^T += V^T P^T  (rows = channels, columns = query rows).
// A product's result holds in lane group g (16 lanes) the rows 4g .. 4g + 3 of
// every column, and its second operand wants in lane group g the eight
// contraction indices 8g .. 8g + 7 of the column.  The order of keys is free,
// so row 4g + i of score tile s is key 16 g + 4 s + i of the 64: then group g
// has, over the four score tiles, exactly the keys 16 g .. 16 g + 15, which is
// one 16-byte vector of the cache's transposed value tile, and the
// probabilities go from one product into the next without leaving their lane.
//
// Measured: 32 requests of 17 to 8,192 keys, 8 kv heads of 128, e4m3: 64 us,
// 4.1 TB/s of codes (a large copy moves 4.9 TB/s); 16 of 4,096 to 32,768 keys
// with 4 tokens each, 2 kv heads of 256, int8: 104 us, 2.9 TB/s.  There 32 rows
// of sums leave one wave a SIMD, whose conversions (45 % of its cycles) do not
// overlap its waits; partial sums of up to 22 splits are written and read again,
// 9 us of it in the join's own launch.  Workgroups of splits that a request does
// not have leave once they know its length: a bound of 4 times the lengths costs
// nothing measurable, one of 16 times 22 us of the 55 (the first batch) and 9 of
// the 103 (the second).
//
// Keys are split over workgroups in runs of fixed length (split_keys), the
// four waves of a workgroup take tiles in turn, and partial results
// (fp32 sums against the running maximum) are joined in a fixed order, so a
// request's bits do not depend on its batch.
#include <algorithm>
#include <type_traits>

#include "attn_device.h"

namespace gdn {
namespace {

constexpr int kWaves = 4;

// Keys per workgroup: by the head size alone, so that how a request's keys are
// split never depends on its batch.  Fewer make more partial sums to write and
// join, more leave the last workgroups to run alone, or a short request to few
// workgroups: no length is best for all.  Measured, 2 kv heads of 256 (512, 768,
// 1,024, 1,536, 2,048 keys, in us):
//   16 requests of 4,096 to 32,768 keys, 4 tokens  138  130  118  102  119
//   the same, 1 token                               84   77   79   64   78
//   32 requests of 17 to 8,192                      42   35   39   48   45
//   one of 8,192                                    23   26   29   37   44
// 4 kv heads of 256: the long batch of 1 token 150, 134, 130, 129 and 146, the
// batch to 8,192 60, 58, 62, 56 and 63.  8 of 128 (512, 768, 1,024, 2,048): 149,
// 130, 131 and 127, 60, 58, 55 and 60, one of 8,192 keys 17, 18, 19 and 26.
__host__ __device__ constexpr int split_keys(int dim) { return dim == 256 ? 1536 : 1024; }
__host__ __device__ inline int n_splits(int L, int dim) { return L <= 0 ? 1 : (L - 1) / split_keys(dim) + 1; }

struct Partial {
  float* o;    // [B][splits][n_tok * Hq][D]
  float2* ml;  // [B][splits][n_tok * Hq] maximum (of log2 scores), sum
  int splits;
};

template <int D, bool I8, int NT, bool PACKED>
__global__ void __launch_bounds__(64 * kWaves, D == 64 ? 5 - NT : NT * D <= 256 ? 2 : 1) attn_decode_kernel(const AttnArgs a, const Partial part) {
  // Keys of a tile: 64, so that a lane's values are whole vectors; 32 where that
  // lets two waves into a SIMD (32 requests to 8,192 keys, 4 kv heads of 256:
  // 67 us, with 64 a few registers spill and it takes 72).
  constexpr int KT = D == 256 && NT == 1 ? 32 : 64;
  constexpr int KG = KT / 4;    // keys of a lane group
  constexpr int NS = KT / 16;   // score tiles
  constexpr int KL = D / 64;    // 16-byte loads of a key per lane
  constexpr int KS = D / 32;    // contraction steps of a score
  constexpr int OB = D / 16;    // 16-channel blocks of the output
  // Workgroups go to the eight XCDs in turn: heads first, then requests, then
  // splits, and the requests one further on with every split, so that neither
  // the first splits nor a long request's all go to one of them (16 requests of
  // 4,096 to 32,768 keys, 2 kv heads of 256: 114 us, without the turn 155).
  // In a pack (z: more prompts) a workgroup takes all keys of its rows.
  const int sp = PACKED ? 0 : blockIdx.z;
  const int b = PACKED ? (int)(blockIdx.y + blockIdx.z * gridDim.y) : (int)((blockIdx.y + blockIdx.z) % gridDim.y);
  if (PACKED && b >= a.n_seqs) return;
  const int G = a.Hq / a.c.Hkv;
  const int tok0 = PACKED ? a.cu[b] : b * a.n_tok, n_tok = PACKED ? min(a.cu[b + 1], a.n_tokens) - tok0 : a.n_tok;
  if (PACKED && (tok0 < 0 || n_tok < 1 || n_tok > few_rows(D) / G)) return;
  const int R = n_tok * G;
  const int groups = ((PACKED ? a.few * G : R) + 16 * NT - 1) / (16 * NT);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c16 = lane & 15, g = lane >> 4;
  const int hk = blockIdx.x / groups, r0 = (blockIdx.x % groups) * 16 * NT;
  if (PACKED && r0 >= R) return;
  const int shift = a.c.page_shift, pmask = (1 << shift) - 1;
  const int32_t* table = a.table + (int64_t)b * a.max_pages;
  constexpr int kStep = kWaves * KT;
  const int key0 = sp * split_keys(D);
  // the first tile's entries do not wait for the length
  int t0 = key0 + wave * KT;
  auto entry_of = [&](int key) -> int { return a.max_pages > 0 ? table[min(key >> shift, a.max_pages - 1)] : -1; };
  const int ek = entry_of(t0 + KG * (c16 >> 2)), ev = entry_of(t0 + KG * g);
  const int ek1 = entry_of(t0 + kStep + KG * (c16 >> 2)), ev1 = entry_of(t0 + kStep + KG * g);
  const int L = a.kv_len[b];
  const bool bad = L < 0 || L > a.max_kv;
  const int splits = bad || PACKED ? 1 : n_splits(L, D);
  if (sp >= splits) return;

  // this lane's column: its query row per tile, and the last key that it sees
  auto row_of = [&](int t) -> int { return min(r0 + 16 * t + c16, R - 1); };
  int last[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) last[t] = L - n_tok + row_of(t) / G;
  if (bad || L == 0) {
    for (int e = tid; e < 16 * NT * D; e += 64 * kWaves) {
      const int r = r0 + e / D;
      if (r < R) {
        const int i = r / G;
        a.out[((int64_t)(tok0 + i) * a.Hq + hk * G + (r - i * G)) * D + e % D] = bad ? 0x7FC0 : 0;
      }
    }
    return;
  }

  // Queries: in registers, or in LDS (the same for every wave) where the
  // registers are needed for the codes in flight.
  constexpr bool QL = NT * D >= 256;
  constexpr int QN = QL ? NT * KS / kWaves : NT * KS;
  __shared__ union {
    bf16x8 q[QL ? NT * KS : 1][64];
    f32x4 o[kWaves][NT * OB][64];
  } lds;
  auto& ql = lds.q;
  bf16x8 q[QN];
#pragma unroll
  for (int n = 0; n < QN; ++n) {
    const int e = QL ? n * kWaves + wave : n, t = e / KS, k = e % KS, r = row_of(t), i = r / G;
    const uint16_t* p = a.q + (tok0 + i) * a.q_stride + (hk * G + (r - i * G)) * D + 16 * g;
    q[n] = *reinterpret_cast<const bf16x8*>(p + 64 * (k >> 1) + 8 * (k & 1));
  }
  auto query = [&](int t, int k) -> bf16x8 {
    if constexpr (QL) return ql[t * KS + k][lane];
    else return q[t * KS + k];
  };

  const int key1 = PACKED ? L : min(L, key0 + split_keys(D));
  const float log_scale = a.scale * kLog2e;

  // A tile's pages: of the keys whose values (and scores) this lane has, and
  // of the key whose codes it loads (-1: not held, read as page 0 and masked).
  auto page_of = [&](int entry, int key) -> int { return key < key1 && entry < a.c.n_pages ? entry : -1; };
  typedef std::conditional_t<KT == 64, uint4, uint2> Values;   // a lane's KG keys of a channel
  uint4 kc[NS][KL];
  Values vc[OB];
  float ks, vs;
  auto load_keys = [&](int t0, int pk, int pv) {
    const int kk = t0 + KG * (c16 >> 2);
    const uint8_t* kp = a.c.k + page_base(a.c, max(pk, 0), hk) + ((kk & pmask) + (c16 & 3)) * D + 16 * g;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int i = 0; i < KL; ++i) kc[s][i] = *reinterpret_cast<const uint4*>(kp + 4 * s * D + 64 * i);
    ks = a.c.ks[(int64_t)max(pv, 0) * a.c.Hkv + hk];
  };
  auto load_values = [&](int t0, int pv) {
    const int kv = t0 + KG * g;
    const uint8_t* vp = a.c.v + page_base(a.c, max(pv, 0), hk) + ((kv & pmask & ~15) * D + c16 * 16 + (kv & 15));
#pragma unroll
    for (int x = 0; x < OB; ++x) vc[x] = *reinterpret_cast<const Values*>(vp + x * 256);
    vs = a.c.vs[(int64_t)max(pv, 0) * a.c.Hkv + hk];
  };

  // Loads run ahead: a tile's keys are asked for when the scores before them
  // are done, its values after the products before them, its pages a tile
  // earlier.
  int pv = page_of(ev, t0 + KG * g);
  int pk1 = page_of(ek1, t0 + kStep + KG * (c16 >> 2)), pv1 = page_of(ev1, t0 + kStep + KG * g);
  if (t0 < key1) {
    load_keys(t0, page_of(ek, t0 + KG * (c16 >> 2)), pv);
    load_values(t0, pv);
  }
  if constexpr (QL) {
#pragma unroll
    for (int n = 0; n < QN; ++n) ql[n * kWaves + wave][lane] = q[n];
    __syncthreads();
  }
  f32x4 o[NT][OB];
  float m[NT], l[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = -__builtin_inff();
    l[t] = 0.f;
#pragma unroll
    for (int x = 0; x < OB; ++x) o[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  for (; t0 < key1; t0 += kStep) {
    const bool more = t0 + kStep < key1;
    const int kk2 = t0 + 2 * kStep + KG * (c16 >> 2), kv2 = t0 + 2 * kStep + KG * g;
    const int pk2 = page_of(table[min(kk2, key1 - 1) >> shift], kk2), pv2 = page_of(table[min(kv2, key1 - 1) >> shift], kv2);
    const int kv = t0 + KG * g;
    const bool held = pv >= 0;

    f32x4 s4[NT][NS];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int s = 0; s < NS; ++s) s4[t][s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KL; ++i) {
      bf16x8 q0[NT], q1[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        q0[t] = query(t, 2 * i);
        q1[t] = query(t, 2 * i + 1);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const bf16x8 k0 = codes_to_operand<I8>(kc[s][i].x, kc[s][i].y);
        const bf16x8 k1 = codes_to_operand<I8>(kc[s][i].z, kc[s][i].w);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          s4[t][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q0[t], s4[t][s], 0, 0, 0);
          s4[t][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q1[t], s4[t][s], 0, 0, 0);
        }
      }
    }
    const float kf = __builtin_amdgcn_fmed3f(ks * log_scale, -kMostFactor, kMostFactor);
    __builtin_amdgcn_sched_barrier(0);
    if (more) load_keys(t0 + kStep, pk1, pv1);
    __builtin_amdgcn_sched_barrier(0);

    // codes behind the last key (or of a page not held) may be anything, NaN
    // among them, which a probability of 0 would not silence; so would a NaN
    // value that only some rows see: it becomes 0, and its key's score NaN for
    // the rows that see it
    const bool whole = t0 + KT <= key1 - (n_tok - 1);   // every row sees the tile
    uint32_t nan = 0;
    if (!whole || __any(!held)) {
      const int left = held ? key1 - kv : 0;
#pragma unroll
      for (int x = 0; x < OB; ++x) {
        vc[x].x = without_nan<I8>(vc[x].x & first_bytes(left), 0, &nan);
        vc[x].y = without_nan<I8>(vc[x].y & first_bytes(left - 4), 4, &nan);
        if constexpr (KT == 64) {
          vc[x].z = without_nan<I8>(vc[x].z & first_bytes(left - 8), 8, &nan);
          vc[x].w = without_nan<I8>(vc[x].w & first_bytes(left - 12), 12, &nan);
        }
      }
      if constexpr (!I8)
#pragma unroll
        for (int d = 8; d; d >>= 1) nan |= __shfl_xor(nan, d);
    }

    // scores to probabilities; in units of log2
    const float vf = held ? vs : 0.f, over = fmaxf(__builtin_amdgcn_logf(vf) - kLarge, 0.f);
    bf16x8 p[NT][NS / 2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float mx = -__builtin_inff();
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s4[t][s][i] * kf;
          if (!I8 && (nan >> (4 * s + i) & 1)) x = __builtin_nanf("");
          if (!held || (!whole && kv + 4 * s + i > last[t])) x = -__builtin_inff();
          s4[t][s][i] = x;
          mx = fmaxf(mx, x);
        }
      mx += over;
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float m1 = fmaxf(m[t], mx);
      const float base = m1 == -__builtin_inff() ? 0.f : m1;
      if (__any(m1 > m[t])) {
        const float again = exp2_fast(m[t] - base);
        l[t] *= again;
#pragma unroll
        for (int x = 0; x < OB; ++x) o[t][x] *= again;
        m[t] = m1;
      }
      u32x4 w[NS / 2];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = exp2_fast(s4[t][s][i] - base);
          l[t] += e[i];
          e[i] *= vf;   // the probability times its value's scale is rounded to bf16 once
        }
        w[s >> 1][2 * (s & 1)] = pack_bf16(e[0], e[1]);
        w[s >> 1][2 * (s & 1) + 1] = pack_bf16(e[2], e[3]);
      }
#pragma unroll
      for (int u = 0; u < NS / 2; ++u) p[t][u] = __builtin_bit_cast(bf16x8, w[u]);
    }
#pragma unroll
    for (int x = 0; x < OB; ++x) {
      const bf16x8 v0 = codes_to_operand<I8>(vc[x].x, vc[x].y);
#pragma unroll
      for (int t = 0; t < NT; ++t) o[t][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, p[t][0], o[t][x], 0, 0, 0);
      if constexpr (KT == 64) {
        const bf16x8 v1 = codes_to_operand<I8>(vc[x].z, vc[x].w);
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, p[t][1], o[t][x], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (more) load_values(t0 + kStep, pv1);
    pk1 = pk2;
    pv = pv1;
    pv1 = pv2;
  }

  // The waves' sums meet in LDS, each against the common maximum; then each
  // wave adds up a quarter of the 16 x 16 blocks, in the waves' order.
  __shared__ float sm[kWaves][16 * NT], sl[kWaves][16 * NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l[t] += __shfl_xor(l[t], 16);
    l[t] += __shfl_xor(l[t], 32);
    if (g == 0) {
      sm[wave][16 * t + c16] = m[t];
      sl[wave][16 * t + c16] = l[t];
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float mt = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mt = fmaxf(mt, sm[w][16 * t + c16]);
    const float mine = m[t] == -__builtin_inff() ? 0.f : exp2_fast(m[t] - mt);
#pragma unroll
    for (int x = 0; x < OB; ++x) lds.o[wave][t * OB + x][lane] = o[t][x] * mine;
  }
  __syncthreads();
#pragma unroll 1
  for (int n = wave; n < NT * OB; n += kWaves) {
    const int t = n / OB, c = 16 * (n % OB) + 4 * g, r = r0 + 16 * t + c16;
    f32x4 y = lds.o[0][n][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) y += lds.o[w][n][lane];
    float mt = -__builtin_inff(), lt = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mt = fmaxf(mt, sm[w][16 * t + c16]);
    const float base = mt == -__builtin_inff() ? 0.f : mt;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) lt += sl[w][16 * t + c16] * exp2_fast(sm[w][16 * t + c16] - base);
    if (r >= R) continue;
    const int i = r / G;
    const int64_t row = (int64_t)(tok0 + i) * a.Hq + hk * G + (r - i * G);
    if (splits == 1) {
      const float inv = mt == -__builtin_inff() ? 0.f : 1.f / lt;
      *reinterpret_cast<uint2*>(a.out + row * D + c) = make_uint2(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv));
    } else {
      const int rows = a.n_tok * a.Hq;
      const int64_t pr = row + ((int64_t)b * (part.splits - 1) + sp) * rows;   // [b][split][row of the request]
      *reinterpret_cast<f32x4*>(part.o + pr * D + c) = y;
      if (c == 0) part.ml[pr] = make_float2(mt, lt);
    }
  }
}

// Joins the splits of one row, in order: lanes take the splits' maxima and
// sums at once, then all channels of each split.
template <int D>
__global__ void __launch_bounds__(64) attn_join_kernel(const AttnArgs a, const Partial part) {
  const int rows = a.n_tok * a.Hq;
  const int b = (int)(blockIdx.x / rows), r = (int)(blockIdx.x % rows), lane = threadIdx.x;
  const int L = a.kv_len[b];
  if (L < 0 || L > a.max_kv) return;
  const int splits = n_splits(L, D);
  if (splits == 1) return;
  constexpr int C = D / 64;
  const int64_t p0 = (int64_t)b * part.splits * rows + r;
  float mt = -__builtin_inff();
  for (int s = lane; s < splits; s += 64) mt = fmaxf(mt, part.ml[p0 + (int64_t)s * rows].x);
#pragma unroll
  for (int d = 32; d; d >>= 1) mt = fmaxf(mt, __shfl_xor(mt, d));
  const float base = mt == -__builtin_inff() ? 0.f : mt;
  float o[C] = {}, l = 0.f;
  for (int s0 = 0; s0 < splits; s0 += 64) {
    float w = 0.f, lw = 0.f;
    if (s0 + lane < splits) {
      const float2 ml = part.ml[p0 + (int64_t)(s0 + lane) * rows];
      w = exp2_fast(ml.x - base);
      lw = w * ml.y;
    }
    const int n = min(64, splits - s0);
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
      const float ws = __shfl(w, s);
      l += __shfl(lw, s);
      const float* const from = part.o + (p0 + (int64_t)(s0 + s) * rows) * D + C * lane;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] += ws * from[c];
    }
  }
  const float inv = mt == -__builtin_inff() ? 0.f : 1.f / l;
  uint16_t* const out = a.out + ((int64_t)b * rows + r) * D + C * lane;
#pragma unroll
  for (int c = 0; c < C; ++c) out[c] = (uint16_t)pack_bf16(o[c] * inv, 0.f);
}

template <int D, bool I8>
hipError_t launch_d(const AttnArgs& a, const Partial& part, hipStream_t st) {
  const int R = a.n_tok * (a.Hq / a.c.Hkv);
  // Two tiles of rows a wave where there are more than one: they share the
  // codes' conversion (32 rows, 2 kv heads of 128, 16 x 4,096 .. 32,768 keys:
  // 59 us, with one tile a wave 69).  Four leave room for one wave a SIMD only,
  // which loses more than it saves (64 rows of 128: 83 us, with four 113).
  const int nt = R <= 16 ? 1 : 2;
  const dim3 grid(a.c.Hkv * ((R + 16 * nt - 1) / (16 * nt)), a.n_seqs, part.splits), block(64 * kWaves);
  if (nt == 1) hipLaunchKernelGGL((attn_decode_kernel<D, I8, 1, false>), grid, block, 0, st, a, part);
  else hipLaunchKernelGGL((attn_decode_kernel<D, I8, 2, false>), grid, block, 0, st, a, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || part.splits == 1) return e;
  hipLaunchKernelGGL((attn_join_kernel<D>), dim3((uint32_t)(a.n_seqs * a.n_tok * a.Hq)), dim3(64), 0, st, a, part);
  return hipGetLastError();
}

template <int D, bool I8>
hipError_t launch_few_d(const AttnArgs& a, hipStream_t st) {
  const int R = a.few * (a.Hq / a.c.Hkv), nt = few_tiles(D, R);
  const int y = std::min(a.n_seqs, 32768);
  const dim3 grid(a.c.Hkv * ((R + 16 * nt - 1) / (16 * nt)), y, (a.n_seqs + y - 1) / y), block(64 * kWaves);
  const Partial none{};
  if (nt == 1) hipLaunchKernelGGL((attn_decode_kernel<D, I8, 1, true>), grid, block, 0, st, a, none);
  else if constexpr (D < 256) hipLaunchKernelGGL((attn_decode_kernel<D, I8, 2, true>), grid, block, 0, st, a, none);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_few(const AttnArgs& a, hipStream_t st) {
  switch (a.c.dim) {
    case 64: return a.c.i8 ? launch_few_d<64, true>(a, st) : launch_few_d<64, false>(a, st);
    case 128: return a.c.i8 ? launch_few_d<128, true>(a, st) : launch_few_d<128, false>(a, st);
    default: return a.c.i8 ? launch_few_d<256, true>(a, st) : launch_few_d<256, false>(a, st);
  }
}

int attn_decode_splits(int dim, int max_kv) { return n_splits(max_kv, dim); }

int64_t attn_decode_bytes(int dim, int Hq, int batch, int n_tok, int max_kv) {
  const int64_t s = n_splits(max_kv, dim);
  return s == 1 ? 0 : s * batch * n_tok * Hq * (dim + 2) * 4;
}

hipError_t launch_attn_decode(const AttnArgs& a, void* workspace, hipStream_t st) {
  Partial part{static_cast<float*>(workspace), nullptr, n_splits(a.max_kv, a.c.dim)};
  part.ml = reinterpret_cast<float2*>(part.o + (int64_t)a.n_seqs * part.splits * a.n_tok * a.Hq * a.c.dim);
  switch (a.c.dim) {
    case 64: return a.c.i8 ? launch_d<64, true>(a, part, st) : launch_d<64, false>(a, part, st);
    case 128: return a.c.i8 ? launch_d<128, true>(a, part, st) : launch_d<128, false>(a, part, st);
    default: return a.c.i8 ? launch_d<256, true>(a, part, st) : launch_d<256, false>(a, part, st);
  }
}

}  // namespace gdn
