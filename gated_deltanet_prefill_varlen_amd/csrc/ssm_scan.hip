// Packed scan of the state space layers on the matrix cores, in chunks of 32
// tokens.  With cum_t = sum of A dt up to token t of a chunk, S0 the state
// that enters it, L its last token:
//
//   y_t = exp(cum_t) S0 C_t + sum_{s <= t} M_ts x_s + D x_t,
//         M_ts = exp(cum_t - cum_s) dt_s (C_t . B_s)
//   S   = exp(cum_L) S0 + sum_s w_s x_s B_s^T,  w_s = exp(cum_L - cum_s) dt_s
//
// Three launches (the second only where a prompt is cut into segments):
//  1. prepare: per chunk and group the convolved B and C as fp16 operands laid
//     out as the products read them, and the products C . B; per chunk and
//     head the steps, their running sums and the weights w.
//  2. segments: long prompts on few heads would leave most of the chip idle
//     behind the chain of their chunks, so their chunks are dealt to segments
//     by a rule on the prompt's own length; each segment's state from zero,
//     then the states that enter the segments, one after the other.
//  3. scan: a workgroup walks the chunks of a segment for 128 / P heads of one
//     group, one wave per 32 channels of a head, S^T in accumulators.
//
// Precision.  States come back in fp32 and are held to it: x w and B enter
// their product as fp16 pairs hi + lo (hi hi + hi lo + lo hi: 2^-21).  What only
// ends in the bf16 outputs (M, x, C, S as operands) is fp16 once, 2^-11 of the
// value.  fp16's range is met by powers of two: per token on C and, for the state,
// on B (which x w takes back), per chunk on B in C . B, per chunk and channel on x and
// x w, and per channel on S, by a bound of its largest entry that is carried along.
// Below them fp16's smallest step is felt.  Half of it is at most, of x, 2^-28 of its
// channel's largest in the chunk; of x w, 2^-29 of its channel's largest with its
// token's largest B; of B for the state, 2^-38 of its token's largest; of S, 2^-27 of
// its bound; and of the weights M, with the products C . B and their operands,
// 2^-28 of the largest C of the token, B of the chunk and step (as far as it is
// left at the token) together.  A channel's x, as an operand, and its state, as an
// accumulator, lie in the same lanes, so a channel's scale never leaves them but
// for the outputs.  Values below 2^-100 and decays below 2^-126 may count as 0.
//
// Measured: 32 x 1,024 tokens of 64 heads of 64 on 128 with the convolution (0.63
// GB) 305 us, prepare 32 of them; 4 x 8,192 tokens of 32 heads of 128 on 128 in 16
// groups (0.82 GB) 485 us: prepare 114, segments 128 + 19.  Bound by the vector
// instructions of the scan, 715 a wave and chunk beside 68 products, on two waves
// a SIMD (189 registers); a third wave's 168 would spill into the loop.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "cache_device.h"
#include "ssm_device.h"

namespace gdn {
namespace {

constexpr int kChunk = 32;
constexpr int kTab = 128;                 // floats of a (chunk, head)'s table: dt, cum, w, scalars, 32 powers as int8
constexpr int kTiles = 3;                 // 16 x 16 tiles of C . B on and below the diagonal
// Powers of two that the largest values are brought to: B of a token for the state
// and of a chunk for C . B (and S, where the products of x w and B fill it), C of a
// token, and the products C . B, whose sums over N stay below 2^(kTopB + kTopC + 7).
constexpr int kTopB = 14, kTopS = 30, kTopS16 = 14, kTopC = 14, kTopCB = 15, kCB = kTopB + kTopC + 7 - kTopCB;
constexpr int kPlainX = 11;               // x as it is used where no channel asks for another power: below 2^4
constexpr float kLog2e = 1.44269504088896341f;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 mma(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

__device__ __forceinline__ f16x2 pack_f16(float a, float b) { return __builtin_convertvector(f32x2{a, b}, f16x2); }

// x < 2^pow2_above(x) for finite x >= 0; -100 at least.
__device__ __forceinline__ int pow2_above(float x) { return max((int)(__float_as_uint(x) >> 23 & 0xFF) - 126, -100); }

// Whether one of two values >= 0 lies below `low`, other than 0 itself.
__device__ __forceinline__ bool small_but_not_0(const float (&x)[2], float low) {
  return min(__float_as_uint(x[0]) - 1u, __float_as_uint(x[1]) - 1u) < __float_as_uint(low) - 1u;
}

// x of another lane.
__device__ __forceinline__ int from_lane(int x, int src) { return __builtin_amdgcn_ds_bpermute(src << 2, x); }
__device__ __forceinline__ float from_lane(float x, int src) { return __int_as_float(from_lane(__float_as_int(x), src)); }
// A value that the compiler takes for a new one: what is computed from it in a
// rare path stays there, instead of in registers over the whole loop.
__device__ __forceinline__ int anew(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

template <typename Op>
__device__ __forceinline__ float over_half(float x, Op op) {
  x = op(x, dpp_f32<0xB1>(x));
  x = op(x, dpp_f32<0x4E>(x));
  x = op(x, dpp_f32<0x141>(x));
  x = op(x, dpp_f32<0x140>(x));
  return op(x, __shfl_xor(x, 16));
}
struct MaxOp { __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); } };
// The largest of values >= 0, by their bits: over the lane groups (the lanes that
// hold the same channels), and over a wave of what is the same in its lane groups.
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float over_groups(float v) {
  uint32_t x = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return __uint_as_float(max((uint32_t)b[0], (uint32_t)b[1]));
}
__device__ __forceinline__ float over_wave16(float v) {
  return __uint_as_float(max_dpp<0x140>(max_dpp<0x141>(max_dpp<0x4E>(max_dpp<0xB1>(__float_as_uint(v))))));
}

// ------------------------------------------------------------ the layout --
// Chunk c of prompt s has slot cu[s] / 32 + s + c: no two chunks share one,
// and none passes n_tokens / 32 + n_seqs.  Segments alike, by 256 tokens.
struct Ws {
  char* bc;              // [slots][G]: C operands, B^T hi, B^T lo (32 N halves each)
  _Float16* gt;          // [slots][G][4][64][4]: the tiles of C . B on and below the diagonal; in place of the
                         // fourth kb, the power of two on the chunk's B, and per token (from the 32nd dword on)
                         // that on C and (from the 64th on) 2^(kb - that on B), which stands with x w
  float* tab;            // [slots][H][kTab]
  float* seg;            // [segment slots][H][P][N]
  float* seg_sum;        // [segment slots][H]: log2 of the segment's decay
  int32_t slots, seg_slots;
  int64_t bytes;
};

constexpr int kSegUnit = 8;               // chunks a segment has at least

// Chunks of a segment for a prompt of nc chunks whose chunk row takes hb
// workgroups: as many segments as make 256 workgroups of the prompt alone, where
// it has more than 40 chunks.  The rule looks at one prompt, so that its bits do
// not depend on the pack, and stands between a lone prompt, which gains, and many,
// which pay for states that they did not need early.
// The 40: from there on a lone prompt gains more than 32 at once lose.  Uncut and
// cut, us, of 64 heads of 64 on 128, and of 32 heads of 128 in 16 groups:
//   tokens      768      1,024      1,280       1,536       2,048
//   1 prompt    89 / 70  115 / 72   140 / 73    166 / 75    217 / 80
//   32          242 / 590  313 / 589  390 / 793   458 / 886   599 / 1211
//   1 prompt    76 / 60  99 / 63    120 / 65    140 / 67    182 / 70
//   32          263 / 440  348 / 594  433 / 755   521 / 931   685 / 1260
// The 256: with 128 and 512 in its place, 32 heads of 128 in 16 groups, one prompt
// of 8,192 tokens takes 311 and 147 us for 191, four take 487 and 534 for 483; one
// of 2,048 takes 96 and 69 for 69, sixteen take 509 and 611 for 609.
__host__ __device__ inline int seg_chunks(int nc, int hb) {
  if (nc <= 40) return nc > 0 ? nc : 1;
  const int want = (256 + hb - 1) / hb, most = nc / kSegUnit, n = want < most ? want : most;
  return (nc + n - 1) / n;
}

inline int64_t up(int64_t x) { return (x + 255) / 256 * 256; }

inline Ws layout(const SsmLayer& l, int32_t n_seqs, int64_t n_tokens, bool split, void* base) {
  Ws w{};
  w.slots = (int32_t)(n_tokens / kChunk + n_seqs);
  w.seg_slots = split ? (int32_t)(n_tokens / (kChunk * kSegUnit) + n_seqs) : 0;
  char* p = static_cast<char*>(base);
  int64_t at = 0;
  auto take = [&](int64_t bytes) { const int64_t here = at; at += up(bytes); return p + here; };
  const int64_t sg = (int64_t)w.slots * l.G;
  w.bc = take(sg * 3 * kChunk * l.N * 2);
  w.gt = reinterpret_cast<_Float16*>(take(sg * 4 * 256 * 2));
  w.tab = reinterpret_cast<float*>(take((int64_t)w.slots * l.H * kTab * 4 + 512));
  w.seg = reinterpret_cast<float*>(take((int64_t)w.seg_slots * l.H * l.P * l.N * 4));
  w.seg_sum = reinterpret_cast<float*>(take((int64_t)w.seg_slots * l.H * 4));
  w.bytes = at;
  return w;
}

// Heads of a workgroup: 128 / P (four waves), or the largest power of two below
// it that divides a group's heads.
inline int heads_per_group(const SsmLayer& l) { return l.H / l.G; }
inline int heads_per_wg(const SsmLayer& l) {
  int n = 128 / l.P;
  while (heads_per_group(l) % n != 0) n /= 2;
  return n;
}

inline int max_segments(const SsmLayer& l, int32_t n_seqs, const int32_t* cu) {
  const int hb = l.H / heads_per_wg(l);
  int most = 1;
  for (int s = 0; s < n_seqs; ++s) {
    const int nc = (cu[s + 1] - cu[s] + kChunk - 1) / kChunk, per = seg_chunks(nc, hb);
    most = std::max(most, (nc + per - 1) / per);
  }
  return most;
}

// The prompt s that owns slot b where prompt s begins at cu[s] / unit + s.
__device__ __forceinline__ int owner(const int32_t* cu_ptr, int n_seqs, int unit, int b) {
  typedef const int32_t __attribute__((address_space(4)))* ConstI32;
  const ConstI32 cu = (ConstI32)cu_ptr;
  int lo = 0, hi = n_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] / unit + mid <= b) lo = mid; else hi = mid;
  }
  return lo;
}

// The order of sums.  A product of 32 takes 8 elements from each lane group g.
// Over a chunk's tokens, element j is token slot_of(g, j): the rows that the two
// accumulator tiles of 16 hold in the lane group.  Over N, it is column
// 32 ks + 8 g + j, where row r of the tile 2 ks + q of S^T is column 32 ks + 2 r +
// q: element j lies in tile j % 2, so an accumulator of S^T is an operand too,
// rows of C are read as they lie, and a lane's entries of S are 8 in a row.
__device__ __forceinline__ constexpr int slot_of(int g, int j) { return 16 * (j / 4) + 4 * g + j % 4; }

// ---------------------------------------------------------------- inputs --
// What a wave keeps of a chunk's inputs: the two channels 2 r, 2 r + 1 of its 32
// in one dword, at the tokens of its lane group (runs of four: 16 run + 4 g ..)
// and the three before each run.
struct RawX { uint32_t v[2][7]; };

// Where a wave's inputs lie.
struct XRef {
  const uint16_t* x;       // the prompt's first row
  const uint16_t* hist;    // the prompt's window [3][conv_dim], or nullptr
  int64_t stride;
  int conv_dim, len, ch0;  // ch0: this lane's first channel
};

// Rows past the prompt's end read as 0 by the buffer's range check, as do the
// ones before its start, whose place the window takes.
template <bool CONV>
__device__ __forceinline__ void load_x(const XRef& f, int c, int g, RawX& x) {
  uint32_t row = (uint32_t)f.stride * 2;
  asm volatile("" : "+s"(row));   // (offsets kept over the chunks would take 28 registers)
  const __amdgpu_buffer_rsrc_t buf = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(f.x + (int64_t)(c * kChunk - 3) * f.stride), 0, (min(f.len - c * kChunk, kChunk) + 3) * row, 0x00020000);
  const bool before = c == 0 && g == 0;
#pragma unroll
  for (int i = CONV ? 0 : 3; i < 7; ++i) {
    const uint32_t at = (4 * g + i) * row + 2 * f.ch0;
    x.v[0][i] = __builtin_amdgcn_raw_buffer_load_b32(buf, i < 3 && before ? 0xFFFFFFF0u : at, 0, 0);
#pragma unroll
    for (int run = 1; run < 2; ++run) x.v[run][i] = __builtin_amdgcn_raw_buffer_load_b32(buf, at + 16 * run * row, 0, 0);
  }
  if (CONV && c == 0 && f.hist) {
    const uint16_t* p = f.hist + anew(f.ch0);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (g == 0) x.v[0][i] = *reinterpret_cast<const uint32_t*>(p + (int64_t)i * f.conv_dim);
  }
}

// The convolution of a channel pair, times 2^POW2; v[q][run][i]: channel 2 r + q
// at token 16 run + 4 g + i.
struct ConvW { float w0[2], w1[2], w2[2], w3[2], b[2]; };
template <bool CONV, int POW2 = 0>
__device__ __forceinline__ void conv_run(const uint32_t (&x)[7], const ConvW& k, float (&v0)[4], float (&v1)[4]) {
  float in[2][7];
#pragma unroll
  for (int i = CONV ? 0 : 3; i < 7; ++i) { in[0][i] = lo_bf16(x[i]); in[1][i] = hi_bf16(x[i]); }
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      (q ? v1 : v0)[i] = CONV ? conv4_bias_silu<POW2>(k.b[q], k.w0[q], k.w1[q], k.w2[q], k.w3[q], in[q][i], in[q][i + 1], in[q][i + 2], in[q][i + 3])
                              : POW2 == 0 ? in[q][i + 3] : in[q][i + 3] * (float)(1 << POW2);
}

__device__ __forceinline__ void load_conv(const SsmLayer& l, int ch, ConvW& k) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float4 t = reinterpret_cast<const float4*>(l.conv_w)[ch + q];
    k.w0[q] = conv_tap(t.x); k.w1[q] = conv_tap(t.y); k.w2[q] = conv_tap(t.z); k.w3[q] = conv_tap(t.w);
    k.b[q] = l.conv_bias ? conv_tap(l.conv_bias[ch + q]) : 0.f;
  }
}

__device__ __forceinline__ f16x8 join(f16x2 a, f16x2 b, f16x2 c, f16x2 d) { return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]}; }

// --------------------------------------------------------------- prepare --
template <int N, bool CONV>
__device__ __forceinline__ void prepare_bc(const SsmScanArgs& a, const Ws& w, int s, int c, int grp, _Float16* rows, float* red) {
  constexpr int ROW = N + 8, PAIRS = N / 32, KN = N / 32, TILES = (2 * PAIRS + 3) / 4;   // tiles of 32 channels a wave
  const SsmLayer& l = a.l;
  const int tid = threadIdx.x, wave = tid / 64, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int t0 = a.cu[s], len = a.cu[s + 1] - t0, inner = l.H * l.P, left = len - c * kChunk;
  const int64_t sg = (int64_t)(t0 / kChunk + s + c) * l.G + grp;
  float v[TILES][2][2][4];
  float top[TILES][2][4] = {};        // the largest of each token in a tile
  RawX x[TILES];
  auto tile_of = [&](int k) { return wave + 4 * k; };     // below PAIRS: of B, then of C
  auto col_of = [&](int t) { return t < PAIRS ? inner + grp * N + 32 * t : inner + (l.G + grp) * N + 32 * (t - PAIRS); };
#pragma unroll
  for (int k = 0; k < TILES; ++k) {
    if (tile_of(k) >= 2 * PAIRS) continue;
    const XRef f{a.x + (int64_t)t0 * a.x_stride, a.conv_in ? a.conv_in + (int64_t)s * 3 * l.conv_dim : nullptr, a.x_stride, l.conv_dim, len,
                 col_of(tile_of(k)) + 2 * r};
    load_x<CONV>(f, c, g, x[k]);
  }
#pragma unroll
  for (int k = 0; k < TILES; ++k) {
    if (tile_of(k) >= 2 * PAIRS) continue;
    ConvW cw;
    if (CONV) load_conv(l, col_of(tile_of(k)) + 2 * r, cw);
#pragma unroll
    for (int run = 0; run < 2; ++run) {
      conv_run<CONV>(x[k].v[run], cw, v[k][0][run], v[k][1][run]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float& u0 = v[k][0][run][i];
        float& u1 = v[k][1][run][i];
        if (16 * run + 4 * g + i >= left) u0 = u1 = 0.f;
        top[k][run][i] = fmaxf(finite_abs(u0), finite_abs(u1));
      }
    }
  }
  // [B, C][token][tile]
#pragma unroll
  for (int k = 0; k < TILES; ++k) {
    if (tile_of(k) >= 2 * PAIRS) continue;
    float* const to = red + (tile_of(k) / PAIRS * kChunk + 4 * g) * PAIRS + tile_of(k) % PAIRS;
#pragma unroll
    for (int run = 0; run < 2; ++run)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float m = over_wave16(top[k][run][i]);
        if (r == 0) to[(16 * run + i) * PAIRS] = m;
      }
  }
  __syncthreads();
  // lane t of each wave: token t's power on B, lane 32 + t: on C
  float most = red[lane * PAIRS];
#pragma unroll
  for (int i = 1; i < PAIRS; ++i) most = fmaxf(most, red[lane * PAIRS + i]);
  const int power = (lane < 32 ? kTopB : kTopC) - pow2_above(most);
  int kb = lane < 32 ? power : INT_MAX;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) kb = min(kb, from_lane(kb, lane ^ d));
  kb = __builtin_amdgcn_readfirstlane(kb);
  if (wave == 0) {
    int* const powers = reinterpret_cast<int*>(w.gt + sg * 4 * 256 + 3 * 256);
    if (lane == 0) powers[0] = kb;
    powers[32 + (lane ^ 32)] = lane < 32 ? __float_as_int(ldexpf(1.f, kb - power)) : power;
  }
  f16x8* ops = reinterpret_cast<f16x8*>(w.bc + sg * 3 * kChunk * N * 2);
#pragma unroll
  for (int k = 0; k < TILES; ++k) {
    const int t = tile_of(k);
    if (t >= 2 * PAIRS) continue;
    const bool is_c = t >= PAIRS;
    _Float16* to = rows + (is_c ? kChunk * ROW + 32 * (t - PAIRS) : 32 * t) + 2 * r;
#pragma unroll
    for (int run = 0; run < 2; ++run)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int own = from_lane(power, (is_c ? 32 : 0) + 16 * run + 4 * g + i), all = is_c ? own : kb;
        *reinterpret_cast<f16x2*>(to + (16 * run + 4 * g + i) * ROW) = pack_f16(ldexpf(v[k][0][run][i], all), ldexpf(v[k][1][run][i], all));
        v[k][0][run][i] = ldexpf(v[k][0][run][i], own);
        v[k][1][run][i] = ldexpf(v[k][1][run][i], own);
      }
    if (!is_c) {
      f16x8* bt = ops + kChunk * N / 8;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        f16x2 hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v0 = v[k][q][i / 2][2 * (i % 2)], v1 = v[k][q][i / 2][2 * (i % 2) + 1];
          hi[i] = pack_f16(v0, v1);
          lo[i] = pack_f16(fmaf((float)hi[i][0], -1.f, v0), fmaf((float)hi[i][1], -1.f, v1));
        }
        bt[(2 * t + q) * 64 + lane] = join(hi[0], hi[1], hi[2], hi[3]);
        if (CONV) bt[kChunk * N / 8 + (2 * t + q) * 64 + lane] = join(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
  __syncthreads();
  // rows of C as operands, two tiles of 16 by two waves each; the three tiles of C . B by a wave each
  const _Float16* rc = rows + kChunk * ROW + r * ROW + 8 * g;
  for (int ks = wave / 2; ks < KN; ks += 2)
    ops[((wave % 2) * KN + ks) * 64 + lane] = *reinterpret_cast<const f16x8*>(rc + 16 * (wave % 2) * ROW + 32 * ks);
  if (wave < kTiles) {
    const int tt = wave > 0, st = wave > 1;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KN; ++ks)
      acc = mma(*reinterpret_cast<const f16x8*>(rows + (16 * st + r) * ROW + 8 * g + 32 * ks),
                *reinterpret_cast<const f16x8*>(rc + 16 * tt * ROW + 32 * ks), acc);
    acc *= 1.f / (1 << kCB);
    const f16x2 p0 = pack_f16(acc[0], acc[1]), p1 = pack_f16(acc[2], acc[3]);
    reinterpret_cast<f16x4*>(w.gt + sg * 4 * 256)[wave * 64 + lane] = f16x4{p0[0], p0[1], p1[0], p1[1]};
  }
}

// The steps of a chunk for two heads: half a wave each, a lane per token.
__device__ __forceinline__ void prepare_steps(const SsmScanArgs& a, const Ws& w, int s, int c, int h) {
  const int lane = threadIdx.x & 31, t0 = a.cu[s], len = a.cu[s + 1] - t0, p = c * kChunk + lane;
  const float A = a.l.A[h];
  const float dt = p < len ? ssm_step(a.l, a.dt, (int64_t)(t0 + p) * a.dt_stride + h, h) : 0.f;
  // log2 of the token's decay; one of 2^-200 leaves nothing of a state, and
  // longer ones would only take precision from the sums
  float al = A * dt * kLog2e;
  if (al < -200.f) al = -200.f;
  if (p >= len) al = 0.f;
  float cum = al, after = al;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const float x = __shfl_up(cum, d, 32), y = __shfl_down(after, d, 32);
    if (lane >= d) cum += x;
    if (lane + d < 32) after += y;
  }
  const float total = __shfl(cum, 31, 32);
  // sum of the later tokens' decays, from the end: near tokens keep their
  // precision behind a long sum
  after = __shfl_down(after, 1, 32);
  if (lane == 31) after = 0.f;
  const float wt = __builtin_amdgcn_exp2f(after) * dt;
  const float wmax = over_half(finite_abs(wt), MaxOp{});
  // the power of two above the largest step of this token and those before it,
  // decayed (or grown) to this token: what the token's weights hold besides C . B
  float most = (float)pow2_above(finite_abs(dt)) - cum;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const float x = __shfl_up(most, d, 32);
    if (lane >= d) most = fmaxf(most, x);      // (NaN, of later tokens' sums alone, is passed over)
  }
  float* tab = w.tab + ((int64_t)(t0 / kChunk + s + c) * a.l.H + h) * kTab;
  tab[lane] = dt;
  tab[32 + lane] = cum;
  const int kw = -pow2_above(wmax);      // the weights below 1
  tab[64 + lane] = ldexpf(wt, kw);
  if (lane < 3) tab[96 + lane] = lane == 0 ? total : lane == 1 ? __int_as_float(kw) : __builtin_amdgcn_exp2f(total);
  reinterpret_cast<int8_t*>(tab + 100)[lane] = (int8_t)fminf(fmaxf(ceilf(most + cum), -100.f), 127.f);
}

template <int N, bool CONV>
__global__ void __launch_bounds__(256) ssm_prepare_kernel(const SsmScanArgs a, const Ws w) {
  __shared__ __align__(16) _Float16 rows[2 * kChunk * (N + 8)];
  __shared__ __align__(16) float red[2 * kChunk * 4];
  const int b = blockIdx.x, s = owner(a.cu, a.n_seqs, kChunk, b), c = b - (a.cu[s] / kChunk + s);
  if (c * kChunk >= a.cu[s + 1] - a.cu[s]) return;
  if ((int)blockIdx.y < a.l.G) {
    prepare_bc<N, CONV>(a, w, s, c, blockIdx.y, rows, red);
  } else {
    const int h = (blockIdx.y - a.l.G) * 8 + threadIdx.x / 32;
    if (h < a.l.H) prepare_steps(a, w, s, c, h);
  }
}

// ------------------------------------------------------------------ scan --
// Copies 16 bytes a lane from global memory to LDS, from the wave's base on.
// The compiler does not see it and so waits for none before other reads of
// LDS: arrived() and a barrier stand between it and its readers.
__device__ __forceinline__ void to_lds(const void* g, const void* base) {
  const uint32_t at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)base;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(g) : "memory", "m0");
}
// Waits for the wave's accesses to memory.
__device__ __forceinline__ void arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Input of channel c at position p of prompt s (t0 = its first row; p < 0: its history).
__device__ __forceinline__ uint16_t raw_at(const SsmScanArgs& a, int s, int t0, int p, int c) {
  if (p >= 0) return a.x[(int64_t)(t0 + p) * a.x_stride + c];
  return a.conv_in ? a.conv_in[((int64_t)s * 3 + 3 + p) * a.l.conv_dim + c] : 0;
}

// The window behind a prompt's len tokens for a channel pair: its last three
// inputs, all read before the first is written, since conv_out may be conv_in.
__device__ __forceinline__ void move_window(const SsmScanArgs& a, int s, int t0, int len, int pair) {
  uint32_t v[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) v[j] = raw_at(a, s, t0, len - 3 + j, 2 * pair) | (uint32_t)raw_at(a, s, t0, len - 3 + j, 2 * pair + 1) << 16;
#pragma unroll
  for (int j = 0; j < 3; ++j) reinterpret_cast<uint32_t*>(a.conv_out + ((int64_t)s * 3 + j) * a.l.conv_dim)[pair] = v[j];
}

// The power of two on a token's weights: from those on C . B (with C's own, kc)
// and its steps (ad), or what D leaves.
__device__ __forceinline__ int weight_power(int kb, int kc, int ad, int pd_max) { return min(kb + kc - kCB + ad, pd_max); }

// The operand of M^T for 16 tokens t (tile row TT): both tiles of s.  m: the power
// on the weights of this lane's token, cb: the one that they have from C . B.
template <int TT>
__device__ __forceinline__ f16x8 weigh(const f16x4* gt, const float* tab, int lane, int m, int cb, float D) {
  const int r = lane & 15, g = lane >> 4, ad = m - cb;
  const float dm = ldexpf(D, m);
  const float ct = tab[32 + 16 * TT + r] + (float)ad;
  f16x2 o[4];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int st = q;
    if (st > TT) { o[2 * q] = o[2 * q + 1] = f16x2{0, 0}; continue; }
    const f16x4 gv = gt[(TT + st) * 64 + lane];
    const f32x4 cs = *reinterpret_cast<const f32x4*>(tab + 32 + 16 * st + 4 * g);
    const f32x4 ds = *reinterpret_cast<const f32x4*>(tab + 16 * st + 4 * g);
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = (float)gv[j] * (ds[j] * __builtin_amdgcn_exp2f(ct - cs[j]));
      if (st == TT) v[j] = 4 * g + j < r ? v[j] : 4 * g + j == r ? v[j] + dm : 0.f;
    }
    o[2 * q] = pack_f16(v[0], v[1]);
    o[2 * q + 1] = pack_f16(v[2], v[3]);
  }
  return join(o[0], o[1], o[2], o[3]);
}

// LDS of a workgroup of NW waves: C, B^T hi, B^T lo (without the
// convolution B is exact in fp16: no lo), C . B, x, M and the tables.
template <int P, int N, int NW, bool OUT, bool CONV>
struct ScanLds {
  static constexpr int OPS = kChunk * N * 2;
  static constexpr int FIRST = OUT ? 0 : OPS, LAST = CONV ? 3 * OPS : 2 * OPS;   // of the operands in a slot
  static constexpr int GT = OUT ? 2048 : 1024,   // (the states need the powers of two alone)
                        ROWS = CONV ? 35 : 32;
  static constexpr int X = (ROWS * 64 * NW + 1023) / 1024 * 1024, HPW = NW / (P / 32);
  static constexpr int TABS = HPW > 2 ? HPW * kTab * 4 : 1024;     // of a chunk, fetched by 1,024 bytes
  static constexpr int BYTES = LAST - FIRST + GT + 2 * X + (OUT ? HPW * 2048 : 0) + 2 * TABS + (CONV ? 5 * 32 * NW * 4 : 0);
};

template <int P, int N, int NW, bool OUT, bool CONV>
__global__ void __launch_bounds__(64 * NW, 2) ssm_chunk_kernel(const SsmScanArgs a, const Ws w, int split, int grouped, int windows) {
  using L = ScanLds<P, N, NW, OUT, CONV>;
  constexpr int nw = NW, hpw = L::HPW;
  constexpr int WPH = P / 32, NT = N / 16, KN = N / 32, OPS = L::OPS, FIRST = L::FIRST, LAST = L::LAST, GT = L::GT;
  extern __shared__ __align__(16) char lds[];
  const SsmLayer& l = a.l;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int hl = wave / WPH, half = wave % WPH;
  char* const ops = lds;
  char* const gts = ops + (LAST - FIRST);
  char* const xs = gts + GT;
  f16x8 (*const fm)[64] = reinterpret_cast<f16x8 (*)[64]>(xs + 2 * L::X + (OUT ? hl * 2048 : 0));   // this head's M
  char* const tabs = xs + 2 * L::X + (OUT ? hpw * 2048 : 0);
  const int hb = l.H / hpw, per_group = hb / l.G;
  int unit, b;
  if (grouped) {   // the workgroups that read the same B and C go to one XCD (4 x 8,192 tokens: 492 -> 481 us)
    const int q = blockIdx.x / (8 * per_group), rem = blockIdx.x % (8 * per_group), cell = 8 * q + rem % 8;
    unit = cell / l.G;
    b = cell % l.G * per_group + rem / 8;
  } else {
    unit = blockIdx.x / hb;
    b = blockIdx.x % hb;
  }
  const int units = split ? w.seg_slots : a.n_seqs;
  if (unit >= units) return;
  const int s = split ? owner(a.cu, a.n_seqs, kChunk * kSegUnit, unit) : unit;
  const int t0 = a.cu[s], len = a.cu[s + 1] - t0, nc = (len + kChunk - 1) / kChunk;
  const int per = split ? seg_chunks(nc, hb) : max(nc, 1), k = split ? unit - (t0 / (kChunk * kSegUnit) + s) : 0;
  const int n_seg = max(1, (nc + per - 1) / per);
  if (k >= n_seg || (!OUT && k + 1 >= n_seg)) return;
  const int c_first = k * per, c_end = min(nc, c_first + per);

  const int h = b * hpw + hl, grp = h / (l.H / l.G), ch0 = h * P + 32 * half + 2 * r;
  const int64_t hpn = (int64_t)l.P * l.N, slot0 = t0 / kChunk + s;
  const int st_at = (32 * half + 2 * r) * N + 8 * g;       // this lane's entries of a head's state
  // A chunk is fetched while others are worked on, to LDS directly, 16 bytes a
  // lane: its operands once the ones before are through with the products, its
  // x a chunk earlier.
  auto fetch = [&](int c) __attribute__((always_inline)) {
    const int64_t sg = (slot0 + c) * l.G + grp;
    const char* src = w.bc + sg * 3 * OPS;
    for (int i = FIRST / 1024 + wave; i < LAST / 1024; i += nw) to_lds(src + 1024 * i + 16 * lane, ops + 1024 * i - FIRST);
    for (int i = wave; i < GT / 1024; i += nw) to_lds(reinterpret_cast<const char*>(w.gt) + sg * 2048 + 2048 - GT + 1024 * i + 16 * lane, gts + 1024 * i);
    for (int i = wave; i < L::TABS / 1024; i += nw)
      to_lds(w.tab + ((slot0 + c) * l.H + b * hpw) * kTab + 256 * i + 4 * lane, tabs + (c & 1) * L::TABS + 1024 * i);
  };
  // Rows of x (from three before the chunk's first with the convolution; past
  // the prompt's end its last) of the workgroup's channels, 64 bytes a wave.
  // Row p keeps wave w's piece at piece w ^ (p / 4 % 2): rows 4 apart, which two
  // lane groups read together, lie in different banks.
  constexpr int XSWAP = NW > 1 ? 1 : 0;
  auto fetch_x = [&](int c) __attribute__((always_inline)) {
    const char* src = reinterpret_cast<const char*>(a.x + (int64_t)t0 * a.x_stride + b * hpw * P);
    const int p0 = c * kChunk - (CONV ? 3 : 0);
    for (int i = wave; i < L::X / 1024; i += nw) {
      const int at = 64 * i + lane, p = at / (4 * nw), blk = (at % (4 * nw)) ^ (((p >> 2) & XSWAP) << 2);
      to_lds(src + (int64_t)min(max(p0 + p, 0), len - 1) * a.x_stride * 2 + 16 * blk, xs + (c & 1) * L::X + 1024 * i);
    }
  };
  if (c_first < c_end) {
    fetch(c_first);
    fetch_x(c_first);
    if (c_first + 1 < c_end) fetch_x(c_first + 1);
  }
  // the taps of the workgroup's channels, in LDS: [5][32 NW]
  float* const taps = reinterpret_cast<float*>(tabs + 2 * L::TABS) + 32 * wave + 2 * r;
  if (CONV && g == 0) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 t = reinterpret_cast<const float4*>(l.conv_w)[ch0 + q];
      taps[q] = conv_tap(t.x);
      taps[32 * nw + q] = conv_tap(t.y);
      taps[64 * nw + q] = conv_tap(t.z);
      taps[96 * nw + q] = conv_tap(t.w);
      taps[128 * nw + q] = l.conv_bias ? conv_tap(l.conv_bias[ch0 + q]) : 0.f;
    }
  }
  const float D = OUT && l.D ? l.D[h] : 0.f;

  // the state that enters, S^T in tiles [16 n][16 p] (columns of N in the order
  // of the sums), scaled by 2^e; `bound`:
  // no entry of the channel is larger
  f32x4 S[NT][2];
  int e[2] = {0, 0};
  float bound[2] = {0.f, 0.f};
  const float* from = !OUT ? nullptr
                      : k > 0 ? w.seg + (((int64_t)unit - 1) * l.H + h) * hpn
                      : !a.init ? nullptr
                      : n_seg > 1 && a.init == a.final_state ? w.seg + (((int64_t)unit + n_seg - 1) * l.H + h) * hpn
                      : a.init + ((int64_t)s * l.H + h) * hpn;
#pragma unroll
  for (int z = 0; z < KN; ++z)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f32x4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
      if (from) {
        v0 = *reinterpret_cast<const f32x4*>(from + st_at + q * N + 32 * z);
        v1 = *reinterpret_cast<const f32x4*>(from + st_at + q * N + 32 * z + 4);
      }
      S[2 * z][q] = f32x4{v0[0], v0[2], v1[0], v1[2]};
      S[2 * z + 1][q] = f32x4{v0[1], v0[3], v1[1], v1[3]};
    }
  if (from) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) bound[q] = fmaxf(bound[q], finite_abs(S[nt][q][i]));
      bound[q] = over_groups(bound[q]);
      e[q] = kTopS - pow2_above(bound[q]);
      const float f = ldexpf(1.f, e[q]);     // (e is within -98 .. 130: past 127 by parts)
      const float f0 = e[q] > 126 ? 0x1p100f : f, f1 = e[q] > 126 ? ldexpf(1.f, e[q] - 100) : 1.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[nt][q][i] = S[nt][q][i] * f0 * f1;
    }
  }
  auto store_state = [&](float* head) __attribute__((always_inline)) {
    float* to = head + anew(st_at);
#pragma unroll
    for (int z = 0; z < KN; ++z)
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<f32x4*>(to + q * N + 32 * z + 4 * i) =
              f32x4{ldexpf(S[2 * z][q][2 * i], -e[q]), ldexpf(S[2 * z + 1][q][2 * i], -e[q]), ldexpf(S[2 * z][q][2 * i + 1], -e[q]),
                    ldexpf(S[2 * z + 1][q][2 * i + 1], -e[q])};
  };
  int ci = 0, next = INT_MAX;
  if (OUT) {
    ci = lower_bound_i32(a.ckpt, a.n_ckpt, t0 + c_first * kChunk + 1);
    if (ci < a.n_ckpt) next = a.ckpt[ci];
    ci = __builtin_amdgcn_readfirstlane(ci);
    next = __builtin_amdgcn_readfirstlane(next);
  }
  auto keep_until = [&](int end) __attribute__((always_inline)) {
    while (next < end) {
      store_state(a.ckpt_buf + ((int64_t)ci * l.H + h) * hpn);
      ++ci;
      next = __builtin_amdgcn_readfirstlane(ci < a.n_ckpt ? a.ckpt[ci] : INT_MAX);
    }
  };
  float seg_sum = 0.f;
  arrived();
  __syncthreads();   // the first chunk is whole
  if (CONV && c_first == 0 && c_end > 0) {
    // the window takes the place of the three rows before the prompt (rows 0 to 2: not swapped)
    if (lane < 48) {
      const int i = lane / 16;
      reinterpret_cast<uint32_t*>(xs)[16 * (i * nw + wave) + lane % 16] =
          a.conv_in ? *reinterpret_cast<const uint32_t*>(a.conv_in + ((int64_t)s * 3 + i) * l.conv_dim + h * P + 32 * half + 2 * (lane % 16)) : 0u;
    }
    __syncthreads();
  }
  const f16x8* fc = reinterpret_cast<const f16x8*>(ops) + lane;
  const f16x8* bh = reinterpret_cast<const f16x8*>(ops + OPS - FIRST) + lane;
  const f16x8* bl = reinterpret_cast<const f16x8*>(ops + (CONV ? 2 * OPS : OPS) - FIRST) + lane;

  // A chunk's x through the convolution, times 2^kPlainX; x_wide: that power does
  // not serve this lane's values.
  float xv[2][2][4];
  bool x_wide = false;
  auto take_x = [&](int c) __attribute__((always_inline)) {
    // row 16 run + 4 g + j of the tile, from one address for j below 4 and one beyond
    ConvW cw;
    if (CONV) {
      typedef float f32x2a __attribute__((ext_vector_type(2)));
      const float* tp = taps + anew(0);    // (read here: kept over the chunks, they would take 10 registers)
      const f32x2a t0 = *reinterpret_cast<const f32x2a*>(tp), t1 = *reinterpret_cast<const f32x2a*>(tp + 32 * nw),
                   t2 = *reinterpret_cast<const f32x2a*>(tp + 64 * nw), t3 = *reinterpret_cast<const f32x2a*>(tp + 96 * nw),
                   tb = *reinterpret_cast<const f32x2a*>(tp + 128 * nw);
#pragma unroll
      for (int q = 0; q < 2; ++q) { cw.w0[q] = t0[q]; cw.w1[q] = t1[q]; cw.w2[q] = t2[q]; cw.w3[q] = t3[q]; cw.b[q] = tb[q]; }
    }
    const uint32_t* xr[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) xr[j] = reinterpret_cast<const uint32_t*>(xs + (c & 1) * L::X) + r + 16 * (4 * g * nw + (wave ^ ((g + j) & XSWAP)));
#pragma unroll
    for (int run = 0; run < 2; ++run) {
      uint32_t x[7];
#pragma unroll
      for (int i = CONV ? 0 : 3; i < 7; ++i) {
        const int j = i - (CONV ? 0 : 3);
        x[i] = xr[j / 4][16 * nw * (16 * run + j)];
      }
      conv_run<CONV, kPlainX>(x, cw, xv[0][run], xv[1][run]);
    }
    if (CONV && len - c * kChunk < kChunk) {
      // behind the prompt's last row stands that row again, whose convolution may
      // be what no token's is: infinite, say, which a weight of 0 would make NaN
      const int past = len - c * kChunk - anew(4 * g);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (16 * (i / 4) + i % 4 >= past) xv[q][i / 4][i % 4] = 0.f;
    }
    if (OUT) {
      float top[2] = {0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) top[q] = fmaxf(top[q], fabsf(xv[q][i / 4][i % 4]));   // (NaN is passed over)
      x_wide = small_but_not_0(top, ldexpf(1.f, kPlainX - 8)) || fmaxf(top[0], top[1]) >= 32768.f;
    }
  };
  const int pd_max = 14 - pow2_above(fabsf(D));
  if (c_first < c_end) take_x(c_first);

  for (int c = c_first; c < c_end; ++c) {
    const int left = min(kChunk, len - c * kChunk);
    // a checkpoint at the chunk's start gets the state that enters it, and so
    // does one inside, to which a launch behind this one adds the tokens
    if (OUT) keep_until(t0 + c * kChunk + left);
    arrived();
    __syncthreads();   // the chunk's operands and the next x are whole; x is in registers; the last outputs are through with M
    if (c + 2 < c_end) fetch_x(c + 2);
    // the half with the operands goes first on a SIMD: behind its end wait the
    // workgroup's fetches (307 -> 297 us at 32 x 1,024 tokens)
    __builtin_amdgcn_s_setprio(1);
    const int* const powers = reinterpret_cast<const int*>(gts + GT - 512);
    const int kbt = __builtin_amdgcn_readfirstlane(powers[0]);
    const float* tab = reinterpret_cast<const float*>(tabs + (c & 1) * L::TABS) + hl * kTab;
    const float alpha = tab[98];
    const int kw = __float_as_int(tab[97]);
    int kc[2], m[2];           // the powers on C and on the weights of tokens r and 16 + r
    if (OUT) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        kc[tt] = powers[32 + 16 * tt + r];
        m[tt] = weight_power(kbt, kc[tt], -reinterpret_cast<const int8_t*>(tab + 100)[16 * tt + r], pd_max);
      }
    }
    __builtin_amdgcn_sched_barrier(0);

    // the entering state with C: S as an operand times 2^es; y[tt][q]: channel
    // 2 (4 g + i) + q at token 16 tt + r.  One power for the wave and one for x
    // (plain) serve where they leave each channel 2^-27 of its own largest value:
    // where no channel's x, or state, lies far below the wave's.  Else each channel
    // has its own, which the outputs' rows then take from its lanes (in every chunk:
    // 32 x 1,024 tokens 302 -> 346 us).
    f32x4 y[2][2];
    int es[2];
    bool plain = false;
    if (OUT) {
      const float top = over_wave16(fmaxf(bound[0], bound[1]));
      plain = __ballot(x_wide || small_but_not_0(bound, top * 0x1p-12f) || top >= 0x1p60f) == 0;
      float down[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        es[q] = kTopS16 - pow2_above(plain ? top : bound[q]);
        down[q] = bound[q] == 0.f ? 0.f : ldexpf(1.f, es[q] - e[q]);
      }
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int q = 0; q < 2; ++q) y[tt][q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int z = 0; z < KN; ++z) {
        const f16x8 c0 = fc[z * 64], c1 = fc[(KN + z) * 64];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const f16x8 so = join(pack_f16(S[2 * z][q][0] * down[q], S[2 * z + 1][q][0] * down[q]),
                                pack_f16(S[2 * z][q][1] * down[q], S[2 * z + 1][q][1] * down[q]),
                                pack_f16(S[2 * z][q][2] * down[q], S[2 * z + 1][q][2] * down[q]),
                                pack_f16(S[2 * z][q][3] * down[q], S[2 * z + 1][q][3] * down[q]));
          y[0][q] = mma(so, c0, y[0][q]);
          y[1][q] = mma(so, c1, y[1][q]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      // the weights inside the chunk, as operands: element (t = column, s) of M^T
      const f16x4* gt = reinterpret_cast<const f16x4*>(gts);
      if (0 == half) fm[0][lane] = weigh<0>(gt, tab, lane, m[0], kbt + kc[0] - kCB, D);
      if (1 % WPH == half) fm[1][lane] = weigh<1>(gt, tab, lane, m[1], kbt + kc[1] - kCB, D);
    }
    __builtin_amdgcn_sched_barrier(0);

    // x as operand of the outputs, times 2^kx
    int kx[2] = {kPlainX, kPlainX};
    f16x8 xo[2], xh[2], xl[2];
    if (OUT) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (plain) {
          xo[q] = join(pack_f16(xv[q][0][0], xv[q][0][1]), pack_f16(xv[q][0][2], xv[q][0][3]), pack_f16(xv[q][1][0], xv[q][1][1]),
                       pack_f16(xv[q][1][2], xv[q][1][3]));
          continue;
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_abs(xv[q][i / 4][i % 4]));
        const int k = 15 - pow2_above(over_groups(top));
        kx[q] += k;
        f16x2 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_f16(ldexpf(xv[q][i / 2][2 * (i % 2)], k), ldexpf(xv[q][i / 2][2 * (i % 2) + 1], k));
        xo[q] = join(o[0], o[1], o[2], o[3]);
      }
    }
    // x w of the state, in pairs: times 2^(kPlainX + kw + ks), ks a channel's own, and
    // 0 where half the pairs' smallest step is 2^-29 of its largest x w at most
    float grown[2], pmax[2];
    int ks[2], e_new[2];
    {
      const float* const fb = reinterpret_cast<const float*>(powers) + 64;
      const f32x4 wt[2] = {*reinterpret_cast<const f32x4*>(tab + 64 + 4 * g) * *reinterpret_cast<const f32x4*>(fb + 4 * g),
                           *reinterpret_cast<const f32x4*>(tab + 80 + 4 * g) * *reinterpret_cast<const f32x4*>(fb + 16 + 4 * g)};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        pmax[q] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xv[q][i / 4][i % 4] *= wt[i / 4][i % 4];
          pmax[q] = fmaxf(pmax[q], fabsf(xv[q][i / 4][i % 4]));      // (NaN is passed over)
        }
      }
    }
    if (__ballot(!(fmaxf(pmax[0], pmax[1]) < __builtin_inff()))) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        pmax[q] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) pmax[q] = fmaxf(pmax[q], finite_abs(xv[q][i / 4][i % 4]));
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      pmax[q] = over_groups(pmax[q]);
      // no entry of the channel will be larger: 32 products below 2^(kTopB - kbt) each
      grown[q] = fmaf(alpha, bound[q], ldexpf(pmax[q], 5 + kTopB - kbt - kw - kPlainX));
      ks[q] = pmax[q] == 0.f || (pmax[q] >= 16.f && pmax[q] < 32768.f) ? 0 : 15 - pow2_above(pmax[q]);
      ks[q] = min(ks[q], 90 - pow2_above(grown[q]) - kbt - kw - kPlainX);     // the state stays inside fp32
      e_new[q] = kbt + kw + kPlainX + ks[q];
    }
    if (__ballot((ks[0] | ks[1]) != 0)) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) xv[q][i / 4][i % 4] = ldexpf(xv[q][i / 4][i % 4], ks[q]);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f16x2 hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p0 = xv[q][i / 2][2 * (i % 2)], p1 = xv[q][i / 2][2 * (i % 2) + 1];
        hi[i] = pack_f16(p0, p1);
        lo[i] = pack_f16(fmaf((float)hi[i][0], -1.f, p0), fmaf((float)hi[i][1], -1.f, p1));
      }
      xh[q] = join(hi[0], hi[1], hi[2], hi[3]);
      xl[q] = join(lo[0], lo[1], lo[2], lo[3]);
    }

    // the state: S^T[n, p] += B^T[n, s] (x w)^T[s, p]
    float mul[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      // A state of zeros has no power of its own, and the change from any to the
      // next may pass 2^127, whose infinity would make NaN of its zeros.  (Where
      // it holds anything, mul times an entry of 2^e bound stays below 2^90.)
      mul[q] = ldexpf(alpha, bound[q] == 0.f ? -126 : e_new[q] - e[q]);
      e[q] = e_new[q];
      bound[q] = grown[q];
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt % 2 == 0) __builtin_amdgcn_sched_barrier(0);
      const f16x8 fh = bh[nt * 64];
      f16x8 fl;
      if (CONV) fl = bl[nt * 64];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int i = 0; i < 4; ++i) S[nt][q][i] *= mul[q];
        S[nt][q] = mma(fh, xh[q], S[nt][q]);
        S[nt][q] = mma(fh, xl[q], S[nt][q]);
        if (CONV) S[nt][q] = mma(fl, xh[q], S[nt][q]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (!OUT) seg_sum += tab[96];
    // the outputs' decays from the start of the chunk, before the tables may be fetched over
    float fe[2];
    if (OUT) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) fe[tt] = __builtin_amdgcn_exp2f(tab[32 + 16 * tt + r]);
    }
    __builtin_amdgcn_s_setprio(0);
    __syncthreads();   // M is whole; the products are through with the operands
    if (c + 1 < c_end) fetch(c + 1);
    if (OUT) {
      // a value of x that is not finite has left none of its channel's state
      // finite; in the products inside the chunk it would reach the tokens
      // before it, at weights of 0
      int first_bad[2] = {INT_MAX, INT_MAX};
      const bool bad = __ballot(!(fabsf(S[0][0][0]) + fabsf(S[0][1][0]) < __builtin_inff())) != 0;
      if (bad) {
        const int g2 = anew(g), lane2 = anew(lane);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
          for (int j = 7; j >= 0; --j) {
            if (!(fabsf((float)xo[q][j]) < __builtin_inff())) {
              first_bad[q] = slot_of(g2, j);
              xo[q][j] = (_Float16)0.f;
            }
          }
          first_bad[q] = min(first_bad[q], from_lane(first_bad[q], lane2 ^ 16));
          first_bad[q] = min(first_bad[q], from_lane(first_bad[q], lane2 ^ 32));
        }
      }
      uint16_t* to = a.out + ((int64_t)(t0 + c * kChunk) * l.H + h) * P + 32 * half;
      const uint32_t out_at = (uint32_t)(r * l.H * P + 8 * g);
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const f16x8 mf = fm[tt][lane];
        float o[8];
        const f32x4 z = {0.f, 0.f, 0.f, 0.f}, y2[2] = {mma(xo[0], mf, z), mma(xo[1], mf, z)};
        if (plain) {
          const float f1 = ldexpf(fe[tt], -(es[0] + kc[tt])), f2 = ldexpf(1.f, -(m[tt] + kPlainX));
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[2 * i + q] = fmaf(y2[q][i], f2, y[tt][q][i] * f1);
        } else {
          const int row = anew(4 * g);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[2 * i + q] = ldexpf(y2[q][i], -(m[tt] + from_lane(kx[q], row + i))) +
                             ldexpf(y[tt][q][i] * fe[tt], -(from_lane(es[q], row + i) + kc[tt]));
        }
        const int t = 16 * tt + r;
        if (bad) {
          const int row = anew(4 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q)
              if (t >= from_lane(first_bad[q], row + i)) o[2 * i + q] = __builtin_nanf("");
        }
        if (t < left)
          *reinterpret_cast<uint4*>(to + (int64_t)16 * tt * l.H * P + out_at) =
              make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (c + 1 < c_end) take_x(c + 1);
  }
  if (!OUT) {
    store_state(w.seg + ((int64_t)unit * l.H + h) * hpn);
    if (lane == 0 && half == 0) w.seg_sum[(int64_t)unit * l.H + h] = seg_sum;
  } else {
    keep_until(min(t0 + len, t0 + c_end * kChunk) + 1);
    if (a.final_state && k + 1 == n_seg) store_state(a.final_state + ((int64_t)s * l.H + h) * hpn);
    if (CONV && windows) {   // the window behind an unsplit prompt: this workgroup's x, and its group's B and C by the group's first
      const int inner = l.H * P / 2, first = b % per_group == 0;
      for (int i = tid; i < 16 * nw + (first ? N : 0); i += 64 * nw) {
        const int j = i - 16 * nw;
        move_window(a, s, t0, len, j < 0 ? b * 16 * nw + i : inner + (j < N / 2 ? grp * (N / 2) + j : (l.G + grp - 1) * (N / 2) + j));
      }
    }
  }
}

// The state at a checkpoint inside a chunk, from the one that enters the chunk,
// token by token (31 at most): a workgroup per 32 channels of a head, whose N
// columns lie on N / 16 lanes.
template <int N>
__global__ void __launch_bounds__(2 * N) ssm_ckpt_kernel(const SsmScanArgs a) {
  constexpr int LPR = N / 16, NCH = 32 + N;
  const SsmLayer& l = a.l;
  const int i = blockIdx.x, h = blockIdx.y, row0 = blockIdx.z * 32, pos = a.ckpt[i], s = seq_of_token(a.cu, a.n_seqs, pos - 1);
  const int t0 = a.cu[s], upto = pos - t0, first = (upto - 1) / kChunk * kChunk;
  if (upto == first + kChunk || pos == a.cu[s + 1]) return;      // the chunk's end: it is there already
  const int tid = threadIdx.x, rg = tid / LPR, jl = tid % LPR, grp = h / (l.H / l.G), inner = l.H * l.P;
  float* p = a.ckpt_buf + (((int64_t)i * l.H + h) * l.P + row0 + rg) * N + 4 * jl;
  float S[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) S[k] = p[4 * LPR * (k / 4) + k % 4];
  __shared__ float u[NCH];
  const float A = l.A[h];
  for (int t = first; t < upto; ++t) {
    __syncthreads();
    for (int e = tid; e < NCH; e += 2 * N) {
      const int c = e < 32 ? h * l.P + row0 + e : inner + grp * N + e - 32;
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j == 3 || l.conv_w) x[j] = bf16_to_f32(raw_at(a, s, t0, t - 3 + j, c));
      if (l.conv_w) {
        const float4 k = reinterpret_cast<const float4*>(l.conv_w)[c];
        x[3] = conv4_bias_silu(l.conv_bias ? conv_tap(l.conv_bias[c]) : 0.f, conv_tap(k.x), conv_tap(k.y), conv_tap(k.z),
                               conv_tap(k.w), x[0], x[1], x[2], x[3]);
      }
      u[e] = x[3];
    }
    const float dt = ssm_step(l, a.dt, (int64_t)(t0 + t) * a.dt_stride + h, h), alpha = expf(A * dt);
    __syncthreads();
    const float dx = dt * u[rg];
#pragma unroll
    for (int k = 0; k < 16; ++k) S[k] = fmaf(alpha, S[k], dx * u[32 + 4 * LPR * (k / 4) + 4 * jl + k % 4]);
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) p[4 * LPR * (k / 4) + k % 4] = S[k];
}

// The states that enter a prompt's segments: segment k's slot, which holds its
// state from zero, gets the state behind it (the one that enters k + 1).  Where
// final_state is init_state, the prompt's last segment may write it before the
// first reads it: the first then has its own from the last one's slot.
__global__ void __launch_bounds__(256) ssm_pass_kernel(const SsmScanArgs a, const Ws w, int hb) {
  const SsmLayer& l = a.l;
  const int s = blockIdx.x, h = blockIdx.y, i = (blockIdx.z * 256 + threadIdx.x) * 4;
  const int64_t hpn = (int64_t)l.P * l.N;
  const int t0 = a.cu[s], nc = (a.cu[s + 1] - t0 + kChunk - 1) / kChunk, per = seg_chunks(nc, hb), n_seg = (nc + per - 1) / per;
  if (n_seg < 2 || i >= hpn) return;
  const int64_t first = t0 / (kChunk * kSegUnit) + s;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (a.init) S = *reinterpret_cast<const f32x4*>(a.init + ((int64_t)s * l.H + h) * hpn + i);
  if (a.init && a.init == a.final_state) *reinterpret_cast<f32x4*>(w.seg + ((first + n_seg - 1) * l.H + h) * hpn + i) = S;
  for (int k = 0; k + 1 < n_seg; ++k) {
    f32x4* p = reinterpret_cast<f32x4*>(w.seg + ((first + k) * l.H + h) * hpn + i);
    const float al = __builtin_amdgcn_exp2f(w.seg_sum[(first + k) * l.H + h]);
    const f32x4 own = *p;
#pragma unroll
    for (int j = 0; j < 4; ++j) S[j] = fmaf(al, S[j], own[j]);
    *p = S;
  }
}

// The three inputs before each checkpoint (blockIdx.x < n_ck), and behind each
// prompt.  conv_out may be conv_in: the checkpoints that read conv_in, at most
// two tokens into their prompt, are written by the prompt's own threads, ahead
// of its window.
__global__ void __launch_bounds__(256) ssm_scan_window_kernel(const SsmScanArgs a, int n_ck) {
  const int c = blockIdx.y * 256 + threadIdx.x, dim = a.l.conv_dim, i = blockIdx.x;
  if (2 * c >= dim) return;
  auto keep = [&](int i, int s, int t0) {
    for (int j = 0; j < 3; ++j)
      for (int q = 0; q < 2; ++q) a.conv_ckpt[((int64_t)i * 3 + j) * dim + 2 * c + q] = raw_at(a, s, t0, a.ckpt[i] - t0 - 3 + j, 2 * c + q);
  };
  if (i < n_ck) {
    const int s = seq_of_token(a.cu, a.n_seqs, a.ckpt[i] - 1), t0 = a.cu[s];
    if (a.ckpt[i] - t0 >= 3) keep(i, s, t0);
    return;
  }
  const int s = i - n_ck, t0 = a.cu[s], len = a.cu[s + 1] - t0;
  if (n_ck > 0)
    for (int k = lower_bound_i32(a.ckpt, n_ck, t0 + 1); k < n_ck && a.ckpt[k] <= t0 + min(len, 2); ++k) keep(k, s, t0);
  if (a.conv_out) move_window(a, s, t0, len, c);
}

template <int P, int N, int NW>
hipError_t launch(const SsmScanArgs& a, const Ws& w, int segs, bool inside, int windows, hipStream_t st) {
  const SsmLayer& l = a.l;
  hipError_t e = hipSuccess;
  if (a.n_tokens > 0) {
    const dim3 prep(w.slots, l.G + (l.H + 7) / 8);
    if (l.conv_w) hipLaunchKernelGGL((ssm_prepare_kernel<N, true>), prep, dim3(256), 0, st, a, w);
    else hipLaunchKernelGGL((ssm_prepare_kernel<N, false>), prep, dim3(256), 0, st, a, w);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const int hb = l.H / (NW / (P / 32)), split = segs > 1;
  const int64_t units = split ? w.seg_slots : a.n_seqs, cells = units * l.G;
  const int grouped = cells >= 32;
  const dim3 grid((uint32_t)(grouped ? (cells + 7) / 8 * 8 * (hb / l.G) : units * hb));
  auto scan = [&](auto out, auto conv) {
    constexpr bool O = decltype(out)::value, C = decltype(conv)::value;
    constexpr int bytes = ScanLds<P, N, NW, O, C>::BYTES;
    static_assert(bytes <= 64 * 1024, "past what a launch has without asking");
    hipLaunchKernelGGL((ssm_chunk_kernel<P, N, NW, O, C>), grid, dim3(64 * NW), bytes, st, a, w, split, grouped, windows);
    return hipGetLastError();
  };
  using T = std::true_type;
  using F = std::false_type;
  if (split) {
    if ((e = l.conv_w ? scan(F{}, T{}) : scan(F{}, F{})) != hipSuccess) return e;
    hipLaunchKernelGGL(ssm_pass_kernel, dim3(a.n_seqs, l.H, (P * N + 1023) / 1024), dim3(256), 0, st, a, w, hb);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  e = l.conv_w ? scan(T{}, T{}) : scan(T{}, F{});
  if (e != hipSuccess || !inside) return e;
  hipLaunchKernelGGL((ssm_ckpt_kernel<N>), dim3(a.n_ckpt, l.H, P / 32), dim3(2 * N), 0, st, a);
  return hipGetLastError();
}

template <int P, int N>
hipError_t launch_n(const SsmScanArgs& a, const Ws& w, int segs, bool inside, int windows, hipStream_t st) {
  const int nw = heads_per_wg(a.l) * (P / 32);
  if constexpr (P <= 64) {
    if (nw == 2) return launch<P, N, 2>(a, w, segs, inside, windows, st);
  }
  if constexpr (P == 32) {
    if (nw == 1) return launch<P, N, 1>(a, w, segs, inside, windows, st);
  }
  return launch<P, N, 4>(a, w, segs, inside, windows, st);
}

template <int P>
hipError_t launch_p(const SsmScanArgs& a, const Ws& w, int segs, bool inside, int windows, hipStream_t st) {
  return a.l.N == 32 ? launch_n<P, 32>(a, w, segs, inside, windows, st) : a.l.N == 64 ? launch_n<P, 64>(a, w, segs, inside, windows, st)
                                                                             : launch_n<P, 128>(a, w, segs, inside, windows, st);
}

}  // namespace

int64_t ssm_scan_bytes(const SsmLayer& l, int32_t n_seqs, const int32_t* cu) {
  if (n_seqs == 0 || cu[n_seqs] == 0) return 0;
  return layout(l, n_seqs, cu[n_seqs], max_segments(l, n_seqs, cu) > 1, nullptr).bytes;
}

int64_t ssm_scan_groups(const SsmLayer& l, int32_t n_seqs, int64_t n_tokens) {
  const int64_t hb = l.H / heads_per_wg(l), units = n_tokens / (kChunk * kSegUnit) + n_seqs;
  return std::max((units * l.G + 8) * (hb / l.G), n_tokens / kChunk + n_seqs);
}

// Whether a checkpoint lies inside a chunk.
static bool ckpt_inside(const SsmScanArgs& a, const int32_t* cu, const int32_t* ckpt) {
  int s = 0;
  for (int i = 0; i < a.n_ckpt; ++i) {
    while (cu[s + 1] < ckpt[i]) ++s;
    if ((ckpt[i] - cu[s]) % kChunk != 0 && ckpt[i] != cu[s + 1]) return true;
  }
  return false;
}

hipError_t launch_ssm_scan(const SsmScanArgs& a, const int32_t* cu_host, const int32_t* ckpt_host, void* workspace,
                           hipStream_t st) {
  const bool inside = ckpt_inside(a, cu_host, ckpt_host);
  const int segs = max_segments(a.l, a.n_seqs, cu_host);
  const Ws w = layout(a.l, a.n_seqs, a.n_tokens, segs > 1, workspace);
  const int n_ck = a.conv_ckpt ? a.n_ckpt : 0;
  // The scan moves the windows itself (one launch less of 4 us: 25.7 -> 23.3 us
  // for a prompt of 100 tokens) where each channel of conv_in has one reader, the
  // workgroup that writes it, and none comes later.
  const int windows = a.conv_out && segs == 1 && n_ck == 0 && !inside;
  hipError_t e = a.l.P == 32   ? launch_p<32>(a, w, segs, inside, windows, st)
                 : a.l.P == 64 ? launch_p<64>(a, w, segs, inside, windows, st)
                               : launch_p<128>(a, w, segs, inside, windows, st);
  if (e == hipSuccess && !windows && a.n_seqs > 0 && (a.conv_out || n_ck > 0)) {
    hipLaunchKernelGGL(ssm_scan_window_kernel, dim3(n_ck + a.n_seqs, (a.l.conv_dim + 511) / 512), dim3(256), 0, st, a, n_ck);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace gdn
