// Rotary positions with the cache's write, and the cache's read back.
//
// One launch rotates the queries and writes the keys and values.  A workgroup
// of the write owns one (page, kv head) of one prompt, because the page's
// scale depends on every token that this call puts there: it loads the page's
// new keys and values once into registers, rotates the keys, takes both
// maxima, settles the scales and stores the codes.  A query workgroup forms
// the angles of its tokens once in LDS and turns every head with them.
// Measured: 32 prompts of 1,024 tokens (32 query heads, 8 kv heads of 128)
// 160 us, HBM bound (0.74 GB, 4.6 TB/s); a decode step of 64 tokens 9.6 us,
// the latency of the way from the prompts' offsets over slots and rows to the
// scale and the codes.  Pages of 128 tokens with heads of 256 (keys and values
// of 256 registers, two waves a SIMD): 16 prompts of 500 to 1,500 tokens, 4 kv
// heads, with their read 138 us, 3.3 TB/s, where heads of 128 reach 4.4.
#include <algorithm>

#include "cache_device.h"

namespace gdn {
namespace {


// cos and sin of position * freq, to 0.86 ulp at any size that the call takes
// (|freq| <= 2^16, so angles up to 2^47).  The angle, a product of
// 31 and 24 bits, is held in two doubles, and 2 / pi in two: the nearest whole
// number of quarter turns comes off exactly, and what is left of the angle is
// right to 2^-54 turns.  It is x + x_lo, at most 0.8, where the Taylor sums
// through x^9 and x^10 leave 2e-9 and 1.4e-10.  Each sum's last addition is the
// only rounding at the result's size: the lower part of x, of x^2 and of
// 1 - x^2/2 goes into the small terms.
__device__ __forceinline__ void cos_sin(int pos, float freq, float scale, float* c, float* s) {
  constexpr double kQuarters = 0.63661977236758134308, kQuartersLow = -3.935735335036497e-17;   // 2 / pi
  const double angle = (double)pos * (double)freq, angle_lo = fma((double)pos, (double)freq, -angle);
  const double n = rint(angle * kQuarters);
  const double xd = (fma(angle, kQuarters, -n) + fma(angle, kQuartersLow, angle_lo * kQuarters)) * 1.57079632679489661923;   // pi / 2
  const float x = (float)xd, x_lo = (float)(xd - (double)x);
  const float y = x * x, y_lo = fmaf(2.f * x, x_lo, fmaf(x, x, -y));
  float sn = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);
  sn = fmaf(y, sn, 8.3333333e-3f);
  sn = fmaf(y, sn, -1.6666667e-1f);
  sn = x + fmaf(x * y, sn, x_lo);
  float cs = fmaf(y, -2.7557319e-7f, 2.4801587e-5f);
  cs = fmaf(y, cs, -1.3888889e-3f);
  cs = fmaf(y, cs, 4.1666667e-2f);
  const float h = 0.5f * y, w = 1.f - h;
  cs = w + ((1.f - w) - h + fmaf(y * y, cs, -0.5f * y_lo));
  const int k = (int)(long long)n & 3;
  const float a = (k & 1) ? sn : cs, b = (k & 1) ? cs : sn;
  *c = scale * (k == 1 || k == 2 ? -a : a);
  *s = scale * (k >= 2 ? -b : b);
}

// Positions of a token on every axis.
struct Positions {
  int32_t p[4];
  __device__ __forceinline__ void load(const AppendArgs& a, int t) {
#pragma unroll
    for (int x = 0; x < 4; ++x) p[x] = x < a.rope.n_axes ? a.pos[x * a.pos_stride + t] : 0;
  }
  __device__ __forceinline__ int32_t at(int axis) const {
    return axis == 0 ? p[0] : axis == 1 ? p[1] : axis == 2 ? p[2] : p[3];
  }
};

// A head's channels in chunks of 16: two groups of 8, at e0 and e1.  The first
// rot / 16 chunks hold the pairs 8 chunk .. 8 chunk + 7.
struct Chunk {
  int e0, e1;
  bool turned;
  __device__ __forceinline__ Chunk(const RopeRef& r, int c) {
    turned = c < r.rot / 16;
    e0 = turned && !r.adjacent ? 8 * c : 16 * c;
    e1 = turned && !r.adjacent ? e0 + r.rot / 2 : e0 + 8;
  }
};

__device__ __forceinline__ float at_most_largest(float x) {
  return __builtin_amdgcn_fmed3f(x, -0x1.fffffep127f, 0x1.fffffep127f);
}

// Turns the 8 pairs of a chunk (x: 16 channels, e0's 8 then e1's 8).
template <typename CosSin>
__device__ __forceinline__ void turn(float* x, int adjacent, CosSin cs) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float c, s;
    cs(i, &c, &s);
    float& a = adjacent ? x[2 * i] : x[i];
    float& b = adjacent ? x[2 * i + 1] : x[8 + i];
    // the second product's rounding error goes back in, so that fewer results
    // land on the other side of a bf16 step; an infinite product's is taken
    // against the largest number, so that it is infinite too and not NaN
    const float bs = b * s, bc = b * c;
    const float es = fmaf(b, s, -at_most_largest(bs)), ec = fmaf(b, c, -at_most_largest(bc));
    const float ra = fmaf(a, c, -bs) - es, rb = fmaf(a, s, bc) + ec;
    a = ra;
    b = rb;
  }
}

__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo_bf16(u[i]);
    x[2 * i + 1] = hi_bf16(u[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// ---------------------------------------------------------------- queries --
template <int T>
__device__ __forceinline__ void rotate_q(const AppendArgs& a, int dim, int t0, int n, float2* cs) {
  const int half = a.rope.rot / 2;
  for (int e = threadIdx.x; e < n * half; e += T) {
    const int t = e / half, i = e - t * half;
    float c, s;
    cos_sin(a.pos[a.rope.axis[i] * a.pos_stride + t0 + t], a.rope.freq[i], a.rope.scale, &c, &s);
    cs[e] = make_float2(c, s);
  }
  __syncthreads();
  const int chunks = dim / 16, per = a.Hq * chunks;
  for (int e = threadIdx.x; e < n * per; e += T) {
    const int t = e / per, hc = e - t * per, h = hc / chunks, c = hc - h * chunks;
    const Chunk ch(a.rope, c);
    const uint16_t* src = a.q + (t0 + t) * a.q_stride + (int64_t)h * dim;
    uint16_t* dst = a.q_out + (t0 + t) * a.qo_stride + (int64_t)h * dim;
    uint4 w0 = *reinterpret_cast<const uint4*>(src + ch.e0);
    uint4 w1 = *reinterpret_cast<const uint4*>(src + ch.e1);
    if (ch.turned) {
      float x[16];
      unpack8(w0, x);
      unpack8(w1, x + 8);
      const float2* row = cs + t * half + 8 * c;
      turn(x, a.rope.adjacent, [&](int i, float* co, float* si) { *co = row[i].x; *si = row[i].y; });
      w0 = pack8(x);
      w1 = pack8(x + 8);
    }
    *reinterpret_cast<uint4*>(dst + ch.e0) = w0;
    *reinterpret_cast<uint4*>(dst + ch.e1) = w1;
  }
}

// Largest value over the workgroup of x >= 0 and y >= 0.
template <int T>
__device__ __forceinline__ void block_max(float* x, float* y, float2* lds) {
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    *x = fmaxf(*x, __shfl_xor(*x, d));
    *y = fmaxf(*y, __shfl_xor(*y, d));
  }
  if constexpr (T == 64) return;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = make_float2(*x, *y);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < T / 64; ++i) {
    *x = fmaxf(*x, lds[i].x);
    *y = fmaxf(*y, lds[i].y);
  }
}

__device__ __forceinline__ float old_scale(float s) {
  return s >= kMinScale && s < __builtin_inff() ? s : kMinScale;   // a page never written holds anything
}

// ---------------------------------------------------------- keys, values --
// NV: value items (16 tokens x 2 channels) per thread; a key item (1 token x
// 16 channels) is half as large, so there are 2 NV of them.
template <int D, bool I8, int NV, int T>
__device__ __forceinline__ void write_page(const AppendArgs& a, int unit, int h, uint8_t* valid, float2* red) {
  const int tid = threadIdx.x, shift = a.c.page_shift, P = 1 << shift;
  // all of a thread's key items have the same channels: their frequencies and
  // axes are under way before anything else is known
  const int kc = tid % (D / 16);
  const Chunk ch(a.rope, kc);
  float freq[8];
  uint64_t axes = 0;
  if (ch.turned && tid / (D / 16) < P) {
#pragma unroll
    for (int i = 0; i < 8; ++i) freq[i] = a.rope.freq[8 * kc + i];
    axes = *reinterpret_cast<const uint64_t*>(a.rope.axis + 8 * kc);
  }
  // unit -> (prompt s, its j-th page of this call): prompt s has the units
  // cu[s] / P + 2 s on, more than its ceil(len / P) + 1 pages
  // (counted 64 prompts at a time: one round through memory, not log2 n)
  int lo = -1;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 64) {
    const int s = s0 + (tid & 63);
    lo += __popcll(__ballot(s < a.n_seqs && (a.cu[min(s, a.n_seqs)] >> shift) + 2 * s <= unit));
  }
  const int j = unit - (a.cu[lo] >> shift) - 2 * lo;
  const int i0 = a.cu[lo], i1 = min(a.cu[lo + 1], a.n_tokens);
  if (i0 < 0 || i0 >= i1 || j < 0) return;
  const int64_t slot0 = a.slot[i0];
  const int off0 = slot0 >= 0 ? (int)(slot0 & (P - 1)) : 0;
  const int64_t begin = j == 0 ? i0 : (int64_t)i0 + ((int64_t)j << shift) - off0;
  if (begin >= i1) return;
  const int tl = (int)begin, off = j == 0 ? off0 : 0;
  const int cnt = min(P - off, i1 - tl);
  // the page's slots in one trip, then its scales beside its rows
  const bool inside = tid >= off && tid < off + cnt;
  const int64_t lead = a.slot[tl], own = inside ? a.slot[tl + tid - off] : 0;
  if (lead < 0 || (lead & (P - 1)) != off || (lead >> shift) >= a.c.n_pages) return;
  const int64_t page = lead >> shift;
  float* const ksp = a.c.ks + page * a.c.Hkv + h;
  float* const vsp = a.c.vs + page * a.c.Hkv + h;
  const float k_was = *ksp, v_was = *vsp;

  if (tid < P) valid[tid] = inside && own == lead + (tid - off);
  __syncthreads();

  uint32_t v[NV][16];
  float vmax = 0.f, kmax = 0.f;
  const int tiles = P / 16;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int item = tid + n * T, u = item / (D / 2), c2 = item % (D / 2);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int o = u * 16 + i;
      v[n][i] = 0;
      if (u < tiles && valid[o])
        v[n][i] = *reinterpret_cast<const uint32_t*>(a.v + (tl + o - off) * a.v_stride + (int64_t)h * D + 2 * c2);
    }
  }
  uint4 k[2 * NV][2];
  constexpr int AHEAD = NV <= 2 ? 2 * NV : 0;   // items whose positions are asked for with the keys (registers)
  Positions pos[AHEAD + 1];
#pragma unroll
  for (int n = 0; n < 2 * NV; ++n) {
    const int o = (tid + n * T) / (D / 16);
    k[n][0] = k[n][1] = make_uint4(0, 0, 0, 0);
    if (o < P && valid[o]) {
      const int t = tl + o - off;
      const uint16_t* src = a.k + t * a.k_stride + (int64_t)h * D;
      k[n][0] = *reinterpret_cast<const uint4*>(src + ch.e0);
      k[n][1] = *reinterpret_cast<const uint4*>(src + ch.e1);
      if (n < AHEAD && ch.turned) pos[n].load(a, t);
    }
  }
#pragma unroll
  for (int n = 0; n < 2 * NV; ++n) {
    const int o = (tid + n * T) / (D / 16);
    if (o >= P || !valid[o]) continue;
    float x[16];
    unpack8(k[n][0], x);
    unpack8(k[n][1], x + 8);
    if (ch.turned) {
      Positions& at = pos[n < AHEAD ? n : AHEAD];
      if (n >= AHEAD) at.load(a, tl + o - off);
      turn(x, a.rope.adjacent, [&](int i, float* co, float* si) {
        cos_sin(at.at((int)(axes >> (8 * i) & 255)), freq[i], a.rope.scale, co, si);
      });
      k[n][0] = pack8(x);
      k[n][1] = pack8(x + 8);
      unpack8(k[n][0], x);
      unpack8(k[n][1], x + 8);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) kmax = fmaxf(kmax, finite_abs(x[i]));
  }
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      vmax = fmaxf(vmax, fmaxf(finite_abs(lo_bf16(v[n][i])), finite_abs(hi_bf16(v[n][i]))));
  block_max<T>(&kmax, &vmax, red);

  const float k_old = off ? old_scale(k_was) : kMinScale, v_old = off ? old_scale(v_was) : kMinScale;
  const float k_new = fmaxf(k_old, scale_for<I8>(kmax)), v_new = fmaxf(v_old, scale_for<I8>(vmax));
  __syncthreads();   // every thread has the old scales
  if (tid == 0) {
    *ksp = k_new;
    *vsp = v_new;
  }
  // powers of two up to 2^121: the reciprocals are exact and normal
  const float k_inv = 1.f / k_new, v_inv = 1.f / v_new;
  const float k_ratio = k_old * k_inv, v_ratio = v_old * v_inv;
  const bool k_grew = k_new > k_old, v_grew = v_new > v_old;

  uint8_t* const kb = a.c.k + page_base(a.c, page, h);
#pragma unroll
  for (int n = 0; n < 2 * NV; ++n) {
    const int o = (tid + n * T) / (D / 16);
    if (o >= P) continue;
    uint2* const d0 = reinterpret_cast<uint2*>(kb + o * D + ch.e0);
    uint2* const d1 = reinterpret_cast<uint2*>(kb + o * D + ch.e1);
    if (valid[o]) {
      float x[16];
      unpack8(k[n][0], x);
      unpack8(k[n][1], x + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= k_inv;
      *d0 = make_uint2(encode4<I8>(x), encode4<I8>(x + 4));
      *d1 = make_uint2(encode4<I8>(x + 8), encode4<I8>(x + 12));
    } else if (o < off && k_grew) {
      const uint2 w0 = *d0, w1 = *d1;
      *d0 = make_uint2(recode4<I8>(w0.x, k_ratio), recode4<I8>(w0.y, k_ratio));
      *d1 = make_uint2(recode4<I8>(w1.x, k_ratio), recode4<I8>(w1.y, k_ratio));
    }
  }

  uint8_t* const vb = a.c.v + page_base(a.c, page, h);
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int item = tid + n * T, u = item / (D / 2), c2 = item % (D / 2);
    if (u >= tiles) continue;
    uint32_t mask[4];   // the bytes of this tile that are new
    bool any = false, all = true;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      mask[g] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (valid[u * 16 + 4 * g + i]) mask[g] |= 0xFFu << (8 * i);
      any |= mask[g] != 0;
      all &= mask[g] == 0xFFFFFFFFu;
    }
    const bool again = v_grew && u * 16 < off;
    if (!any && !again) continue;
    uint4* const dst = reinterpret_cast<uint4*>(vb + (u * D + 2 * c2) * 16);
    uint4 old[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (!all) {
      old[0] = dst[0];
      old[1] = dst[1];
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t w[4] = {old[half].x, old[half].y, old[half].z, old[half].w};
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (again) {
          const int before = off - (u * 16 + 4 * g);   // older tokens among these four
          const uint32_t m = before >= 4 ? 0xFFFFFFFFu : before <= 0 ? 0u : (1u << (8 * before)) - 1;
          w[g] = (recode4<I8>(w[g], v_ratio) & m) | (w[g] & ~m);
        }
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two = v[n][4 * g + i];
          x[i] = (half ? hi_bf16(two) : lo_bf16(two)) * v_inv;
        }
        w[g] = (encode4<I8>(x) & mask[g]) | (w[g] & ~mask[g]);
      }
      dst[half] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Workgroups of 256, or of one wave where a page and head have no more than
// 2,048 codes to write: a wave has enough loads of those, and needs no barrier
// for its maxima (16 prompts of 500 to 1,500 tokens, 4 kv heads of 64, pages of
// 16, with their read: 51 us in workgroups of 256, 35 us).
template <int D, bool I8, int NV, int T>
__global__ void __launch_bounds__(T, NV == 4 ? 2 : 5 - NV) rope_append_kernel(const AppendArgs a, const int64_t page_blocks) {
  constexpr int Q = T / 64;   // tokens of a query workgroup
  __shared__ union {
    struct { uint8_t valid[128]; float2 red[T / 64]; } w;
    float2 cs[Q * 128];
  } lds;
  const int64_t b = blockIdx.x;
  if (b < page_blocks) {
    write_page<D, I8, NV, T>(a, (int)(b / a.c.Hkv), (int)(b % a.c.Hkv), lds.w.valid, lds.w.red);
  } else {
    const int t0 = (int)(b - page_blocks) * Q;
    rotate_q<T>(a, D, t0, min(Q, a.n_tokens - t0), lds.cs);
  }
}

// ---------------------------------------------------------------- gather --
// A workgroup reads back 16 rows of one head.  Keys: 16 channels of a row per
// thread.  Values lie 16 tokens to a vector, so a wave takes 4 rows, reads a
// vector per channel for each run of rows that lie in one 16-token tile (one or
// two for rows that follow each other) and hands its bytes out row by row; the
// next run's vectors are on their way meanwhile.  Bound by HBM: 32,768 rows of 8
// heads of 128 take 31 us, 0.20 GB (6.4 TB/s with a part of it still cached,
// 48 us from cold); a prefix of 1,000 rows takes 4 us.  16 rows a wave read
// each vector once, but are no faster anywhere (49 and 5.4 us).
constexpr int kThreads = 256;

template <int D, bool I8>
__global__ void __launch_bounds__(kThreads) cache_gather_kernel(const GatherArgs a) {
  constexpr int C = D / 64;   // a lane's channels of the values
  constexpr int R = 4;        // a wave's rows
  const int h = blockIdx.y;
  const int64_t row0 = (int64_t)blockIdx.x * (4 * R);
  const int lane = threadIdx.x & 63;
  const int64_t t0 = row0 + R * (threadIdx.x >> 6);
  const int n = (int)max(min((int64_t)R, a.n_tokens - t0), (int64_t)0);
  const int64_t slots = (int64_t)a.c.n_pages << a.c.page_shift;
  const int page_mask = (1 << a.c.page_shift) - 1;

  // the wave's slots, a lane each; -1 for one outside the cache (which ends
  // with a tile's end, so a tile is inside as a whole or not at all)
  int64_t mine = lane < n ? a.slot[t0 + lane] : -1;
  if (mine < 0 || mine >= slots) mine = -1;
  const int64_t before = __shfl_up(mine, 1);
  uint64_t runs = __ballot(lane < n && (lane == 0 || (mine >> 4) != (before >> 4)));
  uint4 w[C], next[C];
  float scale = 0.f, next_scale = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) w[c] = next[c] = make_uint4(0, 0, 0, 0);
  auto slot_of = [&](int r) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(mine >> 32), r) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane((int)mine, r));
  };
  auto load = [&](int r, uint4 (&to)[C], float& to_scale) {
    const int64_t s = slot_of(r);
    to_scale = 0.f;
    if (s < 0) return;
    const int64_t page = s >> a.c.page_shift;
    const uint8_t* p = a.c.v + page_base(a.c, page, h) + (((s & page_mask) >> 4) * D + C * lane) * 16;
#pragma unroll
    for (int c = 0; c < C; ++c) to[c] = reinterpret_cast<const uint4*>(p)[c];
    to_scale = a.c.vs[page * a.c.Hkv + h];
  };
  if (a.v_out && n) load(0, w, scale);

  if (a.k_out) {
#pragma unroll
    for (int e = threadIdx.x; e < R * D / 4; e += kThreads) {   // 4 R rows x D / 16 chunks
      const int64_t t = row0 + e / (D / 16);
      const int c = e % (D / 16);
      if (t >= a.n_tokens) continue;
      const int64_t s = a.slot[t];
      const bool ok = s >= 0 && s < slots;
      uint4 k = make_uint4(0, 0, 0, 0);
      float k_scale = 0.f;
      if (ok) {
        const int64_t page = s >> a.c.page_shift;
        k = *reinterpret_cast<const uint4*>(a.c.k + page_base(a.c, page, h) + (s & page_mask) * D + 16 * c);
        k_scale = a.c.ks[page * a.c.Hkv + h];
      }
      float x[16];
      decode4<I8>(k.x, x);
      decode4<I8>(k.y, x + 4);
      decode4<I8>(k.z, x + 8);
      decode4<I8>(k.w, x + 12);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = ok ? x[i] * k_scale : 0.f;
      uint4* dst = reinterpret_cast<uint4*>(a.k_out + (t * a.c.Hkv + h) * D + 16 * c);
      dst[0] = pack8(x);
      dst[1] = pack8(x + 8);
    }
  }
  if (!a.v_out) return;
  while (runs) {
    const int r0 = __builtin_ctzll(runs);
    runs &= runs - 1;
    const int r1 = runs ? __builtin_ctzll(runs) : n;
    if (runs) load(r1, next, next_scale);
    const bool ok = slot_of(r0) >= 0;
    for (int r = r0; r < r1; ++r) {
      const int o = (int)(slot_of(r) & 15);
      const uint32_t pick = (uint32_t)(o & 7) | 0x0C0C0C00u;   // that byte, zeros above
      float x[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[4];
        decode4<I8>(o < 8 ? __builtin_amdgcn_perm(w[c].y, w[c].x, pick) : __builtin_amdgcn_perm(w[c].w, w[c].z, pick), f);
        x[c] = ok ? f[0] * scale : 0.f;
      }
      uint16_t* dst = a.v_out + ((t0 + r) * a.c.Hkv + h) * D + C * lane;
      if constexpr (C == 1) {
        dst[0] = (uint16_t)pack_bf16(x[0], 0.f);
      } else {
#pragma unroll
        for (int c = 0; c < C; c += 2) reinterpret_cast<uint32_t*>(dst)[c / 2] = pack_bf16(x[c], x[c + 1]);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = next[c];
    scale = next_scale;
  }
}

template <int D, bool I8, int NV, int T>
hipError_t append(const AppendArgs& a, hipStream_t st) {
  const int64_t units = (a.n_tokens >> a.c.page_shift) + 2 * (int64_t)a.n_seqs;
  const int64_t page_blocks = units * a.c.Hkv;
  const int64_t q_blocks = a.q ? ((int64_t)a.n_tokens + T / 64 - 1) / (T / 64) : 0;
  hipLaunchKernelGGL((rope_append_kernel<D, I8, NV, T>), dim3((uint32_t)(page_blocks + q_blocks)), dim3(T), 0, st, a, page_blocks);
  return hipGetLastError();
}

template <int D, bool I8>
hipError_t append_d(const AppendArgs& a, hipStream_t st) {
  const int codes = D << a.c.page_shift;
  if constexpr (D < 256)
    if (codes <= 2048) return append<D, I8, 1, 64>(a, st);
  if constexpr (D > 128)
    if (codes > 16384) return append<D, I8, 4, 256>(a, st);
  if constexpr (D > 64)
    if (codes > 8192) return append<D, I8, 2, 256>(a, st);
  return append<D, I8, 1, 256>(a, st);
}

}  // namespace

hipError_t launch_rope_append(const AppendArgs& a, hipStream_t st) {
  switch (a.c.dim) {
    case 64: return a.c.i8 ? append_d<64, true>(a, st) : append_d<64, false>(a, st);
    case 128: return a.c.i8 ? append_d<128, true>(a, st) : append_d<128, false>(a, st);
    default: return a.c.i8 ? append_d<256, true>(a, st) : append_d<256, false>(a, st);
  }
}

hipError_t launch_cache_gather(const GatherArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)(((int64_t)a.n_tokens + 15) / 16), a.c.Hkv);
  const dim3 block(kThreads);
  switch (a.c.dim) {
    case 64:
      if (a.c.i8) hipLaunchKernelGGL((cache_gather_kernel<64, true>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((cache_gather_kernel<64, false>), grid, block, 0, st, a);
      break;
    case 128:
      if (a.c.i8) hipLaunchKernelGGL((cache_gather_kernel<128, true>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((cache_gather_kernel<128, false>), grid, block, 0, st, a);
      break;
    default:
      if (a.c.i8) hipLaunchKernelGGL((cache_gather_kernel<256, true>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((cache_gather_kernel<256, false>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace gdn
