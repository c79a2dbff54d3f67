// Page planner: block tables, the pack of new tokens and its slot map from
// the lengths that requests hold and want, without a host round trip.
//
// One workgroup plans: prefix sums over the requests turn lengths into stack
// positions and pack offsets, and the pages and tokens are then dealt out flat,
// each finding its request by a binary search of the prefix in LDS, so a
// request of many pages does not hold up its lane.  Everything is integer work
// on a few kB, so the number of dependent steps through memory bounds it.  Up
// to 1,024 requests there are two: the lengths, and then everything else at
// once, since the page at any place of the stack is known without the stack
// having been written (below its old top it is read there, above it it comes
// from the row that gives it back): a step of 64 requests takes 6.2 us, where
// the way through the stack takes 10.0.  More requests go 1,024 at a time,
// through the stack in memory.
#include "cache_internal.h"
#include "gdn_device.h"

namespace gdn {
namespace {

constexpr int kPlan = 1024;
constexpr int kFill = 256;

struct PlanLds {
  int64_t pre[kPlan + 1];   // exclusive prefix of the quantity being dealt out
  int32_t first[kPlan];     // a request's first page column or token index
  int32_t row[kPlan];       // granted (tokens are slotted) or not
  int64_t wave[kPlan / 64];
  int64_t total;
};

// Exclusive prefix sum over the workgroup; the total goes to every lane.
__device__ __forceinline__ int64_t block_scan(int64_t x, PlanLds& l, int64_t* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int64_t s = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(s, d);
    if (lane >= d) s += y;
  }
  __syncthreads();   // the arrays' last readers
  if (lane == 63) l.wave[w] = s;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPlan / 64; ++i) {
    const int64_t y = l.wave[i];
    if (i < w) before += y;
    all += y;
  }
  *total = all;
  return before + s - x;
}

// The request e belongs to: pre[i] <= e < pre[i + 1].
__device__ __forceinline__ int owner(const int64_t* pre, int n, int64_t e) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= e) lo = mid; else hi = mid;
  }
  return lo;
}

struct Lengths {
  int64_t kv, want;
  int32_t status, have, need;
};

__device__ __forceinline__ Lengths lengths_of(const PlanArgs& a, int i) {
  Lengths r{0, 0, 3, 0, 0};
  if (i >= a.n_seqs) return r;
  r.kv = a.kv[i];
  r.want = a.want[i];
  const int64_t most = (int64_t)a.max_pages << a.page_shift, round = (1 << a.page_shift) - 1;
  if (r.kv < 0 || r.want < 0 || r.kv > most) return r;
  r.have = (int32_t)((r.kv + round) >> a.page_shift);
  r.need = r.have;
  r.status = r.want > most ? 2 : 0;
  if (!r.status) r.need = (int32_t)((r.want + round) >> a.page_shift);
  return r;
}

__device__ __forceinline__ int64_t slot_of(const PlanArgs& a, int i, int64_t p) {
  const int32_t id = a.table[(int64_t)i * a.max_pages + (p >> a.page_shift)];
  if (id < 0 || id >= a.n_pages) return -1;
  return ((int64_t)id << a.page_shift) + (p & ((1 << a.page_shift) - 1));
}

struct SmallLds {
  int64_t back[kPlan + 1], more[kPlan + 1], fresh[kPlan + 1];   // exclusive prefixes
  int32_t kv[kPlan], have[kPlan], need[kPlan], status[kPlan];
  int64_t wave[kPlan / 64][3];
  unsigned long long got;
};

// n_seqs <= kPlan
__global__ void __launch_bounds__(kPlan) plan_few_kernel(const PlanArgs a, const int fill) {
  __shared__ SmallLds l;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int n = a.n_seqs, shift = a.page_shift;
  const int64_t old_top = min(max(*a.free_count, 0), a.n_pages);
  const Lengths r = lengths_of(a, tid);
  int64_t x[3];   // given back, asked for, new tokens
  x[2] = r.status != 3 && r.want > r.kv ? r.want - r.kv : 0;
  x[0] = r.have > r.need ? r.have - r.need : 0;
  // (a request refused for the slot map's end asks for no pages, but then no
  // later one gets any either)
  x[1] = r.status == 0 && r.need > r.have ? r.need - r.have : 0;
  int64_t s[3] = {x[0], x[1], x[2]};
#pragma unroll
  for (int d = 1; d < 64; d <<= 1)
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int64_t y = __shfl_up(s[q], d);
      if (lane >= d) s[q] += y;
    }
  if (lane == 63)
#pragma unroll
    for (int q = 0; q < 3; ++q) l.wave[w][q] = s[q];
  if (tid == 0) l.got = 0;
  __syncthreads();
  int64_t all[3] = {0, 0, 0};
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    s[q] -= x[q];
    for (int i = 0; i * 64 < n; ++i) {
      const int64_t y = l.wave[i][q];
      if (i < w) s[q] += y;
      all[q] += y;
    }
  }
  const int64_t left = min(old_top + all[0], (int64_t)a.n_pages);   // the stack's top after the pushes
  int32_t status = r.status;
  if (status == 0 && x[2] && s[2] + x[2] > a.slot_cap) status = 4;
  // granted: every page asked for up to here is there; the requests that take
  // pages are so a prefix of those that ask, and take the first ones
  if (status == 0 && x[1] && s[1] + x[1] > left) status = 1;
  l.back[tid] = s[0];
  l.more[tid] = s[1];
  l.fresh[tid] = s[2];
  l.kv[tid] = (int32_t)r.kv;
  l.have[tid] = r.have;
  l.need[tid] = r.need;
  l.status[tid] = status;
  if (status == 0 && x[1]) atomicMax(&l.got, (unsigned long long)(s[1] + x[1]));
  __syncthreads();
  const int64_t got = (int64_t)l.got;
  if (tid < n) {
    a.kv_out[tid] = (int32_t)(status == 0 ? r.want : r.kv);
    a.status[tid] = status;
    a.cu[tid] = (int32_t)min(s[2], (int64_t)INT32_MAX);
  }
  if (tid == 0) {
    a.cu[n] = (int32_t)min(all[2], (int64_t)INT32_MAX);
    *a.free_count_out = (int32_t)(left - got);
  }
  auto given_back = [&](int64_t e) -> int32_t {   // the e-th page pushed
    const int i = owner(l.back, n, e);
    return a.table[(int64_t)i * a.max_pages + l.need[i] + (e - l.back[i])];
  };
  auto page_at = [&](int64_t place) -> int32_t { return place < old_top ? a.free_pages[place] : given_back(place - old_top); };
  if (fill)
    for (int64_t t = tid; t < a.slot_cap; t += kPlan) {
      int64_t slot = -1, p = 0;
      if (t < all[2]) {
        const int i = owner(l.fresh, n, t);
        p = l.kv[i] + (t - l.fresh[i]);
        if (l.status[i] == 0) {
          const int32_t col = (int32_t)(p >> shift);
          const int32_t id = col < l.have[i] ? a.table[(int64_t)i * a.max_pages + col]
                                             : page_at(left - 1 - (l.more[i] + (col - l.have[i])));
          if (id >= 0 && id < a.n_pages) slot = ((int64_t)id << shift) + (p & ((1 << shift) - 1));
        }
      }
      a.slot[t] = slot;
      if (a.pos) a.pos[t] = (int32_t)p;
    }
  for (int64_t e = tid; e < got; e += kPlan) {
    const int i = owner(l.more, n, e);
    a.table[(int64_t)i * a.max_pages + l.have[i] + (e - l.more[i])] = page_at(left - 1 - e);
  }
  for (int64_t e = tid; e < all[0] && old_top + e < a.n_pages; e += kPlan) a.free_pages[old_top + e] = given_back(e);
}

__global__ void __launch_bounds__(kPlan) plan_pages_kernel(const PlanArgs a, const int fill) {
  __shared__ PlanLds l;
  const int tid = threadIdx.x;
  int64_t total;
  int64_t left = min(max(*a.free_count, 0), a.n_pages);   // free pages; the stack's top

  // given back: pushed in request order
  for (int r0 = 0; r0 < a.n_seqs; r0 += kPlan) {
    const Lengths r = lengths_of(a, r0 + tid);
    const int64_t pre = block_scan(r.have > r.need ? r.have - r.need : 0, l, &total);
    if (total) {
      l.pre[tid] = pre;
      l.first[tid] = r.need;
      __syncthreads();
      for (int64_t e = tid; e < total; e += kPlan) {
        const int i = owner(l.pre, kPlan, e);
        if (left + e < a.n_pages)
          a.free_pages[left + e] = a.table[(int64_t)(r0 + i) * a.max_pages + l.first[i] + (e - l.pre[i])];
      }
      left = min(left + total, (int64_t)a.n_pages);
    }
  }
  __syncthreads();   // pushes before pops

  int64_t asked = 0, taken = 0, tokens = 0;
  for (int r0 = 0; r0 < a.n_seqs; r0 += kPlan) {
    const int me = r0 + tid;
    const Lengths r = lengths_of(a, me);
    int32_t status = r.status;
    const int64_t fresh = status != 3 && r.want > r.kv ? r.want - r.kv : 0;
    int64_t n_new;
    const int64_t pre_new = block_scan(fresh, l, &n_new);
    if (status == 0 && fresh && tokens + pre_new + fresh > a.slot_cap) status = 4;
    const int64_t more = status == 0 && r.need > r.have ? r.need - r.have : 0;
    const int64_t pre = block_scan(more, l, &total);
    // granted: every page asked for up to here is there; the requests that
    // take pages are so a prefix of those that ask, and take the first ones
    if (more && asked + pre + more > left) status = 1;
    int64_t got;
    (void)block_scan(status == 0 ? more : 0, l, &got);
    l.pre[tid] = pre;
    l.first[tid] = r.have;
    if (me < a.n_seqs) {
      a.kv_out[me] = (int32_t)(status == 0 ? r.want : r.kv);
      a.status[me] = status;
      a.cu[me] = (int32_t)min(tokens + pre_new, (int64_t)INT32_MAX);
    }
    __syncthreads();
    for (int64_t e = tid; e < got; e += kPlan) {
      const int i = owner(l.pre, kPlan, e);
      a.table[(int64_t)(r0 + i) * a.max_pages + l.first[i] + (e - l.pre[i])] = a.free_pages[left - 1 - asked - e];
    }
    if (fill) {
      __syncthreads();
      l.pre[tid] = pre_new;
      l.first[tid] = (int32_t)r.kv;
      l.row[tid] = status == 0;
      __syncthreads();
      for (int64_t e = tid; e < n_new && tokens + e < a.slot_cap; e += kPlan) {
        const int i = owner(l.pre, kPlan, e);
        const int64_t p = l.first[i] + (e - l.pre[i]);
        a.slot[tokens + e] = l.row[i] ? slot_of(a, r0 + i, p) : -1;
        if (a.pos) a.pos[tokens + e] = (int32_t)p;
      }
    }
    asked += total;
    taken += got;
    tokens += n_new;
  }
  if (tid == 0) {
    a.cu[a.n_seqs] = (int32_t)min(tokens, (int64_t)INT32_MAX);
    *a.free_count_out = (int32_t)(left - taken);
  }
  if (fill)
    for (int64_t t = tokens + tid; t < a.slot_cap; t += kPlan) {
      a.slot[t] = -1;
      if (a.pos) a.pos[t] = 0;
    }
}

// The slot map of a large pack, after the plan: one thread per token.
__global__ void __launch_bounds__(kFill) plan_slots_kernel(const PlanArgs a) {
  const int64_t t = (int64_t)blockIdx.x * kFill + threadIdx.x;
  if (t >= a.slot_cap) return;
  int64_t slot = -1, p = 0;
  if (a.n_seqs > 0 && t < a.cu[a.n_seqs]) {
    const int i = seq_of_token(a.cu, a.n_seqs, (int)t);
    const int ok = a.status[i] == 0;
    // the request's new tokens end at its length where they were granted
    p = (ok ? a.kv_out[i] - (a.cu[i + 1] - a.cu[i]) : a.kv_out[i]) + (t - a.cu[i]);
    if (ok) slot = slot_of(a, i, p);
  }
  a.slot[t] = slot;
  if (a.pos) a.pos[t] = (int32_t)p;
}

}  // namespace

hipError_t launch_plan_pages(const PlanArgs& a, hipStream_t st) {
  const int fill = a.slot_cap <= 4 * kPlan;
  if (a.n_seqs <= kPlan) hipLaunchKernelGGL(plan_few_kernel, dim3(1), dim3(kPlan), 0, st, a, fill);
  else hipLaunchKernelGGL(plan_pages_kernel, dim3(1), dim3(kPlan), 0, st, a, fill);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || fill) return e;
  hipLaunchKernelGGL(plan_slots_kernel, dim3((a.slot_cap + kFill - 1) / kFill), dim3(kFill), 0, st, a);
  return hipGetLastError();
}

}  // namespace gdn
