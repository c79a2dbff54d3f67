// Internal interface between the C-ABI host layer and the launchers of the
// paged 8-bit key/value cache and the attention over it.  Every struct here is
// filled only after the host layer validated the call.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

// The paged 8-bit key/value cache as the kernels see it.
struct CacheRef {
  int32_t Hkv, dim;
  int32_t page_shift;      // log2 of the page's tokens
  int32_t n_pages;
  int32_t i8;              // codes are int8 (else e4m3)
  uint8_t* k;              // [n_pages, Hkv, page, dim]
  uint8_t* v;              // [n_pages, Hkv, page/16, dim, 16]
  float* ks;               // [n_pages, Hkv]
  float* vs;
};

struct PlanArgs {
  int32_t page_shift, n_seqs, max_pages, n_pages, slot_cap;
  const int32_t* want;
  const int32_t* kv;
  int32_t* kv_out;         // may equal kv
  int32_t* table;          // [n_seqs, max_pages]
  int32_t* free_pages;     // [n_pages]
  const int32_t* free_count;
  int32_t* free_count_out; // may equal free_count
  int32_t* cu;             // [n_seqs + 1]
  int64_t* slot;           // [slot_cap]
  int32_t* pos;            // [slot_cap] or nullptr
  int32_t* status;         // [n_seqs]
};

struct RopeRef {
  int32_t rot, n_axes, adjacent;
  float scale;
  float freq[128];
  uint8_t axis[128];
};

struct AppendArgs {
  RopeRef rope;
  CacheRef c;
  int32_t Hq, n_seqs, n_tokens;
  const int32_t* cu;
  const uint16_t* q;       // [T, Hq, d] or nullptr
  const uint16_t* k;       // [T, Hkv, d]
  const uint16_t* v;
  uint16_t* q_out;
  int64_t q_stride, k_stride, v_stride, qo_stride;
  const int32_t* pos;      // axis a of token t at a * pos_stride + t
  int64_t pos_stride;
  const int64_t* slot;     // [T]
};

struct GatherArgs {
  CacheRef c;
  int32_t n_tokens;
  const int64_t* slot;
  uint16_t* k_out;         // [T, Hkv, d] or nullptr
  uint16_t* v_out;
};

// A packed prompt with no more rows than this (tokens x Hq / Hkv) is computed
// as a decoding request is, four waves sharing its keys.  The rule goes by the
// prompt's own rows, so its bits do not depend on the pack.  Measured with it
// and without it, 4 kv heads of 64, 128 and 256, int8, in us:
//   1 prompt of 16 rows on 4,096 keys    32 and  92   40 and 115   72 and 237
//   8 of 64 rows on 3,000                36 and  71   47 and  88   65 and 180
//   64 of 64 rows on 2,000               37 and  65   54 and  82  154 and 158
//   8 of 128 rows on 3,000               38 and  71   49 and  90   70 and 184 *
//   64 of 128 rows on 2,000              62 and  66   98 and  86  295 and 169 *
// (* with a limit of 128, which heads of 256 do not have.)  64 prompts fill the
// card: there 128 rows of 128 cost a seventh more with the rule, against the
// half that it saves where they are few.
constexpr int few_rows(int dim) { return dim == 256 ? 64 : 128; }

// 16-row tiles of a wave there, for `rows` rows of the longest of them (heads
// of 256: one for all, as the steps differ in length, and with them the bits).
constexpr int few_tiles(int dim, int rows) { return rows <= 16 || dim == 256 ? 1 : 2; }

struct AttnArgs {
  CacheRef c;
  int32_t Hq, n_seqs, n_tokens;
  int32_t n_tok;           // rows per request (decode), 0 = rows by cu
  int32_t few, many;       // packed: tokens of the longest prompt of up to few_rows() rows; prompts with more
  float scale;
  const int32_t* cu;
  const int32_t* kv_len;   // [n_seqs]
  const int32_t* table;    // [n_seqs, max_pages]
  int32_t max_pages;
  int32_t max_kv;          // lengths over it make NaN rows
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;           // [T, Hq, d]
};

hipError_t launch_plan_pages(const PlanArgs& a, hipStream_t stream);
hipError_t launch_rope_append(const AppendArgs& a, hipStream_t stream);
hipError_t launch_cache_gather(const GatherArgs& a, hipStream_t stream);
hipError_t launch_attn_packed(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_few(const AttnArgs& a, hipStream_t stream);   // the packed prompts of few rows
int attn_decode_splits(int dim, int max_kv);   // workgroups that share a request's keys
int64_t attn_decode_bytes(int dim, int Hq, int batch, int n_tok, int max_kv);
hipError_t launch_attn_decode(const AttnArgs& a, void* workspace, hipStream_t stream);

}  // namespace gdn
