// Host-side launches of the rotary and cache kernels (rope.cu, cache.cu).
#pragma once

#include "common.h"

namespace attn {

// Up to three tensors of `heads` heads each; element offset of (b, head, n) is
// b * sb + head * sh + n * st.  With slots, tensors 1 and 2 go to rows
// slots[n] of caches [num_slots, heads, d].
struct RopeKParams {
  const uint16_t* src[3];
  uint16_t* dst[3];
  long long sb[3], sh[3], st[3];
  long long db[3], dh[3], dt[3];
  int heads[3];
  int rotated;                 // tensors 0 .. rotated - 1 are rotated
  const float* cos;            // [max_pos, rot / 2]
  const float* sin;
  const int* positions;        // [B * N], or nullptr: the row's index n, or with
  const int* cu_seqlens;       // [requests + 1] and seq_lens the last positions of
  const int* seq_lens;         // the request that owns the row
  int requests;
  const long long* slots;      // [N], or nullptr
  long long num_slots;
  int* status;
  int B, N, d, rot, max_pos;
  int inverse;
  int heads_per_chunk;
};

attn_status_t launch_rope_table(float* cos_out, float* sin_out, long long n, int rot, double base,
                                double factor, long long orig_len, double low, double high,
                                double attn_factor, long long first, cudaStream_t stream);

struct TablesParams {
  int* block_table;          // [B, max_pages], entries of new pages written
  const int* old_lens;       // [B]
  const int* new_lens;       // [B]
  const int* free_pages;     // [n_free]
  int* seq_lens;             // [B]
  int* cu_seqlens;           // [B + 1]
  long long* slots;          // [capacity]
  int* positions;            // [capacity]
  int* used;                 // [1]
  int B, max_pages, n_free, page_size, capacity;
};
attn_status_t launch_block_tables(const TablesParams& p, cudaStream_t stream);

// New keys and values [total, H_kv, 128] of packed requests into an e4m3 paged
// cache with one descale per (page, head).
struct AppendFp8Params {
  const void* k;
  const void* v;
  long long kt, kh, vt, vh;      // element strides of tokens and heads
  uint8_t* k_cache;              // [num_pages, page_size, H_kv, 128]
  uint8_t* v_cache;
  float* k_descale;              // [num_pages, H_kv]
  float* v_descale;
  const int* block_table;        // [B, max_pages]
  const int* seq_lens;           // [B], the new tokens counted
  const int* cu_seqlens;         // [B + 1]
  const float* cos;              // or nullptr
  const float* sin;
  const float* signs;            // or nullptr
  int* status;
  int B, total, H_kv, num_pages, page_size, max_pages, rot, max_pos;
};
// q: query rows to rotate in the same launch (heads[0] = 0: none).
attn_status_t launch_append_fp8(AppendFp8Params p, RopeKParams q, int fp16, int interleaved,
                                cudaStream_t stream);
attn_status_t launch_rope(RopeKParams p, int fp16, int interleaved, cudaStream_t stream);

}  // namespace attn
