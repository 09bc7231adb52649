// The 4-bit paged cache: its layout on the device, and how a call's rows name
// sequences, positions and places.
#pragma once
#include <stdint.h>

#include "kv4_slot.h"

namespace wpk {

struct Kv4Dev {
  uint8_t* pages;        // [n_blocks][n_kv][page_bytes]
  const int32_t* table;  // [batch][max_blocks]
  int64_t n_blocks;
  int batch, max_blocks, n_kv, page_tokens, page_bytes;
  uint64_t page_magic;   // kv4_page_magic(page_tokens)
  const int32_t* pos;     // [batch] position of a sequence's first new token; < 0 = idle
  const int32_t* indptr;  // [batch + 1], or NULL: `each` tokens per sequence
  const int32_t* n_seq;   // sequences in use (device), or NULL: batch
  int total, each;
  int rope_positions;     // positions with a rotation (INT_MAX without a rope table)
};

__device__ __forceinline__ int kv4_sequences(const Kv4Dev& c) { return c.n_seq ? min(c.batch, *c.n_seq) : c.batch; }

__device__ __forceinline__ int kv4_slot(const Kv4Dev& c, int position) { return kv4_slot_of(position, c.page_magic); }

// First byte of (block, kv head)'s page.
__device__ __forceinline__ uint8_t* kv4_page(const Kv4Dev& c, int block, int head) {
  return c.pages + ((int64_t)block * c.n_kv + head) * c.page_bytes;
}

// New tokens [q0, q0 + n) of sequence b, cut to the rows that the call has.
__device__ __forceinline__ void kv4_new(const Kv4Dev& c, int b, int* q0, int* n) {
  int lo, hi;
  if (c.indptr) {
    lo = c.indptr[b];
    hi = min(c.indptr[b + 1], c.total);
  } else {
    lo = b * c.each;
    hi = lo + c.each;
  }
  *q0 = lo;
  *n = lo < 0 || hi < lo ? 0 : hi - lo;
}

}  // namespace wpk
