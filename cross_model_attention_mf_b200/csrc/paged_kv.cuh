// The receiver's paged key-value cache as the kernels see it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mf_internal.cuh"

namespace mfi {

// n / d by a product, 0 <= n < 2^31: with 2^l >= d and mul = floor(2^(31+l) / d) + 1 the product
// exceeds n 2^(31+l) / d by at most n 2^l / d, too little to reach the next quotient.
struct Divider {
  uint32_t mul;
  int shift;
  Divider(int d = 1) {
    int l = 0;
    while (((int64_t)1 << l) < d) ++l;
    shift = 31 + l;
    mul = (uint32_t)((uint64_t(1) << shift) / (uint64_t)d + 1);
  }
  __device__ int of(int n) const { return (int)(((uint64_t)(uint32_t)n * mul) >> shift); }
};

struct KvView {
  char* K;
  char* V;
  int64_t page_bytes;  // between pages
  int32_t slot_bytes;  // h_kv * d * element: one slot's rows of every key head
  int32_t row_bytes;   // d * element: one key head's row
  int n_pages, page_size, max_pages, nseq, max_len;
  Divider by_page;     // by page_size
  int top;             // the longest length: max_len, or the slots of the table
  const int32_t* table;
  const int32_t* lens;
  uint32_t* status;
};

inline KvView kv_view(const mf_paged_kv& k, uint32_t* status) {
  const int e = k.dtype == MF_F32 ? 4 : 2;
  KvView v;
  v.K = static_cast<char*>(k.K);
  v.V = static_cast<char*>(k.V);
  v.row_bytes = k.d * e;
  v.slot_bytes = k.h_kv * v.row_bytes;
  v.page_bytes = k.page_stride ? k.page_stride * e : (int64_t)k.page_size * v.slot_bytes;
  v.n_pages = k.n_pages;
  v.page_size = k.page_size;
  v.by_page = Divider(k.page_size);
  v.top = (int)std::min<int64_t>(k.max_len, (int64_t)k.max_pages * k.page_size);
  v.max_pages = k.max_pages;
  v.nseq = k.nseq;
  v.max_len = k.max_len;
  v.table = k.block_table;
  v.lens = k.seq_lens;
  v.status = status;
  return v;
}

// sequence length, within [0, max_len] and the table's slots; `report` sets the status bit for
// one that is not
__device__ __forceinline__ int kv_len(const KvView& v, int s, bool report) {
  const int len = v.lens[s];
  if ((unsigned)len <= (unsigned)v.top) return len;
  if (report) atomicOr(v.status, ST_INDEX);
  return len < 0 ? 0 : v.top;
}

// floor of a / b for a >= 0, b > 0 (a 64-bit division takes four times the instructions)
__device__ __forceinline__ int64_t div_floor(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// where a slot lies: its page's place in the table, its row in the page
struct KvPlace {
  int page, row;
};
__device__ __forceinline__ KvPlace kv_place(const KvView& v, int slot) {
  const int page = v.by_page.of(slot);
  return {page, slot - page * v.page_size};
}
// the page id of sequence s in that place
__device__ __forceinline__ int kv_page(const KvView& v, int s, const KvPlace& at) {
  return v.table[(int64_t)s * v.max_pages + at.page];
}
// byte offset (from K or V) of the slot's first head row in page `id`, -1 for an id out of range
__device__ __forceinline__ int64_t kv_offset(const KvView& v, int id, const KvPlace& at) {
  if ((unsigned)id >= (unsigned)v.n_pages) {
    atomicOr(v.status, ST_PAGE);
    return -1;
  }
  return (int64_t)id * v.page_bytes + (int64_t)at.row * v.slot_bytes;
}
__device__ __forceinline__ int64_t kv_slot(const KvView& v, int s, int slot) {
  const KvPlace at = kv_place(v, slot);
  return kv_offset(v, kv_page(v, s, at), at);
}

}  // namespace mfi
