// The receiver's paged key-value cache as the kernels see it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "mf_internal.cuh"

namespace mfi {

// Raises a kernel's limit of dynamic shared memory to `bytes`, once per device.
template <auto Kernel> cudaError_t allow_smem(int dev, int bytes) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

struct KvView {
  char* K;
  char* V;
  int64_t page_bytes;  // between pages
  int32_t slot_bytes;  // h_kv * d * element: one slot's rows of every key head
  int32_t row_bytes;   // d * element: one key head's row
  int n_pages, page_size, max_pages, nseq, max_len;
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
  const int64_t room = (int64_t)v.max_pages * v.page_size;
  const int top = room < v.max_len ? (int)room : v.max_len;
  if (len >= 0 && len <= top) return len;
  if (report) atomicOr(v.status, ST_INDEX);
  return len < 0 ? 0 : top;
}

// page of a slot of sequence s, as the table has it
__device__ __forceinline__ int kv_page(const KvView& v, int s, int slot) {
  return v.table[(int64_t)s * v.max_pages + slot / v.page_size];
}
// byte offset (from K or V) of a slot's first head row in that page, -1 for a page id out of range
__device__ __forceinline__ int64_t kv_offset(const KvView& v, int page, int slot) {
  if (page < 0 || page >= v.n_pages) {
    atomicOr(v.status, ST_PAGE);
    return -1;
  }
  return (int64_t)page * v.page_bytes + (int64_t)(slot % v.page_size) * v.slot_bytes;
}
__device__ __forceinline__ int64_t kv_slot(const KvView& v, int s, int slot) {
  return kv_offset(v, kv_page(v, s, slot), slot);
}

}  // namespace mfi
