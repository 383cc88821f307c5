// Internal declarations shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <string>

#include "mf.h"

namespace mfi {

// bits of the per-device status word
enum : uint32_t {
  ST_INDEX = 1u,     // BSR row/column index out of range
  ST_CAPACITY = 2u,  // more kept blocks than capacity
  ST_TIMEOUT = 4u,   // a pipeline wait gave up
  ST_ALIGN = 8u,     // a sequence's map offset is not 16-byte aligned
  ST_PAGE = 16u,     // a page id out of range
  ST_SINGULAR = 32u, // a calibration Gram that is not positive definite
};

// limit of every pipeline wait in the tensor-core kernels (ns) and the test stall flag, as set
// by mf_set_wait_limit (read at each launch)
uint64_t wait_limit_ns();
int wait_stall();
constexpr uint64_t DRAIN_NS = 2000000000ull;  // bound of the waits for work already issued

// scratch of mf_compress (carved out of the caller's workspace)
struct CompressWs {
  int64_t* meta;      // [4 + 4 * nseq]: total rows, total causal blocks, selection ticket, -,
                      // then per sequence (L, nqb, row_base, cb_base)
  double* mass;       // [max_cb] head-summed block masses
  unsigned long long* flags;  // [max_rows] selection look-back: count or prefix per row
  int32_t* kept_row;  // [capacity] BSR row of each kept block
  int64_t max_cb, max_rows;
};

// Computes the layout; with base == nullptr only the size is returned.
size_t compress_ws_layout(const mf_compress_desc& d, CompressWs* ws, void* base);

cudaError_t launch_compress(const mf_compress_desc& d, const CompressWs& ws, uint32_t* status,
                            cudaStream_t st);

// the geometry pass of compression (per-sequence meta; off may be NULL: no map offsets)
cudaError_t launch_meta(const int32_t* cu, const int64_t* off, int nseq, int max_seqlen, int B,
                        int elem_bytes, const CompressWs& ws, uint32_t* status, int32_t* row_ptr,
                        int32_t* nnz_out, cudaStream_t st);
// selection and BSR index build from the masses of every causal block
cudaError_t launch_select(const CompressWs& ws, int nseq, int max_seqlen, int B, const double* mass,
                          double tau, int32_t* row_ptr, int32_t* col_idx, int32_t* nnz_out,
                          int64_t capacity, uint32_t* status, cudaStream_t st);

// scratch of mf_compress_qk beyond CompressWs
struct QkWs {
  float2* ml;         // [h_s][cb_stride][B] per-block max and exp-sum of each row
  float* lse2;        // [h_s][T] row log2-sum-exp
  int64_t cb_stride;  // causal-block capacity of the pack
};
size_t compress_qk_ws_layout(const mf_compress_qk_desc& d, CompressWs* ws, QkWs* q, void* base);
bool launch_compress_qk(const mf_compress_qk_desc& d, const CompressWs& ws, const QkWs& q,
                        uint32_t* status, cudaStream_t st, std::string* err);

// one receiver layer's pointers
struct RetrieveLayer {
  const int32_t* row_ptr;
  const int32_t* col_idx;
  const void* values;
  int64_t capacity;
  const float* W;  // [h_r][h_s] of this layer
  const void* V;   // this layer's V
  void* O;         // this layer's O
};

cudaError_t launch_retrieve_simt(const mf_retrieve_desc& d, const RetrieveLayer& l,
                                 uint32_t* status, cudaStream_t st);

bool tc_supported(const mf_retrieve_desc& d);

// one launch for n (1..4) receivers that share the sender BSR layer and the query / key
// packing; returns false and fills *err on a host-side failure (tensor-map encoding, launch).
// Every launch may start while the previous kernel on the stream still runs (programmatic
// dependent launch).  first: the call's first launch, which waits for that kernel before its
// first global access; later launches of one call read nothing the earlier ones write.
bool launch_retrieve_tc(const mf_retrieve_desc* const* ds, const RetrieveLayer* ls, int n,
                        uint32_t* status, cudaStream_t st, std::string* err, bool first = true);

// prefix-hash block cache
struct BlockCache;
BlockCache* cache_create(const mf_cache_desc& d);
void cache_destroy(BlockCache* c);
int64_t cache_put(BlockCache* c, int layer, const mf_bsr& bsr, const int32_t* row_ptr_host,
                  const int32_t* col_idx_host, int64_t row0, int nrows, const uint64_t* hashes,
                  cudaStream_t st);
bool cache_get(BlockCache* c, int layer, const uint64_t* hashes, int nrows, int32_t* row_ptr,
               int32_t* col_idx, void* values, int64_t capacity, int* hit, cudaStream_t st);
void cache_stats(BlockCache* c, int64_t* out6);

// head-map calibration
size_t calib_ws_bytes(const mf_calib_desc& d);
int calib_path(const mf_calib_desc& d);
// returns false and fills *err on a host-side failure
bool launch_calib_gram(const mf_calib_desc& d, void* ws, uint32_t* status, cudaStream_t st,
                       std::string* err);
cudaError_t launch_calib_solve(const double* gram, int h_s, int h_r, double ridge, float* W,
                               double* residual, uint32_t* status, cudaStream_t st);

// Raises a kernel's limit of dynamic shared memory to `bytes`, once per device: the most that any
// call takes, for the limit is the process's, and another thread's call may be about to launch.
template <auto Kernel> cudaError_t allow_smem(int dev, int bytes) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launches of the paged cache's calls overlap with the end of the kernel before them in the stream:
// every kernel is launched with `launch_early` and waits with `await_earlier`, in every CTA, before
// its first access to memory that another kernel may touch (a call's second kernel may read its
// inputs before that, if the first one has waited for them).  `allow_later` lets the next kernel
// take its place already; only a kernel that another one of its call follows does so: CTAs of a
// next call that wait in the SMs cost more than their launch (131072 slots cut to an eighth 50.8 us
// instead of 44.8, without early launches 47.2; a decode of one short sequence 4.4, 4.1 and 6.2).
__device__ __forceinline__ void await_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_later() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                         cudaStream_t st, const A&... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// single-token attention over the paged cache: scratch carved out of the caller's workspace
struct PagedDecodeWs {
  int32_t* pre;     // [nseq + 1] tiles before each sequence
  int64_t* per;     // tiles of a CTA
  float* lse2;      // [nseq][h_r]
  float* part_O;    // parts of the units cut between CTAs
  float2* part_ml;
  float* S;         // x_j of every query head and key (with score_out)
};
size_t paged_decode_ws(const mf_paged_decode_desc& d, PagedDecodeWs* ws, void* base);
cudaError_t launch_paged_decode(const mf_paged_decode_desc& d, const PagedDecodeWs& ws,
                                uint32_t* status, cudaStream_t st);

cudaError_t launch_kv_append(const mf_kv_append_desc& d, uint32_t* status, cudaStream_t st);

// eviction: the rows to move, per (sequence, key head)
struct KvEvictWs {
  int32_t* count;   // [nseq][h_kv] rows to move
  int32_t* len;     // [nseq] new lengths
  int32_t* dst;     // [nseq][h_kv][moves]
  int32_t* src;
  int64_t moves;    // most rows that one (sequence, key head) can move
};
size_t kv_evict_ws(const mf_kv_evict_desc& d, KvEvictWs* ws, void* base);
cudaError_t launch_kv_evict(const mf_kv_evict_desc& d, const KvEvictWs& ws, uint32_t* status,
                            cudaStream_t st);

// weights gathered in a prefill: [slots][h_kv][B] column sums of mixed blocks, one slot per
// stretch of blocks that a CTA shares with no other
struct KeyScoresWs {
  float* part;
};
size_t key_scores_ws(const mf_key_scores_desc& d, KeyScoresWs* ws, void* base);
cudaError_t launch_key_scores(const mf_key_scores_desc& d, const KeyScoresWs& ws, uint32_t* status,
                              cudaStream_t st);

}  // namespace mfi
