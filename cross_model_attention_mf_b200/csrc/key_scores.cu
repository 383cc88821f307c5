// Weights every key gathered in a prefill that reused a sender's maps (mf_map_key_scores):
//   score[g][j] = sum_{r in g} sum_{i >= j} sum_s W[r][s] A_s[i][j]
//               = sum_s wg[g][s] colsum_s[j],   wg[g][s] = sum_{r in g} W[r][s],
// over the kept blocks.  Every kept value is read once (nnz h_s B^2 elements, one addition each),
// which bounds the call by HBM bandwidth; the mix of the column sums is B times smaller.
//
// k_colsum   the (block, sender head) tiles of the BSR lie on a line that the CTAs share evenly.
//            A warp sums one B x B tile's columns (16-byte loads, each lane a fixed chunk of
//            columns), the CTA mixes its heads' sums per block and writes one [h_kv][B] part per
//            block it touches: part n + c for block n and CTA c, since a block is shared only
//            by consecutive CTAs.
// k_colmerge CTA (sequence, key block): finds the block's column in every later query-block row
//            (binary search of the ascending columns), then adds the parts in ascending order in
//            float64.
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>

#include "mf_internal.cuh"

namespace mfi {
namespace {

constexpr int CS_WARPS = 8;
constexpr int CS_THR = 32 * CS_WARPS;
constexpr int CS_GRID = 592;   // most CTAs of k_colsum
constexpr int CS_HEADS = 32;   // sender heads mixed at a time

struct ColParams {
  const int32_t* row_ptr;
  const int32_t* col_idx;
  const char* values;
  int64_t capacity, n_rows;
  int h_s, h_r, h_kv;
  const float* W;
  const int32_t* cu;
  const int32_t* base;
  int nseq, max_len, nqb_max;
  float* score;
  int64_t stride;
  float* part;
  int grid;
  uint32_t* status;
};

// blocks of the BSR, within its capacity
__device__ __forceinline__ int64_t block_count(const ColParams& p, bool report) {
  const int64_t n = p.row_ptr[p.n_rows];
  if (n >= 0 && n <= p.capacity) return n;
  if (report) atomicOr(p.status, ST_INDEX);
  return n < 0 ? 0 : p.capacity;
}
__device__ __forceinline__ int64_t tiles_per_cta(int64_t n_blocks, int h_s, int grid) {
  return max((int64_t)1, (n_blocks * h_s + grid - 1) / grid);
}

template <typename T, int B>
__global__ void __launch_bounds__(CS_THR) k_colsum(const __grid_constant__ ColParams p) {
  constexpr int E = 16 / sizeof(T);        // elements per 16-byte chunk
  constexpr int CPR = B / E;               // chunks per tile row
  constexpr int RPI = 32 / CPR;            // rows a warp reads per load
  constexpr int NL = B / RPI;              // loads per tile
  constexpr int UNR = NL < 8 ? NL : 8;
  extern __shared__ float sm[];
  float* wg = sm;                          // [h_s][h_kv]
  float* acc = wg + p.h_s * p.h_kv;        // [h_kv][B]
  float* col = acc + p.h_kv * B;           // [CS_HEADS][B]
  __shared__ int s_live[2];                // query block minus key block, rows inside the sequence
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t nb = block_count(p, blockIdx.x == 0 && tid == 0);
  const int64_t per = tiles_per_cta(nb, p.h_s, p.grid);
  int64_t x = per * blockIdx.x;
  const int64_t end = min(nb * p.h_s, x + per);
  if (x >= end) return;
  const int gs = p.h_r / p.h_kv;
  for (int i = tid; i < p.h_s * p.h_kv; i += CS_THR) {
    const int h = i / p.h_kv, g = i - h * p.h_kv;
    float w = 0.0f;
    for (int r = 0; r < gs; ++r) w += p.W[(int64_t)(g * gs + r) * p.h_s + h];
    wg[i] = w;
  }
  const int chunk = lane % CPR, row0 = lane / CPR;
  while (x < end) {
    const int64_t n = x / p.h_s;
    const int h_lo = (int)(x - n * p.h_s), h_hi = (int)min((int64_t)p.h_s, h_lo + (end - x));
    x += h_hi - h_lo;
    if (tid == 0) s_live[0] = -1;
    for (int i = tid; i < p.h_kv * B; i += CS_THR) acc[i] = 0.0f;
    __syncthreads();
    // the block's row, and the sequence the row belongs to
    for (int s = warp; s < p.nseq; s += CS_WARPS) {
      const int L = p.cu[s + 1] - p.cu[s];
      const int nq = (L + B - 1) / B, b = p.base[s];
      if (L <= 0 || L > p.max_len || b < 0 || (int64_t)b + nq > p.n_rows) continue;
      if (p.row_ptr[b] > n || p.row_ptr[b + nq] <= n) continue;
      for (int q = lane; q < nq; q += 32)
        if (p.row_ptr[b + q] <= n && n < p.row_ptr[b + q + 1]) {
          const int c = p.col_idx[n];
          if (c < 0 || c > q) {
            atomicOr(p.status, ST_INDEX);
          } else {
            s_live[0] = q - c;
            s_live[1] = L - q * B;
          }
        }
    }
    __syncthreads();
    const int diff = s_live[0], rows = s_live[1];
    if (diff >= 0) {  // a block of no sequence, or with a bad column, counts for nothing
      const bool masked = diff == 0 || rows < B;
      for (int h0 = h_lo; h0 < h_hi; h0 += CS_HEADS) {
        const int hn = min(CS_HEADS, h_hi - h0);
        for (int h = warp; h < hn; h += CS_WARPS) {
          const uint4* t = reinterpret_cast<const uint4*>(p.values + (n * p.h_s + h0 + h) * (int64_t)(B * B * sizeof(T))) + lane;
          float c[E];
#pragma unroll
          for (int k = 0; k < E; ++k) c[k] = 0.0f;
#pragma unroll 1
          for (int i0 = 0; i0 < NL; i0 += UNR) {
            uint4 v[UNR];
#pragma unroll
            for (int i = 0; i < UNR; ++i) v[i] = __ldcs(t + (i0 + i) * 32);
#pragma unroll
            for (int i = 0; i < UNR; ++i) {
              const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
              const int row = (i0 + i) * RPI + row0;
#pragma unroll
              for (int k = 0; k < E; ++k) {
                float f;
                if (sizeof(T) == 4) f = __uint_as_float(w[k & 3]);
                else f = __uint_as_float(k & 1 ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16);
                if (masked && (row >= rows || (diff == 0 && chunk * E + k > row))) f = 0.0f;
                c[k] += f;
              }
            }
          }
#pragma unroll
          for (int o = CPR; o < 32; o <<= 1)
#pragma unroll
            for (int k = 0; k < E; ++k) c[k] += __shfl_xor_sync(~0u, c[k], o);
          if (row0 == 0)
#pragma unroll
            for (int k = 0; k < E; ++k) col[h * B + chunk * E + k] = c[k];
        }
        __syncthreads();
        for (int i = tid; i < p.h_kv * B; i += CS_THR) {
          const int g = i / B, j = i % B;
          float a = acc[i];
          for (int h = 0; h < hn; ++h) a = fmaf(wg[(h0 + h) * p.h_kv + g], col[h * B + j], a);
          acc[i] = a;
        }
        __syncthreads();
      }
    }
    float* out = p.part + (n + blockIdx.x) * p.h_kv * B;
    for (int i = tid; i < p.h_kv * B; i += CS_THR) out[i] = acc[i];
    __syncthreads();
  }
}

constexpr int CM_THR = 256;

__global__ void __launch_bounds__(CM_THR) k_colmerge(const __grid_constant__ ColParams p, int B) {
  extern __shared__ int32_t s_n[];  // block of every query-block row, -1 where it was not kept
  const int s = blockIdx.x / p.nqb_max, kb = blockIdx.x - s * p.nqb_max;
  const int tid = threadIdx.x;
  const int L = p.cu[s + 1] - p.cu[s];
  const int b = p.base[s];
  const int nq = (int)(((int64_t)L + B - 1) / B);
  if (L < 0 || L > p.max_len || b < 0 || (int64_t)b + nq > p.n_rows) {
    if (kb == 0 && tid == 0) atomicOr(p.status, ST_INDEX);
    return;
  }
  if (kb >= nq) return;
  for (int q = kb + tid; q < nq; q += CM_THR) {
    int lo = p.row_ptr[b + q], hi = p.row_ptr[b + q + 1];
    int at = -1;
    if (lo < 0 || hi < lo || hi > p.capacity) {
      atomicOr(p.status, ST_INDEX);
    } else {
      const int top = hi;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.col_idx[mid] < kb) lo = mid + 1; else hi = mid;
      }
      if (lo < top && p.col_idx[lo] == kb) at = lo;
    }
    s_n[q - kb] = at;
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t nb = block_count(p, false);
  const int64_t per = tiles_per_cta(nb, p.h_s, p.grid);
  const int width = min(B, L - kb * B);
  for (int i = tid; i < p.h_kv * width; i += CM_THR) {
    const int g = i / width, j = i - g * width;
    double sum = 0.0;
    for (int q = 0; q < nq - kb; ++q) {
      const int n = s_n[q];
      if (n < 0 || n >= nb) continue;
      const int64_t c0 = (int64_t)n * p.h_s / per, c1 = ((int64_t)n * p.h_s + p.h_s - 1) / per;
      for (int64_t c = c0; c <= c1; ++c) sum += (double)p.part[((n + c) * p.h_kv + g) * B + j];
    }
    p.score[((int64_t)s * p.h_kv + g) * p.stride + (int64_t)kb * B + j] = (float)sum;
  }
}

}  // namespace

size_t key_scores_ws(const mf_key_scores_desc& d, KeyScoresWs* ws, void* base) {
  if (ws) ws->part = static_cast<float*>(base);
  const size_t n = ((size_t)d.bsr.capacity_blocks + CS_GRID) * d.h_kv * d.B * sizeof(float);
  return (n + 255) & ~size_t(255);
}

cudaError_t launch_key_scores(const mf_key_scores_desc& d, const KeyScoresWs& ws, uint32_t* status,
                              cudaStream_t st) {
  ColParams p{};
  p.row_ptr = d.bsr.row_ptr;
  p.col_idx = d.bsr.col_idx;
  p.values = static_cast<const char*>(d.bsr.values);
  p.capacity = d.bsr.capacity_blocks;
  p.n_rows = d.n_rows;
  p.h_s = d.h_s;
  p.h_r = d.h_r;
  p.h_kv = d.h_kv;
  p.W = d.W;
  p.cu = d.cu_seqlens;
  p.base = d.qblock_base;
  p.nseq = d.nseq;
  p.max_len = d.max_seqlen;
  p.nqb_max = (d.max_seqlen + d.B - 1) / d.B;
  p.score = d.score;
  p.stride = d.score_stride;
  p.part = ws.part;
  p.status = status;
  if (p.nqb_max == 0) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  p.grid = std::min(CS_GRID, 4 * sms);
  const size_t smem = sizeof(float) * ((size_t)d.h_s * d.h_kv + (size_t)d.h_kv * d.B + (size_t)CS_HEADS * d.B);
  auto launch = [&](auto kern) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return;
    kern<<<p.grid, CS_THR, smem, st>>>(p);
    e = cudaGetLastError();
  };
  if (d.map_dtype == MF_F32) {
    if (d.B == 32) launch(k_colsum<float, 32>);
    else if (d.B == 64) launch(k_colsum<float, 64>);
    else launch(k_colsum<float, 128>);
  } else {
    if (d.B == 32) launch(k_colsum<__nv_bfloat16, 32>);
    else if (d.B == 64) launch(k_colsum<__nv_bfloat16, 64>);
    else launch(k_colsum<__nv_bfloat16, 128>);
  }
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  cfg.gridDim = dim3((unsigned)((int64_t)p.nseq * p.nqb_max));
  cfg.blockDim = dim3(CM_THR);
  cfg.dynamicSmemBytes = 4 * (size_t)p.nqb_max;
  cfg.stream = st;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_colmerge, p, d.B);
}

}  // namespace mfi
