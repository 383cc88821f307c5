// Weights every key gathered in a prefill that reused a sender's maps (mf_map_key_scores):
//   score[g][j] = sum_{r in g} sum_{i >= j} sum_s W[r][s] A_s[i][j]
//               = sum_s wg[g][s] colsum_s[j],   wg[g][s] = sum_{r in g} W[r][s],
// over the kept blocks.  Every kept value is read once (nnz h_s B^2 elements, one addition each),
// which bounds the call by HBM bandwidth; the mix of the column sums is B times smaller.
//
// k_colsum   the (block, sender head) tiles of the BSR lie on a line that the CTAs share evenly.
//            A warp sums one B x B tile's columns (16-byte loads, each lane a fixed chunk of
//            columns) and fetches the start of its next tile before it leaves the present one,
//            so that loads are on their way while the CTA finds a block's row, mixes its heads'
//            sums and writes one [h_kv][B] part per block it touches: part n + c for block n and
//            CTA c, since a block is shared only by consecutive CTAs.
// k_colmerge CTA (sequence, key block): lists the parts of the block's column in every later
//            query-block row (binary search of the ascending columns; this runs beside k_colsum),
//            then adds them in float64, in slices of the list that are joined in order.
//
// Measured (one B200; copy rate 6469 GB/s): 1.17 GB of kept blocks (4 sequences, 40 sender heads)
// 198 us, 91% of that rate (k_colsum 187: masked tiles have a loop of their own, without which it
// was bound by instructions at 236); 58 MB (8192 tokens, 3% of the blocks) 19.5 us: 4 us until the
// first block's row is known, 10 for two or three tiles a warp, 3 for the merge.  Three CTAs of
// k_colsum to an SM: two took 205 us, four (with spills) 197 and 21 for the small case.
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "mf_internal.cuh"

namespace mfi {
namespace {

constexpr int CS_WARPS = 8;
constexpr int CS_THR = 32 * CS_WARPS;
constexpr int CS_CTAS = 3;     // resident on an SM
constexpr int CS_GRID = 592;   // most CTAs of k_colsum
constexpr int CS_HEADS = 32;   // sender heads mixed at a time
constexpr int MAX_SENDERS = 256, MAX_KEY_HEADS = 64;  // h_s and h_kv, as the entry point checks

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
  if (p.n_rows == 0) return 0;
  const int64_t n = p.row_ptr[p.n_rows];
  if (n >= 0 && n <= p.capacity) return n;
  if (report) atomicOr(p.status, ST_INDEX);
  return n < 0 ? 0 : p.capacity;
}
__device__ __forceinline__ int64_t tiles_per_cta(int64_t n_blocks, int h_s, int grid) {
  return max((int64_t)1, (n_blocks * h_s + grid - 1) / grid);
}

// k-th element of 16 bytes
template <typename T> __device__ __forceinline__ float element(const uint4& v, int k) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (sizeof(T) == 4) return __uint_as_float(w[k & 3]);
  return __uint_as_float(k & 1 ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16);
}

template <typename T, int B>
__global__ void __launch_bounds__(CS_THR, CS_CTAS) k_colsum(const __grid_constant__ ColParams p) {
  constexpr int E = 16 / sizeof(T);        // elements per 16-byte chunk
  constexpr int CPR = B / E;               // chunks per tile row
  constexpr int RPI = 32 / CPR;            // rows a warp reads per load
  constexpr int NL = B / RPI;              // loads per tile
  constexpr int UNR = NL < 8 ? NL : 8;
  constexpr int TILE = B * B * sizeof(T);
  extern __shared__ float sm[];
  float* wg = sm;                          // [h_s][h_kv]
  float* acc = wg + p.h_s * p.h_kv;        // [h_kv][B]
  float* col = acc + p.h_kv * B;           // [CS_HEADS][B]
  __shared__ uint32_t s_lo, s_hi;          // least and largest (query block, live rows) that a sequence gives the row
  await_earlier();
  allow_later();  // k_colmerge reads the maps' indices before it waits: not before this kernel may
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t nb = block_count(p, blockIdx.x == 0 && tid == 0);
  const int64_t per = tiles_per_cta(nb, p.h_s, p.grid);
  int64_t x = per * blockIdx.x;
  const int64_t end = min(nb * p.h_s, x + per);
  if (x >= end) return;
  const int chunk = lane % CPR, row0 = lane / CPR;
  uint4 v[UNR];
  auto fetch = [&](int64_t tile, int i0) {
    const uint4* t = reinterpret_cast<const uint4*>(p.values + tile * TILE) + i0 * 32 + lane;
#pragma unroll
    for (int i = 0; i < UNR; ++i) v[i] = __ldcs(t + i * 32);
  };
  int64_t n = x / p.h_s;
  int h_lo = (int)(x - n * p.h_s);
  int h_hi = (int)min((int64_t)p.h_s, h_lo + (end - x));
  if (h_lo + warp < h_hi) fetch(x + warp, 0);
  int kb = p.col_idx[n];
  const int gs = p.h_r / p.h_kv;
  for (int i = tid; i < p.h_s * p.h_kv; i += CS_THR) {
    const int h = i / p.h_kv, g = i - h * p.h_kv;
    float w = 0.0f;
#pragma unroll 4
    for (int r = 0; r < gs; ++r) w += p.W[(int64_t)(g * gs + r) * p.h_s + h];
    wg[i] = w;
  }
  int64_t row_end = 0;  // blocks before it belong to the row that was found last
  int qb = -1, rows = 0;  // its query block (-1: a row of no sequence) and the rows inside the sequence
  while (x < end) {
    if (tid == 0) s_lo = ~0u, s_hi = 0;
    for (int i = tid; i < p.h_kv * B; i += CS_THR) acc[i] = 0.0f;
    __syncthreads();
    if (n >= row_end) {
      // the row of block n: every thread probes one row, until one is left
      int64_t r = 0, top = p.n_rows;
      while (top - r > 1) {
        const int64_t step = (top - r + CS_THR - 1) / CS_THR;
        const int64_t at = r + (tid + 1) * step;
        const int k = __syncthreads_count(at < top && p.row_ptr[at] <= n);
        r += k * step;
        top = min(top, r + step);
      }
      row_end = p.row_ptr[r + 1];
      const bool good = p.row_ptr[r] <= n && n < row_end;
      // the sequence that holds the row; several may, if they agree on what it holds
      for (int s = tid; s < p.nseq; s += CS_THR) {
        const int L = p.cu[s + 1] - p.cu[s], b = p.base[s];
        const int nq = (int)(((int64_t)L + B - 1) / B);
        if (L <= 0 || L > p.max_len || b < 0 || (int64_t)b + nq > p.n_rows || r < b || r >= (int64_t)b + nq) continue;
        const int q = (int)(r - b);
        const uint32_t what = (uint32_t)q << 8 | (uint32_t)min(B, L - q * B);
        atomicMin(&s_lo, what);
        atomicMax(&s_hi, what);
      }
      __syncthreads();
      qb = -1, rows = 0;
      if (good && s_lo == s_hi) {
        qb = (int)(s_lo >> 8);
        rows = (int)(s_lo & 255u);
      } else if (tid == 0 && (!good || s_lo < s_hi)) {
        atomicOr(p.status, ST_INDEX);
      }
      if (!good) row_end = n + 1;
    }
    int live = rows;
    const int diff = qb - kb;
    if (qb < 0) {
      live = 0;
    } else if (kb < 0 || diff < 0) {
      if (tid == 0) atomicOr(p.status, ST_INDEX);
      live = 0;
    }
    if (n + 1 < nb) kb = p.col_idx[n + 1];
    const bool masked = diff == 0 || live < B;
    // a warp without a head in this block goes on to the next
    const int64_t ahead = (n + 1) * p.h_s + warp;
    if (h_lo + warp >= h_hi && warp < p.h_s && ahead < end) fetch(ahead, 0);
    for (int h0 = h_lo; h0 < h_hi; h0 += CS_HEADS) {
      const int hn = min(CS_HEADS, h_hi - h0);
      for (int h = h0 + warp; h < h0 + hn; h += CS_WARPS) {
        float c[E];
#pragma unroll
        for (int k = 0; k < E; ++k) c[k] = 0.0f;
#pragma unroll 1
        for (int i0 = 0; i0 < NL; i0 += UNR) {
          if (masked) {
#pragma unroll
            for (int i = 0; i < UNR; ++i) {
              const int row = (i0 + i) * RPI + row0;
              // columns of the chunk that the row may see
              const int see = row >= live ? 0 : diff == 0 ? row - chunk * E + 1 : E;
#pragma unroll
              for (int k = 0; k < E; ++k) c[k] += k < see ? element<T>(v[i], k) : 0.0f;
            }
          } else {
#pragma unroll
            for (int i = 0; i < UNR; ++i)
#pragma unroll
              for (int k = 0; k < E; ++k) c[k] += element<T>(v[i], k);
          }
          // on to the rest of the tile, the warp's next head, or its first head of the next block
          if (i0 + UNR < NL) {
            fetch(n * p.h_s + h, i0 + UNR);
          } else {
            const int64_t next = h + CS_WARPS < h_hi ? n * p.h_s + h + CS_WARPS : ahead;
            if (next < end && (h + CS_WARPS < h_hi || warp < p.h_s)) fetch(next, 0);
          }
        }
#pragma unroll
        for (int o = CPR; o < 32; o <<= 1)
#pragma unroll
          for (int k = 0; k < E; ++k) c[k] += __shfl_xor_sync(~0u, c[k], o);
        if (row0 == 0)
#pragma unroll
          for (int k = 0; k < E; ++k) col[(h - h0) * B + chunk * E + k] = c[k];
      }
      __syncthreads();
      for (int i = tid; i < p.h_kv * B; i += CS_THR) {
        const int g = i / B, j = i % B;
        float a = acc[i];
#pragma unroll 4
        for (int h = 0; h < hn; ++h) a = fmaf(wg[(h0 + h) * p.h_kv + g], col[h * B + j], a);
        acc[i] = a;
      }
      __syncthreads();
    }
    float* out = p.part + (n + blockIdx.x) * p.h_kv * B;
    for (int i = tid; i < p.h_kv * B; i += CS_THR) out[i] = acc[i];
    x += h_hi - h_lo;
    ++n;
    h_lo = 0;
    h_hi = (int)min((int64_t)p.h_s, end - x);
  }
}

constexpr int CM_THR = 256;
constexpr int CM_UN = 8;  // parts a thread loads at a time

// entries of the list of a key block's parts: one for every query block, and one more for every
// CTA of k_colsum that starts inside a block
__host__ __device__ inline int merge_list(int nqb_max, int grid) { return nqb_max + grid; }

__global__ void __launch_bounds__(CM_THR) k_colmerge(const __grid_constant__ ColParams p, int B) {
  extern __shared__ uint32_t s_part[];  // rows of the part array, in ascending order
  __shared__ int s_w[CM_THR / 32];
  __shared__ double s_sum[CM_THR][4];
  const int s = blockIdx.x / p.nqb_max, kb = blockIdx.x - s * p.nqb_max;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = p.cu[s + 1] - p.cu[s];
  const int b = p.base[s];
  const int nq = (int)(((int64_t)L + B - 1) / B);
  if (L < 0 || L > p.max_len || b < 0 || (int64_t)b + nq > p.n_rows) {
    if (kb == 0 && tid == 0) atomicOr(p.status, ST_INDEX);
    await_earlier();
    return;
  }
  if (kb >= nq) {
    await_earlier();
    return;
  }
  const int64_t nb = block_count(p, false);
  const int64_t per = tiles_per_cta(nb, p.h_s, p.grid);
  const int room = merge_list(p.nqb_max, p.grid);
  int count = 0;
  for (int q0 = kb; q0 < nq; q0 += CM_THR) {
    const int q = q0 + tid;
    int at = -1;
    if (q < nq) {
      int lo = p.row_ptr[b + q], hi = p.row_ptr[b + q + 1];
      if (lo < 0 || hi < lo || hi > nb) {
        atomicOr(p.status, ST_INDEX);
      } else {
        const int top = hi;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (p.col_idx[mid] < kb) lo = mid + 1; else hi = mid;
        }
        if (lo < top && p.col_idx[lo] == kb) at = lo;
      }
    }
    int64_t c0 = 0;
    int parts = 0;
    if (at >= 0) {
      c0 = (int64_t)at * p.h_s / per;
      parts = (int)(((int64_t)at * p.h_s + p.h_s - 1) / per - c0) + 1;
    }
    int incl = parts;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_w[warp] = incl;
    __syncthreads();
    int to = count + incl - parts;
    for (int w = 0; w < CM_THR / 32; ++w) {
      if (w < warp) to += s_w[w];
      count += s_w[w];
    }
    for (int k = 0; k < parts && to + k < room; ++k) s_part[to + k] = (uint32_t)(at + c0 + k);
    __syncthreads();
  }
  count = min(count, room);  // more only if rows overlap, which is reported above
  await_earlier();
  // a thread takes four columns of the key head's row; h_kv B is a multiple of 32
  const int cols = p.h_kv * B / 4;
  const int ns = cols >= CM_THR ? 1 : CM_THR / cols;  // slices of the list
  const float4* part = reinterpret_cast<const float4*>(p.part);
  for (int i0 = 0; i0 < cols; i0 += CM_THR) {
    const int i = ns > 1 ? tid % cols : i0 + tid, sl = ns > 1 ? tid / cols : 0;
    double a[4] = {0.0, 0.0, 0.0, 0.0};
    if (i < cols && sl < ns)
      for (int k0 = sl; k0 < count; k0 += CM_UN * ns) {
        float4 v[CM_UN];
#pragma unroll
        for (int k = 0; k < CM_UN; ++k)
          v[k] = k0 + k * ns < count ? part[(int64_t)s_part[k0 + k * ns] * cols + i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < CM_UN; ++k) {
          a[0] += v[k].x;
          a[1] += v[k].y;
          a[2] += v[k].z;
          a[3] += v[k].w;
        }
      }
    if (ns > 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s_sum[tid][k] = a[k];
      __syncthreads();
      if (sl == 0)
        for (int m = 1; m < ns; ++m)
#pragma unroll
          for (int k = 0; k < 4; ++k) a[k] += s_sum[m * cols + i][k];
    }
    if (i < cols && sl == 0) {
      const int g = 4 * i / B, j = 4 * i % B;
      float* out = p.score + ((int64_t)s * p.h_kv + g) * p.stride + (int64_t)kb * B + j;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (kb * B + j + k < L) out[k] = (float)a[k];
    }
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
  p.grid = std::min(CS_GRID, CS_CTAS * sms);
  auto smem = [&](int h_s, int h_kv) { return sizeof(float) * ((size_t)h_s * h_kv + (size_t)h_kv * d.B + (size_t)CS_HEADS * d.B); };
  auto launch = [&](auto kernel) {
    constexpr auto K = decltype(kernel)::value;
    // the largest call's limit: one of this call's size would fail a larger call of another thread
    // that has set its own already
    e = allow_smem<K>(dev, (int)smem(MAX_SENDERS, MAX_KEY_HEADS));
    if (e == cudaSuccess) e = launch_early(K, p.grid, CS_THR, smem(d.h_s, d.h_kv), 1, st, p);
  };
  auto launch_for = [&](auto type) {
    using T = decltype(type);
    using std::integral_constant;
    if (d.B == 32) launch(integral_constant<void (*)(ColParams), &k_colsum<T, 32>>{});
    else if (d.B == 64) launch(integral_constant<void (*)(ColParams), &k_colsum<T, 64>>{});
    else launch(integral_constant<void (*)(ColParams), &k_colsum<T, 128>>{});
  };
  if (d.map_dtype == MF_F32) launch_for(float{});
  else launch_for(__nv_bfloat16{});
  if (e != cudaSuccess) return e;
  return launch_early(k_colmerge, (unsigned)((int64_t)p.nseq * p.nqb_max), CM_THR, 4 * (size_t)merge_list(p.nqb_max, p.grid), 1,
                      st, p, d.B);
}

}  // namespace mfi
