// The paged cache's upkeep: new tokens in (mf_kv_append), rows out by gathered weight
// (mf_kv_evict).  Both move bytes and are bounded by HBM bandwidth, or by launch latency for the
// few rows of a decode step.
//
// Eviction keeps `budget` of a (sequence, key head)'s slots.  With k_j the 32-bit key whose
// unsigned order is the order of preference (protected slots above all, then the score),
// the kept set is the `budget` largest keys, equal keys by slot.  k_evict_select finds the
// smallest kept key by counting: three rounds over 11, 11 and 10 bits, each a histogram of the
// slots that still share the prefix, walked from the top.  A cluster of CTAs shares one (sequence,
// key head): the keys stay in its shared memory, the histograms are added over distributed shared
// memory, so scores and positions are read once however long the cache.
// Attention does not depend on the order of the slots, so kept rows below the budget stay where
// they are and only the kept rows above it move, into the dropped slots: every source lies at or
// above the budget and every target below, so all moves are independent and k_evict_move makes
// them in any order.
#include <cooperative_groups.h>
#include <stdint.h>

#include <algorithm>

#include "paged_kv.cuh"

namespace cg = cooperative_groups;

namespace mfi {
namespace {

// ------------------------------------------------------------------ append
constexpr int AP_THR = 256;
constexpr int AP_VECS = 4 * AP_THR;  // 16-byte vectors of K (and of V) a CTA copies

struct AppendParams {
  KvView kv;
  const char* K;
  const char* V;
  int64_t new_bytes;   // between the rows of two new tokens
  int64_t total_new;
  const int32_t* cu;
  const int32_t* n_seen;
  float* score;
  int32_t* pos;
  int64_t stride;
  int max_new, h_kv, toks;  // tokens per CTA
  int chunks;
};

__global__ void __launch_bounds__(AP_THR) k_append(const __grid_constant__ AppendParams p) {
  const int s = blockIdx.x / p.chunks, chunk = blockIdx.x - s * p.chunks;
  const int c0 = p.cu[s], n = p.cu[s + 1] - c0;
  const int len = kv_len(p.kv, s, chunk == 0 && threadIdx.x == 0);
  if (n < 0 || n > p.max_new || n > len || c0 < 0 || (int64_t)c0 + n > p.total_new) {
    if (chunk == 0 && threadIdx.x == 0) atomicOr(p.kv.status, ST_INDEX);
    return;
  }
  const int t0 = chunk * p.toks, t1 = min(n, t0 + p.toks);
  const int nv = p.kv.slot_bytes >> 4;
  const int slot0 = len - n;
  const int work = (t1 - t0) * nv;  // <= 0 past the sequence's new tokens
  for (int i0 = threadIdx.x; i0 < work; i0 += 4 * AP_THR) {
    uint4 k[4], v[4];
    int64_t to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * AP_THR;
      to[j] = -1;
      if (i < work) {
        const int t = t0 + i / nv, c = i % nv;
        const int64_t src = (int64_t)(c0 + t) * p.new_bytes + 16 * c;
        k[j] = __ldg(reinterpret_cast<const uint4*>(p.K + src));
        v[j] = __ldg(reinterpret_cast<const uint4*>(p.V + src));
        const int64_t at = kv_slot(p.kv, s, slot0 + t);
        if (at >= 0) to[j] = at + 16 * c;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (to[j] >= 0) {
        *reinterpret_cast<uint4*>(p.kv.K + to[j]) = k[j];
        *reinterpret_cast<uint4*>(p.kv.V + to[j]) = v[j];
      }
  }
  if (!p.score && !p.pos) return;
  const int first = (p.n_seen ? p.n_seen[s] : len) - n;
  const int nt = t1 - t0;
  for (int i = threadIdx.x; i < nt * p.h_kv; i += AP_THR) {
    const int g = i / nt, t = t0 + i - g * nt;
    const int64_t at = ((int64_t)s * p.h_kv + g) * p.stride + slot0 + t;
    if (p.score) p.score[at] = 0.0f;
    if (p.pos) p.pos[at] = first + t;
  }
}

// ------------------------------------------------------------------ eviction: selection
constexpr int EV_THR = 512;
constexpr int EV_WARPS = EV_THR / 32;
constexpr int BINS = 2048;
constexpr int EV_KEYS = 32768;    // keys a CTA keeps in shared memory; later ones are read again
constexpr int EV_CLUSTER = 8;     // portable cluster size
constexpr int EV_SLOTS = 4096;    // slots a CTA takes before the cluster grows

struct EvictParams {
  KvView kv;
  const float* score_in;
  const int32_t* pos_in;
  float* score_out;
  int32_t* pos_out;
  int64_t stride;
  const int32_t* n_seen;
  int budget, sink, window, h_kv;
  int32_t* lens_out;
  KvEvictWs ws;
  int keys;           // capacity of the shared key array
};

// unsigned order = preference: NaN below -inf, then ascending scores, protected slots on top
__device__ __forceinline__ uint32_t evict_key(float score, int pos, int sink, int64_t recent) {
  if (pos < sink || pos >= recent) return 0xFFFFFFFFu;
  if (score != score) return 0u;
  const uint32_t b = __float_as_uint(score == 0.0f ? 0.0f : score);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// exclusive scan of one count per thread over the CTA
__device__ __forceinline__ uint32_t scan_excl(uint32_t a, uint32_t* s_w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = a;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += u;
  }
  if (lane == 31) s_w[warp] = x;
  __syncthreads();
  uint32_t r = x - a;
#pragma unroll
  for (int w = 0; w < EV_WARPS; ++w)
    if (w < warp) r += s_w[w];
  __syncthreads();
  return r;
}

__global__ void __launch_bounds__(EV_THR) k_evict_select(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_hist[BINS];
  __shared__ uint32_t s_a[EV_WARPS], s_b[EV_WARPS];
  __shared__ uint32_t s_pick[2];    // bin of the smallest kept key, keys still to take from it
  __shared__ uint32_t s_count[2];   // this CTA's counts, read by the cluster
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int job = blockIdx.x / C;
  const int s = job / p.h_kv;
  const int tid = threadIdx.x;
  // the move kernel may take its place; it waits for this grid before its first access
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int len = kv_len(p.kv, s, rank == 0 && tid == 0 && job == s * p.h_kv);
  const int left = min(len, p.budget);
  const int64_t row = (int64_t)job * p.stride;
  const float* sc = p.score_in + row;
  const int32_t* po = p.pos_in + row;
  const bool cut = len > p.budget;
  // slots of this CTA
  const int per = (len + C - 1) / C;
  const int lo = min(len, rank * per), hi = min(len, lo + per);
  const int64_t recent = (int64_t)(p.n_seen ? p.n_seen[s] : len) - p.window;
  if (job == s * p.h_kv && rank == 0 && tid == 0) p.ws.len[s] = left;

  if (!cut) {  // nothing goes: the rows stay, copies follow
    if (rank == 0 && tid == 0) p.ws.count[job] = 0;
    for (int j = lo + tid; j < hi; j += EV_THR) {
      if (p.score_out != p.score_in) p.score_out[row + j] = sc[j];
      if (p.pos_out != p.pos_in) p.pos_out[row + j] = po[j];
    }
    return;  // the whole cluster: len is the same for its CTAs
  }

  auto key_of = [&](int j) -> uint32_t {
    const int i = j - lo;
    return i < p.keys ? s_key[i] : evict_key(sc[j], po[j], p.sink, recent);
  };
  uint32_t prefix = 0, need = (uint32_t)p.budget;
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    const uint32_t mask = round == 2 ? 1023u : 2047u;
    const int top = round == 0 ? 32 : shift + (round == 1 ? 11 : 10);  // bits above are the prefix
    for (int b = tid; b < BINS; b += EV_THR) s_hist[b] = 0;
    __syncthreads();
    for (int j = lo + tid; j < hi; j += EV_THR) {
      uint32_t k;
      if (round == 0) {
        k = evict_key(sc[j], po[j], p.sink, recent);
        if (j - lo < p.keys) s_key[j - lo] = k;
      } else {
        k = key_of(j);
      }
      if (round == 0 || k >> top == prefix) atomicAdd(&s_hist[(k >> shift) & mask], 1u);
    }
    cl.sync();
    // every CTA adds up the cluster's histograms and walks them from the top: thread t owns bins
    // 4 t .. 4 t + 3 counted from the highest
    uint32_t c[4];
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = BINS - 1 - (4 * tid + i);
      uint32_t v = 0;
      for (int r = 0; r < C; ++r) v += *cl.map_shared_rank(&s_hist[b], r);
      c[i] = v;
      sum += v;
    }
    uint32_t above = scan_excl(sum, s_a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (above < need && need <= above + c[i]) {
        s_pick[0] = (uint32_t)(BINS - 1 - (4 * tid + i));
        s_pick[1] = need - above;
      }
      above += c[i];
    }
    cl.sync();  // the histograms have been read everywhere, and s_pick is written
    prefix = round == 0 ? s_pick[0] : (prefix << (round == 1 ? 11 : 10)) | s_pick[0];
    need = s_pick[1];
  }
  const uint32_t bar = prefix;  // smallest kept key; `need` of the slots that equal it are kept

  // slots in order, a contiguous run per warp, 32 at a time: the equal keys before a slot decide
  // its fate
  const int lane = tid & 31, warp = tid >> 5;
  const uint32_t below = (1u << lane) - 1u;
  const int run = ((hi - lo + EV_THR - 1) / EV_THR) * 32;
  const int w0 = min(hi, lo + warp * run), w1 = min(hi, w0 + run);
  uint32_t eq = 0;
  for (int j = w0; j < w1; j += 32) eq += __popc(__ballot_sync(~0u, j + lane < w1 && key_of(j + lane) == bar));
  if (lane == 0) s_a[warp] = eq;
  __syncthreads();
  uint32_t eq_before = 0;
  if (tid == 0) s_count[0] = 0;
  for (int w = 0; w < EV_WARPS; ++w) {
    if (w < warp) eq_before += s_a[w];
    if (tid == 0) s_count[0] += s_a[w];
  }
  cl.sync();
  for (int r = 0; r < rank; ++r) eq_before += *cl.map_shared_rank(&s_count[0], r);
  // holes: dropped slots below the new length; movers: kept slots at or above it
  uint32_t e = eq_before, holes = 0, movers = 0;
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t k = j < w1 ? key_of(j) : 0u;
    const uint32_t eqm = __ballot_sync(~0u, j < w1 && k == bar);
    const bool kept = k > bar || (k == bar && e + __popc(eqm & below) < need);
    e += __popc(eqm);
    holes += __popc(__ballot_sync(~0u, j < w1 && !kept && j < left));
    movers += __popc(__ballot_sync(~0u, j < w1 && kept && j >= left));
  }
  if (lane == 0) {
    s_a[warp] = holes;
    s_b[warp] = movers;
  }
  cl.sync();  // the equal keys' counts have been read everywhere
  uint32_t h = 0, mv = 0, th = 0, tm = 0;
  for (int w = 0; w < EV_WARPS; ++w) {
    if (w < warp) {
      h += s_a[w];
      mv += s_b[w];
    }
    th += s_a[w];
    tm += s_b[w];
  }
  if (tid == 0) {
    s_count[0] = th;
    s_count[1] = tm;
  }
  cl.sync();
  uint32_t total = 0;
  for (int r = 0; r < C; ++r) {
    const uint32_t m = *cl.map_shared_rank(&s_count[1], r);
    if (r < rank) {
      h += *cl.map_shared_rank(&s_count[0], r);
      mv += m;
    }
    total += m;
  }
  if (rank == 0 && tid == 0) p.ws.count[job] = (int32_t)total;
  int32_t* dst = p.ws.dst + (int64_t)job * p.ws.moves;
  int32_t* src = p.ws.src + (int64_t)job * p.ws.moves;
  e = eq_before;
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int j = j0 + lane;
    const bool in = j < w1;
    const uint32_t k = in ? key_of(j) : 0u;
    const uint32_t eqm = __ballot_sync(~0u, in && k == bar);
    const bool kept = k > bar || (k == bar && e + __popc(eqm & below) < need);
    e += __popc(eqm);
    const uint32_t hm = __ballot_sync(~0u, in && !kept && j < left);
    const uint32_t mm = __ballot_sync(~0u, in && kept && j >= left);
    if (in) {
      if (j < left) {
        if (!kept) {
          dst[h + __popc(hm & below)] = j;
        } else {
          if (p.score_out != p.score_in) p.score_out[row + j] = sc[j];
          if (p.pos_out != p.pos_in) p.pos_out[row + j] = po[j];
        }
      } else if (kept) {
        src[mv + __popc(mm & below)] = j;  // its score and position move with the row
      } else {
        p.score_out[row + j] = 0.0f;
        p.pos_out[row + j] = -1;
      }
    }
    h += __popc(hm);
    mv += __popc(mm);
  }
  cl.sync();  // no CTA leaves while another still reads its counts
}

// ------------------------------------------------------------------ eviction: moves
constexpr int MV_THR = 256;
constexpr int MV_ROWS = 64;  // moves per CTA

__global__ void __launch_bounds__(MV_THR) k_evict_move(const __grid_constant__ EvictParams p, int chunks) {
  const int job = blockIdx.x / chunks, chunk = blockIdx.x - job * chunks;
  const int s = job / p.h_kv, g = job - s * p.h_kv;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (chunk == 0 && g == 0 && threadIdx.x == 0) p.lens_out[s] = p.ws.len[s];
  const int n = p.ws.count[job];
  const int m0 = chunk * MV_ROWS, m1 = min(n, m0 + MV_ROWS);
  if (m0 >= m1) return;
  __shared__ int64_t s_src[MV_ROWS], s_dst[MV_ROWS];
  for (int i = m0 + threadIdx.x; i < m1; i += MV_THR) {
    const int a = p.ws.src[(int64_t)job * p.ws.moves + i], b = p.ws.dst[(int64_t)job * p.ws.moves + i];
    const int64_t row = (int64_t)job * p.stride;
    const float sv = p.score_in[row + a];
    const int pv = p.pos_in[row + a];
    p.score_out[row + b] = sv;
    p.pos_out[row + b] = pv;
    p.score_out[row + a] = 0.0f;
    p.pos_out[row + a] = -1;
    const int64_t off = (int64_t)g * p.kv.row_bytes;
    const int64_t x = kv_slot(p.kv, s, a), y = kv_slot(p.kv, s, b);
    s_src[i - m0] = x < 0 ? -1 : x + off;
    s_dst[i - m0] = y < 0 ? -1 : y + off;
  }
  __syncthreads();
  const int nv = p.kv.row_bytes >> 4;
  const int work = (m1 - m0) * nv;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int i0 = threadIdx.x; i0 < work; i0 += 4 * MV_THR) {
    uint4 k[4], v[4];
    int64_t to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * MV_THR;
      to[j] = -1;
      if (i < work) {
        const int m = i / nv, c = (i - m * nv) * 16;
        const int64_t a = s_src[m];
        k[j] = a >= 0 ? *reinterpret_cast<const uint4*>(p.kv.K + a + c) : zero;
        v[j] = a >= 0 ? *reinterpret_cast<const uint4*>(p.kv.V + a + c) : zero;
        if (s_dst[m] >= 0) to[j] = s_dst[m] + c;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (to[j] >= 0) {
        *reinterpret_cast<uint4*>(p.kv.K + to[j]) = k[j];
        *reinterpret_cast<uint4*>(p.kv.V + to[j]) = v[j];
      }
  }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

cudaError_t launch_kv_append(const mf_kv_append_desc& d, uint32_t* status, cudaStream_t st) {
  AppendParams p{};
  p.kv = kv_view(d.kv, status);
  const int e = d.kv.dtype == MF_F32 ? 4 : 2;
  p.K = static_cast<const char*>(d.K_new);
  p.V = static_cast<const char*>(d.V_new);
  p.new_bytes = d.new_stride ? d.new_stride * e : p.kv.slot_bytes;
  p.total_new = d.total_new;
  p.cu = d.cu_seqlens_new;
  p.n_seen = d.n_seen;
  p.score = d.score;
  p.pos = d.pos;
  p.stride = d.score_stride;
  p.max_new = d.max_new;
  p.h_kv = d.kv.h_kv;
  p.toks = std::max(1, AP_VECS / (p.kv.slot_bytes / 16));
  p.chunks = std::max(1, (d.max_new + p.toks - 1) / p.toks);
  k_append<<<(unsigned)((int64_t)p.chunks * d.kv.nseq), AP_THR, 0, st>>>(p);
  return cudaGetLastError();
}

size_t kv_evict_ws(const mf_kv_evict_desc& d, KvEvictWs* ws, void* base) {
  // at most `budget` rows can move, and at most the slots past the budget
  const int64_t moves = std::max<int64_t>(0, std::min<int64_t>(d.budget, (int64_t)d.kv.max_len - d.budget));
  const size_t jobs = (size_t)d.kv.nseq * d.kv.h_kv;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    int32_t* q = base ? reinterpret_cast<int32_t*>(static_cast<char*>(base) + at) : nullptr;
    at += up256(bytes);
    return q;
  };
  KvEvictWs w;
  w.count = take(4 * jobs);
  w.len = take(4 * (size_t)d.kv.nseq);
  w.dst = take(4 * jobs * (size_t)moves);
  w.src = take(4 * jobs * (size_t)moves);
  w.moves = moves;
  if (ws) *ws = w;
  return at;
}

cudaError_t launch_kv_evict(const mf_kv_evict_desc& d, const KvEvictWs& ws, uint32_t* status,
                            cudaStream_t st) {
  EvictParams p{};
  p.kv = kv_view(d.kv, status);
  p.score_in = d.score_in;
  p.pos_in = d.pos_in;
  p.score_out = d.score_out;
  p.pos_out = d.pos_out;
  p.stride = d.score_stride;
  p.n_seen = d.n_seen;
  p.budget = d.budget;
  p.sink = d.sink;
  p.window = d.window;
  p.h_kv = d.kv.h_kv;
  p.lens_out = d.seq_lens_out;
  p.ws = ws;
  const int jobs = d.kv.nseq * d.kv.h_kv;
  int C = 1;
  while (C < EV_CLUSTER && (int64_t)C * EV_SLOTS < d.kv.max_len) C *= 2;
  p.keys = (int)std::min<int64_t>(EV_KEYS, ((int64_t)d.kv.max_len + C - 1) / C);
  const size_t smem = 4 * (size_t)p.keys;
  cudaError_t e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       4 * EV_KEYS);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  cfg.gridDim = dim3((unsigned)((int64_t)jobs * C));
  cfg.blockDim = dim3(EV_THR);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_evict_select, p);
  if (e != cudaSuccess) return e;

  const int chunks = (int)std::max<int64_t>(1, (ws.moves + MV_ROWS - 1) / MV_ROWS);
  cudaLaunchConfig_t mv{};
  mv.gridDim = dim3((unsigned)((int64_t)jobs * chunks));
  mv.blockDim = dim3(MV_THR);
  mv.stream = st;
  cudaLaunchAttribute pa[1];
  pa[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pa[0].val.programmaticStreamSerializationAllowed = 1;
  mv.attrs = pa;
  mv.numAttrs = 1;
  return cudaLaunchKernelEx(&mv, k_evict_move, p, chunks);
}

}  // namespace mfi
