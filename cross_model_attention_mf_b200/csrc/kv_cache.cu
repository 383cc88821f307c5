// The paged cache's upkeep: new tokens in (mf_kv_append), rows out by gathered weight
// (mf_kv_evict).  Both move bytes and are bounded by HBM bandwidth, or by launch latency for the
// few rows of a decode step.
//
// Eviction keeps `budget` of a (sequence, key head)'s slots.  With k_j the 32-bit key whose
// unsigned order is the order of preference (protected slots above all, then the score),
// the kept set is the `budget` largest keys, equal keys by slot.  k_evict_select finds the
// smallest kept key by counting: up to three rounds over 11, 11 and 10 bits, each a histogram of
// the slots that still share the prefix, walked from the top; a round whose bin is kept whole is
// the last.  A CTA, or a cluster of them, has one (sequence, key head): the keys stay in its shared
// memory, a cluster's histograms are added over distributed shared memory, so scores and positions
// are read once; outputs that are not the inputs are written from the registers of that read.
// With kb(j) kept slots before slot j, hole j is the (j - kb(j))-th and mover j the
// (kb(j) - kb(new length))-th: one count over the cluster places both.
// What bounds the selection is the number of instructions per slot, next to the latency of a
// round (histogram, barrier, walk), not the bytes.
// Attention does not depend on the order of the slots, so kept rows below the budget stay where
// they are and only the kept rows above it move, into the dropped slots: every source lies at or
// above the budget and every target below, so all moves are independent and k_evict_move makes
// them in any order.
//
// Measured (one B200; copy rate 6469 GB/s): append of 15938 rows of 8 x 128 bf16 for K and V 26.6 us
// (92%), of 64 rows 3.5 us (launch); one slot out of each of 512 rows of 2049 12.7 us (the selection
// 12 of them); 16 prompts of 1024 to 8192 tokens cut to 2048 35.9 us (selection 12, moves 22: 117 MB
// at 82%); 8 rows of 131072 cut to 16384 46 us (selection 23 on 64 SMs, moves 21).
#include <cooperative_groups.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

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

// One 16-byte vector of K and of V per thread and step, four steps in flight; a CTA takes about 16 KB
// of each, whole tokens.
__global__ void __launch_bounds__(AP_THR) k_append(const __grid_constant__ AppendParams p) {
  const int s = blockIdx.x / p.chunks, chunk = blockIdx.x - s * p.chunks;
  await_earlier();
  const int c0 = p.cu[s], n = p.cu[s + 1] - c0;
  const int len = kv_len(p.kv, s, chunk == 0 && threadIdx.x == 0);
  if (n < 0 || n > p.max_new || n > len || c0 < 0 || (int64_t)c0 + n > p.total_new) {
    if (chunk == 0 && threadIdx.x == 0) atomicOr(p.kv.status, ST_INDEX);
    return;
  }
  const int t0 = chunk * p.toks, t1 = min(n, t0 + p.toks);
  if (t0 >= n) return;  // past the sequence's new tokens: max_new may be 2^30, and t1 - t0 far below 0
  const int nv = p.kv.slot_bytes >> 4;
  const int slot0 = len - n;
  const int work = (t1 - t0) * nv;  // at most toks tokens: AP_VECS vectors, or one token's
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
constexpr int BINS = 2048;
constexpr int EV_CLUSTER = 8;     // portable cluster size
constexpr int EV_LOADS = 8;       // slots a thread loads at a time
constexpr int EV_THR = 256;       // threads of a CTA for rows of up to
constexpr int EV_SHORT = 4096;    // slots, and
constexpr int EV_WIDE = 512;      // threads for longer ones
constexpr int EV_SLOTS = 4096;    // slots a CTA of a cluster is left with where SMs would be idle

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
};

// unsigned order = preference: NaN below -inf, then ascending scores, protected slots on top
__device__ __forceinline__ uint32_t evict_key(float score, int pos, int sink, int recent) {
  const uint32_t b = __float_as_uint(score + 0.0f);  // -0 becomes 0
  uint32_t k = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
  if (score != score) k = 0u;
  if (pos < sink || pos >= recent) k = 0xFFFFFFFFu;
  return k;
}

__device__ __forceinline__ uint32_t scan_warp(uint32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += u;
  }
  return x;
}

// the lowest n set bits of m
__device__ __forceinline__ uint32_t lowest_bits(uint32_t m, uint32_t n) {
  if (n >= __popc(m)) return m;
  uint32_t r = 0;
  for (; n && m; --n) {
    r |= m & (0u - m);
    m &= m - 1;
  }
  return r;
}

// Keys in registers and loops unrolled over a thread's slots took 26 us for 512 rows of 2049 slots:
// the code left the instruction cache.  Loops over shared memory with few instructions: 12.6.
// A CTA's slots are one tile of at most 32 THR, whose keys stay in shared memory, or are read
// again, tile by tile, in every pass.  A warp owns up to 32 groups of 32 neighbouring slots of a
// tile; ballots mark a group's keys above the bar and at it, and lane q keeps the marks of group
// q: what is kept, a hole or a mover is then found for 1024 slots at once.
// SOLO: one CTA has the row to itself.
template <int THR, bool SOLO>
__global__ void __launch_bounds__(THR, 1024 / THR) k_evict_select(const __grid_constant__ EvictParams p) {
  constexpr int WARPS = THR / 32, TILE = THR * 32;
  static_assert(BINS == 64 * 32, "two levels of the walk");
  extern __shared__ __align__(16) uint32_t s_key[];
  __shared__ __align__(16) uint32_t s_hist[2][BINS];
  __shared__ __align__(8) uint32_t s_coarse[2][64];
  __shared__ uint32_t s_pick[2][3];           // bin of the smallest kept key, keys to take from it, keys in it
  __shared__ int s_in[2];                     // the row's length, the tokens seen
  __shared__ uint2 s_cnt[WARPS];              // keys above and at the bar, per warp of the tile
  __shared__ __align__(16) uint32_t s_tot[4]; // of the CTA: above, at the bar; and of those, below the new length
  cg::cluster_group cl = cg::this_cluster();
  const int C = SOLO ? 1 : (int)cl.num_blocks(), rank = SOLO ? 0 : (int)cl.block_rank();
  const int job = blockIdx.x / C;
  const int s = job / p.h_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first = job == s * p.h_kv && rank == 0 && tid == 0;
  for (int i = tid; i < 2 * BINS / 4; i += THR) reinterpret_cast<uint4*>(s_hist)[i] = make_uint4(0, 0, 0, 0);
  if (tid < 4) s_tot[tid] = 0;
  if (tid < 6) s_pick[tid / 3][tid % 3] = 0;
  await_earlier();
  allow_later();
  auto sync = [&] {
    if (SOLO) __syncthreads(); else cl.sync();
  };
  int len, seen;
  if (SOLO) {
    seen = p.n_seen ? p.n_seen[s] : 0;
    len = kv_len(p.kv, s, first);
  } else {
    // one thread reads the length for the whole cluster: no CTA may leave while others read its
    // memory, not even if the caller lets the length change meanwhile
    if (rank == 0 && tid == 0) {
      s_in[0] = kv_len(p.kv, s, first);
      s_in[1] = p.n_seen ? p.n_seen[s] : 0;
    }
    cl.sync();
    const int* in0 = cl.map_shared_rank(s_in, 0);
    len = in0[0], seen = in0[1];
  }
  // a bound below -2^31 protects every slot, as -2^31 does
  const int recent = (int)max((int64_t)INT32_MIN, (int64_t)(p.n_seen ? seen : len) - p.window);
  const int left = min(len, p.budget);
  const int64_t row = (int64_t)job * p.stride;
  const float* sc = p.score_in + row;
  const int32_t* po = p.pos_in + row;
  float* so = p.score_out + row;
  int32_t* qo = p.pos_out + row;
  const bool copy_s = so != sc, copy_p = qo != po;
  // slots of this CTA
  const int per = (len + C - 1) / C;
  const int lo = min(len, rank * per), hi = min(len, lo + per);
  if (first) p.ws.len[s] = left;
  if (len <= p.budget) {  // nothing goes: the rows stay, copies follow
    if (rank == 0 && tid == 0) p.ws.count[job] = 0;
    if (copy_s || copy_p)
#pragma unroll 8
      for (int j = lo + tid; j < hi; j += THR) {
        if (copy_s) so[j] = sc[j];
        if (copy_p) qo[j] = po[j];
      }
    if (!SOLO) cl.sync();  // the first CTA's length has been read
    return;
  }
  const bool one = hi - lo <= TILE;
  // Keys of the tile's n slots.  The first pass counts their upper bits, and writes outputs that
  // are not the inputs: slots below the new length as they are (the movers overwrite the holes
  // later), cleared ones above it.
  auto load = [&](int t0, int n, bool begin) {
    for (int i0 = tid; i0 < n; i0 += EV_LOADS * THR) {
      const int rem = n - i0, keep = left - t0 - i0;
      const float* ps = sc + t0 + i0;
      const int32_t* pp = po + t0 + i0;
      float a[EV_LOADS];
      int b[EV_LOADS];
#pragma unroll
      for (int k = 0; k < EV_LOADS; ++k)
        if (k * THR < rem) {
          a[k] = ps[k * THR];
          b[k] = pp[k * THR];
        }
      uint32_t* pk = s_key + i0;
#pragma unroll
      for (int k = 0; k < EV_LOADS; ++k)
        if (k * THR < rem) {
          const uint32_t key = evict_key(a[k], b[k], p.sink, recent);
          pk[k * THR] = key;
          if (begin) atomicAdd(&s_hist[0][key >> 21], 1u);
        }
      if (begin && copy_s) {
        float* out = so + t0 + i0;
#pragma unroll
        for (int k = 0; k < EV_LOADS; ++k)
          if (k * THR < rem) out[k * THR] = k * THR < keep ? a[k] : 0.0f;
      }
      if (begin && copy_p) {
        int32_t* out = qo + t0 + i0;
#pragma unroll
        for (int k = 0; k < EV_LOADS; ++k)
          if (k * THR < rem) out[k * THR] = k * THR < keep ? b[k] : -1;
      }
    }
    // the last vector of keys is read whole: zeros count below every budget
    if (tid < (-n & 3)) s_key[n + tid] = 0;
  };
  __syncthreads();
  for (int t0 = lo; t0 < hi; t0 += TILE) load(t0, min(TILE, hi - t0), true);

  uint32_t prefix = 0, need = (uint32_t)p.budget;
  int shift = 32;  // bits below the prefix
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int top = shift, buf = round & 1;
    shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    uint32_t* hist = s_hist[buf];
    if (round > 0) {
      const uint32_t mask = (1u << (top - shift)) - 1u;
      for (int t0 = lo; t0 < hi; t0 += TILE) {
        const int n = min(TILE, hi - t0);
        if (!one) {
          __syncthreads();
          load(t0, n, false);
          __syncthreads();
        }
#pragma unroll 2
        for (int i = tid; i < (n + 3) >> 2; i += THR) {
          const uint4 v = reinterpret_cast<const uint4*>(s_key)[i];
          if (v.x >> top == prefix) atomicAdd(&hist[(v.x >> shift) & mask], 1u);
          if (v.y >> top == prefix) atomicAdd(&hist[(v.y >> shift) & mask], 1u);
          if (v.z >> top == prefix) atomicAdd(&hist[(v.z >> shift) & mask], 1u);
          if (v.w >> top == prefix) atomicAdd(&hist[(v.w >> shift) & mask], 1u);
        }
      }
    }
    __syncthreads();
    // sums of 32 neighbouring bins
    for (int i = tid; i < BINS / 4; i += THR) {
      const uint4 v = reinterpret_cast<const uint4*>(hist)[i];
      uint32_t sum = v.x + v.y + v.z + v.w;
      sum += __shfl_xor_sync(~0u, sum, 1);
      sum += __shfl_xor_sync(~0u, sum, 2);
      sum += __shfl_xor_sync(~0u, sum, 4);
      if (i % 8 == 0) s_coarse[buf][i / 8] = sum;
    }
    sync();
    // The cluster's histograms are walked from the top: by one warp, 64 sums, then 32 bins
    if (warp == 0) {
      uint2 two = make_uint2(0, 0);  // sums 63 - 2 lane and 62 - 2 lane
#pragma unroll
      for (int r = 0; r < (SOLO ? 1 : EV_CLUSTER); ++r)
        if (r < C) {
          const uint32_t* from = SOLO ? s_coarse[buf] : cl.map_shared_rank(s_coarse[buf], r);
          const uint2 v = *reinterpret_cast<const uint2*>(from + 62 - 2 * lane);
          two.x += v.y, two.y += v.x;
        }
      uint32_t above = scan_warp(two.x + two.y, lane) - two.x - two.y;
      const bool here = above < need && need <= above + two.x + two.y;
      const int from_lane = __ffs(__ballot_sync(~0u, here)) - 1;
      const bool second = need > above + two.x;
      above = __shfl_sync(~0u, second ? above + two.x : above, from_lane);
      const int coarse = __shfl_sync(~0u, 63 - 2 * lane - (second ? 1 : 0), from_lane);
      uint32_t c = 0;  // bin 31 - lane of the 32
#pragma unroll
      for (int r = 0; r < (SOLO ? 1 : EV_CLUSTER); ++r)
        if (r < C) c += (SOLO ? hist : cl.map_shared_rank(hist, r))[32 * coarse + 31 - lane];
      above += scan_warp(c, lane) - c;
      if (above < need && need <= above + c) {
        s_pick[buf][0] = (uint32_t)(32 * coarse + 31 - lane);
        s_pick[buf][1] = need - above;
        s_pick[buf][2] = c;
      }
    } else if (round == 1) {  // the first histogram has been read everywhere: it serves the third round
      for (int i = tid - 32; i < BINS / 4; i += THR - 32) reinterpret_cast<uint4*>(s_hist[0])[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    prefix = (prefix << (top - shift)) | s_pick[buf][0];
    need = s_pick[buf][1];
    if (s_pick[buf][2] == need) break;  // the same in the whole cluster
  }
  // kept: keys whose upper bits are above the prefix, and the first `need` of those that equal it

  uint32_t mg = 0, me = 0;      // marks of this lane's group: above the bar, at it
  uint32_t lm = 0, vm = 0;      // its slots below the new length, its slots
  int g0 = 0, groups = 0;       // the warp's first slot, its groups
  auto marks = [&](int t0, int n) {
    groups = (n + THR - 1) / THR;
    g0 = warp * groups * 32;
    const uint32_t* pk = s_key + g0 + lane;
    const int rem = n - g0 - lane;
    mg = me = 0;
#pragma unroll 4
    for (int q = 0; q < groups; ++q) {
      const uint32_t u = 32 * q < rem ? pk[32 * q] >> shift : 0u;
      const uint32_t g = __ballot_sync(~0u, u > prefix), e = __ballot_sync(~0u, u == prefix);
      if (lane == q) mg = g, me = e;
    }
    auto first_bits = [](int k) { return k >= 32 ? ~0u : k <= 0 ? 0u : (1u << k) - 1u; };
    vm = lane < groups ? first_bits(n - g0 - 32 * lane) : 0u;
    lm = first_bits(left - t0 - g0 - 32 * lane);
    me &= vm;  // slots past the end count as keys of 0
  };
  for (int t0 = lo; t0 < hi; t0 += TILE) {
    const int n = min(TILE, hi - t0);
    if (!one) {
      __syncthreads();
      load(t0, n, false);
    }
    __syncthreads();
    marks(t0, n);
    const uint32_t gt = __reduce_add_sync(~0u, __popc(mg)), eq = __reduce_add_sync(~0u, __popc(me));
    const uint32_t gt_l = __reduce_add_sync(~0u, __popc(mg & lm)), eq_l = __reduce_add_sync(~0u, __popc(me & lm));
    if (lane == 0) {
      s_cnt[warp] = make_uint2(gt, eq);
      atomicAdd(&s_tot[0], gt);
      atomicAdd(&s_tot[1], eq);
      atomicAdd(&s_tot[2], gt_l);
      atomicAdd(&s_tot[3], eq_l);
    }
  }
  sync();
  uint32_t gt_before, eq_before, kept_l;  // before this CTA; kept below the new length
  {
    uint4 t = make_uint4(0, 0, 0, 0);
    if (lane < C) t = *reinterpret_cast<const uint4*>(SOLO ? s_tot : cl.map_shared_rank(s_tot, lane));
    gt_before = __reduce_add_sync(~0u, lane < rank ? t.x : 0u);
    eq_before = __reduce_add_sync(~0u, lane < rank ? t.y : 0u);
    kept_l = __reduce_add_sync(~0u, t.z) + min(need, __reduce_add_sync(~0u, t.w));
  }
  if (!SOLO) cl.barrier_arrive();  // no CTA leaves while another still reads its totals: awaited below
  const int moves = (int)p.ws.moves;
  if (rank == 0 && tid == 0) p.ws.count[job] = min(max(p.budget - (int32_t)kept_l, 0), moves);
  int32_t* dst = p.ws.dst + (int64_t)job * p.ws.moves;
  int32_t* src = p.ws.src + (int64_t)job * p.ws.moves;
  const uint32_t below = (1u << lane) - 1u;
  for (int t0 = lo; t0 < hi; t0 += TILE) {
    const int n = min(TILE, hi - t0);
    if (!one) {
      __syncthreads();
      load(t0, n, false);
      __syncthreads();
      marks(t0, n);
      const uint32_t gt = __reduce_add_sync(~0u, __popc(mg)), eq = __reduce_add_sync(~0u, __popc(me));
      if (lane == 0) s_cnt[warp] = make_uint2(gt, eq);
      __syncthreads();
    }
    const uint2 c = lane < WARPS ? s_cnt[lane] : make_uint2(0, 0);
    // keys above and at the bar before the lane's group
    const uint32_t g = gt_before + __reduce_add_sync(~0u, lane < warp ? c.x : 0u) + scan_warp(__popc(mg), lane) - __popc(mg);
    const uint32_t e = eq_before + __reduce_add_sync(~0u, lane < warp ? c.y : 0u) + scan_warp(__popc(me), lane) - __popc(me);
    gt_before += __reduce_add_sync(~0u, c.x);
    eq_before += __reduce_add_sync(~0u, c.y);
    const uint32_t kept = mg | lowest_bits(me, need > e ? min(need - e, 32u) : 0u);
    const uint32_t kb = g + min(need, e);  // kept before the lane's group
    const uint32_t holes = ~kept & vm & lm, movers = kept & ~lm, gone = ~kept & vm & ~lm;
    const int j0 = t0 + g0;
    const int at_h = j0 + 32 * lane - (int)kb, at_m = max(0, (int)(kb - kept_l));
    const bool clear = !copy_s || !copy_p;  // the first pass did it otherwise
    const uint32_t some = __ballot_sync(~0u, (holes | movers | (clear ? gone : 0u)) != 0);
#pragma unroll 4
    for (int q = some ? __ffs(some) - 1 : 0; q < 32 - __clz(some); ++q) {
      const uint32_t mh = __shfl_sync(~0u, holes, q), mm = __shfl_sync(~0u, movers, q);
      const int ah = __shfl_sync(~0u, at_h, q), am = __shfl_sync(~0u, at_m, q);
      const int j = j0 + 32 * q + lane;
      // (places within the lists, also if scores change between the passes over a row of several tiles)
      const int th = ah + __popc(mh & below), tm = am + __popc(mm & below);
      if ((mh >> lane & 1u) && th >= 0 && th < moves) dst[th] = j;
      if ((mm >> lane & 1u) && tm < moves) src[tm] = j;  // its score and position move with the row
      if (clear && (__shfl_sync(~0u, gone, q) >> lane & 1u)) {
        so[j] = 0.0f;
        qo[j] = -1;
      }
    }
  }
  if (!SOLO) cl.barrier_wait();
}

// ------------------------------------------------------------------ eviction: moves
constexpr int MV_THR = 256;
constexpr int MV_ROWS = 16;                        // rows a warp moves
constexpr int MV_CHUNK = MV_ROWS * (MV_THR / 32);  // moves per CTA

// A warp looks its rows up together (lanes 0..15 the sources, 16..31 the targets), then copies
// them, four loads of K and of V on their way in every lane.  The warps need not wait for one
// another, so that some look up while others copy.
__global__ void __launch_bounds__(MV_THR, 4) k_evict_move(const __grid_constant__ EvictParams p, int chunks) {
  const int job = blockIdx.x / chunks, chunk = blockIdx.x - job * chunks;
  const int s = job / p.h_kv, g = job - s * p.h_kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  await_earlier();
  if (chunk == 0 && g == 0 && threadIdx.x == 0) p.lens_out[s] = p.ws.len[s];
  const int m0 = chunk * MV_CHUNK + warp * MV_ROWS;
  const int rows = min(MV_ROWS, p.ws.count[job] - m0);
  if (rows <= 0) return;
  const int mine = lane & (MV_ROWS - 1);
  int slot = -1;  // of the cache (checked, as the selection's places are)
  int64_t off = -1;
  if (mine < rows) {
    slot = (lane < MV_ROWS ? p.ws.src : p.ws.dst)[(int64_t)job * p.ws.moves + m0 + mine];
    if ((unsigned)slot >= (unsigned)p.kv.top) slot = -1;
    const int64_t at = slot < 0 ? -1 : kv_slot(p.kv, s, slot);
    if (at >= 0) off = at + (int64_t)g * p.kv.row_bytes;
  }
  const int to_slot = __shfl_down_sync(~0u, slot, MV_ROWS);
  if (lane < rows && slot >= 0 && to_slot >= 0) {
    const int64_t row = (int64_t)job * p.stride;
    const float sv = p.score_in[row + slot];
    const int pv = p.pos_in[row + slot];
    p.score_out[row + to_slot] = sv;
    p.pos_out[row + to_slot] = pv;
    p.score_out[row + slot] = 0.0f;
    p.pos_out[row + slot] = -1;
  }
  // nv vectors of 16 bytes to a row; short rows are copied several at a time
  const int nv = p.kv.row_bytes >> 4;
  const int together = nv < 32 ? 32 / nv : 1;
  const int sub = nv < 32 ? lane / nv : 0, col = nv < 32 ? lane - sub * nv : lane;
  for (int c0 = 0; c0 < nv; c0 += 32)
    for (int r0 = 0; r0 < rows; r0 += 4 * together) {
      uint4 k[4], v[4];
      int64_t to[4];
      const int c = (c0 + col) * 16;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + j * together + sub;
        const int64_t from = __shfl_sync(~0u, off, r & (MV_ROWS - 1));
        to[j] = __shfl_sync(~0u, off, MV_ROWS + (r & (MV_ROWS - 1)));
        k[j] = v[j] = make_uint4(0, 0, 0, 0);
        if (r >= rows || sub >= together || c0 + col >= nv) {
          to[j] = -1;
        } else if (from >= 0) {
          k[j] = *reinterpret_cast<const uint4*>(p.kv.K + from + c);
          v[j] = *reinterpret_cast<const uint4*>(p.kv.V + from + c);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (to[j] >= 0) {
          *reinterpret_cast<uint4*>(p.kv.K + to[j] + c) = k[j];
          *reinterpret_cast<uint4*>(p.kv.V + to[j] + c) = v[j];
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
  return launch_early(k_append, (unsigned)((int64_t)p.chunks * d.kv.nseq), AP_THR, 0, 1, st, p);
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
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // CTAs of a row: as few as hold its keys, for a barrier of a cluster takes a microsecond; a row
  // of more than 8192 slots takes more of them, down to EV_SLOTS slots each, while SMs would be
  // idle otherwise.  16 x 8 rows of 16000: alone 18.4 us, four CTAs each 20.5; 4 x 8 of them: 17.8
  // and 12.8; 8 rows of 6000: 11.3 and (two each) 12.1
  const int thr = d.kv.max_len <= EV_SHORT ? EV_THR : EV_WIDE;
  int C = 1;
  while (C < EV_CLUSTER && ((int64_t)C * 32 * thr < d.kv.max_len ||
                            (d.kv.max_len > 2 * EV_SLOTS && (int64_t)C * EV_SLOTS < d.kv.max_len &&
                             2 * (int64_t)C * jobs <= sms))) C *= 2;
  const int keys = (int)std::min<int64_t>(32 * thr, ((int64_t)d.kv.max_len + C - 1) / C);
  const size_t smem = (4 * (size_t)keys + 15) & ~size_t(15);
  auto launch = [&](auto kernel) {
    constexpr auto K = decltype(kernel)::value;
    e = allow_smem<K>(dev, 4 * 32 * EV_WIDE);
    if (e == cudaSuccess) e = launch_early(K, (unsigned)((int64_t)jobs * C), thr, smem, C, st, p);
  };
  using std::integral_constant;
  if (C == 1 && thr == EV_WIDE) launch(integral_constant<void (*)(EvictParams), &k_evict_select<EV_WIDE, true>>{});
  else if (C == 1) launch(integral_constant<void (*)(EvictParams), &k_evict_select<EV_THR, true>>{});
  else launch(integral_constant<void (*)(EvictParams), &k_evict_select<EV_WIDE, false>>{});
  if (e != cudaSuccess) return e;

  const int chunks = (int)std::max<int64_t>(1, (ws.moves + MV_CHUNK - 1) / MV_CHUNK);
  return launch_early(k_evict_move, (unsigned)((int64_t)jobs * chunks), MV_THR, 0, 1, st, p, chunks);
}

}  // namespace mfi
