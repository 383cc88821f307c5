// Attention of one new token per sequence over the paged key-value cache (mf_paged_decode).
//
//   x_j = c2 q.K[j] (c2 = scale log2 e),  m = max x_j,  l = sum 2^(x_j - m),
//   O = sum 2^(x_j - m) V[j] / l,  lse = (m + log2 l) ln 2,
// with (m, l, O) of two sets of keys joined by 2^(m_a - m), 2^(m_b - m).  K and V are read once:
// 4 len h_r d operations on 2 len h_kv d elements, so HBM bandwidth bounds long calls at any group
// size, and the chain of launch, table lookup, first tiles and join bounds short ones.
//
// Cores.  bf16: S^T = K Q^T and O^T = V^T P^T per warp on 16 keys and 8 (or 16) heads, with the
// warp-wide m16n8k16 product: a tile's 16 x 8 scores stay in registers from one product to the
// next.  The tcgen05 tile (64 rows at least, accumulators in TMEM) would take every score through
// TMEM and back for a tensor pipe that these loads cannot fill.  float32: FMA.
//
// Measured (one B200; copy rate 6469 GB/s; 8 key heads, bf16, groups of 4 and d = 128 where nothing
// else is said): 64 x 8192 tokens, weights carried on, 364 to 374 us, 93 to 90% of that rate;
// 131072 tokens with weights 96 us (88%: 86 the main kernel, the rest join and ends that differ by
// 7 us among CTAs); 16 x 8192 without weights 87 us (95%), groups of 16 102 (81%), d = 64 55 (75%),
// 192 130 (96%), 256 176 to 190 (94 to 87%), 256 with groups of 16 294 (56%); 100 tokens 4.0 us,
// 8.2 under a bound of 8192.  float32, 16 x 4096 tokens: groups of up to 4 91 us (91%), of 8 121 to
// 125 (67%); d = 64 70 (59%) and 97 (43%): instructions of the exchanges and of shared memory.
//
// Split.  A unit is (sequence, key head, block of up to HT query heads of its group).  The units
// of a sequence go in F bundles of P; the bundles of the batch, cut into tiles of TK keys, lie one
// after another on a line that groups of P CTAs share evenly, each CTA with a unit of the bundle:
// whatever the lengths, every CTA gets the same number of tiles, and the CTAs of a group walk
// through the same slots together, whose rows are neighbours in memory.  (With every unit on a line
// of its own, rows of 160 bytes cost 1.5 times their bytes in DRAM traffic.)  A CTA finishes a unit
// that lies wholly inside its stretch; a unit cut by a stretch's end leaves (m, l, O) in the
// workspace, at most two per CTA, and k_decode_join adds the parts in order.  Within a CTA the
// four warps take tiles in turn, each with its own ring of asynchronous copies and its own
// (m, l, O): no CTA barrier inside a unit.
//
// Gathered weights need the final lse, so the main kernel stores x_j (4 bytes per query head and
// key, against 2 d elements per key head) and the join kernel turns them into weights.
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "paged_kv.cuh"

namespace mfi {
namespace {

constexpr int WARPS = 4;
constexpr int NTHR = 32 * WARPS;
constexpr int MAX_GRID = 512;     // CTAs of the main kernel (two partial results each)
constexpr int MIN_TILES = WARPS;  // tiles a CTA takes at least: one per warp
constexpr int ALIGN = WARPS;      // ALIGN, 2 ALIGN or 4 ALIGN tiles to a CTA where units have their own
constexpr int MAX_SEQS = 4096;    // as the entry point checks
constexpr int JOIN_THR = 256;
constexpr int JOIN_KEYS = 1024;   // keys whose weights a CTA of the join kernel adds up at a time
constexpr int JOIN_CTAS = 4;      // its CTAs on an SM
constexpr int MAX_JOINERS = 2048; // CTAs of the join kernel that add up parts
constexpr float LN2 = 0.693147180559945309f;

struct DecodeParams {
  KvView kv;
  const char* Q;
  int64_t q_bytes;     // between the rows of two sequences
  int h_r, h_kv, G, GP, hb, U, d;
  float c2;
  char* O;
  int o_f32;
  float* lse;          // or null
  float* S;            // [nseq][h_kv][max_len][GP] x_j, or null
  const float* score_in;
  float* score_out;    // or null
  int64_t score_stride;
  int32_t* pre;        // [nseq + 1] tiles before each sequence
  int64_t* per;        // tiles of a CTA
  float* lse2;         // [nseq][h_r] of the units finished by one CTA
  float* part_O;       // [2 grid][HT][d]
  float2* part_ml;     // [2 grid][HT]
  int P, F, groups;    // units of a bundle, bundles of a sequence, groups of CTAs
  int groups_each;     // groups / F
  Divider by_P, by_groups;
  int whole;           // every unit is finished by one CTA
  int own_scores;      // and its group has no other unit: the CTA adds up the weights too
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes to shared memory, zeros when bytes == 0
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy) : "memory");
}
// Keys and values are read once and leave L2 first: 16 ragged sequences 57.1 -> 55.2 us.  With
// gathered weights they do not: 64 x 8192 tokens took 380 us so and 369 otherwise.
__device__ __forceinline__ uint64_t cache_policy(bool scores) {
  uint64_t first, normal;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
  return scores ? normal : first;
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8x8 transpose of 16-bit values across the warp
__device__ __forceinline__ uint32_t mov_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// one warp's share of a unit
struct Unit {
  int s, hk, h0, nh, len;  // sequence, key head, first query head, heads, sequence length
  int t0, t1;              // tiles [t0, t1) of the unit belong to this CTA
};

// What the two cores (bf16 on the tensor cores, float32 on the FMA pipes) share: TK keys per
// tile, HT query heads per unit, DP the padded head dim, STAGES tiles in a warp's ring.
// run() leaves the warp's m, l in sm / sl [HT] and its O in buf [HT][DP + PAD].

template <int DP_, int NT>
struct CoreBf16 {
  static constexpr int DP = DP_, TK = 16, HT = 8 * NT, ESZ = 2;
  static constexpr int CPR = DP / 8;                 // 16-byte chunks per row
  static constexpr int HALF = TK * DP * ESZ;         // K rows, then V rows
  static constexpr int TILE = 2 * HALF;
  static constexpr int STAGES = DP == 64 ? 6 : DP == 128 ? 3 : DP == 192 ? 2 : 3;
  // eight rows' chunks of one column fall on different banks
  __device__ static uint32_t place(int row, int c) { return (row * CPR + (c ^ (row & 7))) * 16; }
  static constexpr int CTAS = DP == 256 ? 1 : 2;
  static constexpr int LDB = DP + 4;                 // conflict-free writes of the fragments
  static_assert(HT * LDB * 4 <= STAGES * TILE, "O fits the warp's ring");

  __device__ static void run(const DecodeParams& p, const Unit& u, uint8_t* ring, float* sm, float* sl, int warp,
                             int lane) {
    const KvView& kv = p.kv;
    const int g = lane >> 2, t = lane & 3;
    const int nch = p.d >> 3;
    const int first = u.t0 + warp;
    const int n_my = first < u.t1 ? (u.t1 - first + WARPS - 1) / WARPS : 0;
    const uint32_t sring = smem_u32(ring);
    const int64_t hoff = (int64_t)u.hk * kv.row_bytes;
    const uint64_t policy = cache_policy(p.S != nullptr);
    // byte offset of key row `lane` (< 16) of the k-th tile, -1 past the end
    auto key_of = [&](int k) { return (first + k * WARPS) * TK + (lane & 15); };
    auto held = [&](int k) { return k < n_my && key_of(k) < u.len; };
    auto rows_of = [&](int k) -> int64_t { return held(k) ? kv_slot(kv, u.s, key_of(k)) : -1; };
    auto issue = [&](int stage, int64_t off) {
      const uint32_t base = sring + stage * TILE;
#pragma unroll
      for (int i = 0; i < CPR / 2; ++i) {
        const int idx = i * 32 + lane;
        const int row = idx / CPR, c = idx % CPR;
        const int64_t ro = __shfl_sync(~0u, off, row);
        const bool ok = ro >= 0 && c < nch;
        const int64_t a = ok ? ro + hoff + c * 16 : 0;
        const uint32_t dst = base + place(row, c);
        cp16(dst, kv.K + a, ok ? 16u : 0u, policy);
        cp16(dst + HALF, kv.V + a, ok ? 16u : 0u, policy);
      }
    };
    // the first tiles' pages are looked up together
    KvPlace at[STAGES];
    int id[STAGES];
#pragma unroll
    for (int k = 0; k < STAGES; ++k) {
      at[k] = kv_place(kv, held(k) ? key_of(k) : 0);
      id[k] = held(k) ? kv_page(kv, u.s, at[k]) : 0;
    }
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) {
      if (k < n_my) issue(k, held(k) ? kv_offset(kv, id[k], at[k]) : -1);
      cp_commit();
    }
    int64_t next = held(STAGES - 1) ? kv_offset(kv, id[STAGES - 1], at[STAGES - 1]) : -1;
    // Q^T fragments: head g (+ 8 per head tile), dims 16 k + 2 t (+ 8)
    uint32_t q[DP / 16][NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = g + 8 * n;
      const char* qr = p.Q + (int64_t)u.s * p.q_bytes + (int64_t)(u.h0 + h) * p.d * 2;
#pragma unroll
      for (int k = 0; k < DP / 16; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = 16 * k + 2 * t + 8 * j;
          q[k][n][j] = h < u.nh && c < p.d ? *reinterpret_cast<const uint32_t*>(qr + 2 * c) : 0u;
        }
    }
    float o[DP / 16][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < DP / 16; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[k][n][j] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }
    int stage = 0, fill = STAGES - 1;
    float* S = p.S ? p.S + ((int64_t)u.s * p.h_kv + u.hk) * kv.max_len * p.GP : nullptr;
    const int hg = u.h0 - u.hk * p.G;  // first head within the group
    for (int k = 0; k < n_my; ++k) {
      cp_wait<STAGES - 2>();
      __syncwarp();
      if (k + STAGES - 1 < n_my) issue(fill, next);
      cp_commit();
      next = rows_of(k + STAGES);
      const uint32_t kb = sring + stage * TILE, vb = kb + HALF;
      if (++stage == STAGES) stage = 0;
      if (++fill == STAGES) fill = 0;

      // S^T[key][head]: rows g and g + 8, heads 2t, 2t + 1; two chains of accumulators
      float sc[2][NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[0][n][j] = sc[1][n][j] = 0.0f;
      {
        const int row = lane & 15, hi = lane >> 4;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
          uint32_t a[4];
          ldm4(a, kb + place(row, 2 * ks + hi));
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(sc[ks & 1][n], a, q[ks][n][0], q[ks][n][1]);
        }
      }
      const int key = (first + k * WARPS) * TK + g;
      const bool in0 = key < u.len, in1 = key + 8 < u.len;
      uint32_t pw[NT][3][2];
      float al[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = (sc[0][n][j] + sc[1][n][j]) * p.c2;
        if (!in0) x[0] = x[1] = -INFINITY;
        if (!in1) x[2] = x[3] = -INFINITY;
        if (S) {
          const int h = 8 * n + 2 * t;
          if (h < u.nh) {  // GP is even: the pair stays inside the key's row
            if (in0) *reinterpret_cast<float2*>(S + (int64_t)key * p.GP + hg + h) = make_float2(x[0], x[1]);
            if (in1) *reinterpret_cast<float2*>(S + (int64_t)(key + 8) * p.GP + hg + h) = make_float2(x[2], x[3]);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mx = fmaxf(x[j], x[j + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
          const float mn = fmaxf(m[n][j], mx);
          const float mu = mn == -INFINITY ? 0.0f : mn;
          al[n][j] = ex2(m[n][j] - mu);
          m[n][j] = mn;
          x[j] = ex2(x[j] - mu);
          x[j + 2] = ex2(x[j + 2] - mu);
          l[n][j] = l[n][j] * al[n][j] + (x[j] + x[j + 2]);
        }
        // Weights transposed into the B operand (head g, keys 2t, 2t + 1 (+ 8)), each as the sum of
        // three bf16: 8 bits of its 24 in each, so that the product takes the float32 weight as it is.
        // (Two terms left float32 outputs up to 6.5e-6 off.  The third costs 1% where HBM is the
        // bound, 64 x 8192 tokens with weights 363 -> 366 us, and 15% at 16 heads of 256: 254 -> 294.)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float a = x[2 * j], b = x[2 * j + 1];
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const uint32_t w = pack_bf16(a, b);
            a -= __uint_as_float(w << 16);
            b -= __uint_as_float(w & 0xFFFF0000u);
            pw[n][i][j] = mov_trans(w);
          }
        }
      }
      // O^T[dim][head] = O^T al + V^T P^T.  A tile's product has accumulators of its own, and the sum
      // over the tiles is made here, rounded to nearest: the tensor cores cut their sums off towards
      // zero, and in one chain of them 8192 keys put O 4.9e-6 off, 131072 2.8e-6 (2-norm; so 4e-7 and
      // 5e-7).  It costs nothing where HBM is the bound; 16 x 8192 tokens: 4 heads of 256 170 -> 176
      // us, 16 of 128 94 -> 102.  Several products at a time, since three in a row on the same
      // accumulators wait for one another (one at a time: 198 and 104).
      {
        constexpr int NI = NT == 1 ? 4 : 2;
        const int row = (lane & 7) + 8 * (lane >> 4), hi = (lane >> 3) & 1;
#pragma unroll
        for (int i0 = 0; i0 < DP / 16; i0 += NI) {
          uint32_t a[NI][4];
          float c[NI][NT][4];
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            ldm4t(a[i], vb + place(row, 2 * (i0 + i) + hi));
#pragma unroll
            for (int n = 0; n < NT; ++n) c[i][n][0] = c[i][n][1] = c[i][n][2] = c[i][n][3] = 0.0f;
          }
#pragma unroll
          for (int j = 2; j >= 0; --j)  // the small terms first
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816(c[i][n], a[i], pw[n][j][0], pw[n][j][1]);
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[i0 + i][n][j] = fmaf(o[i0 + i][n][j], al[n][j & 1], c[i][n][j]);
        }
      }
    }
    cp_wait<0>();
    __syncwarp();
    float* buf = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v = l[n][j];
        v += __shfl_xor_sync(~0u, v, 4);
        v += __shfl_xor_sync(~0u, v, 8);
        v += __shfl_xor_sync(~0u, v, 16);
        if (g == 0) {
          sm[8 * n + 2 * t + j] = m[n][j];
          sl[8 * n + 2 * t + j] = v;
        }
      }
#pragma unroll
      for (int i = 0; i < DP / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          buf[(8 * n + 2 * t + (j & 1)) * LDB + 16 * i + g + 8 * (j >> 1)] = o[i][n][j];
    }
  }
};

// A lane owns the same dims of Q, K, V and O (DIMS at a time), so that rows are read as they lie
// and Q stays in registers; a lane's share of 4 heads x 8 keys is added up over the warp by
// exchanges that halve the number of values, until lane (head r = lane / 8, key = lane % 8) holds
// one score.  Reading Q from shared memory for every tile took three times as long.
template <int DP_>
struct CoreF32 {
  static constexpr int DP = DP_, TK = 8, HT = 8, ESZ = 4;
  static constexpr int CPR = DP / 4;
  static constexpr int TILE = 2 * TK * DP * ESZ;
  static constexpr int STAGES = DP == 64 ? 6 : DP == 128 ? 3 : DP == 192 ? 2 : 3;
  static constexpr int CTAS = DP == 256 ? 1 : 2;
  static constexpr int LDB = DP;
  static constexpr int DIMS = DP == 64 ? 2 : 4;      // neighbouring dims of a lane
  static constexpr int NV = (DP / DIMS + 31) / 32;   // such groups of dims per lane
  static_assert(HT * LDB * 4 <= STAGES * TILE, "O fits the warp's ring");

  struct Vec {
    float v[DIMS];
  };
  __device__ static bool in_row(int lane, int i) { return DIMS * (lane + 32 * i) < DP; }
  __device__ static Vec load(const float* row, int lane, int i) {
    Vec r;
    if (!in_row(lane, i)) {
#pragma unroll
      for (int c = 0; c < DIMS; ++c) r.v[c] = 0.0f;
    } else if (DIMS == 4) {
      const float4 t = reinterpret_cast<const float4*>(row)[lane + 32 * i];
      r.v[0] = t.x, r.v[1] = t.y, r.v[DIMS - 2] = t.z, r.v[DIMS - 1] = t.w;
    } else {
      const float2 t = reinterpret_cast<const float2*>(row)[lane + 32 * i];
      r.v[0] = t.x, r.v[1] = t.y;
    }
    return r;
  }

  __device__ static void run(const DecodeParams& p, const Unit& u, uint8_t* ring, float* sm, float* sl, int warp,
                             int lane) {
    const KvView& kv = p.kv;
    const int nch = p.d >> 2;
    const int first = u.t0 + warp;
    const int n_my = first < u.t1 ? (u.t1 - first + WARPS - 1) / WARPS : 0;
    const uint32_t sring = smem_u32(ring);
    const int64_t hoff = (int64_t)u.hk * kv.row_bytes;
    const uint64_t policy = cache_policy(p.S != nullptr);
    auto key_of = [&](int k) { return (first + k * WARPS) * TK + (lane & 7); };
    auto held = [&](int k) { return k < n_my && key_of(k) < u.len; };
    auto rows_of = [&](int k) -> int64_t { return held(k) ? kv_slot(kv, u.s, key_of(k)) : -1; };
    auto issue = [&](int stage, int64_t off) {
      const uint32_t base = sring + stage * TILE;
#pragma unroll
      for (int i = 0; i < CPR / 4; ++i) {
        const int idx = i * 32 + lane;
        const int row = idx / CPR, c = idx % CPR;
        const int64_t ro = __shfl_sync(~0u, off, row);
        const bool ok = ro >= 0 && c < nch;
        const int64_t a = ok ? ro + hoff + c * 16 : 0;
        const uint32_t dst = base + idx * 16;
        cp16(dst, kv.K + a, ok ? 16u : 0u, policy);
        cp16(dst + TK * DP * ESZ, kv.V + a, ok ? 16u : 0u, policy);
      }
    };
    // the first tiles' pages are looked up together
    KvPlace at[STAGES];
    int id[STAGES];
#pragma unroll
    for (int k = 0; k < STAGES; ++k) {
      at[k] = kv_place(kv, held(k) ? key_of(k) : 0);
      id[k] = held(k) ? kv_page(kv, u.s, at[k]) : 0;
    }
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) {
      if (k < n_my) issue(k, held(k) ? kv_offset(kv, id[k], at[k]) : -1);
      cp_commit();
    }
    int64_t next = held(STAGES - 1) ? kv_offset(kv, id[STAGES - 1], at[STAGES - 1]) : -1;
    Vec q[HT][NV], o[HT][NV];
#pragma unroll
    for (int h = 0; h < HT; ++h)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < DIMS; ++c) {
          const int dim = DIMS * (lane + 32 * i) + c;
          o[h][i].v[c] = 0.0f;
          q[h][i].v[c] = h < u.nh && dim < p.d
              ? reinterpret_cast<const float*>(p.Q + (int64_t)u.s * p.q_bytes)[(int64_t)(u.h0 + h) * p.d + dim] : 0.0f;
        }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // of head 4 b + r; l over the lane's keys
    int stage = 0, fill = STAGES - 1;
    float* S = p.S ? p.S + ((int64_t)u.s * p.h_kv + u.hk) * kv.max_len * p.GP : nullptr;
    const int hg = u.h0 - u.hk * p.G;
    const int kl = lane & 7, r = lane >> 3;
    for (int k = 0; k < n_my; ++k) {
      cp_wait<STAGES - 2>();
      __syncwarp();
      if (k + STAGES - 1 < n_my) issue(fill, next);
      cp_commit();
      next = rows_of(k + STAGES);
      const float* Kt = reinterpret_cast<const float*>(ring + stage * TILE);
      const float* Vt = Kt + TK * DP;
      if (++stage == STAGES) stage = 0;
      if (++fill == STAGES) fill = 0;
      const int key = (first + k * WARPS) * TK + kl;
      const bool in = key < u.len;
      float w[2] = {0.0f, 0.0f}, al[2] = {1.0f, 1.0f};
      bool moved = false;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (4 * b >= u.nh) break;  // the same in the whole warp
        float x[4][8];
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
          for (int j = 0; j < 8; ++j) x[h][j] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const Vec t = load(Kt + j * DP, lane, i);
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
              for (int c = 0; c < DIMS; ++c) x[h][j] = fmaf(t.v[c], q[4 * b + h][i].v[c], x[h][j]);
          }
        // keys over lane bits 2, 1, 0
#pragma unroll
        for (int n = 4; n; n >>= 1)
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int j = 0; j < n; ++j) {
              const bool up = lane & n;
              const float give = up ? x[h][j] : x[h][j + n], keep = up ? x[h][j + n] : x[h][j];
              x[h][j] = keep + __shfl_xor_sync(~0u, give, n);
            }
        // heads over lane bits 4, 3
#pragma unroll
        for (int n = 2; n; n >>= 1)
#pragma unroll
          for (int h = 0; h < n; ++h) {
            const bool up = lane & (8 * n);
            const float give = up ? x[h][0] : x[h + n][0], keep = up ? x[h + n][0] : x[h][0];
            x[h][0] = keep + __shfl_xor_sync(~0u, give, 8 * n);
          }
        const float v = in ? x[0][0] * p.c2 : -INFINITY;
        if (S && in && 4 * b + r < u.nh) S[(int64_t)key * p.GP + hg + 4 * b + r] = v;
        float mx = v;
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
        const float mn = fmaxf(m[b], mx);
        const float mu = mn == -INFINITY ? 0.0f : mn;
        al[b] = ex2(m[b] - mu);
        moved |= mn != m[b];
        m[b] = mn;
        w[b] = ex2(v - mu);
        l[b] = l[b] * al[b] + w[b];
      }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          const float f = __shfl_sync(~0u, al[h >> 2], 8 * (h & 3));
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int c = 0; c < DIMS; ++c) o[h][i].v[c] *= f;
        }
      }
#pragma unroll
      for (int j = 0; j < TK; ++j) {
        Vec t[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) t[i] = load(Vt + j * DP, lane, i);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (4 * b >= u.nh) break;
#pragma unroll
          for (int h = 4 * b; h < 4 * b + 4; ++h) {
            const float f = __shfl_sync(~0u, w[b], 8 * (h & 3) + j);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
              for (int c = 0; c < DIMS; ++c) o[h][i].v[c] = fmaf(f, t[i].v[c], o[h][i].v[c]);
          }
        }
      }
    }
    cp_wait<0>();
    __syncwarp();
    float* buf = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float v = l[b];
      v += __shfl_xor_sync(~0u, v, 1);
      v += __shfl_xor_sync(~0u, v, 2);
      v += __shfl_xor_sync(~0u, v, 4);
      if (kl == 0) {
        sm[4 * b + r] = m[b];
        sl[4 * b + r] = v;
      }
    }
#pragma unroll
    for (int h = 0; h < HT; ++h)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in_row(lane, i))
#pragma unroll
          for (int c = 0; c < DIMS; ++c) buf[h * LDB + DIMS * (lane + 32 * i) + c] = o[h][i].v[c];
  }
};

__device__ __forceinline__ int tiles_of(int len, int tk) { return max(1, (len + tk - 1) / tk); }

// Tiles before each sequence on the line of one bundle (`pre`, shared memory), and the tiles of a
// CTA, which are returned.  A sequence of length 0 takes one (empty) tile, so that its outputs
// are written like any other's.  If every unit can have CTAs of its own, ALIGN << k tiles each, its
// stretch of the line is rounded up to them: no CTA then starts over with a second unit, which
// takes 2 us of the 11 that a small call lasts.
__device__ inline int64_t scan_tiles(const DecodeParams& p, int tk, int32_t* pre, bool report) {
  __shared__ int s_w[WARPS];
  __shared__ int s_n[3];
  const KvView& kv = p.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < 3) s_n[threadIdx.x] = 0;
  __syncthreads();
  int c[3] = {0, 0, 0};
  for (int s = threadIdx.x; s < kv.nseq; s += NTHR) {
    const int n = tiles_of(kv_len(kv, s, report), tk);
    pre[s] = n;
#pragma unroll
    for (int k = 0; k < 3; ++k) c[k] += min((n + (ALIGN << k) - 1) / (ALIGN << k), MAX_GRID + 1);
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    c[k] = __reduce_add_sync(~0u, c[k]);
    if (lane == 0) atomicAdd(&s_n[k], c[k]);
  }
  __syncthreads();
  int align = 0;
#pragma unroll
  for (int k = 2; k >= 0; --k)
    if (s_n[k] <= p.groups_each) align = ALIGN << k;
  int base = 0;
  for (int s0 = 0; s0 < kv.nseq; s0 += NTHR) {
    const int s = s0 + threadIdx.x;
    int n = s < kv.nseq ? pre[s] : 0;
    if (align) n = (n + align - 1) & -align;  // a power of two
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_w[warp] = x;
    __syncthreads();
    int add = base, tot = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) add += s_w[w];
      tot += s_w[w];
    }
    if (s < kv.nseq) pre[s] = add + x - n;
    base += tot;
    __syncthreads();
  }
  if (threadIdx.x == 0) pre[kv.nseq] = base;
  __syncthreads();
  if (align) return align;
  const int64_t up = (int64_t)base * p.F + p.groups - 1;
  return max((int64_t)MIN_TILES, up >> 31 == 0 ? p.by_groups.of((int)up) : up / p.groups);
}

// sum of 2^(x - lse2) over the first n of V heads (the others are padding); an empty row, of x = -inf
// and any lse2, adds 0
template <int V>
__device__ __forceinline__ float weights(const float (&x)[V], const float* lse2, int n) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n) sum += ex2(x[i] - lse2[i]);
  return sum;
}
template <int V> __device__ __forceinline__ void load_x(const float* x, float (&v)[V]) {
  if (V == 4) {
    const float4 t = __ldcs(reinterpret_cast<const float4*>(x));
    v[0] = t.x, v[1] = t.y, v[V - 2] = t.z, v[V - 1] = t.w;
  } else {
    const float2 t = __ldcs(reinterpret_cast<const float2*>(x));
    v[0] = t.x, v[1] = t.y;
  }
}

// Keys j0 .. j1 of one row: the group's weights, V heads to a load.  A thread's first loads go out
// before `ready` has found lse2 (shared memory).
template <int V, int THR, class Ready>
__device__ __forceinline__ void add_weights(const DecodeParams& p, int64_t row, int j0, int j1, const float* lse2,
                                            Ready ready) {
  constexpr int UN = 4;
  for (int j = j0 + threadIdx.x; j < j1 || j - j0 < THR; j += UN * THR) {
    const float* S = p.S + (row * p.kv.max_len + j) * p.GP;
    const float* in = p.score_in ? p.score_in + row * p.score_stride + j : nullptr;
    float* out = p.score_out + row * p.score_stride + j;
    const int rem = j1 - j;
    float old[UN], x[UN][V];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      old[i] = 0.0f;
      if (i * THR < rem) {
        if (in) old[i] = in[i * THR];
        load_x<V>(S + i * THR * p.GP, x[i]);
      }
    }
    if (j - j0 < THR) ready();
    float sum[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) sum[i] = i * THR < rem ? weights<V>(x[i], lse2, p.G) : 0.0f;
    for (int h = V; h < p.GP; h += V) {
#pragma unroll
      for (int i = 0; i < UN; ++i)
        if (i * THR < rem) load_x<V>(S + i * THR * p.GP + h, x[i]);
#pragma unroll
      for (int i = 0; i < UN; ++i)
        if (i * THR < rem) sum[i] += weights<V>(x[i], lse2 + h, p.G - h);
    }
#pragma unroll
    for (int i = 0; i < UN; ++i)
      if (i * THR < rem) out[i * THR] = old[i] + sum[i];
  }
}

template <class Core>
__global__ void __launch_bounds__(NTHR, Core::CTAS) k_decode(const __grid_constant__ DecodeParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[WARPS][Core::HT], s_l[WARPS][Core::HT], s_f[WARPS][Core::HT], s_lse2[Core::HT];
  constexpr int RING = Core::STAGES * Core::TILE;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * RING;
  int32_t* pre = reinterpret_cast<int32_t*>(smem + WARPS * RING);

  await_earlier();
  if (!p.whole || (p.S && !p.own_scores)) allow_later();  // k_decode_join follows
  int64_t x, end;
  int s = 0, member = 0;
  if (p.whole) {
    // one unit per CTA: nothing to share out
    x = blockIdx.x;
    end = x + 1;
    s = (int)(x / p.U);
  } else {
    const int64_t per = scan_tiles(p, Core::TK, pre, blockIdx.x == 0);
    if (blockIdx.x == 0) {
      for (int i = threadIdx.x; i <= p.kv.nseq; i += NTHR) p.pre[i] = pre[i];
      if (threadIdx.x == 0) *p.per = per;
    }
    const int64_t total = (int64_t)pre[p.kv.nseq] * p.F;
    const int group = p.by_P.of(blockIdx.x);
    member = blockIdx.x - group * p.P;
    x = per * group;
    end = min(total, x + per);
    int hi = p.kv.nseq;  // the sequence whose stretch holds x
    while (hi - s > 1) {
      const int mid = (s + hi) >> 1;
      if ((int64_t)pre[mid] * p.F <= x) s = mid; else hi = mid;
    }
  }
  while (x < end) {
    Unit u;
    bool begins, whole;
    int ui;
    u.s = s;
    u.len = kv_len(p.kv, s, p.whole);
    if (p.whole) {
      ui = (int)(x - (int64_t)s * p.U);
      u.t0 = 0;
      u.t1 = tiles_of(u.len, Core::TK);
      begins = whole = true;
      ++x;
    } else {
      const int nt = pre[s + 1] - pre[s];
      const int64_t rel = x - (int64_t)pre[s] * p.F;
      const int bundle = p.F == 1 ? 0 : (int)div_floor(rel, nt);
      ui = bundle * p.P + member;
      u.t0 = (int)(rel - (int64_t)bundle * nt);
      const int to = (int)min((int64_t)nt, u.t0 + (end - x));
      u.t1 = min(to, tiles_of(u.len, Core::TK));  // past it the stretch is rounded up
      begins = u.t0 == 0;
      whole = begins && to == nt;
      x += to - u.t0;
      if (bundle == p.F - 1 && to == nt) ++s;
    }
    u.hk = p.hb == 1 ? ui : ui / p.hb;
    const int in_group = (ui - u.hk * p.hb) * Core::HT;
    u.h0 = u.hk * p.G + in_group;
    u.nh = min(Core::HT, p.G - in_group);

    Core::run(p, u, ring, s_m[warp], s_l[warp], warp, lane);
    __syncthreads();
    // join the warps: their shares first, a head to a thread
    const int64_t slot = 2 * (int64_t)blockIdx.x + (begins ? 1 : 0);
    if (threadIdx.x < u.nh) {
      const int h = threadIdx.x;
      float M = s_m[0][h];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) M = fmaxf(M, s_m[w][h]);
      const float mu = M == -INFINITY ? 0.0f : M;
      float f[WARPS], L = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        f[w] = ex2(s_m[w][h] - mu);
        L = fmaf(f[w], s_l[w][h], L);
      }
      const float inv = !whole ? 1.0f : L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) s_f[w][h] = f[w] * inv;
      if (whole) {
        const float v = L == 0.0f ? -INFINITY : mu + log2f(L);
        const int64_t r = (int64_t)u.s * p.h_r + u.h0 + h;
        p.lse2[r] = v;
        if (p.lse) p.lse[r] = v * LN2;
        s_lse2[h] = v == -INFINITY ? 0.0f : v;
      } else {
        p.part_ml[slot * Core::HT + h] = make_float2(M, L);
      }
    }
    __syncthreads();
    // a finished unit writes O, a cut one its part
    const int columns = p.d >> 2;
    for (int i = threadIdx.x; i < u.nh * columns; i += NTHR) {
      const int h = i / columns, c = 4 * (i - h * columns);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = s_f[w][h];
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * RING) + h * Core::LDB + c);
        a.x = fmaf(f, v.x, a.x);
        a.y = fmaf(f, v.y, a.y);
        a.z = fmaf(f, v.z, a.z);
        a.w = fmaf(f, v.w, a.w);
      }
      const int64_t at = ((int64_t)u.s * p.h_r + u.h0 + h) * p.d + c;
      if (!whole) *reinterpret_cast<float4*>(p.part_O + (slot * Core::HT + h) * p.d + c) = a;
      else if (p.o_f32) *reinterpret_cast<float4*>(p.O + 4 * at) = a;
      else *reinterpret_cast<uint2*>(p.O + 2 * at) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
    }
    __syncthreads();
  }
  if (p.own_scores) {  // the CTA had a whole group: it turns the x_j that it stored into weights itself
    const int row = blockIdx.x, len = kv_len(p.kv, row / p.h_kv, false);  // one unit to a key head
    auto ready = [] {};
    if (p.GP % 4 == 0) add_weights<4, NTHR>(p, row, 0, len, s_lse2, ready);
    else add_weights<2, NTHR>(p, row, 0, len, s_lse2, ready);
  }
}

// Parts of one unit: n CTAs, P apart, hold one each; n is 1 when one CTA finished it.
struct Parts {
  int first, P, n;
  __device__ int slot(int k) const { return 2 * (first + k * P) + (k == 0); }
};

__device__ __forceinline__ Parts unit_parts(const DecodeParams& p, int s, int ui) {
  if (p.whole) return {0, 1, 1};
  const int before = p.pre[s], nt = p.pre[s + 1] - before;
  const int64_t per = *p.per;
  const int bundle = p.by_P.of(ui);
  const int64_t at = (int64_t)before * p.F + (int64_t)bundle * nt;
  const int g0 = (int)div_floor(at, per);
  return {g0 * p.P + (ui - bundle * p.P), p.P, (int)div_floor(at + nt - 1, per) - g0 + 1};
}

// m (0 for an empty row) and l of head h over the parts: one warp, the same in every lane
__device__ __forceinline__ float2 join_stats(const DecodeParams& p, const Parts& u, int HT, int h, int lane) {
  float M = -INFINITY;
  for (int k = lane; k < u.n; k += 32) M = fmaxf(M, p.part_ml[u.slot(k) * HT + h].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
  const float mu = M == -INFINITY ? 0.0f : M;
  float L = 0.0f;
  for (int k = lane; k < u.n; k += 32) {
    const float2 ml = p.part_ml[u.slot(k) * HT + h];
    L = fmaf(ex2(ml.x - mu), ml.y, L);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(~0u, L, o);
  return make_float2(mu, L);
}

// a += the parts first, first + step, .. of four columns of head h; part k is scaled to the row's m
__device__ __forceinline__ void add_parts(const DecodeParams& p, const Parts& u, int HT, int h, float mu, int column,
                                          int first, int step, float4& a) {
#pragma unroll 4
  for (int k = first; k < u.n; k += step) {
    const int at = u.slot(k) * HT + h;
    const float f = ex2(p.part_ml[at].x - mu);
    const float4 v = reinterpret_cast<const float4*>(p.part_O + (int64_t)at * p.d)[column];
    a.x = fmaf(f, v.x, a.x);
    a.y = fmaf(f, v.y, a.y);
    a.z = fmaf(f, v.z, a.z);
    a.w = fmaf(f, v.w, a.w);
  }
}
__device__ __forceinline__ void write_row(const DecodeParams& p, int row, int column, const float4& a, const float2& ml) {
  const float inv = ml.y == 0.0f ? 0.0f : 1.0f / ml.y;
  const int64_t at = (int64_t)row * p.d + 4 * column;
  if (p.o_f32) *reinterpret_cast<float4*>(p.O + 4 * at) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
  else *reinterpret_cast<uint2*>(p.O + 2 * at) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
  if (column == 0 && p.lse) p.lse[row] = ml.y == 0.0f ? -INFINITY : (ml.x + log2f(ml.y)) * LN2;
}

// The first `adders` CTAs, one per (key chunk, sequence, key head), turn the x_j into weights and
// add them up over the group.  The others add up the parts of the units that were cut: a warp
// takes a query head, or with `many` parts to a row a CTA does, in slices of the parts that are
// added up in order.  Both find the row's lse from the parts' (m, l), lanes over parts.
__global__ void __launch_bounds__(JOIN_THR, JOIN_CTAS) k_decode_join(const __grid_constant__ DecodeParams p, int HT,
                                                                     int adders, int keys, int many) {
  __shared__ float s_lse2[256];
  __shared__ float4 s_acc[JOIN_THR];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  await_earlier();
  if ((int)blockIdx.x >= adders) {
    const int nc = p.d >> 2, ns = JOIN_THR / nc;  // 16-byte columns of a row, slices
    const int per = many ? 1 : JOIN_THR / 32;     // rows a CTA takes at a time
    for (int64_t r0 = (int64_t)(blockIdx.x - adders) * per; r0 < (int64_t)p.kv.nseq * p.h_r; r0 += (int64_t)(gridDim.x - adders) * per) {
      const int row = (int)r0 + (many ? 0 : warp);
      if (row >= p.kv.nseq * p.h_r) continue;  // a warp on its own: rows of a CTA's are below
      const int s = row / p.h_r, r = row - s * p.h_r;
      const int hk = r / p.G, b = (r - hk * p.G) / HT, h = r - hk * p.G - b * HT;
      const Parts u = unit_parts(p, s, hk * p.hb + b);
      if (u.n == 1) continue;
      const float2 ml = join_stats(p, u, HT, h, lane);
      if (!many) {
        for (int c = lane; c < nc; c += 32) {
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
          add_parts(p, u, HT, h, ml.x, c, 0, 1, a);
          write_row(p, row, c, a, ml);
        }
        continue;
      }
      const int c = tid % nc, sl = tid / nc;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (sl < ns) add_parts(p, u, HT, h, ml.x, c, sl, ns, a);
      s_acc[tid] = a;
      __syncthreads();
      if (tid < nc) {
        for (int k = 1; k < min(ns, u.n); ++k) {
          const float4 v = s_acc[k * nc + tid];
          a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
        write_row(p, row, tid, a, ml);
      }
      __syncthreads();
    }
    return;
  }
  const int rows = p.kv.nseq * p.h_kv, job = blockIdx.x;
  const int chunk = job / rows, sg = job - chunk * rows;
  const int s = sg / p.h_kv, hk = sg - s * p.h_kv;
  const int len = kv_len(p.kv, s, false);
  const int64_t j0 = (int64_t)chunk * keys;
  if (j0 >= len) return;
  auto ready = [&] {  // lse2 of the group's heads (0 for an empty row)
    for (int h = warp; h < p.G; h += JOIN_THR / 32) {
      const int b = h / HT;
      const Parts u = unit_parts(p, s, hk * p.hb + b);
      float v;
      if (u.n == 1) {
        v = p.lse2[(int64_t)s * p.h_r + hk * p.G + h];
      } else {
        const float2 ml = join_stats(p, u, HT, h - b * HT, lane);
        v = ml.x + log2f(ml.y);
      }
      if (lane == 0) s_lse2[h] = v == -INFINITY ? 0.0f : v;
    }
    __syncthreads();
  };
  const int j1 = (int)min((int64_t)len, j0 + keys);
  if (p.GP % 4 == 0) add_weights<4, JOIN_THR>(p, sg, (int)j0, j1, s_lse2, ready);
  else add_weights<2, JOIN_THR>(p, sg, (int)j0, j1, s_lse2, ready);
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

constexpr int WHOLE_BF16 = 512;  // see whole_keys

// query heads per unit and keys per tile of the kernel that serves a descriptor
int head_tile(const mf_paged_decode_desc& d) {
  if (d.kv.dtype != MF_BF16 || d.h_r / d.kv.h_kv <= 8) return 8;
  // Groups of more than 8 heads: 16 at a time read the keys once (16 x 8192 tokens, groups of 16:
  // 102 us, 8 at a time 118).  Few short sequences leave SMs idle, and 8 at a time are done sooner
  // (32 key heads of 300 keys 7.0 us, 16 at a time 10.3; 64 of them 7.2 and 10.4; 32 of 512 keys 9.5
  // and 14.2); with weights they would need the join.
  const bool few = d.kv.max_len <= WHOLE_BF16 && (int64_t)d.kv.nseq * d.kv.h_kv <= 64;
  return few && !d.score_out ? 8 : 16;
}

// One CTA per unit, without a second launch, for bounds max_len up to this many keys: a split call
// takes 8 us at any length, one CTA's time grows with its keys.  Alone and split, us:
//   bf16     512 keys: 8 units 8.6 and 8.6, 64 units 9.5 and 11.2, 512 units 25.4 and 29.4;
//            700 keys: 11.4 and 9.0, 12.4 and 12.9, 32.8 and 36.8;
//            512 keys with weights: 10.7 and 8.8, 12.9 and 13.3, 32.6 and 35.9;
//   float32  128 keys: 8 units 6.7 and 8.8, 64 units 7.1 and 9.8; 256 keys: 11.2 and 9.2, 12.0 and 12.1;
//            512 units, more than CTAs: 256 keys 29.9 and 33.1, 350 keys 38.0 and 41.1.
int whole_keys(const mf_paged_decode_desc& d, bool fill) { return d.kv.dtype == MF_BF16 ? WHOLE_BF16 : fill ? 256 : 128; }

}  // namespace

size_t paged_decode_ws(const mf_paged_decode_desc& d, PagedDecodeWs* ws, void* base) {
  const int HT = head_tile(d), G = d.h_r / d.kv.h_kv, GP = (G + 1) & ~1;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* q = base ? static_cast<char*>(base) + at : nullptr;
    at += up256(bytes);
    return q;
  };
  char* pre = take(4 * ((size_t)d.kv.nseq + 1));
  char* per = take(sizeof(int64_t));
  char* lse2 = take(4 * (size_t)d.kv.nseq * d.h_r);
  char* po = take(sizeof(float) * 2 * MAX_GRID * (size_t)HT * d.kv.d);
  char* ml = take(sizeof(float2) * 2 * MAX_GRID * (size_t)HT);
  char* S = d.score_out ? take(4 * (size_t)d.kv.nseq * d.kv.h_kv * d.kv.max_len * GP) : nullptr;
  if (ws) {
    ws->pre = reinterpret_cast<int32_t*>(pre);
    ws->per = reinterpret_cast<int64_t*>(per);
    ws->lse2 = reinterpret_cast<float*>(lse2);
    ws->part_O = reinterpret_cast<float*>(po);
    ws->part_ml = reinterpret_cast<float2*>(ml);
    ws->S = reinterpret_cast<float*>(S);
  }
  return at;
}

cudaError_t launch_paged_decode(const mf_paged_decode_desc& d, const PagedDecodeWs& ws, uint32_t* status,
                                cudaStream_t st) {
  DecodeParams p{};
  p.kv = kv_view(d.kv, status);
  const int e = d.kv.dtype == MF_F32 ? 4 : 2;
  p.Q = static_cast<const char*>(d.Q);
  p.h_r = d.h_r;
  p.h_kv = d.kv.h_kv;
  p.d = d.kv.d;
  p.G = d.h_r / d.kv.h_kv;
  p.GP = (p.G + 1) & ~1;
  const int HT = head_tile(d);
  p.hb = (p.G + HT - 1) / HT;
  p.U = p.h_kv * p.hb;
  p.q_bytes = (d.q_stride ? d.q_stride : (int64_t)d.h_r * p.d) * e;
  const double scale = d.scale > 0.0f ? (double)d.scale : 1.0 / std::sqrt((double)p.d);
  p.c2 = (float)(scale * 1.4426950408889634074);
  p.O = static_cast<char*>(d.O);
  p.o_f32 = d.kv.dtype == MF_F32 || (d.flags & MF_DECODE_O_F32);
  p.lse = d.lse;
  p.S = d.score_out ? ws.S : nullptr;
  p.score_in = d.score_in;
  p.score_out = d.score_out;
  p.score_stride = d.score_stride;
  p.pre = ws.pre;
  p.per = ws.per;
  p.lse2 = ws.lse2;
  p.part_O = ws.part_O;
  p.part_ml = ws.part_ml;

  int dev = 0, sms = 0;
  cudaError_t e0 = cudaGetDevice(&dev);
  if (e0 == cudaSuccess) e0 = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e0 != cudaSuccess) return e0;

  cudaError_t err = cudaSuccess;
  int grid = 0;
  auto launch = [&](auto core) {
    using Core = decltype(core);
    const int resident = std::min(MAX_GRID, sms * Core::CTAS), units = p.kv.nseq * p.U;
    p.whole = d.kv.max_len <= whole_keys(d, units > resident);
    p.own_scores = p.whole && p.S && p.hb == 1;
    // the widest bundle whose groups of CTAs leave few of the resident ones without work
    p.P = p.U;
    while (p.U % p.P || 20 * (resident / p.P * p.P) < 19 * resident) --p.P;  // 1 leaves none
    p.F = p.U / p.P;
    p.groups = resident / p.P;
    p.groups_each = p.groups / p.F;
    p.by_P = Divider(p.P);
    p.by_groups = Divider(p.groups);
    grid = p.whole ? units : p.groups * p.P;
    const size_t smem = (size_t)WARPS * Core::STAGES * Core::TILE + (p.whole ? 0 : 4 * ((size_t)p.kv.nseq + 1));
    // room for the scan of the largest batch
    err = allow_smem<&k_decode<Core>>(dev, WARPS * Core::STAGES * Core::TILE + 4 * (MAX_SEQS + 1));
    if (err != cudaSuccess) return;
    err = launch_early(k_decode<Core>, grid, NTHR, smem, 1, st, p);
  };
  const int D = p.d <= 64 ? 64 : p.d <= 128 ? 128 : p.d <= 192 ? 192 : 256;
  if (d.kv.dtype == MF_F32) {
    if (D == 64) launch(CoreF32<64>{});
    else if (D == 128) launch(CoreF32<128>{});
    else if (D == 192) launch(CoreF32<192>{});
    else launch(CoreF32<256>{});
  } else if (HT == 8) {
    if (D == 64) launch(CoreBf16<64, 1>{});
    else if (D == 128) launch(CoreBf16<128, 1>{});
    else if (D == 192) launch(CoreBf16<192, 1>{});
    else launch(CoreBf16<256, 1>{});
  } else {
    if (D == 64) launch(CoreBf16<64, 2>{});
    else if (D == 128) launch(CoreBf16<128, 2>{});
    else if (D == 192) launch(CoreBf16<192, 2>{});
    else launch(CoreBf16<256, 2>{});
  }
  if (err != cudaSuccess || (p.whole && (!p.score_out || p.own_scores))) return err;

  // parts of a row if all were equally long: from 8 on its join is split over a CTA's warps
  const int many = grid >= 8 * p.kv.nseq * p.U;
  const int joiners = p.whole ? 0 : std::min(MAX_JOINERS, many ? p.kv.nseq * p.h_r : (p.kv.nseq * p.h_r + 7) / 8);
  // keys of an adder: the adders fill the GPU once, since each looks its row up first
  const int rows = p.kv.nseq * p.h_kv;
  const int64_t share = p.kv.max_len / std::max(1, JOIN_CTAS * sms / rows);
  const int keys = (int)std::max<int64_t>(1, (share + JOIN_KEYS - 1) / JOIN_KEYS) * JOIN_KEYS;
  const int adders = p.score_out ? (int)(((int64_t)p.kv.max_len + keys - 1) / keys) * rows : 0;
  const unsigned ctas = (unsigned)adders + (unsigned)joiners;
  if (ctas == 0) return cudaSuccess;
  return launch_early(k_decode_join, ctas, JOIN_THR, 0, 1, st, p, HT, adders, keys, many);
}

}  // namespace mfi
