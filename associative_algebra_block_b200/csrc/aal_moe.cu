// One decode step of a mixture of algebraic SwiGLU experts: for every entry
// the router's logits, the top-k experts and their weights, the experts' row-
// typed gate, up and down products, and their weighted sum plus the residual.
//
//   l = x Wr;  e_1..e_k = the k largest logits (ties: the lower index)
//   w_j = softmax(l)[e_j], or softmax over the chosen logits alone
//   y = (r) + sum_j w_j (silu(x * Wg_e) . (x * Wu_e)) * Wd_e,   e = e_j
//
// with every "*" row t = position mod q of the table.  Three launches chained
// by programmatic dependent launch:
//   k_moe_router   a cluster an entry (or four): logits, top-k, weights
//   k_moe_up       gate, up and SiLU of one expert's 64 columns a CTA
//   k_moe_down     64 columns of y a cluster, its CTAs dealing the experts out
// The experts' weights are the work: each weight block that some entry needs
// is read once for all entries that share the expert.
#include "aal_internal.h"

#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

namespace aal {
namespace moe {

namespace cg = cooperative_groups;

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;"); }

constexpr int kMaxTopK = 32;
constexpr int kChunk = 128;  // entries of one chain of launches

// ------------------------------------------------------------------- router
// A cluster of kRouterCtas CTAs takes TB entries: CTA r the input rows of
// slice r, a thread VEC adjacent experts on every RL-th row of it.  The logits
// are sums of exact products in fp64 (an expert chosen or not by a rounding
// would change the whole row), added over the row lanes and the CTAs in a
// fixed order.
constexpr int kRouterCtas = 8, kRouterThreads = 256;

struct RouterArgs {
  const void *x, *wr;
  const int64_t* positions;
  int* ids;
  float* weights;
  long long ldx, ldr;
  int B, D, E, k, renorm;
};

template <typename T>
__device__ __forceinline__ double widen(T v) { return (double)ld_elem(&v); }

template <typename T, int VEC, int TB>
__global__ void __cluster_dims__(kRouterCtas, 1, 1) __launch_bounds__(kRouterThreads) k_moe_router(const RouterArgs a) {
  extern __shared__ double sm[];
  double* part = sm;                        // [TB][E] this CTA's sums
  double* red = part + (size_t)TB * a.E;    // [threads][VEC] (one entry at a time)
  double* logit = red + kRouterThreads * VEC;  // [TB][E] (rank 0)
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tid = threadIdx.x;
  pdl_release();
  pdl_wait();
  const int b0 = (int)(blockIdx.x / kRouterCtas) * TB;
  const int nb = min(TB, a.B - b0);
  const int ds = (a.D + kRouterCtas - 1) / kRouterCtas;
  const int d0 = min(a.D, rank * ds), d1 = min(a.D, d0 + ds);
  const int ncv = (a.E + VEC - 1) / VEC;
  int cvb = 1;  // column vectors a pass
  while (cvb < ncv && cvb < kRouterThreads) cvb <<= 1;
  const int rl = kRouterThreads / cvb;  // row lanes
  const T *x = (const T*)a.x, *wr = (const T*)a.wr;
  for (int c0 = 0; c0 < ncv; c0 += cvb) {
    const int cv = c0 + tid % cvb, lane_r = tid / cvb;
    double acc[TB][VEC];
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[b][j] = 0.0;
    if (cv < ncv) {
#pragma unroll 4
      for (int d = d0 + lane_r; d < d1; d += rl) {
        T w[VEC];
        if constexpr (VEC == 1) {
          w[0] = wr[(long long)d * a.ldr + cv];
        } else {
          const uint4 u = *reinterpret_cast<const uint4*>(wr + (long long)d * a.ldr + (long long)cv * VEC);
          memcpy(w, &u, 16);
        }
        double xv[TB];
#pragma unroll
        for (int b = 0; b < TB; ++b) xv[b] = b < nb ? widen(x[(long long)(b0 + b) * a.ldx + d]) : 0.0;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const double wv = widen(w[j]);
#pragma unroll
          for (int b = 0; b < TB; ++b) acc[b][j] = fma(wv, xv[b], acc[b][j]);
        }
      }
    }
    for (int b = 0; b < TB; ++b) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) red[j * kRouterThreads + tid] = 0.0;
#pragma unroll
      for (int bb = 0; bb < TB; ++bb)
        if (bb == b) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) red[j * kRouterThreads + tid] = acc[bb][j];
        }
      __syncthreads();
      for (int i = tid; i < cvb * VEC; i += kRouterThreads) {
        const int j = i / cvb, c = i - j * cvb, e = (c0 + c) * VEC + j;
        if (e < a.E) {
          double s = 0.0;
          for (int l = 0; l < rl; ++l) s += red[j * kRouterThreads + l * cvb + c];
          part[(size_t)b * a.E + e] = s;
        }
      }
      __syncthreads();
    }
  }
  cl.sync();
  if (rank == 0) {
    for (int i = tid; i < nb * a.E; i += kRouterThreads) {
      double s = 0.0;
#pragma unroll
      for (int r = 0; r < kRouterCtas; ++r) s += cl.map_shared_rank(part, r)[i];
      logit[i] = s;
    }
  }
  cl.sync();  // the peers' sums have been read
  if (rank != 0) return;
  const int warp = tid >> 5, lane = tid & 31;
  if (warp >= nb) return;
  const int b = b0 + warp;
  double* l = logit + (size_t)warp * a.E;
  int* ids = a.ids + (long long)b * a.k;
  float* wts = a.weights + (long long)b * a.k;
  if (a.positions[b] < 0) {  // skipped: no expert, no output row
    if (lane == 0) flag_device_error(kDevBounds);
    for (int j = lane; j < a.k; j += 32) {
      ids[j] = -1;
      wts[j] = 0.f;
    }
    return;
  }
  // the largest logit (NaN where one is NaN) and the softmax's sum
  double mx = -INFINITY;
  bool nan = false;
  for (int e = lane; e < a.E; e += 32) {
    const double v = l[e];
    nan |= isnan(v);
    mx = v > mx ? v : mx;
  }
  for (int o = 16; o > 0; o >>= 1) {
    const double v = __shfl_xor_sync(0xffffffffu, mx, o);
    mx = v > mx ? v : mx;
  }
  nan = __any_sync(0xffffffffu, nan);
  float sum = 0.f;
  if (!a.renorm) {
    for (int e = lane; e < a.E; e += 32) sum += expf((float)(l[e] - mx));
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  // k rounds of the largest not yet taken; a NaN ranks as -infinity, so the
  // chosen indices are always k different experts
  float mine = 0.f;               // lane j: the weight of choice j
  unsigned long long taken = 0;   // bit i: expert lane + 32 i (kMaxExperts fit)
  for (int j = 0; j < a.k; ++j) {
    double best = -INFINITY;
    int at = INT_MAX;
    for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
      if ((taken >> i) & 1ull) continue;
      double v = l[e];
      if (isnan(v)) v = -INFINITY;
      if (at == INT_MAX || v > best) { best = v; at = e; }
    }
    for (int o = 16; o > 0; o >>= 1) {
      const double v = __shfl_xor_sync(0xffffffffu, best, o);
      const int i = __shfl_xor_sync(0xffffffffu, at, o);
      if (i != INT_MAX && (at == INT_MAX || v > best || (v == best && i < at))) { best = v; at = i; }
    }
    const float p = nan ? NAN : expf((float)(best - mx));
    if (a.renorm) sum += p;
    if (lane == j) {
      mine = p;
      ids[j] = at;
    }
    if ((at & 31) == lane) taken |= 1ull << (at >> 5);
  }
  if (lane < a.k) wts[lane] = mine / sum;
}

// ------------------------------------------------- experts, tensor-core path
// A warp multiplies 64 weight columns by up to 8 NT entries with
// mma.sync.m16n8k16: M = the columns, N = the entries, K = weight rows, 16 a
// step.  The order of K inside a step is free as long as both operands agree,
// so lane (g, t) = (lane / 4, lane % 4) takes rows 4t..4t+3 of the step and
// columns 8g..8g+7: one 16-byte load a row, whole 128-byte lines a warp, and
// the fragments of the four 16-column tiles are byte permutes of those
// registers (tile i holds columns 8g + 2i and 8g + 2i + 1).  The weights
// therefore go from global memory to the matrix instruction without shared
// memory, and a warp keeps kDepth steps (kDepth * 2 KB) in flight.
constexpr int kDepth = 4;
constexpr int kTile = 64;       // output columns of a CTA's tile
constexpr int kUpThreads = 256, kDownThreads = 256;
constexpr int kMaxQ = 256;

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// The entries (slots) of one expert, gathered by the whole CTA.
struct Slots {
  int n;            // slots of the expert
  int* slot;        // [n] ascending
};

// Collects the slots s < n with ids[s] == e in ascending order into ``out``;
// every thread returns their number.  ``cnt``: 32 ints of shared memory.
__device__ __forceinline__ int collect(const int* ids, int n, int e, int* out, int* cnt) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int total = 0;
  for (int s0 = 0; s0 < n; s0 += blockDim.x) {
    const int s = s0 + (int)threadIdx.x;
    const bool hit = s < n && ids[s] == e;
    const unsigned m = __ballot_sync(0xffffffffu, hit);
    if (lane == 0) cnt[warp] = __popc(m);
    __syncthreads();
    int before = total;
    for (int w = 0; w < nw; ++w) {
      const int c = cnt[w];
      if (w < warp) before += c;
      total += c;
    }
    if (hit) out[before + __popc(m & ((1u << lane) - 1u))] = s;
    __syncthreads();
  }
  return total;
}

// The expert of unit u.  With at least as many slots as experts a unit is an
// expert; with fewer a unit is a slot, which stands for its expert if it is
// the first one to choose it.  -1: the unit has no work.
__device__ __forceinline__ int unit_expert(const int* ids, int n, int E, int u) {
  if (n >= E) return u;
  const int e = ids[u];
  if (e < 0) return -1;
  bool seen = false;
  for (int s = threadIdx.x; s < u; s += blockDim.x) seen |= ids[s] == e;
  return __syncthreads_or(seen) ? -1 : e;
}

// The groups that some of the n entries needs for output group kg, as a list
// in ascending order; returns how many (every thread).
__device__ __forceinline__ int used_groups(int law, int q, const int* types, int n, int kg, unsigned* mask,
                                           uint16_t* list, int* count) {
  for (int i = threadIdx.x; i < kMaxQ / 32; i += blockDim.x) mask[i] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int m[4];
    const int c = table_members(law, q, types[i], kg, m);
    for (int j = 0; j < c; ++j) atomicOr(&mask[m[j] >> 5], 1u << (m[j] & 31));
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int at = 0;
    for (int w = 0; w < kMaxQ / 32; ++w) {
      const unsigned v = mask[w];
      const int lane = threadIdx.x;
      if ((v >> lane) & 1u) list[at + __popc(v & ((1u << lane) - 1u))] = (uint16_t)(w * 32 + lane);
      at += __popc(v);
    }
    if (threadIdx.x == 0) *count = at;
  }
  __syncthreads();
  return *count;
}

// Accumulates acc[i][nt] += (64 columns at ``w``) x (entries of the chunk) over
// the steps first, first + stride, ... of the used groups.  ``w`` points at
// row 0, column 8g of the tile (lanes past its width pass wide = false and
// load nothing); xrow[nt]: the input row of entry nt * 8 + g, or null.
template <int NT>
__device__ __forceinline__ void stream_tile(const __nv_bfloat16* w, long long ldw, bool wide, int law, int kg,
                                            int nused, const uint16_t* used, int gw, int first, int stride,
                                            const __nv_bfloat16* const* xrow, const int* xtype,
                                            float (&acc)[4][NT][4]) {
  const int t4 = (threadIdx.x & 3) * 4;
  const int spg = gw >> 4;  // steps a group
  int gi = first / spg, in = first - gi * spg;
  while (gi < nused) {
    uint4 wv[kDepth][4];
    uint2 xv[kDepth][NT];
    int pg = gi, pi = in;
#pragma unroll
    for (int s = 0; s < kDepth; ++s) {
      const bool on = pg < nused;
      const int grp = on ? used[pg] : 0;
      const long long r = (long long)grp * gw + pi * 16 + t4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        wv[s][i] = (on && wide) ? __ldg(reinterpret_cast<const uint4*>(w + (r + i) * ldw)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        xv[s][nt] = (on && xrow[nt] && in_table(law, xtype[nt], kg, grp))
                        ? *reinterpret_cast<const uint2*>(xrow[nt] + r)
                        : make_uint2(0, 0);
      pi += stride;
      while (pi >= spg) { pi -= spg; ++pg; }
    }
#pragma unroll
    for (int s = 0; s < kDepth; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w0 = word(wv[s][0], i), w1 = word(wv[s][1], i), w2 = word(wv[s][2], i), w3 = word(wv[s][3], i);
        const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
        const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(acc[i][nt], a0, a1, a2, a3, xv[s][nt].x, xv[s][nt].y);
      }
    }
    gi = pg;
    in = pi;
  }
}

// Writes a warp's accumulators to red[n][64].
template <int NT>
__device__ __forceinline__ void spill(float* red, const float (&acc)[4][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* p = red + (size_t)(nt * 8 + 2 * t) * kTile + 8 * g + 2 * i;
      *reinterpret_cast<float2*>(p) = make_float2(acc[i][nt][0], acc[i][nt][2]);
      *reinterpret_cast<float2*>(p + kTile) = make_float2(acc[i][nt][1], acc[i][nt][3]);
    }
}

struct ExpertArgs {
  const int64_t* positions;
  const int* ids;
  const float* weights;
  const __nv_bfloat16 *x, *wg, *wu, *wd, *r;
  __nv_bfloat16 *h, *y;
  long long ldx, ldg, ldu, ldd, ldh, ldr, ldy;
  int law, q, B, k, E, D, F;
  int tiles;   // column tiles of an output group
  int units;
  int zsplit;  // k_moe_up: CTAs of a cluster; k_moe_down: CTAs that share an expert
};

// Lists one chunk's entries for this thread: the input rows and types of
// entries nt * 8 + g.
template <int NT>
__device__ __forceinline__ void chunk_rows(const __nv_bfloat16* base, long long ld, const int* rows, const int* types,
                                           int n0, int n, const __nv_bfloat16** xrow, int* xtype) {
  const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int i = n0 + nt * 8 + g;
    xrow[nt] = i < n ? base + (long long)rows[i] * ld : nullptr;
    xtype[nt] = i < n ? types[i] : 0;
  }
}

// h of one expert's 64 columns: warps 0-3 stream the gate's weights, warps
// 4-7 the up projection's, each every 4 zsplit-th step; a cluster of zsplit
// CTAs splits K further where there are few tiles and adds its parts in rank
// order through distributed shared memory.
template <int NT>
__global__ void __launch_bounds__(kUpThreads, 2) k_moe_up(const ExpertArgs a) {
  extern __shared__ float smf[];
  __shared__ int cnt[32], nu;
  __shared__ unsigned gmask[kMaxQ / 32];
  __shared__ uint16_t glist[kMaxQ];
  __shared__ int slot[kChunk], type[kChunk], tok[kChunk];
  float* red = smf;                          // [8 warps][8 NT][64]
  float* gu = red + 8 * 8 * NT * kTile;      // [2][8 NT][64] this CTA's gate and up sums
  cg::cluster_group cl = cg::this_cluster();
  const int z = a.zsplit, rank = (int)(blockIdx.x % z), tile = (int)(blockIdx.x / z);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_release();  // after the wait: a dependent that starts now finds the router's results complete
  const int nslots = a.B * a.k;
  const int e = unit_expert(a.ids, nslots, a.E, (int)blockIdx.y);
  if (e < 0) return;
  // an expert's slots belong to different entries, so there are at most kChunk
  const int n = collect(a.ids, nslots, e, slot, cnt);
  if (n == 0) return;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    tok[i] = slot[i] / a.k;
    type[i] = (int)(a.positions[tok[i]] % a.q);
  }
  __syncthreads();
  const int bi = a.D / a.q, bo = a.F / a.q;
  const int kg = tile / a.tiles, c0 = kg * bo + (tile - kg * a.tiles) * kTile;
  const int width = min(kTile, (kg + 1) * bo - c0);
  const int nused = used_groups(a.law, a.q, type, n, kg, gmask, glist, &nu);
  const bool wide = 8 * (lane >> 2) < width;
  const bool up = warp >= 4;
  const long long ldw = up ? a.ldu : a.ldg;
  const __nv_bfloat16* w = (up ? a.wu : a.wg) + (long long)e * a.D * ldw + c0 + 8 * (lane >> 2);
  for (int n0 = 0; n0 < n; n0 += 8 * NT) {
    const __nv_bfloat16* xrow[NT];
    int xtype[NT];
    chunk_rows<NT>(a.x, a.ldx, tok, type, n0, n, xrow, xtype);
    float acc[4][NT][4] = {};
    stream_tile<NT>(w, ldw, wide, a.law, kg, nused, glist, bi, rank * 4 + (warp & 3), 4 * z, xrow, xtype, acc);
    spill<NT>(red + warp * 8 * NT * kTile, acc);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * 8 * NT * kTile; i += blockDim.x) {
      const int m = i / (8 * NT * kTile), j = i - m * 8 * NT * kTile;
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < 4; ++v) s += red[(m * 4 + v) * 8 * NT * kTile + j];
      gu[i] = s;
    }
    if (z > 1) cl.sync();
    else __syncthreads();
    // the cluster's CTAs finish the entries n mod z == rank
    const int nc = min(8 * NT, n - n0);
    for (int i = threadIdx.x; i < nc * kTile; i += blockDim.x) {
      const int m = i / kTile, c = i - m * kTile;
      if (m % z != rank || c >= width) continue;
      float g = 0.f, u = 0.f;
      for (int v = 0; v < z; ++v) {
        const float* p = z > 1 ? cl.map_shared_rank(gu, v) : gu;
        g += p[i];
        u += p[8 * NT * kTile + i];
      }
      a.h[(long long)slot[n0 + m] * a.ldh + c0 + c] = __float2bfloat16_rn(g / (1.f + expf(-g)) * u);
    }
    if (z > 1) cl.sync();
    else __syncthreads();
  }
}

// 64 columns of y: the cluster's CTAs take the experts in turn (zsplit of
// them share one expert's K range where there are few experts), add each
// expert's weighted product to the CTA's sums in shared memory, and the
// cluster adds the CTAs' sums in rank order with the residual.
constexpr int kDownCtas = 8;
template <int NT>
__global__ void __cluster_dims__(kDownCtas, 1, 1) __launch_bounds__(kDownThreads, 2) k_moe_down(const ExpertArgs a) {
  extern __shared__ float smf[];
  __shared__ int cnt[32], nu;
  __shared__ unsigned gmask[kMaxQ / 32];
  __shared__ uint16_t glist[kMaxQ];
  __shared__ int slot[kChunk], type[kChunk];
  float* red = smf;                       // [8 warps][8 NT][64]
  float* ys = red + 8 * 8 * NT * kTile;   // [B][64]
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tile = (int)(blockIdx.x / kDownCtas);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < a.B * kTile; i += blockDim.x) ys[i] = 0.f;
  pdl_wait();
  pdl_release();
  const int nslots = a.B * a.k;
  const int bi = a.F / a.q, bo = a.D / a.q;
  const int kg = tile / a.tiles, c0 = kg * bo + (tile - kg * a.tiles) * kTile;
  const int width = min(kTile, (kg + 1) * bo - c0);
  const bool wide = 8 * (lane >> 2) < width;
  const int z = a.zsplit, lanes = kDownCtas / z;
  for (int u = rank / z; u < a.units; u += lanes) {
    const int e = unit_expert(a.ids, nslots, a.E, u);
    if (e < 0) continue;
    const int n = collect(a.ids, nslots, e, slot, cnt);
    if (n == 0) continue;
    for (int i = threadIdx.x; i < n; i += blockDim.x) type[i] = (int)(a.positions[slot[i] / a.k] % a.q);
    __syncthreads();
    const int nused = used_groups(a.law, a.q, type, n, kg, gmask, glist, &nu);
    const __nv_bfloat16* w = a.wd + (long long)e * a.F * a.ldd + c0 + 8 * (lane >> 2);
    for (int n0 = 0; n0 < n; n0 += 8 * NT) {
      const __nv_bfloat16* xrow[NT];
      int xtype[NT];
      chunk_rows<NT>(a.h, a.ldh, slot, type, n0, n, xrow, xtype);
      float acc[4][NT][4] = {};
      stream_tile<NT>(w, a.ldd, wide, a.law, kg, nused, glist, bi, (rank % z) * 8 + warp, 8 * z, xrow, xtype, acc);
      spill<NT>(red + warp * 8 * NT * kTile, acc);
      __syncthreads();
      const int nc = min(8 * NT, n - n0);
      for (int i = threadIdx.x; i < nc * kTile; i += blockDim.x) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < 8; ++v) s += red[v * 8 * NT * kTile + i];
        const int sl = slot[n0 + i / kTile];
        ys[sl / a.k * kTile + i % kTile] += a.weights[sl] * s;
      }
      __syncthreads();
    }
  }
  cl.sync();
  // the cluster's CTAs finish the entries b mod 8 == rank
  for (int i = threadIdx.x; i < a.B * kTile; i += blockDim.x) {
    const int b = i / kTile, c = i - b * kTile;
    if (b % kDownCtas != rank || c >= width || a.positions[b] < 0) continue;
    float s = a.r ? __bfloat162float(a.r[(long long)b * a.ldr + c0 + c]) : 0.f;
    for (int v = 0; v < kDownCtas; ++v) s += cl.map_shared_rank(ys, v)[i];
    a.y[(long long)b * a.ldy + c0 + c] = __float2bfloat16_rn(s);
  }
  cl.sync();  // the peers' sums have been read
}

// ---------------------------------------------------------- experts, any shape
// 32 output columns a CTA, the K range dealt to its 8 warps.  One (entry,
// choice) a CTA row for gate/up, one entry for down.
template <typename T>
struct GenArgs {
  const int64_t* positions;
  const int* ids;
  const float* weights;
  const T *x, *wg, *wu, *wd, *r;
  T *h, *y;
  long long ldx, ldg, ldu, ldd, ldh, ldr, ldy;
  int law, q, k, D, F;
};

template <typename T>
__global__ void __launch_bounds__(256) k_moe_up_general(const GenArgs<T> a) {
  __shared__ float sg[8][33], su[8][33];
  pdl_wait();
  pdl_release();
  const int s = (int)blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = a.ids[s];
  if (e < 0) return;
  const int b = s / a.k, t = (int)(a.positions[b] % a.q);
  const int c = (int)blockIdx.x * 32 + lane;
  const int bi = a.D / a.q, bo = a.F / a.q;
  float g = 0.f, u = 0.f;
  if (c < a.F) {
    int m[4];
    const int n = table_members(a.law, a.q, t, c / bo, m);
    for (int i = 0; i < n; ++i) {
      const T* x = a.x + (long long)b * a.ldx + (long long)m[i] * bi;
      const T* wg = a.wg + ((long long)e * a.D + (long long)m[i] * bi) * a.ldg + c;
      const T* wu = a.wu + ((long long)e * a.D + (long long)m[i] * bi) * a.ldu + c;
#pragma unroll 8
      for (int j = warp; j < bi; j += 8) {
        const float xv = ld_elem(x + j);
        g = fmaf(xv, ld_elem(wg + (long long)j * a.ldg), g);
        u = fmaf(xv, ld_elem(wu + (long long)j * a.ldu), u);
      }
    }
  }
  sg[warp][lane] = g;
  su[warp][lane] = u;
  __syncthreads();
  if (warp || c >= a.F) return;
  g = u = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g += sg[i][lane];
    u += su[i][lane];
  }
  st_elem(a.h + (long long)s * a.ldh + c, g / (1.f + expf(-g)) * u);
}

template <typename T>
__global__ void __launch_bounds__(256) k_moe_down_general(const GenArgs<T> a) {
  __shared__ float sy[8][33];
  pdl_wait();
  pdl_release();
  const int b = (int)blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long pos = a.positions[b];
  if (pos < 0) return;
  const int t = (int)(pos % a.q);
  const int c = (int)blockIdx.x * 32 + lane;
  const int bi = a.F / a.q, bo = a.D / a.q;
  float y = 0.f;
  if (c < a.D) {
    int m[4];
    const int n = table_members(a.law, a.q, t, c / bo, m);
    for (int j = 0; j < a.k; ++j) {
      const int s = b * a.k + j, e = a.ids[s];
      float p = 0.f;
      for (int i = 0; i < n; ++i) {
        const T* h = a.h + (long long)s * a.ldh + (long long)m[i] * bi;
        const T* wd = a.wd + ((long long)e * a.F + (long long)m[i] * bi) * a.ldd + c;
#pragma unroll 8
        for (int r = warp; r < bi; r += 8) p = fmaf(ld_elem(h + r), ld_elem(wd + (long long)r * a.ldd), p);
      }
      y = fmaf(a.weights[s], p, y);
    }
  }
  sy[warp][lane] = y;
  __syncthreads();
  if (warp || c >= a.D) return;
  y = a.r ? ld_elem(a.r + (long long)b * a.ldr + c) : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) y += sy[i][lane];
  st_elem(a.y + (long long)b * a.ldy + c, y);
}

// ------------------------------------------------------------------ launches
// A launch that may start while the stream's previous kernel runs (the kernels
// wait for it before they touch global memory); ``cluster`` > 0 sets a cluster
// size at launch.
template <typename... A>
static aal_status launch(void (*k)(A...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, A... args) {
  if (smem > 32 * 1024 &&  // the static arrays count too
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return AAL_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 0) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
  note_launch();
  return cuda_status(e);
}

template <typename T, int VEC, int TB>
static aal_status run_router(const RouterArgs& a, cudaStream_t s) {
  const size_t smem = ((size_t)2 * TB * a.E + (size_t)kRouterThreads * VEC) * sizeof(double);
  return launch(k_moe_router<T, VEC, TB>, dim3((unsigned)((a.B + TB - 1) / TB * kRouterCtas)), kRouterThreads, smem, 0,
                s, a);
}
template <typename T, int VEC>
static aal_status run_router_tb(const RouterArgs& a, cudaStream_t s) {
  return a.B <= 16 ? run_router<T, VEC, 1>(a, s) : run_router<T, VEC, 4>(a, s);
}

// The widest router the kernel holds in shared memory.
constexpr int kMaxExperts = 2048;

static bool vec16(const aal_mat& m) {
  const size_t es = m.dtype == AAL_F32 ? 4 : 2;
  return !m.ptr || (((uintptr_t)m.ptr % 16) == 0 && (m.ld * es) % 16 == 0);
}

template <int NT>
static aal_status run_experts(ExpertArgs a, cudaStream_t s) {
  const int sms = device_sms();
  const int bo = a.F / a.q, bi = a.D / a.q;
  a.tiles = (bo + kTile - 1) / kTile;
  const int utiles = a.q * a.tiles;
  // split K over a cluster while that fills SMs and leaves every warp a step
  const int steps = (a.q < 2 ? 1 : 2) * (bi >> 4);
  int z = 1;
  while (z < 8 && (long long)utiles * a.units * z * 2 <= 2LL * sms && steps >= 8 * z) z *= 2;
  a.zsplit = z;
  aal_status st = timed(AAL_KERNEL_MOE_UP, s, [&] {
    return launch(k_moe_up<NT>, dim3((unsigned)(utiles * z), (unsigned)a.units), kUpThreads,
                  (size_t)(8 + 2) * 8 * NT * kTile * sizeof(float), z > 1 ? z : 0, s, a);
  });
  if (st != AAL_OK) return st;
  a.tiles = (bi + kTile - 1) / kTile;
  a.zsplit = a.units >= 8 ? 1 : a.units >= 4 ? 2 : a.units >= 2 ? 4 : 8;
  return timed(AAL_KERNEL_MOE_DOWN, s, [&] {
    return launch(k_moe_down<NT>, dim3((unsigned)(a.q * a.tiles * kDownCtas)), kDownThreads,
                  ((size_t)8 * 8 * NT + a.B) * kTile * sizeof(float), 0, s, a);
  });
}

template <typename T>
static aal_status run_general(int law, int q, const int64_t* positions, const aal_mat& x, const aal_mat& Wg,
                              const aal_mat& Wu, const aal_mat& Wd, const aal_mat& R, const int* ids,
                              const float* weights, int k, const aal_mat& h, const aal_mat& y, int B, int D, int F,
                              cudaStream_t s) {
  GenArgs<T> a = {positions, ids, weights, (const T*)x.ptr, (const T*)Wg.ptr, (const T*)Wu.ptr, (const T*)Wd.ptr,
                  (const T*)R.ptr, (T*)h.ptr, (T*)y.ptr, x.ld, Wg.ld, Wu.ld, Wd.ld, h.ld, R.ld, y.ld, law, q, k, D, F};
  aal_status st = timed(AAL_KERNEL_MOE_UP, s, [&] {
    return launch(k_moe_up_general<T>, dim3((unsigned)((F + 31) / 32), (unsigned)(B * k)), 256, 0, 0, s, a);
  });
  if (st != AAL_OK) return st;
  return timed(AAL_KERNEL_MOE_DOWN, s, [&] {
    return launch(k_moe_down_general<T>, dim3((unsigned)((D + 31) / 32), (unsigned)B), 256, 0, 0, s, a);
  });
}

}  // namespace moe
}  // namespace aal

using namespace aal;

extern "C" aal_status aal_moe_decode(int32_t law, int32_t q, const int64_t* positions, aal_mat x, aal_mat Wr, aal_mat Wg,
                                     aal_mat Wu, aal_mat Wd, aal_mat R, int32_t top_k, int32_t renormalize,
                                     int32_t* ids, float* weights, aal_mat h, aal_mat y, void* stream) {
  if (!valid_law(law, q) || !valid_mat(x) || !valid_mat(Wr) || !valid_mat(Wg) || !valid_mat(Wu) || !valid_mat(Wd) ||
      (R.ptr && !valid_mat(R)) || !valid_mat(h) || !valid_mat(y))
    return AAL_ERR_INVALID_ARG;
  const int dt = x.dtype;
  if (Wr.dtype != dt || Wg.dtype != dt || Wu.dtype != dt || Wd.dtype != dt || (R.ptr && R.dtype != dt) ||
      h.dtype != dt || y.dtype != dt)
    return AAL_ERR_UNSUPPORTED;
  const long long B = x.rows, D = x.cols, E = Wr.cols, F = Wg.cols;
  if (top_k < 1 || E < 1 || top_k > E) return AAL_ERR_INVALID_ARG;
  if (Wr.rows != D || Wg.rows != E * D || Wu.rows != E * D || Wu.cols != F || Wd.rows != E * F || Wd.cols != D ||
      (R.ptr && (R.rows != B || R.cols != D)) || h.rows != B * top_k || h.cols != F || y.rows != B || y.cols != D)
    return AAL_ERR_INVALID_ARG;
  if (D % q || F % q) return AAL_ERR_INVALID_ARG;
  if (((uintptr_t)positions % 8) || ((uintptr_t)ids % 4) || ((uintptr_t)weights % 4)) return AAL_ERR_INVALID_ARG;
  if (B > 0 && (!positions || !ids || !weights)) return AAL_ERR_INVALID_ARG;
  if (top_k > moe::kMaxTopK || E > moe::kMaxExperts || D > INT_MAX || F > INT_MAX) return AAL_ERR_UNSUPPORTED;
  note_path(0);
  if (B == 0 || D == 0 || F == 0) return AAL_OK;
  cudaStream_t s = (cudaStream_t)stream;
  const bool fast = t_policy != AAL_PATH_GENERAL && dt == AAL_BF16 && q <= moe::kMaxQ && (D / q) % 16 == 0 &&
                    (F / q) % 16 == 0 && moe::vec16(x) && moe::vec16(Wg) && moe::vec16(Wu) && moe::vec16(Wd) &&
                    moe::vec16(h);
  if (!fast && t_policy == AAL_PATH_TENSOR) return AAL_ERR_UNSUPPORTED;
  const size_t es = dt == AAL_F32 ? 4 : 2;
  const bool rvec = moe::vec16(Wr) && (E * es) % 16 == 0;
  auto at = [&](const aal_mat& m, long long row) { return m.ptr ? (char*)m.ptr + row * m.ld * es : nullptr; };
  aal_status st = AAL_OK;
  for (long long b0 = 0; b0 < B && st == AAL_OK; b0 += moe::kChunk) {
    const int nb = (int)(B - b0 < moe::kChunk ? B - b0 : moe::kChunk);
    int* id = ids + b0 * top_k;
    float* wt = weights + b0 * top_k;
    moe::RouterArgs ra = {at(x, b0), Wr.ptr, positions + b0, id, wt, x.ld, Wr.ld, nb, (int)D, (int)E, top_k,
                          renormalize != 0};
    st = timed(AAL_KERNEL_MOE_ROUTER, s, [&] {
      if (dt == AAL_F32)
        return rvec ? moe::run_router_tb<float, 4>(ra, s) : moe::run_router_tb<float, 1>(ra, s);
      return rvec ? moe::run_router_tb<__nv_bfloat16, 8>(ra, s) : moe::run_router_tb<__nv_bfloat16, 1>(ra, s);
    });
    if (st != AAL_OK) return st;
    if (fast) {
      using bf = __nv_bfloat16;
      moe::ExpertArgs a = {positions + b0, id, wt, (const bf*)at(x, b0), (const bf*)Wg.ptr, (const bf*)Wu.ptr,
                           (const bf*)Wd.ptr, (const bf*)at(R, b0), (bf*)at(h, b0 * top_k), (bf*)at(y, b0), x.ld, Wg.ld,
                           Wu.ld, Wd.ld, h.ld, R.ld, y.ld, law, q, nb, top_k, (int)E, (int)D, (int)F, 0,
                           (int)(nb * top_k < E ? nb * top_k : E), 0};
      st = nb <= 8 ? moe::run_experts<1>(a, s) : moe::run_experts<2>(a, s);
    } else {
      aal_mat xs = x, Rs = R, hs = h, ys = y;
      xs.ptr = at(x, b0);
      Rs.ptr = at(R, b0);
      hs.ptr = at(h, b0 * top_k);
      ys.ptr = at(y, b0);
      st = dt == AAL_F32 ? moe::run_general<float>(law, q, positions + b0, xs, Wg, Wu, Wd, Rs, id, wt, top_k, hs, ys,
                                                   nb, (int)D, (int)F, s)
                         : moe::run_general<__nv_bfloat16>(law, q, positions + b0, xs, Wg, Wu, Wd, Rs, id, wt, top_k,
                                                           hs, ys, nb, (int)D, (int)F, s);
    }
  }
  if (st == AAL_OK) note_path(fast ? AAL_PATH_DECODE : AAL_PATH_GENERAL);
  return st;
}
