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
//   k_moe_router   a cluster an entry (or two): logits, top-k, weights
//   k_moe_up       gate, up and SiLU of one expert's 64 columns a piece
//   k_moe_down     64 columns of y a cluster, its warps dealing the experts out
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
constexpr int kChunk = 128;   // entries of one chain of launches,
constexpr int kSlots = 1024;  // and choices: what a CTA's tables hold beside its ring for 2048 experts

// ------------------------------------------------------------------- router
// A cluster of kRouterCtas CTAs takes TB entries: CTA r the input rows of
// slice r, a thread VEC adjacent experts on every RL-th row of it, all its
// weight loads in flight before the first product.  The logits are sums of
// exact products in fp64 (an expert chosen or not by a rounding would change
// the whole row), added over the row lanes and the CTAs in a fixed order; CTA
// b of the cluster then ranks entry b's.
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

// Unsigned keys in the order of the doubles; NaN lowest, -0 as +0.
__device__ __forceinline__ unsigned long long order_key(double v) {
  if (isnan(v)) return 0ull;
  const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

// Writes the entry's k choices: the experts of the k largest logits l[0..E),
// ties to the lower index, NaN last, and their softmax weights.  Up to
// kCountExperts an expert's place is the number of experts before it, counted
// by 256 / E threads each; beyond that a warp picks the largest k times (a
// step of one entry and 128 experts 17.9 us counted, 19.7 picked; the router
// of 1024 experts 82 counted, 36 picked).
constexpr int kCountExperts = 512;
__device__ __forceinline__ void write_weights(const double* l, const double* top, int E, int k, int renorm, bool nan,
                                              float* wts) {
  const int lane = threadIdx.x & 31;
  const double mx = top[0];
  const float p = lane < k ? expf((float)(top[lane] - mx)) : 0.f;
  float sum = p;
  if (!renorm) {  // the softmax over every logit
    sum = 0.f;
    for (int e = lane; e < E; e += 32) sum += expf((float)(l[e] - mx));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < k) wts[lane] = nan ? NAN : p / sum;
}
__device__ void rank_logits(const double* l, unsigned long long* key, double* top, int E, int k, int renorm, int* ids,
                            float* wts) {
  const int tid = threadIdx.x, lane = tid & 31;
  bool nan = false;
  for (int e = tid; e < E; e += kRouterThreads) {
    nan |= isnan(l[e]);
    key[e] = order_key(l[e]);
  }
  nan = __syncthreads_or(nan);
  if (E <= kCountExperts) {
    int per = 1;  // threads an expert, neighbours in a warp
    while (per < 32 && E * per * 2 <= kRouterThreads) per *= 2;
    for (int e0 = 0; e0 < E; e0 += kRouterThreads / per) {  // the whole CTA, for the shuffles
      const int e = e0 + tid / per;
      const unsigned long long mine = e < E ? key[e] : 0ull;
      int before = 0;
#pragma unroll 8
      for (int j = tid % per; j < E; j += per) {
        const unsigned long long other = key[j];
        before += other > mine || (other == mine && j < e);
      }
      for (int o = per >> 1; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
      if (e < E && tid % per == 0 && before < k) {
        ids[before] = e;
        top[before] = l[e];
      }
    }
  } else if (tid < 32) {
    // the lane's best of the experts lane, lane + 32, ... not yet taken
    unsigned long long taken = 0;  // bit i: expert lane + 32 i (kMaxExperts fit)
    unsigned long long best = 0;
    int at = INT_MAX;
    auto scan = [&] {
      best = 0;
      at = INT_MAX;
      for (int e = lane, i = 0; e < E; e += 32, ++i) {
        if ((taken >> i) & 1ull) continue;
        if (at == INT_MAX || key[e] > best) { best = key[e]; at = e; }
      }
    };
    scan();
    for (int j = 0; j < k; ++j) {
      // the largest key, then the lowest expert that has it
      const unsigned hi = __reduce_max_sync(0xffffffffu, (unsigned)(best >> 32));
      const bool in_hi = (unsigned)(best >> 32) == hi;
      const unsigned lo = __reduce_max_sync(0xffffffffu, in_hi ? (unsigned)best : 0u);
      const int e = (int)__reduce_min_sync(0xffffffffu, in_hi && (unsigned)best == lo ? (unsigned)at : 0x7fffffffu);
      if (lane == 0) {
        ids[j] = e;
        top[j] = l[e];
      }
      if ((e & 31) == lane) {
        taken |= 1ull << (e >> 5);
        scan();
      }
    }
  }
  __syncthreads();
  if (tid < 32) write_weights(l, top, E, k, renorm, nan, wts);
}

template <typename T, int VEC, int TB>
__global__ void __cluster_dims__(kRouterCtas, 1, 1) __launch_bounds__(kRouterThreads) k_moe_router(const RouterArgs a) {
  constexpr int U = 16;  // weight loads in flight
  extern __shared__ double sm[];
  __shared__ double top[kMaxTopK];
  double* part = sm;                                 // [TB][E] this CTA's sums
  double* red = part + (size_t)TB * a.E;             // [TB][VEC][threads]
  double* xs = red + (size_t)TB * VEC * kRouterThreads;  // [slice][TB]
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tid = threadIdx.x;
  pdl_release();
  pdl_wait();
  const int b0 = (int)(blockIdx.x / kRouterCtas) * TB;
  const int nb = min(TB, a.B - b0);
  const int ds = (a.D + kRouterCtas - 1) / kRouterCtas;
  const int d0 = min(a.D, rank * ds), nd = min(a.D, d0 + ds) - d0;
  const int ncv = (a.E + VEC - 1) / VEC;
  int cvb = 1;  // column vectors a pass
  while (cvb < ncv && cvb < kRouterThreads) cvb <<= 1;
  const int rl = kRouterThreads / cvb;  // row lanes
  const T *x = (const T*)a.x, *wr = (const T*)a.wr + (long long)d0 * a.ldr;
  for (int c0 = 0; c0 < ncv; c0 += cvb) {
    const int cv = c0 + tid % cvb, lane_r = tid / cvb;
    const bool on = cv < ncv;
    double acc[TB][VEC];
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[b][j] = 0.0;
    for (int r0 = lane_r; r0 < nd || r0 == lane_r; r0 += U * rl) {
      T w[U][VEC];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int r = r0 + i * rl;
        if constexpr (VEC == 1) {
          w[i][0] = on && r < nd ? wr[(long long)r * a.ldr + cv] : T(0.f);
        } else {
          uint4 u = make_uint4(0, 0, 0, 0);
          if (on && r < nd) u = __ldg(reinterpret_cast<const uint4*>(wr + (long long)r * a.ldr + (long long)cv * VEC));
          memcpy(w[i], &u, 16);
        }
      }
      if (c0 == 0 && r0 == lane_r) {
        // the entries' inputs, widened once, while the first weights are on their way
#pragma unroll
        for (int b = 0; b < TB; ++b)
          for (int r = tid; r < nd; r += kRouterThreads)
            xs[(size_t)r * TB + b] = b < nb ? widen(x[(long long)(b0 + b) * a.ldx + d0 + r]) : 0.0;
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int r = r0 + i * rl;
        if (r >= nd) break;
        double xv[TB];
#pragma unroll
        for (int b = 0; b < TB; ++b) xv[b] = xs[(size_t)r * TB + b];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const double wv = widen(w[i][j]);
#pragma unroll
          for (int b = 0; b < TB; ++b) acc[b][j] = fma(wv, xv[b], acc[b][j]);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int j = 0; j < VEC; ++j) red[(size_t)(b * VEC + j) * kRouterThreads + tid] = acc[b][j];
    __syncthreads();
    for (int i = tid; i < TB * VEC * cvb; i += kRouterThreads) {
      const int bj = i / cvb, c = i - bj * cvb, e = (c0 + c) * VEC + bj % VEC;
      if (e < a.E) {
        double s = 0.0;
#pragma unroll 8
        for (int l = 0; l < rl; ++l) s += red[(size_t)bj * kRouterThreads + l * cvb + c];
        part[(size_t)(bj / VEC) * a.E + e] = s;
      }
    }
    __syncthreads();
  }
  cl.sync();
  double* logit = red;        // this CTA's entry
  unsigned long long* key = reinterpret_cast<unsigned long long*>(red + a.E);
  if (rank < nb) {
    for (int e = tid; e < a.E; e += kRouterThreads) {
      double s = 0.0;
#pragma unroll
      for (int r = 0; r < kRouterCtas; ++r) s += cl.map_shared_rank(part, r)[(size_t)rank * a.E + e];
      logit[e] = s;
    }
  }
  cl.barrier_arrive();  // the peers' sums have been read
  if (rank < nb) {
    const int b = b0 + rank;
    int* ids = a.ids + (long long)b * a.k;
    float* wts = a.weights + (long long)b * a.k;
    if (a.positions[b] < 0) {  // skipped: no expert, no output row
      if (tid == 0) flag_device_error(kDevBounds);
      if (tid < a.k) {
        ids[tid] = -1;
        wts[tid] = 0.f;
      }
    } else {
      __syncthreads();
      rank_logits(logit, key, top, a.E, a.k, a.renorm, ids, wts);
    }
  }
  cl.barrier_wait();
}

// ------------------------------------------------- experts, tensor-core path
// A warp multiplies 64 weight columns by up to 8 NT entries with
// mma.sync.m16n8k16: M = the columns, N = the entries, K = weight rows, 16 a
// step.  The order of K inside a step is free as long as both operands agree,
// so lane (g, t) = (lane / 4, lane % 4) multiplies rows 4t..4t+3 of the step
// and columns 8g..8g+7: one 16-byte word a row, and the fragments of the four
// 16-column tiles are byte permutes of those words (tile i holds columns
// 8g + 2i and 8g + 2i + 1).  The step's 16 rows of 128 bytes come in with
// cp.async, eight lanes a row (lanes spread over four rows asked L2 for twice
// the sectors), at a chunk position xored with 2t so that the four rows a
// quarter warp reads together fall into different banks.  A warp's ring of
// steps is its own: it takes no CTA barrier and runs on from one piece of work
// (an expert's tile) to the next, so the next piece is in flight while the CTA
// adds up this one.
constexpr int kTile = 64;   // output columns of a CTA's tile
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxQ = 32;   // groups of a table row fit one word

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Copies of 16 bytes (past L1: weights are read once) and of 8 bytes; with
// ``bytes`` 0 they fill zeros and read nothing.
__device__ __forceinline__ void copy(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct ExpertArgs {
  const int64_t* positions;
  const int* ids;
  const float* weights;
  const __nv_bfloat16 *x, *wg, *wu, *wd, *r;
  __nv_bfloat16 *h, *y;
  long long ldx, ldg, ldu, ldd, ldh, ldr, ldy;
  int law, q, B, k, E, D, F;
  int passes;        // upper bound of the number of passes
  int zsplit;        // k_moe_up: CTAs of a cluster
  int tiles, ntile;  // column tiles of an output group, and of all groups
  tc::FastDiv by_tiles, by_ntile, by_k;
};

// Up to 8 NT entries of one expert; ``types``: the row types of all of the
// expert's entries, one bit each.
struct Pass {
  int expert, first, n;
  unsigned types;
};

// What a CTA knows of the step, in dynamic shared memory.
struct Tables {
  Pass* pass;      // [passes]
  int* first;      // [E] place of the expert's first entry in ``slot``
  unsigned* tmask; // [E] row types of its entries
  unsigned* who;   // [E][words] its entries, one bit each
  int* id;         // [B k] the router's choices
  float* weight;   // [B k] and their weights
  int* slot;       // [B k] choices by expert, then by entry
  int* entry;      // [B k] and their entries
  int* type;       // [B]
  int words;
  __host__ __device__ static size_t bytes(int passes, int E, int B, int k) {
    const size_t words = (B + 31) / 32;
    return (sizeof(Pass) * passes + sizeof(int) * ((2 + words) * E + 4 * (size_t)B * k + B) + 15) / 16 * 16;
  }
  __device__ explicit Tables(unsigned char* p, const ExpertArgs& a) {
    words = (a.B + 31) / 32;
    pass = reinterpret_cast<Pass*>(p);
    first = reinterpret_cast<int*>(pass + a.passes);
    tmask = reinterpret_cast<unsigned*>(first + a.E);
    who = tmask + a.E;
    id = reinterpret_cast<int*>(who + a.E * words);
    weight = reinterpret_cast<float*>(id + a.B * a.k);
    slot = reinterpret_cast<int*>(weight + a.B * a.k);
    entry = slot + a.B * a.k;
    type = entry + a.B * a.k;
  }
};

// Sorts the choices by expert and entry and cuts every expert's entries into
// passes of up to ``width``; returns the number of passes (every thread).  All
// CTAs of a launch come to the same order: an entry chooses an expert at most
// once, so a bit a (expert, entry) holds the choices whatever the order of
// the atomics, and an entry's place is the number of bits below its own.
__device__ __forceinline__ int build_tables(const ExpertArgs& a, const Tables& tb, int width) {
  __shared__ int s_passes;
  const int n = a.B * a.k, W = tb.words;
  for (int s = threadIdx.x; s < n; s += blockDim.x) {
    const int e = __ldcg(a.ids + s);
    const float w = __ldcg(a.weights + s);
    tb.id[s] = e < a.E ? e : -1;
    tb.weight[s] = w;
  }
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const long long pos = __ldcg((const long long*)a.positions + b);
    tb.type[b] = pos < 0 ? 0 : (int)(pos % a.q);
  }
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) tb.tmask[e] = 0u;
  for (int i = threadIdx.x; i < a.E * W; i += blockDim.x) tb.who[i] = 0u;
  __syncthreads();
  for (int s = threadIdx.x; s < n; s += blockDim.x) {
    const int e = tb.id[s], b = (int)tc::fdiv((uint32_t)s, a.by_k);
    if (e >= 0) {
      atomicOr(&tb.who[e * W + (b >> 5)], 1u << (b & 31));
      atomicOr(&tb.tmask[e], 1u << (tb.type[b] & 31));  // (read where q <= 32)
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int base = 0, np = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + (int)threadIdx.x;
      int c = 0;
      if (e < a.E)
        for (int w = 0; w < W; ++w) c += __popc(tb.who[e * W + w]);
      const int p = (c + width - 1) / width;
      int ci = c, pi = p;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, ci, o), v = __shfl_up_sync(0xffffffffu, pi, o);
        if ((int)threadIdx.x >= o) {
          ci += u;
          pi += v;
        }
      }
      const int first = base + ci - c;
      for (int j = 0; j < p; ++j) {
        const int done = j * width;
        tb.pass[np + pi - p + j] = Pass{e, first + done, min(width, c - done), tb.tmask[e]};
      }
      if (e < a.E) tb.first[e] = first;
      base += __shfl_sync(0xffffffffu, ci, 31);
      np += __shfl_sync(0xffffffffu, pi, 31);
    }
    if (threadIdx.x == 0) s_passes = np;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < n; s += blockDim.x) {
    const int e = tb.id[s], b = (int)tc::fdiv((uint32_t)s, a.by_k);
    if (e < 0) continue;
    int at = tb.first[e] + __popc(tb.who[e * W + (b >> 5)] & ((1u << (b & 31)) - 1u));
    for (int w = 0; w < (b >> 5); ++w) at += __popc(tb.who[e * W + w]);
    tb.slot[at] = s;
    tb.entry[at] = b;
  }
  __syncthreads();
  return s_passes;
}

// The input groups that output group kg needs for entries of the given types.
__device__ __forceinline__ unsigned groups_of(int law, int q, unsigned types, int kg) {
  if (law == AAL_LAW_Q) return types | (1u << kg);
  unsigned m = 0;
  for (int t = 0; t < 4; ++t)
    if ((types >> t) & 1u)
      for (int g = 0; g < 4; ++g)
        if (in_table(law, t, kg, g)) m |= 1u << g;
  return m;
}

// A warp's walk over the K steps of one piece: steps first, first + stride,
// ... of the used groups in ascending order.  Inside a group a step is a
// constant distance from the one before.
template <int NT>
struct Walk {
  const __nv_bfloat16* w;      // row lane / 8, column chunk lane % 8 of K step 0
  const __nv_bfloat16* x[NT];  // input rows of entries nt * 8 + g from element 4t on
  bool have[NT];               // the entry exists
  int type[NT];
  long long ldw;
  unsigned left;               // used groups from the current one on (0: the walk is over)
  int in, spg, stride, kg;
  int wsize;                   // bytes copied per word: 16, or 0 past the tile's width
  // the current step
  const __nv_bfloat16* at;
  int k;
  int xsize[NT];
  // Moves to the group that step ``in`` falls into.
  __device__ __forceinline__ void settle(int law) {
    while (in >= spg && left) {
      in -= spg;
      left &= left - 1u;
    }
    if (!left) return;
    const int grp = __ffs(left) - 1;
    k = (grp * spg + in) * 16;
    at = w + (long long)k * ldw;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xsize[nt] = have[nt] && in_table(law, type[nt], kg, grp) ? 8 : 0;
  }
  __device__ __forceinline__ void start(int law, unsigned groups, int first) {
    left = groups;
    in = first;
    settle(law);
  }
  __device__ __forceinline__ void next(int law) {
    in += stride;
    if (in < spg) {
      k += stride * 16;
      at += (long long)(stride * 16) * ldw;
    } else {
      settle(law);
    }
  }
};
// Number of steps such a walk takes.
__device__ __forceinline__ int walk_steps(unsigned groups, int spg, int first, int stride) {
  const int total = __popc(groups) * spg;
  return first < total ? (total - first + stride - 1) / stride : 0;
}

template <int NT, int S>
struct Ring {
  static constexpr uint32_t kStep = 2048 + 256 * NT;  // bytes of one step
  uint32_t put, get;   // this lane's places in slot 0: words copied, words read
  uint32_t xpos;       // the entries' 8 bytes, copied and read by the same lane
  uint32_t head = 0;   // slot the next step goes to (bytes)
  uint32_t tail = 0;   // slot the next product reads (bytes)
  __device__ Ring(unsigned char* mem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t p = tc::smem_u32(mem) + warp * S * kStep;
    const int g = lane >> 2, t = lane & 3;
    put = p + (lane >> 3) * 128;  // row lane / 8 of each four; the chunk's xor depends on the row
    get = p + t * 512 + ((g ^ (2 * t)) << 4);
    xpos = p + 2048 + lane * 8;
  }
  // Issues the copies of the walk's step: its weights, and its entries'
  // inputs.
  __device__ __forceinline__ void issue_weights(const Walk<NT>& k) {
    const uint32_t chunk = threadIdx.x & 7, d = put + head;
    const __nv_bfloat16* w = k.at;
    const long long four = 4 * k.ldw;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // rows 4i .. 4i + 3
      copy(d + i * 512 + ((chunk ^ (2 * i)) << 4), w, k.wsize);
      w += four;
    }
  }
  __device__ __forceinline__ void issue_inputs(const Walk<NT>& k) {
    const uint32_t dx = xpos + head;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) copy8(dx + nt * 256, k.x[nt] + k.k, k.xsize[nt]);
  }
  __device__ __forceinline__ void advance() { head = head + kStep == S * kStep ? 0 : head + kStep; }
  // The products of the oldest step.
  __device__ __forceinline__ void multiply(float (&acc)[4][NT][4]) {
    const uint32_t s = get + tail, sx = xpos + tail;
    uint4 v[4];
    uint32_t b[NT][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                   : "r"(s + i * 128)
                   : "memory");
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(b[nt][0]), "=r"(b[nt][1]) : "r"(sx + nt * 256) : "memory");
    const uint32_t w0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, w1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
    const uint32_t w2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, w3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a0 = __byte_perm(w0[i], w1[i], 0x5410), a1 = __byte_perm(w0[i], w1[i], 0x7632);
      const uint32_t a2 = __byte_perm(w2[i], w3[i], 0x5410), a3 = __byte_perm(w2[i], w3[i], 0x7632);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma16816(acc[i][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
    }
    tail = tail + kStep == S * kStep ? 0 : tail + kStep;
  }
};

// A warp's sums of up to 8 NT entries by 64 columns in shared memory.  Even
// entries come first and rows are 66 floats apart, so the fragments' stores
// meet no bank twice.
template <int NT>
struct Sums {
  static constexpr int kRow = kTile + 2, kFloats = 8 * NT * kRow;
  __device__ static __forceinline__ int at(int entry, int col) {
    return ((entry >> 1) + (entry & 1) * 4 * NT) * kRow + col;
  }
  __device__ static __forceinline__ void put(float* red, const float (&acc)[4][NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = nt * 8 + 2 * t, c = 8 * g + 2 * i;
        *reinterpret_cast<float2*>(red + at(n, c)) = make_float2(acc[i][nt][0], acc[i][nt][2]);
        *reinterpret_cast<float2*>(red + at(n + 1, c)) = make_float2(acc[i][nt][1], acc[i][nt][3]);
      }
  }
};

// The loop both expert kernels share: ``open(i, walk)`` describes the warp's
// piece i, ``steps(i)`` is its number of steps, and ``close(i, sums)`` takes its
// products.  ``ready`` is called once, before the first input is read and after
// the first steps' weights are on their way.
template <int NT, int S, typename Open, typename Steps, typename Close, typename Ready>
__device__ __forceinline__ void run_pieces(unsigned char* ring_mem, int law, int pieces, Open open, Steps steps,
                                           Close close, Ready ready) {
  Ring<NT, S> ring(ring_mem);
  Walk<NT> walk;
  walk.left = 0;
  int ahead = 0;  // next piece to open
  auto produce_weights = [&] {
    while (!walk.left && ahead < pieces) open(ahead++, walk);
    if (walk.left) {
      ring.issue_weights(walk);
      ring.advance();
      walk.next(law);
    }
  };
  for (int i = 0; i < S - 1; ++i) produce_weights();
  ready();
  // the same steps again, for their inputs
  walk.left = 0;
  ahead = 0;
  ring.head = 0;
  auto produce = [&](bool weights) {
    while (!walk.left && ahead < pieces) open(ahead++, walk);
    if (walk.left) {
      if (weights) ring.issue_weights(walk);
      ring.issue_inputs(walk);
      ring.advance();
      walk.next(law);
    }
    copy_commit();  // empty once the work has run out, so that the waits still count
  };
  for (int i = 0; i < S - 1; ++i) produce(false);
  for (int i = 0; i < pieces; ++i) {
    float acc[4][NT][4] = {};
    for (int n = steps(i); n > 0; --n) {
      copy_wait<S - 2>();  // the oldest step's copies of this lane have landed,
      __syncwarp();        // and so have the others'; nor does any still read the slot before it
      ring.multiply(acc);
      produce(true);       // into the slot read in the round before
    }
    close(i, acc);
  }
  copy_wait<0>();
}

// h of the passes' 64-column tiles.  A piece is (pass, tile); warps 0-3 stream
// the gate's weights, warps 4-7 the up projection's, every fourth step each.
// Where the pieces leave SMs without one, a cluster of zsplit CTAs takes each:
// they split K further and add their parts in rank order through distributed
// shared memory.
// Measured with 768 columns of 2048 rows: 8 entries of 128 experts, dense, 63
// us for 325 MB (5.1 TB/s: the copies in flight, less the start and the last
// pieces); 64 entries under Q_16 60 us for 217 MB (3.6 TB/s: of every row 96
// bytes are used and DRAM delivers 128, and a piece is four K steps a warp).
template <int NT, int S>
__global__ void __launch_bounds__(kThreads, 2) k_moe_up(const ExpertArgs a) {
  extern __shared__ __align__(128) unsigned char mem[];
  constexpr int kRed = Sums<NT>::kFloats;
  unsigned char* ring_mem = mem;
  float* red = reinterpret_cast<float*>(mem + kWarps * S * Ring<NT, S>::kStep);
  const Tables tb(reinterpret_cast<unsigned char*>(red + kWarps * kRed), a);
  cg::cluster_group cl = cg::this_cluster();
  const int z = a.zsplit, rank = (int)(blockIdx.x % z);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_release();
  const int np = build_tables(a, tb, 8 * NT);
  const int bi = a.D / a.q, bo = a.F / a.q, spg = bi >> 4;
  const int total = np * a.ntile;
  const int team = (int)(blockIdx.x / z), teams = (int)(gridDim.x / z);
  const int pieces = team < total ? (total - team + teams - 1) / teams : 0;
  // piece i: its pass, output group and first column
  auto piece = [&](int i, int& kg, int& c0) {
    const int id = team + i * teams;
    const int p = (int)tc::fdiv((uint32_t)id, a.by_ntile), tile = id - p * a.ntile;
    kg = (int)tc::fdiv((uint32_t)tile, a.by_tiles);
    c0 = kg * bo + (tile - kg * a.tiles) * kTile;
    return p;
  };
  const int first = rank * 4 + (warp & 3), stride = 4 * z;
  const long long ldw = warp >= 4 ? a.ldu : a.ldg;
  const __nv_bfloat16* wbase = (warp >= 4 ? a.wu : a.wg) + (long long)(lane >> 3) * ldw;
  auto open = [&](int i, Walk<NT>& w) {
    int kg, c0;
    const Pass p = tb.pass[piece(i, kg, c0)];
    const int col = 8 * (lane & 7);
    const bool wide = col < (kg + 1) * bo - c0;
    w.wsize = wide ? 16 : 0;
    w.ldw = ldw;
    w.w = wbase + (long long)p.expert * a.D * ldw + c0 + (wide ? col : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = nt * 8 + (lane >> 2);
      w.have[nt] = n < p.n;
      const int b = tb.entry[p.first + (n < p.n ? n : 0)];
      w.x[nt] = a.x + (long long)b * a.ldx + 4 * (lane & 3);
      w.type[nt] = tb.type[b];
    }
    w.spg = spg;
    w.stride = stride;
    w.kg = kg;
    w.start(a.law, groups_of(a.law, a.q, p.types, kg), first);
  };
  auto steps = [&](int i) {
    int kg, c0;
    const int p = piece(i, kg, c0);
    return walk_steps(groups_of(a.law, a.q, tb.pass[p].types, kg), spg, first, stride);
  };
  auto close = [&](int i, const float (&acc)[4][NT][4]) {
    Sums<NT>::put(red + warp * kRed, acc);
    if (z > 1) cl.sync();
    else __syncthreads();
    int kg, c0;
    const Pass p = tb.pass[piece(i, kg, c0)];
    const int width = min(kTile, (kg + 1) * bo - c0);
    for (int j = threadIdx.x; j < p.n * kTile; j += kThreads) {
      const int m = j / kTile, c = j % kTile, o = Sums<NT>::at(m, c);
      if (c >= width || (z > 1 && m % z != rank)) continue;  // a cluster's CTAs finish every z-th entry
      float g = 0.f, u = 0.f;
      for (int v = 0; v < z; ++v) {
        const float* from = z > 1 ? cl.map_shared_rank(red, v) : red;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          g += from[w * kRed + o];
          u += from[(w + 4) * kRed + o];
        }
      }
      a.h[(long long)tb.slot[p.first + m] * a.ldh + c0 + c] = __float2bfloat16_rn(g / (1.f + expf(-g)) * u);
    }
    if (z > 1) cl.sync();
    else __syncthreads();
  };
  run_pieces<NT, S>(ring_mem, a.law, pieces, open, steps, close, [] {});
}

// 64 columns of y a cluster.  A unit of work is a pass, or one of its kparts
// interleaved parts along K where there are few; the cluster's warps take
// units in turn, each from first weight row to last on its own, and add the
// weighted products to their CTA's sums in shared memory one after another in
// unit order, so results do not depend on timing.  Then the cluster adds the CTAs' sums in rank order with the
// residual.  (With a unit to all of a CTA's warps, summed and handed over with
// barriers, 64 entries under Q_16 took 55 us: two K steps a warp and unit; now
// 39, and 37 for 8 entries of 128 dense experts, 162 MB.)
constexpr int kDownCtas = 8;
constexpr int kYRow = kTile + 2;  // floats between entries' sums

// The turn goes from warp w to warp w + 1 through named barrier w + 1 of the
// two.  (A flag in shared memory needs a fence, and a fence waits for the
// warp's copies in flight: 0.7 us a turn.)
__device__ __forceinline__ void take_turn(int warp) {
  asm volatile("barrier.cta.sync %0, 64;" ::"r"((warp + kWarps - 1) % kWarps + 1) : "memory");
}
__device__ __forceinline__ void pass_turn(int warp) {
  asm volatile("barrier.cta.arrive %0, 64;" ::"r"(warp + 1) : "memory");
}

// CL: CTAs of a cluster, 8, or 4 for little work, so that all of them find
// room beside k_moe_up's and have their weights when it ends.
template <int NT, int S, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(kThreads, 2) k_moe_down(const ExpertArgs a) {
  constexpr int kUnits = CL * kWarps;  // units the cluster's warps take at once
  extern __shared__ __align__(128) unsigned char mem[];
  float* ys = reinterpret_cast<float*>(mem + kWarps * S * Ring<NT, S>::kStep);  // [B][kYRow]
  const Tables tb(reinterpret_cast<unsigned char*>(ys + (a.B * kYRow + 3) / 4 * 4), a);
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tile = (int)(blockIdx.x / CL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < a.B * kYRow; i += kThreads) ys[i] = 0.f;
  const int bi = a.F / a.q, bo = a.D / a.q, spg = bi >> 4;
  const int kg = tile / a.tiles, c0 = kg * bo + (tile - kg * a.tiles) * kTile;
  const int width = min(kTile, (kg + 1) * bo - c0);
  // The router's results are complete here although this kernel has not waited
  // yet: it starts once every CTA of k_moe_up has released it, which each does
  // after its own wait for the router.  So the tables and the first weights
  // come in while k_moe_up still runs; only its h needs the wait.
  const int np = build_tables(a, tb, 8 * NT);
  // Parts a pass: the fewest K steps a warp takes, where adding a unit's
  // products costs about as much as a step.
  int kparts = 1;
  {
    const int steps = (a.q < 2 ? 1 : 2) * spg;
    int best = INT_MAX;
    for (int k = 1; k <= 16 && steps >= 2 * k; k *= 2) {
      const int c = (np * k + kUnits - 1) / kUnits * (steps + k) * (16 / k);
      if (c < best) {
        best = c;
        kparts = k;
      }
    }
  }
  const int shift = __ffs(kparts) - 1;
  // unit u = i * kUnits + warp * CL + rank
  const int units = np << shift, mine = warp * CL + rank;
  const int pieces = mine < units ? (units - mine + kUnits - 1) / kUnits : 0;
  const int col = 8 * (lane & 7);
  const bool wide = col < width;
  const __nv_bfloat16* wbase = a.wd + (long long)(lane >> 3) * a.ldd + c0 + (wide ? col : 0);
  auto open = [&](int i, Walk<NT>& w) {
    const int u = i * kUnits + mine;
    const Pass p = tb.pass[u >> shift];
    w.wsize = wide ? 16 : 0;
    w.ldw = a.ldd;
    w.w = wbase + (long long)p.expert * a.F * a.ldd;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = nt * 8 + (lane >> 2), at = p.first + (n < p.n ? n : 0);
      w.have[nt] = n < p.n;
      w.x[nt] = a.h + (long long)tb.slot[at] * a.ldh + 4 * (lane & 3);
      w.type[nt] = tb.type[tb.entry[at]];
    }
    w.spg = spg;
    w.stride = kparts;
    w.kg = kg;
    w.start(a.law, groups_of(a.law, a.q, p.types, kg), u & (kparts - 1));
  };
  auto steps = [&](int i) {
    const int u = i * kUnits + mine;
    return walk_steps(groups_of(a.law, a.q, tb.pass[u >> shift].types, kg), spg, u & (kparts - 1), kparts);
  };
  auto close = [&](int i, const float (&acc)[4][NT][4]) {
    const Pass p = tb.pass[(i * kUnits + mine) >> shift];
    const int g = lane >> 2, t = lane & 3;
    float* y[NT][2];
    float wt[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int n = nt * 8 + 2 * t + o, at = p.first + (n < p.n ? n : 0);
        wt[nt][o] = tb.weight[tb.slot[at]];
        y[nt][o] = ys + tb.entry[at] * kYRow + 8 * g;
      }
    if (i > 0 || warp > 0) take_turn(warp);
    // all loads before the stores: the sums' round trip is what the next warp waits for
    float2 v[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[nt][o][k] = *reinterpret_cast<const float2*>(y[nt][o] + 2 * k);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int o = 0; o < 2; ++o)
        if (nt * 8 + 2 * t + o < p.n) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<float2*>(y[nt][o] + 2 * k) =
                make_float2(fmaf(wt[nt][o], acc[k][nt][o], v[nt][o][k].x), fmaf(wt[nt][o], acc[k][nt][2 + o], v[nt][o][k].y));
        }
    // to the next unit of this CTA, if there is one
    if ((warp + 1 < kWarps ? i * kUnits + mine + CL : (i + 1) * kUnits + rank) < units) pass_turn(warp);
  };
  run_pieces<NT, S>(mem, a.law, pieces, open, steps, close, [] {
    pdl_wait();
    pdl_release();
  });
  cl.sync();
  // the cluster's CTAs finish the entries b mod CL == rank
  for (int i = threadIdx.x; i < a.B * kTile; i += kThreads) {
    const int b = i / kTile, c = i % kTile;
    if (b % CL != rank || c >= width || a.positions[b] < 0) continue;
    float s = a.r ? __bfloat162float(a.r[(long long)b * a.ldr + c0 + c]) : 0.f;
#pragma unroll
    for (int v = 0; v < CL; ++v) s += cl.map_shared_rank(ys, v)[b * kYRow + c];
    a.y[(long long)b * a.ldy + c0 + c] = __float2bfloat16_rn(s);
  }
  cl.sync();  // the peers' sums have been read
}

// ---------------------------------------------------------- experts, any shape
// fp32, and widths off the matrix instruction's grid.  The pieces of work are
// the same passes and tiles, 32 columns wide here: a lane takes VEC adjacent
// columns (16 bytes of an aligned row, else one) and multiplies every weight
// it loads with the pass's entries, whose inputs wait in shared memory, zeroed
// where an entry's table row does not use the group.  A CTA's warps deal the
// rows of the used groups out, kLoads loads a lane at a time so that as many
// are in flight, and meet in shared memory.  (24 loads of an element or 8 of a
// vector: exchanged, 5 fp32 entries of 8 experts at 768 x 1536 took 49.5 us a
// step against 36.8, and with fewer elements in flight odd bf16 rows 85.4
// against 83.0.)  Bound by instructions and the loads' latency: 32.7 us for
// those 5 entries, of whose 57 MB HBM would need 8.7; 27 entries of 64 bf16
// experts at 1113 x 979, element by element, 506 (57).
constexpr int kGenTile = 32, kGenEntries = 8, kGenRows = 512;

template <typename T>
struct GenArgs {
  ExpertArgs e;  // (its matrices are not used: those below have their type)
  const T *x, *wg, *wu, *wd, *r;
  T *h, *y;
  tc::FastDiv by_bi;
};

// The groups that output group kg needs for a pass's entries (at most
// kGenEntries + 1 under Q_q, 4 under Q2 x Q2); warp 0 lists them.
__device__ __forceinline__ int list_groups(const ExpertArgs& a, const Tables& tb, const Pass& p, int kg, int* list) {
  const int lane = threadIdx.x & 31;
  if (a.q <= 32) {  // from the expert's types, which may be more than the pass's
    const unsigned m = groups_of(a.law, a.q, p.types, kg);
    if ((m >> lane) & 1u) list[__popc(m & ((1u << lane) - 1u))] = lane;
    return __popc(m);
  }
  int n = 0;  // law Q_q: kg and the entries' types, each once
  if (lane == 0) list[0] = kg;
  n = 1;
  for (int i = 0; i < p.n; ++i) {
    const int t = tb.type[tb.entry[p.first + i]];
    bool seen = t == kg;
    for (int l = 0; l < i; ++l) seen |= tb.type[tb.entry[p.first + l]] == t;
    if (!seen) {
      if (lane == 0) list[n] = t;
      ++n;
    }
  }
  return n;
}

struct GenShared {
  float x[kGenRows][kGenEntries];
  int row[kGenRows];
  float part[kWarps][kGenEntries][kGenTile];
  int groups[32];
  int ngroups;
};

// This warp's products of one matrix (row 0 at ``w``, the lane's columns) with
// a pass's entries, in sh.part[warp].  The used groups' rows part / parts of
// the way through are dealt to ``warps`` warps, of which this is number ``wi``;
// ``in`` gives the input row of the choice at a place.
// NE: the most entries of the pass that are multiplied (the instructions are
// what bounds this path: 27 entries of 64 experts, about two a pass, took 567
// us a step with eight each).
template <typename T, int VEC, int NE, typename In>
__device__ __forceinline__ void gen_multiply_entries(const GenArgs<T>& g, const Tables& tb, GenShared& sh, const Pass& p, int kg,
                                             int bi, const T* w, long long ldw, bool on, int wi, int warps, int part,
                                             int parts, In in) {
  constexpr int kLoads = VEC == 1 ? 24 : 8;
  constexpr int kLanes = kGenTile / VEC, kSub = 32 / kLanes;  // lanes a row, rows a load instruction
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / kLanes;
  float acc[NE][VEC] = {};
  __syncthreads();  // the shared arrays are free
  if (warp == 0) {
    const int n = list_groups(g.e, tb, p, kg, sh.groups);
    if (lane == 0) sh.ngroups = n;
  }
  __syncthreads();
  const int total = sh.ngroups * bi;
  const int lo = (int)((long long)total * part / parts), hi = (int)((long long)total * (part + 1) / parts);
  for (int r0 = lo; r0 < hi; r0 += kGenRows) {
    const int n = min(kGenRows, hi - r0);
    for (int r = threadIdx.x; r < n; r += kThreads) {
      const int gi = (int)tc::fdiv((uint32_t)(r0 + r), g.by_bi);
      const int grp = sh.groups[gi], k = grp * bi + (r0 + r - gi * bi);
      sh.row[r] = k;
      float v[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int at = p.first + (i < p.n ? i : 0);
        v[i] = i < p.n && in_table(g.e.law, tb.type[tb.entry[at]], kg, grp) ? ld_elem(in(at) + k) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < NE; i += 2) *reinterpret_cast<float2*>(&sh.x[r][i]) = make_float2(v[i], v[i + 1]);
    }
    __syncthreads();
    for (int b = wi * kLoads * kSub; b < n; b += warps * kLoads * kSub) {
      float v[kLoads][VEC];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = b + j * kSub + sub;
        const T* src = w + (long long)sh.row[r < n ? r : 0] * ldw;
#pragma unroll
        for (int c = 0; c < VEC; ++c) v[j][c] = 0.f;
        if (on && r < n) {
          if constexpr (VEC == 1) {
            v[j][0] = ld_elem(src);
          } else {
            static_assert(sizeof(T) * VEC == 16, "a 16-byte vector");
            const float4 f = __ldg(reinterpret_cast<const float4*>(src));
            v[j][0] = f.x;
            v[j][1] = f.y;
            v[j][2] = f.z;
            v[j][3] = f.w;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = b + j * kSub + sub;
        const float* xr = sh.x[r < n ? r : 0];
        float xe[NE];
        if constexpr (NE == 2) {
          const float2 f = *reinterpret_cast<const float2*>(xr);
          xe[0] = f.x;
          xe[1] = f.y;
        } else {
#pragma unroll
          for (int i = 0; i < NE; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(xr + i);
            xe[i] = f.x;
            xe[i + 1] = f.y;
            xe[i + 2] = f.z;
            xe[i + 3] = f.w;
          }
        }
#pragma unroll
        for (int i = 0; i < NE; ++i)
#pragma unroll
          for (int c = 0; c < VEC; ++c) acc[i][c] = fmaf(v[j][c], xe[i], acc[i][c]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < NE; ++i)
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      float v = acc[i][c];
      for (int o = kLanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (sub == 0) sh.part[warp][i][lane * VEC + c] = v;
    }
  __syncthreads();
}

template <typename T, int VEC, typename In>
__device__ __forceinline__ void gen_multiply(const GenArgs<T>& g, const Tables& tb, GenShared& sh, const Pass& p, int kg,
                                             int bi, const T* w, long long ldw, bool on, int wi, int warps, int part,
                                             int parts, In in) {
  if (p.n <= 2) gen_multiply_entries<T, VEC, 2>(g, tb, sh, p, kg, bi, w, ldw, on, wi, warps, part, parts, in);
  else if (p.n <= 4) gen_multiply_entries<T, VEC, 4>(g, tb, sh, p, kg, bi, w, ldw, on, wi, warps, part, parts, in);
  else gen_multiply_entries<T, VEC, kGenEntries>(g, tb, sh, p, kg, bi, w, ldw, on, wi, warps, part, parts, in);
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 2) k_moe_up_general(const GenArgs<T> g) {
  extern __shared__ __align__(128) unsigned char mem[];
  __shared__ __align__(16) GenShared sh;
  const ExpertArgs& a = g.e;
  const Tables tb(mem, a);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_release();
  const int np = build_tables(a, tb, kGenEntries);
  const int bi = a.D / a.q, bo = a.F / a.q;
  const int total = np * a.ntile;
  const bool up = warp >= kWarps / 2;
  const long long ldw = up ? a.ldu : a.ldg;
  for (int id = blockIdx.x; id < total; id += gridDim.x) {
    const int pi = (int)tc::fdiv((uint32_t)id, a.by_ntile), tile = id - pi * a.ntile;
    const Pass p = tb.pass[pi];
    const int kg = (int)tc::fdiv((uint32_t)tile, a.by_tiles);
    const int in_group = (tile - kg * a.tiles) * kGenTile, col = lane % (kGenTile / VEC) * VEC;
    const bool on = in_group + col < bo;
    const T* w = (up ? g.wu : g.wg) + (long long)p.expert * a.D * ldw + kg * bo + in_group + (on ? col : 0);
    gen_multiply<T, VEC>(g, tb, sh, p, kg, bi, w, ldw, on, warp % (kWarps / 2), kWarps / 2, 0, 1,
                         [&](int at) { return g.x + (long long)tb.entry[at] * a.ldx; });
    // warp i finishes entry i
    if (warp < p.n && in_group + lane < bo) {
      float gs = 0.f, us = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps / 2; ++v) {
        gs += sh.part[v][warp][lane];
        us += sh.part[v + kWarps / 2][warp][lane];
      }
      st_elem(g.h + (long long)tb.slot[p.first + warp] * a.ldh + kg * bo + in_group + lane, gs / (1.f + expf(-gs)) * us);
    }
  }
}

// 32 columns of y a cluster, as in k_moe_down: its CTAs take the passes in
// turn, or split the rows of each where there are fewer passes than CTAs.
template <typename T, int VEC>
__global__ void __cluster_dims__(kDownCtas, 1, 1) __launch_bounds__(kThreads, 2) k_moe_down_general(const GenArgs<T> g) {
  extern __shared__ __align__(128) unsigned char mem[];
  __shared__ __align__(16) GenShared sh;
  const ExpertArgs& a = g.e;
  float* ys = reinterpret_cast<float*>(mem);  // [B][32]
  const Tables tb(mem + (size_t)a.B * kGenTile * sizeof(float), a);
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tile = (int)(blockIdx.x / kDownCtas);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < a.B * kGenTile; i += kThreads) ys[i] = 0.f;
  const int bi = a.F / a.q, bo = a.D / a.q;
  const int kg = tile / a.tiles, in_group = (tile - kg * a.tiles) * kGenTile, col = lane % (kGenTile / VEC) * VEC;
  const bool on = in_group + col < bo;
  // (k_moe_up_general has waited for the router before it lets this kernel start)
  const int np = build_tables(a, tb, kGenEntries);
  pdl_wait();
  pdl_release();
  // the passes past the last full round are split along their rows, z ways
  const int whole = np / kDownCtas, left = np - whole * kDownCtas;
  const int z = left > 4 ? 1 : left > 2 ? 2 : left == 2 ? 4 : 8;
  for (int i = 0; i < whole + (rank / z < left ? 1 : 0); ++i) {
    const bool split = i >= whole;
    const Pass p = tb.pass[split ? whole * kDownCtas + rank / z : i * kDownCtas + rank];
    const T* w = g.wd + (long long)p.expert * a.F * a.ldd + kg * bo + in_group + (on ? col : 0);
    gen_multiply<T, VEC>(g, tb, sh, p, kg, bi, w, a.ldd, on, warp, kWarps, split ? rank % z : 0, split ? z : 1,
                         [&](int at) { return g.h + (long long)tb.slot[at] * a.ldh; });
    if (warp < p.n) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) s += sh.part[v][warp][lane];
      const int at = p.first + warp;
      ys[tb.entry[at] * kGenTile + lane] += tb.weight[tb.slot[at]] * s;
    }
  }
  cl.sync();
  for (int i = threadIdx.x; i < a.B * kGenTile; i += kThreads) {
    const int b = i / kGenTile, l = i % kGenTile;
    if (b % kDownCtas != rank || in_group + l >= bo || a.positions[b] < 0) continue;
    const long long c = kg * bo + in_group + l;
    float s = g.r ? ld_elem(g.r + (long long)b * a.ldr + c) : 0.f;
#pragma unroll
    for (int v = 0; v < kDownCtas; ++v) s += cl.map_shared_rank(ys, v)[i];
    st_elem(g.y + (long long)b * a.ldy + c, s);
  }
  cl.sync();  // the peers' sums have been read
}

// ------------------------------------------------------------------ launches
using norm::launch_pdl;

template <typename T, int VEC, int TB>
static aal_status run_router(const RouterArgs& a, cudaStream_t s) {
  const size_t ds = (a.D + kRouterCtas - 1) / kRouterCtas;
  // an entry's logits and their keys take the place of the products afterwards
  size_t red = (size_t)TB * VEC * kRouterThreads + TB * ds;
  if (red < 2 * (size_t)a.E) red = 2 * (size_t)a.E;
  const size_t smem = ((size_t)TB * a.E + red) * sizeof(double);
  if (smem > 200 * 1024) return AAL_ERR_UNSUPPORTED;
  return launch_pdl<k_moe_router<T, VEC, TB>>(dim3((unsigned)((a.B + TB - 1) / TB * kRouterCtas)), kRouterThreads, smem,
                                              0, s, a);
}
// Two entries a cluster share its weight loads and conversions (four need more
// registers than the loads in flight leave: 25 against 17 us at 64 entries;
// one 23, and at 16 entries the same within a microsecond);
// one entry a cluster leaves more SMs to few entries, and serves what does not
// fit.
template <typename T, int VEC>
static aal_status run_router_tb(const RouterArgs& a, cudaStream_t s) {
  if (a.B > 16) {
    const aal_status st = run_router<T, VEC, 2>(a, s);
    if (st != AAL_ERR_UNSUPPORTED) return st;
  }
  return run_router<T, VEC, 1>(a, s);
}

// The widest router the kernel holds in shared memory.
constexpr int kMaxExperts = 2048;
constexpr long long kMaxWidth = 1 << 20;  // of x and of h

static bool vec16(const aal_mat& m) {
  const size_t es = m.dtype == AAL_F32 ? 4 : 2;
  return !m.ptr || (((uintptr_t)m.ptr % 16) == 0 && (m.ld * es) % 16 == 0);
}

template <int NT, int S>
static size_t up_bytes() {
  return (size_t)kWarps * (S * Ring<NT, S>::kStep + Sums<NT>::kFloats * sizeof(float));
}
template <int NT, int S>
static size_t down_bytes(int B) {
  return (size_t)kWarps * S * Ring<NT, S>::kStep + (size_t)(B * kYRow + 3) / 4 * 4 * sizeof(float);
}
constexpr size_t kHalfSm = 113 * 1024;  // shared memory of a CTA that leaves room for a second one

template <int NT, int S>
static aal_status run_up(ExpertArgs a, size_t tables, cudaStream_t s) {
  const int sms = device_sms();
  const int bo = a.F / a.q, bi = a.D / a.q;
  a.tiles = (bo + kTile - 1) / kTile;
  a.ntile = a.q * a.tiles;
  a.by_tiles = tc::make_fastdiv((uint32_t)a.tiles);
  a.by_ntile = tc::make_fastdiv((uint32_t)a.ntile);
  const long long pieces = (long long)a.ntile * a.passes, room = 2LL * sms;
  // clusters while each piece has one to itself and every warp two steps (one
  // token of 2 experts, 24 pieces: 20.5 us a step against 22.8 without; of 8,
  // 96 pieces in turns: 36.1 against 33.2; clusters of two for one token of 8
  // experts under Q_16, 128 pieces: 21.4 against 18.1)
  const int steps = (a.q < 2 ? 1 : 2) * (bi >> 4);
  const int z = 4 * pieces <= room && steps >= 32 ? 4 : 1;
  a.zsplit = z;
  return timed(AAL_KERNEL_MOE_UP, s, [&] {
    return launch_pdl<k_moe_up<NT, S>>(dim3((unsigned)(pieces * z < room ? pieces * z : room)), kThreads, up_bytes<NT, S>() + tables,
                  z > 1 ? z : 0, s, a);
  });
}
template <int NT, int S>
static aal_status run_down(ExpertArgs a, size_t tables, cudaStream_t s) {
  const int bo = a.D / a.q;
  a.tiles = (bo + kTile - 1) / kTile;
  a.ntile = a.q * a.tiles;
  const size_t smem = down_bytes<NT, S>(a.B) + tables;
  // Clusters of 4 against 8: one token of 8 experts under Q_16 17.8 against
  // 21.9 us a step (all three kernels), 16 entries of 4 experts 40.8 against
  // 34.1 us.
  const bool little = a.passes <= 16;
  return timed(AAL_KERNEL_MOE_DOWN, s, [&] {
    return little ? launch_pdl<k_moe_down<NT, S, 4>>(dim3((unsigned)(a.ntile * 4)), kThreads, smem, 0, s, a)
                  : launch_pdl<k_moe_down<NT, S, 8>>(dim3((unsigned)(a.ntile * 8)), kThreads, smem, 0, s, a);
  });
}
// NT tiles of 8 entries a pass; a ring of four steps where two CTAs still
// share a SM, else of three (8 entries of 128 dense experts: 109 against 119 us
// a step when measured with shared left-overs).
template <int NT>
static aal_status run_experts(ExpertArgs a, cudaStream_t s) {
  // every expert's last pass may be part full
  const int slots = a.B * a.k, used = slots < a.E ? slots : a.E;
  const int most = used + slots / (8 * NT);
  a.passes = slots < most ? slots : most;
  a.by_k = tc::make_fastdiv((uint32_t)a.k);
  const size_t tables = Tables::bytes(a.passes, a.E, a.B, a.k);
  const aal_status st = up_bytes<NT, 4>() + tables <= kHalfSm ? run_up<NT, 4>(a, tables, s) : run_up<NT, 3>(a, tables, s);
  if (st != AAL_OK) return st;
  return down_bytes<NT, 4>(a.B) + tables <= kHalfSm ? run_down<NT, 4>(a, tables, s) : run_down<NT, 3>(a, tables, s);
}

template <typename T, int VEC>
static aal_status run_general(const ExpertArgs& e, const aal_mat& x, const aal_mat& Wg, const aal_mat& Wu,
                              const aal_mat& Wd, const aal_mat& R, const aal_mat& h, const aal_mat& y, cudaStream_t s) {
  GenArgs<T> g = {e, (const T*)x.ptr, (const T*)Wg.ptr, (const T*)Wu.ptr, (const T*)Wd.ptr, (const T*)R.ptr, (T*)h.ptr,
                  (T*)y.ptr, {}};
  ExpertArgs& a = g.e;
  const int slots = a.B * a.k, used = slots < a.E ? slots : a.E, most = used + slots / kGenEntries;
  a.passes = slots < most ? slots : most;
  a.by_k = tc::make_fastdiv((uint32_t)a.k);
  const size_t tables = Tables::bytes(a.passes, a.E, a.B, a.k);
  const int sms = device_sms();
  auto divisor = [](int n) { return tc::make_fastdiv((uint32_t)(n > 0 ? n : 1)); };  // (of an empty width: not used)
  auto tiles = [&](int bo, int bi) {
    a.tiles = (bo + kGenTile - 1) / kGenTile;
    a.ntile = a.q * a.tiles;
    a.by_tiles = divisor(a.tiles);
    a.by_ntile = divisor(a.ntile);
    g.by_bi = divisor(bi);
  };
  tiles(a.F / a.q, a.D / a.q);
  const long long pieces = (long long)a.ntile * a.passes, room = 2LL * sms;
  // F = 0: one CTA without a piece, so that the down kernel still starts after
  // the router's end
  const unsigned grid = pieces < 1 ? 1 : (unsigned)(pieces < room ? pieces : room);
  aal_status st = timed(AAL_KERNEL_MOE_UP, s, [&] {
    return launch_pdl<k_moe_up_general<T, VEC>>(dim3(grid), kThreads, tables, 0, s, g);
  });
  if (st != AAL_OK) return st;
  if (a.D == 0) return AAL_OK;  // y has no elements
  tiles(a.D / a.q, a.F / a.q);
  return timed(AAL_KERNEL_MOE_DOWN, s, [&] {
    return launch_pdl<k_moe_down_general<T, VEC>>(dim3((unsigned)(a.ntile * kDownCtas)), kThreads,
                  (size_t)a.B * kGenTile * sizeof(float) + tables, 0, s, g);
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
  // (pieces of a launch, 32 columns of 1024 passes at most, are counted in 32 bits)
  if (top_k > moe::kMaxTopK || E > moe::kMaxExperts || D > moe::kMaxWidth || F > moe::kMaxWidth)
    return AAL_ERR_UNSUPPORTED;
  if (Wr.rows != D || Wg.rows != E * D || Wu.rows != E * D || Wu.cols != F || Wd.rows != E * F || Wd.cols != D ||
      (R.ptr && (R.rows != B || R.cols != D)) || h.rows != B * top_k || h.cols != F || y.rows != B || y.cols != D)
    return AAL_ERR_INVALID_ARG;
  if (D % q || F % q) return AAL_ERR_INVALID_ARG;
  if (((uintptr_t)positions % 8) || ((uintptr_t)ids % 4) || ((uintptr_t)weights % 4)) return AAL_ERR_INVALID_ARG;
  if (B > 0 && (!positions || !ids || !weights)) return AAL_ERR_INVALID_ARG;
  note_path(0);
  if (B == 0) return AAL_OK;
  cudaStream_t s = (cudaStream_t)stream;
  // (empty widths leave no tile to multiply: the general path takes the empty sums)
  const bool fast = t_policy != AAL_PATH_GENERAL && dt == AAL_BF16 && q <= moe::kMaxQ && D > 0 && F > 0 &&
                    (D / q) % 16 == 0 && (F / q) % 16 == 0 && moe::vec16(x) && moe::vec16(Wg) && moe::vec16(Wu) &&
                    moe::vec16(Wd) && moe::vec16(h);
  if (!fast && t_policy == AAL_PATH_TENSOR) return AAL_ERR_UNSUPPORTED;
  const size_t es = dt == AAL_F32 ? 4 : 2;
  const bool wvec = moe::vec16(Wg) && moe::vec16(Wu) && moe::vec16(Wd) && (D / q) % 4 == 0 && (F / q) % 4 == 0;
  const bool rvec = moe::vec16(Wr) && (E * es) % 16 == 0;
  auto at = [&](const aal_mat& m, long long row) { return m.ptr ? (char*)m.ptr + row * m.ld * es : nullptr; };
  aal_status st = AAL_OK;
  const int chunk = moe::kSlots / top_k < moe::kChunk ? moe::kSlots / top_k : moe::kChunk;
  for (long long b0 = 0; b0 < B && st == AAL_OK; b0 += chunk) {
    const int nb = (int)(B - b0 < chunk ? B - b0 : chunk);
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
    using bf = __nv_bfloat16;
    aal_mat xs = x, Rs = R, hs = h, ys = y;
    xs.ptr = at(x, b0);
    Rs.ptr = at(R, b0);
    hs.ptr = at(h, b0 * top_k);
    ys.ptr = at(y, b0);
    moe::ExpertArgs a = {positions + b0, id, wt, (const bf*)xs.ptr, (const bf*)Wg.ptr, (const bf*)Wu.ptr,
                         (const bf*)Wd.ptr, (const bf*)Rs.ptr, (bf*)hs.ptr, (bf*)ys.ptr, x.ld, Wg.ld, Wu.ld, Wd.ld, h.ld,
                         R.ld, y.ld, law, q, nb, top_k, (int)E, (int)D, (int)F, 0, 0, 0, 0, {}, {}, {}};
    // two tiles of entries a pass where experts get more than six on average
    // (32 entries, 2 of 8 experts each: 45.4 us against 51.3 with one; 16
    // entries, 4 of 64 each: 38.9 against 33.8)
    if (fast) st = (long long)nb * top_k <= 6 * E ? moe::run_experts<1>(a, s) : moe::run_experts<2>(a, s);
    else if (dt == AAL_F32 && wvec) st = moe::run_general<float, 4>(a, xs, Wg, Wu, Wd, Rs, hs, ys, s);
    else if (dt == AAL_F32) st = moe::run_general<float, 1>(a, xs, Wg, Wu, Wd, Rs, hs, ys, s);
    else st = moe::run_general<bf, 1>(a, xs, Wg, Wu, Wd, Rs, hs, ys, s);
  }
  if (st == AAL_OK) note_path(fast ? AAL_PATH_DECODE : AAL_PATH_GENERAL);
  return st;
}
