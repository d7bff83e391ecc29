// Layer norm of the rows of a matrix, forward and backward: the norm ahead of
// the feed-forward block (and, with R, the residual add that precedes it).
//
//   s = x (+ r),  mu = mean(s),  v = mean((s - mu)^2),  rstd = 1 / sqrt(v + eps)
//   y = (s - mu) rstd gamma + beta
//   backward, with xh = (s - mu) rstd and g = dy gamma:
//   dx = rstd (g - mean(g) - xh mean(g xh)) (+ dr)
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Every byte of the matrices crosses HBM once while two rows of every input fit
// the ring: up to 16,384 columns, but 14,464 for fp32 rows with R and backward
// with fp32 gamma, 8,264 for fp32 rows backward, and 8,192 where rows start
// anywhere.  Wider rows are walked several times.  A row comes into shared memory
// while the ones before it are reduced, the variance is the
// mean of the squared distances from the mean (no cancellation), and the
// backward keeps dgamma and dbeta of a thread's own columns in fp32 registers
// over all the rows its CTA visits.  The CTAs' column sums go to the caller's
// workspace and a second, programmatically dependent launch adds them in CTA
// order, so results do not depend on timing.
//
// Measured, microseconds a call in a graph, against the bytes at the copy rate
// of 6.53 TB/s:  forward 12288 x 768 bf16 with residual 16.3 (11.6), 2048 x
// 4096 fp32 17.0 (10.3), 4099 x 1003 bf16 10.1 (2.5);  backward 32768 x 5120
// bf16 with dR 208 (205), 12288 x 768 22.5 (11.6), 2047 x 1001 fp32 17-18
// (3.8), 96 x 2048 7.4.  Large calls are bound by HBM; those of a few rows a
// CTA by the ring's start, the reductions of the rows and, backward, the second
// launch.
#include "aal_internal.h"

#include <math.h>

#include <atomic>
#include <type_traits>

namespace aal {
namespace norm {

// Two fp32 values in a register pair: Blackwell adds and multiplies pairs in
// one instruction, and these kernels issue more than they wait for memory.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(f32x2 v) {
  float a, b;
  unpair(v, a, b);
  return a + b;
}

// Elements of a 16-byte vector of T, and that many elements of a parameter
// vector of type TP (one or two 16-byte words), as pairs of fp32.
template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T), pairs = n / 2;
};
__device__ __forceinline__ void widen(const uint4& u, f32x2 (&o)[4], __nv_bfloat16) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void widen(const uint4& u, f32x2 (&o)[2], float) {
  o[0] = pair(__uint_as_float(u.x), __uint_as_float(u.y));
  o[1] = pair(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint4 narrow(const f32x2 (&v)[4], __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpair(v[i], a, b);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    memcpy(&w[i], &h, 4);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 narrow(const f32x2 (&v)[2], float) {
  float a, b, c, d;
  unpair(v[0], a, b);
  unpair(v[1], c, d);
  return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}
// A shared-memory load that stays where it is written: the backward reads its
// row twice rather than hold it in registers across the reduction.
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr));
  return u;
}
template <typename T, typename TP>
struct Param {
  static constexpr int words = Vec<T>::n * sizeof(TP) / 16;
  uint4 u[words];
  __device__ __forceinline__ void load(const TP* p) {
#pragma unroll
    for (int i = 0; i < words; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void load_shared(uint32_t addr) {
#pragma unroll
    for (int i = 0; i < words; ++i) u[i] = lds128(addr + i * 16);
  }
  __device__ __forceinline__ void get(f32x2 (&o)[Vec<T>::pairs]) const {
    if constexpr (words == 2) {
      f32x2 a[2], b[2];
      widen(u[0], a, 0.f);
      widen(u[1], b, 0.f);
      o[0] = a[0];
      o[1] = a[1];
      o[2] = b[0];
      o[3] = b[1];
    } else {
      widen(u[0], o, TP());
    }
  }
};
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the block's warps of (a, b) in one barrier.  ``buf`` alternates
// between two arrays so that the next call cannot overwrite values another
// warp has yet to read.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2 (*buf)[32], int& turn) {
  a = warp_sum(a);
  b = warp_sum(b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) buf[turn][warp] = make_float2(a, b);
  __syncthreads();
  const float2 r = lane < nw ? buf[turn][lane] : make_float2(0.f, 0.f);
  turn ^= 1;
  return make_float2(warp_sum(r.x), warp_sum(r.y));
}

__device__ __forceinline__ void pdl_begin() {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}


// ------------------------------------------------- rows through shared memory
// Rows come in with bulk asynchronous copies: a group (a warp for narrow rows,
// the CTA for wide ones) owns a ring of stages, each holding its next row (or
// rows, several narrow ones share a warp) of every input array, and one thread
// refills a stage as soon as the group is done with it.  The next rows are so
// in flight while one is reduced, about 100 KB a SM, which plain loads could
// not do: their registers held one row and nothing moved during the
// reductions.
//
// A bulk copy moves whole 16-byte words.  Where rows start on them (the vector
// form) a thread takes 16-byte vectors; elsewhere (the element form) the copy
// brings the words that lie inside the row, a few threads fetch the elements
// before and after them (a row ahead, through registers), and a thread takes
// elements TPR apart.
constexpr int kMaxRing = 4;
constexpr int kRowsPerCta = 8;  // groups of a CTA of warps
constexpr unsigned long long kRingWaitNs = 2000000000ull, kRingLostNs = 100000ull;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}
// Bounded wait for a stage.  A copy that has not landed after two seconds never
// will: the status word is set (in place of any other error) and the caller goes
// on with what is there, so that every thread still reaches the kernel's barriers.
// From then on every wait is short, the ones for copies still in flight and the
// ones for rows that will not come (refill), so that the kernel ends within
// seconds whatever the number of rows.
__device__ __forceinline__ void ring_wait(uint64_t* bar, uint32_t parity) {
  if (tc::mbar_try_wait(bar, parity)) return;
  const unsigned long long t0 = tc::gtime();
  for (uint32_t i = 0; !tc::mbar_try_wait(bar, parity); ++i)
    if ((i & 255u) == 255u &&
        tc::gtime() - t0 > (*(volatile int*)&g_device_status == kDevTimeout ? kRingLostNs : kRingWaitNs)) {
      atomicExch(&g_device_status, kDevTimeout);
      return;
    }
}

// Bytes of a stage's copy of one array: ``rows`` rows of d elements, in the
// element form with room for the row's offset from a 16-byte boundary.
__host__ __device__ __forceinline__ uint32_t region_bytes(long long d, int es, int rows, bool elem) {
  return elem ? (uint32_t)((d * es + 30) / 16 * 16) : (uint32_t)(d * es * rows);
}

// Where the pieces of a row lie (element form).
struct Edges {
  uint32_t off;         // bytes from the region's start to element 0
  uint32_t from, size;  // the whole words inside the row: offset from element 0, bytes
  int head, tail;       // elements before and after them
};
template <typename T>
__device__ __forceinline__ Edges edges_of(const T* row, int d) {
  const uint32_t a = (uint32_t)((uintptr_t)row & 15), len = (uint32_t)(d * sizeof(T));
  Edges e;
  e.off = a;
  e.from = (16u - a) & 15u;
  const uint32_t end = (a + len) & ~15u;  // past the last whole word, from the boundary below the row
  if (e.from >= len || end <= a + e.from) {
    e.from = e.size = 0;
    e.head = d;  // no whole word: fewer than 16 bytes either side
    e.tail = 0;
  } else {
    e.size = end - a - e.from;
    e.head = (int)(e.from / sizeof(T));
    e.tail = (int)((a + len - end) / sizeof(T));
  }
  return e;
}
constexpr int kEdgeThreads = 32;  // threads 0-15 take elements before the words, 16-31 after them
// The element of the row's edges that thread t fetches, or -1.
__device__ __forceinline__ int edge_index(const Edges& e, int d, int t) {
  if (t < 16) return t < e.head ? t : -1;
  return t - 16 < e.tail ? d - e.tail + t - 16 : -1;
}

// What a group knows of its place in the launch.
template <int TPR, bool SUB>
struct Group {
  static constexpr bool BLOCK = TPR != 32;
  int tpr, t, lane;     // threads a row, this thread's place in its row, in its group
  int index;            // group within the CTA
  int rpw, sub;         // rows a group takes at once, this thread's one of them
  long long first, step;  // blocks of rpw rows
  __device__ __forceinline__ explicit Group(int lpr) {
    lane = BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & 31);
    index = BLOCK ? 0 : (int)(threadIdx.x >> 5);
    tpr = SUB ? lpr : TPR ? TPR : (int)blockDim.x;
    rpw = SUB ? 32 / lpr : 1;
    sub = SUB ? lane / lpr : 0;
    t = SUB ? lane % lpr : lane;
    first = BLOCK ? (long long)blockIdx.x : (long long)blockIdx.x * kRowsPerCta + index;
    step = BLOCK ? (long long)gridDim.x : (long long)gridDim.x * kRowsPerCta;
  }
  __device__ __forceinline__ void sync() const {
    if (BLOCK) __syncthreads();
    else __syncwarp();
  }
  // Sum of (a, b) over the row's threads.
  __device__ __forceinline__ float2 sum(float a, float b, float2 (*buf)[32], int& turn) const {
    if (BLOCK) return block_sum2(a, b, buf, turn);
    return make_float2(sum(a), sum(b));
  }
  __device__ __forceinline__ float sum(float a, float2 (*buf)[32], int& turn) const {
    return BLOCK ? block_sum2(a, 0.f, buf, turn).x : sum(a);
  }
  __device__ __forceinline__ float sum(float a) const {
    if constexpr (SUB) {
      for (int o = tpr >> 1; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
      return a;
    } else {
      return warp_sum(a);
    }
  }
};

// Copies the rows of block rb of one array into a stage's region.
template <typename T, bool SUB, bool ELEM>
__device__ __forceinline__ void fill_region(uint32_t dst, const T* p, long long ld, int d, long long rb, int rpw,
                                            int rows, uint64_t* bar) {
  const T* src = p + rb * rpw * ld;
  if constexpr (ELEM) {
    const Edges e = edges_of(src, d);
    if (e.size) bulk_load(dst + e.off + e.from, (const char*)src + e.from, e.size, bar);
  } else if constexpr (!SUB) {
    bulk_load(dst, src, (uint32_t)(d * sizeof(T)), bar);
  } else if (ld == d) {
    bulk_load(dst, src, (uint32_t)(d * sizeof(T)) * rows, bar);
  } else {
    for (int i = 0; i < rows; ++i)
      bulk_load(dst + i * (uint32_t)(d * sizeof(T)), src + i * ld, (uint32_t)(d * sizeof(T)), bar);
  }
}
// and how many bytes that is.
template <typename T, bool ELEM>
__device__ __forceinline__ uint32_t fill_bytes(const T* p, long long ld, int d, long long rb, int rpw, int rows) {
  return ELEM ? edges_of(p + rb * rpw * ld, d).size : (uint32_t)(d * sizeof(T)) * rows;
}

// A thread's vector i of a row in shared memory (16 bytes, or that many
// elements TPR apart), as pairs; elements past the row read as zero.
template <typename T, bool ELEM, int TPR>
__device__ __forceinline__ void row_get(uint32_t row, int i, int tpr, int left, f32x2 (&v)[Vec<T>::pairs]) {
  constexpr int n = Vec<T>::n;
  if constexpr (!ELEM) {
    widen(lds128(row + i * tpr * 16), v, T());
  } else {
    float e[n];
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const int k = (i * n + j) * TPR;
      e[j] = 0.f;
      if (k < left) {
        if constexpr (sizeof(T) == 2) {
          unsigned short h;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(row + k * 2));
          e[j] = __uint_as_float((uint32_t)h << 16);
        } else {
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(e[j]) : "r"(row + k * 4));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < Vec<T>::pairs; ++j) v[j] = pair(e[2 * j], e[2 * j + 1]);
  }
}
// A thread's vector i of a row less the row's mean.  bf16 elements are widened by
// the addition itself, one mixed-precision instruction an element (32768 x 5120
// backward 208 us; with a pair addition after the widening 217).
template <typename T, bool ELEM, int TPR>
__device__ __forceinline__ void row_get_less(uint32_t row, int i, int tpr, int left, float mean,
                                             f32x2 (&v)[Vec<T>::pairs]) {
  if constexpr (!ELEM && sizeof(T) == 2) {
    const uint4 u = lds128(row + i * tpr * 16);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("{\n\t.reg .b16 lo, hi;\n\t.reg .f32 a, b;\n\tmov.b32 {lo, hi}, %1;\n\tadd.rn.f32.bf16 a, lo, %2;\n\t"
          "add.rn.f32.bf16 b, hi, %2;\n\tmov.b64 %0, {a, b};\n\t}"
          : "=l"(v[j])
          : "r"(w[j]), "f"(-mean));
  } else {
    row_get<T, ELEM, TPR>(row, i, tpr, left, v);
#pragma unroll
    for (int j = 0; j < Vec<T>::pairs; ++j) v[j] = add2(v[j], pair(-mean, -mean));
  }
}
template <typename T, bool ELEM, int TPR>
__device__ __forceinline__ void row_put(T* row, int i, int tpr, int left, const f32x2 (&v)[Vec<T>::pairs]) {
  constexpr int n = Vec<T>::n;
  if constexpr (!ELEM) {
    *reinterpret_cast<uint4*>(row + i * tpr * n) = narrow(v, T());
  } else {
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const int k = (i * n + j) * TPR;
      float a, b;
      unpair(v[j / 2], a, b);
      if (k < left) row[k] = from_f32<T>(j & 1 ? b : a);
    }
  }
}
// A thread's part of a parameter vector in registers.
template <typename T, typename TP, bool ELEM, int TPR>
struct ParamPart {
  static constexpr int n = Vec<T>::n;
  std::conditional_t<ELEM, float[n], Param<T, TP>> u;
  __device__ __forceinline__ void load(const TP* p, int i, int tpr, int left) {
    if constexpr (ELEM) {
#pragma unroll
      for (int j = 0; j < n; ++j) u[j] = (i * n + j) * TPR < left ? as_f32(p[(i * n + j) * TPR]) : 0.f;
    } else {
      u.load(p + i * tpr * n);
    }
  }
  __device__ __forceinline__ void get(f32x2 (&o)[Vec<T>::pairs]) const {
    if constexpr (ELEM) {
#pragma unroll
      for (int j = 0; j < Vec<T>::pairs; ++j) o[j] = pair(u[2 * j], u[2 * j + 1]);
    } else {
      u.get(o);
    }
  }
};

struct FwdArgs {
  const void *x, *r, *gamma, *beta;
  void *s, *y;
  float *mean, *rstd;
  long long rows, d, ldx, ldr, lds, ldy;
  float eps;
  int ring;  // stages
  int lpr;   // lanes a row (warps)
};

// TPR: 32 a warp a row (SUB: lpr lanes of one), 0 the CTA of any size, else the
// CTA of that size.  NV vectors a thread.  MAXT, MINB: the largest CTA, and
// how many of them a SM is to hold.
template <typename T, typename TP, int NV, int TPR, bool SUB, bool ELEM, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_ln_fwd(const FwdArgs a) {
  constexpr int VEC = Vec<T>::n, P = Vec<T>::pairs;
  constexpr bool BLOCK = TPR != 32;
  extern __shared__ __align__(128) unsigned char ring_mem[];
  __shared__ float2 buf[2][32];
  __shared__ __align__(8) uint64_t bars[(BLOCK ? 1 : kRowsPerCta) * kMaxRing];
  __shared__ volatile int lost[BLOCK ? 1 : kRowsPerCta];  // by group: a copy has not landed
  const Group<TPR, SUB> gr(a.lpr);
  const int t = gr.t, tpr = gr.tpr, d = (int)a.d, S = a.ring;
  const T *x = (const T*)a.x, *r = (const T*)a.r;
  const TP *gm = (const TP*)a.gamma, *bt = (const TP*)a.beta;
  const uint32_t region = region_bytes(d, sizeof(T), gr.rpw, ELEM), stage = region * (r ? 2u : 1u);
  const uint32_t mem = tc::smem_u32(ring_mem) + (uint32_t)gr.index * S * stage;
  uint64_t* bar = bars + gr.index * kMaxRing;
  if (gr.lane == 0) {
    lost[gr.index] = 0;
    for (int i = 0; i < S; ++i) tc::mbar_init(&bar[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tc::fence_async_smem();
  }
  pdl_begin();
  auto rows_of = [&](long long rb) { return SUB ? (int)min((long long)gr.rpw, a.rows - rb * gr.rpw) : 1; };
  auto fill = [&](long long rb, int st) {
    const int n = rows_of(rb);
    tc::mbar_expect_tx(&bar[st], fill_bytes<T, ELEM>(x, a.ldx, d, rb, gr.rpw, n) +
                                     (r ? fill_bytes<T, ELEM>(r, a.ldr, d, rb, gr.rpw, n) : 0u));
    fill_region<T, SUB, ELEM>(mem + st * stage, x, a.ldx, d, rb, gr.rpw, n, &bar[st]);
    if (r) fill_region<T, SUB, ELEM>(mem + st * stage + region, r, a.ldr, d, rb, gr.rpw, n, &bar[st]);
  };
  // A stage takes the next row once the one before has landed.  After a loss none
  // does: the barrier's turn is not over, and must not get a second arrival.
  auto refill = [&](long long rb, int st, uint32_t phase) {
    if (!tc::mbar_try_wait(&bar[st], phase)) lost[gr.index] = 1;
    if (!lost[gr.index]) fill(rb, st);
  };
  const long long blocks = SUB ? (a.rows + gr.rpw - 1) / gr.rpw : a.rows;
  if (gr.lane == 0)
    for (int i = 0; i < S; ++i)
      if (gr.first + i * gr.step < blocks) fill(gr.first + i * gr.step, i);
  gr.sync();
  // this thread's edge elements of row ``row``
  T ex = T(0.f), er = T(0.f);
  auto edges = [&](long long row) {
    if (!ELEM || gr.lane >= kEdgeThreads || row >= a.rows) return;
    const int i = edge_index(edges_of(x + row * a.ldx, d), d, gr.lane);
    if (i >= 0) ex = x[row * a.ldx + i];
    if (r) {
      const int j = edge_index(edges_of(r + row * a.ldr, d), d, gr.lane);
      if (j >= 0) er = r[row * a.ldr + j];
    }
  };
  auto put_edge = [&](uint32_t where, const T* row, T v) {
    const Edges e = edges_of(row, d);
    const int i = edge_index(e, d, gr.lane);
    if (i >= 0) *reinterpret_cast<T*>(ring_mem + (where - tc::smem_u32(ring_mem)) + e.off + i * sizeof(T)) = v;
  };
  edges(gr.first);
  const int left = ELEM ? d - t : (d - t * VEC + VEC - 1) / VEC;  // elements (vectors: elements / VEC) from this thread's on
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = ELEM ? i * VEC * TPR < left : (i * tpr + t) * VEC < d;
  ParamPart<T, TP, ELEM, TPR> pg[NV], pb[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (in[i]) {
      if (gm) pg[i].load(gm + t * (ELEM ? 1 : VEC), i, tpr, left);
      if (bt) pb[i].load(bt + t * (ELEM ? 1 : VEC), i, tpr, left);
    }
  const float inv_d = 1.0f / (float)d;
  int turn = 0, st = 0, before = S - 1;  // this block's stage and the one before's
  uint32_t ph = 0;
  for (long long rb = gr.first; rb < blocks; rb += gr.step) {
    const long long row = rb * gr.rpw + gr.sub;
    const bool on = !SUB || row < a.rows;
    uint32_t m = mem + st * stage;
    uint32_t mr = m + region;
    if (ELEM) {
      if (gr.lane < kEdgeThreads) {
        put_edge(m, x + row * a.ldx, ex);
        if (r) put_edge(mr, r + row * a.ldr, er);
        tc::fence_async_smem();  // before the copy that refills the stage
      }
      edges(row + gr.step);
      m += (uint32_t)((uintptr_t)(x + row * a.ldx) & 15) + t * sizeof(T);
      if (r) mr += (uint32_t)((uintptr_t)(r + row * a.ldr) & 15) + t * sizeof(T);
    } else {
      m += gr.sub * (uint32_t)(d * sizeof(T)) + t * 16;
      mr += gr.sub * (uint32_t)(d * sizeof(T)) + t * 16;
    }
    ring_wait(&bar[st], ph);
    if (ELEM) gr.sync();
    f32x2 v[NV][P];
    f32x2 sum = 0;  // two zeros
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < P; ++j) v[i][j] = 0;
      if (in[i] && on) {
        row_get<T, ELEM, TPR>(m, i, tpr, left, v[i]);
        if (r) {
          f32x2 w[P];
          row_get<T, ELEM, TPR>(mr, i, tpr, left, w);
#pragma unroll
          for (int j = 0; j < P; ++j) v[i][j] = add2(v[i][j], w[j]);
        }
#pragma unroll
        for (int j = 0; j < P; ++j) sum = add2(sum, v[i][j]);
      }
    }
    const float mu = gr.sum(sum2(sum), buf, turn) * inv_d;
    // A warp has its rows in registers, all its lanes' past the barrier; a CTA's
    // threads are all done with the row before this one (the sum's barrier).
    // The sum over a row's lanes alone would not order the other rows' reads
    // before the copy that refills their stage.
    if (!BLOCK) __syncwarp();
    const long long next = rb + (BLOCK ? S - 1 : S) * gr.step;
    if (gr.lane == 0 && next < blocks && (!BLOCK || rb != gr.first))
      refill(next, BLOCK ? before : st, BLOCK && st == 0 ? ph ^ 1u : ph);
    before = st;
    if (++st == S) { st = 0; ph ^= 1u; }
    const f32x2 nmu = pair(-mu, -mu);
    f32x2 sq = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          f32x2 e = add2(v[i][j], nmu);
          if (ELEM) {  // elements past the row are zeros, not members of the sum
            float e0, e1;
            unpair(e, e0, e1);
            e = pair((i * VEC + 2 * j) * TPR < left ? e0 : 0.f, (i * VEC + 2 * j + 1) * TPR < left ? e1 : 0.f);
          }
          sq = fma2(e, e, sq);
        }
      }
    const float var = gr.sum(sum2(sq), buf, turn) * inv_d;
    const float rs = 1.0f / sqrtf(var + a.eps);
    if (!on) continue;
    if (t == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = rs;
    }
    const f32x2 rs2 = pair(rs, rs);
    T* yo = (T*)a.y + row * a.ldy + t * (ELEM ? 1 : VEC);
    T* so = (T*)a.s + row * a.lds + t * (ELEM ? 1 : VEC);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      // the stored sum is rounded to the matrix type; the norm itself uses
      // the unrounded one
      if (a.s) row_put<T, ELEM, TPR>(so, i, tpr, left, v[i]);
      f32x2 e[P], w[P];
#pragma unroll
      for (int j = 0; j < P; ++j) e[j] = mul2(add2(v[i][j], nmu), rs2);
      if (gm) {
        pg[i].get(w);
#pragma unroll
        for (int j = 0; j < P; ++j) e[j] = mul2(e[j], w[j]);
      }
      if (bt) {
        pb[i].get(w);
#pragma unroll
        for (int j = 0; j < P; ++j) e[j] = add2(e[j], w[j]);
      }
      row_put<T, ELEM, TPR>(yo, i, tpr, left, e);
    }
  }
}

// Rows too wide for registers: the CTA walks its row three times (the second
// and third pass hit L2).  S and Y are written in the last pass only, each
// element after its own last read, so they may be X or R.
template <typename T, typename TP>
__global__ void __launch_bounds__(1024) k_ln_fwd_wide(const FwdArgs a) {
  __shared__ float2 buf[2][32];
  pdl_begin();
  const TP *gm = (const TP*)a.gamma, *bt = (const TP*)a.beta;
  int turn = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ldx;
    const T* r = a.r ? (const T*)a.r + row * a.ldr : nullptr;
    float sum = 0.f;
    for (long long c = threadIdx.x; c < a.d; c += blockDim.x) sum += as_f32(x[c]) + (r ? as_f32(r[c]) : 0.f);
    const float mu = block_sum2(sum, 0.f, buf, turn).x / (float)a.d;
    float sq = 0.f;
    for (long long c = threadIdx.x; c < a.d; c += blockDim.x) {
      const float e = as_f32(x[c]) + (r ? as_f32(r[c]) : 0.f) - mu;
      sq = fmaf(e, e, sq);
    }
    const float rs = 1.0f / sqrtf(block_sum2(sq, 0.f, buf, turn).x / (float)a.d + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = rs;
    }
    for (long long c = threadIdx.x; c < a.d; c += blockDim.x) {
      const float s = as_f32(x[c]) + (r ? as_f32(r[c]) : 0.f);
      float e = (s - mu) * rs;
      if (gm) e *= as_f32(gm[c]);
      if (bt) e += as_f32(bt[c]);
      if (a.s) ((T*)a.s)[row * a.lds + c] = from_f32<T>(s);
      ((T*)a.y)[row * a.ldy + c] = from_f32<T>(e);
    }
  }
}

struct BwdArgs {
  const void *x, *gamma, *dy, *dr;
  const float *mean, *rstd;
  void* dx;
  float* part;  // [grid][2][d] column sums of each CTA, or null
  long long rows, d, ldx, lddy, lddr, lddx;
  int ring;  // stages
  int lpr;   // lanes a row (warps)
  uint32_t ring_bytes;
};

// dx = rstd (g - mean(g) - xh mean(g xh)) as g rstd + A + B (x - mu), the row's
// two numbers folded once.  The mean is subtracted from x, where the difference
// is rounded against itself: with -B mu folded into A instead, two large numbers
// would cancel in rows far from zero (relative error of dx 5e-5 instead of 8e-8
// at a mean of 1000 standard deviations).
struct RowFold {
  float A, B;
};
__device__ __forceinline__ RowFold fold_row(float rs, float mg, float mgx) {
  RowFold f;
  f.A = -rs * mg;
  f.B = -rs * (rs * mgx);
  return f;
}

template <typename T, typename TP, int NV, int TPR, bool SUB, bool ELEM, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_ln_bwd(const BwdArgs a) {
  constexpr int VEC = Vec<T>::n, P = Vec<T>::pairs;
  constexpr bool BLOCK = TPR != 32;
  extern __shared__ __align__(128) unsigned char ring_mem[];
  __shared__ float2 buf[2][32];
  __shared__ __align__(8) uint64_t bars[(BLOCK ? 1 : kRowsPerCta) * kMaxRing];
  __shared__ volatile int lost[BLOCK ? 1 : kRowsPerCta];  // by group: a copy has not landed
  const Group<TPR, SUB> gr(a.lpr);
  const int t = gr.t, tpr = gr.tpr, d = (int)a.d, S = a.ring;
  const T *x = (const T*)a.x, *dy = (const T*)a.dy, *dr = (const T*)a.dr;
  const TP* gm = (const TP*)a.gamma;
  const uint32_t region = region_bytes(d, sizeof(T), gr.rpw, ELEM), stage = region * (dr ? 3u : 2u);
  const uint32_t mem = tc::smem_u32(ring_mem) + (uint32_t)gr.index * S * stage;
  uint64_t* bar = bars + gr.index * kMaxRing;
  if (gr.lane == 0) {
    lost[gr.index] = 0;
    for (int i = 0; i < S; ++i) tc::mbar_init(&bar[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tc::fence_async_smem();
  }
  pdl_begin();
  auto rows_of = [&](long long rb) { return SUB ? (int)min((long long)gr.rpw, a.rows - rb * gr.rpw) : 1; };
  auto fill = [&](long long rb, int st) {
    const int n = rows_of(rb);
    tc::mbar_expect_tx(&bar[st], fill_bytes<T, ELEM>(x, a.ldx, d, rb, gr.rpw, n) +
                                     fill_bytes<T, ELEM>(dy, a.lddy, d, rb, gr.rpw, n) +
                                     (dr ? fill_bytes<T, ELEM>(dr, a.lddr, d, rb, gr.rpw, n) : 0u));
    fill_region<T, SUB, ELEM>(mem + st * stage, x, a.ldx, d, rb, gr.rpw, n, &bar[st]);
    fill_region<T, SUB, ELEM>(mem + st * stage + region, dy, a.lddy, d, rb, gr.rpw, n, &bar[st]);
    if (dr) fill_region<T, SUB, ELEM>(mem + st * stage + 2 * region, dr, a.lddr, d, rb, gr.rpw, n, &bar[st]);
  };
  // A stage takes the next row once the one before has landed.  After a loss none
  // does: the barrier's turn is not over, and must not get a second arrival.
  auto refill = [&](long long rb, int st, uint32_t phase) {
    if (!tc::mbar_try_wait(&bar[st], phase)) lost[gr.index] = 1;
    if (!lost[gr.index]) fill(rb, st);
  };
  const long long blocks = SUB ? (a.rows + gr.rpw - 1) / gr.rpw : a.rows;
  if (gr.lane == 0)
    for (int i = 0; i < S; ++i)
      if (gr.first + i * gr.step < blocks) fill(gr.first + i * gr.step, i);
  gr.sync();
  T ex = T(0.f), ey = T(0.f), er = T(0.f);  // this thread's edge elements
  auto edge = [&](const T* row) {
    const int i = edge_index(edges_of(row, d), d, gr.lane);
    return i >= 0 ? row[i] : T(0.f);
  };
  auto edges = [&](long long row) {
    if (!ELEM || gr.lane >= kEdgeThreads || row >= a.rows) return;
    ex = edge(x + row * a.ldx);
    ey = edge(dy + row * a.lddy);
    if (dr) er = edge(dr + row * a.lddr);
  };
  auto put_edge = [&](uint32_t where, const T* row, T v) {
    const Edges e = edges_of(row, d);
    const int i = edge_index(e, d, gr.lane);
    if (i >= 0) *reinterpret_cast<T*>(ring_mem + (where - tc::smem_u32(ring_mem)) + e.off + i * sizeof(T)) = v;
  };
  edges(gr.first);
  const int left = ELEM ? d - t : (d - t * VEC + VEC - 1) / VEC;
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = ELEM ? i * VEC * TPR < left : (i * tpr + t) * VEC < d;
  // gamma of this thread's columns: in registers (element form), else in
  // shared memory behind the rings (registers would cost rows in flight)
  ParamPart<T, TP, ELEM, TPR> pg[ELEM ? NV : 1];
  const uint32_t gs = tc::smem_u32(ring_mem) + a.ring_bytes;
  if (ELEM && gm) {
#pragma unroll
    for (int i = 0; i < (ELEM ? NV : 1); ++i) pg[i].load(gm + t, i, tpr, left);
  }
  if (!ELEM && gm) {
    const uint4* from = reinterpret_cast<const uint4*>(gm);
    uint4* to = reinterpret_cast<uint4*>(ring_mem + a.ring_bytes);
    for (int c = threadIdx.x; c < d * (int)sizeof(TP) / 16; c += blockDim.x) to[c] = from[c];
    __syncthreads();
  }
  auto gamma = [&](int i, f32x2 (&w)[P]) {
    if constexpr (ELEM) {
      pg[i].get(w);
    } else {
      Param<T, TP> g;
      g.load_shared(gs + (i * tpr + t) * VEC * (uint32_t)sizeof(TP));
      g.get(w);
    }
  };
  const float inv_d = 1.0f / (float)d;
  f32x2 dg[NV][P], db[NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) dg[i][j] = db[i][j] = 0;
  int turn = 0, st = 0, before = S - 1;
  uint32_t ph = 0;
  auto stats = [&](long long rb, float& mu, float& rs) {
    const long long row = rb * gr.rpw + gr.sub;
    mu = rs = 0.f;
    if (row < a.rows) {
      mu = a.mean[row];
      rs = a.rstd[row];
    }
  };
  float mu, rs;
  stats(gr.first, mu, rs);
  for (long long rb = gr.first; rb < blocks; rb += gr.step) {
    const long long row = rb * gr.rpw + gr.sub;
    const bool on = !SUB || row < a.rows;
    float mu_next, rs_next;
    stats(rb + gr.step, mu_next, rs_next);
    uint32_t m = mem + st * stage, my = m + region, mr = my + region;
    if (ELEM) {
      if (gr.lane < kEdgeThreads) {
        put_edge(m, x + row * a.ldx, ex);
        put_edge(my, dy + row * a.lddy, ey);
        if (dr) put_edge(mr, dr + row * a.lddr, er);
        tc::fence_async_smem();  // before the copy that refills the stage
      }
      edges(row + gr.step);
      m += (uint32_t)((uintptr_t)(x + row * a.ldx) & 15) + t * sizeof(T);
      my += (uint32_t)((uintptr_t)(dy + row * a.lddy) & 15) + t * sizeof(T);
      if (dr) mr += (uint32_t)((uintptr_t)(dr + row * a.lddr) & 15) + t * sizeof(T);
    } else {
      const uint32_t o = gr.sub * (uint32_t)(d * sizeof(T)) + t * 16;
      m += o;
      my += o;
      mr += o;
    }
    ring_wait(&bar[st], ph);
    if (ELEM) gr.sync();
    f32x2 sg = 0, sgx = 0;
    const f32x2 rs2 = pair(rs, rs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i] || !on) continue;
      f32x2 xv[P], yv[P], w[P];
      row_get_less<T, ELEM, TPR>(m, i, tpr, left, mu, xv);
      row_get<T, ELEM, TPR>(my, i, tpr, left, yv);  // zero past the row, and with it every product below
      if (gm) gamma(i, w);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const f32x2 xh = mul2(xv[j], rs2);
        const f32x2 g = gm ? mul2(yv[j], w[j]) : yv[j];
        sg = add2(sg, g);
        sgx = fma2(g, xh, sgx);
        dg[i][j] = fma2(yv[j], xh, dg[i][j]);
        db[i][j] = add2(db[i][j], yv[j]);
      }
    }
    const float2 s = gr.sum(sum2(sg), sum2(sgx), buf, turn);
    // past a CTA's barrier every thread is done with the row before this one
    if (BLOCK) {
      const long long next = rb + (S - 1) * gr.step;
      if (gr.lane == 0 && next < blocks && rb != gr.first) refill(next, before, st == 0 ? ph ^ 1u : ph);
    }
    if (a.dx && on) {
      const RowFold f = fold_row(rs, s.x * inv_d, s.y * inv_d);
      const f32x2 A = pair(f.A, f.A), B = pair(f.B, f.B);
      T* o = (T*)a.dx + row * a.lddx + t * (ELEM ? 1 : VEC);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!in[i]) continue;
        f32x2 xv[P], yv[P], w[P];
        row_get_less<T, ELEM, TPR>(m, i, tpr, left, mu, xv);
        row_get<T, ELEM, TPR>(my, i, tpr, left, yv);
        if (gm) gamma(i, w);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const f32x2 g = gm ? mul2(yv[j], w[j]) : yv[j];
          xv[j] = fma2(g, rs2, fma2(xv[j], B, A));  // xv: x - mu
        }
        if (dr) {
          row_get<T, ELEM, TPR>(mr, i, tpr, left, w);
#pragma unroll
          for (int j = 0; j < P; ++j) xv[j] = add2(xv[j], w[j]);
        }
        row_put<T, ELEM, TPR>(o, i, tpr, left, xv);
      }
    }
    if (!BLOCK) {
      __syncwarp();
      const long long next = rb + S * gr.step;
      if (gr.lane == 0 && next < blocks) refill(next, st, ph);
    }
    before = st;
    if (++st == S) { st = 0; ph ^= 1u; }
    mu = mu_next;
    rs = rs_next;
  }
  if (!a.part) return;
  float* out = a.part + (long long)blockIdx.x * 2 * d;
  // A CTA's threads have columns of their own.  A warp's sums go where its
  // ring was (two stages hold them), after those of its several rows have met,
  // and the CTA adds its warps' in order.
  float* mine = BLOCK ? out : reinterpret_cast<float*>(ring_mem + (size_t)gr.index * S * stage);
  if (!BLOCK) {
    __syncwarp();
    for (int o = tpr; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j) {
          dg[i][j] = add2(dg[i][j], __shfl_xor_sync(0xffffffffu, dg[i][j], o));
          db[i][j] = add2(db[i][j], __shfl_xor_sync(0xffffffffu, db[i][j], o));
        }
    }
  }
  if (gr.sub == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      if (ELEM) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int k = (i * VEC + j) * TPR;
          float g0, g1, b0, b1;
          unpair(dg[i][j / 2], g0, g1);
          unpair(db[i][j / 2], b0, b1);
          if (k < left) {
            mine[t + k] = j & 1 ? g1 : g0;
            mine[d + t + k] = j & 1 ? b1 : b0;
          }
        }
      } else {
        const int c = (i * tpr + t) * VEC;
#pragma unroll
        for (int j = 0; j < P; ++j) {
          *reinterpret_cast<f32x2*>(mine + c + 2 * j) = dg[i][j];
          *reinterpret_cast<f32x2*>(mine + d + c + 2 * j) = db[i][j];
        }
      }
    }
  }
  if (BLOCK) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsPerCta; ++w) v += reinterpret_cast<const float*>(ring_mem + (size_t)w * S * stage)[c];
    out[c] = v;
  }
}

// dX of rows too wide for registers (two passes over the row).
template <typename T, typename TP>
__global__ void __launch_bounds__(1024) k_ln_bwd_wide(const BwdArgs a) {
  __shared__ float2 buf[2][32];
  pdl_begin();
  const TP* gm = (const TP*)a.gamma;
  int turn = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *x = (const T*)a.x + row * a.ldx, *dy = (const T*)a.dy + row * a.lddy;
    const T* dr = a.dr ? (const T*)a.dr + row * a.lddr : nullptr;
    const float mu = a.mean[row], rs = a.rstd[row];
    float sg = 0.f, sgx = 0.f;
    for (long long c = threadIdx.x; c < a.d; c += blockDim.x) {
      const float g = as_f32(dy[c]) * (gm ? as_f32(gm[c]) : 1.f);
      sg += g;
      sgx = fmaf(g, (as_f32(x[c]) - mu) * rs, sgx);
    }
    const float2 s = block_sum2(sg, sgx, buf, turn);
    sg = s.x / (float)a.d;
    sgx = s.y / (float)a.d;
    for (long long c = threadIdx.x; c < a.d; c += blockDim.x) {
      const float g = as_f32(dy[c]) * (gm ? as_f32(gm[c]) : 1.f);
      float e = rs * (g - sg - (as_f32(x[c]) - mu) * rs * sgx);
      if (dr) e += as_f32(dr[c]);
      ((T*)a.dx)[row * a.lddx + c] = from_f32<T>(e);
    }
  }
}

// dgamma and dbeta straight from X and dY, 32 columns a CTA and the rows
// dealt to its 32 warps: what runs without a workspace, or for rows too wide
// for registers.
template <typename T>
__global__ void __launch_bounds__(1024) k_ln_bwd_cols(const BwdArgs a, void* dgamma, void* dbeta, int pf32,
                                                      int accumulate) {
  __shared__ float sg[32][33], sb[32][33];
  pdl_begin();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long c = (long long)blockIdx.x * 32 + lane;
  float g = 0.f, b = 0.f;
  if (c < a.d)
    for (long long row = w; row < a.rows; row += 32) {
      const float y = as_f32(((const T*)a.dy)[row * a.lddy + c]);
      g = fmaf(y, (as_f32(((const T*)a.x)[row * a.ldx + c]) - a.mean[row]) * a.rstd[row], g);
      b += y;
    }
  sg[w][lane] = g;
  sb[w][lane] = b;
  __syncthreads();
  if (w >= 2 || c >= a.d) return;
  void* out = w ? dbeta : dgamma;
  if (!out) return;
  float v = 0.f;
  for (int i = 0; i < 32; ++i) v += w ? sb[i][lane] : sg[i][lane];
  if (pf32) {
    float* o = (float*)out + c;
    *o = accumulate ? *o + v : v;
  } else {
    __nv_bfloat16* o = (__nv_bfloat16*)out + c;
    *o = __float2bfloat16_rn(accumulate ? __bfloat162float(*o) + v : v);
  }
}

// dgamma and dbeta from the CTAs' column sums: 32 columns a CTA, the n sums of
// a column dealt to its warps and added in a fixed order.  The sums are in L2;
// 9 us for 296 of 5120 columns, of which the call sees less: the launch and
// first loads hide behind the pass before it.
template <int kReduceWarps>
__global__ void __launch_bounds__(32 * kReduceWarps) k_ln_bwd_reduce(const float* part, int n, long long d,
                                                                     void* dgamma, void* dbeta, int pf32,
                                                                     int accumulate) {
  __shared__ float acc[kReduceWarps][33];
  pdl_begin();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long c = (long long)blockIdx.x * 32 + lane;
  void* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  float v = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int i = w; i < n; i += kReduceWarps) v += part[((long long)i * 2 + blockIdx.y) * d + c];
  }
  acc[w][lane] = v;
  __syncthreads();
  if (w || c >= d) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kReduceWarps; ++i) v += acc[i][lane];
  if (pf32) {
    float* o = (float*)out + c;
    *o = accumulate ? *o + v : v;
  } else {
    __nv_bfloat16* o = (__nv_bfloat16*)out + c;
    *o = __float2bfloat16_rn(accumulate ? __bfloat162float(*o) + v : v);
  }
}

// ------------------------------------------------------------------ planning
struct Plan {
  bool elem;    // element by element (rows that start anywhere), else 16-byte vectors
  int nv;       // vectors a thread
  bool block;   // the CTA a row (else a warp, or lpr lanes of one)
  int threads;  // CTA size
  int lpr;
  bool wide;    // the row does not fit: the kernels that walk it several times
  int stages, per_sm;  // the ring, and CTAs a SM
  size_t bytes;        // the rings' shared memory
  size_t gamma;        // and gamma's behind it (backward)
};

// A warp takes a row of up to 4 vectors a lane (12288 x 768 bf16: forward 16.1
// us against 19.7 with a CTA a row, backward 22.5 against 31.2), several rows
// of up to half a vector a lane (30000 x 64: 6.0 against 14.0 with a row a
// warp, backward 9.4 against 18.3), a CTA one of 16 elements a thread.  A SM
// holds up to 1024 threads of such CTAs forward (2048 x 4096 fp32: 17.0 us
// against 20.5 with 512) and 640 backward (32768 x 5120: 208 against 290 with
// 320; each CTA leaves a row of column sums).  ``arrays``: input arrays of a
// stage (3 for the backward); pes: bytes of a gamma element.
static Plan plan(long long d, int es, bool aligned, int arrays, int pes) {
  Plan p = {};
  const int vec = 16 / es;
  p.elem = !(aligned && (d * es) % 16 == 0);
  p.wide = d == 0 || d > (p.elem ? 512 * 16 : 1024 * 16);  // (no element: only the statistics, 0 / 0)
  p.block = !p.wide && d > (p.elem ? 32 * 16 : 32 * 4 * vec);
  p.nv = 1;
  p.lpr = 32;
  p.threads = 32 * kRowsPerCta;
  if (!p.wide && !p.block) {
    while (p.nv * 32 * vec < d) ++p.nv;
    if (p.elem && p.nv == 3) p.nv = 4;
    if (!p.elem)
      while (p.nv == 1 && p.lpr > 4 && p.lpr / 2 * vec >= d) p.lpr /= 2;
  } else if (p.block) {
    p.nv = 16 / vec;
    p.threads = (int)((d + 16 * 32 - 1) / (16 * 32)) * 32;
    if (p.elem) {  // 64, 128, 256 or 512 threads: the offsets are then constants
      int th = 64;
      while (th < p.threads) th *= 2;
      p.threads = th;
    }
  }
  if (!p.wide) {
    const size_t stage = (size_t)region_bytes(d, es, 32 / p.lpr, p.elem) * arrays * (p.block ? 1 : kRowsPerCta);
    constexpr size_t kSm = 226 * 1024;  // of 227 KB; the static arrays take the rest
    p.gamma = arrays == 3 && !p.elem ? (size_t)d * pes : 0;
    const bool bwd = arrays == 3;
    const int most = p.threads <= 128 ? (bwd ? 8 : 16) : (bwd ? 2 : 4);
    int want = p.block ? (bwd ? 640 : 1024) / p.threads : 2;
    want = want < 1 ? 1 : want > most ? most : want;
    for (p.per_sm = want; p.per_sm > 1; --p.per_sm)
      if (2 * stage + p.gamma <= kSm / p.per_sm - 1024) break;
    const size_t room = kSm / p.per_sm - (p.per_sm > 1 ? 1024 : 0);  // 1 KB of every CTA's is the system's
    p.stages = room > p.gamma ? (int)((room - p.gamma) / stage) : 0;
    if (p.stages > kMaxRing) p.stages = kMaxRing;
    p.bytes = p.stages * stage;
    // the warps' column sums go where their rings were
    if (p.stages < 2 || (!p.block && arrays == 3 && 2 * d * 4 > (long long)(p.bytes / kRowsPerCta))) p.wide = true;
  }
  if (p.wide) {
    p.block = true;
    p.threads = 1024;
    p.per_sm = 2;
  }
  return p;
}

static int grid_of(const Plan& p, long long rows) {
  const long long per = p.block ? 1 : (long long)kRowsPerCta * (32 / p.lpr);
  const long long most = (long long)device_sms() * p.per_sm, n = (rows + per - 1) / per;
  return (int)(n < most ? n : most);
}

static bool rows_aligned(const aal_mat& m) {
  const size_t es = m.dtype == AAL_F32 ? 4 : 2;
  return !m.ptr || (((uintptr_t)m.ptr % 16) == 0 && (m.rows <= 1 || (m.ld * es) % 16 == 0));
}

// Raises kernel K's limit of dynamic shared memory on the current device to all
// that its static arrays leave, once (the driver call costs as much as a short
// kernel).  Without it 48 KB hold, of static and dynamic memory together: what
// a launch may ask for then depends on the kernel's static arrays, so every
// kernel with dynamic memory is raised, whatever its first launch needs.
template <auto K>
static cudaError_t allow_shared(size_t bytes) {
  constexpr int kDevices = 64;
  static std::atomic<size_t> allowed[kDevices];
  if (bytes == 0) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<size_t>* a = dev >= 0 && dev < kDevices ? &allowed[dev] : nullptr;
  if (a && a->load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  // two threads may come here together: both raise the limit to the same value
  int most = 0;
  e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  cudaFuncAttributes f;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&f, K);
  if (e != cudaSuccess) return e;
  const size_t limit = (size_t)most - f.sharedSizeBytes;
  if (bytes > limit) return cudaErrorInvalidValue;
  e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)limit);
  if (e == cudaSuccess && a) a->store(limit, std::memory_order_relaxed);
  return e;
}

// A launch that may start while the stream's previous kernel still runs (the
// kernels wait for it before they touch what it writes); ``cluster`` > 0 sets a
// cluster size at launch.
template <auto K, typename... A>
static aal_status launch_pdl(dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, A... args) {
  if (const aal_status st = cuda_status(allow_shared<K>(smem)); st != AAL_OK) return st;
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, K, args...);
  note_launch();
  return cuda_status(e);
}

// Calls f with the kernel's compile-time shape: vectors a thread, threads a
// row, several rows a warp, the element form, the largest CTA and CTAs a SM.
// The forward's wide rows run two CTAs of 512 threads a SM (64 registers); the
// backward's column sums need more registers than that leaves.
template <typename T, bool BWD, typename F>
static aal_status with_shape(const Plan& p, F f) {
  constexpr int W = 32 * kRowsPerCta, N = 16 / Vec<T>::n;
  if (p.elem) {
    if (p.block) {
      switch (p.threads) {
        case 64: return f.template run<N, 64, false, true, 64, 8>();
        case 128: return f.template run<N, 128, false, true, 128, 4>();
        case 256: return f.template run<N, 256, false, true, 256, 2>();
        default: return f.template run<N, 512, false, true, 512, BWD ? 1 : 2>();
      }
    }
    switch (p.nv) {
      case 1: return f.template run<1, 32, false, true, W, 2>();
      case 2: return f.template run<2, 32, false, true, W, 2>();
      default: return f.template run<N, 32, false, true, W, 2>();
    }
  }
  if (p.block) {
    if constexpr (BWD) {
      if (p.threads <= 320) return f.template run<N, 0, false, false, 320, 2>();
    }
    return p.threads <= 512 ? f.template run<N, 0, false, false, 512, BWD ? 1 : 2>()
                            : f.template run<N, 0, false, false, 1024, 1>();
  }
  switch (p.nv) {
    case 1:
      return p.lpr < 32 ? f.template run<1, 32, true, false, W, 2>() : f.template run<1, 32, false, false, W, 2>();
    case 2: return f.template run<2, 32, false, false, W, 2>();
    case 3: return f.template run<3, 32, false, false, W, 2>();
    default: return f.template run<4, 32, false, false, W, 2>();
  }
}

template <typename T, typename TP>
struct FwdLaunch {
  FwdArgs a;
  const Plan& p;
  cudaStream_t s;
  template <int NV, int TPR, bool SUB, bool ELEM, int MAXT, int MINB>
  aal_status run() {
    a.ring = p.stages;
    a.lpr = p.lpr;
    return launch_pdl<k_ln_fwd<T, TP, NV, TPR, SUB, ELEM, MAXT, MINB>>(dim3((unsigned)grid_of(p, a.rows)), p.threads, p.bytes, 0,
                                                                       s, a);
  }
};
template <typename T, typename TP>
static aal_status run_fwd(const FwdArgs& a, const Plan& p, cudaStream_t s) {
  if (p.wide) return launch_pdl<k_ln_fwd_wide<T, TP>>(dim3((unsigned)grid_of(p, a.rows)), p.threads, 0, 0, s, a);
  return with_shape<T, false>(p, FwdLaunch<T, TP>{a, p, s});
}

template <typename T, typename TP>
struct BwdLaunch {
  BwdArgs a;
  const Plan& p;
  cudaStream_t s;
  template <int NV, int TPR, bool SUB, bool ELEM, int MAXT, int MINB>
  aal_status run() {
    a.ring = p.stages;
    a.lpr = p.lpr;
    a.ring_bytes = (uint32_t)p.bytes;
    return launch_pdl<k_ln_bwd<T, TP, NV, TPR, SUB, ELEM, MAXT, MINB>>(dim3((unsigned)grid_of(p, a.rows)), p.threads,
                                                                       p.bytes + p.gamma, 0, s, a);
  }
};

// A parameter vector (gamma, beta or a gradient of one): [1, d], the call's
// dtype or fp32; a null pointer stands for one that is not there.
static bool valid_vec(const aal_mat& m, long long d, int dtype) {
  if (!m.ptr) return true;
  return valid_mat(m) && m.rows == 1 && m.cols == d && (m.dtype == dtype || m.dtype == AAL_F32);
}

// Partial column sums of the backward: CTAs times two rows of d floats.
static long long bwd_part_bytes(long long rows, long long d, int es, bool aligned, int pes) {
  const Plan p = plan(d, es, aligned, 3, pes);
  return p.wide ? 0 : (long long)grid_of(p, rows) * 2 * d * 4;
}

}  // namespace norm
}  // namespace aal

using namespace aal;

extern "C" {

aal_status aal_layer_norm_fwd(aal_mat X, aal_mat R, aal_mat gamma, aal_mat beta, float eps, aal_mat S, aal_mat Y,
                              float* mean, float* rstd, void* stream) {
  const int dt = X.dtype;
  const long long M = X.rows, d = X.cols;
  if (!valid_mat(X) || !valid_mat(Y) || (R.ptr && !valid_mat(R)) || (S.ptr && !valid_mat(S)))
    return AAL_ERR_INVALID_ARG;
  if (Y.dtype != dt || (R.ptr && R.dtype != dt) || (S.ptr && S.dtype != dt)) return AAL_ERR_UNSUPPORTED;
  auto is = [&](const aal_mat& m) { return m.rows == M && m.cols == d; };
  if (!is(Y) || (R.ptr && !is(R)) || (S.ptr && !is(S)) || (S.ptr && !R.ptr)) return AAL_ERR_INVALID_ARG;
  if (!norm::valid_vec(gamma, d, dt) || !norm::valid_vec(beta, d, dt)) return AAL_ERR_INVALID_ARG;
  if (gamma.ptr && beta.ptr && gamma.dtype != beta.dtype) return AAL_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || isinf(eps)) return AAL_ERR_INVALID_ARG;
  if (((uintptr_t)mean | (uintptr_t)rstd) % 4) return AAL_ERR_INVALID_ARG;
  if (M > 0 && d > 0 && S.ptr && S.ptr == Y.ptr) return AAL_ERR_INVALID_ARG;
  note_path(0);
  if (M == 0 || (d == 0 && !mean && !rstd)) return AAL_OK;
  const int pdt = gamma.ptr ? gamma.dtype : beta.ptr ? beta.dtype : dt;
  const bool al = norm::rows_aligned(X) && norm::rows_aligned(R) && norm::rows_aligned(S) && norm::rows_aligned(Y) &&
                  norm::rows_aligned(gamma) && norm::rows_aligned(beta);
  const norm::Plan p = norm::plan(d, dt == AAL_F32 ? 4 : 2, al, R.ptr ? 2 : 1, 0);
  norm::FwdArgs a = {X.ptr, R.ptr, gamma.ptr, beta.ptr, S.ptr, Y.ptr, mean, rstd, M, d, X.ld, R.ld, S.ld, Y.ld, eps, 0, 0};
  cudaStream_t s = (cudaStream_t)stream;
  const aal_status st = timed(AAL_KERNEL_NORM_FWD, s, [&] {
    if (dt == AAL_F32) return norm::run_fwd<float, float>(a, p, s);
    if (pdt == AAL_F32) return norm::run_fwd<__nv_bfloat16, float>(a, p, s);
    return norm::run_fwd<__nv_bfloat16, __nv_bfloat16>(a, p, s);
  });
  if (st == AAL_OK) note_path(AAL_PATH_GENERAL);
  return st;
}

int64_t aal_layer_norm_bwd_workspace_size(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return -1;
  if (rows == 0 || cols == 0) return 0;
  // the largest of what the element types and alignments need
  long long n = 0;
  for (int es = 2; es <= 4; es += 2)
    for (int al = 0; al < 2; ++al)
      for (int pes = es; pes <= 4; pes += 2) {
        const long long b = norm::bwd_part_bytes(rows, cols, es, al != 0, pes);
        n = b > n ? b : n;
      }
  return n;
}

aal_status aal_layer_norm_bwd(aal_mat X, aal_mat gamma, const float* mean, const float* rstd, aal_mat dY, aal_mat dR,
                              aal_mat dX, aal_mat dgamma, aal_mat dbeta, int32_t accumulate, void* stream) {
  const int dt = X.dtype;
  const long long M = X.rows, d = X.cols;
  if (!valid_mat(X) || !valid_mat(dY) || (dR.ptr && !valid_mat(dR)) || (dX.ptr && !valid_mat(dX)))
    return AAL_ERR_INVALID_ARG;
  if (dY.dtype != dt || (dR.ptr && dR.dtype != dt) || (dX.ptr && dX.dtype != dt)) return AAL_ERR_UNSUPPORTED;
  auto is = [&](const aal_mat& m) { return m.rows == M && m.cols == d; };
  if (!is(dY) || (dR.ptr && !is(dR)) || (dX.ptr && !is(dX)) || (dR.ptr && !dX.ptr)) return AAL_ERR_INVALID_ARG;
  if (!norm::valid_vec(gamma, d, dt) || !norm::valid_vec(dgamma, d, dt) || !norm::valid_vec(dbeta, d, dt))
    return AAL_ERR_INVALID_ARG;
  if (dgamma.ptr && dbeta.ptr && (dgamma.dtype != dbeta.dtype || dgamma.ptr == dbeta.ptr)) return AAL_ERR_INVALID_ARG;
  if (M > 0 && (!mean || !rstd)) return AAL_ERR_INVALID_ARG;
  if (((uintptr_t)mean | (uintptr_t)rstd) % 4) return AAL_ERR_INVALID_ARG;
  note_path(0);
  const bool cols = dgamma.ptr || dbeta.ptr;
  if (d == 0 || (!cols && (M == 0 || !dX.ptr))) return AAL_OK;
  cudaStream_t s = (cudaStream_t)stream;
  const int pf32 = (dgamma.ptr ? dgamma.dtype : dbeta.dtype) == AAL_F32;
  const int gdt = gamma.ptr ? gamma.dtype : dt;
  const bool al = norm::rows_aligned(X) && norm::rows_aligned(dY) && norm::rows_aligned(dR) &&
                  norm::rows_aligned(dX) && norm::rows_aligned(gamma);
  const norm::Plan p = norm::plan(d, dt == AAL_F32 ? 4 : 2, al, 3, gdt == AAL_F32 ? 4 : 2);
  norm::BwdArgs a = {X.ptr, gamma.ptr, dY.ptr, dR.ptr, mean, rstd, dX.ptr, nullptr, M, d, X.ld, dY.ld, dR.ld, dX.ld, 0, 0, 0};
  const int grid = norm::grid_of(p, M);
  const unsigned gx = (unsigned)((d + 31) / 32);
  if ((d + 31) / 32 > 0x7fffffffLL) return AAL_ERR_UNSUPPORTED;
  uint64_t have = 0;
  float* ws = (float*)current_workspace(&have);
  const bool parts = cols && M > 0 && !p.wide && ws && have >= (uint64_t)grid * 2 * d * 4;
  const aal_status st = timed(AAL_KERNEL_NORM_BWD, s, [&] {
    aal_status e = AAL_OK;
    if (cols && M > 0 && !parts) {  // first: dX may be written over X, dY or dR
      e = dt == AAL_F32 ? norm::launch_pdl<norm::k_ln_bwd_cols<float>>(dim3(gx), 1024, 0, 0, s, a, dgamma.ptr, dbeta.ptr, pf32,
                                                                    (int)accumulate)
                        : norm::launch_pdl<norm::k_ln_bwd_cols<__nv_bfloat16>>(dim3(gx), 1024, 0, 0, s, a, dgamma.ptr, dbeta.ptr, pf32,
                                                                            (int)accumulate);
    }
    a.part = parts ? ws : nullptr;
    if (e == AAL_OK && M > 0 && (dX.ptr || parts)) {
      if (p.wide) {  // (without column sums: parts is false)
        const dim3 g((unsigned)grid);
        e = dt == AAL_F32     ? norm::launch_pdl<norm::k_ln_bwd_wide<float, float>>(g, p.threads, 0, 0, s, a)
            : gdt == AAL_F32 ? norm::launch_pdl<norm::k_ln_bwd_wide<__nv_bfloat16, float>>(g, p.threads, 0, 0, s, a)
                             : norm::launch_pdl<norm::k_ln_bwd_wide<__nv_bfloat16, __nv_bfloat16>>(g, p.threads, 0, 0, s, a);
      } else if (dt == AAL_F32) {
        e = norm::with_shape<float, true>(p, norm::BwdLaunch<float, float>{a, p, s});
      } else if (gdt == AAL_F32) {
        e = norm::with_shape<__nv_bfloat16, true>(p, norm::BwdLaunch<__nv_bfloat16, float>{a, p, s});
      } else {
        e = norm::with_shape<__nv_bfloat16, true>(p, norm::BwdLaunch<__nv_bfloat16, __nv_bfloat16>{a, p, s});
      }
    }
    if (e == AAL_OK && cols && (parts || M == 0)) {
      // few sums are sooner added by few warps (96 of 2048 columns: 7.4 us for
      // the call against 9.5; 296 of 768: 24.0 against 22.5 with many)
      const int n = M == 0 ? 0 : grid;
      e = n <= 128 ? norm::launch_pdl<norm::k_ln_bwd_reduce<8>>(dim3(gx, 2), 256, 0, 0, s, (const float*)ws, n, (long long)d,
                                                                dgamma.ptr, dbeta.ptr, pf32, (int)accumulate)
                   : norm::launch_pdl<norm::k_ln_bwd_reduce<32>>(dim3(gx, 2), 1024, 0, 0, s, (const float*)ws, n, (long long)d,
                                                                 dgamma.ptr, dbeta.ptr, pf32, (int)accumulate);
    }
    return e;
  });
  if (st == AAL_OK) note_path(AAL_PATH_GENERAL);
  return st;
}

}  // extern "C"
