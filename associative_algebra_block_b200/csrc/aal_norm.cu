// Layer norm of the rows of a matrix, forward and backward: the norm ahead of
// the feed-forward block (and, with R, the residual add that precedes it).
//
//   s = x (+ r),  mu = mean(s),  v = mean((s - mu)^2),  rstd = 1 / sqrt(v + eps)
//   y = (s - mu) rstd gamma + beta
//   backward, with xh = (s - mu) rstd and g = dy gamma:
//   dx = rstd (g - mean(g) - xh mean(g xh)) (+ dr)
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Every byte of the matrices crosses HBM once: a row lives in registers from
// its load to its store (up to 4 vectors a thread), the variance is the mean
// of the squared distances from the mean (no cancellation), and the backward
// keeps dgamma and dbeta of a thread's own columns in fp32 registers over all
// the rows its CTA visits.  The CTAs' column sums go to the caller's workspace
// and a second, programmatically dependent launch adds them in CTA order, so
// results do not depend on timing.
#include "aal_internal.h"

#include <math.h>

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
// The vector kernels bring their rows in with bulk asynchronous copies: a
// group (the warp of a narrow row, the CTA of a wide one) owns a ring of
// stages, each one row of every input array, and one of its threads refills a
// stage as soon as the group is done with it, so the next rows are in flight
// while one is reduced.  That keeps about 100 KB a SM moving with 16 warps,
// which plain loads could not: their registers held one row a warp and nothing
// moved during the reductions.
constexpr int kMaxRing = 4;
constexpr unsigned long long kRingWaitNs = 2000000000ull;

__device__ __forceinline__ void ring_init(uint64_t* bar) { tc::mbar_init(bar, 1); }
__device__ __forceinline__ void ring_init_done() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  tc::fence_async_smem();
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}
// Bounded wait for a stage.  A copy that has not landed after two seconds
// never will: the status word is set and the caller goes on with what is
// there, so that every thread still reaches the kernel's barriers.
__device__ __forceinline__ void ring_wait(uint64_t* bar, uint32_t parity) {
  if (tc::mbar_try_wait(bar, parity)) return;
  const unsigned long long t0 = tc::gtime();
  for (uint32_t i = 0; !tc::mbar_try_wait(bar, parity); ++i)
    if ((i & 255u) == 255u && tc::gtime() - t0 > kRingWaitNs) {
      flag_device_error(kDevTimeout);
      return;
    }
}

struct FwdArgs {
  const void *x, *r, *gamma, *beta;
  void *s, *y;
  float *mean, *rstd;
  long long rows, d, ldx, ldr, lds, ldy;
  float eps;
  int ring;  // stages of the pipelined kernels
};

constexpr int kRowsPerCta = 8;  // warp-per-row kernels: one row a warp

// The vector kernel: NV 16-byte vectors a thread, at most MAXT threads.
template <typename T, typename TP, int NV, bool BLOCK, int MAXT>
__global__ void __launch_bounds__(MAXT, BLOCK ? 1 : 2) k_ln_fwd_ring(const FwdArgs a) {
  constexpr int VEC = Vec<T>::n, P = Vec<T>::pairs;
  extern __shared__ __align__(128) unsigned char ring_mem[];
  __shared__ float2 buf[2][32];
  __shared__ __align__(8) uint64_t bars[(BLOCK ? 1 : kRowsPerCta) * kMaxRing];
  const int tpr = BLOCK ? (int)blockDim.x : 32;
  const int t = BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & 31);
  const int group = BLOCK ? 0 : (int)(threadIdx.x >> 5);
  const long long r0 = BLOCK ? blockIdx.x : (long long)blockIdx.x * kRowsPerCta + group;
  const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * kRowsPerCta;
  const T *x = (const T*)a.x, *r = (const T*)a.r;
  const TP *gm = (const TP*)a.gamma, *bt = (const TP*)a.beta;
  const int d = (int)a.d, S = a.ring;
  const uint32_t bytes = (uint32_t)(d * sizeof(T));
  const uint32_t stage = bytes * (r ? 2u : 1u);
  unsigned char* mem = ring_mem + (size_t)group * S * stage;
  uint64_t* bar = bars + group * kMaxRing;
  if (t == 0) {
    for (int i = 0; i < S; ++i) ring_init(&bar[i]);
    ring_init_done();
  }
  pdl_begin();
  auto fill = [&](long long row, int st) {
    tc::mbar_expect_tx(&bar[st], stage);
    const uint32_t dst = tc::smem_u32(mem) + st * stage;
    bulk_load(dst, x + row * a.ldx, bytes, &bar[st]);
    if (r) bulk_load(dst + bytes, r + row * a.ldr, bytes, &bar[st]);
  };
  if (t == 0)
    for (int i = 0; i < S; ++i)
      if (r0 + i * step < a.rows) fill(r0 + i * step, i);
  if (BLOCK) __syncthreads();
  else __syncwarp();
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = (i * tpr + t) * VEC < d;
  Param<T, TP> pg[NV], pb[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (in[i]) {
      if (gm) pg[i].load(gm + (i * tpr + t) * VEC);
      if (bt) pb[i].load(bt + (i * tpr + t) * VEC);
    }
  const float inv_d = 1.0f / (float)d;
  int turn = 0, st = 0, before = S - 1;  // this row's stage and the previous row's
  uint32_t ph = 0;
  for (long long row = r0; row < a.rows; row += step) {
    ring_wait(&bar[st], ph);
    const unsigned char* m = mem + (size_t)st * stage + t * 16;
    f32x2 v[NV][P];
    f32x2 sum = 0;  // two zeros
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < P; ++j) v[i][j] = 0;
      if (in[i]) {
        widen(*reinterpret_cast<const uint4*>(m + i * tpr * 16), v[i], T());
        if (r) {
          f32x2 w[P];
          widen(*reinterpret_cast<const uint4*>(m + bytes + i * tpr * 16), w, T());
#pragma unroll
          for (int j = 0; j < P; ++j) v[i][j] = add2(v[i][j], w[j]);
        }
#pragma unroll
        for (int j = 0; j < P; ++j) sum = add2(sum, v[i][j]);
      }
    }
    float mu;
    if (BLOCK) {
      mu = block_sum2(sum2(sum), 0.f, buf, turn).x * inv_d;
      // past that barrier every thread is done with the previous row's stage
      const long long next = row + (S - 1) * step;
      if (t == 0 && row != r0 && next < a.rows) fill(next, before);
    } else {
      mu = warp_sum(sum2(sum)) * inv_d;
      const long long next = row + S * step;
      if (t == 0 && next < a.rows) fill(next, st);  // the row is in registers
    }
    before = st;
    if (++st == S) { st = 0; ph ^= 1u; }
    const f32x2 nmu = pair(-mu, -mu);
    f32x2 sq = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const f32x2 e = add2(v[i][j], nmu);
          sq = fma2(e, e, sq);
        }
      }
    const float var = (BLOCK ? block_sum2(sum2(sq), 0.f, buf, turn).x : warp_sum(sum2(sq))) * inv_d;
    const float rs = 1.0f / sqrtf(var + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = rs;
    }
    const f32x2 rs2 = pair(rs, rs);
    T* yo = (T*)a.y + row * a.ldy + t * VEC;
    T* so = (T*)a.s + row * a.lds + t * VEC;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      // the stored sum is rounded to the matrix type; the norm itself uses
      // the unrounded one
      if (a.s) *reinterpret_cast<uint4*>(so + i * tpr * VEC) = narrow(v[i], T());
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
      *reinterpret_cast<uint4*>(yo + i * tpr * VEC) = narrow(e, T());
    }
  }
}

// The element-by-element kernel, for rows that start anywhere: TPR threads a
// row (a warp, kRowsPerCta rows a CTA, or the CTA), NV elements a thread.
template <typename T, typename TP, int NV, int TPR>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kRowsPerCta : TPR) k_ln_fwd(const FwdArgs a) {
  constexpr bool BLOCK = TPR > 32;
  __shared__ float2 buf[2][32];
  pdl_begin();
  const int t = (int)threadIdx.x % TPR;
  const long long r0 = BLOCK ? blockIdx.x : (long long)blockIdx.x * kRowsPerCta + (threadIdx.x >> 5);
  const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * kRowsPerCta;
  const TP *gm = (const TP*)a.gamma, *bt = (const TP*)a.beta;
  const int left = (int)a.d - t;  // element i of this thread is i * TPR < left
  const float inv_d = 1.0f / (float)(int)a.d;
  float g[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    g[i] = gm && i * TPR < left ? as_f32(gm[i * TPR + t]) : 1.f;
    b[i] = bt && i * TPR < left ? as_f32(bt[i * TPR + t]) : 0.f;
  }
  int turn = 0;
  for (long long row = r0; row < a.rows; row += step) {
    const T* x = (const T*)a.x + row * a.ldx + t;
    float v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = i * TPR < left ? as_f32(x[i * TPR]) : 0.f;
    if (a.r) {
      const T* r = (const T*)a.r + row * a.ldr + t;
      T w[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * TPR < left) w[i] = r[i * TPR];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * TPR < left) v[i] += as_f32(w[i]);
    }
    float sum = 0.f, sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) sum += v[i];
    const float mu = (BLOCK ? block_sum2(sum, 0.f, buf, turn).x : warp_sum(sum)) * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * TPR < left) sq = fmaf(v[i] - mu, v[i] - mu, sq);
    const float var = (BLOCK ? block_sum2(sq, 0.f, buf, turn).x : warp_sum(sq)) * inv_d;
    const float rs = 1.0f / sqrtf(var + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = rs;
    }
    if (a.s) {
      T* so = (T*)a.s + row * a.lds + t;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * TPR < left) so[i * TPR] = from_f32<T>(v[i]);
    }
    T* yo = (T*)a.y + row * a.ldy + t;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * TPR < left) yo[i * TPR] = from_f32<T>((v[i] - mu) * rs * g[i] + b[i]);
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
  int ring;  // stages of the pipelined kernels
};

// dx = rstd (g - mean(g) - xh mean(g xh)) as g rstd + A + B x with
// A = rstd (mean xh-term, below) and B = -rstd^2 mean(g xh): the row's two
// numbers are folded once instead of recomputing xh for every element.
struct RowFold {
  float A, B;
};
__device__ __forceinline__ RowFold fold_row(float mu, float rs, float mg, float mgx) {
  RowFold f;
  f.B = -rs * rs * mgx;
  f.A = -rs * mg - f.B * mu;
  return f;
}

template <typename T, typename TP, int NV, bool BLOCK, int MAXT>
__global__ void __launch_bounds__(MAXT, BLOCK ? 1 : 2) k_ln_bwd_ring(const BwdArgs a) {
  constexpr int VEC = Vec<T>::n, P = Vec<T>::pairs;
  extern __shared__ __align__(128) unsigned char ring_mem[];
  __shared__ float2 buf[2][32];
  __shared__ __align__(8) uint64_t bars[(BLOCK ? 1 : kRowsPerCta) * kMaxRing];
  const int tpr = BLOCK ? (int)blockDim.x : 32;
  const int t = BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & 31);
  const int group = BLOCK ? 0 : (int)(threadIdx.x >> 5);
  const long long r0 = BLOCK ? blockIdx.x : (long long)blockIdx.x * kRowsPerCta + group;
  const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * kRowsPerCta;
  const T *x = (const T*)a.x, *dy = (const T*)a.dy, *dr = (const T*)a.dr;
  const TP* gm = (const TP*)a.gamma;
  const int d = (int)a.d, S = a.ring;
  const uint32_t bytes = (uint32_t)(d * sizeof(T));
  const uint32_t stage = bytes * (dr ? 3u : 2u);
  unsigned char* mem = ring_mem + (size_t)group * S * stage;
  uint64_t* bar = bars + group * kMaxRing;
  if (t == 0) {
    for (int i = 0; i < S; ++i) ring_init(&bar[i]);
    ring_init_done();
  }
  pdl_begin();
  auto fill = [&](long long row, int st) {
    tc::mbar_expect_tx(&bar[st], stage);
    const uint32_t dst = tc::smem_u32(mem) + st * stage;
    bulk_load(dst, x + row * a.ldx, bytes, &bar[st]);
    bulk_load(dst + bytes, dy + row * a.lddy, bytes, &bar[st]);
    if (dr) bulk_load(dst + 2 * bytes, dr + row * a.lddr, bytes, &bar[st]);
  };
  if (t == 0)
    for (int i = 0; i < S; ++i)
      if (r0 + i * step < a.rows) fill(r0 + i * step, i);
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = (i * tpr + t) * VEC < d;
  // gamma waits in shared memory, behind the rings
  TP* gs = reinterpret_cast<TP*>(ring_mem + (size_t)(BLOCK ? 1 : kRowsPerCta) * S * stage);
  if (gm)
    for (int c = threadIdx.x; c < d; c += blockDim.x) gs[c] = gm[c];
  const uint32_t gsa = tc::smem_u32(gs) + t * VEC * (uint32_t)sizeof(TP);
  __syncthreads();
  const float inv_d = 1.0f / (float)d;
  f32x2 dg[NV][P], db[NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) dg[i][j] = db[i][j] = 0;
  int turn = 0, st = 0, before = S - 1;
  uint32_t ph = 0;
  float mu = 0.f, rs = 0.f;
  if (r0 < a.rows) {
    mu = a.mean[r0];
    rs = a.rstd[r0];
  }
  for (long long row = r0; row < a.rows; row += step) {
    float mu_next = 0.f, rs_next = 0.f;
    if (row + step < a.rows) {
      mu_next = a.mean[row + step];
      rs_next = a.rstd[row + step];
    }
    ring_wait(&bar[st], ph);
    const uint32_t m = tc::smem_u32(mem) + st * stage + t * 16;
    f32x2 sg = 0, sgx = 0;
    const f32x2 nmu = pair(-mu, -mu), rs2 = pair(rs, rs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      f32x2 xv[P], yv[P], w[P];
      widen(lds128(m + i * tpr * 16), xv, T());
      widen(lds128(m + bytes + i * tpr * 16), yv, T());
      if (gm) {
        Param<T, TP> pg;
        pg.load_shared(gsa + i * tpr * VEC * (uint32_t)sizeof(TP));
        pg.get(w);
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const f32x2 xh = mul2(add2(xv[j], nmu), rs2);
        const f32x2 g = gm ? mul2(yv[j], w[j]) : yv[j];
        sg = add2(sg, g);
        sgx = fma2(g, xh, sgx);
        dg[i][j] = fma2(yv[j], xh, dg[i][j]);
        db[i][j] = add2(db[i][j], yv[j]);
      }
    }
    float mg = sum2(sg), mgx = sum2(sgx);
    if (BLOCK) {
      const float2 s = block_sum2(mg, mgx, buf, turn);
      mg = s.x;
      mgx = s.y;
      // past that barrier every thread is done with the previous row's stage
      const long long next = row + (S - 1) * step;
      if (t == 0 && row != r0 && next < a.rows) fill(next, before);
    } else {
      mg = warp_sum(mg);
      mgx = warp_sum(mgx);
    }
    if (a.dx) {
      const RowFold f = fold_row(mu, rs, mg * inv_d, mgx * inv_d);
      const f32x2 A = pair(f.A, f.A), B = pair(f.B, f.B);
      T* o = (T*)a.dx + row * a.lddx + t * VEC;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!in[i]) continue;
        f32x2 xv[P], yv[P], w[P];
        widen(lds128(m + i * tpr * 16), xv, T());
        widen(lds128(m + bytes + i * tpr * 16), yv, T());
        if (gm) {
          Param<T, TP> pg;
          pg.load_shared(gsa + i * tpr * VEC * (uint32_t)sizeof(TP));
          pg.get(w);
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const f32x2 g = gm ? mul2(yv[j], w[j]) : yv[j];
          xv[j] = fma2(g, rs2, fma2(xv[j], B, A));
        }
        if (dr) {
          widen(lds128(m + 2 * bytes + i * tpr * 16), w, T());
#pragma unroll
          for (int j = 0; j < P; ++j) xv[j] = add2(xv[j], w[j]);
        }
        *reinterpret_cast<uint4*>(o + i * tpr * VEC) = narrow(xv, T());
      }
    }
    if (!BLOCK) {
      __syncwarp();
      const long long next = row + S * step;
      if (t == 0 && next < a.rows) fill(next, st);
    }
    before = st;
    if (++st == S) { st = 0; ph ^= 1u; }
    mu = mu_next;
    rs = rs_next;
  }
  if (!a.part) return;
  float* out = a.part + (long long)blockIdx.x * 2 * d;
  if (BLOCK) {  // every thread has columns of its own
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      const int c = (i * tpr + t) * VEC;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        *reinterpret_cast<f32x2*>(out + c + 2 * j) = dg[i][j];
        *reinterpret_cast<f32x2*>(out + d + c + 2 * j) = db[i][j];
      }
    }
    return;
  }
  // a warp's sums go where its ring was (a ring of two rows holds them), then
  // the CTA adds its warps' in order
  float* mine = reinterpret_cast<float*>(mem);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!in[i]) continue;
    const int c = (i * 32 + t) * VEC;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      *reinterpret_cast<f32x2*>(mine + c + 2 * j) = dg[i][j];
      *reinterpret_cast<f32x2*>(mine + d + c + 2 * j) = db[i][j];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsPerCta; ++w) v += reinterpret_cast<const float*>(ring_mem + (size_t)w * S * stage)[c];
    out[c] = v;
  }
}

template <typename T, typename TP, int NV, int TPR>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kRowsPerCta : TPR) k_ln_bwd(const BwdArgs a) {
  constexpr bool BLOCK = TPR > 32;
  __shared__ float2 buf[2][32];
  extern __shared__ float cols[];  // a warp a row: [warps][2][d] column sums
  pdl_begin();
  const int t = (int)threadIdx.x % TPR;
  const long long r0 = BLOCK ? blockIdx.x : (long long)blockIdx.x * kRowsPerCta + (threadIdx.x >> 5);
  const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * kRowsPerCta;
  const TP* gm = (const TP*)a.gamma;
  const int d = (int)a.d, left = d - t;  // element i of this thread is i * TPR < left
  const float inv_d = 1.0f / (float)d;
  float gam[NV], dg[NV], db[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    gam[i] = gm && i * TPR < left ? as_f32(gm[i * TPR + t]) : 1.f;
    dg[i] = db[i] = 0.f;
  }
  int turn = 0;
  for (long long row = r0; row < a.rows; row += step) {
    const T *x = (const T*)a.x + row * a.ldx + t, *dy = (const T*)a.dy + row * a.lddy + t;
    const float mu = a.mean[row], rs = a.rstd[row];
    T px[NV], py[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * TPR < left) {
        px[i] = x[i * TPR];
        py[i] = dy[i * TPR];
      }
    float mg = 0.f, mgx = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * TPR < left) {
        const float xh = (as_f32(px[i]) - mu) * rs, y = as_f32(py[i]), g = y * gam[i];
        mg += g;
        mgx = fmaf(g, xh, mgx);
        dg[i] = fmaf(y, xh, dg[i]);
        db[i] += y;
      }
    if (!a.dx) continue;
    if (BLOCK) {
      const float2 s = block_sum2(mg, mgx, buf, turn);
      mg = s.x;
      mgx = s.y;
    } else {
      mg = warp_sum(mg);
      mgx = warp_sum(mgx);
    }
    const RowFold f = fold_row(mu, rs, mg * inv_d, mgx * inv_d);
    T* o = (T*)a.dx + row * a.lddx + t;
    const T* dr = a.dr ? (const T*)a.dr + row * a.lddr + t : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * TPR < left) {
        float e = fmaf(as_f32(py[i]) * gam[i], rs, fmaf(as_f32(px[i]), f.B, f.A));
        if (dr) e += as_f32(dr[i * TPR]);
        o[i * TPR] = from_f32<T>(e);
      }
  }
  if (!a.part) return;
  float* out = a.part + (long long)blockIdx.x * 2 * d;
  float* mine = BLOCK ? out : cols + (size_t)(threadIdx.x >> 5) * 2 * d;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i * TPR < left) {
      mine[i * TPR + t] = dg[i];
      mine[d + i * TPR + t] = db[i];
    }
  if (BLOCK) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsPerCta; ++w) v += cols[(size_t)w * 2 * d + c];
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
// a column dealt to its warps and added in a fixed order.
constexpr int kReduceWarps = 16;
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
  bool vec;     // 16-byte vectors (the pipelined kernels), else element by element
  int nv;       // vectors (elements) a thread
  bool block;   // the CTA a row (else a warp a row)
  int threads;  // CTA size
  bool wide;    // the row does not fit: the three-pass kernels
};

// Vectors need 16-byte aligned rows and parameters and whole vectors a row;
// other shapes go element by element, still coalesced.  A warp takes a row of
// up to 4 vectors (16 elements) a lane, a CTA one of 16 elements a thread.
static Plan plan(long long d, int es, bool aligned) {
  Plan p;
  p.vec = aligned && (d * es) % 16 == 0;
  const int vec = p.vec ? 16 / es : 1;
  const long long n = (d + vec - 1) / vec;
  const int most = p.vec ? 4 : 16, cta = 16 / vec;  // vectors a lane, vectors a thread of a CTA
  p.wide = n > (p.vec ? 1024LL : 512LL) * cta;
  p.block = p.wide || n > 32LL * most;
  p.nv = 1;
  p.threads = p.wide ? 1024 : 32 * kRowsPerCta;
  if (p.wide) return p;
  if (!p.block) {
    while (p.nv * 32 < n) p.nv = p.vec ? p.nv + 1 : p.nv * 2;
  } else {
    p.nv = cta;
    p.threads = (int)(((n + cta - 1) / cta + 31) / 32 * 32);
    if (!p.vec) {  // 64, 128, 256 or 512 threads: the offsets are then constants
      int th = 64;
      while (th < p.threads) th *= 2;
      p.threads = th;
    }
  }
  return p;
}

static bool rows_aligned(const aal_mat& m) {
  const size_t es = m.dtype == AAL_F32 ? 4 : 2;
  return !m.ptr || (((uintptr_t)m.ptr % 16) == 0 && (m.rows <= 1 || (m.ld * es) % 16 == 0));
}

template <typename... A>
static aal_status launch_pdl(void (*k)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  if (smem > 32 * 1024 &&  // the static arrays count too
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return AAL_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
  note_launch();
  return cuda_status(e);
}

// Calls f with the kernel's compile-time shape.  V: elements of a vector.
template <int V, typename F>
static aal_status with_shape(const Plan& p, F f) {
  constexpr int W = 32 * kRowsPerCta;
  if (!p.vec) {
    if (p.block) {
      switch (p.threads) {
        case 64: return f.template scalar<16, 64>();
        case 128: return f.template scalar<16, 128>();
        case 256: return f.template scalar<16, 256>();
        default: return f.template scalar<16, 512>();
      }
    }
    switch (p.nv) {
      case 1: return f.template scalar<1, 32>();
      case 2: return f.template scalar<2, 32>();
      case 4: return f.template scalar<4, 32>();
      case 8: return f.template scalar<8, 32>();
      default: return f.template scalar<16, 32>();
    }
  }
  if (p.block) return p.threads <= 512 ? f.template ring<16 / V, true, 512>() : f.template ring<16 / V, true, 1024>();
  switch (p.nv) {
    case 1: return f.template ring<1, false, W>();
    case 2: return f.template ring<2, false, W>();
    case 3: return f.template ring<3, false, W>();
    default: return f.template ring<4, false, W>();
  }
}

// Stages of a group's ring and CTAs of a SM: two CTAs a SM where a CTA's
// rings of two stages fit half of its shared memory, and as many stages as
// then fit, up to kMaxRing.
struct Ring {
  int stages;
  int per_sm;
  size_t bytes;
};
static Ring ring_plan(const Plan& p, long long d, int es, int arrays) {
  const size_t extra = arrays == 3 ? (size_t)d * 4 : 0;  // gamma of the backward
  Ring r = {0, 0, 0};
  const size_t stage = (size_t)d * es * arrays * (p.block ? 1 : kRowsPerCta);
  constexpr size_t kSm = 220 * 1024;
  // registers: about 100 a thread of a row's CTA, at most 128 of a warp's row
  int want = p.block ? 640 / p.threads : 2;
  want = want < 1 ? 1 : want > 4 ? 4 : want;
  for (r.per_sm = want; r.per_sm > 1; --r.per_sm)
    if (2 * stage + extra <= kSm / r.per_sm) break;
  r.stages = (int)((kSm / r.per_sm - extra) / stage);
  if (r.stages > kMaxRing) r.stages = kMaxRing;
  r.bytes = r.stages * stage + extra;
  return r;
}

static int grid_of(const Plan& p, long long rows, int per_sm) {
  const long long per = p.block ? 1 : kRowsPerCta;
  const long long most = (long long)device_sms() * per_sm, n = (rows + per - 1) / per;
  return (int)(n < most ? n : most);
}
// CTAs a SM of the kernels without a ring: what their registers allow for the
// forward, few for the backward, whose CTAs each leave a row of column sums.
static int plain_per_sm(const Plan& p, bool bwd) {
  const int fit = 1024 / p.threads;
  const int most = bwd ? 4 : 8;
  return p.wide ? 2 : fit < 1 ? 1 : fit < most ? fit : most;
}
// A row whose ring does not hold two stages takes the three-pass kernels.
static Plan ring_or_wide(Plan p, long long d, int es, int arrays) {
  if (p.vec && !p.wide && ring_plan(p, d, es, arrays).stages < 2) {
    p.wide = p.block = true;
    p.threads = 1024;
  }
  return p;
}
static Plan fwd_plan(long long d, int es, bool aligned) { return ring_or_wide(plan(d, es, aligned), d, es, 2); }
static Plan bwd_plan(long long d, int es, bool aligned) { return ring_or_wide(plan(d, es, aligned), d, es, 3); }
// CTAs of the backward (its workspace holds two rows of sums for each).
static int bwd_grid(const Plan& p, long long rows, long long d, int es) {
  if (!p.vec) return grid_of(p, rows, plain_per_sm(p, true));
  return grid_of(p, rows, ring_plan(p, d, es, 3).per_sm);
}

template <typename T, typename TP>
struct FwdLaunch {
  FwdArgs a;
  const Plan& p;
  cudaStream_t s;
  template <int NV, int TPR>
  aal_status scalar() {
    return launch_pdl(k_ln_fwd<T, TP, NV, TPR>, dim3((unsigned)grid_of(p, a.rows, plain_per_sm(p, false))), p.threads,
                      0, s, a);
  }
  template <int NV, bool BLOCK, int MAXT>
  aal_status ring() {
    const Ring r = ring_plan(p, a.d, sizeof(T), a.r ? 2 : 1);
    a.ring = r.stages;
    return launch_pdl(k_ln_fwd_ring<T, TP, NV, BLOCK, MAXT>,
                      dim3((unsigned)grid_of(p, a.rows, r.per_sm)), p.threads, r.bytes, s, a);
  }
};
template <typename T, typename TP>
static aal_status run_fwd(const FwdArgs& a, const Plan& p, cudaStream_t s) {
  if (p.wide)
    return launch_pdl(k_ln_fwd_wide<T, TP>, dim3((unsigned)grid_of(p, a.rows, 2)), p.threads, 0, s, a);
  return with_shape<16 / sizeof(T)>(p, FwdLaunch<T, TP>{a, p, s});
}

template <typename T, typename TP>
struct BwdLaunch {
  BwdArgs a;
  const Plan& p;
  int grid;
  cudaStream_t s;
  template <int NV, int TPR>
  aal_status scalar() {
    return launch_pdl(k_ln_bwd<T, TP, NV, TPR>, dim3((unsigned)grid), p.threads,
                      TPR == 32 ? (size_t)a.d * 2 * kRowsPerCta * sizeof(float) : 0, s, a);
  }
  template <int NV, bool BLOCK, int MAXT>
  aal_status ring() {
    // the stages fit three arrays; with two the ring is no longer, only lighter
    const Ring r = ring_plan(p, a.d, sizeof(T), 3);
    a.ring = r.stages;
    return launch_pdl(k_ln_bwd_ring<T, TP, NV, BLOCK, MAXT>, dim3((unsigned)grid), p.threads, r.bytes, s, a);
  }
};

// A parameter vector (gamma, beta or a gradient of one): [1, d], the call's
// dtype or fp32; a null pointer stands for one that is not there.
static bool valid_vec(const aal_mat& m, long long d, int dtype) {
  if (!m.ptr) return true;
  return valid_mat(m) && m.rows == 1 && m.cols == d && (m.dtype == dtype || m.dtype == AAL_F32);
}

// Partial column sums of the backward: CTAs times two rows of d floats.
static long long bwd_part_bytes(long long rows, long long d, int es, bool aligned) {
  const Plan p = bwd_plan(d, es, aligned);
  return p.wide ? 0 : (long long)bwd_grid(p, rows, d, es) * 2 * d * 4;
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
  if (M == 0 || d == 0) return AAL_OK;
  const int pdt = gamma.ptr ? gamma.dtype : beta.ptr ? beta.dtype : dt;
  const bool al = norm::rows_aligned(X) && norm::rows_aligned(R) && norm::rows_aligned(S) && norm::rows_aligned(Y) &&
                  norm::rows_aligned(gamma) && norm::rows_aligned(beta);
  const norm::Plan p = norm::fwd_plan(d, dt == AAL_F32 ? 4 : 2, al);
  norm::FwdArgs a = {X.ptr, R.ptr, gamma.ptr, beta.ptr, S.ptr, Y.ptr, mean, rstd, M, d, X.ld, R.ld, S.ld, Y.ld, eps, 0};
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
    for (int al = 0; al < 2; ++al) {
      const long long b = norm::bwd_part_bytes(rows, cols, es, al != 0);
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
  const int es = dt == AAL_F32 ? 4 : 2;
  const norm::Plan p = norm::bwd_plan(d, es, al);
  norm::BwdArgs a = {X.ptr, gamma.ptr, dY.ptr, dR.ptr, mean, rstd, dX.ptr, nullptr, M, d, X.ld, dY.ld, dR.ld, dX.ld, 0};
  const int grid = p.wide ? 0 : norm::bwd_grid(p, M, d, es);
  const unsigned gx = (unsigned)((d + 31) / 32);
  if ((d + 31) / 32 > 0x7fffffffLL) return AAL_ERR_UNSUPPORTED;
  uint64_t have = 0;
  float* ws = (float*)current_workspace(&have);
  const bool parts = cols && M > 0 && !p.wide && ws && have >= (uint64_t)grid * 2 * d * 4;
  const aal_status st = timed(AAL_KERNEL_NORM_BWD, s, [&] {
    aal_status e = AAL_OK;
    if (cols && M > 0 && !parts) {  // first: dX may be written over X, dY or dR
      e = dt == AAL_F32 ? norm::launch_pdl(norm::k_ln_bwd_cols<float>, dim3(gx), 1024, 0, s, a, dgamma.ptr, dbeta.ptr,
                                           pf32, (int)accumulate)
                        : norm::launch_pdl(norm::k_ln_bwd_cols<__nv_bfloat16>, dim3(gx), 1024, 0, s, a, dgamma.ptr,
                                           dbeta.ptr, pf32, (int)accumulate);
    }
    a.part = parts ? ws : nullptr;
    if (e == AAL_OK && M > 0 && (dX.ptr || parts)) {
      if (p.wide) {  // (without column sums: parts is false)
        const dim3 g((unsigned)norm::grid_of(p, M, 2));
        e = dt == AAL_F32     ? norm::launch_pdl(norm::k_ln_bwd_wide<float, float>, g, p.threads, 0, s, a)
            : gdt == AAL_F32 ? norm::launch_pdl(norm::k_ln_bwd_wide<__nv_bfloat16, float>, g, p.threads, 0, s, a)
                             : norm::launch_pdl(norm::k_ln_bwd_wide<__nv_bfloat16, __nv_bfloat16>, g, p.threads, 0, s, a);
      } else if (dt == AAL_F32) {
        e = norm::with_shape<4>(p, norm::BwdLaunch<float, float>{a, p, grid, s});
      } else if (gdt == AAL_F32) {
        e = norm::with_shape<8>(p, norm::BwdLaunch<__nv_bfloat16, float>{a, p, grid, s});
      } else {
        e = norm::with_shape<8>(p, norm::BwdLaunch<__nv_bfloat16, __nv_bfloat16>{a, p, grid, s});
      }
    }
    if (e == AAL_OK && cols && (parts || M == 0))
      e = norm::launch_pdl(norm::k_ln_bwd_reduce, dim3(gx, 2), 32 * norm::kReduceWarps, 0, s, (const float*)ws,
                           M == 0 ? 0 : grid, (long long)d, dgamma.ptr, dbeta.ptr, pf32, (int)accumulate);
    return e;
  });
  if (st == AAL_OK) note_path(AAL_PATH_GENERAL);
  return st;
}

}  // extern "C"
