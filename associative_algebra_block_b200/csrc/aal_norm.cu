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

// VEC adjacent elements, loaded and stored in 16-byte pieces (one element when
// VEC is 1).
template <typename T, int VEC>
struct Pack {
  T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ void load_pack(const T* p, Pack<T, VEC>& o) {
  if constexpr (VEC == 1) {
    o.v[0] = *p;
  } else {
    static_assert((sizeof(T) * VEC) % 16 == 0, "16-byte pieces");
    constexpr int n = sizeof(T) * VEC / 16;
    uint4 u[n];
#pragma unroll
    for (int i = 0; i < n; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    memcpy(o.v, u, sizeof(u));
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, VEC>& o) {
  if constexpr (VEC == 1) {
    *p = o.v[0];
  } else {
    constexpr int n = sizeof(T) * VEC / 16;
    uint4 u[n];
    memcpy(u, o.v, sizeof(u));
#pragma unroll
    for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
  }
}
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

struct FwdArgs {
  const void *x, *r, *gamma, *beta;
  void *s, *y;
  float *mean, *rstd;
  long long rows, d, ldx, ldr, lds, ldy;
  float eps;
};

constexpr int kRowsPerCta = 8;  // warp-per-row kernels: one row a warp

// BLOCK false: a warp a row, kRowsPerCta rows a CTA; true: the CTA a row.
// NV vectors of VEC elements a thread.
template <typename T, typename TP, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 32 * kRowsPerCta) k_ln_fwd(const FwdArgs a) {
  __shared__ float2 buf[2][32];
  pdl_begin();
  const int tpr = BLOCK ? (int)blockDim.x : 32;
  const int t = BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & 31);
  const long long r0 = BLOCK ? blockIdx.x : (long long)blockIdx.x * kRowsPerCta + (threadIdx.x >> 5);
  const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * kRowsPerCta;
  const T *x = (const T*)a.x, *r = (const T*)a.r;
  const TP *gm = (const TP*)a.gamma, *bt = (const TP*)a.beta;
  const int d = (int)a.d;
  const float inv_d = 1.0f / (float)d;
  int turn = 0;
  for (long long row = r0; row < a.rows; row += step) {
    float v[NV][VEC];
    Pack<T, VEC> px[NV], pr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
      if (c < d) load_pack<T, VEC>(x + row * a.ldx + c, px[i]);
    }
    if (r) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
        if (c < d) load_pack<T, VEC>(r + row * a.ldr + c, pr[i]);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float e = 0.f;
        if (c < d) {
          e = as_f32(px[i].v[j]);
          if (r) e += as_f32(pr[i].v[j]);
        }
        v[i][j] = e;
        sum += e;
      }
    }
    sum = BLOCK ? block_sum2(sum, 0.f, buf, turn).x : warp_sum(sum);
    const float mu = sum * inv_d;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float e = c < d ? v[i][j] - mu : 0.f;
        sq = fmaf(e, e, sq);
      }
    }
    sq = BLOCK ? block_sum2(sq, 0.f, buf, turn).x : warp_sum(sq);
    const float rs = 1.0f / sqrtf(sq * inv_d + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = rs;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
      if (c >= d) continue;
      if (a.s) {
        // the stored sum is rounded to the matrix type; the norm itself uses
        // the unrounded one
        Pack<T, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) o.v[j] = from_f32<T>(v[i][j]);
        store_pack<T, VEC>((T*)a.s + row * a.lds + c, o);
      }
      Pack<TP, VEC> pg, pb;
      if (gm) load_pack<TP, VEC>(gm + c, pg);
      if (bt) load_pack<TP, VEC>(bt + c, pb);
      Pack<T, VEC> o;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float e = (v[i][j] - mu) * rs;
        if (gm) e *= as_f32(pg.v[j]);
        if (bt) e += as_f32(pb.v[j]);
        o.v[j] = from_f32<T>(e);
      }
      store_pack<T, VEC>((T*)a.y + row * a.ldy + c, o);
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
};

template <typename T, typename TP, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 32 * kRowsPerCta) k_ln_bwd(const BwdArgs a) {
  __shared__ float2 buf[2][32];
  extern __shared__ float cols[];  // warp-per-row: [2][d] column sums of the CTA
  pdl_begin();
  const int tpr = BLOCK ? (int)blockDim.x : 32;
  const int t = BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & 31);
  const long long r0 = BLOCK ? blockIdx.x : (long long)blockIdx.x * kRowsPerCta + (threadIdx.x >> 5);
  const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * kRowsPerCta;
  const T *x = (const T*)a.x, *dy = (const T*)a.dy, *dr = (const T*)a.dr;
  const TP* gm = (const TP*)a.gamma;
  const int d = (int)a.d;
  const float inv_d = 1.0f / (float)d;
  float dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[i][j] = db[i][j] = 0.f;
  int turn = 0;
  for (long long row = r0; row < a.rows; row += step) {
    Pack<T, VEC> px[NV], py[NV], pr[NV];
    const float mu = a.mean[row], rs = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
      if (c < d) {
        load_pack<T, VEC>(x + row * a.ldx + c, px[i]);
        load_pack<T, VEC>(dy + row * a.lddy + c, py[i]);
      }
    }
    if (dr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
        if (c < d) load_pack<T, VEC>(dr + row * a.lddr + c, pr[i]);
      }
    }
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
      if (c >= d) continue;
      Pack<TP, VEC> pg;
      if (gm) load_pack<TP, VEC>(gm + c, pg);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float xh = (as_f32(px[i].v[j]) - mu) * rs, y = as_f32(py[i].v[j]);
        const float g = gm ? y * as_f32(pg.v[j]) : y;
        sg += g;
        sgx = fmaf(g, xh, sgx);
        dg[i][j] = fmaf(y, xh, dg[i][j]);
        db[i][j] += y;
      }
    }
    if (a.dx) {
      if (BLOCK) {
        const float2 s = block_sum2(sg, sgx, buf, turn);
        sg = s.x;
        sgx = s.y;
      } else {
        sg = warp_sum(sg);
        sgx = warp_sum(sgx);
      }
      sg *= inv_d;
      sgx *= inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
        if (c >= d) continue;
        Pack<TP, VEC> pg;
        if (gm) load_pack<TP, VEC>(gm + c, pg);
        Pack<T, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (as_f32(px[i].v[j]) - mu) * rs, y = as_f32(py[i].v[j]);
          const float g = gm ? y * as_f32(pg.v[j]) : y;
          float e = rs * (g - sg - xh * sgx);
          if (dr) e += as_f32(pr[i].v[j]);
          o.v[j] = from_f32<T>(e);
        }
        store_pack<T, VEC>((T*)a.dx + row * a.lddx + c, o);
      }
    }
  }
  if (!a.part) return;
  float* out = a.part + (long long)blockIdx.x * 2 * d;
  if (BLOCK) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (c < d) {
          out[c + j] = dg[i][j];
          out[d + c + j] = db[i][j];
        }
    }
    return;
  }
  // the warps add their columns one after another: a fixed order
  for (int w = 0; w < kRowsPerCta; ++w) {
    if ((int)(threadIdx.x >> 5) == w) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * 32 + t) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c < d) {
            cols[c + j] = w ? cols[c + j] + dg[i][j] : dg[i][j];
            cols[d + c + j] = w ? cols[d + c + j] + db[i][j] : db[i][j];
          }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) out[c] = cols[c];
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
  int vec;      // elements a vector: 16 bytes, or 1
  int nv;       // vectors a thread
  bool block;   // the CTA a row (else a warp a row)
  int threads;  // CTA size
  bool wide;    // the row does not fit registers
};

// Vectors need 16-byte aligned rows and parameters and whole vectors a row;
// other shapes go element by element, still coalesced.
static Plan plan(long long d, int es, bool aligned) {
  Plan p;
  p.vec = (aligned && (d * es) % 16 == 0) ? 16 / es : 1;
  const long long n = (d + p.vec - 1) / p.vec;
  const int most = p.vec == 1 ? 16 : 4;  // vectors a thread
  p.wide = n > 1024LL * most;
  p.block = n > 32LL * most;
  p.nv = 1;
  p.threads = 32 * kRowsPerCta;
  if (p.wide) {
    p.block = true;
    p.threads = 1024;
    return p;
  }
  if (!p.block) {
    while (p.nv * 32 < n) p.nv = p.vec == 1 ? p.nv * 2 : p.nv + 1;
  } else {
    p.nv = most;
    p.threads = (int)(((n + most - 1) / most + 31) / 32 * 32);
  }
  return p;
}

static bool rows_aligned(const aal_mat& m) {
  const size_t es = m.dtype == AAL_F32 ? 4 : 2;
  return !m.ptr || (((uintptr_t)m.ptr % 16) == 0 && (m.rows <= 1 || (m.ld * es) % 16 == 0));
}

template <typename... A>
static aal_status launch_pdl(void (*k)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
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

// Calls f with the kernel's compile-time shape: f.template operator()<VEC, NV, BLOCK>().
template <int V, typename F>
static aal_status with_shape(const Plan& p, F f) {
  if (p.vec == 1) {
    if (p.block) return f.template operator()<1, 16, true>();
    switch (p.nv) {
      case 1: return f.template operator()<1, 1, false>();
      case 2: return f.template operator()<1, 2, false>();
      case 4: return f.template operator()<1, 4, false>();
      case 8: return f.template operator()<1, 8, false>();
      default: return f.template operator()<1, 16, false>();
    }
  }
  if (p.block) return f.template operator()<V, 4, true>();
  switch (p.nv) {
    case 1: return f.template operator()<V, 1, false>();
    case 2: return f.template operator()<V, 2, false>();
    case 3: return f.template operator()<V, 3, false>();
    default: return f.template operator()<V, 4, false>();
  }
}

static int fwd_grid(const Plan& p, long long rows) {
  const long long per = p.block ? 1 : kRowsPerCta;
  const long long most = (long long)device_sms() * (p.block ? 2048 / p.threads : 8);
  const long long n = (rows + per - 1) / per;
  return (int)(n < most ? n : most);
}
static int bwd_grid(const Plan& p, long long rows) {
  const long long per = p.block ? 1 : kRowsPerCta;
  const int res = p.block ? (p.threads >= 512 ? 1 : p.threads >= 256 ? 2 : 3) : 2;
  const long long most = (long long)device_sms() * res;
  const long long n = (rows + per - 1) / per;
  return (int)(n < most ? n : most);
}

template <typename T, typename TP>
struct FwdLaunch {
  const FwdArgs& a;
  const Plan& p;
  cudaStream_t s;
  template <int VEC, int NV, bool BLOCK>
  aal_status operator()() {
    return launch_pdl(k_ln_fwd<T, TP, VEC, NV, BLOCK>, dim3((unsigned)fwd_grid(p, a.rows)), p.threads, 0, s, a);
  }
};
template <typename T, typename TP>
static aal_status run_fwd(const FwdArgs& a, const Plan& p, cudaStream_t s) {
  if (p.wide)
    return launch_pdl(k_ln_fwd_wide<T, TP>, dim3((unsigned)fwd_grid(p, a.rows)), p.threads, 0, s, a);
  return with_shape<16 / sizeof(T)>(p, FwdLaunch<T, TP>{a, p, s});
}

template <typename T, typename TP>
struct BwdLaunch {
  const BwdArgs& a;
  const Plan& p;
  int grid;
  cudaStream_t s;
  template <int VEC, int NV, bool BLOCK>
  aal_status operator()() {
    return launch_pdl(k_ln_bwd<T, TP, VEC, NV, BLOCK>, dim3((unsigned)grid), p.threads,
                      BLOCK ? 0 : (size_t)a.d * 2 * sizeof(float), s, a);
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
  const Plan p = plan(d, es, aligned);
  return p.wide ? 0 : (long long)bwd_grid(p, rows) * 2 * d * 4;
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
  const norm::Plan p = norm::plan(d, dt == AAL_F32 ? 4 : 2, al);
  norm::FwdArgs a = {X.ptr, R.ptr, gamma.ptr, beta.ptr, S.ptr, Y.ptr, mean, rstd, M, d, X.ld, R.ld, S.ld, Y.ld, eps};
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
  const norm::Plan p = norm::plan(d, dt == AAL_F32 ? 4 : 2, al);
  norm::BwdArgs a = {X.ptr, gamma.ptr, dY.ptr, dR.ptr, mean, rstd, dX.ptr, nullptr, M, d, X.ld, dY.ld, dR.ld, dX.ld};
  const int grid = norm::bwd_grid(p, M);
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
      if (p.wide) {
        const dim3 g((unsigned)norm::fwd_grid(p, M));
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
