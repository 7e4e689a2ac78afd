// ckda_layernorm.cu -- layer norm over the last axis, forward and backward.
//
// Per row x of D values, with mean m and r = 1 / sqrt(var + eps) (var the
// mean of (x - m)^2):
//     y_i  = (x_i - m) r w_i + b_i
//     dx_i = r [ t_i - mean(t) - xh_i mean(t xh) ],  t = dy w,  xh = (x - m) r
//     dw_i = sum over rows of dy_i xh_i,   db_i = sum over rows of dy_i
// Everything is fp32 between the load and the store; the variance is taken
// from centred values held in registers, so a row with a large offset loses
// nothing to cancellation.
//
// The work is a few flop per element, so HBM bandwidth is the bound: x once in
// and y once out (forward), x and dy in and dx out (backward).  A row is held
// in registers by the lanes that own it, in vectors of VEC elements:
//   - narrow rows: LPR lanes (8, 16 or 32) to a row, several rows to a warp,
//     and kRowsInFlight rows a lane group at once, so that enough loads are in
//     flight with 16 bytes a lane;
//   - wide rows: a block to a row;
//   - rows wider than a block's registers hold: a block to a row, read again
//     for each of the sums (the second and third reads hit L2).
// The weight gradients are sums over rows for every column: a block walks its
// rows with one fp32 partial sum a column in the registers of the thread that
// owns the column, writes one partial row to the workspace, and a second
// kernel adds the partial rows in a fixed order.  No atomics: two calls on the
// same input give the same bits.
#include "ckda_internal.cuh"

namespace ckda {
namespace {

constexpr int kSms = 152;
constexpr int kBlock = 256;

struct NormArgs {
  const void* x;
  const void* dy;
  const void* w;
  const void* b;
  void* y;  // dx in the backward pass
  float* mean;
  float* rstd;
  float* part;  // [2][parts][D] partial dw and db
  void* dw;
  void* db;
  long long rows;
  int D;
  int parts;
  float eps;
};

template <typename IO, int VEC>
struct alignas(sizeof(IO) * VEC) Pack {
  IO v[VEC];
};
template <typename IO>
__device__ __forceinline__ float to_f(IO x) {
  return ld_io(&x);
}
template <typename IO, int VEC>
__device__ __forceinline__ void load_vec(const void* base, long long at, float (&f)[VEC]) {
  const Pack<IO, VEC> p = *reinterpret_cast<const Pack<IO, VEC>*>(static_cast<const IO*>(base) + at);
#pragma unroll
  for (int e = 0; e < VEC; ++e) f[e] = to_f(p.v[e]);
}
template <typename IO, int VEC>
__device__ __forceinline__ void store_vec(void* base, long long at, const float (&f)[VEC]) {
  Pack<IO, VEC> p;
#pragma unroll
  for (int e = 0; e < VEC; ++e) st_io(&p.v[e], f[e]);
  *reinterpret_cast<Pack<IO, VEC>*>(static_cast<IO*>(base) + at) = p;
}
// Weights are few and stay in L1/L2: one element at a time in their own type.
template <typename W>
__device__ __forceinline__ float weight_at(const void* w, int i, float none) {
  return w ? ld_io(static_cast<const W*>(w) + i) : none;
}

template <int LPR>
__device__ __forceinline__ float lane_sum(float s) {
#pragma unroll
  for (int m = LPR / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  return s;
}
// Sum over the block, the same value (and order) in every thread.  `red` has
// one float a warp and may be used again after the next barrier pair.
__device__ __forceinline__ float block_sum(float s, float* red) {
  s = lane_sum<32>(s);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) t += red[i];
  return t;
}

// ------------------------------------------------------------------ forward
template <typename IO, typename W, int VEC, int LPR, int NV, int RIF>
__global__ void __launch_bounds__(kBlock) norm_fwd_rows_kernel(NormArgs a) {
  constexpr int kGroups = kBlock / LPR;
  const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const float inv_d = 1.f / (float)a.D;
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = (n * LPR + lane) * VEC + e;
      w[n][e] = i < a.D ? weight_at<W>(a.w, i, 1.f) : 0.f;
      b[n][e] = i < a.D ? weight_at<W>(a.b, i, 0.f) : 0.f;
    }
  for (long long r0 = (long long)blockIdx.x * kGroups * RIF; r0 < a.rows;
       r0 += (long long)gridDim.x * kGroups * RIF) {
    float x[RIF][NV][VEC];
#pragma unroll
    for (int k = 0; k < RIF; ++k) {
      const long long r = r0 + k * kGroups + grp;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int i = (n * LPR + lane) * VEC;
        if (r < a.rows && i < a.D)
          load_vec<IO, VEC>(a.x, r * a.D + i, x[k][n]);
        else
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[k][n][e] = 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < RIF; ++k) {
      const long long r = r0 + k * kGroups + grp;
      float s = 0.f;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += x[k][n][e];
      const float mean = lane_sum<LPR>(s) * inv_d;
      float s2 = 0.f;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float c = x[k][n][e] - mean;
          x[k][n][e] = c;
          if ((n * LPR + lane) * VEC < a.D) s2 = fmaf(c, c, s2);
        }
      const float rstd = 1.f / sqrtf(lane_sum<LPR>(s2) * inv_d + a.eps);
      if (r < a.rows) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const int i = (n * LPR + lane) * VEC;
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[k][n][e] = fmaf(x[k][n][e] * rstd, w[n][e], b[n][e]);
          if (i < a.D) store_vec<IO, VEC>(a.y, r * a.D + i, x[k][n]);
        }
        if (lane == 0) {
          a.mean[r] = mean;
          a.rstd[r] = rstd;
        }
      }
    }
  }
}

template <typename IO, typename W, int VEC, int NV>
__global__ void __launch_bounds__(kBlock) norm_fwd_block_kernel(NormArgs a) {
  __shared__ float red[kBlock / 32];
  const float inv_d = 1.f / (float)a.D;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float x[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = (n * kBlock + threadIdx.x) * VEC;
      if (i < a.D)
        load_vec<IO, VEC>(a.x, r * a.D + i, x[n]);
      else
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[n][e] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += x[n][e];
    const float mean = block_sum(s, red) * inv_d;
    float s2 = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if ((n * kBlock + threadIdx.x) * VEC < a.D)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x[n][e] -= mean;
          s2 = fmaf(x[n][e], x[n][e], s2);
        }
    const float rstd = 1.f / sqrtf(block_sum(s2, red) * inv_d + a.eps);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = (n * kBlock + threadIdx.x) * VEC;
      if (i >= a.D) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        x[n][e] = fmaf(x[n][e] * rstd, weight_at<W>(a.w, i + e, 1.f), weight_at<W>(a.b, i + e, 0.f));
      store_vec<IO, VEC>(a.y, r * a.D + i, x[n]);
    }
    if (threadIdx.x == 0) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
  }
}

template <typename IO, typename W>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(NormArgs a) {
  __shared__ float red[32];
  const float inv_d = 1.f / (float)a.D;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const IO* x = static_cast<const IO*>(a.x) + r * a.D;
    IO* y = static_cast<IO*>(a.y) + r * a.D;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 1024) s += ld_io(x + i);
    const float mean = block_sum(s, red) * inv_d;
    float s2 = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 1024) {
      const float c = ld_io(x + i) - mean;
      s2 = fmaf(c, c, s2);
    }
    const float rstd = 1.f / sqrtf(block_sum(s2, red) * inv_d + a.eps);
    for (int i = threadIdx.x; i < a.D; i += 1024)
      st_io(y + i, fmaf((ld_io(x + i) - mean) * rstd, weight_at<W>(a.w, i, 1.f),
                        weight_at<W>(a.b, i, 0.f)));
    if (threadIdx.x == 0) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
  }
}

// ----------------------------------------------------------------- backward
// One partial row of dw and db for each block.
template <typename IO, typename W, int VEC, int LPR, int NV, int RIF>
__global__ void __launch_bounds__(kBlock) norm_bwd_rows_kernel(NormArgs a) {
  constexpr int kGroups = kBlock / LPR;
  extern __shared__ float part_s[];  // [kGroups][D], when weight gradients are wanted
  const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const float inv_d = 1.f / (float)a.D;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = (n * LPR + lane) * VEC + e;
      w[n][e] = i < a.D ? weight_at<W>(a.w, i, 1.f) : 0.f;
      dw[n][e] = db[n][e] = 0.f;
    }
  for (long long r0 = (long long)blockIdx.x * kGroups * RIF; r0 < a.rows;
       r0 += (long long)gridDim.x * kGroups * RIF) {
    float x[RIF][NV][VEC], dy[RIF][NV][VEC], mean[RIF], rstd[RIF];
#pragma unroll
    for (int k = 0; k < RIF; ++k) {
      const long long r = r0 + k * kGroups + grp;
      const bool in = r < a.rows;
      mean[k] = in ? a.mean[r] : 0.f;
      rstd[k] = in ? a.rstd[r] : 0.f;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int i = (n * LPR + lane) * VEC;
        if (in && i < a.D) {
          load_vec<IO, VEC>(a.x, r * a.D + i, x[k][n]);
          load_vec<IO, VEC>(a.dy, r * a.D + i, dy[k][n]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            x[k][n][e] = mean[k];
            dy[k][n][e] = 0.f;
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < RIF; ++k) {
      const long long r = r0 + k * kGroups + grp;
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (x[k][n][e] - mean[k]) * rstd[k], g = dy[k][n][e], t = g * w[n][e];
          dw[n][e] = fmaf(g, xh, dw[n][e]);
          db[n][e] += g;
          s1 += t;
          s2 = fmaf(t, xh, s2);
          x[k][n][e] = xh;
          dy[k][n][e] = t;
        }
      const float m1 = lane_sum<LPR>(s1) * inv_d, m2 = lane_sum<LPR>(s2) * inv_d;
      if (r < a.rows) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const int i = (n * LPR + lane) * VEC;
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            x[k][n][e] = rstd[k] * (dy[k][n][e] - m1 - x[k][n][e] * m2);
          if (i < a.D) store_vec<IO, VEC>(a.y, r * a.D + i, x[k][n]);
        }
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int i = (n * LPR + lane) * VEC + e;
        if (i < a.D) part_s[grp * a.D + i] = which ? db[n][e] : dw[n][e];
      }
    __syncthreads();
    float* out = a.part + ((size_t)which * a.parts + blockIdx.x) * a.D;
    for (int i = threadIdx.x; i < a.D; i += kBlock) {
      float s = 0.f;
#pragma unroll 8
      for (int g = 0; g < kGroups; ++g) s += part_s[g * a.D + i];
      out[i] = s;
    }
  }
}

template <typename IO, typename W, int VEC, int NV>
__global__ void __launch_bounds__(kBlock) norm_bwd_block_kernel(NormArgs a) {
  __shared__ float red[2][kBlock / 32];
  const float inv_d = 1.f / (float)a.D;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = (n * kBlock + threadIdx.x) * VEC + e;
      w[n][e] = i < a.D ? weight_at<W>(a.w, i, 1.f) : 0.f;
      dw[n][e] = db[n][e] = 0.f;
    }
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float x[NV][VEC], dy[NV][VEC];
    const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = (n * kBlock + threadIdx.x) * VEC;
      if (i < a.D) {
        load_vec<IO, VEC>(a.x, r * a.D + i, x[n]);
        load_vec<IO, VEC>(a.dy, r * a.D + i, dy[n]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x[n][e] = mean;
          dy[n][e] = 0.f;
        }
      }
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (x[n][e] - mean) * rstd, g = dy[n][e], t = g * w[n][e];
        dw[n][e] = fmaf(g, xh, dw[n][e]);
        db[n][e] += g;
        s1 += t;
        s2 = fmaf(t, xh, s2);
        x[n][e] = xh;
        dy[n][e] = t;
      }
    // both sums through one pair of barriers
    s1 = lane_sum<32>(s1);
    s2 = lane_sum<32>(s2);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      red[0][threadIdx.x >> 5] = s1;
      red[1][threadIdx.x >> 5] = s2;
    }
    __syncthreads();
    float m1 = 0.f, m2 = 0.f;
#pragma unroll
    for (int i = 0; i < kBlock / 32; ++i) {
      m1 += red[0][i];
      m2 += red[1][i];
    }
    m1 *= inv_d;
    m2 *= inv_d;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = (n * kBlock + threadIdx.x) * VEC;
      if (i >= a.D) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[n][e] = rstd * (dy[n][e] - m1 - x[n][e] * m2);
      store_vec<IO, VEC>(a.y, r * a.D + i, x[n]);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = (n * kBlock + threadIdx.x) * VEC + e;
      if (i >= a.D) continue;
      a.part[(size_t)blockIdx.x * a.D + i] = dw[n][e];
      a.part[((size_t)a.parts + blockIdx.x) * a.D + i] = db[n][e];
    }
}

// Rows wider than a block's registers: the block keeps its partial sums of dw
// and db in its row of the workspace.
template <typename IO, typename W>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(NormArgs a) {
  __shared__ float red[32];
  const float inv_d = 1.f / (float)a.D;
  float* pw = a.part ? a.part + (size_t)blockIdx.x * a.D : nullptr;
  float* pb = a.part ? a.part + ((size_t)a.parts + blockIdx.x) * a.D : nullptr;
  bool first = true;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const IO* x = static_cast<const IO*>(a.x) + r * a.D;
    const IO* dy = static_cast<const IO*>(a.dy) + r * a.D;
    IO* dx = static_cast<IO*>(a.y) + r * a.D;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 1024) {
      const float xh = (ld_io(x + i) - mean) * rstd, g = ld_io(dy + i);
      const float t = g * weight_at<W>(a.w, i, 1.f);
      s1 += t;
      s2 = fmaf(t, xh, s2);
      if (pw) {  // column i of this block's partial row belongs to this thread
        pw[i] = fmaf(g, xh, first ? 0.f : pw[i]);
        pb[i] = g + (first ? 0.f : pb[i]);
      }
    }
    first = false;
    const float m1 = block_sum(s1, red) * inv_d, m2 = block_sum(s2, red) * inv_d;
    for (int i = threadIdx.x; i < a.D; i += 1024) {
      const float xh = (ld_io(x + i) - mean) * rstd;
      const float t = ld_io(dy + i) * weight_at<W>(a.w, i, 1.f);
      st_io(dx + i, rstd * (t - m1 - xh * m2));
    }
  }
}

// dw and db from the partial rows: 32 columns to a block, 8 threads a column
// over the partial rows, joined in a fixed order.
template <typename W>
__global__ void __launch_bounds__(256) norm_weight_grad_kernel(NormArgs a) {
  __shared__ float s[8][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + c;
  const float* p = a.part + (size_t)blockIdx.y * a.parts * a.D;
  float t = 0.f;
  if (i < a.D)
    for (int r = g; r < a.parts; r += 8) t += p[(size_t)r * a.D + i];
  s[g][c] = t;
  __syncthreads();
  if (g == 0 && i < a.D) {
#pragma unroll
    for (int k = 1; k < 8; ++k) t += s[k][c];
    st_io(static_cast<W*>(blockIdx.y ? a.db : a.dw) + i, t);
  }
}

// ----------------------------------------------------------------- dispatch
// Vectors of 16 bytes where the width and every row-indexed pointer allow it,
// single elements otherwise.
inline bool vector_ok(int D, int vec, const void* p0, const void* p1, const void* p2) {
  const uintptr_t m = reinterpret_cast<uintptr_t>(p0) | reinterpret_cast<uintptr_t>(p1) |
                      reinterpret_cast<uintptr_t>(p2);
  return D % vec == 0 && (m & 15) == 0;
}
inline int blocks_for(long long units, int per_sm) {
  const long long most = (long long)kSms * per_sm;
  return (int)(units < most ? (units < 1 ? 1 : units) : most);
}
// Partial rows of the weight gradients: at most four a SM, fewer for few rows.
inline int weight_parts(long long rows, int D) {
  (void)D;
  return blocks_for(rows, 4);
}

template <typename IO, typename W, int VEC>
cudaError_t fwd_vec(const NormArgs& a, cudaStream_t s) {
  const int D = a.D;
#define NORM_ROWS(LPR, NV, RIF)                                                                \
  {                                                                                            \
    const int per = (kBlock / LPR) * RIF;                                                      \
    norm_fwd_rows_kernel<IO, W, VEC, LPR, NV, RIF>                                             \
        <<<blocks_for((a.rows + per - 1) / per, 8), kBlock, 0, s>>>(a);                        \
  }
  // few rows: one row a lane group, so that the rows spread over more SMs
  if (D <= 8 * VEC) NORM_ROWS(8, 1, 2)
  else if (D <= 16 * VEC) NORM_ROWS(16, 1, 2)
  else if (D <= 32 * VEC) NORM_ROWS(32, 1, 2)
  else if (D <= 64 * VEC) NORM_ROWS(32, 2, 1)
  else if (D <= 128 * VEC && a.rows >= 8 * kSms) NORM_ROWS(32, 4, 1)
  else if (D <= 1 * kBlock * VEC)
    norm_fwd_block_kernel<IO, W, VEC, 1><<<blocks_for(a.rows, 8), kBlock, 0, s>>>(a);
  else if (D <= 2 * kBlock * VEC)
    norm_fwd_block_kernel<IO, W, VEC, 2><<<blocks_for(a.rows, 8), kBlock, 0, s>>>(a);
  else if (D <= 4 * kBlock * VEC)
    norm_fwd_block_kernel<IO, W, VEC, 4><<<blocks_for(a.rows, 8), kBlock, 0, s>>>(a);
  else if (D <= 8 * kBlock * VEC)
    norm_fwd_block_kernel<IO, W, VEC, 8><<<blocks_for(a.rows, 8), kBlock, 0, s>>>(a);
  else
    norm_fwd_long_kernel<IO, W><<<blocks_for(a.rows, 2), 1024, 0, s>>>(a);
#undef NORM_ROWS
  return cudaGetLastError();
}

template <typename IO, typename W, int VEC>
cudaError_t bwd_vec(const NormArgs& a, cudaStream_t s) {
  const int D = a.D;
  const int grid = a.parts;
#define NORM_ROWS(LPR, NV, RIF)                                                       \
  norm_bwd_rows_kernel<IO, W, VEC, LPR, NV, RIF>                                      \
      <<<grid, kBlock, a.part ? (size_t)(kBlock / LPR) * D * sizeof(float) : 0, s>>>(a)
  if (D <= 8 * VEC) NORM_ROWS(8, 1, 2);
  else if (D <= 16 * VEC) NORM_ROWS(16, 1, 2);
  else if (D <= 32 * VEC) NORM_ROWS(32, 1, 2);
  else if (D <= 64 * VEC) NORM_ROWS(32, 2, 1);
  else if (D <= 1 * kBlock * VEC)
    norm_bwd_block_kernel<IO, W, VEC, 1><<<grid, kBlock, 0, s>>>(a);
  else if (D <= 2 * kBlock * VEC)
    norm_bwd_block_kernel<IO, W, VEC, 2><<<grid, kBlock, 0, s>>>(a);
  else if (D <= 4 * kBlock * VEC)
    norm_bwd_block_kernel<IO, W, VEC, 4><<<grid, kBlock, 0, s>>>(a);
  else
    norm_bwd_long_kernel<IO, W><<<grid, 1024, 0, s>>>(a);
#undef NORM_ROWS
  return cudaGetLastError();
}

template <typename IO, typename W>
cudaError_t launch_norm(const NormArgs& a, bool back, cudaStream_t s) {
  constexpr int kVec = 16 / sizeof(IO);
  const bool vec = vector_ok(a.D, kVec, a.x, a.y, back ? a.dy : a.x);
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    e = back ? (vec ? bwd_vec<IO, W, kVec>(a, s) : bwd_vec<IO, W, 1>(a, s))
             : (vec ? fwd_vec<IO, W, kVec>(a, s) : fwd_vec<IO, W, 1>(a, s));
    if (e != cudaSuccess) return e;
  }
  if (back && a.part) {
    NormArgs b = a;
    if (a.rows == 0) b.parts = 0;  // the sums over no rows are zero
    norm_weight_grad_kernel<W><<<dim3((a.D + 31) / 32, 2), 256, 0, s>>>(b);
    e = cudaGetLastError();
  }
  return e;
}

cudaError_t launch_any(const NormArgs& a, ckda_dtype io, ckda_dtype wt, bool back, cudaStream_t s) {
  if (io == CKDA_F32)
    return wt == CKDA_F32 ? launch_norm<float, float>(a, back, s)
                          : launch_norm<float, __nv_bfloat16>(a, back, s);
  return wt == CKDA_F32 ? launch_norm<__nv_bfloat16, float>(a, back, s)
                        : launch_norm<__nv_bfloat16, __nv_bfloat16>(a, back, s);
}

ckda_status check_norm(long long rows, int width, ckda_dtype io, ckda_dtype wt) {
  if (io != CKDA_F32 && io != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
  if (wt != CKDA_F32 && wt != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
  if (rows < 0 || width < 1) return CKDA_ERR_INVALID_ARG;
  if (rows > 0x7fffffffLL) return CKDA_ERR_UNSUPPORTED;
  return CKDA_OK;
}

}  // namespace
}  // namespace ckda

using namespace ckda;

extern "C" {

ckda_status ckda_layernorm_fwd(const void* x, const void* weight, const void* bias, void* y,
                               float* mean, float* rstd, long long rows, int width,
                               ckda_dtype io_dtype, ckda_dtype weight_dtype, float eps,
                               void* stream) {
  const ckda_status st = check_norm(rows, width, io_dtype, weight_dtype);
  if (st != CKDA_OK) return st;
  if (!(eps >= 0.f) || eps > 3.0e38f) return CKDA_ERR_INVALID_ARG;
  if (rows == 0) return CKDA_OK;
  if (!x || !y || !mean || !rstd) return CKDA_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = x; a.w = weight; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd;
  a.rows = rows; a.D = width; a.eps = eps;
  return launch_any(a, io_dtype, weight_dtype, false, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? CKDA_OK
             : CKDA_ERR_CUDA;
}

size_t ckda_layernorm_bwd_workspace_bytes(long long rows, int width) {
  if (rows < 0 || width < 1) return 0;
  return (size_t)2 * weight_parts(rows, width) * width * sizeof(float);
}

ckda_status ckda_layernorm_bwd(const void* dy, const void* x, const float* mean,
                               const float* rstd, const void* weight, void* dx, void* dweight,
                               void* dbias, long long rows, int width, ckda_dtype io_dtype,
                               ckda_dtype weight_dtype, void* workspace, size_t workspace_bytes,
                               void* stream) {
  const ckda_status st = check_norm(rows, width, io_dtype, weight_dtype);
  if (st != CKDA_OK) return st;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return CKDA_ERR_INVALID_ARG;
  if ((dweight == nullptr) != (dbias == nullptr)) return CKDA_ERR_INVALID_ARG;
  if (dweight) {
    if (!workspace || workspace_bytes < ckda_layernorm_bwd_workspace_bytes(rows, width))
      return CKDA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 15) != 0) return CKDA_ERR_WORKSPACE;
  }
  NormArgs a{};
  a.x = x; a.dy = dy; a.w = weight; a.y = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.part = dweight ? static_cast<float*>(workspace) : nullptr;
  a.dw = dweight; a.db = dbias;
  a.rows = rows; a.D = width;
  a.parts = weight_parts(rows, width);
  return launch_any(a, io_dtype, weight_dtype, true, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? CKDA_OK
             : CKDA_ERR_CUDA;
}

}  // extern "C"
