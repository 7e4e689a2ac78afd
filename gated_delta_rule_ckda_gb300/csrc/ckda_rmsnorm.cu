// ckda_rmsnorm.cu -- root-mean-square norm over the last axis with the addition of a
// residual before it, forward (outputs in the I/O type, or in 8 bits with scales) and
// backward.
//
// Per row of D values, with r = 1 / sqrt(mean(h^2) + eps):
//     h_i  = x_i + residual_i         (rounded to the I/O type: the norm is of what is kept)
//     y_i  = h_i r w_i
//     dx_i = r [ t_i - xh_i mean(t xh) ] + dh_i,   t = dy w,  xh = h r
//     dw_i = sum over rows of dy_i xh_i
// In 8 bits, for a group of columns (or the row) with largest |y| = m:
//     scale = max(m, 2^-100) / 448,   y8_i = e4m3(y_i 448 / max(m, 2^-100))
// from y in fp32, so that a value is rounded once; the bound on m keeps the quotient
// finite for rows of zeros.
//
// A few flop per element: HBM bandwidth is the bound, each tensor once.  Rows are held in
// registers by 8, 16 or 32 lanes or by a block, in vectors of VEC elements, and come
// through a ring of S rows in shared memory that each thread fills for itself with
// cp.async.  The weight gradients go by a partial row a block and a second kernel that
// adds them in a fixed order and carries along what its additions round off: no atomics,
// the same bits every time.  (A thread's own sum, over its rows, is fp32: 1.6e-7 of dw over
// 16,384 rows is mostly that.)
#include <cuda_fp8.h>
#include "ckda_launch.cuh"
#include "ckda_rows.cuh"

namespace ckda {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kLeastMax = 7.888609052210118e-31f;  // 2^-100

struct RmsArgs {
  const void* x;    // forward: x; backward: h
  const void* add;  // forward: residual; backward: dh (each may be null)
  const void* dy;
  const void* w;
  void* h;
  void* y;  // dx in the backward pass
  float* scale;
  float* rstd;
  float* part;  // [parts][D] partial dw
  void* dw;
  long long rows;
  int D;
  int group;  // columns of a scale, 0: the row
  int parts;
  int w_bf16;
  float eps;
};

__device__ __forceinline__ float weight_of(const RmsArgs& a, int i) {
  if (!a.w) return 1.f;
  return a.w_bf16 ? ld_io(static_cast<const __nv_bfloat16*>(a.w) + i)
                  : static_cast<const float*>(a.w)[i];
}
template <typename IO>
__device__ __forceinline__ float rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ float rounded<__nv_bfloat16>(float v) {
  return __bfloat162float(__float2bfloat16_rn(v));
}
template <int VEC>
__device__ __forceinline__ void store_e4m3(void* base, long long at, const float (&f)[VEC]) {
  Pack<__nv_fp8_storage_t, VEC> p;
#pragma unroll
  for (int e = 0; e < VEC; ++e) p.v[e] = __nv_cvt_float_to_fp8(f[e], __NV_SATFINITE, __NV_E4M3);
  *reinterpret_cast<Pack<__nv_fp8_storage_t, VEC>*>(static_cast<uint8_t*>(base) + at) = p;
}
// The larger one, a NaN if either is: a scale shows what its values hold.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Rows ahead of up to MOST tensors (as many as are given) in shared memory: a thread
// copies what it reads itself.
template <typename IO, int VEC, int TB, int LPR, int NV, int S, int MOST>
struct Ahead {
  static constexpr int kBytes = sizeof(IO) * VEC;
  static constexpr bool kAsync = kBytes >= 4;
  using P = Pack<IO, VEC>;
  P* ring;
  const IO* src[MOST];
  int n_src, D, lane;
  static size_t smem(int n) { return kAsync ? (size_t)S * n * NV * TB * kBytes : 0; }
  __device__ __forceinline__ P* at(int stage, int t, int n) {
    return ring + ((size_t)(stage * n_src + t) * NV + n) * TB + threadIdx.x;
  }
  __device__ __forceinline__ void fetch(int stage, long long row, bool in) {
    if (!kAsync) return;
    if (in) {
#pragma unroll
      for (int t = 0; t < MOST; ++t)
        if (t < n_src)
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            const int i = (n * LPR + lane) * VEC;
            if (i < D) copy_async<kBytes >= 16 ? 16 : 4>(at(stage, t, n), src[t] + row * D + i);
          }
    }
    copy_commit();
  }
  __device__ __forceinline__ void read(int stage, long long row, int t, int n, float (&f)[VEC]) {
    const int i = (n * LPR + lane) * VEC;
    unpack<IO, VEC>(kAsync ? *at(stage, t, n) : *reinterpret_cast<const P*>(src[t] + row * D + i), f);
  }
};

template <int LANES>
__device__ __forceinline__ float lane_max(float s) {
#pragma unroll
  for (int m = LANES / 2; m >= 1; m >>= 1) s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, m));
  return s;
}
template <int TB, int LPR>
__device__ __forceinline__ float row_max(float s, float* red, int& turn) {
  if (LPR <= 32) return lane_max<LPR <= 32 ? LPR : 32>(s);
  s = lane_max<32>(s);
  float* r = red + (turn ^= 1) * (TB / 32);
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = s;
  __syncthreads();
  float t = r[0];
#pragma unroll
  for (int i = 1; i < TB / 32; ++i) t = max_nan(t, r[i]);
  return t;
}

// ------------------------------------------------------------------ forward
template <typename IO, bool OUT8, int VEC, int TB, int LPR, int NV, int S>
__global__ void __launch_bounds__(TB) rms_fwd_kernel(RmsArgs a) {
  constexpr int kGroups = TB / LPR;
  extern __shared__ __align__(16) char sm[];
  __shared__ float red[2 * TB / 32];
  using Ring = Ahead<IO, VEC, TB, LPR, NV, S, 2>;
  Ring ring;
  ring.ring = reinterpret_cast<typename Ring::P*>(sm);
  ring.src[0] = static_cast<const IO*>(a.x);
  ring.src[1] = static_cast<const IO*>(a.add);
  ring.n_src = a.add ? 2 : 1;
  ring.D = a.D;
  const int lane = ring.lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  const long long stride = (long long)gridDim.x * kGroups;
  long long r0 = (long long)blockIdx.x * kGroups;  // (the same in a block: barriers)
#pragma unroll
  for (int s = 0; s < S - 1; ++s) ring.fetch(s, r0 + s * stride + grp, r0 + s * stride + grp < a.rows);
  float w[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = (n * LPR + lane) * VEC + e;
      w[n][e] = i < a.D ? weight_of(a, i) : 0.f;
    }
  for (int stage = 0; r0 < a.rows; r0 += stride, stage = stage + 1 == S ? 0 : stage + 1) {
    const long long r = r0 + grp, ahead = r + (S - 1) * stride;
    const bool in = r < a.rows;
    ring.fetch(stage == 0 ? S - 1 : stage - 1, ahead, ahead < a.rows);
    if (Ring::kAsync) copy_wait<S - 1>();
    float x[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = (n * LPR + lane) * VEC;
      if (in && i < a.D) {
        ring.read(stage, r, 0, n, x[n]);
        if (a.add) {
          float f[VEC];
          ring.read(stage, r, 1, n, f);
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[n][e] = rounded<IO>(x[n][e] + f[e]);
          store_vec<IO, VEC>(a.h, r * a.D + i, x[n]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[n][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) s = fmaf(x[n][e], x[n][e], s);
    }
    const float rstd = 1.f / sqrtf(row_sum<TB, LPR>(s, red, turn) * inv_d + a.eps);
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[n][e] = x[n][e] * rstd * w[n][e];
    if (in && lane == 0) a.rstd[r] = rstd;
    if (!OUT8) {
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int i = (n * LPR + lane) * VEC;
        if (in && i < a.D) store_vec<IO, VEC>(a.y, r * a.D + i, x[n]);
      }
    } else {
      float m[NV];
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        m[n] = fabsf(x[n][0]);
#pragma unroll
        for (int e = 1; e < VEC; ++e) m[n] = max_nan(m[n], fabsf(x[n][e]));
      }
      if (a.group == 0) {
#pragma unroll
        for (int n = 1; n < NV; ++n) m[0] = max_nan(m[0], m[n]);
        const float top = max_nan(row_max<TB, LPR>(m[0], red, turn), kLeastMax);
        if (in && lane == 0) a.scale[r] = top / kE4m3Max;
#pragma unroll
        for (int n = 0; n < NV; ++n) m[n] = kE4m3Max / top;
      } else {  // a group is group / VEC lanes of one warp
        const int width = a.group / VEC;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          for (int k = width >> 1; k >= 1; k >>= 1)
            m[n] = max_nan(m[n], __shfl_xor_sync(0xffffffffu, m[n], k));
          const float top = max_nan(m[n], kLeastMax);
          const int i = (n * LPR + lane) * VEC;
          if (in && i < a.D && (lane & (width - 1)) == 0)
            a.scale[r * (a.D / a.group) + i / a.group] = top / kE4m3Max;
          m[n] = kE4m3Max / top;
        }
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int i = (n * LPR + lane) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[n][e] *= m[n];
        if (in && i < a.D) store_e4m3<VEC>(a.y, r * a.D + i, x[n]);
      }
    }
  }
}

// Rows wider than a block's registers: h is read again for the maximum and the output.
template <typename IO, bool OUT8>
__global__ void __launch_bounds__(1024) rms_fwd_long_kernel(RmsArgs a) {
  __shared__ float red[64];
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const IO* h = static_cast<const IO*>(a.x) + r * a.D;
    float s = 0.f;
    if (a.add) {
      const IO* x = h;
      const IO* res = static_cast<const IO*>(a.add) + r * a.D;
      IO* sum = static_cast<IO*>(a.h) + r * a.D;
      for (int i = threadIdx.x; i < a.D; i += 1024) {
        const float v = rounded<IO>(ld_io(x + i) + ld_io(res + i));
        st_io(sum + i, v);  // (read again by this thread alone)
        s = fmaf(v, v, s);
      }
      h = sum;
    } else {
      for (int i = threadIdx.x; i < a.D; i += 1024) s = fmaf(ld_io(h + i), ld_io(h + i), s);
    }
    const float rstd = 1.f / sqrtf(row_sum<1024, 1024>(s, red, turn) * inv_d + a.eps);
    if (threadIdx.x == 0) a.rstd[r] = rstd;
    if (!OUT8) {
      IO* y = static_cast<IO*>(a.y) + r * a.D;
      for (int i = threadIdx.x; i < a.D; i += 1024) st_io(y + i, ld_io(h + i) * rstd * weight_of(a, i));
    } else {
      // groups are runs of `group` threads within the 1024 columns of a step; a warp is in
      // one group or holds whole ones
      uint8_t* y = static_cast<uint8_t*>(a.y) + r * a.D;
      const int per = a.group == 0 ? a.D : a.group;
      float top = 0.f;
      if (a.group == 0) {
        for (int i = threadIdx.x; i < a.D; i += 1024)
          top = max_nan(top, fabsf(ld_io(h + i) * rstd * weight_of(a, i)));
        top = max_nan(row_max<1024, 1024>(top, red, turn), kLeastMax);
        if (threadIdx.x == 0) a.scale[r] = top / kE4m3Max;
      }
      for (int i0 = 0; i0 < a.D; i0 += 1024) {
        const int i = i0 + (int)threadIdx.x;
        const float v = i < a.D ? ld_io(h + i) * rstd * weight_of(a, i) : 0.f;
        if (a.group != 0) {
          const int warps = per / 32;
          float m = lane_max<32>(fabsf(v));
          float* q = red + (turn ^= 1) * 32;
          if ((threadIdx.x & 31) == 0) q[threadIdx.x >> 5] = m;
          __syncthreads();
          const int first = (int)(threadIdx.x >> 5) / warps * warps;
          m = q[first];
          for (int k = 1; k < warps; ++k) m = max_nan(m, q[first + k]);
          top = max_nan(m, kLeastMax);
          if (i < a.D && i % per == 0) a.scale[r * (a.D / per) + i / per] = top / kE4m3Max;
        }
        if (i < a.D) y[i] = __nv_cvt_float_to_fp8(v * (kE4m3Max / top), __NV_SATFINITE, __NV_E4M3);
      }
    }
  }
}

// ----------------------------------------------------------------- backward
template <typename IO, int VEC, int TB, int LPR, int NV, int S>
__global__ void __launch_bounds__(TB) rms_bwd_kernel(RmsArgs a) {
  let_next_start();
  constexpr int kGroups = TB / LPR;
  extern __shared__ __align__(16) char sm[];
  __shared__ float red[2 * TB / 32];
  using Ring = Ahead<IO, VEC, TB, LPR, NV, S, 3>;
  Ring ring;
  ring.ring = reinterpret_cast<typename Ring::P*>(sm);
  ring.src[0] = static_cast<const IO*>(a.x);
  ring.src[1] = static_cast<const IO*>(a.dy);
  ring.src[2] = static_cast<const IO*>(a.add);
  ring.n_src = a.add ? 3 : 2;
  ring.D = a.D;
  const int lane = ring.lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  using V = typename Pairs<VEC>::V;
  constexpr int kN = Pairs<VEC>::kN;
  const long long stride = (long long)gridDim.x * kGroups;
  long long r0 = (long long)blockIdx.x * kGroups;
#pragma unroll
  for (int s = 0; s < S - 1; ++s) ring.fetch(s, r0 + s * stride + grp, r0 + s * stride + grp < a.rows);
  float rstd_next = r0 + grp < a.rows ? a.rstd[r0 + grp] : 0.f;
  V w[NV][kN], dw[NV][kN];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = (n * LPR + lane) * VEC + e;
      f[e] = i < a.D ? weight_of(a, i) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      w[n][e] = reinterpret_cast<const V*>(f)[e];
      dw[n][e] = both<V>(0.f);
    }
  }
  for (int stage = 0; r0 < a.rows; r0 += stride, stage = stage + 1 == S ? 0 : stage + 1) {
    const long long r = r0 + grp, ahead = r + (S - 1) * stride;
    const bool in = r < a.rows;
    ring.fetch(stage == 0 ? S - 1 : stage - 1, ahead, ahead < a.rows);
    const float rstd = rstd_next;  // (a row ahead: its load would add its latency to every row)
    if (r + stride < a.rows) rstd_next = a.rstd[r + stride];
    if (Ring::kAsync) copy_wait<S - 1>();
    V xh[NV][kN], t[NV][kN];
    V p = both<V>(0.f);
    const V scale = both<V>(rstd);
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (in && (n * LPR + lane) * VEC < a.D) {
        float x[VEC], g[VEC];
        ring.read(stage, r, 0, n, x);
        ring.read(stage, r, 1, n, g);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const V gv = reinterpret_cast<const V*>(g)[e];
          xh[n][e] = mul_(reinterpret_cast<const V*>(x)[e], scale);
          dw[n][e] = fma_(gv, xh[n][e], dw[n][e]);
          t[n][e] = mul_(gv, w[n][e]);
          p = fma_(t[n][e], xh[n][e], p);
        }
      }
    const float m = row_sum<TB, LPR>(sum_of(p), red, turn) * inv_d;
    const V minus_m = both<V>(-m);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = (n * LPR + lane) * VEC;
      if (in && i < a.D) {
        float o[VEC], f[VEC];
        if (a.add) {
          ring.read(stage, r, 2, n, f);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) f[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < kN; ++e)
          reinterpret_cast<V*>(o)[e] = fma_(fma_(xh[n][e], minus_m, t[n][e]), scale,
                                            reinterpret_cast<const V*>(f)[e]);
        store_vec<IO, VEC>(a.y, r * a.D + i, o);
      }
    }
  }
  if (!a.part) return;
  if (LPR > 32) {
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int i = (n * LPR + lane) * VEC + e;
        if (i < a.D) a.part[(size_t)blockIdx.x * a.D + i] = reinterpret_cast<const float*>(dw[n])[e];
      }
    return;
  }
  // the block's groups, through shared memory ([kGroups][D]), in order
  float* part_s = reinterpret_cast<float*>(sm);
  if (Ring::kAsync) copy_wait<0>();
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = (n * LPR + lane) * VEC + e;
      if (i < a.D) part_s[grp * a.D + i] = reinterpret_cast<const float*>(dw[n])[e];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < a.D; i += TB) {
    CarriedSum s;
#pragma unroll 8
    for (int g = 0; g < kGroups; ++g) s.add(part_s[g * a.D + i]);
    a.part[(size_t)blockIdx.x * a.D + i] = s.sum;
  }
}

// Rows wider than a block's registers: the block keeps its partial sums in its row of
// the workspace.
template <typename IO>
__global__ void __launch_bounds__(1024) rms_bwd_long_kernel(RmsArgs a) {
  let_next_start();
  __shared__ float red[64];
  const float inv_d = 1.f / (float)a.D;
  float* pw = a.part ? a.part + (size_t)blockIdx.x * a.D : nullptr;
  bool first = true;
  int turn = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const IO* h = static_cast<const IO*>(a.x) + r * a.D;
    const IO* dy = static_cast<const IO*>(a.dy) + r * a.D;
    const IO* dh = a.add ? static_cast<const IO*>(a.add) + r * a.D : nullptr;
    IO* dx = static_cast<IO*>(a.y) + r * a.D;
    const float rstd = a.rstd[r];
    float s = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 1024) {
      const float xh = ld_io(h + i) * rstd, g = ld_io(dy + i);
      s = fmaf(g * weight_of(a, i), xh, s);
      if (pw) pw[i] = fmaf(g, xh, first ? 0.f : pw[i]);  // (column i is this thread's)
    }
    first = false;
    const float m = row_sum<1024, 1024>(s, red, turn) * inv_d;
    for (int i = threadIdx.x; i < a.D; i += 1024) {
      const float xh = ld_io(h + i) * rstd, t = ld_io(dy + i) * weight_of(a, i);
      st_io(dx + i, fmaf(t - xh * m, rstd, dh ? ld_io(dh + i) : 0.f));
    }
  }
}

// dw from the partial rows: 32 columns to a block, 32 threads a column over the partial
// rows, joined in a fixed order by a warp a column.
__global__ void __launch_bounds__(1024) rms_weight_grad_kernel(RmsArgs a) {
  after_previous();
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + c;
  CarriedSum t;
  if (i < a.D)
#pragma unroll 8
    for (int r = g; r < a.parts; r += 32) t.add(a.part[(size_t)r * a.D + i]);
  s[g][c] = t.sum;
  __syncthreads();
  const float all = lane_sum<32>(s[c][g]);  // of the block's column g
  const int own = blockIdx.x * 32 + g;
  if (c == 0 && own < a.D) {
    if (a.w_bf16)
      st_io(static_cast<__nv_bfloat16*>(a.dw) + own, all);
    else
      static_cast<float*>(a.dw)[own] = all;
  }
}

// ------------------------------------------------------- widths of odd bytes
// Rows whose bytes are no multiple of 16, on bases that are: a row starts somewhere in a
// 16-byte vector, so whole vectors come to shared memory as they lie, threads take single
// columns of it (LPR apart, NV each: weights stay with their columns), leave the results in
// its place, and whole vectors go out again; what a row shares a vector with stays untouched.
// Rows of whole vectors that are wider than a block's registers hold in vectors (fp32 past
// 8192 columns) go this way too.  One warp a row, or a block.  8,489 rows of 4853 in bf16 with
// a residual: 103 us forward (48% of the copy bandwidth), 153 backward, which took 363 by
// single elements from memory.
template <typename IO>
struct OddRow {
  const long long start;  // the row's first byte
  const int shift, bytes, vecs;
  __device__ __forceinline__ OddRow(long long row, int D, int size)
      : start(row * D * size), shift((int)(start & 15)), bytes(D * size), vecs((shift + bytes + 15) / 16) {}
  // (a vector past the tensor's end is copied as far as the tensor goes)
  __device__ __forceinline__ void fetch(char* to, const void* base, long long total, int lane, int lanes) const {
    const char* from = static_cast<const char*>(base) + (start - shift);
    for (int v = lane; v < vecs; v += lanes) {
      const long long left = total - (start - shift) - 16LL * v;
      const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to + 16 * v));
      const int n = left < 16 ? (int)left : 16;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from + 16 * v), "r"(n) : "memory");
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(void* base, const char* from, int lane, int lanes) const {
    char* to = static_cast<char*>(base) + (start - shift);
    for (int v = lane; v < vecs; v += lanes) {
      const int lo = v == 0 ? shift : 0, hi = 16 * v + 16 <= shift + bytes ? 16 : shift + bytes - 16 * v;
      if (lo == 0 && hi == 16) {
        *reinterpret_cast<uint4*>(to + 16 * v) = *reinterpret_cast<const uint4*>(from + 16 * v);
      } else {
        for (int i = lo; i < hi; i += (int)sizeof(T))
          *reinterpret_cast<T*>(to + 16 * v + i) = *reinterpret_cast<const T*>(from + 16 * v + i);
      }
    }
  }
};
template <int LPR>
__device__ __forceinline__ void row_sync() {
  if (LPR <= 32)
    __syncwarp();
  else
    __syncthreads();
}
// Bytes of a row in shared memory.
inline __host__ __device__ int odd_span(int D, int size) { return (D * size + 15) / 16 * 16 + 16; }

template <typename IO, bool OUT8, int TB, int LPR, int NV>
__global__ void __launch_bounds__(TB) rms_fwd_odd_kernel(RmsArgs a, int stages) {
  extern __shared__ __align__(16) char sm[];
  __shared__ float red[2 * TB / 32];
  constexpr int kGroups = TB / LPR;
  const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, n_in = a.add ? 2 : 1;
  const int span = odd_span(a.D, sizeof(IO));
  char* const buf = sm + (size_t)grp * stages * n_in * span;
  const long long total = a.rows * a.D * (long long)sizeof(IO);
  const long long stride = (long long)gridDim.x * kGroups;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  const auto fetch = [&](long long r, int stage) {
    if (r < a.rows) {
      const OddRow<IO> row(r, a.D, sizeof(IO));
      row.fetch(buf + (size_t)stage * n_in * span, a.x, total, lane, LPR);
      if (a.add) row.fetch(buf + ((size_t)stage * n_in + 1) * span, a.add, total, lane, LPR);
    }
    copy_commit();
  };
  long long r0 = (long long)blockIdx.x * kGroups;  // (the same in a block: barriers)
  for (int s = 0; s < stages; ++s) fetch(r0 + grp + s * stride, s);
  float w[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) w[n] = n * LPR + lane < a.D ? weight_of(a, n * LPR + lane) : 0.f;
  for (int stage = 0; r0 < a.rows; r0 += stride, stage = stage + 1 == stages ? 0 : stage + 1) {
    const long long r = r0 + grp;
    const bool in = r < a.rows;
    if (stages == 1)
      copy_wait<0>();
    else
      copy_wait<1>();
    row_sync<LPR>();
    const OddRow<IO> row(in ? r : 0, a.D, sizeof(IO));
    char* const raw = buf + (size_t)stage * n_in * span;
    IO* const x = reinterpret_cast<IO*>(raw + row.shift);
    IO* const res = reinterpret_cast<IO*>(raw + span + row.shift);
    float h[NV];
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = n * LPR + lane;
      h[n] = 0.f;
      if (in && i < a.D) {
        h[n] = ld_io(x + i);
        if (a.add) {
          h[n] = rounded<IO>(h[n] + ld_io(res + i));
          st_io(x + i, h[n]);
        }
      }
      s = fmaf(h[n], h[n], s);
    }
    const float rstd = 1.f / sqrtf(row_sum<TB, LPR>(s, red, turn) * inv_d + a.eps);
    if (in && lane == 0) a.rstd[r] = rstd;
    float top = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      h[n] = h[n] * rstd * w[n];
      if (OUT8) top = max_nan(top, fabsf(h[n]));
    }
    // y in the place of the residual, or of x where nothing else goes out from there
    char* const out = a.add ? raw + span : raw;
    if (OUT8) {
      top = max_nan(row_max<TB, LPR>(top, red, turn), kLeastMax);
      if (in && lane == 0) a.scale[r] = top / kE4m3Max;
      const float scale = kE4m3Max / top;
      uint8_t* const y = reinterpret_cast<uint8_t*>(out) + (r * a.D & 15);
      row_sync<LPR>();  // (bytes lie over other columns)
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (in && n * LPR + lane < a.D)
          y[n * LPR + lane] = __nv_cvt_float_to_fp8(h[n] * scale, __NV_SATFINITE, __NV_E4M3);
    } else {
      IO* const y = reinterpret_cast<IO*>(out + row.shift);
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (in && n * LPR + lane < a.D) st_io(y + n * LPR + lane, h[n]);
    }
    row_sync<LPR>();
    if (in) {
      if (a.add) row.template store<IO>(a.h, raw, lane, LPR);
      if (OUT8)
        OddRow<IO>(r, a.D, 1).template store<uint8_t>(a.y, out, lane, LPR);
      else
        row.template store<IO>(a.y, out, lane, LPR);
    }
    row_sync<LPR>();
    fetch(r + stages * stride, stage);
  }
}

template <typename IO, int TB, int LPR, int NV>
__global__ void __launch_bounds__(TB) rms_bwd_odd_kernel(RmsArgs a, int stages) {
  let_next_start();
  extern __shared__ __align__(16) char sm[];
  __shared__ float red[2 * TB / 32];
  constexpr int kGroups = TB / LPR;
  const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, n_in = a.add ? 3 : 2;
  const int span = odd_span(a.D, sizeof(IO));
  char* const buf = sm + (size_t)grp * stages * n_in * span;
  const long long total = a.rows * a.D * (long long)sizeof(IO);
  const long long stride = (long long)gridDim.x * kGroups;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  const auto fetch = [&](long long r, int stage) {
    if (r < a.rows) {
      const OddRow<IO> row(r, a.D, sizeof(IO));
      char* const to = buf + (size_t)stage * n_in * span;
      row.fetch(to, a.x, total, lane, LPR);
      row.fetch(to + span, a.dy, total, lane, LPR);
      if (a.add) row.fetch(to + 2 * span, a.add, total, lane, LPR);
    }
    copy_commit();
  };
  long long r0 = (long long)blockIdx.x * kGroups;
  for (int s = 0; s < stages; ++s) fetch(r0 + grp + s * stride, s);
  float w[NV], dw[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    w[n] = n * LPR + lane < a.D ? weight_of(a, n * LPR + lane) : 0.f;
    dw[n] = 0.f;
  }
  for (int stage = 0; r0 < a.rows; r0 += stride, stage = stage + 1 == stages ? 0 : stage + 1) {
    const long long r = r0 + grp;
    const bool in = r < a.rows;
    const float rstd = in ? a.rstd[r] : 0.f;
    if (stages == 1)
      copy_wait<0>();
    else
      copy_wait<1>();
    row_sync<LPR>();
    const OddRow<IO> row(in ? r : 0, a.D, sizeof(IO));
    char* const raw = buf + (size_t)stage * n_in * span;
    const IO* const h = reinterpret_cast<const IO*>(raw + row.shift);
    IO* const dy = reinterpret_cast<IO*>(raw + span + row.shift);
    const IO* const dh = reinterpret_cast<const IO*>(raw + 2 * span + row.shift);
    float xh[NV], t[NV];
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = n * LPR + lane;
      xh[n] = t[n] = 0.f;
      if (in && i < a.D) {
        const float g = ld_io(dy + i);
        xh[n] = ld_io(h + i) * rstd;
        dw[n] = fmaf(g, xh[n], dw[n]);
        t[n] = g * w[n];
      }
      s = fmaf(t[n], xh[n], s);
    }
    const float m = row_sum<TB, LPR>(s, red, turn) * inv_d;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = n * LPR + lane;
      if (in && i < a.D) st_io(dy + i, fmaf(t[n] - xh[n] * m, rstd, a.add ? ld_io(dh + i) : 0.f));
    }
    row_sync<LPR>();
    if (in) row.template store<IO>(a.y, raw + span, lane, LPR);
    row_sync<LPR>();
    fetch(r + stages * stride, stage);
  }
  if (!a.part) return;
  if (LPR > 32) {
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (n * LPR + lane < a.D) a.part[(size_t)blockIdx.x * a.D + n * LPR + lane] = dw[n];
    return;
  }
  // the block's warps, through shared memory ([kGroups][D]), in order
  float* part_s = reinterpret_cast<float*>(sm);
  copy_wait<0>();
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NV; ++n)
    if (n * LPR + lane < a.D) part_s[grp * a.D + n * LPR + lane] = dw[n];
  __syncthreads();
  for (int i = threadIdx.x; i < a.D; i += TB) {
    CarriedSum s;
    for (int g = 0; g < kGroups; ++g) s.add(part_s[g * a.D + i]);
    a.part[(size_t)blockIdx.x * a.D + i] = s.sum;
  }
}

// ----------------------------------------------------------------- dispatch
template <typename F>
cudaError_t allow_smem(F kernel, size_t smem) {
  if (smem <= 40 * 1024) return cudaSuccess;  // (the static part counts towards the default 48 KB)
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}
inline int weight_parts(long long rows, int D) { return blocks_for(rows, D <= 2048 ? 8 : 3); }

template <typename IO, bool OUT8, int VEC, int TB, int LPR, int NV, int S>
cudaError_t run_fwd(const RmsArgs& a, int per_sm, cudaStream_t s) {
  const size_t smem = Ahead<IO, VEC, TB, LPR, NV, S, 2>::smem(a.add ? 2 : 1);
  const auto kernel = rms_fwd_kernel<IO, OUT8, VEC, TB, LPR, NV, S>;
  const cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  constexpr int kGroups = TB / LPR;
  kernel<<<blocks_for((a.rows + kGroups - 1) / kGroups, per_sm), TB, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename IO, int VEC, int TB, int LPR, int NV, int S>
cudaError_t run_bwd(RmsArgs& a, int per_sm, cudaStream_t s) {
  const size_t ring = Ahead<IO, VEC, TB, LPR, NV, S, 3>::smem(a.add ? 3 : 2);
  const size_t join = LPR <= 32 ? (size_t)(TB / LPR) * a.D * sizeof(float) : 0;
  const size_t smem = ring > join ? ring : join;
  const auto kernel = rms_bwd_kernel<IO, VEC, TB, LPR, NV, S>;
  const cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  const int parts = blocks_for((a.rows + TB / LPR - 1) / (TB / LPR), per_sm);
  a.parts = parts < a.parts ? parts : a.parts;
  kernel<<<a.parts, TB, smem, s>>>(a);
  return cudaGetLastError();
}

// Threads of a row by its width, as for layer norm: the fewest lanes that hold it in one
// or two vectors each, a warp at most, else a block.  16,384 rows of 4096 with a residual,
// forward in 8 bits: blocks of 256 threads, three an SM 83 us, four 89, six 81; of 128
// threads 87, of 512 94.  Backward: 128 threads of four vectors, three blocks an SM, 100
// us; 256 of two, two blocks 116, three 142 (three tensors' rows in shorter runs).
template <typename IO, bool OUT8, int VEC>
cudaError_t fwd_by_width(const RmsArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 8 * VEC) return run_fwd<IO, OUT8, VEC, 256, 8, 1, 4>(a, 8, s);
  if (D <= 16 * VEC) return run_fwd<IO, OUT8, VEC, 256, 16, 1, 4>(a, 8, s);
  if (D <= 32 * VEC) return run_fwd<IO, OUT8, VEC, 256, 32, 1, 4>(a, 8, s);
  if (D <= 64 * VEC) return run_fwd<IO, OUT8, VEC, 256, 32, 2, 3>(a, 8, s);
  if (D <= 128 * VEC) return run_fwd<IO, OUT8, VEC, 128, 128, 1, 4>(a, 16, s);
  if (D <= 256 * VEC) return run_fwd<IO, OUT8, VEC, 128, 128, 2, 4>(a, 12, s);
  if (D <= 512 * VEC) return run_fwd<IO, OUT8, VEC, 256, 256, 2, 3>(a, 6, s);
  if (D <= 1024 * VEC) return run_fwd<IO, OUT8, VEC, 512, 512, 2, 3>(a, 2, s);
  if (D <= 2048 * VEC) return run_fwd<IO, OUT8, VEC, 512, 512, 4, 2>(a, 2, s);
  rms_fwd_long_kernel<IO, OUT8><<<blocks_for(a.rows, 2), 1024, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename IO, int VEC>
cudaError_t bwd_by_width(RmsArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 8 * VEC) return run_bwd<IO, VEC, 256, 8, 1, 4>(a, 4, s);
  if (D <= 16 * VEC) return run_bwd<IO, VEC, 256, 16, 1, 4>(a, 4, s);
  if (D <= 32 * VEC) return run_bwd<IO, VEC, 256, 32, 1, 4>(a, 4, s);
  if (D <= 64 * VEC) return run_bwd<IO, VEC, 256, 32, 2, 3>(a, 4, s);
  if (D <= 128 * VEC) return run_bwd<IO, VEC, 128, 128, 1, 4>(a, 8, s);
  if (D <= 256 * VEC) return run_bwd<IO, VEC, 128, 128, 2, 3>(a, 4, s);
  if (D <= 512 * VEC) return run_bwd<IO, VEC, 128, 128, 4, 3>(a, 3, s);
  if (D <= 1024 * VEC) return run_bwd<IO, VEC, 512, 512, 2, 2>(a, 2, s);
  if constexpr (VEC > 1)
    if (D <= 2048 * VEC) return run_bwd<IO, VEC, 1024, 1024, 2, 2>(a, 1, s);
  if (VEC == 1 && D <= 2048) return run_bwd<IO, VEC, 512, 512, VEC == 1 ? 4 : 2, 2>(a, 2, s);
  a.parts = blocks_for(a.rows, 2);
  rms_bwd_long_kernel<IO><<<a.parts, 1024, 0, s>>>(a);
  return cudaGetLastError();
}

// Two rows on their way to a warp or block where they fit, and as many blocks an SM as
// shared memory and 64 registers a thread leave room for.
struct OddPlan {
  int stages, blocks;
  size_t smem;
};
inline OddPlan odd_plan(long long rows, int D, int size, int n_in, int TB, int LPR, bool join) {
  OddPlan p;
  const size_t one = (size_t)(TB / LPR) * n_in * odd_span(D, size);
  p.stages = 2 * one <= 200 * 1024 ? 2 : 1;
  p.smem = p.stages * one;
  const size_t sums = join ? (size_t)(TB / LPR) * D * sizeof(float) : 0;
  if (p.smem < sums) p.smem = sums;
  int per_sm = (int)(220 * 1024 / (p.smem + 1024));
  if (per_sm > 1024 / TB) per_sm = 1024 / TB;
  if (per_sm < 1) per_sm = 1;
  p.blocks = blocks_for((rows + TB / LPR - 1) / (TB / LPR), per_sm);
  return p;
}
template <typename IO, bool OUT8, int TB, int LPR, int NV>
cudaError_t run_fwd_odd(const RmsArgs& a, cudaStream_t s) {
  const OddPlan p = odd_plan(a.rows, a.D, sizeof(IO), a.add ? 2 : 1, TB, LPR, false);
  const auto kernel = rms_fwd_odd_kernel<IO, OUT8, TB, LPR, NV>;
  const cudaError_t e = allow_smem(kernel, p.smem);
  if (e != cudaSuccess) return e;
  kernel<<<p.blocks, TB, p.smem, s>>>(a, p.stages);
  return cudaGetLastError();
}
template <typename IO, int TB, int LPR, int NV>
cudaError_t run_bwd_odd(RmsArgs& a, cudaStream_t s) {
  OddPlan p = odd_plan(a.rows, a.D, sizeof(IO), a.add ? 3 : 2, TB, LPR, LPR <= 32);
  if (p.blocks > a.parts) p.blocks = a.parts;
  const auto kernel = rms_bwd_odd_kernel<IO, TB, LPR, NV>;
  const cudaError_t e = allow_smem(kernel, p.smem);
  if (e != cudaSuccess) return e;
  a.parts = p.blocks;
  kernel<<<p.blocks, TB, p.smem, s>>>(a, p.stages);
  return cudaGetLastError();
}
// The widest rows that these kernels hold, and the widest in vectors of VEC elements.  Rows
// between the two (fp32, 4096 of 16,384 columns) with a residual take 213 us forward, 207 to 8
// bits and 292 backward; by the kernels that read a row again, which wider ones need, 242,
// 441 and 574.  (A few rows are as long under way in both: 7 of them 20 to 29 us and 18 to 26.)
constexpr int kOddMost = 16384;
template <int VEC>
constexpr int kVectorsMost = 2048 * VEC;
template <typename IO, bool OUT8>
cudaError_t fwd_odd(const RmsArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 128) return run_fwd_odd<IO, OUT8, 256, 32, 4>(a, s);
  if (D <= 512) return run_fwd_odd<IO, OUT8, 256, 32, 16>(a, s);
  if (D <= 1024) return run_fwd_odd<IO, OUT8, 64, 64, 16>(a, s);
  if (D <= 2048) return run_fwd_odd<IO, OUT8, 128, 128, 16>(a, s);
  if (D <= 4096) return run_fwd_odd<IO, OUT8, 256, 256, 16>(a, s);
  if (D <= 8192) return run_fwd_odd<IO, OUT8, 512, 512, 16>(a, s);
  return run_fwd_odd<IO, OUT8, 1024, 1024, 16>(a, s);
}
template <typename IO>
cudaError_t bwd_odd(RmsArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 128) return run_bwd_odd<IO, 256, 32, 4>(a, s);
  if (D <= 512) return run_bwd_odd<IO, 256, 32, 16>(a, s);
  if (D <= 1024) return run_bwd_odd<IO, 64, 64, 16>(a, s);
  if (D <= 2048) return run_bwd_odd<IO, 128, 128, 16>(a, s);
  if (D <= 4096) return run_bwd_odd<IO, 256, 256, 16>(a, s);
  if (D <= 8192) return run_bwd_odd<IO, 512, 512, 16>(a, s);
  return run_bwd_odd<IO, 1024, 1024, 16>(a, s);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename IO, bool OUT8>
cudaError_t launch_fwd_rows(const RmsArgs& a, cudaStream_t s) {
  constexpr int kVec = 16 / sizeof(IO);
  // (8-bit outputs are stored in vectors of kVec bytes)
  const bool aligned = aligned16(a.x) && aligned16(a.add) && aligned16(a.h) && aligned16(a.y);
  const bool held = aligned && a.D <= kOddMost && a.group == 0;
  if (aligned && a.D % kVec == 0 && (a.D <= kVectorsMost<kVec> || !held)) return fwd_by_width<IO, OUT8, kVec>(a, s);
  if (held) return fwd_odd<IO, OUT8>(a, s);
  if (OUT8 && a.group != 0) {  // groups across warps: the kernel that reads again
    rms_fwd_long_kernel<IO, OUT8><<<blocks_for(a.rows, 2), 1024, 0, s>>>(a);
    return cudaGetLastError();
  }
  return fwd_by_width<IO, OUT8, 1>(a, s);
}
template <typename IO>
cudaError_t launch_bwd_rows(RmsArgs a, cudaStream_t s) {
  constexpr int kVec = 16 / sizeof(IO);
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    const bool aligned = aligned16(a.x) && aligned16(a.dy) && aligned16(a.add) && aligned16(a.y);
    const bool held = aligned && a.D <= kOddMost;
    if (aligned && a.D % kVec == 0 && (a.D <= kVectorsMost<kVec> || !held))
      e = bwd_by_width<IO, kVec>(a, s);
    else
      e = held ? bwd_odd<IO>(a, s) : bwd_by_width<IO, 1>(a, s);
    if (e != cudaSuccess) return e;
  }
  if (a.part) {
    if (a.rows == 0) a.parts = 0;  // the sums over no rows are zero
    e = launch_next(a.rows > 0, rms_weight_grad_kernel, dim3((a.D + 31) / 32), 1024, 0, s, a);
  }
  return e;
}

ckda_status check_rms(long long rows, int width, ckda_dtype io, ckda_dtype wt) {
  if (io != CKDA_F32 && io != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
  if (wt != CKDA_F32 && wt != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
  if (rows < 0 || width < 1) return CKDA_ERR_INVALID_ARG;
  // (columns are counted in 32 bits, up to a block's step past the row)
  if (rows > 0x7fffffffLL || width > 1 << 30) return CKDA_ERR_UNSUPPORTED;
  return CKDA_OK;
}
ckda_status forward(const void* x, const void* residual, const void* weight, void* h, void* y,
                    float* scale, float* rstd, long long rows, int width, int group,
                    ckda_dtype io, ckda_dtype wt, float eps, bool out8, void* stream) {
  const ckda_status st = check_rms(rows, width, io, wt);
  if (st != CKDA_OK) return st;
  if (!(eps >= 0.f) || eps > 3.0e38f) return CKDA_ERR_INVALID_ARG;
  if ((residual == nullptr) != (h == nullptr)) return CKDA_ERR_INVALID_ARG;
  if (group != 0 && ((group != 32 && group != 64 && group != 128) || width % group != 0))
    return CKDA_ERR_INVALID_ARG;
  if (rows == 0) return CKDA_OK;
  if (!x || !y || !rstd || (out8 && !scale) || h == y) return CKDA_ERR_INVALID_ARG;
  // (a block that writes a row runs beside blocks that still read others)
  const size_t io_bytes = io == CKDA_F32 ? 4 : 2, in = rows_bytes(rows, width, width, io_bytes),
               out = out8 ? rows_bytes(rows, width, width, 1) : in;
  if (clash(h, x, rows, width, width, io_bytes) || clash(h, residual, rows, width, width, io_bytes) ||
      overlap(h, in, y, out))
    return CKDA_ERR_INVALID_ARG;
  if (out8 ? overlap(y, out, x, in) || overlap(y, out, residual, in)
           : clash(y, x, rows, width, width, io_bytes) || clash(y, residual, rows, width, width, io_bytes))
    return CKDA_ERR_INVALID_ARG;
  RmsArgs a{};
  a.x = x; a.add = residual; a.w = weight; a.h = h; a.y = y; a.scale = scale; a.rstd = rstd;
  a.rows = rows; a.D = width; a.group = group; a.w_bf16 = wt == CKDA_BF16; a.eps = eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      io == CKDA_F32 ? (out8 ? launch_fwd_rows<float, true>(a, s) : launch_fwd_rows<float, false>(a, s))
                     : (out8 ? launch_fwd_rows<__nv_bfloat16, true>(a, s)
                             : launch_fwd_rows<__nv_bfloat16, false>(a, s));
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // namespace
}  // namespace ckda

using namespace ckda;

extern "C" {

ckda_status ckda_rmsnorm_fwd(const void* x, const void* residual, const void* weight, void* h,
                             void* y, float* rstd, long long rows, int width, ckda_dtype io_dtype,
                             ckda_dtype weight_dtype, float eps, void* stream) {
  return forward(x, residual, weight, h, y, nullptr, rstd, rows, width, 0, io_dtype, weight_dtype,
                 eps, false, stream);
}

ckda_status ckda_rmsnorm_fwd8(const void* x, const void* residual, const void* weight, void* h,
                              void* y8, float* scale, float* rstd, long long rows, int width,
                              int group, ckda_dtype io_dtype, ckda_dtype weight_dtype, float eps,
                              void* stream) {
  return forward(x, residual, weight, h, y8, scale, rstd, rows, width, group, io_dtype,
                 weight_dtype, eps, true, stream);
}

size_t ckda_rmsnorm_bwd_workspace_bytes(long long rows, int width) {
  if (rows < 0 || width < 1) return 0;
  return (size_t)weight_parts(rows, width) * width * sizeof(float);
}

ckda_status ckda_rmsnorm_bwd(const void* dy, const void* h, const float* rstd, const void* weight,
                             const void* dh, void* dx, void* dweight, long long rows, int width,
                             ckda_dtype io_dtype, ckda_dtype weight_dtype, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const ckda_status st = check_rms(rows, width, io_dtype, weight_dtype);
  if (st != CKDA_OK) return st;
  if (rows > 0 && (!dy || !h || !rstd || !dx)) return CKDA_ERR_INVALID_ARG;
  if (dweight) {
    if (!workspace || workspace_bytes < ckda_rmsnorm_bwd_workspace_bytes(rows, width) ||
        !aligned16(workspace))
      return CKDA_ERR_WORKSPACE;
  }
  const size_t io = io_dtype == CKDA_F32 ? 4 : 2;
  for (const void* in : {dy, h, dh})
    if (clash(dx, in, rows, width, width, io)) return CKDA_ERR_INVALID_ARG;
  RmsArgs a{};
  a.x = h; a.dy = dy; a.add = dh; a.w = weight; a.y = dx;
  a.rstd = const_cast<float*>(rstd);
  a.part = dweight ? static_cast<float*>(workspace) : nullptr;
  a.dw = dweight;
  a.rows = rows; a.D = width; a.w_bf16 = weight_dtype == CKDA_BF16;
  a.parts = weight_parts(rows, width);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = io_dtype == CKDA_F32 ? launch_bwd_rows<float>(a, s)
                                             : launch_bwd_rows<__nv_bfloat16>(a, s);
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // extern "C"
