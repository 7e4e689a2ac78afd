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
// in registers by the threads that own it, in vectors of VEC elements: LPR = 8,
// 16 or 32 lanes for narrow rows (several to a warp), a block for wide
// ones.  What keeps enough bytes in flight is a ring of S rows a thread group in
// shared memory, filled with cp.async: a thread copies only what it will read
// itself, so the ring needs no barrier and the loads no registers.
// Rows wider than a block's registers hold are read again for each of the sums
// (the second and third reads hit L2).
//
// The weight gradients are sums over rows for every column: a block walks its
// rows with one fp32 partial sum a column in the registers of the thread that
// owns the column, writes one partial row to the workspace, and a second
// kernel adds the partial rows in a fixed order.  No atomics: two calls on the
// same input give the same bits.
//
// Measured, bf16 with fp32 weights: forward of 1,048,576 rows of 128 94 us, 85% of the
// copy bandwidth; backward of 16,384 rows of 4096 82 us, 72% (76 us the rows, the rest
// the second kernel and its start); backward of 2,999 rows of 1031 in fp32 25 to 28 us,
// 17 and 5 of them the kernels, the rest launches and the host.
#include "ckda_internal.cuh"
#include "ckda_launch.cuh"

namespace ckda {
namespace {

constexpr int kSms = 152;

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
template <typename IO, int VEC>
__device__ __forceinline__ void unpack(const Pack<IO, VEC>& p, float (&f)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) f[e] = ld_io(&p.v[e]);
}
template <typename IO, int VEC>
__device__ __forceinline__ void store_vec(void* base, long long at, const float (&f)[VEC]) {
  Pack<IO, VEC> p;
#pragma unroll
  for (int e = 0; e < VEC; ++e) st_io(&p.v[e], f[e]);
  *reinterpret_cast<Pack<IO, VEC>*>(static_cast<IO*>(base) + at) = p;
}
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The backward pass works on pairs, one fma.f32x2 for two columns: at 24 scalar
// instructions an element it was issue-bound short of HBM.  Odd columns alone.
__device__ __forceinline__ unsigned long long u64(float2 a) {
  return *reinterpret_cast<unsigned long long*>(&a);
}
__device__ __forceinline__ float2 f2(unsigned long long a) { return *reinterpret_cast<float2*>(&a); }
__device__ __forceinline__ float2 fma_(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(u64(a)), "l"(u64(b)), "l"(u64(c)));
  return f2(d);
}
__device__ __forceinline__ float2 add_(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(u64(a)), "l"(u64(b)));
  return f2(d);
}
__device__ __forceinline__ float2 mul_(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(u64(a)), "l"(u64(b)));
  return f2(d);
}
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float add_(float a, float b) { return a + b; }
__device__ __forceinline__ float mul_(float a, float b) { return a * b; }
template <typename V>
__device__ __forceinline__ V both(float a);
template <>
__device__ __forceinline__ float both<float>(float a) { return a; }
template <>
__device__ __forceinline__ float2 both<float2>(float a) { return make_float2(a, a); }
__device__ __forceinline__ float sum_of(float a) { return a; }
__device__ __forceinline__ float sum_of(float2 a) { return a.x + a.y; }
template <int VEC>
struct Pairs {
  using V = float2;
  static constexpr int kN = VEC / 2;
};
template <>
struct Pairs<1> {
  using V = float;
  static constexpr int kN = 1;
};
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

// The rows of one group of LPR threads, a ring of S ahead.  Vectors of at least
// four bytes come through cp.async, smaller ones by plain loads.
template <typename IO, int VEC, int TB, int LPR, int NV, int S, int TENSORS>
struct RowRing {
  static constexpr int kBytes = sizeof(IO) * VEC;
  static constexpr bool kAsync = kBytes >= 4;
  static constexpr size_t kSmem = kAsync ? (size_t)S * TENSORS * NV * TB * kBytes : 0;
  using P = Pack<IO, VEC>;
  P* ring;
  const IO* src[TENSORS];
  int D, lane;
  __device__ __forceinline__ P* at(int stage, int t, int n) {
    return ring + ((size_t)(stage * TENSORS + t) * NV + n) * TB + threadIdx.x;
  }
  __device__ __forceinline__ void fetch(int stage, long long row, bool in) {
    if (kAsync) {
      if (in) {
#pragma unroll
        for (int t = 0; t < TENSORS; ++t)
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            const int i = (n * LPR + lane) * VEC;
            if (i < D) copy_async<kBytes >= 16 ? 16 : 4>(at(stage, t, n), src[t] + row * D + i);
          }
      }
      copy_commit();
    }
  }
  __device__ __forceinline__ void read(int stage, long long row, int t, int n, float (&f)[VEC]) {
    const int i = (n * LPR + lane) * VEC;
    unpack<IO, VEC>(kAsync ? *at(stage, t, n) : *reinterpret_cast<const P*>(src[t] + row * D + i), f);
  }
};

// Sum over the row's threads, the same in each.  A block's sum alternates
// between two buffers, so that one barrier a sum is enough.
template <int TB, int LPR>
__device__ __forceinline__ float row_sum(float s, float* red, int& turn) {
  if (LPR <= 32) return lane_sum<LPR>(s);
  s = lane_sum<32>(s);
  float* r = red + (turn ^= 1) * (TB / 32);
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = s;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < TB / 32; ++i) t += r[i];
  return t;
}

// ------------------------------------------------------------------ forward
template <typename IO, typename W, int VEC, int TB, int LPR, int NV, int S>
__global__ void __launch_bounds__(TB) norm_fwd_kernel(NormArgs a) {
  constexpr int kGroups = TB / LPR;
  extern __shared__ __align__(16) char sm[];
  __shared__ float red[2 * TB / 32];
  using Ring = RowRing<IO, VEC, TB, LPR, NV, S, 1>;
  Ring ring;
  ring.ring = reinterpret_cast<typename Ring::P*>(sm);
  ring.src[0] = static_cast<const IO*>(a.x);
  ring.D = a.D;
  const int lane = ring.lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = (n * LPR + lane) * VEC + e;
      w[n][e] = i < a.D ? weight_at<W>(a.w, i, 1.f) : 0.f;
      b[n][e] = i < a.D ? weight_at<W>(a.b, i, 0.f) : 0.f;
    }
  const long long stride = (long long)gridDim.x * kGroups;
  long long r0 = (long long)blockIdx.x * kGroups;  // (the same in a block: barriers)
#pragma unroll
  for (int s = 0; s < S - 1; ++s) ring.fetch(s, r0 + s * stride + grp, r0 + s * stride + grp < a.rows);
  for (int stage = 0; r0 < a.rows; r0 += stride, stage = stage + 1 == S ? 0 : stage + 1) {
    const long long r = r0 + grp, ahead = r + (S - 1) * stride;
    const bool in = r < a.rows;
    ring.fetch(stage == 0 ? S - 1 : stage - 1, ahead, ahead < a.rows);
    if (Ring::kAsync) copy_wait<S - 1>();
    float x[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if (in && (n * LPR + lane) * VEC < a.D)
        ring.read(stage, r, 0, n, x[n]);
      else
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[n][e] = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += x[n][e];
    }
    const float mean = row_sum<TB, LPR>(s, red, turn) * inv_d;
    float s2 = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if ((n * LPR + lane) * VEC < a.D)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x[n][e] -= mean;
          s2 = fmaf(x[n][e], x[n][e], s2);
        }
    const float rstd = 1.f / sqrtf(row_sum<TB, LPR>(s2, red, turn) * inv_d + a.eps);
    if (in) {
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int i = (n * LPR + lane) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[n][e] = fmaf(x[n][e] * rstd, w[n][e], b[n][e]);
        if (i < a.D) store_vec<IO, VEC>(a.y, r * a.D + i, x[n]);
      }
      if (lane == 0) {
        a.mean[r] = mean;
        a.rstd[r] = rstd;
      }
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
template <typename IO, typename W, int VEC, int TB, int LPR, int NV, int S>
__global__ void __launch_bounds__(TB) norm_bwd_kernel(NormArgs a) {
  after_previous();
  let_next_start();
  constexpr int kGroups = TB / LPR;
  extern __shared__ __align__(16) char sm[];
  __shared__ float red[4 * TB / 32];
  using Ring = RowRing<IO, VEC, TB, LPR, NV, S, 2>;
  Ring ring;
  ring.ring = reinterpret_cast<typename Ring::P*>(sm);
  ring.src[0] = static_cast<const IO*>(a.x);
  ring.src[1] = static_cast<const IO*>(a.dy);
  ring.D = a.D;
  const int lane = ring.lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  using V = typename Pairs<VEC>::V;
  constexpr int kN = Pairs<VEC>::kN;
  V w[NV][kN], dw[NV][kN], db[NV][kN];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = (n * LPR + lane) * VEC + e;
      f[e] = i < a.D ? weight_at<W>(a.w, i, 1.f) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      w[n][e] = reinterpret_cast<const V*>(f)[e];
      dw[n][e] = db[n][e] = both<V>(0.f);
    }
  }
  const long long stride = (long long)gridDim.x * kGroups;
  long long r0 = (long long)blockIdx.x * kGroups;
#pragma unroll
  for (int s = 0; s < S - 1; ++s) ring.fetch(s, r0 + s * stride + grp, r0 + s * stride + grp < a.rows);
  // (a row's own two numbers, one row ahead: a load at their use would add its
  // latency to every row)
  float mean_next = r0 + grp < a.rows ? a.mean[r0 + grp] : 0.f;
  float rstd_next = r0 + grp < a.rows ? a.rstd[r0 + grp] : 0.f;
  for (int stage = 0; r0 < a.rows; r0 += stride, stage = stage + 1 == S ? 0 : stage + 1) {
    const long long r = r0 + grp, ahead = r + (S - 1) * stride;
    const bool in = r < a.rows;
    ring.fetch(stage == 0 ? S - 1 : stage - 1, ahead, ahead < a.rows);
    const float mean = mean_next, rstd = rstd_next;
    if (r + stride < a.rows) {
      mean_next = a.mean[r + stride];
      rstd_next = a.rstd[r + stride];
    }
    if (Ring::kAsync) copy_wait<S - 1>();
    V xh[NV][kN], t[NV][kN];
    V p1 = both<V>(0.f), p2 = both<V>(0.f);
    const V minus_mean = both<V>(-mean), scale = both<V>(rstd);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if (in && (n * LPR + lane) * VEC < a.D) {
        float x[VEC], g[VEC];
        ring.read(stage, r, 0, n, x);
        ring.read(stage, r, 1, n, g);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const V gv = reinterpret_cast<const V*>(g)[e];
          xh[n][e] = mul_(add_(reinterpret_cast<const V*>(x)[e], minus_mean), scale);
          dw[n][e] = fma_(gv, xh[n][e], dw[n][e]);
          db[n][e] = add_(db[n][e], gv);
          t[n][e] = mul_(gv, w[n][e]);
          p1 = add_(p1, t[n][e]);
          p2 = fma_(t[n][e], xh[n][e], p2);
        }
      }
    }
    float s1 = sum_of(p1), s2 = sum_of(p2);
    float m1, m2;
    if (LPR <= 32) {
      m1 = lane_sum<LPR <= 32 ? LPR : 32>(s1) * inv_d;
      m2 = lane_sum<LPR <= 32 ? LPR : 32>(s2) * inv_d;
    } else {  // both sums through one barrier
      s1 = lane_sum<32>(s1);
      s2 = lane_sum<32>(s2);
      float* q = red + (turn ^= 1) * (2 * TB / 32);
      if ((threadIdx.x & 31) == 0) {
        q[threadIdx.x >> 5] = s1;
        q[TB / 32 + (threadIdx.x >> 5)] = s2;
      }
      __syncthreads();
      m1 = m2 = 0.f;
#pragma unroll
      for (int i = 0; i < TB / 32; ++i) {
        m1 += q[i];
        m2 += q[TB / 32 + i];
      }
      m1 *= inv_d;
      m2 *= inv_d;
    }
    const V minus_m1 = both<V>(-m1), minus_m2 = both<V>(-m2);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = (n * LPR + lane) * VEC;
      if (in && i < a.D) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < kN; ++e)
          reinterpret_cast<V*>(o)[e] =
              mul_(fma_(xh[n][e], minus_m2, add_(t[n][e], minus_m1)), scale);
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
        if (i >= a.D) continue;
        a.part[(size_t)blockIdx.x * a.D + i] = reinterpret_cast<const float*>(dw[n])[e];
        a.part[((size_t)a.parts + blockIdx.x) * a.D + i] = reinterpret_cast<const float*>(db[n])[e];
      }
    return;
  }
  // the block's groups, through shared memory ([kGroups][D]), in order
  float* part_s = reinterpret_cast<float*>(sm);
  if (Ring::kAsync) copy_wait<0>();
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int i = (n * LPR + lane) * VEC + e;
        if (i < a.D) part_s[grp * a.D + i] = reinterpret_cast<const float*>(which ? db[n] : dw[n])[e];
      }
    __syncthreads();
    float* out = a.part + ((size_t)which * a.parts + blockIdx.x) * a.D;
    for (int i = threadIdx.x; i < a.D; i += TB) {
      float s = 0.f;
#pragma unroll 8
      for (int g = 0; g < kGroups; ++g) s += part_s[g * a.D + i];
      out[i] = s;
    }
  }
}

// Rows wider than a block's registers: the block keeps its partial sums of dw
// and db in its row of the workspace.
template <typename IO, typename W>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(NormArgs a) {
  after_previous();
  let_next_start();
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

// dw and db from the partial rows: 32 columns to a block, 32 threads a column
// over the partial rows, joined in a fixed order.
template <typename W>
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(NormArgs a) {
  after_previous();
  let_next_start();
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + c;
  const float* p = a.part + (size_t)blockIdx.y * a.parts * a.D;
  float t = 0.f;
  if (i < a.D)
#pragma unroll 8
    for (int r = g; r < a.parts; r += 32) t += p[(size_t)r * a.D + i];
  s[g][c] = t;
  __syncthreads();
  if (g == 0 && i < a.D) {
#pragma unroll
    for (int k = 1; k < 32; ++k) t += s[k][c];
    st_io(static_cast<W*>(blockIdx.y ? a.db : a.dw) + i, t);
  }
}

// ----------------------------------------------------------------- dispatch
// Vectors of 16 bytes where the width and every row-indexed pointer allow it,
// single elements otherwise (16,384 rows of 4096, backward: 84 us and 355 us).
inline bool vector_ok(int D, int vec, const void* p0, const void* p1, const void* p2) {
  const uintptr_t m = reinterpret_cast<uintptr_t>(p0) | reinterpret_cast<uintptr_t>(p1) |
                      reinterpret_cast<uintptr_t>(p2);
  return D % vec == 0 && (m & 15) == 0;
}
inline int blocks_for(long long units, int per_sm) {
  const long long most = (long long)kSms * per_sm;
  return (int)(units < most ? (units < 1 ? 1 : units) : most);
}
// Partial rows of the weight gradients, at most: a block each.
inline int weight_parts(long long rows, int D) { return blocks_for(rows, D <= 2048 ? 8 : 3); }

template <typename IO, typename W, int VEC, int TB, int LPR, int NV, int S>
cudaError_t run_fwd(const NormArgs& a, int per_sm, cudaStream_t s) {
  constexpr size_t smem = RowRing<IO, VEC, TB, LPR, NV, S, 1>::kSmem;
  const auto kernel = norm_fwd_kernel<IO, W, VEC, TB, LPR, NV, S>;
  if (smem > 40 * 1024) {  // (the static part counts towards the default 48 KB)
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  constexpr int kGroups = TB / LPR;
  kernel<<<blocks_for((a.rows + kGroups - 1) / kGroups, per_sm), TB, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename IO, typename W, int VEC, int TB, int LPR, int NV, int S>
cudaError_t run_bwd(NormArgs& a, int per_sm, cudaStream_t s) {
  constexpr size_t ring = RowRing<IO, VEC, TB, LPR, NV, S, 2>::kSmem;
  constexpr size_t join = LPR <= 32 ? (size_t)TB * VEC * NV * sizeof(float) : 0;
  constexpr size_t smem = ring > join ? ring : join;
  const auto kernel = norm_bwd_kernel<IO, W, VEC, TB, LPR, NV, S>;
  if (smem > 40 * 1024) {  // (the static part counts towards the default 48 KB)
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int parts = blocks_for((a.rows + TB / LPR - 1) / (TB / LPR), per_sm);
  a.parts = parts < a.parts ? parts : a.parts;
  kernel<<<a.parts, TB, smem, s>>>(a);
  return cudaGetLastError();
}

// Threads of a row by its width: the fewest lanes that hold it in one or two vectors
// each, a warp at most (rows of 128 by 16 lanes 94 us, by 32 half of which idle 194 us);
// wider rows a block, of 128 threads first (rows of 768 to 2048 by 256 threads took
// 246 to 116 us for 2^27 elements, by 128 it is 124 to 89), and three vectors a thread
// before twice the threads (2560: 97 us and 115; 5120: 106 and 128; backward 2560: 150
// and 168, but 5120: 208 and 184).  The ring is as deep as keeps 40 KB or more of an
// SM in flight.
//
// Backward, blocks an SM: a row of 4096 takes 141 us with its two numbers loaded at
// their use, then 100 with three blocks, 97 with four and 84 with two, whose rows
// come to the memory in longer runs; a row by 512 threads takes 109.  Rows of 1024 by
// blocks of 128 threads: 392 us with two, 227 with four, 179 with six, 160 with eight.
// The widest rows in registers (8192 in fp32, 16384 in bf16): one block of 1024
// threads, 325 and 313 us; read again for each sum 634 and 627.
template <typename IO, typename W, int VEC>
cudaError_t fwd_vec(const NormArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 8 * VEC) return run_fwd<IO, W, VEC, 256, 8, 1, 4>(a, 8, s);
  if (D <= 16 * VEC) return run_fwd<IO, W, VEC, 256, 16, 1, 4>(a, 8, s);
  if (D <= 32 * VEC) return run_fwd<IO, W, VEC, 256, 32, 1, 4>(a, 8, s);
  if (D <= 64 * VEC) return run_fwd<IO, W, VEC, 256, 32, 2, 3>(a, 8, s);
  if (D <= 128 * VEC) return run_fwd<IO, W, VEC, 128, 128, 1, 4>(a, 16, s);
  if (D <= 256 * VEC) return run_fwd<IO, W, VEC, 128, 128, 2, 4>(a, 12, s);
  if (D <= 384 * VEC) return run_fwd<IO, W, VEC, 128, 128, 3, 3>(a, 8, s);
  if (D <= 512 * VEC) return run_fwd<IO, W, VEC, 256, 256, 2, 4>(a, 4, s);
  if (D <= 768 * VEC) return run_fwd<IO, W, VEC, 256, 256, 3, 3>(a, 4, s);
  if (D <= 1024 * VEC) return run_fwd<IO, W, VEC, 512, 512, 2, 4>(a, 4, s);
  if (D <= 2048 * VEC) return run_fwd<IO, W, VEC, 512, 512, 4, 2>(a, 4, s);
  norm_fwd_long_kernel<IO, W><<<blocks_for(a.rows, 2), 1024, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename IO, typename W, int VEC>
cudaError_t bwd_vec(NormArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 8 * VEC) return run_bwd<IO, W, VEC, 256, 8, 1, 4>(a, 4, s);
  if (D <= 16 * VEC) return run_bwd<IO, W, VEC, 256, 16, 1, 4>(a, 4, s);
  if (D <= 32 * VEC) return run_bwd<IO, W, VEC, 256, 32, 1, 4>(a, 4, s);
  if (D <= 64 * VEC) return run_bwd<IO, W, VEC, 256, 32, 2, 3>(a, 4, s);
  if (D <= 128 * VEC) return run_bwd<IO, W, VEC, 128, 128, 1, 4>(a, 8, s);
  if (D <= 256 * VEC) return run_bwd<IO, W, VEC, 128, 128, 2, 3>(a, 4, s);
  if (D <= 384 * VEC) return run_bwd<IO, W, VEC, 128, 128, 3, 3>(a, 3, s);
  if (D <= 512 * VEC) return run_bwd<IO, W, VEC, 256, 256, 2, 4>(a, 2, s);
  if (D <= 1024 * VEC) return run_bwd<IO, W, VEC, 512, 512, 2, 3>(a, 2, s);
  if constexpr (VEC > 1)
    if (D <= 2048 * VEC) return run_bwd<IO, W, VEC, 1024, 1024, 2, 2>(a, 1, s);
  // (single elements: odd widths, four a thread)
  if (VEC == 1 && D <= 2048) return run_bwd<IO, W, VEC, 512, 512, VEC == 1 ? 4 : 2, 3>(a, 2, s);
  a.parts = blocks_for(a.rows, 2);
  norm_bwd_long_kernel<IO, W><<<a.parts, 1024, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename IO, typename W>
cudaError_t launch_norm(NormArgs a, bool back, cudaStream_t s) {
  constexpr int kVec = 16 / sizeof(IO);
  const bool vec = vector_ok(a.D, kVec, a.x, a.y, back ? a.dy : a.x);
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    e = back ? (vec ? bwd_vec<IO, W, kVec>(a, s) : bwd_vec<IO, W, 1>(a, s))
             : (vec ? fwd_vec<IO, W, kVec>(a, s) : fwd_vec<IO, W, 1>(a, s));
    if (e != cudaSuccess) return e;
  }
  if (back && a.part) {
    if (a.rows == 0) a.parts = 0;  // the sums over no rows are zero
    e = launch_next(a.rows > 0, norm_weight_grad_kernel<W>, dim3((a.D + 31) / 32, 2), 1024, 0, s, a);
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
  // (columns are counted in 32 bits, up to a block's step past the row)
  if (rows > 0x7fffffffLL || width > 1 << 30) return CKDA_ERR_UNSUPPORTED;
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
