// ckda_rows.cuh -- what the kernels over rows and channels share: vectors in the I/O type,
// pairs of columns in one fp32 instruction, sums over a row's threads, and the ring of
// rows ahead that keeps loads in flight.
#pragma once
#include "ckda_internal.cuh"

namespace ckda {

constexpr int kSms = 152;
// Blocks for so many units of work: each one's, or what runs at once.
inline int blocks_for(long long units, int per_sm) {
  const long long most = (long long)kSms * per_sm;
  return (int)(units < most ? (units < 1 ? 1 : units) : most);
}

// Whether [p, p + n) and [q, q + m) share memory.
inline bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && n > 0 && m > 0 && a < b + m && b < a + n;
}
// From the first of so many rows of D, ld apart, to behind the last.
inline size_t rows_bytes(long long rows, long long D, long long ld, size_t io) {
  return rows > 0 ? (size_t)((rows - 1) * ld + D) * io : 0;
}
// Whether an output of dense rows shares memory with an input of rows ld apart, other than
// element for element: what writes one part may run beside what still reads another.
inline bool clash(const void* out, const void* in, long long rows, long long D, long long ld, size_t io) {
  return !(out == in && (ld == D || rows == 1)) &&
         overlap(out, rows_bytes(rows, D, D, io), in, rows_bytes(rows, D, ld, io));
}

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
  else if (BYTES == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Pairs of columns, one fma.f32x2 for two; odd columns alone.  (Layer norm's backward
// pass, at 24 scalar instructions an element, was issue-bound short of HBM.)
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
// A sum that carries along what its additions round off (Kahan's), so that its error does
// not grow with the number of terms.  A term that is not finite makes it what a plain sum is.
struct CarriedSum {
  float sum = 0.f, lost = 0.f;
  __device__ __forceinline__ void add(float v) {
    v -= lost;
    const float next = sum + v, off = (next - sum) - v;
    lost = off - off == 0.f ? off : 0.f;
    sum = next;
  }
};
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

}  // namespace ckda
