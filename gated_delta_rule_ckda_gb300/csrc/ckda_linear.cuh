// ckda_linear.cuh -- declarations shared by the translation units of linear
// attention with a scalar decay per head:
//     H_t = exp(g_t) H_{t-1} + k_t v_t^T,    o_t = H_t^T (scale q_t)
#pragma once
#include <atomic>
#include "ckda_internal.cuh"
#include "ckda_launch.cuh"

namespace ckda {

constexpr int kLinSms = 152;       // SMs of a GB300
constexpr float kLog2e = 1.4426950408889634f;
// A decay of exp2(-160) is zero in fp32 whatever it multiplies; log decays are
// clamped there so that g = -inf (a reset) leaves sums and differences finite.
constexpr float kMinLog2Decay = -160.f;

struct LinearArgs {
  const void* q;      // io   [B, Hk, T, dk]
  const void* k;      // io   [B, Hk, T, dk]
  const void* v;      // io   [B, H, T, dv]
  const float* g;     // fp32 [B, H, T], or [H] when g_head
  const float* h0;    // fp32 [N, H, dk, dv] or null
  void* o;            // io   [B, H, T, dv]
  float* hT;          // fp32 [N, H, dk, dv] or null
  const int32_t* cu_seqlens;
  const int32_t* order;
  int* status;
  int clear;          // the status word is still to be cleared, by the first kernel
  int N;              // sequences: B, or the packed ones
  int B, H, Hk, T, dk, dv;
  int g_head;
  float scale;
  ckda_dtype io;
  // backward
  const void* dout;   // io   [B, H, T, dv]
  const float* dhT;   // fp32 [N, H, dk, dv] or null
  void* dq;           // io   [B, Hk, T, dk]
  void* dkey;         // io   [B, Hk, T, dk]
  void* dval;         // io   [B, H, T, dv]
  float* dg;          // fp32 [B, H, T], or [H] when g_head
  float* dh0;         // fp32 [N, H, dk, dv] or null
};

// Tokens [t0, t0 + len) of sequence n on the T axis.  Offsets outside [0, T]
// are clamped, so that a bad cu_seqlens reads and writes nothing outside.
__device__ __forceinline__ void seq_range(const LinearArgs& a, int n, int& t0, int& len) {
  t0 = 0;
  len = a.T;
  if (a.cu_seqlens) {
    t0 = min(max(a.cu_seqlens[n], 0), a.T);
    len = max(min(a.cu_seqlens[n + 1], a.T) - t0, 0);
  }
}
__device__ __forceinline__ float log2_decay(float g) {
  // (a NaN stays one)
  const float x = g * kLog2e;
  return x < kMinLog2Decay ? kMinLog2Decay : x;
}

// Lets a kernel have `bytes` of shared memory on the current device; asked once for
// each kernel and device (a call of its own costs a microsecond of the host's part
// of a short prompt).  Calls from several threads at worst ask twice.
template <auto KERNEL>
cudaError_t allow_smem(size_t bytes) {  // the most that any launch of it takes
  static std::atomic<uint64_t> done{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Kernels on CUDA cores: every type and width up to 128.
size_t linear_serial_fwd_bytes(int N, int H, int T, int dk, int dv, bool packed);
cudaError_t linear_serial_fwd(const LinearArgs& a, char* ws, cudaStream_t s);
size_t linear_serial_bwd_bytes(int N, int B, int H, int Hk, int T, int dk, int dv, bool packed);
cudaError_t linear_serial_bwd(const LinearArgs& a, char* ws, cudaStream_t s);

// Shapes and pointers the chunked tensor-core kernels take: TMA wants 16-byte
// aligned rows and bases.
inline bool linear_chunk_path(ckda_dtype io, int dk, int dv) {
  return io == CKDA_BF16 && dk % 8 == 0 && dv % 8 == 0;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// Chunks of 128 tokens on the tensor cores.
size_t linear_chunk_fwd_bytes(int N, int B, int H, int T, int dk, int dv, bool packed);
cudaError_t linear_chunk_fwd(LinearArgs a, char* ws, cudaStream_t s);
size_t linear_chunk_bwd_bytes(int N, int B, int H, int Hk, int T, int dk, int dv, bool packed);
cudaError_t linear_chunk_bwd(const LinearArgs& a, char* ws, cudaStream_t s);

// dg of a decay per head: the sum of fp32 [B, H, T] over B and T.
cudaError_t linear_sum_decay(const LinearArgs& a, const float* dg_full, cudaStream_t s);

}  // namespace ckda
