// ckda_linear_step.cu -- one token of linear attention on a resident fp32 state:
//     S = exp(g) S + k v^T,    o = S^T (scale q),    S updated in place.
//
// Every state element is read once, written once and takes two fmas, so HBM
// bandwidth is the bound (128 KiB moved per head at 128 x 128).  A block owns
// some columns of one (batch, head) state: LANES threads side by side hold VEC
// columns each (16-byte accesses where the width allows), and 256 / LANES row
// groups hold every such rows, all loaded before the token's vectors are
// waited for.  o is the sum over rows, joined through shared memory.
//
// Columns of a block: all 128 when there are enough (batch, head) pairs to
// fill the SMs, else 32, so that a single user's step spreads over four times
// the SMs (each warp still reads whole 128-byte lines).  256 x 32 pairs of 128 x 128:
// 160 us, 99% of the copy bandwidth, and 194 us with 32 columns; 16 pairs, from the
// call to its result: 22.6 us with 32 columns, 23.7 us with 128, most of it the host's.
// Widths that are not multiples of 4, and unaligned states, go by single columns: 256 x 32
// pairs of 128 x 127 in 304 us, 52% of the copy bandwidth.
// Narrower states take as many lanes as they have columns, and half the rows: 1024 x 32
// pairs of 64 x 64 in 175 us, 317 us in blocks for 128 x 128, half of them idle.
#include <type_traits>
#include "ckda_linear.cuh"

namespace ckda {
namespace {

constexpr int kThreads = 256;

struct StepArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  float* state;
  void* o;
  int H, Hk, dk, dv, g_head;
  float scale;
};

// DK: 64 or 128, at least dk.
template <typename IO, int VEC, int LANES, int DK>
__global__ void __launch_bounds__(kThreads) linear_step_kernel(StepArgs a) {
  constexpr int kGroups = kThreads / LANES;
  constexpr int kRows = (DK + kGroups - 1) / kGroups;
  __shared__ float sk[128], sq[128];
  __shared__ float red[kGroups][LANES * VEC];
  const size_t unit = blockIdx.x;
  const int h = unit % a.H;
  const size_t b = unit / a.H, hk = h / (a.H / a.Hk);
  const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const int c = (blockIdx.y * LANES + lane) * VEC;
  const bool in = c < a.dv;
  float* S = a.state + unit * a.dk * a.dv + c;

  struct alignas(4 * VEC) Vec { float f[VEC]; };
  Vec s[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int i = r * kGroups + grp;
    if (in && i < a.dk) s[r] = *reinterpret_cast<const Vec*>(S + (size_t)i * a.dv);
  }
  const IO* k = static_cast<const IO*>(a.k) + (b * a.Hk + hk) * a.dk;
  const IO* q = static_cast<const IO*>(a.q) + (b * a.Hk + hk) * a.dk;
  const IO* v = static_cast<const IO*>(a.v) + unit * a.dv;
  if (threadIdx.x < 128) {
    const bool have = (int)threadIdx.x < a.dk;
    sk[threadIdx.x] = have ? ld_io(k + threadIdx.x) : 0.f;
    sq[threadIdx.x] = have ? a.scale * ld_io(q + threadIdx.x) : 0.f;
  }
  float vv[VEC], acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    vv[e] = in ? ld_io(v + c + e) : 0.f;
    acc[e] = 0.f;
  }
  const float dec = expf(a.g[a.g_head ? (size_t)h : unit]);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int i = r * kGroups + grp;
    if (in && i < a.dk) {
      const float ki = sk[i], qi = sq[i];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        s[r].f[e] = fmaf(dec, s[r].f[e], ki * vv[e]);
        acc[e] = fmaf(s[r].f[e], qi, acc[e]);
      }
      *reinterpret_cast<Vec*>(S + (size_t)i * a.dv) = s[r];
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) red[grp][lane * VEC + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < LANES * VEC) {
    const int col = blockIdx.y * LANES * VEC + threadIdx.x;
    if (col < a.dv) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) t += red[i][threadIdx.x];
      st_io(static_cast<IO*>(a.o) + unit * a.dv + col, t);
    }
  }
}

template <typename IO>
cudaError_t launch_step(const StepArgs& a, int B, cudaStream_t s) {
  const unsigned units = (unsigned)B * a.H;
  const bool vec = a.dv % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
  const auto step = [&](auto dk) {
    constexpr int DK = decltype(dk)::value;
    const bool many = units >= 2 * kLinSms;
    const dim3 by32(units, (a.dv + 31) / 32);
    if (!vec)
      linear_step_kernel<IO, 1, 32, DK><<<by32, kThreads, 0, s>>>(a);
    else if (many && a.dv > 64)
      linear_step_kernel<IO, 4, 32, DK><<<units, kThreads, 0, s>>>(a);
    else if (many && a.dv > 32)
      linear_step_kernel<IO, 4, 16, DK><<<units, kThreads, 0, s>>>(a);
    else
      linear_step_kernel<IO, 4, 8, DK><<<by32, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  };
  return a.dk <= 64 ? step(std::integral_constant<int, 64>()) : step(std::integral_constant<int, 128>());
}

}  // namespace
}  // namespace ckda

using namespace ckda;

extern "C" ckda_status ckda_linear_decode_step(const void* q, const void* k, const void* v,
                                               const float* g, int g_per_head, float* state,
                                               void* o, int B, int H, int Hk, int dk, int dv,
                                               ckda_dtype io_dtype, float scale, void* stream) {
  if (io_dtype != CKDA_F32 && io_dtype != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || Hk < 1 || H % Hk != 0 || dk < 1 || dv < 1) return CKDA_ERR_INVALID_ARG;
  if (!q || !k || !v || !g || !state || !o) return CKDA_ERR_INVALID_ARG;
  if (!(scale == scale)) return CKDA_ERR_INVALID_ARG;
  if (dk > 128 || dv > 128) return CKDA_ERR_UNSUPPORTED;
  if ((long long)B * H > 0x7fffffffLL) return CKDA_ERR_UNSUPPORTED;
  StepArgs a{q, k, v, g, state, o, H, Hk, dk, dv, g_per_head ? 1 : 0, scale};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = io_dtype == CKDA_F32 ? launch_step<float>(a, B, s)
                                             : launch_step<__nv_bfloat16>(a, B, s);
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}
