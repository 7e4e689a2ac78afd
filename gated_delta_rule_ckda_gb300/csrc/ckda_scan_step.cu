// ckda_scan_step.cu -- one token of the selective scan on a resident fp32 state:
//     delta = softplus(dt + dt_bias),   h = exp(delta A) h + delta x B   (in place),
//     y = (sum_n C[n] h[n] + D x) silu(z)
//
// Each state is read and written once for one exponential and three more instructions: HBM
// bandwidth is the bound.  LP lanes share a channel, four states (16 bytes) each; a thread
// loads the states of kChans channels before it waits for any of them.
#include "ckda_scan.cuh"

namespace ckda {
namespace {

constexpr int kThreads = 256;
constexpr int kChans = 4;

// VEC: N a multiple of 4, 16-byte aligned states and rates.
template <typename IO, int LP, bool VEC>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanArgs a) {
  constexpr int kApart = kThreads / LP;
  const int l = threadIdx.x % LP, n0 = 4 * l;
  const long long b = blockIdx.x / a.chan_blocks;
  const int c0 = (int)(blockIdx.x % a.chan_blocks) * kApart * kChans + threadIdx.x / LP;
  float* state = a.hT + b * a.D * a.N;
  float2 h[kChans][2];
#pragma unroll
  for (int j = 0; j < kChans; ++j) {
    const int c = c0 + j * kApart;
    if (VEC) {
      if (c < a.D && n0 < a.N) {
        const float4 v = *reinterpret_cast<const float4*>(state + (long long)c * a.N + n0);
        h[j][0] = make_float2(v.x, v.y);
        h[j][1] = make_float2(v.z, v.w);
      }
    } else {
      load_states<4>(h[j], state, c < a.D ? c : 0, a.N, n0, c < a.D);
    }
  }
  const int dg = a.D / a.G;
#pragma unroll
  for (int j = 0; j < kChans; ++j) {
    const int c = c0 + j * kApart;
    const bool in = c < a.D;
    const int cc = in ? c : 0;
    float2 A[2], B[2], C[2];
    const long long at = (long long)(cc / dg) * a.N;
    if (VEC) {
      const float4 v = in && n0 < a.N ? *reinterpret_cast<const float4*>(a.A + (long long)cc * a.N + n0)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
      A[0] = make_float2(v.x, v.y);
      A[1] = make_float2(v.z, v.w);
    } else {
      load_states<4>(A, a.A, cc, a.N, n0, in);
    }
    float f[4], g[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool have = in && n0 + e < a.N;
      f[e] = have ? ld_io(static_cast<const IO*>(a.B) + b * a.ldb + at + n0 + e) : 0.f;
      g[e] = have ? ld_io(static_cast<const IO*>(a.C) + b * a.ldc + at + n0 + e) : 0.f;
    }
    B[0] = make_float2(f[0], f[1]);
    B[1] = make_float2(f[2], f[3]);
    C[0] = make_float2(g[0], g[1]);
    C[1] = make_float2(g[2], g[3]);
    const float x = ld_io(static_cast<const IO*>(a.x) + b * a.ldx + cc);
    const float raw = ld_io(static_cast<const IO*>(a.dt) + b * a.lddt + cc) + (a.dt_bias ? a.dt_bias[cc] : 0.f);
    const float delta = a.softplus ? softplus(raw) : raw;
    float2 y = both<float2>(0.f);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float2 decay = ex2(mul_(both<float2>(delta), mul_(A[q], both<float2>(kLog2e))));
      h[j][q] = fma_(decay, h[j][q], mul_(both<float2>(delta * x), B[q]));
      y = fma_(C[q], h[j][q], y);
    }
    if (VEC) {
      if (in && n0 < a.N)
        *reinterpret_cast<float4*>(state + (long long)cc * a.N + n0) =
            make_float4(h[j][0].x, h[j][0].y, h[j][1].x, h[j][1].y);
    } else {
      store_states<4>(state, cc, a.N, n0, in, h[j]);
    }
    // (lanes past N hold what they did not load: not summed)
    float s = n0 < a.N && in ? y.x + y.y : 0.f;
#pragma unroll
    for (int m = LP / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (l == 0 && in) {
      s = fmaf(a.skip ? a.skip[cc] : 0.f, x, s);
      if (a.z) s *= scan_silu(ld_io(static_cast<const IO*>(a.z) + b * a.ldz + cc));
      st_io(static_cast<IO*>(a.y) + b * a.D + cc, s);
    }
  }
}

template <typename IO, int LP, bool VEC>
cudaError_t run(ScanArgs a, cudaStream_t s) {
  constexpr int kPer = kThreads / LP * kChans;
  a.chan_blocks = (a.D + kPer - 1) / kPer;
  scan_step_kernel<IO, LP, VEC><<<(unsigned)((long long)a.rows * a.chan_blocks), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename IO, bool VEC>
cudaError_t by_states(const ScanArgs& a, cudaStream_t s) {
  if (a.N <= 4) return run<IO, 1, VEC>(a, s);
  if (a.N <= 8) return run<IO, 2, VEC>(a, s);
  if (a.N <= 16) return run<IO, 4, VEC>(a, s);
  if (a.N <= 32) return run<IO, 8, VEC>(a, s);
  return run<IO, 16, VEC>(a, s);
}

}  // namespace
}  // namespace ckda

using namespace ckda;

extern "C" ckda_status ckda_scan_decode_step(const void* x, const void* dt, const float* A,
                                             const void* Bm, const void* C, const float* D_skip,
                                             const void* z, const float* dt_bias, float* state,
                                             void* y, int B, int D, int N, int G, long long ldx,
                                             long long lddt, long long ldb, long long ldc,
                                             long long ldz, ckda_dtype io_dtype, int softplus,
                                             void* stream) {
  const ckda_status st = check_scan(B, 1, D, N, G, nullptr, 0, io_dtype);
  if (st != CKDA_OK) return st;
  if (!x || !dt || !A || !Bm || !C || !state || !y) return CKDA_ERR_INVALID_ARG;
  if (ldx < D || lddt < D || (z && ldz < D) || ldb < (long long)G * N || ldc < (long long)G * N)
    return CKDA_ERR_INVALID_ARG;
  ScanArgs a{};
  a.x = x; a.dt = dt; a.B = Bm; a.C = C; a.z = z; a.A = A; a.skip = D_skip; a.dt_bias = dt_bias;
  a.hT = state; a.y = y;
  a.ldx = ldx; a.lddt = lddt; a.ldb = ldb; a.ldc = ldc; a.ldz = ldz;
  a.rows = B; a.T = 1; a.D = D; a.N = N; a.G = G; a.seqs = B; a.softplus = softplus != 0;
  const bool vec = N % 4 == 0 && ((reinterpret_cast<uintptr_t>(state) | reinterpret_cast<uintptr_t>(A)) & 15) == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      io_dtype == CKDA_F32 ? (vec ? by_states<float, true>(a, s) : by_states<float, false>(a, s))
                           : (vec ? by_states<__nv_bfloat16, true>(a, s) : by_states<__nv_bfloat16, false>(a, s));
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}
