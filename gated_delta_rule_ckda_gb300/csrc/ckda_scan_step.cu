// ckda_scan_step.cu -- one token of the selective scan on a resident fp32 state:
//     delta = softplus(dt + dt_bias),   h = exp(delta A) h + delta x B   (in place),
//     y = (sum_n C[n] h[n] + D x) silu(z)
//
// Each state is read and written once for one exponential and three more instructions: HBM
// bandwidth is the bound.  LP lanes share a channel, four states (16 bytes) each.  A thread
// takes its channel of four rows of the batch: their states are loaded before any is waited
// for, A and B's unpacking serve all four, and a channel's lanes share the rows' step sizes
// and outputs (one row a lane, handed round by shuffles) instead of each forming all.
#include "ckda_scan.cuh"

namespace ckda {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;

// VEC: N a multiple of 4, states and rates 16-byte aligned, B and C in whole vectors.
template <typename IO, int LP, bool VEC>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanArgs a) {
  constexpr int kApart = kThreads / LP, kOwn = LP < kRows ? kRows / LP : 1;
  const int l = threadIdx.x % LP, n0 = 4 * l;
  const int b0 = (int)(blockIdx.x / a.chan_blocks) * kRows;
  const int chan = (int)(blockIdx.x % a.chan_blocks) * kApart + threadIdx.x / LP;
  const bool in = chan < a.D;
  const int c = in ? chan : 0;
  const bool have = in && n0 < a.N;
  const int rows = a.rows - b0 < kRows ? a.rows - b0 : kRows;
  float* const state = a.hT + (long long)b0 * a.D * a.N;
  const long long row = (long long)a.D * a.N, at = (long long)c * a.N + n0;
  float2 h[kRows][2];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (r >= rows) break;
    if (VEC) {
      if (have) {
        const float4 v = *reinterpret_cast<const float4*>(state + r * row + at);
        h[r][0] = make_float2(v.x, v.y);
        h[r][1] = make_float2(v.z, v.w);
      }
    } else {
      load_states<4>(h[r], state + r * row, c, a.N, n0, in);
    }
  }
  // the rows of this lane: steps, and what finishes the output
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
  float delta[kOwn], u[kOwn], x[kOwn], z[kOwn];
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    const int r = LP < kRows ? l * kOwn + j : l % kRows;
    const long long b = b0 + (r < rows ? r : 0);
    x[j] = ld_io(static_cast<const IO*>(a.x) + b * a.ldx + c);
    const float raw = ld_io(static_cast<const IO*>(a.dt) + b * a.lddt + c) + bias;
    z[j] = a.z ? ld_io(static_cast<const IO*>(a.z) + b * a.ldz + c) : 0.f;
    delta[j] = a.softplus ? softplus(raw) : raw;
    u[j] = delta[j] * x[j];
  }
  float2 A2[2];
  if (VEC) {
    const float4 v = have ? *reinterpret_cast<const float4*>(a.A + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    A2[0] = make_float2(v.x, v.y);
    A2[1] = make_float2(v.z, v.w);
  } else {
    load_states<4>(A2, a.A, c, a.N, n0, in);
  }
  A2[0] = mul_(A2[0], both<float2>(kLog2e));
  A2[1] = mul_(A2[1], both<float2>(kLog2e));
  const long long group = (long long)(c / (a.D / a.G)) * a.N + n0;
  float y[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int from = LP < kRows ? r / kOwn : r;
    const float d = __shfl_sync(0xffffffffu, delta[LP < kRows ? r % kOwn : 0], from, LP);
    const float v = __shfl_sync(0xffffffffu, u[LP < kRows ? r % kOwn : 0], from, LP);
    y[r] = 0.f;
    if (r >= rows || !have) continue;
    float f[4], g[4];
    const IO* pB = static_cast<const IO*>(a.B) + (b0 + r) * a.ldb + group;
    const IO* pC = static_cast<const IO*>(a.C) + (b0 + r) * a.ldc + group;
    if (VEC) {
      unpack<IO, 4>(*reinterpret_cast<const Pack<IO, 4>*>(pB), f);
      unpack<IO, 4>(*reinterpret_cast<const Pack<IO, 4>*>(pC), g);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = n0 + e < a.N ? ld_io(pB + e) : 0.f;
        g[e] = n0 + e < a.N ? ld_io(pC + e) : 0.f;
      }
    }
    float2 s = both<float2>(0.f);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float2 decay = decay_of(both<float2>(d), A2[q]);
      h[r][q] = fma_(decay, h[r][q], mul_(both<float2>(v), make_float2(f[2 * q], f[2 * q + 1])));
      s = fma_(make_float2(g[2 * q], g[2 * q + 1]), h[r][q], s);
    }
    y[r] = s.x + s.y;
    if (VEC)
      *reinterpret_cast<float4*>(state + r * row + at) =
          make_float4(h[r][0].x, h[r][0].y, h[r][1].x, h[r][1].y);
    else
      store_states<4>(state + r * row, c, a.N, n0, true, h[r]);
  }
  fold_values<kRows, LP, 1>(y, l);
  const float skip = a.skip ? a.skip[c] : 0.f;
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    const int r = LP < kRows ? l * kOwn + j : l;
    if (r >= rows || !in) continue;
    float o = fmaf(skip, x[j], y[j]);
    if (a.z) o *= scan_silu(z[j]);
    st_io(static_cast<IO*>(a.y) + (long long)(b0 + r) * a.D + c, o);
  }
}

template <typename IO, int LP, bool VEC>
cudaError_t run(ScanArgs a, cudaStream_t s) {
  constexpr int kPer = kThreads / LP;
  a.chan_blocks = (a.D + kPer - 1) / kPer;
  const long long blocks = (long long)((a.rows + kRows - 1) / kRows) * a.chan_blocks;
  scan_step_kernel<IO, LP, VEC><<<(unsigned)blocks, kThreads, 0, s>>>(a);
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
  const size_t pack = 4 * (io_dtype == CKDA_F32 ? 4 : 2);  // bytes of four states of B and C
  const bool vec = N % 4 == 0 && ldb % 4 == 0 && ldc % 4 == 0 &&
                   ((reinterpret_cast<uintptr_t>(state) | reinterpret_cast<uintptr_t>(A)) & 15) == 0 &&
                   ((reinterpret_cast<uintptr_t>(Bm) | reinterpret_cast<uintptr_t>(C)) & (pack - 1)) == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      io_dtype == CKDA_F32 ? (vec ? by_states<float, true>(a, s) : by_states<float, false>(a, s))
                           : (vec ? by_states<__nv_bfloat16, true>(a, s) : by_states<__nv_bfloat16, false>(a, s));
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}
