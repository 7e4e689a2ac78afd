// ckda_scan_step.cu -- one token of the selective scan on a resident fp32 state:
//     delta = softplus(dt + dt_bias),   h = exp(delta A) h + delta x B   (in place),
//     y = (sum_n C[n] h[n] + D x) silu(z)
//
// Each state is read and written once for one exponential and three more instructions: HBM
// bandwidth is the bound.  LP lanes share a channel, four states (16 bytes) each.  A block
// walks the batch four rows at a time, the states of the next four rows on their way
// through a ring in shared memory (a thread copies what it reads itself); A and its
// products serve all rows, and a channel's lanes share the rows' step sizes and outputs
// (one row a lane, handed round by shuffles) instead of each forming all.
//
// 256 rows of 4096 channels of 16 states: 31 to 33 us, 65 to 69% of the copy bandwidth (each lane its
// own steps and one row after another, 140 instructions a state: 57; four rows held in
// registers 37; eight blocks an SM, with five 37).
#include "ckda_scan.cuh"

namespace ckda {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 4, kStages = 2;
constexpr int kPerSm = 8;

// VEC: N a multiple of 4, states and rates 16-byte aligned, B and C in whole vectors.
template <typename IO, int LP, bool VEC>
__global__ void __launch_bounds__(kThreads, kPerSm) scan_step_kernel(ScanArgs a, int groups) {
  constexpr int kApart = kThreads / LP, kOwn = LP < kRows ? kRows / LP : 1;
  __shared__ float4 ring[VEC ? kStages : 1][kRows][kThreads];
  const int l = threadIdx.x % LP, n0 = 4 * l;
  const int first = (int)(blockIdx.x / a.chan_blocks) * groups * kRows;  // of the block's rows
  const int chan = (int)(blockIdx.x % a.chan_blocks) * kApart + threadIdx.x / LP;
  const bool in = chan < a.D;
  const int c = in ? chan : 0;
  const bool have = in && n0 < a.N;
  const int end = first + groups * kRows < a.rows ? first + groups * kRows : a.rows;
  const long long row = (long long)a.D * a.N;
  float* const state = a.hT + (long long)c * a.N + n0;
  const auto fetch = [&](int b0, int stage) {
    if (VEC) {
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (b0 + r < end && have) copy_async<16>(&ring[VEC ? stage : 0][r][threadIdx.x], state + (b0 + r) * row);
      copy_commit();
    }
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(first + s * kRows, s);
  float2 A2[2];
  load_states<4>(A2, a.A, c, a.N, n0, in);
  A2[0] = mul_(A2[0], both<float2>(kLog2e));
  A2[1] = mul_(A2[1], both<float2>(kLog2e));
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.skip ? a.skip[c] : 0.f;
  const long long group = (long long)(c / (a.D / a.G)) * a.N + n0;
  int stage = 0;
  for (int b0 = first; b0 < end; b0 += kRows, stage = stage + 1 == kStages ? 0 : stage + 1) {
    const int rows = end - b0 < kRows ? end - b0 : kRows;
    // B and C of every row, as they are
    Pack<IO, 4> rowB[kRows], rowC[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r >= rows || !have) break;
      const IO* pB = static_cast<const IO*>(a.B) + (b0 + r) * a.ldb + group;
      const IO* pC = static_cast<const IO*>(a.C) + (b0 + r) * a.ldc + group;
      if (VEC) {
        rowB[r] = *reinterpret_cast<const Pack<IO, 4>*>(pB);
        rowC[r] = *reinterpret_cast<const Pack<IO, 4>*>(pC);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n0 + e < a.N) {
            rowB[r].v[e] = pB[e];
            rowC[r].v[e] = pC[e];
          }
      }
    }
    // the rows of this lane: steps, and what finishes the output
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
    fetch(b0 + (kStages - 1) * kRows, stage == 0 ? kStages - 1 : stage - 1);
    if (VEC) copy_wait<kStages - 1>();
    float y[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int from = LP < kRows ? r / kOwn : r;
      const float d = __shfl_sync(0xffffffffu, delta[LP < kRows ? r % kOwn : 0], from, LP);
      const float v = __shfl_sync(0xffffffffu, u[LP < kRows ? r % kOwn : 0], from, LP);
      y[r] = 0.f;
      if (r >= rows || !have) continue;
      float2 h[2];
      if (VEC) {
        const float4 w = ring[VEC ? stage : 0][r][threadIdx.x];
        h[0] = make_float2(w.x, w.y);
        h[1] = make_float2(w.z, w.w);
      } else {
        load_states<4>(h, state + (b0 + r) * row - n0, 0, a.N, n0, true);
      }
      float f[4], g[4];
      unpack<IO, 4>(rowB[r], f);
      unpack<IO, 4>(rowC[r], g);
      if (!VEC)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n0 + e >= a.N) f[e] = g[e] = 0.f;
      float2 s = both<float2>(0.f);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float2 decay = decay_of(both<float2>(d), A2[q]);
        h[q] = fma_(decay, h[q], mul_(both<float2>(v), make_float2(f[2 * q], f[2 * q + 1])));
        s = fma_(make_float2(g[2 * q], g[2 * q + 1]), h[q], s);
      }
      y[r] = s.x + s.y;
      if (VEC)
        *reinterpret_cast<float4*>(state + (b0 + r) * row) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
      else
        store_states<4>(state + (b0 + r) * row - n0, 0, a.N, n0, true, h);
    }
    fold_values<kRows, LP, 1>(y, l);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const int r = LP < kRows ? l * kOwn + j : l;
      if (r >= rows || !in) continue;
      float o = fmaf(skip, x[j], y[j]);
      if (a.z) o *= scan_silu(z[j]);
      st_io(static_cast<IO*>(a.y) + (long long)(b0 + r) * a.D + c, o);
    }
  }
}

template <typename IO, int LP, bool VEC>
cudaError_t run(ScanArgs a, cudaStream_t s) {
  constexpr int kPer = kThreads / LP;
  a.chan_blocks = (a.D + kPer - 1) / kPer;
  // as few rows to a block as leave all blocks running at once
  const long long room = (long long)kPerSm * kSms;
  const int all = (a.rows + kRows - 1) / kRows;
  long long wide = room / a.chan_blocks;
  if (wide < 1) wide = 1;
  const int groups = (int)((all + wide - 1) / wide);
  const long long blocks = (long long)((all + groups - 1) / groups) * a.chan_blocks;
  scan_step_kernel<IO, LP, VEC><<<(unsigned)blocks, kThreads, 0, s>>>(a, groups);
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
  if (B > 1 << 30) return CKDA_ERR_UNSUPPORTED;  // (rows are counted in 32 bits, some past the last)
  if (!x || !dt || !A || !Bm || !C || !state || !y) return CKDA_ERR_INVALID_ARG;
  if (ldx < D || lddt < D || (z && ldz < D) || ldb < (long long)G * N || ldc < (long long)G * N)
    return CKDA_ERR_INVALID_ARG;
  ScanArgs a{};
  a.x = x; a.dt = dt; a.B = Bm; a.C = C; a.z = z; a.A = A; a.skip = D_skip; a.dt_bias = dt_bias;
  a.hT = state; a.y = y;
  a.ldx = ldx; a.lddt = lddt; a.ldb = ldb; a.ldc = ldc; a.ldz = ldz;
  a.rows = B; a.T = 1; a.D = D; a.N = N; a.G = G; a.seqs = B; a.softplus = softplus != 0;
  const size_t io = io_dtype == CKDA_F32 ? 4 : 2;
  if (scan_clash(a, y, kChannels, io) || scan_clash(a, state, kStates, io) ||
      overlap(y, scan_bytes(a, kChannels, D, io), state, scan_bytes(a, kStates, 0, io)))
    return CKDA_ERR_INVALID_ARG;
  const size_t pack = 4 * io;  // bytes of four states of B and C
  const bool vec = N % 4 == 0 && ldb % 4 == 0 && ldc % 4 == 0 &&
                   ((reinterpret_cast<uintptr_t>(state) | reinterpret_cast<uintptr_t>(A)) & 15) == 0 &&
                   ((reinterpret_cast<uintptr_t>(Bm) | reinterpret_cast<uintptr_t>(C)) & (pack - 1)) == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      io_dtype == CKDA_F32 ? (vec ? by_states<float, true>(a, s) : by_states<float, false>(a, s))
                           : (vec ? by_states<__nv_bfloat16, true>(a, s) : by_states<__nv_bfloat16, false>(a, s));
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}
