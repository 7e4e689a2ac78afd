// ckda_scan_fwd.cu -- selective scan over prompts.  (The formulas and the block's work:
// ckda_scan.cuh.)
//
// What bounds it: N exponentials for every channel of every token, and about five more
// instructions a state, two states to an instruction; memory is read and written once.
//
// Rows with fewer channels than the card has room for are cut into pieces that run side by
// side: a first pass leaves each piece's own end state and the sum of its steps (a state
// decays over a piece by exp(A sum delta)), a scan over the pieces gives the states that
// enter them, and the second pass runs every piece from its own.
#include "ckda_scan.cuh"

namespace ckda {
namespace {

template <typename IO, typename S, bool VEC, bool ENDS>
struct Tile {  // a tile's inputs as a thread loads them
  Eight<IO> x, dt, z;
  GroupTile<IO, S> B, C;
  __device__ __forceinline__ void load(const ScanArgs& a, const ScanPlace& p, int t, int k, int v) {
    const int count = p.t1 - t;
    const long long at = (long long)p.row * a.T + t;
    if (k < count) {
      const int c = p.c0 + 8 * v, n = p.chans - 8 * v;
      x.template load<VEC>(a.x, (at + k) * a.ldx + c, n);
      dt.template load<VEC>(a.dt, (at + k) * a.lddt + c, n);
      if (!ENDS && a.z) z.template load<VEC>(a.z, (at + k) * a.ldz + c, n);
    }
    B.template load<VEC>(a.B, a.ldb, at, count, p.g, a.N);
    if (!ENDS) C.template load<VEC>(a.C, a.ldc, at, count, p.g, a.N);
  }
};

// ENDS: the first pass over pieces, what each leaves by itself.
template <typename IO, typename S, bool VEC, bool ENDS>
__global__ void __launch_bounds__(kScanBlock) scan_fwd_kernel(ScanArgs a) {
  constexpr int LP = S::kLanes, NS = S::kStates, P = S::kChans, K = S::K, NP = S::NP;
  constexpr int kPairs = NS / 2, kApart = kScanBlock / LP;
  __shared__ __align__(16) float2 du[K][S::kRow];
  __shared__ __align__(16) float sB[K * NP], sC[ENDS ? 4 : K * NP];
  __shared__ float sy[ENDS ? 1 : K][S::kRow];
  __shared__ Marks<K> marks;
  after_previous();
  let_next_start();
  const ScanPlace p = scan_place<S::CH>(a);
  const int tid = threadIdx.x, l = tid % LP, pos = tid / LP;
  const int k1 = tid / S::V8, v1 = tid % S::V8;  // steps 1 and 3: token and vector

  if (!ENDS && p.piece == 0 && a.hT && (a.cu || a.T == 0)) empty_states<S::CH>(a, p, a.h0, a.hT);
  if (p.t0 >= p.t1) return;

  float bias[8], skip[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool in = 8 * v1 + e < p.chans;
    bias[e] = in && a.dt_bias ? a.dt_bias[p.c0 + 8 * v1 + e] : 0.f;
    skip[e] = in && a.skip ? a.skip[p.c0 + 8 * v1 + e] : 0.f;
  }
  float2 A2[P][kPairs], h[P][kPairs];
  float span[P];
  bool have[P];
  long long chan[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int c = S::chan_at(pos + j * kApart);
    have[j] = c < p.chans;
    chan[j] = p.c0 + (have[j] ? c : 0);
    load_states<NS>(A2[j], a.A, chan[j], a.N, l * NS, have[j]);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      A2[j][i] = mul_(A2[j][i], both<float2>(kLog2e));
      h[j][i] = both<float2>(0.f);
    }
    span[j] = 0.f;
  }
  ScanSeq seq = scan_seq_at(a, p.row, p.t0);
  const long long unit = (long long)p.row * a.pieces + p.piece;
  if (!ENDS && a.pieces > 1 && seq.begin < p.t0)
#pragma unroll
    for (int j = 0; j < P; ++j)
      load_states<NS>(h[j], a.state, unit * a.D + chan[j], a.N, l * NS, have[j]);

  Tile<IO, S, VEC, ENDS> next;
  next.load(a, p, p.t0, k1, v1);
  for (int t = p.t0; t < p.t1; t += K) {
    const int count = p.t1 - t < K ? p.t1 - t : K;
    // ---- 1
    Eight<IO> x = next.x, z = next.z;
    {
      float delta[8];
      step_sizes(next.dt, bias, a.softplus, k1 < count, delta);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        du[k1][e * S::V8 + v1] = make_float2(delta[e], k1 < count && 8 * v1 + e < p.chans ? delta[e] * x.at(e) : 0.f);
    }
    next.B.template leave<VEC>(sB, count, a.N);
    if (!ENDS) next.C.template leave<VEC>(sC, count, a.N);
    const bool edges = t <= seq.begin || t + count >= seq.end;
    if (edges) marks.fill(a, p.row, t, count);
    __syncthreads();
    if (t + K < p.t1) next.load(a, p, t + K, k1, v1);
    // ---- 2
    const auto recur = [&](auto checked) {
      constexpr bool kChecked = decltype(checked)::value;
#pragma unroll 1
      for (int k0 = 0; k0 < K; k0 += LP) {
        if (k0 >= count) break;
        float ys[P][LP];
#pragma unroll
        for (int i = 0; i < LP; ++i) {
          const int k = k0 + i;
          const int mark = kChecked ? marks.mark[k] : 0;
          if (kChecked && (mark & 1)) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
              if (a.h0)
                load_states<NS>(h[j], a.h0, (long long)marks.n[k] * a.D + chan[j], a.N, l * NS, have[j]);
              else
#pragma unroll
                for (int q = 0; q < kPairs; ++q) h[j][q] = both<float2>(0.f);
            }
          }
          float2 Bk[kPairs], Ck[kPairs];
          from_shared<NS>(Bk, sB + k * NP + l * NS);
          if (!ENDS) from_shared<NS>(Ck, sC + k * NP + l * NS);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const float2 s = du[k][pos + j * kApart];
            if (ENDS) span[j] += s.x;
            const float2 delta = both<float2>(s.x), u = both<float2>(s.y);
            float2 y = both<float2>(0.f);
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
              const float2 decay = ex2(mul_(delta, A2[j][q]));
              h[j][q] = fma_(decay, h[j][q], mul_(u, Bk[q]));
              if (!ENDS) y = fma_(Ck[q], h[j][q], y);
            }
            if (!ENDS) ys[j][i] = y.x + y.y;
            if (!ENDS && kChecked && (mark & 2) && a.hT)
              store_states<NS>(a.hT, (long long)marks.n[k] * a.D + chan[j], a.N, l * NS, have[j], h[j]);
          }
        }
        if (!ENDS)
#pragma unroll
          for (int j = 0; j < P; ++j) sy[k0 + l][pos + j * kApart] = fold<LP>(ys[j], l);
      }
    };
    if (edges)
      recur(std::true_type());
    else
      recur(std::false_type());
    if (t + count >= seq.end && t + count < p.t1) seq = scan_seq_at(a, p.row, t + count);
    __syncthreads();
    // ---- 3
    if (!ENDS && k1 < count) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = fmaf(skip[e], x.at(e), sy[k1][e * S::V8 + v1]);
        if (a.z) y[e] *= scan_silu(z.at(e));
      }
      store_eight<IO, VEC>(a.y, ((long long)p.row * a.T + t + k1) * a.D + p.c0 + 8 * v1, p.chans - 8 * v1, y);
    }
  }
  if (ENDS) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      store_states<NS>(a.state, unit * a.D + chan[j], a.N, l * NS, have[j], h[j]);
      if (l == 0 && have[j]) a.span[unit * a.D + chan[j]] = span[j];
    }
  }
}

// What enters each piece, from what the pieces before it leave: a thread a state.
__global__ void __launch_bounds__(256) scan_join_kernel(ScanArgs a) {
  after_previous();
  let_next_start();
  const long long per = (long long)a.D * a.N;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.rows * per) return;
  const int row = (int)(i / per), last = scan_last(a);
  const int d = (int)(i % per / a.N);
  const float rate = a.A[i % per];
  float h = 0.f;
  for (int s0 = 0; s0 < a.pieces; s0 += 4) {
    float f[4], sum[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s0 + k < a.pieces && (s0 + k) * a.piece_len < last) {
        const long long unit = (long long)row * a.pieces + s0 + k;
        f[k] = a.state[unit * per + i % per];
        sum[k] = a.span[unit * a.D + d];
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (s0 + k >= a.pieces || (s0 + k) * a.piece_len >= last) return;
      const int t0 = (s0 + k) * a.piece_len;
      const int t1 = t0 + a.piece_len < last ? t0 + a.piece_len : last;
      a.state[((long long)row * a.pieces + s0 + k) * per + i % per] = h;
      h = passes(a, row, t0, t1) ? fmaf(expf(rate * sum[k]), h, f[k]) : f[k];
    }
  }
}

template <typename IO, typename S, bool VEC>
cudaError_t run(ScanArgs a, cudaStream_t s) {
  const int dg = a.D / a.G;
  a.chan_blocks = a.G * ((dg + S::CH - 1) / S::CH);
  const unsigned grid = (unsigned)((long long)a.rows * a.pieces * a.chan_blocks);
  cudaError_t e = cudaSuccess;
  if (a.pieces > 1) {
    e = launch_next(false, scan_fwd_kernel<IO, S, VEC, true>, grid, kScanBlock, 0, s, a);
    if (e == cudaSuccess) e = launch_scan_join(true, a, s);
    if (e != cudaSuccess) return e;
  }
  return launch_next(a.pieces > 1, scan_fwd_kernel<IO, S, VEC, false>, grid, kScanBlock, 0, s, a);
}

template <typename IO, bool VEC>
cudaError_t by_states(const ScanArgs& a, cudaStream_t s) {
  if (a.N <= 4) return run<IO, ScanShape<1, 4, 1>, VEC>(a, s);
  if (a.N <= 8) return run<IO, ScanShape<2, 4, 1>, VEC>(a, s);
  if (a.N <= 16) return run<IO, ScanShape<4, 4, 1>, VEC>(a, s);
  if (a.N <= 32) return run<IO, ScanShape<8, 4, 2>, VEC>(a, s);
  return run<IO, ScanShape<8, 8, 2>, VEC>(a, s);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename IO>
cudaError_t launch_io(const ScanArgs& a, cudaStream_t s) {
  constexpr int kV = 16 / sizeof(IO);
  const bool whole = a.N == 4 || a.N == 8 || a.N == 16 || a.N == 32 || a.N == 64;
  const bool vec = a.D / a.G % 8 == 0 && whole && a.ldx % kV == 0 && a.lddt % kV == 0 &&
                   (!a.z || a.ldz % kV == 0) && a.ldb % 4 == 0 && a.ldc % 4 == 0 && aligned16(a.x) &&
                   aligned16(a.dt) && aligned16(a.z) && aligned16(a.B) && aligned16(a.C) && aligned16(a.y);
  return vec ? by_states<IO, true>(a, s) : by_states<IO, false>(a, s);
}

// Channels of a block by the number of states.
inline int block_chans(int N) { return N <= 4 ? 128 : N <= 8 ? 64 : 32; }

void pieces_of(int rows, int T, int D, int N, int G, int* pieces, int* len) {
  scan_pieces(rows, T, D, G, block_chans(N), 4 * kSms, pieces, len);
}

inline size_t state_bytes(int rows, int pieces, int D, int N) {
  return pieces > 1 ? ((size_t)rows * pieces * D * N * 4 + 255) / 256 * 256 : 0;
}

}  // namespace

cudaError_t launch_scan_join(bool next, const ScanArgs& a, cudaStream_t s) {
  const long long n = (long long)a.rows * a.D * a.N;
  return launch_next(next, scan_join_kernel, (unsigned)((n + 255) / 256), 256, 0, s, a);
}

void scan_pieces(int rows, int T, int D, int G, int chans, int room, int* pieces, int* len) {
  const int dg = D / G;
  const long long units = (long long)rows * G * ((dg + chans - 1) / chans);
  int n = 1;
  if (2 * units <= room) {
    n = (int)(room / units);
    const int most = (T + 127) / 128;
    if (n > most) n = most < 1 ? 1 : most;
  }
  const int each = ((T + n - 1) / n + 63) / 64 * 64;  // whole tiles
  *len = each > 0 ? each : 64;
  *pieces = T > 0 ? (T + *len - 1) / *len : 1;
}

ckda_status check_scan(int rows, int T, int D, int N, int G, const int32_t* cu, int num_seqs, ckda_dtype io) {
  if (io != CKDA_F32 && io != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
  if (rows < 1 || T < 0 || D < 1 || N < 1 || G < 1 || D % G != 0) return CKDA_ERR_INVALID_ARG;
  if (cu && (num_seqs < 1 || rows != 1)) return CKDA_ERR_INVALID_ARG;
  if (N > kScanMostStates || D > 1 << 20) return CKDA_ERR_UNSUPPORTED;
  // (tokens of a row and blocks are counted in 32 bits)
  if (T > 1 << 30 || (long long)rows * T > 0x7fffffffLL) return CKDA_ERR_UNSUPPORTED;
  if ((long long)rows * ((T + 127) / 128 + 1) * D > 0x7fffffffLL * 8) return CKDA_ERR_UNSUPPORTED;
  return CKDA_OK;
}

}  // namespace ckda

using namespace ckda;

extern "C" {

size_t ckda_scan_fwd_workspace_bytes(int B, int T, int D, int N, int G) {
  if (B < 1 || T < 0 || D < 1 || N < 1 || G < 1 || D % G != 0) return 0;
  int pieces, len;
  pieces_of(B, T, D, N, G, &pieces, &len);
  return pieces > 1 ? state_bytes(B, pieces, D, N) + (size_t)B * pieces * D * 4 : 0;
}

ckda_status ckda_scan_fwd(const void* x, const void* dt, const float* A, const void* Bm, const void* C,
                          const float* D_skip, const void* z, const float* dt_bias, const float* h0,
                          void* y, float* hT, const int32_t* cu_seqlens, int num_seqs, int B, int T,
                          int D, int N, int G, long long ldx, long long lddt, long long ldb,
                          long long ldc, long long ldz, ckda_dtype io_dtype, int softplus,
                          void* workspace, size_t workspace_bytes, void* stream) {
  const ckda_status st = check_scan(B, T, D, N, G, cu_seqlens, num_seqs, io_dtype);
  if (st != CKDA_OK) return st;
  if (!A || (T > 0 && (!x || !dt || !Bm || !C || !y))) return CKDA_ERR_INVALID_ARG;
  if (ldx < D || lddt < D || (z && ldz < D) || ldb < (long long)G * N || ldc < (long long)G * N)
    return CKDA_ERR_INVALID_ARG;
  // (a block that writes a final state runs beside one that still reads an initial one)
  const size_t states = (size_t)(cu_seqlens ? num_seqs : B) * D * N;
  if (h0 && hT && h0 < hT + states && hT < h0 + states) return CKDA_ERR_INVALID_ARG;
  ScanArgs a{};
  a.x = x; a.dt = dt; a.B = Bm; a.C = C; a.z = z; a.A = A; a.skip = D_skip; a.dt_bias = dt_bias;
  a.h0 = h0; a.y = y; a.hT = hT; a.cu = cu_seqlens;
  a.ldx = ldx; a.lddt = lddt; a.ldb = ldb; a.ldc = ldc; a.ldz = ldz;
  a.rows = B; a.T = T; a.D = D; a.N = N; a.G = G; a.seqs = cu_seqlens ? num_seqs : B;
  a.softplus = softplus != 0;
  pieces_of(B, T, D, N, G, &a.pieces, &a.piece_len);
  if (a.pieces > 1) {
    if (!workspace || workspace_bytes < ckda_scan_fwd_workspace_bytes(B, T, D, N, G) || !aligned16(workspace))
      return CKDA_ERR_WORKSPACE;
    a.state = static_cast<float*>(workspace);
    a.span = reinterpret_cast<float*>(static_cast<char*>(workspace) + state_bytes(B, a.pieces, D, N));
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = io_dtype == CKDA_F32 ? launch_io<float>(a, s) : launch_io<__nv_bfloat16>(a, s);
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // extern "C"
