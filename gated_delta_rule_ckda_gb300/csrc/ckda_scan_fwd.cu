// ckda_scan_fwd.cu -- selective scan over prompts.  (The formulas and the block's work:
// ckda_scan.cuh.)
//
// What bounds it: N exponentials for every channel of every token, four fma-pipe
// instructions of two states each beside every two of them, and the latency between them:
// a warp holds 32 channels with all their states, so the card has few warps (1024 for
// 8 x 2048 tokens of 4096 channels of 16 states, which take 414 us: fma pipe 41%,
// exponentials 36%, issue 48% of the cycles at 1.7 warps a scheduler).  Memory is read and
// written once, 81 us of that.
//
// Rows with fewer channels than the card has room for are cut into pieces that run side by
// side: a first pass leaves each piece's own end state and the sum of its steps (a state
// decays over a piece by exp(A sum delta)), a scan over the pieces gives the states that
// enter them, and the second pass runs every piece from its own.  (Three packed documents
// of 32,768 tokens of 2048 channels: 539 us, 210 of them the first pass.)
#include "ckda_scan.cuh"

namespace ckda {
namespace {

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
  a.chan_blocks = scan_chan_blocks(a.D, a.G);
  cudaError_t e = cudaSuccess;
  if (a.pieces > 1) {
    e = launch_walk<IO, S, VEC, kEnds>(false, a, s);
    if (e == cudaSuccess) e = launch_scan_join(true, a, s);
    if (e != cudaSuccess) return e;
  }
  return launch_walk<IO, S, VEC, kOut>(a.pieces > 1, a, s);
}

// States of a channel to a lane, by their number.  16 states over two lanes of eight take
// 414 us for the batch above and 539 for the documents, over four lanes of four 542 and 690
// (more shuffles), by one lane 408 and 634 (twice the reads of B and C).
template <typename IO, bool VEC>
cudaError_t by_states(const ScanArgs& a, cudaStream_t s) {
  if (a.N <= 4) return run<IO, ScanShape<1, 4>, VEC>(a, s);
  if (a.N <= 8) return run<IO, ScanShape<2, 4>, VEC>(a, s);
  if (a.N <= 16) return run<IO, ScanShape<2, 8>, VEC>(a, s);
  if (a.N <= 32) return run<IO, ScanShape<4, 8>, VEC>(a, s);
  return run<IO, ScanShape<8, 8>, VEC>(a, s);
}

template <typename IO>
cudaError_t launch_io(const ScanArgs& a, cudaStream_t s) {
  return scan_vectors(a, sizeof(IO)) ? by_states<IO, true>(a, s) : by_states<IO, false>(a, s);
}

// Room for 12 warps an SM: the documents take 578 us with 8, 543 with 12, 554 with 16.  Cut
// where that holds four pieces, as every decay is then computed twice.  Rows of 2048 tokens
// of 4096 channels of 16 states, 128 warps each, whole and cut: 1 315 and 92 us, 3 (four
// pieces) 315 and 248, 4 (three) 316 and 322, 5 and 7 (two) 417 and 471, 419 and 475, 8 420
// and 648; of 8 states 3 254 and 178, 4 254 and 262, 7 320 and 386; 1024 tokens of 64 states
// 2 533 and 363, 3 537 and 551, 4 541 and 721.  Rows of up to 128 tokens stay whole: 100
// tokens of 2048 channels take 29 us, cut 39, like 300 of 1024, which whole take 57.
void pieces_of(int rows, int T, int D, int G, int* pieces, int* len) {
  scan_pieces(rows, T, D, G, 12 * kSms, 4, 64, 128, pieces, len);
}

inline size_t state_bytes(int rows, int pieces, int D, int N) {
  return pieces > 1 ? ((size_t)rows * pieces * D * N * 4 + 255) / 256 * 256 : 0;
}

}  // namespace

cudaError_t launch_scan_join(bool next, const ScanArgs& a, cudaStream_t s) {
  const long long n = (long long)a.rows * a.D * a.N;
  return launch_next(next, scan_join_kernel, (unsigned)((n + 255) / 256), 256, 0, s, a);
}

void scan_pieces(int rows, int T, int D, int G, int room, int fewest, int least, int whole, int* pieces, int* len) {
  const long long units = (long long)rows * scan_chan_blocks(D, G);
  int n = 1;
  if (fewest * units <= room && T > whole) {
    n = (int)(room / units);
    const int most = (T + least - 1) / least;
    if (n > most) n = most;
  }
  const int each = ((T + n - 1) / n + kWalkTile - 1) / kWalkTile * kWalkTile;
  *len = each > 0 ? each : kWalkTile;
  *pieces = T > 0 ? (T + *len - 1) / *len : 1;
}

ckda_status check_scan(int rows, int T, int D, int N, int G, const int32_t* cu, int num_seqs, ckda_dtype io) {
  if (io != CKDA_F32 && io != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
  if (rows < 1 || T < 0 || D < 1 || N < 1 || G < 1 || D % G != 0) return CKDA_ERR_INVALID_ARG;
  if (cu && (num_seqs < 1 || rows != 1)) return CKDA_ERR_INVALID_ARG;
  if (N > kScanMostStates || D > 1 << 20) return CKDA_ERR_UNSUPPORTED;
  // (tokens of a row and blocks are counted in 32 bits)
  if (T > 1 << 30 || (long long)rows * T > 0x7fffffffLL) return CKDA_ERR_UNSUPPORTED;
  if ((long long)rows * (T / 64 + 1) * scan_chan_blocks(D, G) > 0x7fffffffLL) return CKDA_ERR_UNSUPPORTED;
  return CKDA_OK;
}

}  // namespace ckda

using namespace ckda;

extern "C" size_t ckda_scan_fwd_workspace_bytes(int B, int T, int D, int N, int G) {
  if (B < 1 || T < 0 || D < 1 || N < 1 || G < 1 || D % G != 0) return 0;
  int pieces, len;
  pieces_of(B, T, D, G, &pieces, &len);
  return pieces > 1 ? state_bytes(B, pieces, D, N) + (size_t)B * pieces * D * 4 : 0;
}

namespace {

ckda_status forward(const void* x, const void* dt, const float* A, const void* Bm, const void* C,
                    const float* D_skip, const void* z, const float* dt_bias, const float* h0, void* y,
                    float* hT, const int32_t* cu_seqlens, int num_seqs, int B, int T, int D, int N, int G,
                    long long ldx, long long lddt, long long ldb, long long ldc, long long ldz,
                    ckda_dtype io_dtype, int softplus, bool fill, void* workspace, size_t workspace_bytes,
                    void* stream) {
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
  a.softplus = softplus != 0; a.fill = fill;
  const size_t io = io_dtype == CKDA_F32 ? 4 : 2;
  if (scan_clash(a, y, kChannels, io) || scan_clash(a, hT, kStates, io) ||
      overlap(y, scan_bytes(a, kChannels, D, io), hT, scan_bytes(a, kStates, 0, io)))
    return CKDA_ERR_INVALID_ARG;
  pieces_of(B, T, D, G, &a.pieces, &a.piece_len);
  if (a.pieces > 1) {
    if (!workspace || workspace_bytes < ckda_scan_fwd_workspace_bytes(B, T, D, N, G) || !scan_aligned(workspace, 16))
      return CKDA_ERR_WORKSPACE;
    a.state = static_cast<float*>(workspace);
    a.span = reinterpret_cast<float*>(static_cast<char*>(workspace) + state_bytes(B, a.pieces, D, N));
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = io_dtype == CKDA_F32 ? launch_io<float>(a, s) : launch_io<__nv_bfloat16>(a, s);
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // namespace

extern "C" {

ckda_status ckda_scan_fwd(const void* x, const void* dt, const float* A, const void* Bm, const void* C,
                          const float* D_skip, const void* z, const float* dt_bias, const float* h0,
                          void* y, float* hT, const int32_t* cu_seqlens, int num_seqs, int B, int T,
                          int D, int N, int G, long long ldx, long long lddt, long long ldb,
                          long long ldc, long long ldz, ckda_dtype io_dtype, int softplus,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return forward(x, dt, A, Bm, C, D_skip, z, dt_bias, h0, y, hT, cu_seqlens, num_seqs, B, T, D, N, G, ldx, lddt,
                 ldb, ldc, ldz, io_dtype, softplus, false, workspace, workspace_bytes, stream);
}
ckda_status ckda_scan_fwd_filled(const void* x, const void* dt, const float* A, const void* Bm, const void* C,
                                 const float* D_skip, const void* z, const float* dt_bias, const float* h0,
                                 void* y, float* hT, const int32_t* cu_seqlens, int num_seqs, int B, int T,
                                 int D, int N, int G, long long ldx, long long lddt, long long ldb,
                                 long long ldc, long long ldz, ckda_dtype io_dtype, int softplus,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  return forward(x, dt, A, Bm, C, D_skip, z, dt_bias, h0, y, hT, cu_seqlens, num_seqs, B, T, D, N, G, ldx, lddt,
                 ldb, ldc, ldz, io_dtype, softplus, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
