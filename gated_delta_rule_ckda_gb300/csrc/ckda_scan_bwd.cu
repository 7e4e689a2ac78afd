// ckda_scan_bwd.cu -- the call of the selective scan's gradients: checks and workspace.
// (The kernels: ckda_scan_grad.cuh.)
#include "ckda_scan_grad.cuh"

namespace ckda {
namespace {

// The workspace's parts, in order, each a multiple of 256 bytes.
struct Layout {
  int pieces, len, chunks;
  size_t chunk, chunk_sum, state, span, grad, part_bc, part_a, part_d, bytes;
};
Layout layout_of(int rows, int T, int D, int N, int G) {
  Layout w{};
  // Room for 24 warps an SM, three times what runs at once: the batch of 512 warps takes
  // 1185 us so, 1329 with 16, 1206 with 32.  Cut where that holds four pieces:
  // rows of 1024 tokens of 4096 channels of 16 states, 128 warps each, whole and cut, 4 1038
  // and 653 us, 7 (four pieces) 1086 and 1041, 8 (three) 1092 and 1270, 14 (two) 1883 and
  // 1984; 512 tokens of 32 states 7 1397 and 1334, 9 1444 and 1694.  More than 32 states give
  // a warp enough to do by itself: 512 tokens of 64 states 2 (fourteen pieces) 1306 and 1098,
  // 3 (nine) 1318 and 1587, 4 1328 and 1936.  Pieces of at least 32 tokens: 2 x
  // 1001 tokens of 480 channels of 12 states take 78 us, with 64 99, with 16 108; 100 of
  // 2048 of 16 states 62, with 64 90.  More than 16 states leave fewer warps at once and
  // have more to take up and leave at a piece's ends: 4096 tokens of 512 channels of 64
  // states take 604 us by 64, by 32 710.
  const int least = N <= 16 ? 32 : 64;
  scan_pieces(rows, T, D, G, 24 * kSms, N <= 32 ? 4 : 12, least, least, &w.pieces, &w.len);
  w.chunks = (T + kScanChunk - 1) / kScanChunk;
  const size_t dn = (size_t)D * N * 4, d = (size_t)D * 4, units = (size_t)rows * w.pieces;
  const bool many = w.pieces > 1;
  const auto take = [&](size_t n) {
    const size_t at = w.bytes;
    w.bytes += (n + 255) / 256 * 256;
    return at;
  };
  w.chunk = take((size_t)rows * w.chunks * dn);
  w.chunk_sum = take(many ? (size_t)rows * w.chunks * d : 0);
  w.state = take(many ? units * dn : 0);
  w.span = take(many ? units * d : 0);
  w.grad = take(many ? units * dn : 0);
  w.part_bc = take((size_t)(scan_chan_blocks(D, G) / G) * rows * T * G * 2 * N * 4);
  w.part_a = take(units * dn);
  w.part_d = take(units * 2 * d);
  return w;
}

}  // namespace
}  // namespace ckda

using namespace ckda;

extern "C" {

size_t ckda_scan_bwd_workspace_bytes(int B, int T, int D, int N, int G) {
  if (B < 1 || T < 0 || D < 1 || N < 1 || G < 1 || D % G != 0) return 0;
  return layout_of(B, T, D, N, G).bytes;
}

ckda_status ckda_scan_bwd(const void* dy, const void* x, const void* dt, const float* A,
                          const void* Bm, const void* C, const float* D_skip, const void* z,
                          const float* dt_bias, const float* h0, const float* dhT, void* dx, void* ddt,
                          float* dA, void* dBm, void* dC, float* dD_skip, void* dz, float* ddt_bias,
                          float* dh0, const int32_t* cu_seqlens, int num_seqs, int B, int T, int D,
                          int N, int G, long long ldx, long long lddt, long long ldb, long long ldc,
                          long long ldz, ckda_dtype io_dtype, int softplus, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const ckda_status st = check_scan(B, T, D, N, G, cu_seqlens, num_seqs, io_dtype);
  if (st != CKDA_OK) return st;
  if (!A || !dA || (T > 0 && (!dy || !x || !dt || !Bm || !C || !dx || !ddt || !dBm || !dC)))
    return CKDA_ERR_INVALID_ARG;
  if (T > 0 && (z == nullptr) != (dz == nullptr)) return CKDA_ERR_INVALID_ARG;
  if (ldx < D || lddt < D || (z && ldz < D) || ldb < (long long)G * N || ldc < (long long)G * N)
    return CKDA_ERR_INVALID_ARG;
  const size_t states = (size_t)(cu_seqlens ? num_seqs : B) * D * N;
  if (dh0 && dhT && dh0 < dhT + states && dhT < dh0 + states) return CKDA_ERR_INVALID_ARG;
  const Layout w = layout_of(B, T, D, N, G);
  if (!workspace || workspace_bytes < w.bytes || !scan_aligned(workspace, 16)) return CKDA_ERR_WORKSPACE;
  if ((long long)B * T * G * 2 * N / 256 + (long long)D * (N + 2) / 256 + 2 > 0x7fffffffLL)
    return CKDA_ERR_UNSUPPORTED;
  char* ws = static_cast<char*>(workspace);
  const auto part = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
  ScanBwdArgs b{};
  ScanArgs& a = b.a;
  a.x = x; a.dt = dt; a.B = Bm; a.C = C; a.z = z; a.A = A; a.skip = D_skip; a.dt_bias = dt_bias;
  a.h0 = h0; a.cu = cu_seqlens;
  a.ldx = ldx; a.lddt = lddt; a.ldb = ldb; a.ldc = ldc; a.ldz = ldz;
  a.rows = B; a.T = T; a.D = D; a.N = N; a.G = G; a.seqs = cu_seqlens ? num_seqs : B;
  a.softplus = softplus != 0;
  a.pieces = w.pieces; a.piece_len = w.len;
  a.state = part(w.state); a.span = part(w.span);
  a.dy = dy; a.dhT = dhT;
  b.dx = dx; b.ddt = ddt; b.dz = dz; b.dB = dBm; b.dC = dC; b.dA = dA;
  b.dskip = dD_skip; b.dbias = ddt_bias; b.dh0 = dh0;
  a.chunk = part(w.chunk); a.chunk_sum = part(w.chunk_sum); a.grad = part(w.grad);
  b.part_bc = part(w.part_bc); b.part_a = part(w.part_a); b.part_d = part(w.part_d);
  a.chunks = w.chunks;
  const size_t io = io_dtype == CKDA_F32 ? 4 : 2;
  const struct { const void* p; ScanRows kind; } out[6] = {{dx, kChannels}, {ddt, kChannels}, {dz, kChannels},
                                                           {dBm, kGroups}, {dC, kGroups}, {dh0, kStates}};
  const auto size = [&](int i) { return scan_bytes(a, out[i].kind, out[i].kind == kChannels ? D : (long long)G * N, io); };
  for (int i = 0; i < 6; ++i) {
    if (scan_clash(a, out[i].p, out[i].kind, io)) return CKDA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, size(i), out[j].p, size(j))) return CKDA_ERR_INVALID_ARG;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = io_dtype == CKDA_F32 ? launch_scan_grads<float>(b, s) : launch_scan_grads<__nv_bfloat16>(b, s);
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // extern "C"
