// ckda_linear.cu -- C ABI of linear attention with a scalar decay per head:
// argument checks, the choice of path and the workspace's layout.
#include "ckda_linear.cuh"

namespace ckda {
namespace {

ckda_status check(int B, int H, int Hk, int T, int dk, int dv, ckda_dtype io, float scale,
                  const int32_t* cu, int num_seqs) {
  if (io != CKDA_F32 && io != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || Hk < 1 || H % Hk != 0 || T < 0 || dk < 1 || dv < 1)
    return CKDA_ERR_INVALID_ARG;
  if (!(scale == scale)) return CKDA_ERR_INVALID_ARG;
  if (cu) {
    if (B != 1 || num_seqs < 1) return CKDA_ERR_INVALID_ARG;
  } else if (num_seqs != 0 && num_seqs != B) {
    return CKDA_ERR_INVALID_ARG;
  }
  if (dk > 128 || dv > 128) return CKDA_ERR_UNSUPPORTED;
  if ((long long)B * H * T > 0x7fffffffLL) return CKDA_ERR_UNSUPPORTED;
  if ((long long)(cu ? num_seqs : B) * H > 0x7fffffffLL) return CKDA_ERR_UNSUPPORTED;
  return CKDA_OK;
}

size_t head_bytes(int num_seqs) {  // status word, order of packed sequences
  const size_t n = num_seqs > 0 ? (size_t)num_seqs : 0;
  return kWsStatusBytes + (n * sizeof(int32_t) + 255) / 256 * 256;
}

// Of a call on the tensor cores (chunked) or on CUDA cores.
size_t fwd_bytes(bool chunked, int num_seqs, int B, int H, int T, int dk, int dv) {
  if (num_seqs < 0 || B < 1 || H < 1 || T < 0 || dk < 1 || dv < 1) return 0;
  const int N = num_seqs > 0 ? num_seqs : B;
  return head_bytes(num_seqs) +
         (chunked ? linear_chunk_fwd_bytes(N, B, H, T, dk, dv, num_seqs > 0)
                  : linear_serial_fwd_bytes(N, H, T, dk, dv, num_seqs > 0));
}
size_t bwd_bytes(bool chunked, int num_seqs, int B, int H, int Hk, int T, int dk, int dv) {
  if (num_seqs < 0 || B < 1 || H < 1 || Hk < 1 || T < 0 || dk < 1 || dv < 1) return 0;
  const int N = num_seqs > 0 ? num_seqs : B;
  return head_bytes(num_seqs) +
         (chunked ? linear_chunk_bwd_bytes(N, B, H, Hk, T, dk, dv, num_seqs > 0)
                  : linear_serial_bwd_bytes(N, B, H, Hk, T, dk, dv, num_seqs > 0));
}
size_t most(size_t a, size_t b) { return a > b ? a : b; }

}  // namespace
}  // namespace ckda

using namespace ckda;

extern "C" {

size_t ckda_linear_fwd_workspace_bytes(int num_seqs, int B, int H, int T, int dk, int dv,
                                       ckda_dtype io_dtype) {
  return most(fwd_bytes(false, num_seqs, B, H, T, dk, dv),
              ckda_linear_fwd_aligned_workspace_bytes(num_seqs, B, H, T, dk, dv, io_dtype));
}

size_t ckda_linear_fwd_aligned_workspace_bytes(int num_seqs, int B, int H, int T, int dk, int dv,
                                               ckda_dtype io_dtype) {
  return fwd_bytes(linear_chunk_path(io_dtype, dk, dv), num_seqs, B, H, T, dk, dv);
}

ckda_status ckda_linear_fwd(const void* q, const void* k, const void* v, const float* g,
                            int g_per_head, const float* h0, void* o, float* hT,
                            const int32_t* cu_seqlens, int num_seqs, int B, int H, int Hk, int T,
                            int dk, int dv, ckda_dtype io_dtype, float scale, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const int N = cu_seqlens ? num_seqs : B;
  const ckda_status st = check(B, H, Hk, T, dk, dv, io_dtype, scale, cu_seqlens, num_seqs);
  if (st != CKDA_OK) return st;
  if (T > 0 && (!q || !k || !v || !g || !o)) return CKDA_ERR_INVALID_ARG;
  const bool chunked = linear_chunk_path(io_dtype, dk, dv) && aligned16(q) && aligned16(k) &&
                       aligned16(v) && aligned16(o);
  if (!workspace ||
      workspace_bytes < fwd_bytes(chunked, cu_seqlens ? num_seqs : 0, B, H, T, dk, dv) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return CKDA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LinearArgs a{};
  a.q = q; a.k = k; a.v = v; a.g = g; a.h0 = h0; a.o = o; a.hT = hT;
  a.cu_seqlens = cu_seqlens;
  a.status = static_cast<int*>(workspace);
  a.N = N; a.B = B; a.H = H; a.Hk = Hk; a.T = T; a.dk = dk; a.dv = dv;
  a.g_head = g_per_head ? 1 : 0;
  a.scale = scale; a.io = io_dtype;
  char* scratch = static_cast<char*>(workspace) + head_bytes(cu_seqlens ? num_seqs : 0);
  cudaError_t e = cudaSuccess;
  if (chunked) {
    a.clear = 1;
    if (cu_seqlens) {
      int32_t* order = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + kWsStatusBytes);
      e = launch_seq_order(cu_seqlens, num_seqs, order, s);
      a.order = order;
    }
    if (e == cudaSuccess) e = linear_chunk_fwd(a, scratch, s);
  } else {
    e = cudaMemsetAsync(workspace, 0, sizeof(int), s);
    if (e == cudaSuccess) e = linear_serial_fwd(a, scratch, s);
  }
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

size_t ckda_linear_bwd_workspace_bytes(int num_seqs, int B, int H, int Hk, int T, int dk, int dv,
                                       ckda_dtype io_dtype) {
  return most(bwd_bytes(false, num_seqs, B, H, Hk, T, dk, dv),
              ckda_linear_bwd_aligned_workspace_bytes(num_seqs, B, H, Hk, T, dk, dv, io_dtype));
}

size_t ckda_linear_bwd_aligned_workspace_bytes(int num_seqs, int B, int H, int Hk, int T, int dk,
                                               int dv, ckda_dtype io_dtype) {
  return bwd_bytes(linear_chunk_path(io_dtype, dk, dv), num_seqs, B, H, Hk, T, dk, dv);
}

ckda_status ckda_linear_bwd(const void* q, const void* k, const void* v, const float* g,
                            int g_per_head, const float* h0, const void* dout, const float* dhT,
                            void* dq, void* dkey, void* dval, float* dg, float* dh0,
                            const int32_t* cu_seqlens, int num_seqs, int B, int H, int Hk, int T,
                            int dk, int dv, ckda_dtype io_dtype, float scale, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const int N = cu_seqlens ? num_seqs : B;
  const ckda_status st = check(B, H, Hk, T, dk, dv, io_dtype, scale, cu_seqlens, num_seqs);
  if (st != CKDA_OK) return st;
  if (T > 0 && (!q || !k || !v || !g || !dout || !dq || !dkey || !dval)) return CKDA_ERR_INVALID_ARG;
  if ((T > 0 || g_per_head) && !dg) return CKDA_ERR_INVALID_ARG;
  const bool chunked = linear_chunk_path(io_dtype, dk, dv) && aligned16(q) && aligned16(k) &&
                       aligned16(v) && aligned16(dout) && aligned16(dq) && aligned16(dkey) &&
                       aligned16(dval);
  if (!workspace ||
      workspace_bytes < bwd_bytes(chunked, cu_seqlens ? num_seqs : 0, B, H, Hk, T, dk, dv) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return CKDA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LinearArgs a{};
  a.q = q; a.k = k; a.v = v; a.g = g; a.h0 = h0;
  a.dout = dout; a.dhT = dhT;
  a.dq = dq; a.dkey = dkey; a.dval = dval; a.dg = dg; a.dh0 = dh0;
  a.cu_seqlens = cu_seqlens;
  a.status = static_cast<int*>(workspace);
  a.N = N; a.B = B; a.H = H; a.Hk = Hk; a.T = T; a.dk = dk; a.dv = dv;
  a.g_head = g_per_head ? 1 : 0;
  a.scale = scale; a.io = io_dtype;
  if (cudaMemsetAsync(workspace, 0, sizeof(int), s) != cudaSuccess) return CKDA_ERR_CUDA;
  char* scratch = static_cast<char*>(workspace) + head_bytes(cu_seqlens ? num_seqs : 0);
  cudaError_t e = cudaSuccess;
  if (chunked) {
    if (cu_seqlens) {
      int32_t* order = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + kWsStatusBytes);
      e = launch_seq_order(cu_seqlens, num_seqs, order, s);
      a.order = order;
    }
    if (e == cudaSuccess) e = linear_chunk_bwd(a, scratch, s);
  } else {
    e = linear_serial_bwd(a, scratch, s);
  }
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // extern "C"
