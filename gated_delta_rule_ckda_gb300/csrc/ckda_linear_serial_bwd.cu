// ckda_linear_serial_bwd.cu -- gradients of linear attention with a scalar decay per
// head on CUDA cores: fp32 I/O, and widths the tensor-core kernels do not take.  Also
// the kernel that finishes the gradient of a decay per head, which the tensor-core
// backward uses as well.
//
// A piece of 64 tokens as matrix products, with H the state entering it, G the
// gradient of the state after it, and D, e, w its decays:
//     B_ij = scale D_ij do_i.v_j          A_ij = scale D_ij q_i.k_j
//     dq_i = scale e_i H do_i + sum_{j <= i} B_ij k_j
//     dk_j = w_j G v_j + sum_{i >= j} B_ij q_i
//     dv_j = w_j G^T k_j + sum_{i >= j} A_ij do_i
// 2 x 6 heads of 48 and 80 channels, three to a key head, 1001 tokens in fp32: 73 us, of
// which 15 are the pieces' own states, 10 their scan and 45 this (token by token, in
// three runs bound by a token's latency, 131 us).  4 x 16 x 2048, 128 channels: 1372 us;
// 8 x 16 x 2048 of 100 channels in bf16 2726 us.
//
// The decay's gradient is dg_t = <H_{t-1} e^{g_t}, dL/dH_t>, in a piece
//     dg_t = e <H, G> + sum_{j<t} w_j k_j.(G v_j)
//            + sum_{i>=t} [ scale e_i q_i.(H do_i) + sum_{j<i} W_ij - sum_{l>i} W_li ],
//     W_ij = B_ij (q_i.k_j)
// with no term that is larger than what it counts: a token's own product W_ii, which no
// decay touches and which is the largest under strong decay, is left out of the sums of dq
// and dk and joins them last.  (The suffix sums of q.dq - k.dk from <H, G> at the piece's
// end are the same in exact arithmetic, but take the products of G that t does not count
// off again: at g = -8 that left dg 1e-3 to 5e-3 of its rms.  It cost 2% less time.)
#include "ckda_linear_piece.cuh"

namespace ckda {
namespace {

struct SerialWs {
  Pieces p;
  float* dq;      // [B, H, T, dk], null unless heads share keys
  float* dk;      // the same
  float* dg;      // [B, H, T] (a decay per head only)
};

// The gradients of one piece of one (sequence, head), 256 threads, everything in
// shared memory in fp32.  Thread (r, c) of 16 x 16 has rows 4 r .. 4 r + 3 (tokens)
// and columns c, c + 16, ... of every product: the sixteen threads of a row read
// one address, and rows padded by four floats keep the others' banks apart.  CK:
// key channels of a slab / 16, CV: value channels / 16.  A state is staged in slabs
// of 64 key channels.  Masks are taken exactly: a token's values, whatever they
// are, enter no gradient that they do not belong to.
//
// 64 tokens of 48 and 80 channels are 1.6 M fmas a piece.  Issue bounds it, of fmas and
// of shared-memory reads about equally, and with few pieces the fetch of its code.
// Paired fmas with their sums in two halves were slower (82 us for 74 then: registers).
size_t grad_smem(int CK, int slabs, int dv) {
  return (size_t)(2 * kTok * (16 * CK * slabs + 4) + (2 * kTok + 16 * CK) * row_floats(dv) +
                  kTok * kPS + 5 * kTok + 8) * sizeof(float);
}

template <typename IO, int CK, int CV>
__global__ void __launch_bounds__(kPieceThreads, 2) piece_grad_kernel(LinearArgs a, SerialWs w,
                                                                     float* dg) {
  after_previous();
  let_next_start();
  extern __shared__ __align__(16) float sm[];
  Where u;
  if (!where(a, w.p, blockIdx.x, u) || u.piece >= u.pieces) return;
  const int slabs = (a.dk + 16 * CK - 1) / (16 * CK), cols = 16 * CK * slabs;
  const int sk = cols + 4, nt = u.len, tid = threadIdx.x;
  const int sv = row_floats(a.dv);
  float *sq = sm, *skey = sq + kTok * sk, *sval = skey + kTok * sk, *sdo = sval + kTok * sv,
        *slab = sdo + kTok * sv, *sp = slab + 16 * CK * sv, *sg = sp + kTok * kPS,
        *se = sg + kTok, *sw = se + kTok, *own = sw + kTok, *sx = own + kTok, *red = sx + kTok;
  const int r = tid >> 4, c = tid & 15, row = 4 * r;
  const size_t states = (size_t)a.dk * a.dv;
  const float* H = w.p.H + (u.slot * a.H + u.h) * states;
  const float* G = w.p.G + (min(u.slot + 1, w.p.slots - 1) * a.H + u.h) * states;
  auto stage_slab = [&](const float* S, int s) {
    stage_rows(slab, sv, S + (size_t)16 * CK * s * a.dv, a.dv, a.dv,
               min(16 * CK, a.dk - 16 * CK * s), 16 * CK, sv - 4);
  };

  stage_rows(sval, sv, static_cast<const IO*>(a.v) + u.vrow * a.dv, a.dv, a.dv, nt, kTok, sv - 4);
  stage_rows(sdo, sv, static_cast<const IO*>(a.dout) + u.vrow * a.dv, a.dv, a.dv, nt, kTok, sv - 4);
  stage_rows(sq, sk, static_cast<const IO*>(a.q) + u.krow * a.dk, a.dk, a.dk, nt, kTok, cols);
  stage_rows(skey, sk, static_cast<const IO*>(a.k) + u.krow * a.dk, a.dk, a.dk, nt, kTok, cols);
  stage_slab(H, 0);
  if (tid < kTok)
    sg[tid] = tid < nt ? (a.g_head ? a.g[u.h] : a.g[u.vrow + tid]) : 0.f;
  __syncthreads();
  piece_decays(sp, se, sw, sg, nt);
  copies_arrived();

  const int dk4 = (a.dk + 3) & ~3, dv4 = (a.dv + 3) & ~3, nt4 = (nt + 3) & ~3;
  float D[4][4];
  {
    float b[4][4] = {};
    add_nt(b, sdo + row * sv, sv, sval + c * sv, sv, dv4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int from = c + 16 * j, at = (row + i) * kPS + from;
        D[i][j] = expf(sp[at]);
        sp[at] = row + i > from ? a.scale * D[i][j] * b[i][j] : 0.f;
        if (row + i == from) own[from] = a.scale * b[i][j];
      }
  }
  __syncthreads();
  // from here on the values go into products with the decay to the piece's end
  for (int i = tid >> 5; i < kTok; i += kPieceThreads / 32)
    for (int j = tid & 31; j < sv - 4; j += 32) sval[i * sv + j] *= sw[i];

  float x[4] = {};  // q.dq - k.dk without G's part of dk, this thread's columns
  // a column of a result, with the token's own part
  auto put = [&](float (&acc)[4][CK], int s, const float* with, IO* out, float* parts) {
    const auto put_to = [&](auto* to) {
      to += (size_t)row * a.dk;
#pragma unroll
      for (int i = 0; i < 4; ++i, to += a.dk)
        if (row + i < nt)
#pragma unroll
          for (int j = 0; j < CK; ++j) {
            const int col = 16 * CK * s + c + 16 * j;
            if (col < a.dk)
              st_io(to + col, fmaf(own[row + i], with[(row + i) * sk + col], acc[i][j]));
          }
    };
    if constexpr (std::is_same_v<IO, float>) {
      put_to(parts ? parts + u.vrow * a.dk : out + u.krow * a.dk);
    } else {
      if (parts)
        put_to(parts + u.vrow * a.dk);
      else
        put_to(out + u.krow * a.dk);
    }
  };
#pragma unroll 1
  for (int s = 0; s < slabs; ++s) {  // dq
    float acc[4][CK] = {};
    add_nt(acc, sdo + row * sv, sv, slab + c * sv, sv, dv4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < CK; ++j) acc[i][j] *= a.scale * se[row + i];
    const float* k = skey + 16 * CK * s + c;
    add_nn<false>(acc, sp + row * kPS, kPS, k, sk, 0, row);
    add_diag<false, false>(acc, sp + row * kPS, kPS, k, sk, row);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < CK; ++j)
        x[i] = fmaf(sq[(row + i) * sk + 16 * CK * s + c + 16 * j], acc[i][j], x[i]);
    put(acc, s, skey, static_cast<IO*>(a.dq), w.dq);
    __syncthreads();
    if (s + 1 < slabs)
      stage_slab(H, s + 1);
    else
      stage_slab(G, 0);
    copies_arrived();
  }
  float dv[4][CV] = {};
  float hg = 0.f;
#pragma unroll 1
  for (int s = 0; s < slabs; ++s) {  // dk, and the state's part of dv
    float acc[4][CK] = {};
    const float* q = sq + 16 * CK * s + c;
    add_diag<true, false>(acc, sp + row, kPS, q, sk, row);
    add_nn<true>(acc, sp + row, kPS, q, sk, row + 4, nt4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < CK; ++j)
        x[i] = fmaf(-skey[(row + i) * sk + 16 * CK * s + c + 16 * j], acc[i][j], x[i]);
    add_nt(acc, sval + row * sv, sv, slab + c * sv, sv, dv4);
    put(acc, s, sq, static_cast<IO*>(a.dkey), w.dk);
    const int rows = min(16 * CK, a.dk - 16 * CK * s);
    // (keys past dk are zeros, as are the slab's rows)
    add_nn<false>(dv, skey + row * sk + 16 * CK * s, sk, slab + c, sv, 0, (rows + 3) & ~3);
    const float* h = H + (size_t)16 * CK * s * a.dv;
#pragma unroll
    for (int i = 0; i < 2 * CK; ++i)  // a warp a row, all its loads in flight
#pragma unroll
      for (int j = 0; j < (CV + 1) / 2; ++j) {
        const int rr = (tid >> 5) + 8 * i, cc = (tid & 31) + 32 * j;
        if (rr < rows && cc < a.dv) hg = fmaf(slab[rr * sv + cc], h[rr * a.dv + cc], hg);
      }
    if (s + 1 < slabs) {
      __syncthreads();
      stage_slab(G, s + 1);
      copies_arrived();
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y = 0.f;  // w k.(G v)
#pragma unroll
    for (int j = 0; j < CV; ++j) {
      if (c + 16 * j < a.dv) y = fmaf(sval[(row + i) * sv + c + 16 * j], dv[i][j], y);
      dv[i][j] *= sw[row + i];
    }
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) {
      x[i] += __shfl_xor_sync(0xffffffffu, x[i], m);
      y += __shfl_xor_sync(0xffffffffu, y, m);
    }
    if (c == 0) {
      sx[row + i] = x[i];
      sg[row + i] = y;  // (the decays have been read)
    }
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) hg += __shfl_xor_sync(0xffffffffu, hg, m);
  if ((tid & 31) == 0) red[tid >> 5] = hg;
  {
    float b[4][4] = {};
    add_nt(b, sq + row * sk, sk, skey + c * sk, sk, dk4);
    __syncthreads();  // B has been read
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sp[(row + i) * kPS + c + 16 * j] = row + i >= c + 16 * j ? a.scale * D[i][j] * b[i][j] : 0.f;
  }
  __syncthreads();
  add_diag<true, true>(dv, sp + row, kPS, sdo + c, sv, row);
  add_nn<true>(dv, sp + row, kPS, sdo + c, sv, row + 4, nt4);
  IO* dval = static_cast<IO*>(a.dval);
#pragma unroll
  for (int j = 0; j < CV; ++j)
    if (c + 16 * j < a.dv)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row + i < nt) st_io(dval + (u.vrow + row + i) * a.dv + c + 16 * j, dv[i][j]);
  if (tid < 32) {  // lane l has tokens l and 32 + l
    // sums of x from a token to the piece's end, and of y over the tokens before it
    float lo = sx[tid], hi = sx[32 + tid], ylo = sg[tid], yhi = sg[32 + tid], all = 0.f;
    for (int i = 0; i < 8; ++i) all += red[i];
    all *= se[kTok - 1];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const float y = __shfl_down_sync(0xffffffffu, lo, m), z = __shfl_down_sync(0xffffffffu, hi, m);
      const float p = __shfl_up_sync(0xffffffffu, ylo, m), o = __shfl_up_sync(0xffffffffu, yhi, m);
      if (tid + m < 32) lo += y, hi += z;
      if (tid >= m) ylo += p, yhi += o;
    }
    lo += __shfl_sync(0xffffffffu, hi, 0);
    yhi += __shfl_sync(0xffffffffu, ylo, 31);
    const float last = __shfl_sync(0xffffffffu, ylo, 31);
    ylo = __shfl_up_sync(0xffffffffu, ylo, 1);  // before the token: shifted, not subtracted
    yhi = __shfl_up_sync(0xffffffffu, yhi, 1);
    if (tid == 0) ylo = 0.f, yhi = last;
    if (tid < nt) dg[u.vrow + tid] = all + ylo + lo;
    if (32 + tid < nt) dg[u.vrow + 32 + tid] = all + yhi + hi;
  }
}

// One thread per element of dq and dk: the sums over the heads that share them.
template <typename IO>
__global__ void sum_heads_kernel(LinearArgs a, const float* dq, const float* dk) {
  after_previous();
  let_next_start();
  const size_t per = (size_t)a.T * a.dk;         // elements of one head
  const size_t total = (size_t)a.B * a.Hk * per;
  const int group = a.H / a.Hk;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (size_t)gridDim.x * blockDim.x) {
    const size_t first = e / per * group * per + e % per;
    float x = 0.f, y = 0.f;
#pragma unroll 4
    for (int i = 0; i < group; ++i) {
      x += dq[first + i * per];
      y += dk[first + i * per];
    }
    st_io(static_cast<IO*>(a.dq) + e, x);
    st_io(static_cast<IO*>(a.dkey) + e, y);
  }
}

// One block a head: B * T values, each thread a strided run in double (the sum
// is long), joined in a fixed order.
__global__ void __launch_bounds__(1024) sum_decay_kernel(LinearArgs a, const float* dg) {
  after_previous();
  let_next_start();
  __shared__ double red[1024];
  const int h = blockIdx.x;
  double s = 0.0;
  for (size_t e = threadIdx.x; e < (size_t)a.B * a.T; e += 1024)
    s += (double)dg[((e / a.T) * a.H + h) * a.T + e % a.T];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int m = 512; m >= 1; m >>= 1) {
    if ((int)threadIdx.x < m) red[threadIdx.x] += red[threadIdx.x + m];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.dg[h] = (float)red[0];
}

struct SerialPlan {
  size_t slots, dq, dk, dg, H, G, dec, slot0, total;
};
SerialPlan serial_plan(int N, int B, int H, int Hk, int T, int dk, int dv, bool packed) {
  SerialPlan p;
  p.slots = slots_of(N, T, packed);
  const size_t states = p.slots * H * dk * dv * 4;
  const size_t rows = (size_t)B * H * T, parts = H == Hk ? 0 : up256(rows * dk * 4);
  size_t at = 0;
  p.dq = at; at += parts;
  p.dk = at; at += parts;
  p.dg = at; at += up256(rows * 4);
  p.H = at; at += up256(states);
  p.G = at; at += up256(states);
  p.dec = at; at += up256(p.slots * H * 4);
  p.slot0 = at; at += up256(((size_t)N + 1) * 4);
  p.total = at;
  return p;
}

template <typename IO, int CK, int CV>
cudaError_t launch_grad(const LinearArgs& a, const SerialWs& w, cudaStream_t s) {
  const size_t smem = grad_smem(CK, (a.dk + 16 * CK - 1) / (16 * CK), a.dv);
  const cudaError_t e = allow_smem<piece_grad_kernel<IO, CK, CV>>(grad_smem(CK, kMostSlabs<CK>, 16 * CV));
  if (e != cudaSuccess) return e;
  return launch_next(true, piece_grad_kernel<IO, CK, CV>, (unsigned)(w.p.slots * a.H),
                     kPieceThreads, smem, s, a, w, a.g_head ? w.dg : a.dg);
}
template <typename IO>
cudaError_t grad(const LinearArgs& a, const SerialWs& w, cudaStream_t s) {
  return with_columns(a.dv, [&](auto cv) {
    return with_slab(a.dk, [&](auto ck) {
      return launch_grad<IO, decltype(ck)::value, decltype(cv)::value>(a, w, s);
    });
  });
}

template <typename IO>
cudaError_t sum_heads(const LinearArgs& a, const SerialWs& w, cudaStream_t s) {
  const size_t total = (size_t)a.B * a.Hk * a.T * a.dk, blocks = (total + 255) / 256;
  const unsigned grid = (unsigned)(blocks < 32 * kLinSms ? blocks : 32 * kLinSms);
  return launch_next(true, sum_heads_kernel<IO>, grid, 256, 0, s, a, w.dq, w.dk);
}

template <typename IO>
cudaError_t serial_bwd_io(const LinearArgs& a, char* ws, cudaStream_t s) {
  const SerialPlan p = serial_plan(a.N, a.B, a.H, a.Hk, a.T, a.dk, a.dv, a.cu_seqlens != nullptr);
  SerialWs w{};
  if (a.H != a.Hk) {
    w.dq = reinterpret_cast<float*>(ws + p.dq);
    w.dk = reinterpret_cast<float*>(ws + p.dk);
  }
  w.dg = reinterpret_cast<float*>(ws + p.dg);
  w.p.slots = p.slots;
  w.p.H = reinterpret_cast<float*>(ws + p.H);
  w.p.G = reinterpret_cast<float*>(ws + p.G);
  w.p.dec = reinterpret_cast<float*>(ws + p.dec);
  cudaError_t e = cudaSuccess;
  if (a.cu_seqlens) {
    int32_t* slot0 = reinterpret_cast<int32_t*>(ws + p.slot0);
    w.p.slot0 = slot0;
    if ((e = linear_plan_slots(a, slot0, s)) != cudaSuccess) return e;
  }
  if ((e = linear_join_pieces(a, w.p, 2, s)) != cudaSuccess) return e;
  if (a.T > 0) {
    if ((e = grad<IO>(a, w, s)) != cudaSuccess) return e;
    if (w.dq && (e = sum_heads<IO>(a, w, s)) != cudaSuccess) return e;
  }
  return a.g_head ? linear_sum_decay(a, w.dg, s) : e;
}

}  // namespace

size_t linear_serial_bwd_bytes(int N, int B, int H, int Hk, int T, int dk, int dv, bool packed) {
  return serial_plan(N, B, H, Hk, T, dk, dv, packed).total;
}

cudaError_t linear_serial_bwd(const LinearArgs& a, char* ws, cudaStream_t s) {
  return a.io == CKDA_F32 ? serial_bwd_io<float>(a, ws, s)
                          : serial_bwd_io<__nv_bfloat16>(a, ws, s);
}

cudaError_t linear_sum_decay(const LinearArgs& a, const float* dg_full, cudaStream_t s) {
  return launch_next(true, sum_decay_kernel, a.H, 1024, 0, s, a, dg_full);
}

}  // namespace ckda
