// ckda_linear_serial.cu -- linear attention with a scalar decay per head, token
// by token on CUDA cores: fp32 I/O, and widths the tensor-core kernels do not
// take.  Also the small kernels that finish the gradients of shared heads and
// of decays, which the tensor-core backward uses as well.
//
// Forward and gradients are four runs of one recurrence.  With a state S of
// "own" rows c and contracted columns r,
//     S = a_t S + y_t x_t^T,    out_t = S z_t
//   o  : forward in time, c over dv, y = v,  x = k,  z = q,  a_t = e^{g_t}
//   dq : forward,         c over dk, y = k,  x = v,  z = do, a_t = e^{g_t}
//   dk : backward,        c over dk, y = q,  x = do, z = v,  a_t = e^{g_{t+1}}
//   dv : backward,        c over dv, y = do, x = q,  z = k,  a_t = e^{g_{t+1}}
// The rows of S do not meet, so a block owns 32 of them and a unit (sequence,
// head) spreads over ceil(rows / 32) blocks; four threads share a row, each
// with every fourth group of four columns in registers.  Per token a thread
// does one fma for the update and one for the readout per column, on x and z
// from shared memory, so the bound is the latency of a token times the tokens
// of a unit, and FMA throughput when the units fill the SMs.
//
// The decay's gradient is dg_t = <H_{t-1} e^{g_t}, dL/dH_t>.  With L the
// cumulative log decay, dL/dL_i = q_i.dq_i - k_i.dk_i, and dg is its suffix
// sum plus <hT, dhT>.  Terms that cancel in it are larger than what is left,
// and two measures keep them small:
//   - a token's own product (its key read by its own query), which no decay
//     touches and which is the largest term under strong decay, is left out:
//     the dq and dk runs read the decayed state before the token's write, and
//     the own part, k_t (v_t.do_t) and q_t (v_t.do_t), joins dq and dk last;
//   - the sum restarts every kCkptTokens tokens from <H, dL/dH> itself: the dq
//     run stores the state there and the dk run, which holds dL/dH in the same
//     layout, takes the product.
#include "ckda_linear.cuh"

namespace ckda {
namespace {

constexpr int kTok = 16;     // tokens staged at a time
constexpr int kOwn = 32;     // state rows of a block
constexpr int kSplit = 4;    // threads of a row

enum { RUN_O, RUN_DQ, RUN_DK, RUN_DV };

struct SerialWs {
  float* dq;      // [B, H, T, dk], without the token's own part
  float* dk;      // [B, H, T, dk], the same
  float* dg;      // [B, H, T] (a decay per head only)
  float* own;     // [B, H, T]: scale v_t.do_t
  float* ckpt;    // [slots][dk][dv]: the state entering each 64-token piece, and the last one
  float* dots;    // [slots][slices]: <H, dL/dH> at each piece's end
  int32_t* slot0; // [N + 1]: first slot of a sequence (packed; times H)
  size_t slots;   // slots of a head in the workspace
};

// Slots of sequence n of len tokens: its pieces, and one for its final state.
__host__ __device__ inline int pieces_of(int len) { return (len + kCkptTokens - 1) / kCkptTokens; }

__device__ __forceinline__ size_t slot_of(const LinearArgs& a, const SerialWs& w, int n, int h,
                                          int piece) {
  const size_t first = a.cu_seqlens ? (size_t)w.slot0[n] : (size_t)n * (pieces_of(a.T) + 1);
  // (offsets that are no packing would run past the workspace)
  const size_t slot = first + piece;
  return (slot < w.slots ? slot : w.slots - 1) * a.H + h;
}

__global__ void slot_plan_kernel(LinearArgs a, int32_t* slot0) {
  // one block; each thread adds up a run of sequences, then the runs are joined
  __shared__ int32_t sum[1024];
  const int per = (a.N + 1023) / 1024, i0 = threadIdx.x * per;
  int32_t s = 0;
  for (int i = i0; i < min(i0 + per, a.N); ++i) {
    int t0, len;
    seq_range(a, i, t0, len);
    s += pieces_of(len) + 1;
  }
  sum[threadIdx.x] = s;
  __syncthreads();
  int32_t before = 0;
  for (int j = 0; j < (int)threadIdx.x; ++j) before += sum[j];
  for (int i = i0; i < min(i0 + per, a.N); ++i) {
    slot0[i] = before;
    int t0, len;
    seq_range(a, i, t0, len);
    before += pieces_of(len) + 1;
  }
}

// R4: columns of a thread / 4 (so R <= 16 R4 contracted columns).
template <typename IO, typename OUT, int RUN, int R4>
__global__ void __launch_bounds__(kOwn* kSplit) serial_kernel(LinearArgs a, SerialWs w, OUT* out) {
  constexpr bool kBack = RUN == RUN_DK || RUN == RUN_DV;
  constexpr bool kOwnV = RUN == RUN_O || RUN == RUN_DV;   // rows are value columns
  constexpr bool kDecayed = RUN == RUN_DQ || RUN == RUN_DK;  // read before the write
  constexpr int kR = 16 * R4;
  __shared__ __align__(16) float sx[kTok][kR], sz[kTok][kR], sy[kTok][kOwn];
  __shared__ float sa[kTok];
  __shared__ float red[kOwn * kSplit / 32];

  const int unit = blockIdx.x, n = unit / a.H, h = unit % a.H;
  const int b = a.cu_seqlens ? 0 : n, hk = h / (a.H / a.Hk);
  int t0, len;
  seq_range(a, n, t0, len);
  const int own_n = kOwnV ? a.dv : a.dk, R = kOwnV ? a.dk : a.dv;
  const size_t krow = ((size_t)b * a.Hk + hk) * a.T + t0;  // first row of q and k
  const size_t vrow = ((size_t)b * a.H + h) * a.T + t0;    // first row of v, do, o, dq, ...
  const IO* q = static_cast<const IO*>(a.q) + krow * a.dk;
  const IO* k = static_cast<const IO*>(a.k) + krow * a.dk;
  const IO* v = static_cast<const IO*>(a.v) + vrow * a.dv;
  const IO* dout = static_cast<const IO*>(a.dout) + vrow * a.dv;
  const IO* X = RUN == RUN_O ? k : RUN == RUN_DQ ? v : RUN == RUN_DK ? dout : q;
  const IO* Y = RUN == RUN_O ? v : RUN == RUN_DQ ? k : RUN == RUN_DK ? q : dout;
  const IO* Z = RUN == RUN_O ? q : RUN == RUN_DQ ? dout : RUN == RUN_DK ? v : k;
  // where the query scale goes: on the readout of o and dq, into the state of dk and dv
  const float out_scale = kBack ? 1.f : a.scale, y_scale = kBack ? a.scale : 1.f;
  const float* g = a.g_head ? a.g + h : a.g + vrow;
  const int gs = a.g_head ? 0 : 1;

  const int own = threadIdx.x / kSplit, p = threadIdx.x % kSplit;
  const int c0 = blockIdx.y * kOwn, c = c0 + own;
  const bool row = c < own_n;
  auto col = [&](int i) { return 4 * (p + kSplit * (i / 4)) + i % 4; };  // of register i
  // element (row c, column r) of a [dk, dv] state
  auto at = [&](int r) { return kOwnV ? (size_t)r * a.dv + c : (size_t)c * a.dv + r; };

  float S[4 * R4];
  const float* init = kBack ? a.dhT : a.h0;
  const size_t st = ((size_t)n * a.H + h) * (size_t)a.dk * a.dv;
#pragma unroll
  for (int i = 0; i < 4 * R4; ++i)
    S[i] = init && row && col(i) < R ? init[st + at(col(i))] : 0.f;

  // <stored state, S> over this block's rows, at the end of a piece (dk run)
  auto take_dot = [&](int piece) {
    const float* ck = w.ckpt + slot_of(a, w, n, h, piece + 1) * (size_t)a.dk * a.dv;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i)
      if (row && col(i) < R) s = fmaf(S[i], ck[at(col(i))], s);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      float t = 0.f;
      for (int i = 0; i < kOwn * kSplit / 32; ++i) t += red[i];
      w.dots[slot_of(a, w, n, h, piece) * gridDim.y + blockIdx.y] = t;
    }
  };
  auto store_ckpt = [&](int piece) {
    float* ck = w.ckpt + slot_of(a, w, n, h, piece) * (size_t)a.dk * a.dv;
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i)
      if (row && col(i) < R) ck[at(col(i))] = S[i];
  };

  for (int s0 = 0; s0 < len; s0 += kTok) {
    const int nt = min(kTok, len - s0);
    __syncthreads();
    for (int e = threadIdx.x; e < kTok * kR; e += kOwn * kSplit) {
      const int tt = e / kR, r = e % kR;
      const size_t t = kBack ? len - 1 - (s0 + tt) : s0 + tt;
      const bool in = tt < nt && r < R;
      sx[tt][r] = in ? ld_io(X + t * R + r) : 0.f;
      sz[tt][r] = in ? ld_io(Z + t * R + r) : 0.f;
    }
    for (int e = threadIdx.x; e < kTok * kOwn; e += kOwn * kSplit) {
      const int tt = e / kOwn, cc = e % kOwn;
      const size_t t = kBack ? len - 1 - (s0 + tt) : s0 + tt;
      sy[tt][cc] = tt < nt && c0 + cc < own_n ? y_scale * ld_io(Y + t * own_n + c0 + cc) : 0.f;
    }
    if (threadIdx.x < kTok && (int)threadIdx.x < nt) {
      const int i = s0 + threadIdx.x;
      // backward, the decay from token t + 1 to t; none into the last token
      sa[threadIdx.x] = kBack ? (i == 0 ? 1.f : expf(g[(size_t)(len - i) * gs]))
                              : expf(g[(size_t)i * gs]);
    }
    __syncthreads();
    for (int tt = 0; tt < nt; ++tt) {
      const int t = kBack ? len - 1 - (s0 + tt) : s0 + tt;
      if (RUN == RUN_DQ && t % kCkptTokens == 0) store_ckpt(t / kCkptTokens);
      const float dec = sa[tt], y = sy[tt][own];
      float acc = 0.f;
      if (kDecayed) {
#pragma unroll
        for (int i = 0; i < 4 * R4; ++i) {
          S[i] *= dec;
          acc = fmaf(S[i], sz[tt][col(i)], acc);
        }
        if (RUN == RUN_DK && (t == len - 1 || t % kCkptTokens == kCkptTokens - 1))
          take_dot(t / kCkptTokens);
#pragma unroll
        for (int i = 0; i < 4 * R4; ++i) S[i] = fmaf(y, sx[tt][col(i)], S[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4 * R4; ++i) {
          S[i] = fmaf(dec, S[i], y * sx[tt][col(i)]);
          acc = fmaf(S[i], sz[tt][col(i)], acc);
        }
      }
      acc += __shfl_xor_sync(0xffffffffu, acc, 1);
      acc += __shfl_xor_sync(0xffffffffu, acc, 2);
      if (p == 0 && row) st_io(out + (vrow + t) * own_n + c, out_scale * acc);
    }
  }
  if (RUN == RUN_DQ) store_ckpt(pieces_of(len));
  if (RUN == RUN_DK && a.dh0) {
    const float dec = len > 0 ? expf(g[0]) : 1.f;
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i)
      if (row && col(i) < R) a.dh0[st + at(col(i))] = dec * S[i];
  }
  if (RUN == RUN_O && a.hT) {
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i)
      if (row && col(i) < R) a.hT[st + at(col(i))] = S[i];
  }
}

template <typename IO, typename OUT, int RUN>
cudaError_t launch_run(const LinearArgs& a, const SerialWs& w, OUT* out, cudaStream_t s) {
  constexpr bool kOwnV = RUN == RUN_O || RUN == RUN_DV;
  const int own = kOwnV ? a.dv : a.dk, R = kOwnV ? a.dk : a.dv;
  const dim3 grid((unsigned)a.N * a.H, (own + kOwn - 1) / kOwn);
  if (R <= 32)
    serial_kernel<IO, OUT, RUN, 2><<<grid, kOwn * kSplit, 0, s>>>(a, w, out);
  else if (R <= 64)
    serial_kernel<IO, OUT, RUN, 4><<<grid, kOwn * kSplit, 0, s>>>(a, w, out);
  else
    serial_kernel<IO, OUT, RUN, 8><<<grid, kOwn * kSplit, 0, s>>>(a, w, out);
  return cudaGetLastError();
}

// dg, a piece of one (sequence, head) at a time: each of the four warps takes
// the dot products of every fourth token, then a thread a token sums a suffix.
template <typename IO>
__global__ void __launch_bounds__(128) serial_dg_kernel(LinearArgs a, SerialWs w, float* dg,
                                                        int slices) {
  __shared__ float x[kCkptTokens];
  const int unit = blockIdx.x, n = unit / a.H, h = unit % a.H;
  const int b = a.cu_seqlens ? 0 : n, hk = h / (a.H / a.Hk);
  int t0, len;
  seq_range(a, n, t0, len);
  const size_t krow = ((size_t)b * a.Hk + hk) * a.T + t0;
  const size_t vrow = ((size_t)b * a.H + h) * a.T + t0;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int piece = blockIdx.y; piece * kCkptTokens < len; piece += gridDim.y) {
    const int p0 = piece * kCkptTokens, nt = min(kCkptTokens, len - p0);
    for (int i = wid; i < kCkptTokens; i += 4) {
      float s = 0.f, own = 0.f;
      if (i < nt) {
        const IO* q = static_cast<const IO*>(a.q) + (krow + p0 + i) * a.dk;
        const IO* k = static_cast<const IO*>(a.k) + (krow + p0 + i) * a.dk;
        const float* dq = w.dq + (vrow + p0 + i) * a.dk;
        const float* dk = w.dk + (vrow + p0 + i) * a.dk;
        for (int r = lane; r < a.dk; r += 32)
          s += fmaf(ld_io(q + r), dq[r], -(ld_io(k + r) * dk[r]));
        const IO* v = static_cast<const IO*>(a.v) + (vrow + p0 + i) * a.dv;
        const IO* dout = static_cast<const IO*>(a.dout) + (vrow + p0 + i) * a.dv;
        for (int c = lane; c < a.dv; c += 32) own = fmaf(ld_io(v + c), ld_io(dout + c), own);
      }
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, m);
        own += __shfl_xor_sync(0xffffffffu, own, m);
      }
      if (lane == 0) {
        x[i] = s;
        if (i < nt) w.own[vrow + p0 + i] = a.scale * own;
      }
    }
    __syncthreads();
    if (threadIdx.x < kCkptTokens && (int)threadIdx.x < nt) {
      float s = 0.f;
      const float* d = w.dots + slot_of(a, w, n, h, piece) * slices;
      for (int i = 0; i < slices; ++i) s += d[i];
      for (int i = kCkptTokens - 1; i >= (int)threadIdx.x; --i) s += x[i];
      dg[vrow + p0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// One thread per element of dq and dk; `own` (may be null) as in SerialWs.
template <typename IO>
__global__ void sum_heads_kernel(LinearArgs a, const float* dq, const float* dk,
                                 const float* own) {
  const size_t per = (size_t)a.T * a.dk;         // elements of one head
  const size_t total = (size_t)a.B * a.Hk * per;
  const int group = a.H / a.Hk;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (size_t)gridDim.x * blockDim.x) {
    const size_t head = e / per, first = head * group * per + e % per;
    float x = 0.f, y = 0.f;
    float o = 0.f;
    for (int i = 0; i < group; ++i) {
      x += dq[first + i * per];
      y += dk[first + i * per];
      if (own) o += own[(head * group + i) * a.T + (e % per) / a.dk];
    }
    if (own) {
      x = fmaf(o, ld_io(static_cast<const IO*>(a.k) + e), x);
      y = fmaf(o, ld_io(static_cast<const IO*>(a.q) + e), y);
    }
    st_io(static_cast<IO*>(a.dq) + e, x);
    st_io(static_cast<IO*>(a.dkey) + e, y);
  }
}

// One block a head: B * T values, each thread a strided run in double (the sum
// is long), joined in a fixed order.
__global__ void __launch_bounds__(1024) sum_decay_kernel(LinearArgs a, const float* dg) {
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

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct SerialPlan {
  size_t slots, dq, dk, dg, own, ckpt, dots, slot0, total;
};
SerialPlan serial_plan(int N, int B, int H, int T, int dk, int dv, bool packed) {
  // packed: each sequence has at most T_n / 64 + 1 pieces, and a final state
  SerialPlan p;
  p.slots = packed ? (size_t)T / kCkptTokens + 2 * (size_t)N : (size_t)N * (pieces_of(T) + 1);
  const size_t slots = p.slots * H;
  const size_t rows = (size_t)B * H * T;
  size_t at = 0;
  p.dq = at; at += up256(rows * dk * 4);
  p.dk = at; at += up256(rows * dk * 4);
  p.dg = at; at += up256(rows * 4);
  p.own = at; at += up256(rows * 4);
  p.ckpt = at; at += up256(slots * dk * dv * 4);
  p.dots = at; at += up256(slots * ((dk + kOwn - 1) / kOwn) * 4);
  p.slot0 = at; at += up256(((size_t)N + 1) * 4);
  p.total = at;
  return p;
}

template <typename IO>
cudaError_t serial_bwd_io(const LinearArgs& a, char* ws, cudaStream_t s) {
  const SerialPlan p = serial_plan(a.N, a.B, a.H, a.T, a.dk, a.dv, a.cu_seqlens != nullptr);
  SerialWs w;
  w.dq = reinterpret_cast<float*>(ws + p.dq);
  w.dk = reinterpret_cast<float*>(ws + p.dk);
  w.dg = reinterpret_cast<float*>(ws + p.dg);
  w.own = reinterpret_cast<float*>(ws + p.own);
  w.ckpt = reinterpret_cast<float*>(ws + p.ckpt);
  w.dots = reinterpret_cast<float*>(ws + p.dots);
  w.slot0 = reinterpret_cast<int32_t*>(ws + p.slot0);
  w.slots = p.slots;
  cudaError_t e = cudaSuccess;
  if (a.cu_seqlens) {
    slot_plan_kernel<<<1, 1024, 0, s>>>(a, w.slot0);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = launch_run<IO, float, RUN_DQ>(a, w, w.dq, s)) != cudaSuccess) return e;
  if ((e = launch_run<IO, float, RUN_DK>(a, w, w.dk, s)) != cudaSuccess) return e;
  if ((e = launch_run<IO, IO, RUN_DV>(a, w, static_cast<IO*>(a.dval), s)) != cudaSuccess) return e;
  if (a.T > 0) {
    const int pieces = pieces_of(a.T);
    const dim3 grid((unsigned)a.N * a.H, pieces < 64 ? pieces : 64);
    float* dg = a.g_head ? w.dg : a.dg;
    serial_dg_kernel<IO><<<grid, 128, 0, s>>>(a, w, dg, (a.dk + kOwn - 1) / kOwn);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = linear_sum_heads(a, w.dq, w.dk, w.own, s)) != cudaSuccess) return e;
  }
  return a.g_head ? linear_sum_decay(a, w.dg, s) : e;
}

}  // namespace

cudaError_t linear_serial_fwd(const LinearArgs& a, cudaStream_t s) {
  SerialWs w{};
  return a.io == CKDA_F32
             ? launch_run<float, float, RUN_O>(a, w, static_cast<float*>(a.o), s)
             : launch_run<__nv_bfloat16, __nv_bfloat16, RUN_O>(
                   a, w, static_cast<__nv_bfloat16*>(a.o), s);
}

size_t linear_serial_bwd_bytes(int N, int B, int H, int T, int dk, int dv, bool packed) {
  return serial_plan(N, B, H, T, dk, dv, packed).total;
}

cudaError_t linear_serial_bwd(const LinearArgs& a, char* ws, cudaStream_t s) {
  return a.io == CKDA_F32 ? serial_bwd_io<float>(a, ws, s)
                          : serial_bwd_io<__nv_bfloat16>(a, ws, s);
}

cudaError_t linear_sum_heads(const LinearArgs& a, const float* dq_part, const float* dk_part,
                             const float* own, cudaStream_t s) {
  const size_t total = (size_t)a.B * a.Hk * a.T * a.dk;
  if (total == 0) return cudaSuccess;
  const size_t blocks = (total + 255) / 256;
  const unsigned grid = (unsigned)(blocks < 32 * kLinSms ? blocks : 32 * kLinSms);
  if (a.io == CKDA_F32)
    sum_heads_kernel<float><<<grid, 256, 0, s>>>(a, dq_part, dk_part, own);
  else
    sum_heads_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a, dq_part, dk_part, own);
  return cudaGetLastError();
}

cudaError_t linear_sum_decay(const LinearArgs& a, const float* dg_full, cudaStream_t s) {
  sum_decay_kernel<<<a.H, 1024, 0, s>>>(a, dg_full);
  return cudaGetLastError();
}

}  // namespace ckda
