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
// The rows of S do not meet, so a block owns 32 of them and a (sequence, head)
// spreads over ceil(rows / 32) blocks; four threads share a row, each with every
// fourth group of four columns in registers.  Per token a thread does one fma
// for the update and one for the readout per column, on x and z from shared
// memory, 64 tokens of which are staged at a time: the bound is the latency of a
// token, and FMA throughput when the blocks fill the SMs.
//
// Tokens are serial, so a sequence is cut into pieces that run side by side: a
// first kernel sums each piece's own contribution to the state (all tokens with
// their decay to the piece's end, in no order), a scan joins them, and then every
// piece's runs start from the state that enters them.  Backward a piece is 64
// tokens, whatever the size; forward as many as leave enough blocks for the SMs,
// or the whole sequence where the heads alone do.
//
// The decay's gradient is dg_t = <H_{t-1} e^{g_t}, dL/dH_t>.  With L the
// cumulative log decay, dL/dL_i = q_i.dq_i - k_i.dk_i, and dg is its suffix
// sum plus <hT, dhT>.  Terms that cancel in it are larger than what is left,
// and two measures keep them small:
//   - a token's own product (its key read by its own query), which no decay
//     touches and which is the largest term under strong decay, is left out:
//     the dq and dk runs read the decayed state before the token's write, and
//     the own part, k_t (v_t.do_t) and q_t (v_t.do_t), joins dq and dk last;
//   - the sum restarts at every piece from <H, dL/dH> itself.
#include <type_traits>
#include "ckda_linear.cuh"

namespace ckda {
namespace {

constexpr int kTok = 64;     // tokens staged at a time
constexpr int kOwn = 32;     // state rows of a block
constexpr int kSplit = 4;    // threads of a row
constexpr int kThreads = kOwn * kSplit;

enum { RUN_O, RUN_DQ, RUN_DK, RUN_DV };

// Pieces of a sequence, and the tables over them.  Slot p of a sequence is the
// state entering its piece p (H) or the gradient of that state (G); the slot
// after its last piece is the final state's.
struct Pieces {
  int tokens;             // of a piece
  const int32_t* slot0;   // packed: [N + 1] first slot of a sequence
  size_t slots;           // of a head
  float* H;               // [slots][H][dk][dv]
  float* G;
};
struct SerialWs {
  Pieces p;
  float* dq;      // [B, H, T, dk], without the token's own part
  float* dk;      // [B, H, T, dk], the same
  float* dg;      // [B, H, T] (a decay per head only)
  float* own;     // [B, H, T]: scale v_t.do_t
};

__host__ __device__ inline int pieces_of(int len, int tokens) { return (len + tokens - 1) / tokens; }

// A piece of one (sequence, head).
struct Where {
  int n, h, piece, pieces;
  int t0, len;            // its tokens on the T axis
  size_t slot;            // of the state entering it
  size_t krow, vrow;      // row of its first token in q, k and in v, do, ...
};
// Block x runs over slots times heads, final states' slots among them; false
// where there is no piece.
__device__ __forceinline__ bool where(const LinearArgs& a, const Pieces& p, size_t block, Where& u) {
  size_t s = block / a.H;
  u.h = block % a.H;
  u.slot = s;
  if (a.cu_seqlens) {
    if (s >= (size_t)p.slot0[a.N]) return false;
    int lo = 0, hi = a.N;  // slot0[lo] <= s < slot0[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((size_t)p.slot0[mid] <= s) lo = mid; else hi = mid;
    }
    u.n = lo;
    u.piece = (int)(s - p.slot0[lo]);
  } else {
    const int per = pieces_of(a.T, p.tokens) + 1;
    u.n = (int)(s / per);
    u.piece = (int)(s % per);
  }
  int t0, len;
  seq_range(a, u.n, t0, len);
  u.pieces = pieces_of(len, p.tokens);
  u.t0 = t0 + u.piece * p.tokens;
  u.len = min(len - u.piece * p.tokens, p.tokens);
  const int b = a.cu_seqlens ? 0 : u.n, hk = u.h / (a.H / a.Hk);
  u.krow = ((size_t)b * a.Hk + hk) * a.T + u.t0;
  u.vrow = ((size_t)b * a.H + u.h) * a.T + u.t0;
  return true;
}

__global__ void slot_plan_kernel(LinearArgs a, int tokens, int32_t* slot0) {
  // one block; each thread adds up a run of sequences, then the runs are joined
  __shared__ int32_t sum[1024];
  const int per = (a.N + 1023) / 1024, i0 = threadIdx.x * per, i1 = min(i0 + per, a.N);
  int32_t s = 0;
  for (int i = i0; i < i1; ++i) {
    int t0, len;
    seq_range(a, i, t0, len);
    s += pieces_of(len, tokens) + 1;
  }
  sum[threadIdx.x] = s;
  __syncthreads();
  if (i0 >= i1) return;
  int32_t before = 0;
  for (int j = 0; j < (int)threadIdx.x; ++j) before += sum[j];
  for (int i = i0; i < i1; ++i) {
    slot0[i] = before;
    int t0, len;
    seq_range(a, i, t0, len);
    before += pieces_of(len, tokens) + 1;
  }
  if (i1 == a.N) slot0[a.N] = before;
}

// Register i of a thread's quarter p of a row: column.
__device__ __forceinline__ int col(int p, int i) { return 4 * (p + kSplit * (i / 4)) + i % 4; }

// Two columns an instruction: issue is what bounds a run that fills the SMs.
struct alignas(8) F2 {
  float x, y;
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ void copy16(float* dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                     __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}

// Stages `nt` tokens of `n` columns from `c0` on into [kTok][WIDTH], the rest
// zeros; back: in reverse, ending with the token at `src`.  Four columns at a
// time where rows and base allow it (fp32 by cp.async, all at once in flight:
// staging one element a load took most of a piece's time).
template <typename IO, int WIDTH>
__device__ __forceinline__ void stage(float* dst, const IO* src, int stride, int c0, int n, int nt,
                                      bool back) {
  constexpr uintptr_t kMask = 4 * sizeof(IO) - 1;
  const bool four = ((stride | n) & 3) == 0 && (reinterpret_cast<uintptr_t>(src) & kMask) == 0;
  if (four) {
#pragma unroll 8
    for (int e = threadIdx.x; e < kTok * WIDTH / 4; e += kThreads) {
      const int tt = e / (WIDTH / 4), c = 4 * (e % (WIDTH / 4));
      const int t = back ? nt - 1 - tt : tt;
      const bool in = tt < nt && c < n;
      const IO* from = in ? src + (size_t)t * stride + c0 + c : src;
      if constexpr (sizeof(IO) == 4)
        copy16(dst + 4 * e, from, in);
      else
        *reinterpret_cast<float4*>(dst + 4 * e) = in ? load4(from) : make_float4(0, 0, 0, 0);
    }
    return;
  }
#pragma unroll 8
  for (int e = threadIdx.x; e < kTok * WIDTH; e += kThreads) {
    const int tt = e / WIDTH, c = e % WIDTH;
    const size_t t = back ? nt - 1 - tt : tt;
    dst[e] = tt < nt && c < n ? ld_io(src + t * stride + c0 + c) : 0.f;
  }
}
__device__ __forceinline__ void staged() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}

// A piece's own contribution to the state after it (block z = 0: over k and v,
// into the slot behind it) or to the gradient of the state before it (z = 1:
// over q and do, into its own slot).  R4: columns of a thread / 4.
template <typename IO, int R4>
__global__ void __launch_bounds__(kThreads) piece_sum_kernel(LinearArgs a, Pieces p, int first_z) {
  constexpr int kR = 16 * R4;
  extern __shared__ __align__(16) float sm[];
  float *sx = sm, *sy = sm + kTok * kR, *sw = sy + kTok * kOwn;
  Where u;
  if (!where(a, p, blockIdx.x, u) || u.piece >= u.pieces) return;
  const bool back = blockIdx.z + first_z == 1;
  const IO* X = back ? static_cast<const IO*>(a.dout) + u.vrow * a.dv
                     : static_cast<const IO*>(a.v) + u.vrow * a.dv;
  const IO* Y = (back ? static_cast<const IO*>(a.q) : static_cast<const IO*>(a.k)) + u.krow * a.dk;
  const float* g = a.g_head ? a.g + u.h : a.g + u.vrow;
  const int gs = a.g_head ? 0 : 1;
  const int own = threadIdx.x / kSplit, part = threadIdx.x % kSplit;
  const int c0 = blockIdx.y * kOwn, c = c0 + own;
  F2 S[2 * R4];
#pragma unroll
  for (int i = 0; i < 2 * R4; ++i) S[i] = F2{0.f, 0.f};
  float* out = (back ? p.G : p.H);
  const size_t slot = min(u.slot + (back ? 0 : 1), p.slots - 1);
  out += (slot * a.H + u.h) * (size_t)a.dk * a.dv;
  // tiles of 64 tokens in the direction of time, backward against it: the
  // decays of later tiles multiply what is there
  for (int s0 = 0; s0 < u.len; s0 += kTok) {
    const int nt = min(kTok, u.len - s0), t0 = back ? u.len - s0 - nt : s0;
    __syncthreads();
    stage<IO, kR>(sx, X + (size_t)t0 * a.dv, a.dv, 0, a.dv, nt, false);
    stage<IO, kOwn>(sy, Y + (size_t)t0 * a.dk, a.dk, c0, min(kOwn, a.dk - c0), nt, false);
    if (threadIdx.x < kTok) sw[kTok + threadIdx.x] =
        (int)threadIdx.x < nt ? g[(size_t)(t0 + threadIdx.x) * gs] : 0.f;
    staged();
    if (threadIdx.x <= kTok) {
      // forward: from after token t to the tile's end; backward: from its start
      // to t; entry kTok: over the tile
      const int t = threadIdx.x;
      float x = 0.f;
      if (t == kTok || back)
        for (int i = 0; i < (t == kTok ? nt : min(t + 1, nt)); ++i) x += sw[kTok + i];
      else
        for (int i = nt - 1; i > t; --i) x += sw[kTok + i];
      sw[t == kTok ? 2 * kTok : t] = (t < kTok && back ? a.scale : 1.f) * expf(x);
    }
    __syncthreads();
    const float all = sw[2 * kTok];
#pragma unroll
    for (int i = 0; i < 2 * R4; ++i) S[i] = mul2(S[i], s0 ? F2{all, all} : F2{1.f, 1.f});
#pragma unroll 2
    for (int t = 0; t < nt; ++t) {
      const float y = sw[t] * sy[t * kOwn + own];
      const float4* x = reinterpret_cast<const float4*>(sx + t * kR) + part;
#pragma unroll
      for (int i = 0; i < R4; ++i) {
        const float4 xv = x[kSplit * i];
        S[2 * i] = fma2(F2{y, y}, F2{xv.x, xv.y}, S[2 * i]);
        S[2 * i + 1] = fma2(F2{y, y}, F2{xv.z, xv.w}, S[2 * i + 1]);
      }
    }
  }
  if (c < a.dk)
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i)
      if (col(part, i) < a.dv) out[(size_t)c * a.dv + col(part, i)] = i % 2 ? S[i / 2].y : S[i / 2].x;
}

// Joins the pieces, in place: H[p + 1] = e^{g over p} H[p] + its own, from h0, and
// G[p] = e^{g over p} G[p + 1] + its own, from dhT (back).
__global__ void __launch_bounds__(256) piece_scan_kernel(LinearArgs a, Pieces p, int first_z) {
  __shared__ float dec[256];
  const bool back = blockIdx.z + first_z == 1;
  const int n = blockIdx.x / a.H, h = blockIdx.x % a.H, b = a.cu_seqlens ? 0 : n;
  int t0, len;
  seq_range(a, n, t0, len);
  const int pieces = pieces_of(len, p.tokens);
  const size_t first = a.cu_seqlens ? (size_t)p.slot0[n]
                                    : (size_t)n * (pieces_of(a.T, p.tokens) + 1);
  const int states = a.dk * a.dv, e = blockIdx.y * 256 + threadIdx.x;
  const float* g = a.g_head ? a.g + h : a.g + ((size_t)b * a.H + h) * a.T + t0;
  const int gs = a.g_head ? 0 : 1;
  auto at = [&](int k) {  // slot k of this sequence
    return (min(first + k, p.slots - 1) * a.H + h) * (size_t)states + e;
  };
  float* S = back ? p.G : p.H;
  const float* from = back ? a.dhT : a.h0;
  const size_t st = ((size_t)n * a.H + h) * states + e;
  float s = from && e < states ? from[st] : 0.f;
  if (e < states) S[at(back ? pieces : 0)] = s;
  for (int k0 = 0; k0 < pieces; k0 += 256) {
    // the decays of up to 256 pieces, a warp a piece in turn
    __syncthreads();
    const int nk = min(256, pieces - k0);
    for (int k = threadIdx.x >> 5; k < nk; k += 8) {
      const int piece = back ? pieces - 1 - (k0 + k) : k0 + k, i0 = piece * p.tokens;
      double x = 0.0;
#pragma unroll 2
      for (int i = i0 + (threadIdx.x & 31); i < min(i0 + p.tokens, len); i += 32)
        x += (double)g[(size_t)i * gs];
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
      if ((threadIdx.x & 31) == 0) dec[k] = (float)exp(x);
    }
    __syncthreads();
    if (e < states) {
      for (int k = 0; k < nk; k += 8) {  // eight loads in flight
        float own[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          own[i] = k + i < nk ? S[at(back ? pieces - 1 - (k0 + k + i) : k0 + k + i + 1)] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < nk) {
            s = fmaf(dec[k + i], s, own[i]);
            S[at(back ? pieces - 1 - (k0 + k + i) : k0 + k + i + 1)] = s;
          }
      }
    }
  }
  if (e < states) {
    if (!back && a.hT) a.hT[st] = s;
    if (back && a.dh0) a.dh0[st] = s;
  }
}

// A run over the tokens of a piece (or, without tables, of a sequence).  R4:
// columns of a thread / 4 (so R <= 16 R4 contracted columns).
template <typename IO, typename OUT, int RUN, int R4>
__device__ __forceinline__ void run_piece(const LinearArgs& a, const Pieces& p, const Where& u,
                                          int slice, OUT* out, float* sm) {
  constexpr bool kBack = RUN == RUN_DK || RUN == RUN_DV;
  constexpr bool kOwnV = RUN == RUN_O || RUN == RUN_DV;   // rows are value columns
  constexpr bool kDecayed = RUN == RUN_DQ || RUN == RUN_DK;  // read before the write
  constexpr int kR = 16 * R4;
  float *sx = sm, *sz = sx + kTok * kR, *sy = sz + kTok * kR, *sa = sy + kTok * kOwn;

  const int own_n = kOwnV ? a.dv : a.dk, R = kOwnV ? a.dk : a.dv;
  const IO* q = static_cast<const IO*>(a.q) + u.krow * a.dk;
  const IO* k = static_cast<const IO*>(a.k) + u.krow * a.dk;
  const IO* v = static_cast<const IO*>(a.v) + u.vrow * a.dv;
  const IO* dout = static_cast<const IO*>(a.dout) + u.vrow * a.dv;
  const IO* X = RUN == RUN_O ? k : RUN == RUN_DQ ? v : RUN == RUN_DK ? dout : q;
  const IO* Y = RUN == RUN_O ? v : RUN == RUN_DQ ? k : RUN == RUN_DK ? q : dout;
  const IO* Z = RUN == RUN_O ? q : RUN == RUN_DQ ? dout : RUN == RUN_DK ? v : k;
  // where the query scale goes: on the readout of o and dq, into the state of dk and dv
  const float out_scale = kBack ? 1.f : a.scale, y_scale = kBack ? a.scale : 1.f;
  const float* g = a.g_head ? a.g + u.h : a.g + u.vrow;
  const int gs = a.g_head ? 0 : 1;

  const int own = threadIdx.x / kSplit, part = threadIdx.x % kSplit;
  const int c0 = slice * kOwn, c = c0 + own;
  const bool row = c < own_n;
  // element (row c, column r) of a [dk, dv] state
  auto at = [&](int r) { return kOwnV ? (size_t)r * a.dv + c : (size_t)c * a.dv + r; };

  F2 S[2 * R4];
  const size_t states = (size_t)a.dk * a.dv;
  const float* init;
  if (kBack)
    init = p.G + (min(u.slot + 1, p.slots - 1) * a.H + u.h) * states;
  else if (p.H)
    init = p.H + (u.slot * a.H + u.h) * states;
  else
    init = a.h0 ? a.h0 + ((size_t)u.n * a.H + u.h) * states : nullptr;
#pragma unroll
  for (int i = 0; i < 4 * R4; ++i)
    (i % 2 ? S[i / 2].y : S[i / 2].x) =
        init && row && col(part, i) < R ? init[at(col(part, i))] : 0.f;

  for (int s0 = 0; s0 < u.len; s0 += kTok) {
    const int nt = min(kTok, u.len - s0), t0 = kBack ? u.len - s0 - nt : s0;
    __syncthreads();
    stage<IO, kR>(sx, X + (size_t)t0 * R, R, 0, R, nt, kBack);
    stage<IO, kR>(sz, Z + (size_t)t0 * R, R, 0, R, nt, kBack);
    stage<IO, kOwn>(sy, Y + (size_t)t0 * own_n, own_n, c0, min(kOwn, own_n - c0), nt, kBack);
    if (threadIdx.x < kTok && (int)threadIdx.x < nt) {
      const int t = kBack ? t0 + nt - 1 - threadIdx.x : t0 + threadIdx.x;
      // backward, the decay from token t + 1 to t; none into the piece's last token
      sa[threadIdx.x] = kBack ? (t == u.len - 1 ? 1.f : expf(g[(size_t)(t + 1) * gs]))
                              : expf(g[(size_t)t * gs]);
    }
    staged();
#pragma unroll 2
    for (int tt = 0; tt < nt; ++tt) {
      const int t = kBack ? t0 + nt - 1 - tt : t0 + tt;
      const float dec = sa[tt], y = y_scale * sy[tt * kOwn + own];
      const float4* x = reinterpret_cast<const float4*>(sx + tt * kR) + part;
      const float4* z = reinterpret_cast<const float4*>(sz + tt * kR) + part;
      const F2 d2{dec, dec}, y2{y, y};
      F2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};  // four chains: the sum is the token's latency
#pragma unroll
      for (int i = 0; i < R4; ++i) {
        const float4 xv = x[kSplit * i], zv = z[kSplit * i];
        const F2 x2[2] = {{xv.x, xv.y}, {xv.z, xv.w}}, z2[2] = {{zv.x, zv.y}, {zv.z, zv.w}};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          F2& S2 = S[2 * i + e];
          if (kDecayed) {
            S2 = mul2(S2, d2);
            acc[e] = fma2(S2, z2[e], acc[e]);
            S2 = fma2(y2, x2[e], S2);
          } else {
            S2 = fma2(d2, S2, mul2(y2, x2[e]));
            acc[e] = fma2(S2, z2[e], acc[e]);
          }
        }
      }
      float s = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (part == 0 && row) st_io(out + (u.vrow + t) * own_n + c, out_scale * s);
    }
  }
  if (RUN == RUN_O && !p.H && a.hT && row) {
    float* to = a.hT + ((size_t)u.n * a.H + u.h) * states;
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i)
      if (col(part, i) < R) to[at(col(part, i))] = i % 2 ? S[i / 2].y : S[i / 2].x;
  }
}

template <typename IO, int R4>
__global__ void __launch_bounds__(kThreads) run_o_kernel(LinearArgs a, Pieces p) {
  extern __shared__ __align__(16) float sm[];
  Where u;
  if (!where(a, p, blockIdx.x, u)) return;
  // (uncut, an empty sequence still hands its state on)
  if (u.piece >= u.pieces && !(u.piece == 0 && !p.H)) return;
  if (u.len < 0) u.len = 0;
  run_piece<IO, IO, RUN_O, R4>(a, p, u, blockIdx.y, static_cast<IO*>(a.o), sm);
}

// dq and dk side by side as block z (they contract over dv), and dv.
template <typename IO, int R4>
__global__ void __launch_bounds__(kThreads) run_dqk_kernel(LinearArgs a, SerialWs w) {
  extern __shared__ __align__(16) float sm[];
  Where u;
  if (!where(a, w.p, blockIdx.x, u) || u.piece >= u.pieces) return;
  if (blockIdx.z == 0)
    run_piece<IO, float, RUN_DQ, R4>(a, w.p, u, blockIdx.y, w.dq, sm);
  else
    run_piece<IO, float, RUN_DK, R4>(a, w.p, u, blockIdx.y, w.dk, sm);
}
template <typename IO, int R4>
__global__ void __launch_bounds__(kThreads) run_dv_kernel(LinearArgs a, SerialWs w) {
  extern __shared__ __align__(16) float sm[];
  Where u;
  if (!where(a, w.p, blockIdx.x, u) || u.piece >= u.pieces) return;
  run_piece<IO, IO, RUN_DV, R4>(a, w.p, u, blockIdx.y, static_cast<IO*>(a.dval), sm);
}

// dg of one piece of one (sequence, head): <H, G> at its end by all 256 threads,
// the dot products of a token by four, then a thread a token sums a suffix.
template <typename IO>
__global__ void __launch_bounds__(256) piece_dg_kernel(LinearArgs a, SerialWs w, float* dg) {
  __shared__ float x[kCkptTokens], red[8];
  Where u;
  if (!where(a, w.p, blockIdx.x, u) || u.piece >= u.pieces) return;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, states = a.dk * a.dv;
  const size_t end = (min(u.slot + 1, w.p.slots - 1) * a.H + u.h) * (size_t)states;
  float s = 0.f;
#pragma unroll 4
  for (int i = threadIdx.x; i < states; i += 256) s = fmaf(w.p.H[end + i], w.p.G[end + i], s);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if (lane == 0) red[wid] = s;
  {  // four threads a token
    const int i = threadIdx.x >> 2, part = threadIdx.x & 3;
    float d = 0.f, own = 0.f;
    if (i < u.len) {
      const IO* q = static_cast<const IO*>(a.q) + (u.krow + i) * a.dk;
      const IO* k = static_cast<const IO*>(a.k) + (u.krow + i) * a.dk;
      const float* dq = w.dq + (u.vrow + i) * a.dk;
      const float* dk = w.dk + (u.vrow + i) * a.dk;
#pragma unroll 4
      for (int r = part; r < a.dk; r += 4)
        d += fmaf(ld_io(q + r), dq[r], -(ld_io(k + r) * dk[r]));
      const IO* v = static_cast<const IO*>(a.v) + (u.vrow + i) * a.dv;
      const IO* dout = static_cast<const IO*>(a.dout) + (u.vrow + i) * a.dv;
#pragma unroll 4
      for (int c = part; c < a.dv; c += 4) own = fmaf(ld_io(v + c), ld_io(dout + c), own);
    }
#pragma unroll
    for (int m = 2; m >= 1; m >>= 1) {
      d += __shfl_xor_sync(0xffffffffu, d, m);
      own += __shfl_xor_sync(0xffffffffu, own, m);
    }
    if (part == 0) {
      x[i] = d;
      if (i < u.len) w.own[u.vrow + i] = a.scale * own;
    }
  }
  __syncthreads();
  if (threadIdx.x < kCkptTokens && (int)threadIdx.x < u.len) {
    float t = 0.f;
    for (int i = 0; i < 8; ++i) t += red[i];
    for (int i = kCkptTokens - 1; i >= (int)threadIdx.x; --i) t += x[i];
    dg[u.vrow + threadIdx.x] = t;
  }
}

// One thread per element of dq and dk; `own` as in SerialWs.
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
      o += own[(head * group + i) * a.T + (e % per) / a.dk];
    }
    x = fmaf(o, ld_io(static_cast<const IO*>(a.k) + e), x);
    y = fmaf(o, ld_io(static_cast<const IO*>(a.q) + e), y);
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

// Bytes of shared memory of a run with R columns (a multiple of 16).
size_t run_smem(int kR) { return (size_t)(2 * kTok * kR + kTok * kOwn + kTok) * sizeof(float); }
size_t sum_smem(int kR) {
  return (size_t)(kTok * kR + kTok * kOwn + 2 * kTok + 1) * sizeof(float);
}

// Calls f with the columns of a thread / 4 that hold R columns, as a constant.
template <typename F>
cudaError_t with_columns(int R, F f) {
  switch ((R + 15) / 16) {
    case 1:
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    default: return f(std::integral_constant<int, 8>());
  }
}

size_t slots_of(int N, int T, int tokens, bool packed) {
  // packed: ceil(len / tokens) pieces of each sequence, and a final state
  return packed ? (size_t)T / tokens + 2 * (size_t)N : (size_t)N * (pieces_of(T, tokens) + 1);
}

// Tokens of a forward piece: 64 and up, so that 608 blocks (four an SM) have one;
// the whole sequence, with no pass before it, where the heads alone make half of
// that (cutting runs the state's update twice).
int fwd_piece(int N, int H, int T, int dv, bool packed) {
  const long long blocks = (long long)N * H * ((dv + kOwn - 1) / kOwn);
  if (blocks >= 2 * kLinSms || T <= 2 * kTok) return 0;
  const long long each = packed ? (long long)H * ((dv + kOwn - 1) / kOwn) : blocks;
  const long long want = (4 * kLinSms + each - 1) / each;  // pieces of the T axis
  const long long tokens = (T + want - 1) / want;
  return (int)((tokens + kTok - 1) / kTok * kTok);
}

// What each piece adds to the states, and the scan.  directions: 1 forward only.
template <typename IO, int R4>
cudaError_t launch_sum(const LinearArgs& a, const Pieces& p, int directions, cudaStream_t s) {
  const size_t smem = sum_smem(16 * R4);
  const cudaError_t e = allow_smem<piece_sum_kernel<IO, R4>>(smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(p.slots * a.H), (a.dk + kOwn - 1) / kOwn, directions);
  piece_sum_kernel<IO, R4><<<grid, kThreads, smem, s>>>(a, p, 0);
  return cudaGetLastError();
}
template <typename IO>
cudaError_t join_pieces(const LinearArgs& a, const Pieces& p, int directions, cudaStream_t s) {
  const cudaError_t e = with_columns(
      a.dv, [&](auto r4) { return launch_sum<IO, decltype(r4)::value>(a, p, directions, s); });
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.N * a.H, (a.dk * a.dv + 255) / 256, directions);
  piece_scan_kernel<<<grid, 256, 0, s>>>(a, p, 0);
  return cudaGetLastError();
}

template <typename IO, int R4>
cudaError_t launch_o(const LinearArgs& a, const Pieces& p, cudaStream_t s) {
  const size_t smem = run_smem(16 * R4);
  const cudaError_t e = allow_smem<run_o_kernel<IO, R4>>(smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(p.slots * a.H), (a.dv + kOwn - 1) / kOwn);
  run_o_kernel<IO, R4><<<grid, kThreads, smem, s>>>(a, p);
  return cudaGetLastError();
}

struct FwdPlan {
  int tokens;
  size_t slots, H, slot0, total;
};
FwdPlan fwd_plan(int N, int H, int T, int dk, int dv, bool packed) {
  FwdPlan p;
  const int cut = fwd_piece(N, H, T, dv, packed);
  p.tokens = cut ? cut : (T > 0 ? T : 1);
  p.slots = slots_of(N, T, p.tokens, packed);
  size_t at = 0;
  p.slot0 = at; at += up256(((size_t)N + 1) * 4);
  p.H = at; at += cut ? up256(p.slots * H * dk * dv * 4) : 0;
  p.total = at;
  return p;
}

template <typename IO>
cudaError_t serial_fwd_io(const LinearArgs& a, char* ws, cudaStream_t s) {
  const FwdPlan f = fwd_plan(a.N, a.H, a.T, a.dk, a.dv, a.cu_seqlens != nullptr);
  const bool cut = fwd_piece(a.N, a.H, a.T, a.dv, a.cu_seqlens != nullptr) != 0;
  Pieces p{};
  p.tokens = f.tokens;
  p.slots = f.slots;
  p.H = cut ? reinterpret_cast<float*>(ws + f.H) : nullptr;
  cudaError_t e = cudaSuccess;
  if (a.cu_seqlens) {
    int32_t* slot0 = reinterpret_cast<int32_t*>(ws + f.slot0);
    p.slot0 = slot0;
    slot_plan_kernel<<<1, 1024, 0, s>>>(a, p.tokens, slot0);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (cut && (e = join_pieces<IO>(a, p, 1, s)) != cudaSuccess) return e;
  return with_columns(a.dk, [&](auto r4) { return launch_o<IO, decltype(r4)::value>(a, p, s); });
}

struct SerialPlan {
  size_t slots, dq, dk, dg, own, H, G, slot0, total;
};
SerialPlan serial_plan(int N, int B, int H, int T, int dk, int dv, bool packed) {
  SerialPlan p;
  p.slots = slots_of(N, T, kCkptTokens, packed);
  const size_t states = p.slots * H * dk * dv * 4;
  const size_t rows = (size_t)B * H * T;
  size_t at = 0;
  p.dq = at; at += up256(rows * dk * 4);
  p.dk = at; at += up256(rows * dk * 4);
  p.dg = at; at += up256(rows * 4);
  p.own = at; at += up256(rows * 4);
  p.H = at; at += up256(states);
  p.G = at; at += up256(states);
  p.slot0 = at; at += up256(((size_t)N + 1) * 4);
  p.total = at;
  return p;
}

template <typename IO, int R4>
cudaError_t launch_dqk(const LinearArgs& a, const SerialWs& w, cudaStream_t s) {
  const size_t smem = run_smem(16 * R4);
  const cudaError_t e = allow_smem<run_dqk_kernel<IO, R4>>(smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(w.p.slots * a.H), (a.dk + kOwn - 1) / kOwn, 2);
  run_dqk_kernel<IO, R4><<<grid, kThreads, smem, s>>>(a, w);
  return cudaGetLastError();
}
template <typename IO, int R4>
cudaError_t launch_dv(const LinearArgs& a, const SerialWs& w, cudaStream_t s) {
  const size_t smem = run_smem(16 * R4);
  const cudaError_t e = allow_smem<run_dv_kernel<IO, R4>>(smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(w.p.slots * a.H), (a.dv + kOwn - 1) / kOwn);
  run_dv_kernel<IO, R4><<<grid, kThreads, smem, s>>>(a, w);
  return cudaGetLastError();
}

template <typename IO>
cudaError_t sum_heads(const LinearArgs& a, const SerialWs& w, cudaStream_t s) {
  const size_t total = (size_t)a.B * a.Hk * a.T * a.dk, blocks = (total + 255) / 256;
  const unsigned grid = (unsigned)(blocks < 32 * kLinSms ? blocks : 32 * kLinSms);
  sum_heads_kernel<IO><<<grid, 256, 0, s>>>(a, w.dq, w.dk, w.own);
  return cudaGetLastError();
}

template <typename IO>
cudaError_t serial_bwd_io(const LinearArgs& a, char* ws, cudaStream_t s) {
  const SerialPlan p = serial_plan(a.N, a.B, a.H, a.T, a.dk, a.dv, a.cu_seqlens != nullptr);
  SerialWs w{};
  w.dq = reinterpret_cast<float*>(ws + p.dq);
  w.dk = reinterpret_cast<float*>(ws + p.dk);
  w.dg = reinterpret_cast<float*>(ws + p.dg);
  w.own = reinterpret_cast<float*>(ws + p.own);
  w.p.tokens = kCkptTokens;
  w.p.slots = p.slots;
  w.p.H = reinterpret_cast<float*>(ws + p.H);
  w.p.G = reinterpret_cast<float*>(ws + p.G);
  cudaError_t e = cudaSuccess;
  if (a.cu_seqlens) {
    int32_t* slot0 = reinterpret_cast<int32_t*>(ws + p.slot0);
    w.p.slot0 = slot0;
    slot_plan_kernel<<<1, 1024, 0, s>>>(a, kCkptTokens, slot0);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = join_pieces<IO>(a, w.p, 2, s)) != cudaSuccess) return e;
  if (a.T > 0) {
    e = with_columns(a.dv, [&](auto r4) { return launch_dqk<IO, decltype(r4)::value>(a, w, s); });
    if (e == cudaSuccess)
      e = with_columns(a.dk, [&](auto r4) { return launch_dv<IO, decltype(r4)::value>(a, w, s); });
    if (e != cudaSuccess) return e;
    piece_dg_kernel<IO><<<(unsigned)(p.slots * a.H), 256, 0, s>>>(a, w, a.g_head ? w.dg : a.dg);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = sum_heads<IO>(a, w, s)) != cudaSuccess) return e;
  }
  return a.g_head ? linear_sum_decay(a, w.dg, s) : e;
}

}  // namespace

size_t linear_serial_fwd_bytes(int N, int H, int T, int dk, int dv, bool packed) {
  return fwd_plan(N, H, T, dk, dv, packed).total;
}

cudaError_t linear_serial_fwd(const LinearArgs& a, char* ws, cudaStream_t s) {
  return a.io == CKDA_F32 ? serial_fwd_io<float>(a, ws, s) : serial_fwd_io<__nv_bfloat16>(a, ws, s);
}

size_t linear_serial_bwd_bytes(int N, int B, int H, int T, int dk, int dv, bool packed) {
  return serial_plan(N, B, H, T, dk, dv, packed).total;
}

cudaError_t linear_serial_bwd(const LinearArgs& a, char* ws, cudaStream_t s) {
  return a.io == CKDA_F32 ? serial_bwd_io<float>(a, ws, s)
                          : serial_bwd_io<__nv_bfloat16>(a, ws, s);
}

cudaError_t linear_sum_decay(const LinearArgs& a, const float* dg_full, cudaStream_t s) {
  sum_decay_kernel<<<a.H, 1024, 0, s>>>(a, dg_full);
  return cudaGetLastError();
}

}  // namespace ckda
