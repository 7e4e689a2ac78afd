// ckda_linear_serial.cu -- linear attention with a scalar decay per head on CUDA
// cores: fp32 I/O, and widths the tensor-core kernels do not take.
//
// Up to 192 tokens run one by one in a single launch.  The state's rows (value
// columns) do not meet, so a block owns 32 of them and a (sequence, head) spreads
// over ceil(dv / 32) blocks; four threads share a row, each with every fourth group
// of four columns in registers.  Per token a thread does one fma for the update and
// one for the readout per column, on k and q from shared memory, 64 tokens of which
// are staged at a time: the bound is the latency of a token.
//
// Longer ones are cut into pieces of 64 tokens that run side by side, as matrix
// products: a first kernel sums each piece's own contribution to the state, a scan
// joins them, and then every piece starts from the state that enters it.  4 x 16
// heads x 2048 tokens of 128 channels in fp32: 568 us in a loop on one input (932 us token
// by token with the longest pieces that fill the SMs), 600 us on inputs that are not in
// L2; bound by FMA issue and shared-memory reads.  8 x 16 x 2048 of 100 channels in bf16,
// which the tensor-core kernels do not take: 1330 us.
#include "ckda_linear_piece.cuh"

namespace ckda {
namespace {

constexpr int kOwn = 32;     // state rows of a block, token by token
constexpr int kSplit = 4;    // threads of a row
constexpr int kThreads = kOwn * kSplit;

__global__ void slot_plan_kernel(LinearArgs a, int32_t* slot0) {
  after_previous();
  let_next_start();
  // one block; each thread adds up a run of sequences, then the runs are joined
  __shared__ int32_t sum[1024];
  const int per = (a.N + 1023) / 1024, i0 = threadIdx.x * per, i1 = min(i0 + per, a.N);
  int32_t s = 0;
  for (int i = i0; i < i1; ++i) {
    int t0, len;
    seq_range(a, i, t0, len);
    s += pieces_of(len) + 1;
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
    before += pieces_of(len) + 1;
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

// Stages `nt` tokens of `n` columns from `c0` on into [kTok][WIDTH], the rest
// zeros.  Four columns at a time where rows and base allow it (fp32 by cp.async,
// all at once in flight: staging one element a load took most of a piece's time).
template <typename IO, int WIDTH>
static __device__ __noinline__ void stage(float* dst, const IO* src, int stride, int c0, int n,
                                      int nt) {
  constexpr uintptr_t kMask = 4 * sizeof(IO) - 1;
  const bool four = ((stride | n) & 3) == 0 && (reinterpret_cast<uintptr_t>(src) & kMask) == 0;
  if (four) {
#pragma unroll 8
    for (int e = threadIdx.x; e < kTok * WIDTH / 4; e += kThreads) {
      const int t = e / (WIDTH / 4), c = 4 * (e % (WIDTH / 4));
      const bool in = t < nt && c < n;
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
    const int t = e / WIDTH, c = e % WIDTH;
    dst[e] = t < nt && c < n ? ld_io(src + (size_t)t * stride + c0 + c) : 0.f;
  }
}
// R4: columns of a thread / 4 (so dk <= 16 R4).
template <typename IO, int R4>
__global__ void __launch_bounds__(kThreads) run_kernel(LinearArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr int kR = 16 * R4;
  float *sx = sm, *sz = sx + kTok * kR, *sy = sz + kTok * kR, *sa = sy + kTok * kOwn;

  const int n = blockIdx.x / a.H, h = blockIdx.x % a.H, b = a.cu_seqlens ? 0 : n;
  int first, len;
  seq_range(a, n, first, len);
  const size_t krow = ((size_t)b * a.Hk + h / (a.H / a.Hk)) * a.T + first;
  const size_t vrow = ((size_t)b * a.H + h) * a.T + first;
  const IO* q = static_cast<const IO*>(a.q) + krow * a.dk;
  const IO* k = static_cast<const IO*>(a.k) + krow * a.dk;
  const IO* v = static_cast<const IO*>(a.v) + vrow * a.dv;
  IO* out = static_cast<IO*>(a.o) + vrow * a.dv;
  const float* g = a.g_head ? a.g + h : a.g + vrow;
  const int gs = a.g_head ? 0 : 1;

  const int own = threadIdx.x / kSplit, part = threadIdx.x % kSplit;
  const int c0 = blockIdx.y * kOwn, c = c0 + own;
  const bool row = c < a.dv;

  F2 S[2 * R4];
  const size_t states = (size_t)a.dk * a.dv;
  const float* init = a.h0 ? a.h0 + ((size_t)n * a.H + h) * states : nullptr;
#pragma unroll
  for (int i = 0; i < 4 * R4; ++i)
    (i % 2 ? S[i / 2].y : S[i / 2].x) =
        init && row && col(part, i) < a.dk ? init[(size_t)col(part, i) * a.dv + c] : 0.f;

  for (int t0 = 0; t0 < len; t0 += kTok) {
    const int nt = min(kTok, len - t0);
    __syncthreads();
    stage<IO, kR>(sx, k + (size_t)t0 * a.dk, a.dk, 0, a.dk, nt);
    stage<IO, kR>(sz, q + (size_t)t0 * a.dk, a.dk, 0, a.dk, nt);
    stage<IO, kOwn>(sy, v + (size_t)t0 * a.dv, a.dv, c0, min(kOwn, a.dv - c0), nt);
    if ((int)threadIdx.x < nt) sa[threadIdx.x] = expf(g[(size_t)(t0 + threadIdx.x) * gs]);
    copies_arrived();
#pragma unroll 2
    for (int t = 0; t < nt; ++t) {
      const float dec = sa[t], y = sy[t * kOwn + own];
      const float4* x = reinterpret_cast<const float4*>(sx + t * kR) + part;
      const float4* z = reinterpret_cast<const float4*>(sz + t * kR) + part;
      const F2 d2{dec, dec}, y2{y, y};
      F2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};  // four chains: the sum is the token's latency
#pragma unroll
      for (int i = 0; i < R4; ++i) {
        const float4 xv = x[kSplit * i], zv = z[kSplit * i];
        const F2 x2[2] = {{xv.x, xv.y}, {xv.z, xv.w}}, z2[2] = {{zv.x, zv.y}, {zv.z, zv.w}};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          F2& S2 = S[2 * i + e];
          S2 = fma2(d2, S2, mul2(y2, x2[e]));
          acc[e] = fma2(S2, z2[e], acc[e]);
        }
      }
      float s = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (part == 0 && row) st_io(out + (size_t)(t0 + t) * a.dv + c, a.scale * s);
    }
  }
  if (a.hT && row) {
    float* to = a.hT + ((size_t)n * a.H + h) * states;
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i)
      if (col(part, i) < a.dk) to[(size_t)col(part, i) * a.dv + c] = i % 2 ? S[i / 2].y : S[i / 2].x;
  }
}

// A piece's own contribution to the state after it (block z = 0: over k and v,
// into the slot behind it) or to the gradient of the state before it (z = 1:
// over q and do, into its own slot), 64 rows a block.  Threads as in the pieces'
// other products; CV: value channels / 16.
template <typename IO, int CV>
__global__ void __launch_bounds__(kPieceThreads) piece_sum_kernel(LinearArgs a, Pieces p) {
  after_previous();
  let_next_start();
  const int sv = row_floats(a.dv);
  extern __shared__ __align__(16) float sm[];
  float *sx = sm, *sy = sx + kTok * sv, *sg = sy + kTok * kPS, *sw = sg + kTok;
  Where u;
  if (!where(a, p, blockIdx.x, u) || u.piece >= u.pieces) return;
  const bool back = blockIdx.z == 1;
  const IO* X = static_cast<const IO*>(back ? a.dout : a.v) + u.vrow * a.dv;
  const IO* Y = static_cast<const IO*>(back ? a.q : a.k) + u.krow * a.dk;
  const int tid = threadIdx.x, nt = u.len, r0 = blockIdx.y * 64, row = 4 * (tid >> 4), c = tid & 15;
  stage_rows(sx, sv, X, a.dv, a.dv, nt, kTok, sv - 4);
  stage_rows(sy, kPS, Y + r0, a.dk, min(64, a.dk - r0), nt, kTok, 64);
  if (tid < kTok) sg[tid] = tid < nt ? (a.g_head ? a.g[u.h] : a.g[u.vrow + tid]) : 0.f;
  __syncthreads();
  if (tid < 32) {
    // lane l has tokens 2 l and 2 l + 1; forward the decay by what follows a
    // token, backward by what leads to it and itself
    const float g0 = sg[2 * tid], g1 = sg[2 * tid + 1];
    float run = g0 + g1;  // over the lanes up to (from) this one
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const float y = back ? __shfl_up_sync(0xffffffffu, run, m) : __shfl_down_sync(0xffffffffu, run, m);
      if (back ? tid >= m : tid + m < 32) run += y;
    }
    if (tid == 0 && !back && blockIdx.y == 0) p.dec[u.slot * a.H + u.h] = expf(run);
    // over the others: shifted, not subtracted
    float other = back ? __shfl_up_sync(0xffffffffu, run, 1) : __shfl_down_sync(0xffffffffu, run, 1);
    if (tid == (back ? 0 : 31)) other = 0.f;
    sw[2 * tid] = back ? a.scale * expf(other + g0) : expf(other + g1);
    sw[2 * tid + 1] = back ? a.scale * expf(other + g0 + g1) : expf(other);
  }
  copies_arrived();
  for (int e = tid; e < kTok * 64; e += kPieceThreads) sy[e / 64 * kPS + e % 64] *= sw[e / 64];
  __syncthreads();
  if (r0 + row >= a.dk) return;
  float acc[4][CV] = {};
  add_nn<true>(acc, sy + row, kPS, sx + c, sv, 0, (nt + 3) & ~3);
  const size_t slot = min(u.slot + (back ? 0 : 1), p.slots - 1);
  float* out = (back ? p.G : p.H) + (slot * a.H + u.h) * (size_t)a.dk * a.dv;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < CV; ++j)
      if (r0 + row + i < a.dk && c + 16 * j < a.dv)
        out[(size_t)(r0 + row + i) * a.dv + c + 16 * j] = acc[i][j];
}

// Joins the pieces, in place: H[p + 1] = e^{g over p} H[p] + its own, from h0, and
// G[p] = e^{g over p} G[p + 1] + its own, from dhT (back).
__global__ void __launch_bounds__(256) piece_scan_kernel(LinearArgs a, Pieces p) {
  after_previous();
  let_next_start();
  const bool back = blockIdx.z == 1;
  const int n = blockIdx.x / a.H, h = blockIdx.x % a.H;
  int t0, len;
  seq_range(a, n, t0, len);
  const int pieces = pieces_of(len);
  const size_t first = a.cu_seqlens ? (size_t)p.slot0[n]
                                    : (size_t)n * (pieces_of(a.T) + 1);
  const int states = a.dk * a.dv, e = blockIdx.y * 256 + threadIdx.x;
  if (e >= states) return;
  auto slot = [&](int k) { return min(first + k, p.slots - 1) * a.H + h; };
  float* S = (back ? p.G : p.H) + e;
  const float* from = back ? a.dhT : a.h0;
  const size_t st = ((size_t)n * a.H + h) * states + e;
  float s = from ? from[st] : 0.f;
  S[slot(back ? pieces : 0) * states] = s;
  for (int k0 = 0; k0 < pieces; k0 += 16) {  // sixteen loads in flight
    float own[16], dec[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = back ? pieces - 1 - (k0 + i) : k0 + i;
      const bool in = k0 + i < pieces;
      own[i] = in ? S[slot(back ? k : k + 1) * states] : 0.f;
      dec[i] = in ? p.dec[slot(k)] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = back ? pieces - 1 - (k0 + i) : k0 + i;
      if (k0 + i < pieces) {
        s = fmaf(dec[i], s, own[i]);
        S[slot(back ? k : k + 1) * states] = s;
      }
    }
  }
  if (!back && a.hT) a.hT[st] = s;
  if (back && a.dh0) a.dh0[st] = s;
}

// The outputs of a piece: o_i = scale e_i H^T q_i + sum_{j <= i} A_ij v_j.
size_t out_smem(int CK, int slabs, int dv) {
  return (size_t)(2 * kTok * (16 * CK * slabs + 4) + (kTok + 16 * CK) * row_floats(dv) +
                  kTok * kPS + 3 * kTok) * sizeof(float);
}
template <typename IO, int CK, int CV>
__global__ void __launch_bounds__(kPieceThreads, 2) piece_out_kernel(LinearArgs a, Pieces p) {
  after_previous();
  let_next_start();
  extern __shared__ __align__(16) float sm[];
  Where u;
  if (!where(a, p, blockIdx.x, u) || u.piece >= u.pieces) return;
  const int slabs = (a.dk + 16 * CK - 1) / (16 * CK), cols = 16 * CK * slabs;
  const int sk = cols + 4, nt = u.len, tid = threadIdx.x;
  const int sv = row_floats(a.dv);
  float *sq = sm, *skey = sq + kTok * sk, *sval = skey + kTok * sk, *slab = sval + kTok * sv,
        *sp = slab + 16 * CK * sv, *sg = sp + kTok * kPS, *se = sg + kTok, *sw = se + kTok;
  const int c = tid & 15, row = 4 * (tid >> 4);
  const float* H = p.H + (u.slot * a.H + u.h) * (size_t)a.dk * a.dv;
  auto stage_slab = [&](int s) {
    stage_rows(slab, sv, H + (size_t)16 * CK * s * a.dv, a.dv, a.dv,
               min(16 * CK, a.dk - 16 * CK * s), 16 * CK, sv - 4);
  };
  stage_rows(sq, sk, static_cast<const IO*>(a.q) + u.krow * a.dk, a.dk, a.dk, nt, kTok, cols);
  stage_rows(skey, sk, static_cast<const IO*>(a.k) + u.krow * a.dk, a.dk, a.dk, nt, kTok, cols);
  stage_rows(sval, sv, static_cast<const IO*>(a.v) + u.vrow * a.dv, a.dv, a.dv, nt, kTok, sv - 4);
  stage_slab(0);
  if (tid < kTok) sg[tid] = tid < nt ? (a.g_head ? a.g[u.h] : a.g[u.vrow + tid]) : 0.f;
  __syncthreads();
  piece_decays(sp, se, sw, sg, nt);
  copies_arrived();

  {
    float b[4][4] = {};
    add_nt(b, sq + row * sk, sk, skey + c * sk, sk, (a.dk + 3) & ~3);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = (row + i) * kPS + c + 16 * j;
        sp[at] = row + i >= c + 16 * j ? expf(sp[at]) * b[i][j] : 0.f;
      }
  }
  float acc[4][CV] = {};
#pragma unroll 1
  for (int s = 0; s < slabs; ++s) {
    add_nn<false>(acc, sq + row * sk + 16 * CK * s, sk, slab + c, sv, 0,
                         (min(16 * CK, a.dk - 16 * CK * s) + 3) & ~3);
    __syncthreads();
    if (s + 1 < slabs) {
      stage_slab(s + 1);
      copies_arrived();
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < CV; ++j) acc[i][j] *= se[row + i];
  add_nn<false>(acc, sp + row * kPS, kPS, sval + c, sv, 0, row);
  add_diag<false, true>(acc, sp + row * kPS, kPS, sval + c, sv, row);
  IO* o = static_cast<IO*>(a.o);
#pragma unroll
  for (int j = 0; j < CV; ++j)
    if (c + 16 * j < a.dv)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row + i < nt) st_io(o + (u.vrow + row + i) * a.dv + c + 16 * j, a.scale * acc[i][j]);
}

// Bytes of shared memory of a run with R columns (a multiple of 16).
size_t run_smem(int kR) { return (size_t)(2 * kTok * kR + kTok * kOwn + kTok) * sizeof(float); }

// Tokens one by one, in one launch, up to three pieces of them: two more launches and
// the pieces' states cost more than the latency of 192 tokens.  One by one against
// pieces, fp32, 16 heads of 128 channels: 34 and 51 us for 128 tokens, 48 and 54 for
// 192, 62 and 53 for 256.  (Packed input counts all its tokens: any one sequence may
// have most of them.)
bool in_pieces(int T) { return T > 3 * kTok; }

size_t sum_smem(int dv) {
  return (size_t)(kTok * row_floats(dv) + kTok * kPS + 2 * kTok) * sizeof(float);
}
template <typename IO>
cudaError_t sum_pieces(const LinearArgs& a, const Pieces& p, int directions, cudaStream_t s) {
  return with_columns(a.dv, [&](auto cv) {
    constexpr int CV = decltype(cv)::value;
    const cudaError_t e = allow_smem<piece_sum_kernel<IO, CV>>(sum_smem(16 * CV));
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(p.slots * a.H), (a.dk + 63) / 64, directions);
    return launch_next(a.cu_seqlens, piece_sum_kernel<IO, CV>, grid, kPieceThreads, sum_smem(a.dv),
                       s, a, p);
  });
}

struct FwdPlan {
  size_t slots, H, dec, slot0, total;
};
FwdPlan fwd_plan(int N, int H, int T, int dk, int dv, bool packed) {
  FwdPlan p{};
  if (!in_pieces(T)) return p;
  p.slots = slots_of(N, T, packed);
  size_t at = 0;
  p.slot0 = at; at += up256(((size_t)N + 1) * 4);
  p.H = at; at += up256(p.slots * H * dk * dv * 4);
  p.dec = at; at += up256(p.slots * H * 4);
  p.total = at;
  return p;
}

template <typename IO>
cudaError_t serial_fwd_io(const LinearArgs& a, char* ws, cudaStream_t s) {
  if (!in_pieces(a.T))
    return with_columns(a.dk, [&](auto r4) {
      constexpr int R4 = decltype(r4)::value;
      const size_t smem = run_smem(16 * R4);
      const cudaError_t e = allow_smem<run_kernel<IO, R4>>(smem);
      if (e != cudaSuccess) return e;
      run_kernel<IO, R4><<<dim3((unsigned)a.N * a.H, (a.dv + kOwn - 1) / kOwn), kThreads, smem, s>>>(a);
      return cudaGetLastError();
    });
  const FwdPlan f = fwd_plan(a.N, a.H, a.T, a.dk, a.dv, a.cu_seqlens != nullptr);
  Pieces p{};
  p.slots = f.slots;
  p.H = reinterpret_cast<float*>(ws + f.H);
  p.dec = reinterpret_cast<float*>(ws + f.dec);
  cudaError_t e = cudaSuccess;
  if (a.cu_seqlens) {
    int32_t* slot0 = reinterpret_cast<int32_t*>(ws + f.slot0);
    p.slot0 = slot0;
    if ((e = linear_plan_slots(a, slot0, s)) != cudaSuccess) return e;
  }
  if ((e = linear_join_pieces(a, p, 1, s)) != cudaSuccess) return e;
  return with_columns(a.dv, [&](auto cv) {
    return with_slab(a.dk, [&](auto ck) {
      constexpr int CK = decltype(ck)::value, CV = decltype(cv)::value;
      const size_t smem = out_smem(CK, (a.dk + 16 * CK - 1) / (16 * CK), a.dv);
      const cudaError_t e =
          allow_smem<piece_out_kernel<IO, CK, CV>>(out_smem(CK, kMostSlabs<CK>, 16 * CV));
      if (e != cudaSuccess) return e;
      return launch_next(true, piece_out_kernel<IO, CK, CV>, (unsigned)(p.slots * a.H),
                         kPieceThreads, smem, s, a, p);
    });
  });
}

}  // namespace

cudaError_t linear_plan_slots(const LinearArgs& a, int32_t* slot0, cudaStream_t s) {
  slot_plan_kernel<<<1, 1024, 0, s>>>(a, slot0);
  return cudaGetLastError();
}

cudaError_t linear_join_pieces(const LinearArgs& a, const Pieces& p, int directions,
                               cudaStream_t s) {
  const cudaError_t e = a.io == CKDA_F32 ? sum_pieces<float>(a, p, directions, s)
                                         : sum_pieces<__nv_bfloat16>(a, p, directions, s);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.N * a.H, (a.dk * a.dv + 255) / 256, directions);
  return launch_next(true, piece_scan_kernel, grid, 256, 0, s, a, p);
}

size_t linear_serial_fwd_bytes(int N, int H, int T, int dk, int dv, bool packed) {
  return fwd_plan(N, H, T, dk, dv, packed).total;
}

cudaError_t linear_serial_fwd(const LinearArgs& a, char* ws, cudaStream_t s) {
  return a.io == CKDA_F32 ? serial_fwd_io<float>(a, ws, s) : serial_fwd_io<__nv_bfloat16>(a, ws, s);
}

}  // namespace ckda
