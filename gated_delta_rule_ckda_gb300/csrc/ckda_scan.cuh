// ckda_scan.cuh -- what the kernels of the selective scan share.
//
// Per channel d with N states, over the tokens of a sequence:
//     delta_t = softplus(dt_t + dt_bias)   (or without the softplus)
//     h_t[n]  = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n]
//     y_t     = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)
//
// Tokens are rows of D channels; B and C are rows of G groups of N, shared by the D / G
// channels of a group.  A warp works by itself, with no barrier of its block: it takes 32
// channels of one group, one to a lane, and walks a piece of one row's tokens in tiles.  A
// lane forms the steps of its own channel and finishes its outputs; the states of LP
// channels are spread over their LP lanes, NS of each channel to a lane, so that a lane
// reads only NS of a token's B and C for its N states: shared memory moves 32 lanes' worth
// even where lanes read the same, and would bound a lane that read all N.  Steps go round
// the LP lanes by shuffles, and so do the parts of the sums over n, each to its own lane.
// Sequence borders (dense rows' ends, packed sequences) are found by ballots in tiles that
// hold one; other tiles run without the checks.
#pragma once
#include <type_traits>
#include "ckda_launch.cuh"
#include "ckda_rows.cuh"

namespace ckda {

// Warps of a block, which do not meet: one or two instead leave 8 x 2048 tokens of 4096
// channels of 16 states at 425 and 418 us for 417.
constexpr int kScanWarps = 4;
constexpr int kScanBlock = 32 * kScanWarps;
constexpr int kScanChunk = 4;  // tokens between the states that the backward pass keeps
constexpr int kScanMostStates = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct ScanArgs {
  const void* x;
  const void* dt;
  const void* B;
  const void* C;
  const void* z;
  const float* A;        // [D][N]
  const float* skip;     // D, [D]
  const float* dt_bias;  // [D]
  const float* h0;       // [seqs][D][N]
  void* y;
  float* hT;
  const int32_t* cu;
  long long ldx, lddt, ldb, ldc, ldz;  // elements from one token to the next
  int rows, T, D, N, G, seqs;
  int softplus;
  int fill;               // rows of y behind the last sequence become zero
  int pieces, piece_len;  // of a row
  int chan_blocks;        // of all channels; per group chan_blocks / G
  float* state;           // [rows][pieces][D][N]: what a piece adds, then what enters it
  float* span;            // [rows][pieces][D]: sum of a piece's steps
  // backward pass
  const void* dy;
  const float* dhT;
  float* chunk;      // [rows][chunks][D][N]: states before chunks, from the piece's own start
  float* chunk_sum;  // [rows][chunks][D]: steps from the piece's start to the chunk (pieces > 1)
  float* grad;       // [rows][pieces][D][N]: what a piece adds to G, then the G that reaches its end
  int chunks;        // of a row
};

// ------------------------------------------------------------------ arithmetic
__device__ __forceinline__ float ex2(float a) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(a));
  return d;
}
__device__ __forceinline__ float2 ex2(float2 a) { return make_float2(ex2(a.x), ex2(a.y)); }
__device__ __forceinline__ float rcp(float a) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(a));
  return d;
}
__device__ __forceinline__ float2 rcp(float2 a) { return make_float2(rcp(a.x), rcp(a.y)); }
// exp(delta A) from A log2(e).  ex2.approx comes out low on average, by 1.4e-8 to 2.7e-8 of
// the value for arguments of 2^-8 to 2^0 and by 5e-9 to 9e-9 for smaller ones (it is exact
// at 0, with the addend too): nothing for one decay, but a state of a memory of 2^-o tokens
// is behind the product of as many.  The addend, which costs nothing, leaves 2e-8 low
// around 2^-7, where memories are short, and 3e-9 high to 2e-9 low below 2^-9: within 6e-6
// over memories of up to 2048 tokens, 9e-6 over 4096.  (No addend: 5.4e-5 over 8192 and
// 1e-4 over 16,384; 2.5e-8, which suits short memories best, 8.8e-5 and 1.8e-4.)
constexpr float kEx2Bias = 1.15e-8f;
__device__ __forceinline__ float2 decay_of(float2 delta, float2 A2) {
  return ex2(fma_(delta, A2, both<float2>(kEx2Bias)));
}
__device__ __forceinline__ float2 scan_sigmoid(float2 p) {
  return rcp(add_(ex2(mul_(p, both<float2>(-kLog2e))), both<float2>(1.f)));
}
__device__ __forceinline__ float scan_sigmoid(float p) { return rcp(1.f + ex2(-kLog2e * p)); }
__device__ __forceinline__ float2 scan_silu(float2 p) { return mul_(p, scan_sigmoid(p)); }
__device__ __forceinline__ float scan_silu(float p) { return p * scan_sigmoid(p); }
// log(1 + e^x) = max(x, 0) + log1p(e^-|x|), and log1p(t) = 2 atanh(t / (2 + t)) by its
// power series: t <= 1 makes the argument at most 1/3, and seven terms leave 2e-8.
// Small steps (x well below 0) keep their relative precision.
__device__ __forceinline__ float2 softplus(float2 x) {
  const float2 t = ex2(mul_(make_float2(fabsf(x.x), fabsf(x.y)), both<float2>(-kLog2e)));
  const float2 s = mul_(t, rcp(add_(t, both<float2>(2.f)))), q = mul_(s, s);
  float2 p = fma_(q, both<float2>(2.f / 13.f), both<float2>(2.f / 11.f));
  p = fma_(q, p, both<float2>(2.f / 9.f));
  p = fma_(q, p, both<float2>(2.f / 7.f));
  p = fma_(q, p, both<float2>(2.f / 5.f));
  p = fma_(q, p, both<float2>(2.f / 3.f));
  p = fma_(q, p, both<float2>(2.f));
  return fma_(s, p, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}
__device__ __forceinline__ float softplus(float x) { return softplus(make_float2(x, x)).x; }

// Sums over LANES lanes, STRIDE apart, of NV values: lane i of them gets the sums of
// values i r to i r + r - 1 in v[0] to v[r - 1], r = NV / LANES; with more lanes than
// values, lane i that of value i % NV.
template <int NV, int LANES, int STRIDE>
__device__ __forceinline__ void fold_values(float (&v)[NV], int i) {
  constexpr int kBoth = NV < LANES ? NV : LANES;
#pragma unroll
  for (int b = kBoth / 2; b >= 1; b /= 2) {
    const int s = b * (NV / kBoth);
    const bool up = (i & b) != 0;
#pragma unroll
    for (int j = 0; j < s; ++j) {
      const float send = up ? v[j] : v[j + s], keep = up ? v[j + s] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, b * STRIDE);
    }
  }
#pragma unroll
  for (int b = kBoth; b < LANES; b *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], b * STRIDE);
}

// ------------------------------------------------------------------- sequences
// Tokens [begin, end) of a row.  Offsets that are out of order or out of range leave
// every access inside the tensors.
struct ScanSeq {
  int n, begin, end;
};
__device__ __forceinline__ int scan_offset(const ScanArgs& a, int n) {
  const int o = a.cu[n];
  return o < 0 ? 0 : o > a.T ? a.T : o;
}
__device__ __forceinline__ ScanSeq scan_seq_at(const ScanArgs& a, int row, int t) {
  if (!a.cu) return {row, 0, a.T};
  int lo = 0, hi = a.seqs;  // the last n with cu[n] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= t) lo = mid; else hi = mid;
  }
  return {lo, scan_offset(a, lo), scan_offset(a, lo + 1)};
}
__device__ __forceinline__ int scan_last(const ScanArgs& a) { return a.cu ? scan_offset(a, a.seqs) : a.T; }
// What enters a piece reaches its end: no sequence starts inside.
__device__ __forceinline__ bool passes(const ScanArgs& a, int row, int t0, int t1) {
  return scan_seq_at(a, row, t1 - 1).begin < t0;
}

// ------------------------------------------------------------------------ tiles
constexpr int kScanChans = 32;  // of a warp

// LP lanes share LP channels' states, NS of each to a lane.
template <int LP, int NS>
struct ScanShape {
  static constexpr int kLanes = LP, kStates = NS, NP = LP * NS;
};

// A tile's inputs of a warp's channels, raw: [K][32] of each tensor, and [K][N] of B and
// C, padded to NP.  VEC: in whole vectors.  They come with cp.async, but for single bf16
// elements, which it does not copy: those are held in registers on their way.
template <typename IO, bool VEC>
constexpr bool kScanAsync = VEC || sizeof(IO) == 4;

template <typename IO, int K>
struct ChanTile {
  IO v[K][kScanChans];
  template <bool VEC>
  __device__ __forceinline__ void fetch(const void* base, long long ld, long long at, int c0, int count, int chans) {
    const int lane = threadIdx.x & 31;
    const IO* from = static_cast<const IO*>(base) + at * ld + c0;
    if constexpr (VEC) {
      constexpr int kV = 16 / sizeof(IO), kPer = kScanChans / kV;  // vectors of a token
      const int c = lane % kPer * kV, k0 = lane / kPer;
      const IO* p = from + k0 * ld + c;
#pragma unroll
      for (int k = 0; k < K; k += 32 / kPer, p += 32 / kPer * ld)
        if (k + k0 < count && c < chans) copy_async<16>(&v[k + k0][c], p);
    } else if constexpr (sizeof(IO) == 4) {
      from += lane;
#pragma unroll
      for (int k = 0; k < K; ++k, from += ld)
        if (k < count && lane < chans) copy_async<4>(&v[k][lane], from);
    }
  }
  __device__ __forceinline__ float2 pair(int k) const {
    const int lane = threadIdx.x & 31;
    return make_float2(ld_io(&v[k][lane]), ld_io(&v[k + 1][lane]));
  }
};
template <typename IO, int K, int NP>
struct GroupTile {
  alignas(16) IO v[K * NP];
  template <bool VEC>
  __device__ __forceinline__ void fetch(const void* base, long long ld, long long at, int count, int g, int N) {
    const int lane = threadIdx.x & 31;
    const IO* from = static_cast<const IO*>(base) + at * ld + (long long)g * N;
    if constexpr (VEC) {  // (N a multiple of 4)
#pragma unroll
      for (int j = 0; j < (K * NP / 4 + 31) / 32; ++j) {
        const int i = (j * 32 + lane) * 4, k = i / NP, n = i % NP;
        if (k < count && n < N) copy_async<4 * sizeof(IO)>(&v[i], from + k * ld + n);
      }
    } else if constexpr (sizeof(IO) == 4) {
#pragma unroll
      for (int j = 0; j < K * NP / 32; ++j) {
        const int i = j * 32 + lane, k = i / NP, n = i % NP;
        if (k < count && n < N) copy_async<4>(&v[i], from + k * ld + n);
      }
    }
  }
  // To fp32, zero where there is no token or no state.
  template <bool VEC>
  __device__ __forceinline__ void unpack_to(float* to, int count, int N) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < (K * NP / 4 + 31) / 32; ++j) {
      const int i = (j * 32 + lane) * 4, k = i / NP, n = i % NP;
      if (K * NP % 128 != 0 && i >= K * NP) break;
      float f[4];
      unpack<IO, 4>(*reinterpret_cast<const Pack<IO, 4>*>(&v[i]), f);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (k >= count || n + (VEC ? 0 : e) >= N) f[e] = 0.f;
      *reinterpret_cast<float4*>(to + i) = make_float4(f[0], f[1], f[2], f[3]);
    }
  }
};
// A tile's elements in registers: load() starts the loads, leave() puts them down.
template <typename IO, int K>
struct HeldChans {
  IO v[K];
  __device__ __forceinline__ void load(const void* base, long long ld, long long at, int c0, int count, int chans) {
    const int lane = threadIdx.x & 31;
    const IO* from = static_cast<const IO*>(base) + at * ld + c0 + lane;
#pragma unroll
    for (int k = 0; k < K; ++k, from += ld)
      if (k < count && lane < chans) v[k] = *from;
  }
  __device__ __forceinline__ void leave(ChanTile<IO, K>& to) const {
#pragma unroll
    for (int k = 0; k < K; ++k) to.v[k][threadIdx.x & 31] = v[k];
  }
};
template <typename IO, int K, int NP>
struct HeldGroups {
  IO v[K * NP / 32];
  __device__ __forceinline__ void load(const void* base, long long ld, long long at, int count, int g, int N) {
    const IO* from = static_cast<const IO*>(base) + at * ld + (long long)g * N;
#pragma unroll
    for (int j = 0; j < K * NP / 32; ++j) {
      const int i = j * 32 + (threadIdx.x & 31), k = i / NP, n = i % NP;
      if (k < count && n < N) v[j] = from[k * ld + n];
    }
  }
  __device__ __forceinline__ void leave(GroupTile<IO, K, NP>& to) const {
#pragma unroll
    for (int j = 0; j < K * NP / 32; ++j) to.v[j * 32 + (threadIdx.x & 31)] = v[j];
  }
};

// Marks of a tile's tokens: bit k of `first` where a sequence starts at token k, of `last`
// where one ends there; lane k has the sequence's number.  Warp-wide.
struct Marks {
  unsigned first, last;
  int n;
  __device__ __forceinline__ void find(const ScanArgs& a, int row, int t, int count) {
    const int k = threadIdx.x & 31;
    ScanSeq s{0, -1, -1};
    if (k < count) s = scan_seq_at(a, row, t + k);
    first = __ballot_sync(0xffffffffu, k < count && t + k == s.begin);
    last = __ballot_sync(0xffffffffu, k < count && t + k + 1 == s.end);
    n = s.n;
  }
  __device__ __forceinline__ int number(int k) const { return __shfl_sync(0xffffffffu, n, k); }
};

// A lane's NS states of one channel, as pairs.
template <int NS>
__device__ __forceinline__ void load_states(float2 (&h)[NS / 2], const float* base, long long chan, int N,
                                            int n0, bool in) {
  const float* p = base + chan * N;
#pragma unroll
  for (int i = 0; i < NS / 2; ++i) {
    h[i].x = in && n0 + 2 * i < N ? p[n0 + 2 * i] : 0.f;
    h[i].y = in && n0 + 2 * i + 1 < N ? p[n0 + 2 * i + 1] : 0.f;
  }
}
template <int NS>
__device__ __forceinline__ void store_states(float* base, long long chan, int N, int n0, bool in,
                                             const float2 (&h)[NS / 2]) {
  if (!in) return;
  float* p = base + chan * N;
  if (NS % 4 == 0 && N % 4 == 0 && (reinterpret_cast<uintptr_t>(base) & 15) == 0) {
#pragma unroll
    for (int i = 0; i < NS / 4; ++i)
      if (n0 + 4 * i < N)
        *reinterpret_cast<float4*>(p + n0 + 4 * i) =
            make_float4(h[2 * i].x, h[2 * i].y, h[2 * i + 1].x, h[2 * i + 1].y);
    return;
  }
#pragma unroll
  for (int i = 0; i < NS / 2; ++i) {
    if (n0 + 2 * i < N) p[n0 + 2 * i] = h[i].x;
    if (n0 + 2 * i + 1 < N) p[n0 + 2 * i + 1] = h[i].y;
  }
}
template <int NS>
__device__ __forceinline__ void from_shared(float2 (&f)[NS / 2], const float* p) {
#pragma unroll
  for (int i = 0; i < NS / 4; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
    f[2 * i] = make_float2(v.x, v.y);
    f[2 * i + 1] = make_float2(v.z, v.w);
  }
}

// Where a warp works: 32 channels of a group from c0, a piece of a row.
struct ScanPlace {
  int row, piece, g, c0, chans;  // chans: that exist
  int t0, t1;
  int block;  // of the group's channels
};
__device__ __forceinline__ bool scan_place(const ScanArgs& a, ScanPlace& p) {
  const long long id = (long long)blockIdx.x * kScanWarps + (threadIdx.x >> 5);
  const int cb = (int)(id % a.chan_blocks);
  const long long unit = id / a.chan_blocks;
  if (unit >= (long long)a.rows * a.pieces) return false;
  p.row = (int)(unit / a.pieces);
  p.piece = (int)(unit % a.pieces);
  const int per = a.chan_blocks / a.G, dg = a.D / a.G;
  p.g = cb / per;
  p.block = cb % per;
  const int first = p.block * kScanChans;
  p.c0 = p.g * dg + first;
  p.chans = dg - first < kScanChans ? dg - first : kScanChans;
  const int last = scan_last(a);
  p.t0 = p.piece * a.piece_len;
  p.t1 = p.t0 + a.piece_len < last ? p.t0 + a.piece_len : last;
  return true;
}
// A warp's part of a [rows][T][D] tensor behind the last sequence: zero.  (What nothing
// writes could be anything, and a NaN there reaches every weight of a layer that takes all
// rows.)
template <typename IO>
__device__ __forceinline__ void zero_behind(const ScanArgs& a, const ScanPlace& p, void* out) {
  const int lane = threadIdx.x & 31;
  const int end = p.t0 + a.piece_len < a.T ? p.t0 + a.piece_len : a.T;
  if (lane < p.chans)
    for (int t = p.t0 > p.t1 ? p.t0 : p.t1; t < end; ++t)
      st_io(static_cast<IO*>(out) + ((long long)p.row * a.T + t) * a.D + p.c0 + lane, 0.f);
}
inline int scan_chan_blocks(int D, int G) { return G * ((D / G + kScanChans - 1) / kScanChans); }
inline unsigned scan_grid(const ScanArgs& a) {
  return (unsigned)(((long long)a.rows * a.pieces * a.chan_blocks + kScanWarps - 1) / kScanWarps);
}

// delta of two channels.
__device__ __forceinline__ float2 step_sizes(float2 dt, float2 bias, int softplus_on) {
  const float2 raw = add_(dt, bias);
  return softplus_on ? softplus(raw) : raw;
}

// States that enter the pieces, from what each adds (ckda_scan_fwd.cu).
cudaError_t launch_scan_join(bool next, const ScanArgs& a, cudaStream_t s);
// Pieces of a row: one where `room` warps have no room for `fewest` or it has no more than
// `whole` tokens; else as many as it has room for, of about `least` tokens or more, in whole
// tiles (in multiples of 64 the batch's gradients took 1235 us for 1194, the documents 555
// for 543).
void scan_pieces(int rows, int T, int D, int G, int room, int fewest, int least, int whole, int* pieces, int* len);

// Empty sequences hand their states on: a warp copies its channels' part of `from` (zero
// if null) to `to`.
__device__ __forceinline__ void empty_states(const ScanArgs& a, const ScanPlace& p, const float* from, float* to) {
  const int lane = threadIdx.x & 31;
  for (int n0 = 0; n0 < (a.cu ? a.seqs : 1); n0 += 32) {
    const int n = n0 + lane;
    const bool empty = a.cu ? n < a.seqs && scan_offset(a, n) >= scan_offset(a, n + 1) : n == 0 && a.T == 0;
    for (unsigned todo = __ballot_sync(0xffffffffu, empty); todo; todo &= todo - 1) {
      const int which = a.cu ? n0 + __ffs(todo) - 1 : p.row;
      const long long at = ((long long)which * a.D + p.c0) * a.N;
      for (int i = lane; i < p.chans * a.N; i += 32) to[at + i] = from ? from[at + i] : 0.f;
    }
  }
}

// Tensors by what their rows are: channels, groups of states, or one state of a sequence.
enum ScanRows { kChannels, kGroups, kStates };
inline size_t scan_bytes(const ScanArgs& a, ScanRows kind, long long ld, size_t io) {
  if (kind == kStates) return (size_t)a.seqs * a.D * a.N * 4;
  return rows_bytes((long long)a.rows * a.T, kind == kChannels ? a.D : (long long)a.G * a.N, ld, io);
}
// Whether a dense output shares memory with an input, other than element for element with one
// of its kind: what writes one part may run beside what still reads another.
inline bool scan_clash(const ScanArgs& a, const void* out, ScanRows kind, size_t io) {
  const long long gn = (long long)a.G * a.N, dense = kind == kChannels ? a.D : gn;
  const struct { const void* p; ScanRows kind; long long ld; } in[8] = {
      {a.x, kChannels, a.ldx}, {a.dt, kChannels, a.lddt}, {a.z, kChannels, a.ldz}, {a.dy, kChannels, a.D},
      {a.B, kGroups, a.ldb},   {a.C, kGroups, a.ldc},     {a.h0, kStates, 0},      {a.dhT, kStates, 0}};
  for (const auto& t : in)
    if (!(out == t.p && kind == t.kind && (kind == kStates || t.ld == dense || (long long)a.rows * a.T == 1)) &&
        overlap(out, scan_bytes(a, kind, dense, io), t.p, scan_bytes(a, t.kind, t.ld, io)))
      return true;
  return false;
}

ckda_status check_scan(int rows, int T, int D, int N, int G, const int32_t* cu, int num_seqs, ckda_dtype io);

// ------------------------------------------------------------- a walk forward
// What a walk over a piece leaves: the outputs (kOut), its end states alone (kEnds), or
// the states before every 4th token for the backward pass (kChunks), then with what the
// piece adds to the gradient that passes it (kGrads, for more than one piece).
enum : int { kOut, kEnds, kChunks, kGrads };

constexpr int kWalkTile = 16;

// Of a warp.
template <typename IO, typename S, int MODE>
struct WalkSmem {
  static constexpr int kTensors = MODE == kOut ? 3 : MODE == kGrads ? 4 : 2;  // x, dt, z or dy, z
  static constexpr bool kC = MODE == kOut || MODE == kGrads;
  alignas(16) ChanTile<IO, kWalkTile> raw[2][kTensors];
  GroupTile<IO, kWalkTile, S::NP> bc[2][kC ? 2 : 1];
  alignas(16) float f[kC ? 2 : 1][kWalkTile * S::NP];  // B and C
};

template <typename IO, typename S, bool VEC, int MODE>
__global__ void __launch_bounds__(kScanBlock) scan_walk_kernel(ScanArgs a) {
  constexpr int LP = S::kLanes, NS = S::kStates, K = kWalkTile, NP = S::NP, kPairs = NS / 2;
  // Tokens of a step of the recurrence's loop: eight (a warp has few others beside it, and
  // 8 x 2048 tokens of 4096 channels of 16 states took 457 us by two, 438 by four, 420 by
  // eight); four where a lane has more states or more to keep.
  constexpr int kTokens = NP <= 16 && MODE != kGrads ? 8 : 4;
  using Smem = WalkSmem<IO, S, MODE>;
  extern __shared__ __align__(16) char sm[];
  Smem& s = reinterpret_cast<Smem*>(sm)[threadIdx.x >> 5];
  after_previous();
  let_next_start();
  ScanPlace p;
  if (!scan_place(a, p)) return;
  const int lane = threadIdx.x & 31, n0 = lane % LP * NS;
  if (MODE == kOut && p.piece == 0 && a.hT && (a.cu || a.T == 0)) empty_states(a, p, a.h0, a.hT);
  if (MODE == kOut && a.fill) zero_behind<IO>(a, p, a.y);
  if (p.t0 >= p.t1) return;

  constexpr bool kAsync = kScanAsync<IO, VEC>;
  HeldChans<IO, kAsync ? 1 : K> held[Smem::kTensors];
  HeldGroups<IO, K, kAsync ? 32 / K : NP> held_bc[2];
  const auto fetch = [&](int t, int stage) {
    const int count = p.t1 - t < K ? p.t1 - t : K;
    const long long at = (long long)p.row * a.T + t;
    const auto chans = [&](int i, const void* base, long long ld) {
      if constexpr (kAsync)
        s.raw[stage][i].template fetch<VEC>(base, ld, at, p.c0, count, p.chans);
      else
        held[i].load(base, ld, at, p.c0, count, p.chans);
    };
    const auto groups = [&](int i, const void* base, long long ld) {
      if constexpr (kAsync)
        s.bc[stage][i].template fetch<VEC>(base, ld, at, count, p.g, a.N);
      else
        held_bc[i].load(base, ld, at, count, p.g, a.N);
    };
    chans(0, a.x, a.ldx);
    chans(1, a.dt, a.lddt);
    if (MODE == kGrads) chans(MODE == kGrads ? 2 : 0, a.dy, a.D);
    if (Smem::kC && a.z) chans(Smem::kTensors - 1, a.z, a.ldz);
    groups(0, a.B, a.ldb);
    if (Smem::kC) groups(Smem::kC ? 1 : 0, a.C, a.ldc);
    copy_commit();
  };
  const auto land = [&](int stage) {
    if constexpr (!kAsync) {
#pragma unroll
      for (int i = 0; i < Smem::kTensors; ++i) held[i].leave(s.raw[stage][i]);
      held_bc[0].leave(s.bc[stage][0]);
      if constexpr (Smem::kC) held_bc[1].leave(s.bc[stage][1]);
    }
  };
  fetch(p.t0, 0);
  land(0);

  const bool own = lane < p.chans;
  const int c = p.c0 + (own ? lane : 0);  // the lane's own channel
  const float2 bias = both<float2>(a.dt_bias ? a.dt_bias[c] : 0.f);
  const float2 skip = both<float2>(MODE == kOut && a.skip ? a.skip[c] : 0.f);
  float2 A2[LP][kPairs], h[LP][kPairs];  // of the channels of lanes lane ^ j
  float2 G[MODE == kGrads ? LP : 1][kPairs], W[MODE == kGrads ? LP : 1][kPairs];  // W: decays from the piece's start
  const auto have = [&](int j) { return (lane ^ j) < p.chans; };
  const auto chan = [&](int j) { return p.c0 + (have(j) ? lane ^ j : 0); };
#pragma unroll
  for (int j = 0; j < LP; ++j) {
    load_states<NS>(A2[j], a.A, chan(j), a.N, n0, have(j));
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      A2[j][q] = mul_(A2[j][q], both<float2>(kLog2e));
      h[j][q] = both<float2>(0.f);
      if (MODE == kGrads) {
        G[j][q] = both<float2>(0.f);
        W[j][q] = both<float2>(1.f);
      }
    }
  }
  float span = 0.f;  // of the own channel's steps
  ScanSeq seq = scan_seq_at(a, p.row, p.t0);
  bool entered = seq.begin < p.t0;  // still in the sequence that entered the piece
  const long long unit = (long long)p.row * a.pieces + p.piece;
  if (MODE == kOut && a.pieces > 1 && entered)
#pragma unroll
    for (int j = 0; j < LP; ++j) load_states<NS>(h[j], a.state, unit * a.D + chan(j), a.N, n0, have(j));
  IO* out = MODE == kOut ? static_cast<IO*>(a.y) + ((long long)p.row * a.T + p.t0) * a.D + c : nullptr;

  int stage = 0;
  for (int t = p.t0; t < p.t1; t += K, stage ^= 1) {
    const int count = p.t1 - t < K ? p.t1 - t : K;
    copy_wait<0>();
    __syncwarp();
    s.bc[stage][0].template unpack_to<VEC>(s.f[0], count, a.N);
    if (Smem::kC) s.bc[stage][Smem::kC ? 1 : 0].template unpack_to<VEC>(s.f[Smem::kC ? 1 : 0], count, a.N);
    const bool edges = t <= seq.begin || t + count >= seq.end;
    const bool whole = count == K && p.chans == kScanChans;
    Marks marks;
    if (edges) marks.find(a, p.row, t, count);
    __syncwarp();
    if (t + K < p.t1) fetch(t + K, stage ^ 1);
    const auto recur = [&](auto checked) {
      constexpr bool kChecked = decltype(checked)::value;
#pragma unroll 1
      for (int k0 = 0; k0 < count; k0 += kTokens) {
        float2 x[kTokens / 2], d[kTokens / 2], u[kTokens / 2], up[kTokens / 2], ys[kTokens / 2];
#pragma unroll
        for (int i = 0; i < kTokens / 2; ++i) {  // two tokens of the own channel
          const int k = k0 + 2 * i;
          x[i] = s.raw[stage][0].pair(k);
          d[i] = step_sizes(s.raw[stage][1].pair(k), bias, a.softplus);
          if (MODE == kGrads) {
            up[i] = s.raw[stage][MODE == kGrads ? 2 : 0].pair(k);
            if (a.z) up[i] = mul_(up[i], scan_silu(s.raw[stage][Smem::kTensors - 1].pair(k)));
          }
          if (!whole) {  // (what there is not was not loaded)
            const bool in0 = own && k < count, in1 = own && k + 1 < count;
            d[i] = make_float2(in0 ? d[i].x : 0.f, in1 ? d[i].y : 0.f);
            x[i] = make_float2(in0 ? x[i].x : 0.f, in1 ? x[i].y : 0.f);
            if (MODE == kGrads) up[i] = make_float2(in0 ? up[i].x : 0.f, in1 ? up[i].y : 0.f);
          }
          u[i] = mul_(d[i], x[i]);
        }
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
          const int k = k0 + i;
          const bool first = kChecked && (marks.first >> k & 1), last = kChecked && (marks.last >> k & 1);
          const int num = kChecked && (first || last) ? marks.number(k) : 0;
          if ((MODE == kChunks || MODE == kGrads) && i % kScanChunk == 0 && k < count) {
            const long long ck = (long long)p.row * a.chunks + (t + k) / kScanChunk;
#pragma unroll
            for (int j = 0; j < LP; ++j) store_states<NS>(a.chunk, ck * a.D + chan(j), a.N, n0, have(j), h[j]);
            if (MODE == kGrads && own) a.chunk_sum[ck * a.D + c] = span + part;
          }
          if (first) {
            entered = false;
#pragma unroll
            for (int j = 0; j < LP; ++j) {
              if (a.h0)
                load_states<NS>(h[j], a.h0, (long long)num * a.D + chan(j), a.N, n0, have(j));
              else
#pragma unroll
                for (int q = 0; q < kPairs; ++q) h[j][q] = both<float2>(0.f);
            }
          }
          const float own_d = i & 1 ? d[i / 2].y : d[i / 2].x, own_u = i & 1 ? u[i / 2].y : u[i / 2].x;
          const float own_up = MODE == kGrads ? (i & 1 ? up[i / 2].y : up[i / 2].x) : 0.f;
          if (MODE != kOut) part += own_d;
          float2 Bk[kPairs], Ck[kPairs];
          from_shared<NS>(Bk, s.f[0] + k * NP + n0);
          if (Smem::kC) from_shared<NS>(Ck, s.f[Smem::kC ? 1 : 0] + k * NP + n0);
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < LP; ++j) {
            const float2 delta = both<float2>(j ? __shfl_xor_sync(0xffffffffu, own_d, j) : own_d);
            const float2 uu = both<float2>(j ? __shfl_xor_sync(0xffffffffu, own_u, j) : own_u);
            float2 upp;
            if (MODE == kGrads) upp = both<float2>(j ? __shfl_xor_sync(0xffffffffu, own_up, j) : own_up);
            float2 y;
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
              const float2 decay = decay_of(delta, A2[j][q]);
              h[j][q] = fma_(decay, h[j][q], mul_(uu, Bk[q]));
              if (MODE == kOut) y = q == 0 ? mul_(Ck[q], h[j][q]) : fma_(Ck[q], h[j][q], y);
              if (MODE == kGrads && entered) {
                W[j][q] = mul_(W[j][q], decay);
                G[j][q] = fma_(W[j][q], mul_(upp, Ck[q]), G[j][q]);
              }
            }
            if (MODE == kOut) sum = j ? sum + __shfl_xor_sync(0xffffffffu, y.x + y.y, j) : y.x + y.y;
            if (MODE == kOut && last && a.hT)
              store_states<NS>(a.hT, (long long)num * a.D + chan(j), a.N, n0, have(j), h[j]);
            if (MODE == kGrads && last && entered && a.dhT) {
              float2 dh[kPairs];
              load_states<NS>(dh, a.dhT, (long long)num * a.D + chan(j), a.N, n0, have(j));
#pragma unroll
              for (int q = 0; q < kPairs; ++q) G[j][q] = fma_(W[j][q], dh[q], G[j][q]);
            }
          }
          (i & 1 ? ys[i / 2].y : ys[i / 2].x) = sum;
        }
        span += part;
        if (MODE == kOut)
#pragma unroll
          for (int i = 0; i < kTokens / 2; ++i) {
            const int k = k0 + 2 * i;
            float2 o = fma_(skip, x[i], ys[i]);
            if (a.z) o = mul_(o, scan_silu(s.raw[stage][Smem::kTensors - 1].pair(k)));
            if (own && k < count) st_io(out, o.x);
            if (own && k + 1 < count) st_io(out + a.D, o.y);
            out += 2 * (long long)a.D;
          }
      }
    };
    if (edges)
      recur(std::true_type());
    else
      recur(std::false_type());
    if (t + count >= seq.end && t + count < p.t1) seq = scan_seq_at(a, p.row, t + count);
    if (t + K < p.t1) land(stage ^ 1);
  }
  if (MODE == kEnds || MODE == kGrads) {
#pragma unroll
    for (int j = 0; j < LP; ++j) {
      store_states<NS>(a.state, unit * a.D + chan(j), a.N, n0, have(j), h[j]);
      if (MODE == kGrads) store_states<NS>(a.grad, unit * a.D + chan(j), a.N, n0, have(j), G[j]);
    }
    if (own) a.span[unit * a.D + c] = span;
  }
}

template <typename IO, typename S, bool VEC, int MODE>
cudaError_t launch_walk(bool next, const ScanArgs& a, cudaStream_t s) {
  const auto kernel = scan_walk_kernel<IO, S, VEC, MODE>;
  constexpr size_t smem = kScanWarps * sizeof(WalkSmem<IO, S, MODE>);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_next(next, kernel, scan_grid(a), kScanBlock, smem, s, a);
}

// Whole vectors: 16-byte rows of channels and packs of four states (2 x 1001 tokens of 480
// channels of 12 states in fp32, backward: 209 us in single elements).
inline bool scan_aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline bool scan_vectors(const ScanArgs& a, size_t io) {
  const int v = (int)(16 / io);
  return a.N % 4 == 0 && a.D / a.G % v == 0 && a.ldx % v == 0 && a.lddt % v == 0 && (!a.z || a.ldz % v == 0) &&
         a.ldb % 4 == 0 && a.ldc % 4 == 0 && scan_aligned(a.x, 16) && scan_aligned(a.dt, 16) &&
         scan_aligned(a.z, 16) && scan_aligned(a.dy, 16) && scan_aligned(a.B, 4 * io) && scan_aligned(a.C, 4 * io);
}

}  // namespace ckda
