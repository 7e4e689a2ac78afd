// ckda_scan.cuh -- what the kernels of the selective scan share.
//
// Per channel d with N states, over the tokens of a sequence:
//     delta_t = softplus(dt_t + dt_bias)   (or without the softplus)
//     h_t[n]  = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n]
//     y_t     = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)
//
// Tokens are rows of D channels; B and C are rows of G groups of N, shared by the D / G
// channels of a group.  A block takes CH channels of one group and walks a piece of one
// row's tokens in tiles of K:
//   1. each thread takes 8 neighbouring channels of one token, forms delta and u = delta x
//      and leaves them in shared memory (B and C of the tile go there as fp32);
//   2. LP lanes share a channel, NS states each in registers, and run the recurrence over
//      the tile; the sums over n are folded over the lanes, LP tokens at a time;
//   3. the threads of step 1 finish their 8 outputs.
// Sequence borders (dense rows' ends, packed sequences) are marked per token in tiles
// that hold one; other tiles run without the checks.
#pragma once
#include "ckda_launch.cuh"
#include "ckda_rows.cuh"

namespace ckda {

constexpr int kScanBlock = 128;
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
  int pieces, piece_len;  // of a row
  int chan_blocks;        // of all channels; per group chan_blocks / G
  float* state;           // [rows][pieces][D][N]: what a piece adds, then what enters it
  float* span;            // [rows][pieces][D]: sum of a piece's steps
};

// ------------------------------------------------------------------ arithmetic
__device__ __forceinline__ float ex2(float a) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(a));
  return d;
}
__device__ __forceinline__ float2 ex2(float2 a) { return make_float2(ex2(a.x), ex2(a.y)); }
__device__ __forceinline__ float scan_sigmoid(float p) { return __fdividef(1.f, 1.f + __expf(-p)); }
__device__ __forceinline__ float scan_silu(float p) { return __fdividef(p, 1.f + __expf(-p)); }
// log(1 + e^x) = max(x, 0) + log1p(e^-|x|), and log1p(t) = 2 atanh(t / (2 + t)) by its
// power series: t <= 1 makes the argument at most 1/3, and seven terms leave 2e-8.
// Small steps (x well below 0) keep their relative precision.
__device__ __forceinline__ float softplus(float x) {
  const float t = expf(-fabsf(x));
  const float s = __fdividef(t, 2.f + t), q = s * s;
  float p = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  p = fmaf(q, p, 1.f / 9.f);
  p = fmaf(q, p, 1.f / 7.f);
  p = fmaf(q, p, 1.f / 5.f);
  p = fmaf(q, p, 1.f / 3.f);
  p = fmaf(q, p, 1.f);
  return fmaf(2.f * s, p, fmaxf(x, 0.f));
}

// Sums over LP neighbouring lanes of LP values: lane l gets the sum of v[l].
template <int LP>
__device__ __forceinline__ float fold(float (&v)[LP], int l) {
#pragma unroll
  for (int s = LP / 2; s >= 1; s /= 2) {
    const bool up = (l & s) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float send = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
    }
  }
  return v[0];
}

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
// KMOST: tokens of a tile at most (then some threads have none in steps 1 and 3).
template <int LP, int NS, int P, int KMOST = 64>
struct ScanShape {
  static constexpr int kLanes = LP, kStates = NS, kChans = P;
  static constexpr int CH = P * kScanBlock / LP;    // channels of a block
  static constexpr int V8 = CH / 8;                 // vectors of 8 channels to a token
  static constexpr int K = kScanBlock / V8 < KMOST ? kScanBlock / V8 : KMOST;  // tokens of a tile
  static constexpr int NP = LP * NS;                // states, padded
  static constexpr int NB = (K * NP + kScanBlock - 1) / kScanBlock;  // elements of B (C) to a thread
  // Channel 8 v + e of a tile stands at e V8 + v, rows padded by V8: the threads of a
  // warp, V8 vectors of several tokens, then write 8 e's without bank conflicts.
  static constexpr int kRow = CH + V8;
  static __device__ __forceinline__ int chan_at(int pos) { return pos % V8 * 8 + pos / V8; }
};

// 8 neighbouring channels of one token, as loaded.
template <typename IO>
struct Eight {
  Pack<IO, 16 / sizeof(IO)> v[sizeof(IO) / 2];
  __device__ __forceinline__ float at(int e) const {
    constexpr int kV = 16 / sizeof(IO);
    return ld_io(&v[e / kV].v[e % kV]);
  }
  template <bool VEC>
  __device__ __forceinline__ void load(const void* base, long long at, int n) {  // n: channels that exist
    constexpr int kV = 16 / sizeof(IO);
    const IO* p = static_cast<const IO*>(base) + at;
    if (VEC) {
      if (n > 0)
#pragma unroll
        for (int j = 0; j < (int)(sizeof(IO) / 2); ++j) v[j] = reinterpret_cast<const Pack<IO, kV>*>(p)[j];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) v[e / kV].v[e % kV] = p[e];
    }
  }
};
template <typename IO, bool VEC>
__device__ __forceinline__ void store_eight(void* base, long long at, int n, const float (&f)[8]) {
  constexpr int kV = 16 / sizeof(IO);
  IO* p = static_cast<IO*>(base) + at;
  if (VEC) {
    if (n > 0)
#pragma unroll
      for (int j = 0; j < 8 / kV; ++j) {
        Pack<IO, kV> o;
#pragma unroll
        for (int e = 0; e < kV; ++e) st_io(&o.v[e], f[j * kV + e]);
        reinterpret_cast<Pack<IO, kV>*>(p)[j] = o;
      }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) st_io(p + e, f[e]);
  }
}

// The tile's part of B or C: NB elements to a thread, of tokens [t, t + count).
template <typename IO, typename S>
struct GroupTile {
  IO v[S::NB];
  template <bool VEC>
  __device__ __forceinline__ void load(const void* base, long long ld, long long t, int count, int g, int N) {
    if (VEC && S::NB % 4 == 0) {  // (N is NP: whole vectors of 4)
#pragma unroll
      for (int j = 0; j < S::NB / 4; ++j) {
        const int i = (j * kScanBlock + (int)threadIdx.x) * 4, k = i / S::NP, n = i % S::NP;
        if (k < count)
          *reinterpret_cast<Pack<IO, 4>*>(&v[j * 4]) = *reinterpret_cast<const Pack<IO, 4>*>(
              static_cast<const IO*>(base) + (t + k) * ld + (long long)g * N + n);
      }
    } else {
#pragma unroll
      for (int j = 0; j < S::NB; ++j) {
        const int i = j * kScanBlock + threadIdx.x, k = i / S::NP, n = i % S::NP;
        if (k < count && n < N) v[j] = static_cast<const IO*>(base)[(t + k) * ld + (long long)g * N + n];
      }
    }
  }
  // (zero where there is no token or no state)
  template <bool VEC>
  __device__ __forceinline__ void leave(float* to, int count, int N) const {
    if (VEC && S::NB % 4 == 0) {
#pragma unroll
      for (int j = 0; j < S::NB / 4; ++j) {
        const int i = (j * kScanBlock + (int)threadIdx.x) * 4;
        const bool in = i / S::NP < count;
        *reinterpret_cast<float4*>(to + i) =
            make_float4(in ? ld_io(&v[j * 4]) : 0.f, in ? ld_io(&v[j * 4 + 1]) : 0.f,
                        in ? ld_io(&v[j * 4 + 2]) : 0.f, in ? ld_io(&v[j * 4 + 3]) : 0.f);
      }
    } else {
#pragma unroll
      for (int j = 0; j < S::NB; ++j) {
        const int i = j * kScanBlock + threadIdx.x;
        if (i < S::K * S::NP) to[i] = i / S::NP < count && i % S::NP < N ? ld_io(&v[j]) : 0.f;
      }
    }
  }
};

// Marks of the tile's tokens: 1 a sequence's first, 2 its last; and its number.
template <int K>
struct Marks {
  int mark[K], n[K];
  __device__ __forceinline__ void fill(const ScanArgs& a, int row, int t, int count) {
    for (int k = threadIdx.x; k < K; k += kScanBlock) {
      int f = 0, num = 0;
      if (k < count) {
        const ScanSeq s = scan_seq_at(a, row, t + k);
        f = (t + k == s.begin ? 1 : 0) | (t + k + 1 == s.end ? 2 : 0);
        num = s.n;
      }
      mark[k] = f;
      n[k] = num;
    }
  }
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

// Where a block works: CH channels of a group from c0, a piece of a row.
struct ScanPlace {
  int row, piece, g, c0, chans;  // chans: that exist
  int t0, t1;
};
template <int CH>
__device__ __forceinline__ ScanPlace scan_place(const ScanArgs& a) {
  ScanPlace p;
  const int cb = (int)(blockIdx.x % a.chan_blocks);
  const int unit = (int)(blockIdx.x / a.chan_blocks);
  p.row = unit / a.pieces;
  p.piece = unit % a.pieces;
  const int per = a.chan_blocks / a.G, dg = a.D / a.G;
  p.g = cb / per;
  const int first = cb % per * CH;
  p.c0 = p.g * dg + first;
  p.chans = dg - first < CH ? dg - first : CH;
  const int last = scan_last(a);
  p.t0 = p.piece * a.piece_len;
  p.t1 = p.t0 + a.piece_len < last ? p.t0 + a.piece_len : last;
  return p;
}

// delta and u = delta x of a thread's 8 channels.
template <typename IO>
__device__ __forceinline__ void step_sizes(const Eight<IO>& dt, const float* bias, int softplus_on, bool in,
                                           float (&delta)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float raw = dt.at(e) + bias[e];
    delta[e] = in ? (softplus_on ? softplus(raw) : raw) : 0.f;
  }
}

// States that enter the pieces, from what each adds (ckda_scan_fwd.cu).
cudaError_t launch_scan_join(bool next, const ScanArgs& a, cudaStream_t s);
// Pieces of a row: one where its channels, `chans` to a block, fill the room of `room`
// blocks; else as many as it has room for, of at least 128 tokens, in whole tiles.
void scan_pieces(int rows, int T, int D, int G, int chans, int room, int* pieces, int* len);

// Empty sequences hand their states on: a block copies its channels' part of `from` (zero
// if null) to `to`.
template <int CH>
__device__ __forceinline__ void empty_states(const ScanArgs& a, const ScanPlace& p, const float* from, float* to) {
  const int tid = threadIdx.x;
  for (int n0 = 0; n0 < (a.cu ? a.seqs : 1); n0 += kScanBlock) {
    const int n = n0 + tid;
    const bool empty = a.cu ? n < a.seqs && scan_offset(a, n) >= scan_offset(a, n + 1) : n == 0 && a.T == 0;
    for (unsigned todo = __ballot_sync(0xffffffffu, empty); todo; todo &= todo - 1) {
      const int which = a.cu ? n0 + (tid & ~31) + __ffs(todo) - 1 : p.row;
      const long long at = ((long long)which * a.D + p.c0) * a.N;
      for (int i = tid & 31; i < p.chans * a.N; i += 32) to[at + i] = from ? from[at + i] : 0.f;
    }
  }
}

ckda_status check_scan(int rows, int T, int D, int N, int G, const int32_t* cu, int num_seqs, ckda_dtype io);

}  // namespace ckda
