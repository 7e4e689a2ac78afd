// ckda_conv.cu -- short causal convolution of each channel, forward, backward and one
// token on a resident state.
//
// Per channel, over the tokens of a sequence, with W = 2, 3 or 4 taps:
//     p_t = b + sum_j w_j x_{t-W+1+j},    y_t = p_t / (1 + exp(-p_t))  or  p_t
// where the inputs before the first token are the W - 1 rows of the initial state (or
// zero) and the last W - 1 inputs are the final state.  With dp = dy silu'(p):
//     dx_i = sum_k w_{W-1-k} dp_{i+k},   dw_j = sum_t dp_t x_{t-W+1+j},   db = sum_t dp_t
// and a final state's gradient adds to the inputs that it holds.
//
// Each input is read once and each output written once; 2 W + 4 flop an element leave HBM
// as the bound.  Channels are the fast axis: a thread has VEC neighbouring channels, in
// pairs, and walks a run of tokens with the last W - 1 inputs in registers, the next 8
// tokens on their way through a ring in shared memory.  A run starts W - 1 tokens early
// (backward: and ends W - 1 late), 5% at 64 tokens and mostly from L2.  Runs go over one
// flat axis of tokens, dense rows or packed sequences alike, and take up the next
// sequence's state where one begins.
//
// The gradients of the weights: sums over a run in registers, over a block's runs in
// shared memory, then one partial row a block in the workspace, added in a fixed order by
// a second kernel that carries along what its additions round off.  No atomics: the same
// bits every time.  (All in fp32; the sum over 64 tokens of a run is most of what is left,
// 1.7e-7 of dw over 16,384 tokens.)
//
// Measured, bf16 with four taps, bias and silu: 24 packed prompts, 50,021 tokens of 4096
// channels, 138 us, 89% of the copy bandwidth (8 channels a thread with the loads held in
// registers 488, 4 channels 176, 2 channels 163); backward of 8 x 2048 tokens 99 us, 61%
// (458 in registers, 202 by groups of tokens in registers, 117 with checks in every token).
// Odd channel counts go by single elements: 4 x 2048 tokens of 4095 in 41 us, 50%.
#include "ckda_launch.cuh"
#include "ckda_rows.cuh"

namespace ckda {
namespace {

constexpr int kBlock = 256;
constexpr int kAhead = 4;
constexpr int kVec = 4;
constexpr float kLog2e = 1.4426950408889634f;

struct ConvArgs {
  const void* x;
  const void* dy;
  const void* w;  // [D][W]
  const void* b;
  const void* h0;  // [seqs][W - 1][D]
  const void* dhT;
  void* y;   // dx in the backward pass
  void* hT;  // dh0 in the backward pass
  void* dw;
  void* db;
  float* part;  // [parts][W + 1][D]: sums of dw by tap, then db
  const int32_t* cu;
  long long ldx;  // elements from one token to the next
  long long tokens;
  int seqs, T, D;  // T: of a dense row
  int w_bf16, silu;
  int fill;        // rows of y behind the last sequence become zero
  int run;         // tokens of a run
  int lanes;       // threads of a token, a power of two
  int chan_blocks, parts;
  long long main_blocks;  // blocks behind these have the states
};

__device__ __forceinline__ float weight_of(const void* w, int bf16, size_t i) {
  return bf16 ? ld_io(static_cast<const __nv_bfloat16*>(w) + i) : static_cast<const float*>(w)[i];
}
// 1 / (1 + 2^a), 0 where 2^a leaves fp32 (p / (1 + e^-p) at p = -inf has no value either way)
__device__ __forceinline__ float one_plus_inverse(float a) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
__device__ __forceinline__ float2 one_plus_inverse(float2 a) {
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(a.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(a.y));
  e = add_(e, both<float2>(1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  return r;
}

// A sequence's tokens [begin, end) on the flat axis.  Offsets that are out of order or out
// of range leave every access inside the tensors.
struct Seq {
  long long begin, end;
  int n;
};
__device__ __forceinline__ long long offset_of(const ConvArgs& a, int n) {
  const long long o = a.cu[n];
  return o < 0 ? 0 : o > a.tokens ? a.tokens : o;
}
__device__ __forceinline__ Seq seq_at(const ConvArgs& a, long long m) {
  Seq s;
  if (!a.cu) {
    s.n = (int)(m / a.T);
    s.begin = (long long)s.n * a.T;
    s.end = s.begin + a.T;
    return s;
  }
  int lo = 0, hi = a.seqs;  // the last n with cu[n] <= m
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= m) lo = mid; else hi = mid;
  }
  s.n = lo;
  s.begin = offset_of(a, lo);
  s.end = offset_of(a, lo + 1);
  return s;
}

template <typename IO, int VEC>
__device__ __forceinline__ Pack<IO, VEC> load_row(const void* base, long long row, long long ld, int c) {
  return *reinterpret_cast<const Pack<IO, VEC>*>(static_cast<const IO*>(base) + row * ld + c);
}
// A thread's VEC channels as pairs.
template <int VEC>
struct Chans {
  using V = typename Pairs<VEC>::V;
  static constexpr int kN = Pairs<VEC>::kN;
  V v[kN];
  __device__ __forceinline__ float* flat() { return reinterpret_cast<float*>(v); }
  __device__ __forceinline__ void fill(float f) {
#pragma unroll
    for (int e = 0; e < kN; ++e) v[e] = both<V>(f);
  }
  template <typename IO>
  __device__ __forceinline__ void from(const Pack<IO, VEC>& p) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) flat()[e] = ld_io(&p.v[e]);
  }
  __device__ __forceinline__ void silu() {  // v / (1 + e^-v)
#pragma unroll
    for (int e = 0; e < kN; ++e) v[e] = mul_(v[e], one_plus_inverse(mul_(v[e], both<V>(-kLog2e))));
  }
  // times the slope g (1 + p (1 - g)), g = 1 / (1 + e^-p)
  __device__ __forceinline__ void times_silu_grad(const Chans& p) {
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const V g = one_plus_inverse(mul_(p.v[e], both<V>(-kLog2e)));
      const V rest = fma_(g, both<V>(-1.f), both<V>(1.f));
      v[e] = mul_(v[e], mul_(g, fma_(p.v[e], rest, both<V>(1.f))));
    }
  }
  template <typename IO>
  __device__ __forceinline__ void store(void* base, long long at) {
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = flat()[e];
    store_vec<IO, VEC>(base, at, f);
  }
};
template <int W, int VEC>
struct Taps {
  Chans<VEC> w[W], b;
  __device__ __forceinline__ void load(const ConvArgs& a, int c) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j].flat()[e] = weight_of(a.w, a.w_bf16, (size_t)(c + e) * W + j);
      b.flat()[e] = a.b ? weight_of(a.b, a.w_bf16, c + e) : 0.f;
    }
  }
  // bias + sum over the taps of the inputs before (oldest first) and x
  __device__ __forceinline__ Chans<VEC> sum(const Chans<VEC> (&in)[W - 1], const Chans<VEC>& x) const {
    Chans<VEC> p;
#pragma unroll
    for (int e = 0; e < Chans<VEC>::kN; ++e) {
      p.v[e] = fma_(w[W - 1].v[e], x.v[e], b.v[e]);
#pragma unroll
      for (int k = W - 2; k >= 0; --k) p.v[e] = fma_(w[k].v[e], in[k].v[e], p.v[e]);
    }
    return p;
  }
};

// Rows of y behind the last sequence, every apart-th from `from` to `to`: zero.  (What
// nothing writes could be anything, and a NaN there reaches every weight of a layer that
// takes all rows.)
template <typename IO, int VEC>
__device__ __forceinline__ void zero_rows(const ConvArgs& a, long long from, long long to, int apart, int c) {
  const float none[VEC] = {};
  for (; from < to; from += apart) store_vec<IO, VEC>(a.y, from * a.D + c, none);
}

// Row i of the inputs before a sequence's token m: i = 0 is W - 1 tokens back.
template <typename IO, int W, int VEC>
__device__ __forceinline__ Chans<VEC> input_before(const ConvArgs& a, const Seq& s, long long m, int i, int c) {
  const long long t = m - (W - 1) + i;
  Chans<VEC> f;
  if (t >= s.begin) {
    f.from(load_row<IO, VEC>(a.x, t, a.ldx, c));
  } else if (a.h0) {
    const long long r = t - s.begin + W - 1;
    f.from(load_row<IO, VEC>(a.h0, (long long)s.n * (W - 1) + (r < 0 ? 0 : r), a.D, c));
  } else {
    f.fill(0.f);
  }
  return f;
}

// ------------------------------------------------------------------ forward
// The final state of every sequence: its last W - 1 inputs, older ones from h0.
template <typename IO, int W, int VEC>
__device__ void final_states(const ConvArgs& a) {
  const int vecs = a.D / VEC;
  const long long n_all = (long long)a.seqs * (W - 1) * vecs;
  const long long step = (long long)(gridDim.x - a.main_blocks) * kBlock;
  for (long long i = ((long long)blockIdx.x - a.main_blocks) * kBlock + threadIdx.x; i < n_all; i += step) {
    const int c = (int)(i % vecs) * VEC;
    const int r = (int)(i / vecs % (W - 1));
    Seq s;
    s.n = (int)(i / vecs / (W - 1));
    s.begin = a.cu ? offset_of(a, s.n) : (long long)s.n * a.T;
    s.end = a.cu ? offset_of(a, s.n + 1) : s.begin + a.T;
    if (s.end < s.begin) s.end = s.begin;
    input_before<IO, W, VEC>(a, s, s.end, r, c).template store<IO>(a.hT, ((long long)s.n * (W - 1) + r) * a.D + c);
  }
}

// The tokens of a run, kAhead to a group, two groups ahead in shared memory: a thread
// copies with cp.async what it reads itself, so the ring needs no barrier and the loads in
// flight no registers.  Single bf16 channels (two bytes) come through registers, a group
// of twice as many at a time.
template <typename IO, int VEC, int TENSORS>
struct TokenRing {
  using P = Pack<IO, VEC>;
  static constexpr bool kAsync = sizeof(P) >= 4;
  static constexpr int kStages = 3, kGroup = kAsync ? kAhead : 2 * kAhead;
  static constexpr size_t kSmem = kAsync ? (size_t)kStages * kGroup * TENSORS * kBlock * sizeof(P) : 0;
  P* base;
  int total;
  const IO* next[TENSORS];
  long long ld[TENSORS];
  P own[kAsync ? 1 : kGroup][TENSORS];
  __device__ __forceinline__ TokenRing(char* sm, int tokens)
      : base(reinterpret_cast<P*>(sm) + threadIdx.x), total(tokens) {}
  __device__ __forceinline__ void from(int t, const IO* p, long long apart) {
    next[t] = p;
    ld[t] = apart;
  }
  __device__ __forceinline__ P& at(P* stage, int u, int t) {
    if constexpr (kAsync)
      return stage[(u * TENSORS + t) * kBlock];
    else
      return own[u][t];
  }
  __device__ __forceinline__ P* stage(int i) const { return base + i * (kGroup * TENSORS * kBlock); }
  __device__ __forceinline__ void one(P* stage, int u) {
#pragma unroll
    for (int t = 0; t < TENSORS; ++t) {
      if constexpr (kAsync)
        copy_async<sizeof(P)>(&at(stage, u, t), next[t]);
      else
        own[u][t] = *reinterpret_cast<const P*>(next[t]);
      next[t] += ld[t];
    }
  }
  __device__ __forceinline__ void fetch(P* stage, int first) {
    if (first + kGroup <= total) {
#pragma unroll
      for (int u = 0; u < kGroup; ++u) one(stage, u);
    } else {
#pragma unroll
      for (int u = 0; u < kGroup; ++u)
        if (first + u < total) one(stage, u);
    }
    if (kAsync) copy_commit();
  }
  // work(stage, u, t, plain) for every token t, in order; `plain` where the whole group is
  // below `to` and not below `from`
  template <typename F>
  __device__ __forceinline__ void each(int from, int to, F work) {
    if (kAsync) {
      fetch(stage(0), 0);
      fetch(stage(1), kGroup);
    }
    int i = 0;
    for (int g = 0; g < total; g += kGroup) {
      P* const at = stage(i);
      if (kAsync) {
        fetch(stage(i == 0 ? 2 : i - 1), g + 2 * kGroup);
        copy_wait<2>();
      } else {
        fetch(at, g);
      }
      if (g >= from && g + kGroup <= to) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u) work(at, u, g + u, true);
      } else {
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
          if (g + u < total) work(at, u, g + u, false);
      }
      i = i == 2 ? 0 : i + 1;
    }
  }
};

template <typename IO, int W, int VEC>
__global__ void __launch_bounds__(kBlock) conv_fwd_kernel(ConvArgs a) {
  extern __shared__ __align__(16) char sm[];
  using Ring = TokenRing<IO, VEC, 1>;
  if (blockIdx.x >= a.main_blocks) {
    final_states<IO, W, VEC>(a);
    return;
  }
  const int chan = (int)(blockIdx.x % a.chan_blocks);
  const long long tok = blockIdx.x / a.chan_blocks;
  const int lane = threadIdx.x % a.lanes, grp = threadIdx.x / a.lanes;
  const int c = (chan * a.lanes + lane) * VEC;
  long long m = (tok * (kBlock / a.lanes) + grp) * a.run;
  long long stop = m + a.run < a.tokens ? m + a.run : a.tokens;
  const long long last = a.cu ? offset_of(a, a.seqs) : a.tokens;
  if (c >= a.D) return;
  if (a.fill) zero_rows<IO, VEC>(a, m > last ? m : last, stop, 1, c);
  if (stop > last) stop = last;
  if (m >= stop) return;
  Taps<W, VEC> taps;
  taps.load(a, c);
  while (m < stop) {  // the run's part of one sequence after another
    const Seq s = seq_at(a, m);
    if (m < s.begin) m = s.begin;
    const long long own = s.end < stop ? s.end : stop;
    const int n = (int)(own - m);
    Chans<VEC> in[W - 1];  // the inputs before the next token, oldest first
#pragma unroll
    for (int i = 0; i < W - 1; ++i) in[i] = input_before<IO, W, VEC>(a, s, m, i, c);
    Ring ring(sm, n);
    ring.from(0, static_cast<const IO*>(a.x) + m * a.ldx + c, a.ldx);
    IO* py = static_cast<IO*>(a.y) + m * a.D + c;
    const auto token = [&](typename Ring::P* stage, int u, int, bool) {
      Chans<VEC> x;
      x.from(ring.at(stage, u, 0));
      Chans<VEC> p = taps.sum(in, x);
      if (a.silu) p.silu();
#pragma unroll
      for (int k = 0; k < W - 2; ++k) in[k] = in[k + 1];
      in[W - 2] = x;
      p.template store<IO>(py, 0);
      py += a.D;
    };
    ring.each(0, n, token);
    m = own > m ? own : stop;
  }
}

// ----------------------------------------------------------------- backward
// The initial state's gradient: row r feeds tap r - k of token k, and a sequence shorter
// than the state hands its row r on as row r - length.
template <typename IO, int W>
__device__ void initial_grads(const ConvArgs& a) {
  const long long n_all = (long long)a.seqs * a.D;
  const long long step = (long long)(gridDim.x - a.main_blocks) * kBlock;
  for (long long i = ((long long)blockIdx.x - a.main_blocks) * kBlock + threadIdx.x; i < n_all; i += step) {
    const int c = (int)(i % a.D);
    Seq s;
    s.n = (int)(i / a.D);
    s.begin = a.cu ? offset_of(a, s.n) : (long long)s.n * a.T;
    s.end = a.cu ? offset_of(a, s.n + 1) : s.begin + a.T;
    const int length = (int)(s.end - s.begin < W - 1 ? (s.end > s.begin ? s.end - s.begin : 0) : W - 1);
    Taps<W, 1> taps;
    taps.load(a, c);
    float dp[W - 1];
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
      dp[t] = 0.f;
      if (t >= length) continue;
      dp[t] = ld_io(static_cast<const IO*>(a.dy) + (s.begin + t) * a.D + c);
      if (!a.silu) continue;
      Chans<1> in[W - 1], x;
      x.v[0] = ld_io(static_cast<const IO*>(a.x) + (s.begin + t) * a.ldx + c);
#pragma unroll
      for (int k = 0; k < W - 1; ++k) in[k] = input_before<IO, W, 1>(a, s, s.begin + t, k, c);
      Chans<1> g;
      g.v[0] = dp[t];
      g.times_silu_grad(taps.sum(in, x));
      dp[t] = g.v[0];
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      float g = 0.f;
#pragma unroll
      for (int t = 0; t <= r; ++t) g = fmaf(taps.w[r - t].v[0], dp[t], g);
      if (a.dhT && r >= length)
        g += ld_io(static_cast<const IO*>(a.dhT) + ((long long)s.n * (W - 1) + r - length) * a.D + c);
      st_io(static_cast<IO*>(a.hT) + ((long long)s.n * (W - 1) + r) * a.D + c, g);
    }
  }
}

template <typename IO, int W, int VEC>
__global__ void __launch_bounds__(kBlock, 2) conv_bwd_kernel(ConvArgs a) {
  extern __shared__ __align__(16) char sm[];
  using Ring = TokenRing<IO, VEC, 2>;
  let_next_start();
  if (blockIdx.x >= a.main_blocks) {
    initial_grads<IO, W>(a);
    return;
  }
  const int chan = (int)(blockIdx.x % a.chan_blocks);
  const long long tok = blockIdx.x / a.chan_blocks;
  const int lane = threadIdx.x % a.lanes, grp = threadIdx.x / a.lanes, groups = kBlock / a.lanes;
  const int c = (chan * a.lanes + lane) * VEC;
  const long long last = a.cu ? offset_of(a, a.seqs) : a.tokens;
  long long m = (tok * groups + grp) * a.run;
  long long stop = m + a.run < last ? m + a.run : last;
  using V = typename Chans<VEC>::V;
  constexpr int kN = Chans<VEC>::kN;
  Chans<VEC> dw[W], db;
  db.fill(0.f);
#pragma unroll
  for (int j = 0; j < W; ++j) dw[j].fill(0.f);
  if (c < a.D && m < stop) {
    Taps<W, VEC> taps;
    taps.load(a, c);
    while (m < stop) {  // the run's part of one sequence after another
      const Seq s = seq_at(a, m);
      if (m < s.begin) m = s.begin;
      const long long own = s.end < stop ? s.end : stop;  // tokens of this run, then W - 1 that its inputs reach
      const int n = (int)(own - m), seen = (int)((s.end < own + W - 1 ? s.end : own + W - 1) - m);
      const int kept = (int)(s.end - (W - 1) - m);  // the first input that the final state holds
      Chans<VEC> in[W - 1], dp[W];                  // dp[k]: of token t - (W - 1) + k
#pragma unroll
      for (int k = 0; k < W - 1; ++k) in[k] = input_before<IO, W, VEC>(a, s, m, k, c);
#pragma unroll
      for (int k = 0; k < W; ++k) dp[k].fill(0.f);
      Ring ring(sm, seen);
      ring.from(0, static_cast<const IO*>(a.x) + m * a.ldx + c, a.ldx);
      ring.from(1, static_cast<const IO*>(a.dy) + m * a.D + c, a.D);
      IO* out = static_cast<IO*>(a.y) + m * a.D + c;
      const auto meet = [&](typename Ring::P* stage, int u, int t, bool plain) {  // token t
        Chans<VEC> x, g;
        x.from(ring.at(stage, u, 0));
        g.from(ring.at(stage, u, 1));
        if (a.silu) g.times_silu_grad(taps.sum(in, x));
#pragma unroll
        for (int k = 0; k < W - 1; ++k) dp[k] = dp[k + 1];
        dp[W - 1] = g;
        if (plain || t < n) {
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            db.v[e] = add_(db.v[e], g.v[e]);
            dw[W - 1].v[e] = fma_(g.v[e], x.v[e], dw[W - 1].v[e]);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) dw[k].v[e] = fma_(g.v[e], in[k].v[e], dw[k].v[e]);
          }
        }
#pragma unroll
        for (int k = 0; k < W - 2; ++k) in[k] = in[k + 1];
        in[W - 2] = x;
      };
      const auto emit = [&](int o, bool plain) {  // input o, which has met all its tokens
        if (!plain && (o < 0 || o >= n)) return;
        Chans<VEC> dx;
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          V sum = mul_(taps.w[W - 1].v[e], dp[0].v[e]);
#pragma unroll
          for (int k = 1; k < W; ++k) sum = fma_(taps.w[W - 1 - k].v[e], dp[k].v[e], sum);
          dx.v[e] = sum;
        }
        if (!plain && o >= kept && a.dhT) {
          Chans<VEC> f;
          f.from(load_row<IO, VEC>(a.dhT, (long long)s.n * (W - 1) + o - kept, a.D, c));
#pragma unroll
          for (int e = 0; e < kN; ++e) dx.v[e] = add_(dx.v[e], f.v[e]);
        }
        dx.template store<IO>(out, 0);
        out += a.D;
      };
      ring.each(W - 1, n < kept ? n : kept, [&](typename Ring::P* stage, int u, int t, bool plain) {
        meet(stage, u, t, plain);
        emit(t - (W - 1), plain);
      });
      for (int t = seen; t < n + W - 1; ++t) {  // the sequence ended
#pragma unroll
        for (int k = 0; k < W - 1; ++k) dp[k] = dp[k + 1];
        dp[W - 1].fill(0.f);
        emit(t - (W - 1), false);
      }
      m = own > m ? own : stop;
    }
  }
  // the runs of a block that share channels, in order
  __shared__ float sum[kBlock][VEC + 1];
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[threadIdx.x][e] = j < W ? dw[j < W ? j : 0].flat()[e] : db.flat()[e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.lanes * VEC; i += kBlock) {
      const int at = chan * a.lanes * VEC + i;
      if (at >= a.D) continue;
      // (of eight, more only where channels are few: carrying what is rounded off took 2 us more)
      float t = 0.f;
      for (int g = 0; g < groups; ++g) t += sum[g * a.lanes + i / VEC][i % VEC];
      a.part[((size_t)tok * (W + 1) + j) * a.D + at] = t;
    }
  }
}

// dw and db from the partial rows: 32 channels to a block, 32 threads a channel over the
// partial rows, joined in a fixed order by a warp a channel (one after another, carrying
// what is rounded off, took 1 us more).  Beside that, dx behind the last sequence (in the
// kernel before, it cost registers, and odd channel counts 3 us).
template <typename IO, int W>
__global__ void __launch_bounds__(1024) conv_weight_grad_kernel(ConvArgs a) {
  after_previous();
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5, j = blockIdx.y;
  const int i = blockIdx.x * 32 + c;
  if (a.cu && i < a.D) zero_rows<IO, 1>(a, offset_of(a, a.seqs) + j * 32 + g, a.tokens, 32 * (W + 1), i);
  CarriedSum t;
  if (i < a.D)
#pragma unroll 8
    for (int r = g; r < a.parts; r += 32) t.add(a.part[((size_t)r * (W + 1) + j) * a.D + i]);
  s[g][c] = t.sum;
  __syncthreads();
  const float all = lane_sum<32>(s[c][g]);  // of the block's channel g
  const int own = blockIdx.x * 32 + g;
  void* out = j < W ? a.dw : a.db;
  if (c == 0 && own < a.D && out) {
    const size_t at = j < W ? (size_t)own * W + j : own;
    if (a.w_bf16)
      st_io(static_cast<__nv_bfloat16*>(out) + at, all);
    else
      static_cast<float*>(out)[at] = all;
  }
}

// --------------------------------------------------------------- single token
template <typename IO, int W, int VEC>
__global__ void __launch_bounds__(kBlock) conv_step_kernel(ConvArgs a) {
  const int vecs = a.D / VEC;
  const long long i = (long long)blockIdx.x * kBlock + threadIdx.x;
  if (i >= a.tokens * vecs) return;
  const long long row = i / vecs;
  const int c = (int)(i % vecs) * VEC;
  IO* st = static_cast<IO*>(a.hT) + row * (W - 1) * a.D + c;
  Pack<IO, VEC> in[W];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) in[k] = *reinterpret_cast<const Pack<IO, VEC>*>(st + (size_t)k * a.D);
  in[W - 1] = load_row<IO, VEC>(a.x, row, a.ldx, c);
  Taps<W, VEC> taps;
  taps.load(a, c);
  float p[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    p[e] = taps.b.flat()[e];
#pragma unroll
    for (int k = W - 1; k >= 0; --k) p[e] = fmaf(taps.w[k].flat()[e], ld_io(&in[k].v[e]), p[e]);
    if (a.silu) p[e] *= one_plus_inverse(-kLog2e * p[e]);
  }
  store_vec<IO, VEC>(a.y, row * a.D + c, p);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) *reinterpret_cast<Pack<IO, VEC>*>(st + (size_t)k * a.D) = in[k + 1];
}

// ----------------------------------------------------------------- dispatch
inline bool aligned(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
// Threads of a token: a warp, fewer where the channels are fewer.
inline int lanes_of(int vecs) {
  int lanes = 1;
  while (lanes < 32 && lanes < vecs) lanes *= 2;
  return lanes;
}
inline int chan_blocks_of(int D, int vec) {
  const int lanes = lanes_of((D + vec - 1) / vec);
  return (D + lanes * vec - 1) / (lanes * vec);
}
// Tokens of a run: 64 where there are enough for every SM (packed prompts 141 us, by 128
// 140, by 256 147; a training batch's gradients 101 each way), shorter ones else.
inline int run_of(long long tokens, int D, int vec) {
  const int lanes = lanes_of((D + vec - 1) / vec);
  int run = 64;
  while (run > 8 && (tokens + (long long)run * (kBlock / lanes) - 1) / (run * (kBlock / lanes)) *
                            chan_blocks_of(D, vec) < 2 * kSms)
    run /= 2;
  return run;
}
inline long long token_blocks(long long tokens, int D, int vec) {
  const long long per = (long long)run_of(tokens, D, vec) * (kBlock / lanes_of((D + vec - 1) / vec));
  return (tokens + per - 1) / per;
}

template <typename F>
cudaError_t allow_smem(F kernel, size_t smem) {
  if (smem <= 32 * 1024) return cudaSuccess;  // (the static part counts towards the default 48 KB)
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

template <int VEC>
void plan(ConvArgs& a) {
  a.lanes = lanes_of((a.D + VEC - 1) / VEC);
  a.chan_blocks = chan_blocks_of(a.D, VEC);
  a.run = run_of(a.tokens, a.D, VEC);
  a.parts = (int)token_blocks(a.tokens, a.D, VEC);
  a.main_blocks = (long long)a.parts * a.chan_blocks;
}

template <typename IO, int W, int VEC>
cudaError_t run_fwd(ConvArgs a, cudaStream_t s) {
  plan<VEC>(a);
  const long long more =
      a.hT ? blocks_for(((long long)a.seqs * (W - 1) * (a.D / VEC) + kBlock - 1) / kBlock, 2) : 0;
  if (a.main_blocks + more == 0) return cudaSuccess;
  constexpr size_t smem = TokenRing<IO, VEC, 1>::kSmem;
  const cudaError_t e = allow_smem(conv_fwd_kernel<IO, W, VEC>, smem);
  if (e != cudaSuccess) return e;
  conv_fwd_kernel<IO, W, VEC><<<(unsigned)(a.main_blocks + more), kBlock, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename IO, int W, int VEC>
cudaError_t run_bwd(ConvArgs a, cudaStream_t s) {
  plan<VEC>(a);
  const long long more = a.hT ? blocks_for(((long long)a.seqs * a.D + kBlock - 1) / kBlock, 2) : 0;
  constexpr size_t smem = TokenRing<IO, VEC, 2>::kSmem;
  cudaError_t e = allow_smem(conv_bwd_kernel<IO, W, VEC>, smem);
  if (e != cudaSuccess) return e;
  if (a.main_blocks + more > 0)
    conv_bwd_kernel<IO, W, VEC><<<(unsigned)(a.main_blocks + more), kBlock, smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_next(a.main_blocks + more > 0, conv_weight_grad_kernel<IO, W>, dim3((a.D + 31) / 32, W + 1),
                     1024, 0, s, a);
}
template <typename IO, int W, int VEC>
cudaError_t run_step(const ConvArgs& a, cudaStream_t s) {
  const long long n = a.tokens * (a.D / VEC);
  conv_step_kernel<IO, W, VEC><<<(unsigned)((n + kBlock - 1) / kBlock), kBlock, 0, s>>>(a);
  return cudaGetLastError();
}

enum class Call { kFwd, kBwd, kStep };

template <typename IO, int W>
cudaError_t launch_taps(const ConvArgs& a, Call call, cudaStream_t s) {
  constexpr int kWide = 16 / sizeof(IO);
  const auto fits = [&](int vec) {
    const size_t bytes = vec * sizeof(IO);
    return a.D % vec == 0 && a.ldx % vec == 0 && aligned(a.x, bytes) && aligned(a.dy, bytes) &&
           aligned(a.h0, bytes) && aligned(a.dhT, bytes) && aligned(a.y, bytes) && aligned(a.hT, bytes);
  };
  if (call == Call::kFwd) return fits(kVec) ? run_fwd<IO, W, kVec>(a, s) : run_fwd<IO, W, 1>(a, s);
  if (call == Call::kBwd) return fits(kVec) ? run_bwd<IO, W, kVec>(a, s) : run_bwd<IO, W, 1>(a, s);
  return fits(kWide) ? run_step<IO, W, kWide>(a, s) : run_step<IO, W, 1>(a, s);
}
template <typename IO>
cudaError_t launch_io(const ConvArgs& a, int W, Call call, cudaStream_t s) {
  if (W == 2) return launch_taps<IO, 2>(a, call, s);
  if (W == 3) return launch_taps<IO, 3>(a, call, s);
  return launch_taps<IO, 4>(a, call, s);
}
ckda_status launch(const ConvArgs& a, int W, ckda_dtype io, Call call, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = io == CKDA_F32 ? launch_io<float>(a, W, call, s)
                                       : launch_io<__nv_bfloat16>(a, W, call, s);
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

ckda_status check_conv(int B, int T, int D, int W, long long ldx, ckda_dtype io, ckda_dtype wt) {
  if (io != CKDA_F32 && io != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
  if (wt != CKDA_F32 && wt != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
  if (B < 1 || T < 0 || D < 1 || ldx < D) return CKDA_ERR_INVALID_ARG;
  if (W < 2 || W > 4 || D > 1 << 24) return CKDA_ERR_UNSUPPORTED;
  // (tokens and blocks are counted in 32 bits on the grid)
  if ((long long)B * T > 0x7fffffffLL || ldx > 1LL << 31) return CKDA_ERR_UNSUPPORTED;
  if ((long long)B * T * ((D + 31) / 32) > 8LL * 0x7fffffffLL) return CKDA_ERR_UNSUPPORTED;
  return CKDA_OK;
}
ckda_status forward(const void* x, const void* weight, const void* bias, const void* h0, void* y, void* hT,
                    const int32_t* cu_seqlens, int num_seqs, int B, int T, int D, int W, long long ldx,
                    ckda_dtype io_dtype, ckda_dtype weight_dtype, int silu, bool fill, void* stream) {
  const ckda_status st = check_conv(B, T, D, W, ldx, io_dtype, weight_dtype);
  if (st != CKDA_OK) return st;
  if (cu_seqlens && (num_seqs < 1 || B != 1)) return CKDA_ERR_INVALID_ARG;
  if (!weight || (T > 0 && (!x || !y))) return CKDA_ERR_INVALID_ARG;
  const int seqs = cu_seqlens ? num_seqs : B;
  const size_t io = io_dtype == CKDA_F32 ? 4 : 2;
  // blocks that write one of these run beside blocks that still read the other
  const size_t states = (size_t)seqs * (W - 1) * D * io, in = rows_bytes((long long)B * T, D, ldx, io),
               out = rows_bytes((long long)B * T, D, D, io);
  if (overlap(h0, states, hT, states) || overlap(x, in, y, out) || overlap(x, in, hT, states) ||
      overlap(y, out, h0, states) || overlap(y, out, hT, states))
    return CKDA_ERR_INVALID_ARG;
  ConvArgs a{};
  a.x = x; a.w = weight; a.b = bias; a.h0 = h0; a.y = y; a.hT = hT; a.cu = cu_seqlens;
  a.ldx = ldx; a.tokens = (long long)B * T; a.seqs = seqs; a.T = T; a.D = D;
  a.w_bf16 = weight_dtype == CKDA_BF16; a.silu = silu != 0; a.fill = fill;
  return launch(a, W, io_dtype, Call::kFwd, stream);
}

}  // namespace
}  // namespace ckda

using namespace ckda;

extern "C" {

ckda_status ckda_conv_fwd(const void* x, const void* weight, const void* bias, const void* h0,
                          void* y, void* hT, const int32_t* cu_seqlens, int num_seqs, int B, int T,
                          int D, int W, long long ldx, ckda_dtype io_dtype, ckda_dtype weight_dtype,
                          int silu, void* stream) {
  return forward(x, weight, bias, h0, y, hT, cu_seqlens, num_seqs, B, T, D, W, ldx, io_dtype, weight_dtype,
                 silu, false, stream);
}
ckda_status ckda_conv_fwd_filled(const void* x, const void* weight, const void* bias, const void* h0,
                                 void* y, void* hT, const int32_t* cu_seqlens, int num_seqs, int B, int T,
                                 int D, int W, long long ldx, ckda_dtype io_dtype, ckda_dtype weight_dtype,
                                 int silu, void* stream) {
  return forward(x, weight, bias, h0, y, hT, cu_seqlens, num_seqs, B, T, D, W, ldx, io_dtype, weight_dtype,
                 silu, true, stream);
}

size_t ckda_conv_bwd_workspace_bytes(int B, int T, int D, int W) {
  if (B < 1 || T < 0 || D < 1 || W < 2 || W > 4) return 0;
  const long long tokens = (long long)B * T;
  const long long parts = D % kVec == 0 && token_blocks(tokens, D, kVec) > token_blocks(tokens, D, 1)
                              ? token_blocks(tokens, D, kVec)
                              : token_blocks(tokens, D, 1);
  return ((size_t)parts * (W + 1) * D + 4) * sizeof(float);
}

ckda_status ckda_conv_bwd(const void* dy, const void* x, const void* weight, const void* bias,
                          const void* h0, const void* dhT, void* dx, void* dweight, void* dbias,
                          void* dh0, const int32_t* cu_seqlens, int num_seqs, int B, int T, int D,
                          int W, long long ldx, ckda_dtype io_dtype, ckda_dtype weight_dtype,
                          int silu, void* workspace, size_t workspace_bytes, void* stream) {
  const ckda_status st = check_conv(B, T, D, W, ldx, io_dtype, weight_dtype);
  if (st != CKDA_OK) return st;
  if (cu_seqlens && (num_seqs < 1 || B != 1)) return CKDA_ERR_INVALID_ARG;
  if (!weight || !dweight || (T > 0 && (!x || !dy || !dx))) return CKDA_ERR_INVALID_ARG;
  const size_t io = io_dtype == CKDA_F32 ? 4 : 2;
  const size_t states = (size_t)(cu_seqlens ? num_seqs : B) * (W - 1) * D * io,
               in = rows_bytes((long long)B * T, D, ldx, io), out = rows_bytes((long long)B * T, D, D, io);
  if (overlap(x, in, dx, out) || overlap(dy, out, dx, out) || overlap(h0, states, dx, out) ||
      overlap(dhT, states, dx, out) || overlap(h0, states, dh0, states) || overlap(dhT, states, dh0, states) ||
      overlap(x, in, dh0, states) || overlap(dy, out, dh0, states) || overlap(dx, out, dh0, states))
    return CKDA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < ckda_conv_bwd_workspace_bytes(B, T, D, W) || !aligned(workspace, 16))
    return CKDA_ERR_WORKSPACE;
  ConvArgs a{};
  a.x = x; a.dy = dy; a.w = weight; a.b = bias; a.h0 = h0; a.dhT = dhT; a.y = dx; a.hT = dh0;
  a.dw = dweight; a.db = dbias; a.part = static_cast<float*>(workspace); a.cu = cu_seqlens;
  a.ldx = ldx; a.tokens = (long long)B * T; a.seqs = cu_seqlens ? num_seqs : B; a.T = T; a.D = D;
  a.w_bf16 = weight_dtype == CKDA_BF16; a.silu = silu != 0;
  return launch(a, W, io_dtype, Call::kBwd, stream);
}

ckda_status ckda_conv_decode_step(const void* x, const void* weight, const void* bias, void* state,
                                  void* y, int B, int D, int W, long long ldx, ckda_dtype io_dtype,
                                  ckda_dtype weight_dtype, int silu, void* stream) {
  const ckda_status st = check_conv(B, 1, D, W, ldx, io_dtype, weight_dtype);
  if (st != CKDA_OK) return st;
  if (!x || !weight || !state || !y) return CKDA_ERR_INVALID_ARG;
  const size_t io = io_dtype == CKDA_F32 ? 4 : 2, states = (size_t)B * (W - 1) * D * io;
  if (clash(y, x, B, D, ldx, io) || overlap(y, rows_bytes(B, D, D, io), state, states) ||
      overlap(x, rows_bytes(B, D, ldx, io), state, states))
    return CKDA_ERR_INVALID_ARG;
  ConvArgs a{};
  a.x = x; a.w = weight; a.b = bias; a.hT = state; a.y = y;
  a.ldx = ldx; a.tokens = B; a.seqs = B; a.T = 1; a.D = D;
  a.w_bf16 = weight_dtype == CKDA_BF16; a.silu = silu != 0;
  return launch(a, W, io_dtype, Call::kStep, stream);
}

}  // extern "C"
