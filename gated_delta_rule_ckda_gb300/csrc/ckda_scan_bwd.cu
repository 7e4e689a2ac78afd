// ckda_scan_bwd.cu -- gradients of the selective scan.  (The formulas of the forward pass
// and a block's work: ckda_scan.cuh.)
//
// With dy' = dy silu(z), a_t = exp(delta_t A) and G the gradient that reaches h_t from
// later tokens (from hT's at a sequence's end):
//     g = G + dy' C,   G <- a g   (at a sequence's start: dh0)
//     dC += dy' h_t,   dB += g u   (sums over a group's channels)
//     q = a g h_{t-1},   dA += q delta
//     dx = delta <g, B> + D dy',   ddelta = <q, A> + <g, B> x,   dz = dy (<C, h> + D x) silu'(z)
//     ddt = ddelta sigmoid(dt + dt_bias) with the softplus, else ddelta
//
// h cannot be run backward (it would be divided by decays), so a first pass walks the
// tokens forward and leaves the state before every 8th one in the workspace; the second
// takes the 8-token chunks in reverse: runs a chunk forward from its state, h and a kept
// in registers, then backward.  That is two exponentials a state for the whole call.
// Rows with few channels are cut into pieces: the first pass then also leaves what each
// piece adds to the gradient that passes it, and a scan joins both directions.
//
// <.,.> are sums over the LP lanes of a channel, dB and dC over the other lanes of the
// warp, then over the block's warps in shared memory; the blocks' parts go through the
// workspace and are added in a fixed order, as are dA's, dD's and ddt_bias's.
#include "ckda_scan.cuh"

namespace ckda {
namespace {

constexpr int kChunk = 8;
constexpr int kWarps = kScanBlock / 32;

struct BwdArgs {
  ScanArgs a;
  const void* dy;
  const float* dhT;
  void* dx;
  void* ddt;
  void* dz;
  void* dB;
  void* dC;
  float* dA;
  float* dskip;
  float* dbias;
  float* dh0;
  float* chunk;      // [rows][chunks][D][N]: states before chunks, from the piece's own start
  float* chunk_sum;  // [rows][chunks][D]: steps from the piece's start to the chunk (pieces > 1)
  float* grad;       // [rows][pieces][D][N]: what a piece adds to G, then the G that reaches its end
  float* part_bc;    // [blocks of a group][rows][T][G][2][N]: dC, dB
  float* part_a;     // [rows][pieces][D][N]
  float* part_d;     // [rows][pieces][2][D]: dD, ddt_bias
  int chunks;        // of a row
};

__device__ __forceinline__ float silu_slope(float z, float g) { return g * fmaf(z, 1.f - g, 1.f); }

// -------------------------------------------------- first pass: states and sums
// GRADS: the pieces' sums of gradients too (more than one piece).
template <typename IO, typename S, bool VEC, bool GRADS>
__global__ void __launch_bounds__(kScanBlock) scan_states_kernel(BwdArgs b) {
  constexpr int LP = S::kLanes, NS = S::kStates, K = S::K, NP = S::NP;
  constexpr int kPairs = NS / 2;
  const ScanArgs& a = b.a;
  __shared__ __align__(16) float4 in[K][S::kRow];  // delta, u, dy'
  __shared__ __align__(16) float sB[K * NP], sC[GRADS ? K * NP : 4];
  __shared__ Marks<K> marks;
  let_next_start();
  const ScanPlace p = scan_place<S::CH>(a);
  if (p.t0 >= p.t1) return;
  const int tid = threadIdx.x, l = tid % LP, pos = tid / LP;
  const int k1 = tid / S::V8, v1 = tid % S::V8;
  float bias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    bias[e] = 8 * v1 + e < p.chans && a.dt_bias ? a.dt_bias[p.c0 + 8 * v1 + e] : 0.f;
  const int c = S::chan_at(pos);
  const bool have = c < p.chans;
  const long long chan = p.c0 + (have ? c : 0);
  float2 A2[kPairs], h[kPairs], G[kPairs], W[kPairs];  // W: product of decays from the piece's start
  load_states<NS>(A2, a.A, chan, a.N, l * NS, have);
#pragma unroll
  for (int q = 0; q < kPairs; ++q) {
    A2[q] = mul_(A2[q], both<float2>(kLog2e));
    h[q] = G[q] = both<float2>(0.f);
    W[q] = both<float2>(1.f);
  }
  float span = 0.f;
  ScanSeq seq = scan_seq_at(a, p.row, p.t0);
  bool first = seq.begin < p.t0;  // in the sequence that entered the piece
  const long long unit = (long long)p.row * a.pieces + p.piece;

  struct Raw {
    Eight<IO> x, dt, dy, z;
    GroupTile<IO, S> B, C;
  } next;
  const auto load = [&](int t) {
    const int count = p.t1 - t;
    const long long at = (long long)p.row * a.T + t;
    if (k1 < K && k1 < count) {
      const int cc = p.c0 + 8 * v1, n = p.chans - 8 * v1;
      next.x.template load<VEC>(a.x, (at + k1) * a.ldx + cc, n);
      next.dt.template load<VEC>(a.dt, (at + k1) * a.lddt + cc, n);
      if (GRADS) {
        next.dy.template load<VEC>(b.dy, (at + k1) * a.D + cc, n);
        if (a.z) next.z.template load<VEC>(a.z, (at + k1) * a.ldz + cc, n);
      }
    }
    next.B.template load<VEC>(a.B, a.ldb, at, count < K ? count : K, p.g, a.N);
    if (GRADS) next.C.template load<VEC>(a.C, a.ldc, at, count < K ? count : K, p.g, a.N);
  };
  load(p.t0);
  for (int t = p.t0; t < p.t1; t += K) {
    const int count = p.t1 - t < K ? p.t1 - t : K;
    if (k1 < K) {
      float delta[8];
      step_sizes(next.dt, bias, a.softplus, k1 < count, delta);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool ok = k1 < count && 8 * v1 + e < p.chans;
        float dy = GRADS && ok ? next.dy.at(e) : 0.f;
        if (GRADS && ok && a.z) dy *= scan_silu(next.z.at(e));
        in[k1][e * S::V8 + v1] = make_float4(delta[e], ok ? delta[e] * next.x.at(e) : 0.f, dy, 0.f);
      }
    }
    next.B.template leave<VEC>(sB, count, a.N);
    if (GRADS) next.C.template leave<VEC>(sC, count, a.N);
    const bool edges = t <= seq.begin || t + count >= seq.end;
    if (edges) marks.fill(a, p.row, t, count);
    __syncthreads();
    if (t + K < p.t1) load(t + K);
    const auto walk = [&](auto checked) {
      constexpr bool kChecked = decltype(checked)::value;
#pragma unroll 1
      for (int k0 = 0; k0 < count; k0 += kChunk) {
        const long long ck = (long long)p.row * b.chunks + (t + k0) / kChunk;
        store_states<NS>(b.chunk, ck * a.D + chan, a.N, l * NS, have, h);
        if (GRADS && l == 0 && have) b.chunk_sum[ck * a.D + chan] = span;
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          const int k = k0 + i;
          const int mark = kChecked ? marks.mark[k] : 0;
          if (kChecked && (mark & 1)) {
            first = false;
            if (a.h0)
              load_states<NS>(h, a.h0, (long long)marks.n[k] * a.D + chan, a.N, l * NS, have);
            else
#pragma unroll
              for (int q = 0; q < kPairs; ++q) h[q] = both<float2>(0.f);
          }
          const float4 s = in[k][pos];
          float2 Bk[kPairs], Ck[kPairs];
          from_shared<NS>(Bk, sB + k * NP + l * NS);
          if (GRADS) from_shared<NS>(Ck, sC + k * NP + l * NS);
          part += s.x;
#pragma unroll
          for (int q = 0; q < kPairs; ++q) {
            const float2 decay = ex2(mul_(both<float2>(s.x), A2[q]));
            h[q] = fma_(decay, h[q], mul_(both<float2>(s.y), Bk[q]));
            if (GRADS && first) {
              W[q] = mul_(W[q], decay);
              G[q] = fma_(W[q], mul_(both<float2>(s.z), Ck[q]), G[q]);
            }
          }
          if (GRADS && kChecked && (mark & 2) && first && b.dhT) {
            float2 last[kPairs];
            load_states<NS>(last, b.dhT, (long long)marks.n[k] * a.D + chan, a.N, l * NS, have);
#pragma unroll
            for (int q = 0; q < kPairs; ++q) G[q] = fma_(W[q], last[q], G[q]);
          }
        }
        span += part;
      }
    };
    if (edges)
      walk(std::true_type());
    else
      walk(std::false_type());
    if (t + count >= seq.end && t + count < p.t1) seq = scan_seq_at(a, p.row, t + count);
    __syncthreads();
  }
  if (GRADS) {
    store_states<NS>(a.state, unit * a.D + chan, a.N, l * NS, have, h);
    store_states<NS>(b.grad, unit * a.D + chan, a.N, l * NS, have, G);
    if (l == 0 && have) a.span[unit * a.D + chan] = span;
  }
}

// The gradient that reaches each piece's end, from what the pieces behind it add: a
// thread a state, from the last piece to the first.
__global__ void __launch_bounds__(256) scan_join_grads_kernel(BwdArgs b) {
  after_previous();
  let_next_start();
  const ScanArgs& a = b.a;
  const long long per = (long long)a.D * a.N;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.rows * per) return;
  const int row = (int)(i / per), last = scan_last(a);
  const int d = (int)(i % per / a.N);
  const float rate = a.A[i % per];
  float g = 0.f;
  for (int s = a.pieces - 1; s >= 0; --s) {
    const int t0 = s * a.piece_len;
    if (t0 >= last) continue;
    const int t1 = t0 + a.piece_len < last ? t0 + a.piece_len : last;
    const long long unit = (long long)row * a.pieces + s;
    const float own = b.grad[unit * per + i % per];
    b.grad[unit * per + i % per] = g;
    if (scan_seq_at(a, row, t0).begin >= t0)
      g = 0.f;
    else
      g = passes(a, row, t0, t1) ? fmaf(expf(rate * a.span[unit * a.D + d]), g, own) : own;
  }
}

// ------------------------------------------------------ second pass: gradients
template <typename IO, typename S>
struct GradSmem {
  Eight<IO> raw[2][4][kScanBlock];       // x, dt, dy, z of a tile, each thread's own
  float4 slot[S::K][S::kRow];            // delta, u, dy'; then delta, <g, B>, <C, h>, <q, A>
  float B[S::K * S::NP], C[S::K * S::NP];
  float red[kWarps][S::K][2 * S::NP];    // dC, dB of the warps' channels
  float bias[S::CH], skip[S::CH];
  Marks<S::K> marks;
};

template <typename IO, typename S, bool VEC>
__global__ void __launch_bounds__(kScanBlock) scan_grad_kernel(BwdArgs b) {
  constexpr int LP = S::kLanes, NS = S::kStates, K = S::K, NP = S::NP;
  constexpr int kPairs = NS / 2, kChanLanes = 32 / LP, kV = 16 / sizeof(IO);
  static_assert(S::kChans == 1 && K % kChunk == 0, "a channel to a thread, whole chunks");
  extern __shared__ __align__(16) char sm[];
  GradSmem<IO, S>& s = *reinterpret_cast<GradSmem<IO, S>*>(sm);
  const ScanArgs& a = b.a;
  after_previous();
  let_next_start();
  const ScanPlace p = scan_place<S::CH>(a);
  const int tid = threadIdx.x, l = tid % LP, pos = tid / LP, warp = tid / 32, ci = tid % 32 / LP;
  const int k1 = tid / S::V8, v1 = tid % S::V8;
  const long long unit = (long long)p.row * a.pieces + p.piece;
  const int c = S::chan_at(pos);
  const bool have = c < p.chans;
  const long long chan = p.c0 + (have ? c : 0);
  if (p.piece == 0 && b.dh0 && (a.cu || a.T == 0)) empty_states<S::CH>(a, p, b.dhT, b.dh0);

  float2 A2[kPairs], g[kPairs], dA[kPairs];
  load_states<NS>(A2, a.A, chan, a.N, l * NS, have);
#pragma unroll
  for (int q = 0; q < kPairs; ++q) {
    A2[q] = mul_(A2[q], both<float2>(kLog2e));
    g[q] = dA[q] = both<float2>(0.f);
  }
  float dskip[8], dbias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dskip[e] = dbias[e] = 0.f;

  if (p.t0 < p.t1) {
    for (int i = tid; i < S::CH; i += kScanBlock) {
      s.bias[i] = i < p.chans && a.dt_bias ? a.dt_bias[p.c0 + i] : 0.f;
      s.skip[i] = i < p.chans && a.skip ? a.skip[p.c0 + i] : 0.f;
    }
    __syncthreads();
    if (a.pieces > 1) load_states<NS>(g, b.grad, unit * a.D + chan, a.N, l * NS, have);
    const int tiles = (p.t1 - p.t0 + K - 1) / K;
    const auto fetch = [&](int tile, int stage) {  // a thread's own vectors of a tile
      const int t = p.t0 + tile * K;
      if (k1 < K && t + k1 < p.t1) {
        const long long at = (long long)p.row * a.T + t + k1;
        const int cc = p.c0 + 8 * v1, n = p.chans - 8 * v1;
        const auto one = [&](int which, const void* base, long long from) {
          Eight<IO>& to = s.raw[stage][which][tid];
          if (VEC) {
            if (n > 0)
#pragma unroll
              for (int j = 0; j < 8 / kV; ++j)
                copy_async<16>(&to.v[j], static_cast<const IO*>(base) + from + j * kV);
          } else {
            to.template load<false>(base, from, n);
          }
        };
        one(0, a.x, at * a.ldx + cc);
        one(1, a.dt, at * a.lddt + cc);
        one(2, b.dy, at * a.D + cc);
        if (a.z) one(3, a.z, at * a.ldz + cc);
      }
      copy_commit();
    };
    GroupTile<IO, S> nextB, nextC;
    const auto fetch_bc = [&](int tile) {
      const int t = p.t0 + tile * K, count = p.t1 - t < K ? p.t1 - t : K;
      const long long at = (long long)p.row * a.T + t;
      nextB.template load<VEC>(a.B, a.ldb, at, count, p.g, a.N);
      nextC.template load<VEC>(a.C, a.ldc, at, count, p.g, a.N);
    };
    fetch(tiles - 1, 0);
    fetch_bc(tiles - 1);
    int stage = 0;
    for (int tile = tiles - 1; tile >= 0; --tile, stage ^= 1) {
      const int t = p.t0 + tile * K, count = p.t1 - t < K ? p.t1 - t : K;
      if (tile > 0)
        fetch(tile - 1, stage ^ 1);
      else
        copy_commit();
      copy_wait<1>();
      // ---- 1
      Eight<IO>* raw = &s.raw[stage][0][tid];  // raw[which * kScanBlock]
      if (k1 < K) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool ok = k1 < count && 8 * v1 + e < p.chans;
          float delta = 0.f, u = 0.f, dy = 0.f;
          if (ok) {
            const float r = raw[kScanBlock].at(e) + s.bias[8 * v1 + e];
            delta = a.softplus ? softplus(r) : r;
            u = delta * raw[0].at(e);
            dy = raw[2 * kScanBlock].at(e);
            if (a.z) dy *= scan_silu(raw[3 * kScanBlock].at(e));
          }
          s.slot[k1][e * S::V8 + v1] = make_float4(delta, u, dy, 0.f);
        }
      }
      nextB.template leave<VEC>(s.B, count, a.N);
      nextC.template leave<VEC>(s.C, count, a.N);
      const ScanSeq seq = scan_seq_at(a, p.row, t);
      const bool edges = t <= seq.begin || t + count >= seq.end;
      if (edges) s.marks.fill(a, p.row, t, count);
      __syncthreads();
      if (tile > 0) fetch_bc(tile - 1);
      // ---- 2
      float2 dA_tile[kPairs];
#pragma unroll
      for (int q = 0; q < kPairs; ++q) dA_tile[q] = both<float2>(0.f);
      const auto walk = [&](auto checked) {
        constexpr bool kChecked = decltype(checked)::value;
#pragma unroll 1
        for (int k0 = (count - 1) / kChunk * kChunk; k0 >= 0; k0 -= kChunk) {
          const long long ck = (long long)p.row * b.chunks + (t + k0) / kChunk;
          float2 h[kPairs], old[kChunk][kPairs], decay[kChunk][kPairs];
          load_states<NS>(h, b.chunk, ck * a.D + chan, a.N, l * NS, have);
          const int begin = kChecked ? scan_seq_at(a, p.row, t + k0).begin : seq.begin;
          if (a.pieces > 1 && begin < p.t0) {  // what entered the piece reaches here
            float2 enter[kPairs];
            load_states<NS>(enter, a.state, unit * a.D + chan, a.N, l * NS, have);
            const float span = have ? b.chunk_sum[ck * a.D + chan] : 0.f;
#pragma unroll
            for (int q = 0; q < kPairs; ++q)
              h[q] = fma_(ex2(mul_(both<float2>(span), A2[q])), enter[q], h[q]);
          }
#pragma unroll
          for (int i = 0; i < kChunk; ++i) {
            const int k = k0 + i;
            if (kChecked && (s.marks.mark[k] & 1)) {
              if (a.h0)
                load_states<NS>(h, a.h0, (long long)s.marks.n[k] * a.D + chan, a.N, l * NS, have);
              else
#pragma unroll
                for (int q = 0; q < kPairs; ++q) h[q] = both<float2>(0.f);
            }
            const float2 step = *reinterpret_cast<const float2*>(&s.slot[k][pos]);
            float2 Bk[kPairs];
            from_shared<NS>(Bk, s.B + k * NP + l * NS);
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
              old[i][q] = h[q];
              decay[i][q] = ex2(mul_(both<float2>(step.x), A2[q]));
              h[q] = fma_(decay[i][q], h[q], mul_(both<float2>(step.y), Bk[q]));
            }
          }
          float yC[kChunk], gB[kChunk], qA[kChunk];
#pragma unroll
          for (int i = kChunk - 1; i >= 0; --i) {
            const int k = k0 + i;
            const int mark = kChecked ? s.marks.mark[k] : 0;
            if (kChecked && (mark & 2)) {
              if (b.dhT)
                load_states<NS>(g, b.dhT, (long long)s.marks.n[k] * a.D + chan, a.N, l * NS, have);
              else
#pragma unroll
                for (int q = 0; q < kPairs; ++q) g[q] = both<float2>(0.f);
            }
            const float4 in = s.slot[k][pos];
            float2 Bk[kPairs], Ck[kPairs];
            from_shared<NS>(Bk, s.B + k * NP + l * NS);
            from_shared<NS>(Ck, s.C + k * NP + l * NS);
            float sums[2 * NS];
            float2 y = both<float2>(0.f), gb = y, qa = y;
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
              // (a sequence's start between leaves its own initial state in old[i + 1])
              const float2 now = kChecked ? fma_(decay[i][q], old[i][q], mul_(both<float2>(in.y), Bk[q]))
                                 : i + 1 < kChunk ? old[i + 1 < kChunk ? i + 1 : i][q] : h[q];
              const float2 dyv = both<float2>(in.z);
              g[q] = fma_(dyv, Ck[q], g[q]);
              y = fma_(Ck[q], now, y);
              gb = fma_(g[q], Bk[q], gb);
              const float2 dC = mul_(dyv, now), dB = mul_(g[q], both<float2>(in.y));
              sums[2 * q] = dC.x;
              sums[2 * q + 1] = dC.y;
              sums[NS + 2 * q] = dB.x;
              sums[NS + 2 * q + 1] = dB.y;
              g[q] = mul_(g[q], decay[i][q]);
              const float2 through = mul_(g[q], old[i][q]);
              qa = fma_(through, A2[q], qa);
              dA_tile[q] = fma_(through, both<float2>(in.x), dA_tile[q]);
            }
            yC[i] = y.x + y.y;
            gB[i] = gb.x + gb.y;
            qA[i] = qa.x + qa.y;
            if (kChecked && (mark & 1)) {
              if (b.dh0)
                store_states<NS>(b.dh0, (long long)s.marks.n[k] * a.D + chan, a.N, l * NS, have, g);
#pragma unroll
              for (int q = 0; q < kPairs; ++q) g[q] = both<float2>(0.f);
            }
            fold_values<2 * NS, kChanLanes, LP>(sums, ci);
            constexpr int kEach = 2 * NS > kChanLanes ? 2 * NS / kChanLanes : 1;
            if (ci * kEach < 2 * NS)
#pragma unroll
              for (int e = 0; e < kEach; ++e) {
                const int at = ci * kEach + e;
                s.red[warp][k][at / NS * NP + l * NS + at % NS] = sums[e];
              }
          }
          fold_values<kChunk, LP, 1>(yC, l);
          fold_values<kChunk, LP, 1>(gB, l);
          fold_values<kChunk, LP, 1>(qA, l);
          __syncwarp();  // the channel's lanes have read their slots
          constexpr int kEach = kChunk > LP ? kChunk / LP : 1;
          if (l * kEach < kChunk)
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
              float4& to = s.slot[k0 + l * kEach + e][pos];
              to.y = gB[e];
              to.z = yC[e];
              to.w = qA[e];
            }
        }
      };
      if (edges)
        walk(std::true_type());
      else
        walk(std::false_type());
#pragma unroll
      for (int q = 0; q < kPairs; ++q) dA[q] = add_(dA[q], dA_tile[q]);
      __syncthreads();
      // ---- 3
      if (k1 < K && k1 < count) {
        const long long at = ((long long)p.row * a.T + t + k1) * a.D + p.c0 + 8 * v1;
        const int n = p.chans - 8 * v1;
        float dx[8], ddt[8], dz[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dx[e] = ddt[e] = dz[e] = 0.f;
          if (e >= n) continue;
          const float4 r = s.slot[k1][e * S::V8 + v1];
          const float x = raw[0].at(e), dy = raw[2 * kScanBlock].at(e), skip = s.skip[8 * v1 + e];
          float up = dy;
          if (a.z) {
            const float z = raw[3 * kScanBlock].at(e), gate = scan_sigmoid(z);
            up = dy * (z * gate);
            dz[e] = dy * fmaf(skip, x, r.z) * silu_slope(z, gate);
          }
          dx[e] = fmaf(r.x, r.y, skip * up);
          ddt[e] = fmaf(r.w, 1.f / kLog2e, r.y * x);
          if (a.softplus) ddt[e] *= scan_sigmoid(raw[kScanBlock].at(e) + s.bias[8 * v1 + e]);
          dskip[e] = fmaf(up, x, dskip[e]);
          dbias[e] += ddt[e];
        }
        store_eight<IO, VEC>(b.dx, at, n, dx);
        store_eight<IO, VEC>(b.ddt, at, n, ddt);
        if (a.z) store_eight<IO, VEC>(b.dz, at, n, dz);
      }
      // the warps' parts of dC and dB
      const int cb = (int)(blockIdx.x % a.chan_blocks) % (a.chan_blocks / a.G);
      float* out = b.part_bc + (((long long)cb * a.rows + p.row) * a.T + t) * a.G * 2 * a.N;
      for (int i = tid; i < count * 2 * NP; i += kScanBlock) {
        const int k = i / (2 * NP), w = i % (2 * NP) / NP, n = i % NP;
        if (n >= a.N) continue;
        float sum = 0.f;
#pragma unroll
        for (int w4 = 0; w4 < kWarps; ++w4) sum += s.red[w4][k][w * NP + n];
        out[((long long)k * a.G + p.g) * 2 * a.N + w * a.N + n] = sum;
      }
      __syncthreads();
    }
  }
  store_states<NS>(b.part_a, unit * a.D + chan, a.N, l * NS, have, dA);
  // dD and ddt_bias: the threads of a vector, in order, through shared memory
  float* join = reinterpret_cast<float*>(sm);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) join[e * kScanBlock + tid] = which ? dbias[e] : dskip[e];
    __syncthreads();
    for (int i = tid; i < p.chans; i += kScanBlock) {
      float sum = 0.f;
      for (int k = 0; k < K; ++k) sum += join[i % 8 * kScanBlock + k * S::V8 + i / 8];
      b.part_d[(unit * 2 + which) * a.D + p.c0 + i] = sum;
    }
  }
}

// dB, dC: sums over the blocks of a group; dA, dD, ddt_bias: over the rows' pieces.
template <typename IO>
__global__ void __launch_bounds__(256) scan_sums_kernel(BwdArgs b, long long bc_blocks) {
  after_previous();
  const ScanArgs& a = b.a;
  if (blockIdx.x < bc_blocks) {
    const long long per = (long long)a.rows * a.T * a.G * 2 * a.N;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= per) return;
    const long long tg = i / (2 * a.N);
    const int w = (int)(i % (2 * a.N)) / a.N, n = (int)(i % a.N);
    if ((int)(tg / a.G % a.T) >= scan_last(a)) return;
    const int blocks = a.chan_blocks / a.G;
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < blocks; ++k) s += b.part_bc[k * per + i];
    st_io(static_cast<IO*>(w ? b.dB : b.dC) + tg * a.N + n, s);
    return;
  }
  const long long i = ((long long)blockIdx.x - bc_blocks) * 256 + threadIdx.x;
  const long long dn = (long long)a.D * a.N;
  const int units = a.rows * a.pieces;
  if (i < dn) {
    float s = 0.f;
#pragma unroll 8
    for (int u = 0; u < units; ++u) s += b.part_a[u * dn + i];
    b.dA[i] = s;
  } else if (i < dn + 2 * a.D) {
    const int w = (int)((i - dn) / a.D), d = (int)((i - dn) % a.D);
    float* out = w ? b.dbias : b.dskip;
    if (!out) return;
    float s = 0.f;
#pragma unroll 8
    for (int u = 0; u < units; ++u) s += b.part_d[(u * 2LL + w) * a.D + d];
    out[d] = s;
  }
}

// ----------------------------------------------------------------- dispatch
template <typename IO, typename S, bool VEC>
cudaError_t run(BwdArgs b, cudaStream_t s) {
  ScanArgs& a = b.a;
  const int dg = a.D / a.G;
  a.chan_blocks = a.G * ((dg + S::CH - 1) / S::CH);
  const unsigned grid = (unsigned)((long long)a.rows * a.pieces * a.chan_blocks);
  cudaError_t e = cudaSuccess;
  if (a.pieces > 1) {
    e = launch_next(false, scan_states_kernel<IO, S, VEC, true>, grid, kScanBlock, 0, s, b);
    if (e == cudaSuccess) e = launch_scan_join(true, a, s);
    const long long n = (long long)a.rows * a.D * a.N;
    if (e == cudaSuccess)
      e = launch_next(true, scan_join_grads_kernel, (unsigned)((n + 255) / 256), 256, 0, s, b);
  } else {
    e = launch_next(false, scan_states_kernel<IO, S, VEC, false>, grid, kScanBlock, 0, s, b);
  }
  if (e != cudaSuccess) return e;
  const auto kernel = scan_grad_kernel<IO, S, VEC>;
  constexpr size_t smem = sizeof(GradSmem<IO, S>);
  static_assert(smem >= 8 * kScanBlock * sizeof(float), "the last sums go through it");
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  e = launch_next(true, kernel, grid, kScanBlock, smem, s, b);
  if (e != cudaSuccess) return e;
  const long long bc = ((long long)a.rows * a.T * a.G * 2 * a.N + 255) / 256;
  const long long ad = ((long long)a.D * (a.N + 2) + 255) / 256;
  return launch_next(true, scan_sums_kernel<IO>, dim3((unsigned)(bc + ad)), 256, 0, s, b, bc);
}

template <typename IO, bool VEC>
cudaError_t by_states(const BwdArgs& b, cudaStream_t s) {
  const int N = b.a.N;
  if (N <= 4) return run<IO, ScanShape<1, 4, 1>, VEC>(b, s);
  if (N <= 8) return run<IO, ScanShape<2, 4, 1>, VEC>(b, s);
  if (N <= 16) return run<IO, ScanShape<4, 4, 1>, VEC>(b, s);
  if (N <= 32) return run<IO, ScanShape<8, 4, 1, 32>, VEC>(b, s);
  return run<IO, ScanShape<16, 4, 1, 16>, VEC>(b, s);
}
inline int block_chans(int N) { return N <= 4 ? 128 : N <= 8 ? 64 : N <= 16 ? 32 : N <= 32 ? 16 : 8; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename IO>
cudaError_t launch_io(const BwdArgs& b, cudaStream_t s) {
  constexpr int kV = 16 / sizeof(IO);
  const ScanArgs& a = b.a;
  const bool whole = a.N == 4 || a.N == 8 || a.N == 16 || a.N == 32 || a.N == 64;
  const bool vec = a.D / a.G % 8 == 0 && whole && a.ldx % kV == 0 && a.lddt % kV == 0 &&
                   (!a.z || a.ldz % kV == 0) && a.ldb % 4 == 0 && a.ldc % 4 == 0 && aligned16(a.x) &&
                   aligned16(a.dt) && aligned16(a.z) && aligned16(a.B) && aligned16(a.C) &&
                   aligned16(b.dy) && aligned16(b.dx) && aligned16(b.ddt) && aligned16(b.dz);
  return vec ? by_states<IO, true>(b, s) : by_states<IO, false>(b, s);
}

// The workspace's parts, in order, each a multiple of 256 bytes.
struct Layout {
  int pieces, len, chunks;
  size_t chunk, chunk_sum, state, span, grad, part_bc, part_a, part_d, bytes;
};
Layout layout_of(int rows, int T, int D, int N, int G) {
  Layout w{};
  const int ch = block_chans(N), dg = D / G;
  scan_pieces(rows, T, D, G, ch, 3 * kSms, &w.pieces, &w.len);
  w.chunks = (T + kChunk - 1) / kChunk;
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
  w.part_bc = take((size_t)((dg + ch - 1) / ch) * rows * T * G * 2 * N * 4);
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
  if (!workspace || workspace_bytes < w.bytes || !aligned16(workspace)) return CKDA_ERR_WORKSPACE;
  if ((long long)B * T * G * 2 * N / 256 + (long long)D * (N + 2) / 256 + 2 > 0x7fffffffLL)
    return CKDA_ERR_UNSUPPORTED;
  char* ws = static_cast<char*>(workspace);
  const auto part = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
  BwdArgs b{};
  ScanArgs& a = b.a;
  a.x = x; a.dt = dt; a.B = Bm; a.C = C; a.z = z; a.A = A; a.skip = D_skip; a.dt_bias = dt_bias;
  a.h0 = h0; a.cu = cu_seqlens;
  a.ldx = ldx; a.lddt = lddt; a.ldb = ldb; a.ldc = ldc; a.ldz = ldz;
  a.rows = B; a.T = T; a.D = D; a.N = N; a.G = G; a.seqs = cu_seqlens ? num_seqs : B;
  a.softplus = softplus != 0;
  a.pieces = w.pieces; a.piece_len = w.len;
  a.state = part(w.state); a.span = part(w.span);
  b.dy = dy; b.dhT = dhT; b.dx = dx; b.ddt = ddt; b.dz = dz; b.dB = dBm; b.dC = dC; b.dA = dA;
  b.dskip = dD_skip; b.dbias = ddt_bias; b.dh0 = dh0;
  b.chunk = part(w.chunk); b.chunk_sum = part(w.chunk_sum); b.grad = part(w.grad);
  b.part_bc = part(w.part_bc); b.part_a = part(w.part_a); b.part_d = part(w.part_d);
  b.chunks = w.chunks;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = io_dtype == CKDA_F32 ? launch_io<float>(b, s) : launch_io<__nv_bfloat16>(b, s);
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // extern "C"
