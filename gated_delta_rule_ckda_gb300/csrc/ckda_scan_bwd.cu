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
// h cannot be run backward (it would be divided by decays), so a first walk forward leaves
// the state before every 4th token in the workspace; the second pass takes these chunks in
// reverse: it runs forward from a chunk's state, the states before its tokens kept in
// registers, then backward over them.  (Chunks of 8 tokens halve the workspace and run
// half of each forward twice, which cost more than the memory's traffic.)
// Rows with few channels are cut into pieces: the first walk then also leaves what each
// piece adds to the gradient that passes it, and a scan joins both directions.
//
// A lane has a channel, as in the forward pass; up to 16 states at a time are spread over
// LP lanes, more in turns (slices).  <.,.> go to their own lane by shuffles; dB and dC are
// sums over a lane's channels, then over the other lanes of the warp; a warp's parts go
// through the workspace and are added in a fixed order, as are dA's, dD's and ddt_bias's.
#include "ckda_scan.cuh"

namespace ckda {
namespace {


struct BwdArgs {
  ScanArgs a;
  void* dx;
  void* ddt;
  void* dz;
  void* dB;
  void* dC;
  float* dA;
  float* dskip;
  float* dbias;
  float* dh0;
  float* part_bc;  // [channel blocks of a group][rows][T][G][2][N]: dC, dB
  float* part_a;   // [rows][pieces][D][N]
  float* part_d;   // [rows][pieces][2][D]: dD, ddt_bias
};

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
  for (int s0 = a.pieces - 1; s0 >= 0; s0 -= 4) {
    float own[4], sum[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s0 - k >= 0 && (s0 - k) * a.piece_len < last) {
        const long long unit = (long long)row * a.pieces + s0 - k;
        own[k] = a.grad[unit * per + i % per];
        sum[k] = a.span[unit * a.D + d];
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (s0 - k < 0) return;
      const int t0 = (s0 - k) * a.piece_len;
      if (t0 >= last) continue;
      const int t1 = t0 + a.piece_len < last ? t0 + a.piece_len : last;
      a.grad[((long long)row * a.pieces + s0 - k) * per + i % per] = g;
      if (scan_seq_at(a, row, t0).begin >= t0)
        g = 0.f;
      else
        g = passes(a, row, t0, t1) ? fmaf(expf(rate * sum[k]), g, own[k]) : own[k];
    }
  }
}

// ------------------------------------------------------ second pass: gradients
constexpr int kTile = 2 * kScanChunk;

// Of a warp; behind it, per slice of 4 LP states, [LP][32] float4 each of A log2(e), of G
// and of dA, each lane's own.
template <typename IO, typename S, bool SLICES>
struct GradSmem {
  alignas(16) ChanTile<IO, kTile> raw[2][4];  // x, dt, dy, z
  float4 slot[kTile][kScanChans];             // delta, u, dy'; then delta, <g, B>, <C, h>, <q, A>
  float sums[SLICES ? kTile : 1][3][kScanChans];  // the last three, over the slices so far
  float4 state[2][S::kLanes][kScanChans];     // states before the two chunks, each lane's own
  float before[2][kScanChans];                // steps before them
};
template <typename IO, int MOST>
struct GradGroups {  // B and C of a tile, MOST states
  GroupTile<IO, kTile, MOST> raw[2][2];
  alignas(16) float f[2][kTile * MOST];
};

// MOST: states, padded; in slices of S::NP.
template <typename IO, typename S, int MOST, bool VEC>
__global__ void __launch_bounds__(kScanBlock, 2) scan_grad_kernel(BwdArgs b) {
  constexpr int LP = S::kLanes, NS = S::kStates, NP = S::NP, kPairs = NS / 2, kGroups = 32 / LP;
  constexpr int kSlices = MOST / NP;
  static_assert(NS == 4, "a lane's states of a channel are one vector");
  using Smem = GradSmem<IO, S, (kSlices > 1)>;
  struct Own {
    Smem s;
    GradGroups<IO, MOST> bc;
    float4 A2[kSlices][LP][32], g[kSlices][LP][32], dA[kSlices][LP][32];
  };
  extern __shared__ __align__(16) char sm[];
  Own& w = reinterpret_cast<Own*>(sm)[threadIdx.x >> 5];
  Smem& s = w.s;
  const ScanArgs& a = b.a;
  after_previous();
  let_next_start();
  ScanPlace p;
  if (!scan_place(a, p)) return;
  const int lane = threadIdx.x & 31, l = lane % LP, grp = lane / LP;
  const long long unit = (long long)p.row * a.pieces + p.piece;
  const bool own = lane < p.chans;
  const int c = p.c0 + (own ? lane : 0);
  const auto have = [&](int j) { return (lane ^ j) < p.chans; };
  const auto chan = [&](int j) { return p.c0 + (have(j) ? lane ^ j : 0); };
  const auto vec = [](const float2 (&f)[kPairs]) { return make_float4(f[0].x, f[0].y, f[1].x, f[1].y); };
  const auto from_vec = [](float2 (&f)[kPairs], const float4& v) {
    f[0] = make_float2(v.x, v.y);
    f[1] = make_float2(v.z, v.w);
  };
  if (p.piece == 0 && b.dh0 && (a.cu || a.T == 0)) empty_states(a, p, a.dhT, b.dh0);
  float dskip = 0.f, dbias = 0.f;
#pragma unroll
  for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
    for (int j = 0; j < LP; ++j) {
      float2 f[kPairs], zero[kPairs] = {both<float2>(0.f), both<float2>(0.f)};
      load_states<NS>(f, a.A, chan(j), a.N, sl * NP + l * NS, have(j));
#pragma unroll
      for (int q = 0; q < kPairs; ++q) f[q] = mul_(f[q], both<float2>(kLog2e));
      w.A2[sl][j][lane] = vec(f);
      w.g[sl][j][lane] = w.dA[sl][j][lane] = vec(zero);
      if (a.pieces > 1 && p.t0 < p.t1) {
        load_states<NS>(f, a.grad, unit * a.D + chan(j), a.N, sl * NP + l * NS, have(j));
        w.g[sl][j][lane] = vec(f);
      }
      s.state[0][j][lane] = s.state[1][j][lane] = vec(zero);  // (lanes without a channel read what nothing writes)
    }

  if (p.t0 < p.t1) {
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.skip ? a.skip[c] : 0.f;
    const int tiles = (p.t1 - p.t0 + kTile - 1) / kTile;
    constexpr bool kAsync = kScanAsync<IO, VEC>;
    const auto fetch = [&](int tile, int stage) {  // a tile's inputs
      const int t = p.t0 + tile * kTile, count = p.t1 - t < kTile ? p.t1 - t : kTile;
      const long long at = (long long)p.row * a.T + t;
      if constexpr (kAsync) {
        s.raw[stage][0].template fetch<VEC>(a.x, a.ldx, at, p.c0, count, p.chans);
        s.raw[stage][1].template fetch<VEC>(a.dt, a.lddt, at, p.c0, count, p.chans);
        s.raw[stage][2].template fetch<VEC>(a.dy, a.D, at, p.c0, count, p.chans);
        if (a.z) s.raw[stage][3].template fetch<VEC>(a.z, a.ldz, at, p.c0, count, p.chans);
        w.bc.raw[stage][0].template fetch<VEC>(a.B, a.ldb, at, count, p.g, a.N);
        w.bc.raw[stage][1].template fetch<VEC>(a.C, a.ldc, at, count, p.g, a.N);
      } else {  // (no registers to hold them beside the recurrence)
        HeldChans<IO, kTile> held[4];
        HeldGroups<IO, kTile, MOST> held_bc[2];
        held[0].load(a.x, a.ldx, at, p.c0, count, p.chans);
        held[1].load(a.dt, a.lddt, at, p.c0, count, p.chans);
        held[2].load(a.dy, a.D, at, p.c0, count, p.chans);
        if (a.z) held[3].load(a.z, a.ldz, at, p.c0, count, p.chans);
        held_bc[0].load(a.B, a.ldb, at, count, p.g, a.N);
        held_bc[1].load(a.C, a.ldc, at, count, p.g, a.N);
#pragma unroll
        for (int i = 0; i < 4; ++i) held[i].leave(s.raw[stage][i]);
        held_bc[0].leave(w.bc.raw[stage][0]);
        held_bc[1].leave(w.bc.raw[stage][1]);
      }
      copy_commit();
    };
    const auto fetch_states = [&](int tile, int sl) {  // the states before its chunks
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = p.t0 + tile * kTile + i * kScanChunk;
        if (t >= p.t1) break;
        const long long ck = (long long)p.row * a.chunks + t / kScanChunk;
#pragma unroll
        for (int j = 0; j < LP; ++j) {
          if (VEC) {
            if (have(j) && sl * NP + l * NS < a.N)
              copy_async<16>(&s.state[i][j][lane], a.chunk + (ck * a.D + chan(j)) * a.N + sl * NP + l * NS);
          } else {
#pragma unroll
            for (int e = 0; e < NS; ++e)
              if (have(j) && sl * NP + l * NS + e < a.N)
                copy_async<4>(reinterpret_cast<float*>(&s.state[i][j][lane]) + e,
                              a.chunk + (ck * a.D + chan(j)) * a.N + sl * NP + l * NS + e);
          }
        }
        if (a.pieces > 1 && sl == 0) copy_async<4>(&s.before[i][lane], a.chunk_sum + ck * a.D + c);
      }
      copy_commit();
    };
    fetch(tiles - 1, 0);
    fetch_states(tiles - 1, 0);
    int stage = 0;
    for (int tile = tiles - 1; tile >= 0; --tile, stage ^= 1) {
      const int t = p.t0 + tile * kTile, count = p.t1 - t < kTile ? p.t1 - t : kTile;
      if (!kAsync && tile + 1 < tiles) fetch(tile, stage);
      copy_wait<0>();
      __syncwarp();
      const bool whole = count == kTile && p.chans == kScanChans;
      // ---- the lane's own channel: steps, and dy through the gate
#pragma unroll
      for (int k = 0; k < kTile; k += 2) {
        float2 x = s.raw[stage][0].pair(k), up = s.raw[stage][2].pair(k);
        float2 d = step_sizes(s.raw[stage][1].pair(k), both<float2>(bias), a.softplus);
        if (a.z) up = mul_(up, scan_silu(s.raw[stage][3].pair(k)));
        if (!whole) {  // (what there is not was not loaded)
          const bool in0 = own && k < count, in1 = own && k + 1 < count;
          d = make_float2(in0 ? d.x : 0.f, in1 ? d.y : 0.f);
          x = make_float2(in0 ? x.x : 0.f, in1 ? x.y : 0.f);
          up = make_float2(in0 ? up.x : 0.f, in1 ? up.y : 0.f);
        }
        const float2 u = mul_(d, x);
        s.slot[k][lane] = make_float4(d.x, u.x, up.x, 0.f);
        s.slot[k + 1][lane] = make_float4(d.y, u.y, up.y, 0.f);
      }
      w.bc.raw[stage][0].template unpack_to<VEC>(w.bc.f[0], count, a.N);
      w.bc.raw[stage][1].template unpack_to<VEC>(w.bc.f[1], count, a.N);
      const ScanSeq seq = scan_seq_at(a, p.row, t);
      const bool edges = t <= seq.begin || t + count >= seq.end;
      Marks marks;
      if (edges) marks.find(a, p.row, t, count);
      __syncwarp();
      if (kAsync && tile > 0) fetch(tile - 1, stage ^ 1);
      float* const out_bc = b.part_bc + ((((long long)p.block * a.rows + p.row) * a.T + t) * a.G + p.g) * 2 * a.N;
      const long long apart_bc = (long long)a.G * 2 * a.N;
      // ---- a slice of the states
      const auto walk = [&](auto checked, int sl) {
        constexpr bool kChecked = decltype(checked)::value;
        const int n0 = sl * NP + l * NS;
        float2 A2[LP][kPairs], g[LP][kPairs], dA[LP][kPairs], h[LP][kPairs];
#pragma unroll
        for (int j = 0; j < LP; ++j) {
          from_vec(A2[j], w.A2[sl][j][lane]);
          from_vec(g[j], w.g[sl][j][lane]);
#pragma unroll
          for (int q = 0; q < kPairs; ++q) dA[j][q] = both<float2>(0.f);
        }
        const auto reset = [&](int k) {  // a sequence starts at token k
          const int num = marks.number(k);
#pragma unroll
          for (int j = 0; j < LP; ++j) {
            if (a.h0)
              load_states<NS>(h[j], a.h0, (long long)num * a.D + chan(j), a.N, n0, have(j));
            else
#pragma unroll
              for (int q = 0; q < kPairs; ++q) h[j][q] = both<float2>(0.f);
          }
        };
#pragma unroll 1
        for (int k0 = (count - 1) / kScanChunk * kScanChunk; k0 >= 0; k0 -= kScanChunk) {
          const int ch = k0 / kScanChunk;
#pragma unroll
          for (int j = 0; j < LP; ++j) from_vec(h[j], s.state[ch][j][lane]);
          const int begin = kChecked ? scan_seq_at(a, p.row, t + k0).begin : seq.begin;
          if (a.pieces > 1 && begin < p.t0) {  // what entered the piece reaches the chunk
#pragma unroll
            for (int j = 0; j < LP; ++j) {
              float2 enter[kPairs];
              load_states<NS>(enter, a.state, unit * a.D + chan(j), a.N, n0, have(j));
              const float2 span = both<float2>(s.before[ch][lane ^ j]);
#pragma unroll
              for (int q = 0; q < kPairs; ++q) h[j][q] = fma_(decay_of(span, A2[j][q]), enter[q], h[j][q]);
            }
          }
          if (k0 == 0) {  // (the states are read: the next ones)
            __syncwarp();
            if (sl + 1 < kSlices)
              fetch_states(tile, sl + 1);
            else if (tile > 0)
              fetch_states(tile - 1, 0);
          }
          float2 old[kScanChunk][LP][kPairs];
#pragma unroll
          for (int i = 0; i < kScanChunk; ++i) {
            const int k = k0 + i;
            if (kChecked && (marks.first >> k & 1)) reset(k);
            float2 Bk[kPairs];
            from_shared<NS>(Bk, w.bc.f[0] + k * MOST + n0);
#pragma unroll
            for (int j = 0; j < LP; ++j) {
              const float2 in = *reinterpret_cast<const float2*>(&s.slot[k][lane ^ j]);
#pragma unroll
              for (int q = 0; q < kPairs; ++q) {
                old[i][j][q] = h[j][q];
                h[j][q] = fma_(decay_of(both<float2>(in.x), A2[j][q]), h[j][q], mul_(both<float2>(in.y), Bk[q]));
              }
            }
          }
          float found[kScanChunk][3];  // <g, B>, <C, h>, <q, A> of the lane's own channel
#pragma unroll
          for (int i = kScanChunk - 1; i >= 0; --i) {
            const int k = k0 + i;
            const bool first = kChecked && (marks.first >> k & 1), last = kChecked && (marks.last >> k & 1);
            const int num = kChecked && (first || last) ? marks.number(k) : 0;
            if (last) {
#pragma unroll
              for (int j = 0; j < LP; ++j) {
                if (a.dhT)
                  load_states<NS>(g[j], a.dhT, (long long)num * a.D + chan(j), a.N, n0, have(j));
                else
#pragma unroll
                  for (int q = 0; q < kPairs; ++q) g[j][q] = both<float2>(0.f);
              }
            }
            float2 Bk[kPairs], Ck[kPairs], sumC[kPairs], sumB[kPairs];
            from_shared<NS>(Bk, w.bc.f[0] + k * MOST + n0);
            from_shared<NS>(Ck, w.bc.f[1] + k * MOST + n0);
#pragma unroll
            for (int j = 0; j < LP; ++j) {
              const float4 in = s.slot[k][lane ^ j];
              const float2 delta = both<float2>(in.x), u = both<float2>(in.y), up = both<float2>(in.z);
              float2 y, gb, qa;
#pragma unroll
              for (int q = 0; q < kPairs; ++q) {
                const float2 decay = decay_of(delta, A2[j][q]);
                // (a sequence's start between leaves its own initial state in old[i + 1])
                const float2 now = kChecked ? fma_(decay, old[i][j][q], mul_(u, Bk[q]))
                                   : i + 1 < kScanChunk ? old[i + 1 < kScanChunk ? i + 1 : i][j][q] : h[j][q];
                g[j][q] = fma_(up, Ck[q], g[j][q]);
                y = q == 0 ? mul_(Ck[q], now) : fma_(Ck[q], now, y);
                gb = q == 0 ? mul_(g[j][q], Bk[q]) : fma_(g[j][q], Bk[q], gb);
                sumC[q] = j == 0 ? mul_(up, now) : fma_(up, now, sumC[q]);
                sumB[q] = j == 0 ? mul_(g[j][q], u) : fma_(g[j][q], u, sumB[q]);
                g[j][q] = mul_(g[j][q], decay);
                const float2 through = mul_(g[j][q], old[i][j][q]);
                qa = q == 0 ? mul_(through, A2[j][q]) : fma_(through, A2[j][q], qa);
                dA[j][q] = fma_(through, delta, dA[j][q]);
              }
              const float s0 = gb.x + gb.y, s1 = y.x + y.y, s2 = qa.x + qa.y;
              found[i][0] = j ? found[i][0] + __shfl_xor_sync(0xffffffffu, s0, j) : s0;
              found[i][1] = j ? found[i][1] + __shfl_xor_sync(0xffffffffu, s1, j) : s1;
              found[i][2] = j ? found[i][2] + __shfl_xor_sync(0xffffffffu, s2, j) : s2;
              if (first) {
                if (b.dh0) store_states<NS>(b.dh0, (long long)num * a.D + chan(j), a.N, n0, have(j), g[j]);
#pragma unroll
                for (int q = 0; q < kPairs; ++q) g[j][q] = both<float2>(0.f);
              }
            }
            float sums[2 * NS] = {sumC[0].x, sumC[0].y, sumC[1].x, sumC[1].y,
                                  sumB[0].x, sumB[0].y, sumB[1].x, sumB[1].y};
            fold_values<2 * NS, kGroups, LP>(sums, grp);
            constexpr int kSums = 2 * NS > kGroups ? 2 * NS / kGroups : 1;
            if (grp * kSums < 2 * NS && k < count)
#pragma unroll
              for (int e = 0; e < kSums; ++e) {
                const int at = grp * kSums + e, n = n0 + at % NS;
                if (n < a.N) out_bc[k * apart_bc + at / NS * a.N + n] = sums[e];
              }
          }
          if (kSlices == 1) {
            __syncwarp();  // the lanes have read these slots
#pragma unroll
            for (int i = 0; i < kScanChunk; ++i) {
              float* to = &s.slot[k0 + i][lane].y;
              to[0] = found[i][0];
              to[1] = found[i][1];
              to[2] = found[i][2];
            }
          } else {
#pragma unroll
            for (int i = 0; i < kScanChunk; ++i)
#pragma unroll
              for (int f = 0; f < 3; ++f) {
                float& to = s.sums[kSlices > 1 ? k0 + i : 0][f][lane];
                to = sl == 0 ? found[i][f] : to + found[i][f];
              }
          }
        }
#pragma unroll
        for (int j = 0; j < LP; ++j) {
          w.g[sl][j][lane] = vec(g[j]);
          float4& to = w.dA[sl][j][lane];
          to = make_float4(to.x + dA[j][0].x, to.y + dA[j][0].y, to.z + dA[j][1].x, to.w + dA[j][1].y);
        }
      };
#pragma unroll 1
      for (int sl = 0; sl < kSlices; ++sl) {
        if (sl > 0) copy_wait<0>();
        if (edges)
          walk(std::true_type(), sl);
        else
          walk(std::false_type(), sl);
      }
      // ---- the lane's own channel: its gradients
      const long long at = ((long long)p.row * a.T + t) * a.D + c;
#pragma unroll
      for (int k = 0; k < kTile; k += 2) {
        const float4 r0 = s.slot[k][lane], r1 = s.slot[k + 1][lane];
        const float2 delta = make_float2(r0.x, r1.x);
        float2 gB, yC, qA;
        if (kSlices == 1) {
          gB = make_float2(r0.y, r1.y);
          yC = make_float2(r0.z, r1.z);
          qA = make_float2(r0.w, r1.w);
        } else {
          const int k2 = kSlices > 1 ? k : 0, k3 = kSlices > 1 ? k + 1 : 0;
          gB = make_float2(s.sums[k2][0][lane], s.sums[k3][0][lane]);
          yC = make_float2(s.sums[k2][1][lane], s.sums[k3][1][lane]);
          qA = make_float2(s.sums[k2][2][lane], s.sums[k3][2][lane]);
        }
        const float2 x = s.raw[stage][0].pair(k);
        float2 up = s.raw[stage][2].pair(k), dz = both<float2>(0.f);
        if (a.z) {
          const float2 z = s.raw[stage][3].pair(k), gate = scan_sigmoid(z), dy = up;
          // silu'(z) = gate (1 + z (1 - gate))
          const float2 slope = mul_(gate, fma_(z, fma_(gate, both<float2>(-1.f), both<float2>(1.f)), both<float2>(1.f)));
          up = mul_(dy, mul_(z, gate));
          dz = mul_(mul_(dy, fma_(both<float2>(skip), x, yC)), slope);
        }
        const float2 dx = fma_(delta, gB, mul_(both<float2>(skip), up));
        float2 ddt = fma_(gB, x, mul_(qA, both<float2>(1.f / kLog2e)));
        if (a.softplus) ddt = mul_(ddt, scan_sigmoid(add_(s.raw[stage][1].pair(k), both<float2>(bias))));
        if (own && k < count) {
          dskip = fmaf(up.x, x.x, dskip);
          dbias += ddt.x;
          st_io(static_cast<IO*>(b.dx) + at + (long long)k * a.D, dx.x);
          st_io(static_cast<IO*>(b.ddt) + at + (long long)k * a.D, ddt.x);
          if (a.z) st_io(static_cast<IO*>(b.dz) + at + (long long)k * a.D, dz.x);
        }
        if (own && k + 1 < count) {
          dskip = fmaf(up.y, x.y, dskip);
          dbias += ddt.y;
          st_io(static_cast<IO*>(b.dx) + at + (long long)(k + 1) * a.D, dx.y);
          st_io(static_cast<IO*>(b.ddt) + at + (long long)(k + 1) * a.D, ddt.y);
          if (a.z) st_io(static_cast<IO*>(b.dz) + at + (long long)(k + 1) * a.D, dz.y);
        }
      }
    }
  }
#pragma unroll
  for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
    for (int j = 0; j < LP; ++j) {
      float2 f[kPairs];
      from_vec(f, w.dA[sl][j][lane]);
      store_states<NS>(b.part_a, unit * a.D + chan(j), a.N, sl * NP + l * NS, have(j), f);
    }
  if (own) {
    b.part_d[unit * 2 * a.D + c] = dskip;
    b.part_d[(unit * 2 + 1) * a.D + c] = dbias;
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
// S1: of the walk forward; S2 and MOST: of the gradients.
template <typename IO, typename S1, typename S2, int MOST, bool VEC>
cudaError_t run(BwdArgs b, cudaStream_t s) {
  ScanArgs& a = b.a;
  a.chan_blocks = scan_chan_blocks(a.D, a.G);
  cudaError_t e = cudaSuccess;
  if (a.pieces > 1) {
    e = launch_walk<IO, S1, VEC, kGrads>(false, a, s);
    if (e == cudaSuccess) e = launch_scan_join(true, a, s);
    const long long n = (long long)a.rows * a.D * a.N;
    if (e == cudaSuccess)
      e = launch_next(true, scan_join_grads_kernel, (unsigned)((n + 255) / 256), 256, 0, s, b);
  } else {
    e = launch_walk<IO, S1, VEC, kChunks>(false, a, s);
  }
  if (e != cudaSuccess) return e;
  const auto kernel = scan_grad_kernel<IO, S2, MOST, VEC>;
  constexpr int kSlices = MOST / S2::NP;
  constexpr size_t smem = kScanWarps * (sizeof(GradSmem<IO, S2, (kSlices > 1)>) + sizeof(GradGroups<IO, MOST>) +
                                        3 * kSlices * S2::kLanes * 32 * sizeof(float4));
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  e = launch_next(true, kernel, scan_grid(a), kScanBlock, smem, s, b);
  if (e != cudaSuccess) return e;
  const long long bc = ((long long)a.rows * a.T * a.G * 2 * a.N + 255) / 256;
  const long long ad = ((long long)a.D * (a.N + 2) + 255) / 256;
  return launch_next(true, scan_sums_kernel<IO>, dim3((unsigned)(bc + ad)), 256, 0, s, b, bc);
}

template <typename IO, bool VEC>
cudaError_t by_states(const BwdArgs& b, cudaStream_t s) {
  const int N = b.a.N;
  if (N <= 4) return run<IO, ScanShape<1, 4>, ScanShape<1, 4>, 4, VEC>(b, s);
  if (N <= 8) return run<IO, ScanShape<2, 4>, ScanShape<2, 4>, 8, VEC>(b, s);
  if (N <= 16) return run<IO, ScanShape<2, 8>, ScanShape<4, 4>, 16, VEC>(b, s);
  if (N <= 32) return run<IO, ScanShape<4, 8>, ScanShape<4, 4>, 32, VEC>(b, s);
  return run<IO, ScanShape<8, 8>, ScanShape<4, 4>, 64, VEC>(b, s);
}

template <typename IO>
cudaError_t launch_io(const BwdArgs& b, cudaStream_t s) {
  return scan_vectors(b.a, sizeof(IO)) ? by_states<IO, true>(b, s) : by_states<IO, false>(b, s);
}

// The workspace's parts, in order, each a multiple of 256 bytes.
struct Layout {
  int pieces, len, chunks;
  size_t chunk, chunk_sum, state, span, grad, part_bc, part_a, part_d, bytes;
};
Layout layout_of(int rows, int T, int D, int N, int G) {
  Layout w{};
  scan_pieces(rows, T, D, G, 24 * kSms, &w.pieces, &w.len);
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
  BwdArgs b{};
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = io_dtype == CKDA_F32 ? launch_io<float>(b, s) : launch_io<__nv_bfloat16>(b, s);
  return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // extern "C"
