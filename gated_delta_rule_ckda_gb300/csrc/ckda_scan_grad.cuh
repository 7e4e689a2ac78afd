// ckda_scan_grad.cuh -- gradients of the selective scan.  (The formulas of the forward pass
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
// half of each forward twice, which costs more than the memory's traffic.)
// Rows with few channels are cut into pieces: the first walk then also leaves what each
// piece adds to the gradient that passes it, and a scan joins both directions.
//
// A lane has a channel, as in the forward pass; up to 16 states at a time are spread over
// LP lanes, more in turns (slices).  <.,.> go to their own lane by shuffles; dB and dC are
// sums over a lane's channels, then over the other lanes of the warp; a warp's parts go
// through the workspace and are added in a fixed order, as are dA's, dD's and ddt_bias's,
// each carrying along what its additions round off.
//
// Bound, like the forward pass, by fma and exponentials on few warps (255 registers leave
// two to a scheduler): 4 x 2048 tokens of 4096 channels of 16 states take 1181 us, 257 of
// them the walk, 867 the gradients (issue 44% of the cycles, fma pipe 35%), 28 the sums of
// dB's and dC's parts; memory 71.  Chunks of 8 tokens, half of them run forward twice,
// took 1350; three blocks an SM with 0.9 KB of a thread's registers in local memory 1620.
#pragma once
#include "ckda_scan.cuh"

namespace ckda {

struct ScanBwdArgs {
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
static __global__ void __launch_bounds__(256) scan_join_grads_kernel(ScanBwdArgs b) {
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
constexpr int kGradTile = 2 * kScanChunk, kSumTiles = 64;

// Of a warp; behind it, per slice of 4 LP states, [LP][32] float4 each of A log2(e), of G
// and of dA, each lane's own.
template <typename IO, typename S, bool SLICES>
struct GradSmem {
  alignas(16) ChanTile<IO, kGradTile> raw[2][4];  // x, dt, dy, z
  float4 slot[kGradTile][kScanChans];             // delta, u, dy'; then delta, <g, B>, <C, h>, <q, A>
  float sums[SLICES ? kGradTile : 1][3][kScanChans];  // the last three, over the slices so far
  float4 state[2][S::kLanes][kScanChans];     // states before the two chunks, each lane's own
  float before[2][kScanChans];                // steps before them
};
template <typename IO, int MOST>
struct GradGroups {  // B and C of a tile, MOST states
  GroupTile<IO, kGradTile, MOST> raw[2][2];
  alignas(16) float f[2][kGradTile * MOST];
};

// MOST: states, padded; in slices of S::NP.
template <typename IO, typename S, int MOST, bool VEC>
__global__ void __launch_bounds__(kScanBlock, 8 / kScanWarps) scan_grad_kernel(ScanBwdArgs b) {
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
  if (a.cu) {
    zero_behind<IO>(a, p, b.dx);
    zero_behind<IO>(a, p, b.ddt);
    if (a.z) zero_behind<IO>(a, p, b.dz);
  }
  // Sums over a piece's tokens, in fp32: dD's and ddt_bias's over a tile, then with what the
  // addition to the rest rounded off carried along; dA's over kSumTiles tiles, then in memory.
  CarriedSum dskip, dbias;
  bool summed = false;
  const auto put_dA = [&]() {
#pragma unroll
    for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
      for (int j = 0; j < LP; ++j) {
        float2 f[kPairs], more[kPairs];
        from_vec(f, w.dA[sl][j][lane]);
        if (summed) {
          load_states<NS>(more, b.part_a, unit * a.D + chan(j), a.N, sl * NP + l * NS, have(j));
#pragma unroll
          for (int q = 0; q < kPairs; ++q) f[q] = add_(f[q], more[q]);
        }
        store_states<NS>(b.part_a, unit * a.D + chan(j), a.N, sl * NP + l * NS, have(j), f);
        w.dA[sl][j][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    summed = true;
  };
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
    const int tiles = (p.t1 - p.t0 + kGradTile - 1) / kGradTile;
    constexpr bool kAsync = kScanAsync<IO, VEC>;
    const auto fetch = [&](int tile, int stage) {  // a tile's inputs
      const int t = p.t0 + tile * kGradTile, count = p.t1 - t < kGradTile ? p.t1 - t : kGradTile;
      const long long at = (long long)p.row * a.T + t;
      if constexpr (kAsync) {
        s.raw[stage][0].template fetch<VEC>(a.x, a.ldx, at, p.c0, count, p.chans);
        s.raw[stage][1].template fetch<VEC>(a.dt, a.lddt, at, p.c0, count, p.chans);
        s.raw[stage][2].template fetch<VEC>(a.dy, a.D, at, p.c0, count, p.chans);
        if (a.z) s.raw[stage][3].template fetch<VEC>(a.z, a.ldz, at, p.c0, count, p.chans);
        w.bc.raw[stage][0].template fetch<VEC>(a.B, a.ldb, at, count, p.g, a.N);
        w.bc.raw[stage][1].template fetch<VEC>(a.C, a.ldc, at, count, p.g, a.N);
      } else {  // (no registers to hold them beside the recurrence)
        HeldChans<IO, kGradTile> held[4];
        HeldGroups<IO, kGradTile, MOST> held_bc[2];
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
        const int t = p.t0 + tile * kGradTile + i * kScanChunk;
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
      const int t = p.t0 + tile * kGradTile, count = p.t1 - t < kGradTile ? p.t1 - t : kGradTile;
      if (!kAsync && tile + 1 < tiles) fetch(tile, stage);
      copy_wait<0>();
      __syncwarp();
      const bool whole = count == kGradTile && p.chans == kScanChans;
      // ---- the lane's own channel: steps, and dy through the gate
#pragma unroll
      for (int k = 0; k < kGradTile; k += 2) {
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
      if (tile % kSumTiles == 0 && tile > 0) put_dA();
      // ---- the lane's own channel: its gradients
      float tile_skip = 0.f, tile_bias = 0.f;
      const long long at = ((long long)p.row * a.T + t) * a.D + c;
#pragma unroll
      for (int k = 0; k < kGradTile; k += 2) {
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
          tile_skip = fmaf(up.x, x.x, tile_skip);
          tile_bias += ddt.x;
          st_io(static_cast<IO*>(b.dx) + at + (long long)k * a.D, dx.x);
          st_io(static_cast<IO*>(b.ddt) + at + (long long)k * a.D, ddt.x);
          if (a.z) st_io(static_cast<IO*>(b.dz) + at + (long long)k * a.D, dz.x);
        }
        if (own && k + 1 < count) {
          tile_skip = fmaf(up.y, x.y, tile_skip);
          tile_bias += ddt.y;
          st_io(static_cast<IO*>(b.dx) + at + (long long)(k + 1) * a.D, dx.y);
          st_io(static_cast<IO*>(b.ddt) + at + (long long)(k + 1) * a.D, ddt.y);
          if (a.z) st_io(static_cast<IO*>(b.dz) + at + (long long)(k + 1) * a.D, dz.y);
        }
      }
      dskip.add(tile_skip);
      dbias.add(tile_bias);
    }
  }
  put_dA();
  if (own) {
    b.part_d[unit * 2 * a.D + c] = dskip.sum;
    b.part_d[(unit * 2 + 1) * a.D + c] = dbias.sum;
  }
}

// dB, dC: sums over the blocks of a group; dA, dD, ddt_bias: over the rows' pieces.
template <typename IO>
__global__ void __launch_bounds__(256) scan_sums_kernel(ScanBwdArgs b, long long bc_blocks) {
  after_previous();
  const ScanArgs& a = b.a;
  if (blockIdx.x < bc_blocks) {
    const long long per = (long long)a.rows * a.T * a.G * 2 * a.N;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= per) return;
    const long long tg = i / (2 * a.N);
    const int w = (int)(i % (2 * a.N)) / a.N, n = (int)(i % a.N);
    // (behind the last sequence there are no parts, and the sum is zero)
    const int blocks = (int)(tg / a.G % a.T) < scan_last(a) ? a.chan_blocks / a.G : 0;
    CarriedSum s;  // (eight at a time: the batch's gradients take 1185 us, one by one 1199)
    int k = 0;
    for (; k + 8 <= blocks; k += 8) {
      float few = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) few += b.part_bc[(k + e) * per + i];
      s.add(few);
    }
    for (; k < blocks; ++k) s.add(b.part_bc[k * per + i]);
    st_io(static_cast<IO*>(w ? b.dB : b.dC) + tg * a.N + n, s.sum);
    return;
  }
  const long long i = ((long long)blockIdx.x - bc_blocks) * 256 + threadIdx.x;
  const long long dn = (long long)a.D * a.N;
  const int units = a.rows * a.pieces;
  if (i < dn) {
    CarriedSum s;
#pragma unroll 8
    for (int u = 0; u < units; ++u) s.add(b.part_a[u * dn + i]);
    b.dA[i] = s.sum;
  } else if (i < dn + 2 * a.D) {
    const int w = (int)((i - dn) / a.D), d = (int)((i - dn) % a.D);
    float* out = w ? b.dbias : b.dskip;
    if (!out) return;
    CarriedSum s;
#pragma unroll 8
    for (int u = 0; u < units; ++u) s.add(b.part_d[(u * 2LL + w) * a.D + d]);
    out[d] = s.sum;
  }
}

// ----------------------------------------------------------------- dispatch
// S1: of the walk forward; S2 and MOST: of the gradients.
template <typename IO, typename S1, typename S2, int MOST, bool VEC>
cudaError_t run_scan_grads(ScanBwdArgs b, cudaStream_t s) {
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
cudaError_t scan_grads_by_states(const ScanBwdArgs& b, cudaStream_t s) {
  const int N = b.a.N;
  if (N <= 4) return run_scan_grads<IO, ScanShape<1, 4>, ScanShape<1, 4>, 4, VEC>(b, s);
  if (N <= 8) return run_scan_grads<IO, ScanShape<2, 4>, ScanShape<2, 4>, 8, VEC>(b, s);
  if (N <= 16) return run_scan_grads<IO, ScanShape<2, 8>, ScanShape<4, 4>, 16, VEC>(b, s);
  if (N <= 32) return run_scan_grads<IO, ScanShape<4, 8>, ScanShape<4, 4>, 32, VEC>(b, s);
  return run_scan_grads<IO, ScanShape<8, 8>, ScanShape<4, 4>, 64, VEC>(b, s);
}

// The whole backward pass in an I/O type (a file for each, to compile beside each other).
template <typename IO>
cudaError_t launch_scan_grads(const ScanBwdArgs& b, cudaStream_t s) {
  return scan_vectors(b.a, sizeof(IO)) ? scan_grads_by_states<IO, true>(b, s) : scan_grads_by_states<IO, false>(b, s);
}
extern template cudaError_t launch_scan_grads<float>(const ScanBwdArgs& b, cudaStream_t s);
extern template cudaError_t launch_scan_grads<__nv_bfloat16>(const ScanBwdArgs& b, cudaStream_t s);

}  // namespace ckda
