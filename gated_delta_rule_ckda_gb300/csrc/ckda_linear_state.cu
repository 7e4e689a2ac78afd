// ckda_linear_state.cu -- the states of chunked linear attention: the state
// entering every chunk for the backward pass, and the segments that long
// sequences are cut into.
#include "ckda_linear_chunk.cuh"

namespace ckda {
namespace {
using namespace chunk;

// ----------------------------------------------------------- states of chunks
// One CTA of 512 threads walks the chunks of one (sequence, head), or of one
// segment of it, forward over (k, v) or backward over (q, do).  IMAGES: it
// starts from the state entering it and writes the state met at each chunk
// and, backward, dh0: two tiles in and an image out, 128 KiB a chunk.  8 x 16 x 2048
// tokens: 42 us a direction for 268 MB, of which 210 MB pass DRAM (58 to 62% of its peak;
// tensor pipe 21%): 128 of 152 SMs, with the tiles of two chunks in flight each.
// Otherwise it starts from zero (at the sequence's end from h0 or dhT) and writes the one
// state that it hands on.
//   warp 0 loads, warp 1 issues the products, warp 2 makes the decays,
//   warps 4-7 scale a chunk's keys (queries) in two bf16 parts,
//   warps 8-15 hold the state: thread (r, s) has its channels 64 s .. + 63 of
//   value column r in fp32 registers.  They stage the image in shared memory
//   and one bulk copy writes it (rows written by their own threads would take
//   an L1 pass for every 16 bytes).
namespace st {
constexpr int kThreads = 512;
constexpr int kSlots = 4;                       // x and y tiles of two chunks
constexpr uint32_t kLo = kSlots * kTile;        // lo part of the scaled tile
constexpr uint32_t kStage = kLo + kTile;        // the image on its way out
constexpr uint32_t kGates = kStage + kImage;
constexpr uint32_t kBars = kGates + sizeof(Gates);
constexpr uint32_t kSmem = kBars + 512;
static_assert(kSmem <= 232448, "shared memory of a CTA");
enum { B_FULL = 0, B_EMPTY = 4, B_KT = 8, B_DF, B_DFREE = B_DF + 2, B_G = B_DFREE + 2, B_GFREE,
       B_END, B_COUNT };
}  // namespace st

// KP: panels of 64 key channels.  Of an image only the panels and value rows that
// exist are written.
template <bool BACK, bool IMAGES, int KP>
__global__ void __launch_bounds__(st::kThreads, 1)
linear_state_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ Split sp,
                    const __grid_constant__ ChunkImages images,
                    const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my) {
  using namespace st;
  extern __shared__ __align__(1024) char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kBars);
  Gates* gates = reinterpret_cast<Gates*>(sm + kGates);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + kBars + 400);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sm + kBars + 404);
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!IMAGES) {
    after_previous();
    let_next_start();
  }
  if (sb & 1023u) {
    if (tid == 0) set_status(a.status, CKDA_ERR_CUDA);
    return;
  }
  // the grid is a bound; without images, only the segments at cuts run
  unsigned block = blockIdx.x;
  if (!IMAGES && a.cu_seqlens) {
    if ((int)(block / a.H) >= sp.item0[a.N + 2]) return;
    block = (sp.cuts[block / a.H].y + (BACK ? 1 : 0)) * a.H + block % a.H;
  }
  if (block >= pieces(a, sp)) return;
  const Piece u = piece_of(a, sp, block);
  // the first segment in this direction, and the one that hands nothing on
  const bool starts = BACK ? u.seg == u.segs - 1 : u.seg == 0;
  const bool ends = BACK ? u.seg == 0 : u.seg == u.segs - 1;
  if (!IMAGES && ends) return;
  const int t0 = u.t0, len = u.len, chunks = u.chunks, xz = u.qz, yz = u.vz;
  const size_t vrow = (size_t)yz * a.T + t0;
  const size_t states = (size_t)a.dk * a.dv, state = ((size_t)u.n * a.H + u.h) * states;
  const float* init = BACK ? a.dhT : a.h0;
  const float* from = starts   ? (init ? init + state : nullptr)
                      : IMAGES ? sp.state + ((size_t)(u.item + (BACK ? 1 : -1)) * a.H + u.h) * states
                               : nullptr;
  auto at = [&](int i) { return BACK ? chunks - 1 - i : i; };  // chunk of step i
  // forward, no chunk of this segment is entered by what its last one leaves
  const int steps = BACK || !IMAGES ? chunks : chunks - 1;

  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i)
      mbar_init(bars + i, i == B_KT                         ? 4
                          : i >= B_DFREE && i < B_DFREE + 2 ? 8
                          : i == B_GFREE                    ? 12
                                                            : 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc(tmem_at, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;

  if (warp == 0) {
    if (lane == 0) {
      int i = 0;
      for (; i < 2 * steps; ++i) {
        const int slot = i % kSlots, use = i / kSlots;
        if (use > 0 && !mbar_wait(bars + B_EMPTY + slot, (use - 1) & 1)) { *abort = 1; break; }
        if (*abort) break;
        // (a second panel of values that no channel reaches is never looked at)
        load_tile(sb + slot * kTile, i & 1 ? &my : &mx, bars + B_FULL + slot, t0 + at(i / 2) * C,
                  i & 1 ? yz : xz, i & 1 ? (a.dv > 64 ? 2 : 1) : KP);
      }
      // (none is left in flight, whatever the others do)
      for (int j = max(0, i - kSlots); j < i; ++j)
        mbar_wait(bars + B_FULL + j % kSlots, (j / kSlots) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      for (int i = 0; i < steps; ++i) {
        const int ix = (2 * i) % kSlots, iy = ix + 1, p = i & 1;
        bool ok = mbar_wait(bars + B_FULL + iy, (i / 2) & 1);
        if (ok && i >= 2) ok = mbar_wait(bars + B_DFREE + p, (i / 2 - 1) & 1);
        if (!ok || !mbar_wait(bars + B_KT, p)) { *abort = 1; break; }
        tc_fence_after();
        mma_ss<true, true, 64 * KP>(tmem + 128 * p, sb + iy * kTile, sb + ix * kTile, 0);
        mma_ss<true, true, 64 * KP>(tmem + 128 * p, sb + iy * kTile, sb + kLo, 1);
        umma_commit(bars + B_DF + p);
        umma_commit(bars + B_EMPTY + ix);
        umma_commit(bars + B_EMPTY + iy);
      }
      umma_commit(bars + B_END);
    }
  } else if (warp == 2) {
    const float* g = a.g_head ? a.g + u.h : a.g + vrow;
    const int gs = a.g_head ? 0 : 1;
    for (int i = 0; i < steps; ++i) {
      const int c = at(i);
      const float4 x = load_decays(g + (size_t)c * C * gs, gs, min(len - c * C, C), lane);
      if (i >= 1 && !warp_wait(bars + B_GFREE, (i - 1) & 1, abort)) break;
      make_gates<false>(gates, x, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_G);
    }
  } else if (warp >= 4 && warp < 8) {
    const int t = tid - 128;
    for (int i = 0; i < steps; ++i) {
      const int ix = (2 * i) % kSlots, valid = min(len - at(i) * C, C);
      const uint32_t par = (i / 2) & 1;
      if (!warp_wait(bars + B_G, i & 1, abort)) break;
      const float wt = BACK ? a.scale * gates->eL[t] : gates->w[t];
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_GFREE);
      if (!warp_wait(bars + B_FULL + ix, par, abort)) break;
      if (a.cu_seqlens && valid < C) {  // tokens of the next sequence behind this one
        if (!warp_wait(bars + B_FULL + ix + 1, par, abort)) break;
        if (t >= valid) zero_row(sm + (ix + 1) * kTile, t);
      }
      if (i >= 1 && !warp_wait(bars + B_DF + ((i - 1) & 1), ((i - 1) / 2) & 1, abort)) break;
      scale_row(sm + ix * kTile, sm + kLo, t, 0, 8 * KP, wt, t < valid);
      warp_publish(bars + B_KT);
    }
  } else if (warp >= 8) {
    const int s = (warp - 8) >> 2, r = (tid - 256) & 127;
    const uint32_t lanes = tmem + ((uint32_t)(r & 96) << 16);
    const size_t first =
        (images.first ? (size_t)images.first[u.n] : (size_t)u.n * ((a.T + C - 1) / C)) + u.c0;
    float S[64], decay = 1.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      const int d = 64 * s + i;
      S[i] = from && r < a.dv && d < a.dk ? from[(size_t)d * a.dv + r] : 0.f;
    }
    bool ok = true;
    int i = 0;
    for (; i < chunks; ++i) {
      const int p = i & 1, c = at(i);
      if (IMAGES) {
        // (offsets that are no packing would run past the workspace)
        const size_t slot = min(first + c, (size_t)images.chunks - 1) * a.H + u.h;
        if (i > 0) {  // the last image has left the stage
          if (tid == 256) store_read_wait();
          named_sync(1, 256);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = S[8 * j + 2 * e], y = S[8 * j + 2 * e + 1];
            hi[e] = pack_bf162(x, y);
            lo[e] = pack_bf162(x - __uint_as_float(hi[e] << 16),
                               y - __uint_as_float(hi[e] & 0xffff0000u));
          }
          char* out = sm + kStage + sw128_chunk(128, r, 8 * s + j);
          *reinterpret_cast<uint4*>(out) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(out + kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
        named_sync(1, 256);
        if (tid == 256)
          for (int z = 0; z < 2 * KP; ++z)  // (part, panel)
            store_bytes(images.img + (slot * 2 * KP + z) * panel_bytes(a.dv),
                        sb + kStage + z / KP * kTile + z % KP * kPanel, panel_bytes(a.dv));
      }
      if (i >= steps) break;
      if (!(ok = warp_wait(bars + B_G, p, abort))) break;
      const float all = gates->all;
      decay *= all;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_GFREE);
      if (!(ok = warp_wait(bars + B_DF + p, (i / 2) & 1, abort))) break;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t x[32];
        tmem_ld32<32>(lanes + 128 * p + 64 * s + 32 * q, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          S[32 * q + e] = fmaf(all, S[32 * q + e], __uint_as_float(x[e]));
      }
      warp_arrive(bars + B_DFREE + p);
    }
    if (IMAGES) leave_group(1, 256, 2 * (chunks - 1 - i));
    if (IMAGES && tid == 256) store_read_wait();
    float* to = !IMAGES ? sp.state + ((size_t)u.item * a.H + u.h) * states
                : BACK && ends && a.dh0 ? a.dh0 + state
                                        : nullptr;
    if (!IMAGES && tid == 256) sp.decay[(size_t)u.item * a.H + u.h] = decay;
    if (ok && to && r < a.dv) {
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        const int d = 64 * s + i;
        if (d < a.dk) to[(size_t)d * a.dv + r] = S[i];
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    if (!mbar_wait(bars + B_END, 0)) *abort = 1;
    if (*abort) set_status(a.status, CKDA_ERR_TIMEOUT);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 3) tmem_dealloc(tmem, 256);
}

// ---------------------------------------------------------------- segments
// Segments of the packed sequences before each, by rank, the table of all, and the
// cuts.  Offsets that are no packing would run past the tables; the bounds are kept.
__global__ void __launch_bounds__(1024) split_plan_kernel(LinearArgs a, int per, int items,
                                                          int most_cuts, int32_t* item0,
                                                          int4* table, int2* cuts) {
  __shared__ int32_t sum[1024], cut[1024];
  after_previous();
  let_next_start();
  if (a.clear && threadIdx.x == 0) *a.status = 0;
  const int share = (a.N + 1023) / 1024, i0 = threadIdx.x * share, i1 = min(i0 + share, a.N);
  auto segments = [&](int i) {
    int t0, len;
    seq_range(a, a.order[i], t0, len);
    return max(1, ((len + C - 1) / C + per - 1) / per);
  };
  int32_t s = 0, n_cut = 0;
  for (int i = i0; i < i1; ++i) {
    const int k = segments(i);
    s += k;
    n_cut += k > 1;
  }
  sum[threadIdx.x] = s;
  cut[threadIdx.x] = n_cut;
  __syncthreads();
  if (i0 >= i1) return;
  int32_t before = 0, cut_before = 0;
  for (int j = 0; j < (int)threadIdx.x; ++j) {
    before += sum[j];
    cut_before += cut[j];
  }
  for (int i = i0; i < i1; ++i) {
    item0[i] = before;
    const int n = a.order[i], segs = segments(i);
    for (int k = 0; k < segs && before + k < items; ++k)
      table[before + k] = make_int4(n, k, segs, 0);
    // segment k of this rank is the (before - i + k)-th that a cut follows
    for (int k = 0; k + 1 < segs && before - i + k < most_cuts; ++k)
      cuts[before - i + k].y = before + k;
    if (segs > 1 && cut_before < most_cuts) cuts[cut_before++].x = i;
    before += segs;
  }
  if (i1 == a.N) {
    item0[a.N] = before;
    item0[a.N + 1] = min(cut_before, most_cuts);
    item0[a.N + 2] = min(before - a.N, most_cuts);
  }
}

// Joins what the segments hand on: in order, each adds its own to the decayed
// state before it.  A thread takes one element of one (sequence, head), and loads
// eight segments' ahead.
__global__ void __launch_bounds__(256) segment_scan_kernel(LinearArgs a, Split sp, int back) {
  after_previous();
  let_next_start();
  const int at = blockIdx.x / a.H, h = blockIdx.x % a.H;
  if (sp.item0 && at >= sp.item0[a.N + 1]) return;
  const int rank = sp.item0 ? sp.cuts[at].x : at;
  const int i0 = sp.item0 ? sp.item0[rank] : rank * sp.per;
  const int segs = sp.item0 ? min(sp.item0[rank + 1], sp.items) - i0 : sp.per;
  const int n = a.dk * a.dv, e = blockIdx.y * 256 + threadIdx.x;
  if (e >= n) return;
  if (!back) {
    const int seq = a.order ? a.order[rank] : rank;
    const size_t st = ((size_t)seq * a.H + h) * n + e;
    sp.begin[st] = a.h0 ? a.h0[st] : 0.f;
  }
  auto slot = [&](int k) { return (size_t)(i0 + (back ? segs - 1 - k : k)) * a.H + h; };
  float s = 0.f;
  for (int k0 = 0; k0 < segs - 1; k0 += 8) {
    float own[8], dec[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      own[k] = k0 + k < segs - 1 ? sp.state[slot(k0 + k) * n + e] : 0.f;
      dec[k] = k0 + k < segs - 1 ? sp.decay[slot(k0 + k)] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k0 + k < segs - 1) {
        s = k0 + k == 0 ? own[k] : fmaf(dec[k], s, own[k]);
        sp.state[slot(k0 + k) * n + e] = s;
      }
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Dense: segments of a sequence, the count with the least time by this model, in
// chunks (3.1 us): rounds of CTAs over the SMs times a segment's chunks and 1.8 for a
// CTA's start and end, the same at 0.6 of the chunks for the states' pass over all
// segments but one, and 7 for the two more launches and the scan.  Measured, us, the
// forward at 128 x 128 uncut, as the model has it, and as counts around it:
//   16 heads, 32,768 tokens   797   9 segments 175   (7: 210, 14: 224, 19: 185)
//   32 heads, 16,384 tokens   403   4 segments 189   (3: 242, 7: 224, 9: 188)
//   64 heads, 8,192 tokens    207   2 segments 196   (3: 215, 4: 208, 7: 200)
//   80 heads, 8,192 tokens    207   uncut            (2: 301, 3: 264, 7: 258)
// Packed: sequences longer than 5/4 of an SM's share of all tokens are cut (24 of
// 50,021 tokens, 16 heads of 64 and 128 channels, in a loop on one set of lengths: 215 us
// with passes over every sequence and a search for each CTA's, 164 us with the tables;
// 164 to 190 us over sets of lengths).
Split linear_split(int N, int B, int H, int T, bool packed) {
  Split sp{};
  const long long chunks = (T + C - 1) / C;
  if (packed) {
    const long long share = (chunks * H * 5 / 4 + kLinSms - 1) / kLinSms;
    sp.per = (int)(share > 8 ? share : 8);
    sp.most_cuts = (int)(chunks / sp.per);
    sp.items = N + sp.most_cuts;
    return sp;
  }
  const long long units = (long long)N * H;
  double best = 0;
  sp.per = 1;
  for (int s = 1; s <= 64 && s <= (chunks > 0 ? chunks : 1); ++s) {
    const double each = (double)((chunks + s - 1) / s);
    const double rounds = (double)((units * s + kLinSms - 1) / kLinSms);
    const double before = (double)((units * (s - 1) + kLinSms - 1) / kLinSms);
    const double cost =
        rounds * (each + 1.8) + (s > 1 ? before * (0.6 * each + 1.8) + 7 : 0);
    if (s == 1 || cost < best) {
      best = cost;
      sp.per = s;
    }
  }
  sp.items = N * sp.per;
  return sp;
}

static size_t plan_bytes(const Split& sp, int N, bool packed) {
  return packed ? up256(((size_t)N + 3) * 4) + up256((size_t)sp.items * 16) +
                      up256((size_t)sp.most_cuts * 8)
                : 0;
}
// The plan and its tables, h0 again, then for each direction the states and decays of the
// segments.
size_t linear_split_bytes(const Split& sp, int N, int H, int dk, int dv, bool packed,
                          int directions) {
  const size_t slots = (size_t)sp.items * H;
  const bool cut = packed || sp.per > 1;
  return plan_bytes(sp, N, packed) +
         (cut ? up256((size_t)N * H * dk * dv * 4) +
                    directions * (up256(slots * dk * dv * 4) + up256(slots * 4))
              : 0);
}

cudaError_t linear_split_plan(const LinearArgs& a, Split& sp, char* ws, cudaStream_t s) {
  if (!a.cu_seqlens) return cudaSuccess;
  int32_t* item0 = reinterpret_cast<int32_t*>(ws);
  int4* table = reinterpret_cast<int4*>(ws + up256(((size_t)a.N + 3) * 4));
  int2* cuts = reinterpret_cast<int2*>(ws + up256(((size_t)a.N + 3) * 4) +
                                       up256((size_t)sp.items * 16));
  sp.item0 = item0;
  sp.table = table;
  sp.cuts = cuts;
  return launch_next(true, split_plan_kernel, 1, 1024, 0, s, a, sp.per, sp.items, sp.most_cuts,
                     item0, table, cuts);
}

template <bool BACK, bool IMAGES, int KP>
static cudaError_t launch_states_of(const LinearArgs& a, const Split& sp, const ChunkImages& out,
                                 cudaStream_t s) {
  CUtensorMap mx{}, my{};
  if (a.T > 0 &&
      (!linear_map(&mx, BACK ? a.q : a.k, (uint64_t)a.B * a.Hk, a.T, a.dk) ||
       !linear_map(&my, BACK ? a.dout : a.v, (uint64_t)a.B * a.H, a.T, a.dv)))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<linear_state_kernel<BACK, IMAGES, KP>>(st::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned blocks =
      (unsigned)(!IMAGES && a.cu_seqlens ? sp.most_cuts : sp.items) * a.H;
  // (early, the kernels that fill the SMs for long cost the one before them more than
  // they save: backward of 8 x 16 x 2048 268 us, and 272 with states and gradients early)
  return launch_next(!IMAGES && (BACK || a.cu_seqlens), linear_state_kernel<BACK, IMAGES, KP>, blocks,
                     st::kThreads, st::kSmem, s, a, sp, out, mx, my);
}

template <bool BACK, bool IMAGES>
static cudaError_t launch_states(const LinearArgs& a, const Split& sp, const ChunkImages& out,
                                 cudaStream_t s) {
  return a.dk <= 64 ? launch_states_of<BACK, IMAGES, 1>(a, sp, out, s)
                    : launch_states_of<BACK, IMAGES, 2>(a, sp, out, s);
}

cudaError_t linear_segment_states(const LinearArgs& a, Split& sp, char* ws, bool back, int dir,
                                  cudaStream_t s) {
  if (!a.cu_seqlens && sp.per == 1) return cudaSuccess;
  const size_t slots = (size_t)sp.items * a.H;
  const size_t states = up256(slots * a.dk * a.dv * 4), decays = up256(slots * 4);
  char* at = ws + plan_bytes(sp, a.N, a.cu_seqlens != nullptr);
  sp.begin = reinterpret_cast<float*>(at);
  at += up256((size_t)a.N * a.H * a.dk * a.dv * 4) + dir * (states + decays);
  sp.state = reinterpret_cast<float*>(at);
  sp.decay = reinterpret_cast<float*>(at + states);
  // packed, every sequence shorter than a segment: nothing to join
  if (a.cu_seqlens && sp.most_cuts == 0) return cudaSuccess;
  cudaError_t e = back ? launch_states<true, false>(a, sp, ChunkImages{}, s)
                       : launch_states<false, false>(a, sp, ChunkImages{}, s);
  if (e != cudaSuccess) return e;
  const unsigned cut = a.cu_seqlens ? sp.most_cuts : a.N;  // sequences, at most
  return launch_next(true, segment_scan_kernel, dim3(cut * a.H, (a.dk * a.dv + 255) / 256), 256, 0,
                     s, a, sp, back ? 1 : 0);
}

cudaError_t linear_chunk_states(const LinearArgs& a, const Split& sp, const ChunkImages& out,
                                bool back, cudaStream_t s) {
  return back ? launch_states<true, true>(a, sp, out, s) : launch_states<false, true>(a, sp, out, s);
}

}  // namespace ckda
