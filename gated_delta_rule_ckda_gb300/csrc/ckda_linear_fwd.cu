// ckda_linear_fwd.cu -- chunked forward of linear attention with a scalar decay
// per head on the tensor cores (bf16 I/O, widths up to 128).
//
// A chunk of 128 tokens, with L_i the cumulative log decay inside it and H the
// state entering it:
//     S = Q K^T,   P_ij = S_ij e^{L_i - L_j} (j <= i),
//     O = P V + e^{L_i} (Q H),
//     H <- e^{L_C} H + sum_j e^{L_C - L_j} k_j v_j^T.
// Every exponent is a sum of log decays, so with g <= 0 no factor exceeds one.
//
// One CTA of 512 threads walks the chunks of one (sequence, head), or of one
// segment of it; the state never leaves the SM.  The floor is HBM: 1 KiB a token at
// 128 x 128 against five 128 x 128 x 128 products a chunk (four and a key part).
// Measured: 4 x 32 x 8192 tokens 209 us, 77% of the copy bandwidth with 128 of 152
// SMs at work; 152 (sequence, head)s reach 86%.  A chunk takes 6,000 cycles, set by
// the latency of its loads through five slots and by the chain S, P, PV, o, H.
// Tried and slower: persistent CTAs over all pieces (221 us: uneven ends), o by
// warps of their own (211 us), the state's product ahead of the next S (219 us),
// tiles ahead into L2 (211 us one or two chunks ahead, 255 us four).
//   warp 0       loads tiles with TMA into a ring of slots, in the order q, k, v
//                of chunk after chunk
//   warp 1       issues the products (tcgen05, one thread)
//   warp 2       the decay factors of a chunk
//   warps 4-7    one row of S a thread: P as bf16 into TMEM, where the product
//                P V reads it; later the row of o, staged in the state's
//                tile (between its readers and the next state) and stored with
//                TMA (a thread's own 256-byte rows cost four times the L1 passes)
//   warps 8-15   the state: thread (r, s) holds one half s of H's rows in column r
//                in fp32 registers, rounded to nearest at every step (tensor-core
//                accumulators truncate, which over thousands of chunks would
//                bias a slowly decaying state).  A chunk's own contribution is
//                a product of its own into fresh TMEM columns, so it does not
//                wait for the state; per chunk the state warps
//                  - write H as bf16 to shared memory for Q H,
//                  - scale the keys by e^{L_C - L_j} in two bf16 parts (hi over
//                    the key tile, lo beside it): the state is an fp32 output,
//                    and one rounding of the keys would leave it with 2^-9,
//                  - read the product and update H.
// Rounded to bf16 are P, and H where it is read by the queries: o is bf16.
#include "ckda_linear_chunk.cuh"

namespace ckda {
namespace {
using namespace chunk;

constexpr int kThreads = 512;

// KD: key channels, 64 or 128 (narrower keys are filled with zeros).  128: a
// ring of five 32 KB slots, one tile each.  64: q and k take 16 KB, and there is
// room for two whole chunks.
template <int KD>
struct Layout {
  static constexpr int kSlots = KD == 128 ? 5 : 6;
  static constexpr int kPanels = KD / 64;
  static constexpr uint32_t kLo = KD == 128 ? 5 * kTile : 4 * kTile;  // lo part of the scaled keys
  static constexpr uint32_t kH = kLo + kPanels * kPanel;              // bf16 state, [dv][dk]; o
  static constexpr uint32_t kGates = kH + kTile;
  static constexpr uint32_t kBars = kGates + sizeof(Gates);
  static constexpr uint32_t kSmem = kBars + 512;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  __device__ static __forceinline__ uint32_t at(int slot) {
    return KD == 128 ? slot * kTile : slot / 3 * 2 * kTile + slot % 3 * kPanel;
  }
};

// A barrier is looked at by the parity of a phase: whoever waits for one has to have seen
// it before anything that the phase after the next one waits for.
enum {
  // B_O and B_DF by chunk parity: the loads wait on them too, and may lag a chunk
  B_FULL = 0, B_S = 6, B_P, B_PV, B_O, B_HREADY = B_O + 2, B_HFREE, B_KT, B_DF, B_G = B_DF + 2,
  B_GFREE, B_END, B_COUNT
};
// TMEM columns
constexpr uint32_t T_S = 0, T_P = 0, T_DF = 128, T_OI = 256, T_O = 384;

template <int KD>
__global__ void __launch_bounds__(kThreads, 1)
linear_fwd_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ Split sp,
                  const __grid_constant__ CUtensorMap mq,
                  const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ CUtensorMap mo) {
  using L = Layout<KD>;
  constexpr int kSlots = L::kSlots, kHalf = KD / 2;
  constexpr uint32_t kLo = L::kLo, kH = L::kH, kGates = L::kGates, kBars = L::kBars;
  extern __shared__ __align__(1024) char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kBars);
  Gates* gates = reinterpret_cast<Gates*>(sm + kGates);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + kBars + 400);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sm + kBars + 404);
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!a.clear) after_previous();
  // (a wait gives up after a second: no other CTA has anything to report yet)
  if (a.clear && blockIdx.x == 0 && tid == 0) *a.status = 0;
  if (sb & 1023u) {  // swizzled tiles need it; no room to align by hand
    if (tid == 0) set_status(a.status, CKDA_ERR_CUDA);
    return;
  }

  if (blockIdx.x >= pieces(a, sp)) return;  // the grid is a bound
  const Piece u = piece_of(a, sp, blockIdx.x);
  const int t0 = u.t0, len = u.len, chunks = u.chunks, qz = u.qz, vz = u.vz;
  const size_t vrow = (size_t)vz * a.T + t0;
  const size_t states = (size_t)a.dk * a.dv, st = ((size_t)u.n * a.H + u.h) * states;
  const float* from = u.seg > 0    ? sp.state + ((size_t)(u.item - 1) * a.H + u.h) * states
                      : u.segs > 1 ? sp.begin + st
                      : a.h0       ? a.h0 + st
                                   : nullptr;

  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      const uint32_t count = i == B_P ? 4
                             : i == B_HREADY || i == B_KT ? 8
                             : i == B_GFREE ? 12
                                            : 1;
      mbar_init(bars + i, count);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc(tmem_at, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;

  if (warp == 0) {
    // ------------------------------------------------------------- loads
    if (lane == 0) {
      int i = 0;
      for (; i < 3 * chunks; ++i) {
        const int slot = i % kSlots, use = i / kSlots, c = i / 3;
        if (use > 0) {  // the slot's last tile has been read: q by Q H, k and v by the state's product
          const int j = i - kSlots, cj = j / 3;
          if (!mbar_wait(bars + (j % 3 == 0 ? B_O : B_DF) + (cj & 1), (cj >> 1) & 1)) *abort = 1;
        }
        if (*abort) break;
        const CUtensorMap* m = i % 3 == 0 ? &mq : i % 3 == 1 ? &mk : &mv;
        // (a second panel of v that no channel reaches is never looked at)
        load_tile(sb + L::at(slot), m, bars + B_FULL + slot, t0 + c * C, i % 3 == 2 ? vz : qz,
                  i % 3 == 2 ? (a.dv > 64 ? 2 : 1) : L::kPanels);
      }
      // (none is left in flight, whatever the others do)
      for (int j = max(0, i - kSlots); j < i; ++j)
        mbar_wait(bars + B_FULL + j % kSlots, (j / kSlots) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- products
    // One thread, so that nothing but a barrier stands between two products.
    // S of the next chunk goes ahead of this chunk's contribution to the state:
    // the warps of P wait for it, while the state has slack.
    if (lane == 0) {
      bool ok = true;
      auto wait = [&](int bar, uint32_t parity) {
        ok = ok && mbar_wait(bars + bar, parity);
        return ok;
      };
      int sq = 0;          // slot of Q, and how often the ring has come round
      uint32_t round = 0;
      for (int c = -1; c < chunks; ++c) {
        int sk = sq + 1, sv = sq + 2;
        uint32_t rk = round, rv = round;
        if (sk >= kSlots) { sk -= kSlots; ++rk; }
        if (sv >= kSlots) { sv -= kSlots; ++rv; }
        const uint32_t par = c & 1;
        if (c >= 0) {
          wait(B_FULL + sv, rv & 1);
          if (!wait(B_P, par)) break;  // and o of the last chunk has been read
          tc_fence_after();
          mma_ts<true>(tmem + T_O, tmem + T_P, sb + L::at(sv), 0);
          umma_commit(bars + B_PV);
          if (!wait(B_HREADY, par)) break;
          tc_fence_after();
          mma_ss<false, false, 128, KD / 16>(tmem + T_OI, sb + L::at(sq), sb + kH, 0);
          umma_commit(bars + B_O + par);
        }
        if (c + 1 < chunks) {
          int nq = c < 0 ? 0 : sv + 1, nk;
          uint32_t rq = c < 0 ? 0 : rv;
          if (nq >= kSlots) { nq -= kSlots; ++rq; }
          nk = nq + 1;
          wait(B_FULL + nq, rq & 1);
          wait(B_FULL + (nk < kSlots ? nk : 0), (rq + (nk >= kSlots)) & 1);
          if (c >= 0) wait(B_PV, par);  // P shares the columns of S
          if (!ok) break;
          tc_fence_after();
          mma_ss<false, false, 128, KD / 16>(tmem + T_S, sb + L::at(nq),
                                             sb + L::at(nk < kSlots ? nk : 0), 0);
          umma_commit(bars + B_S);
        }
        if (c < 0) continue;
        if (!wait(B_KT, par)) break;
        tc_fence_after();
        mma_ss<true, true, KD>(tmem + T_DF, sb + L::at(sv), sb + L::at(sk), 0);
        mma_ss<true, true, KD>(tmem + T_DF, sb + L::at(sv), sb + kLo, 1);
        umma_commit(bars + B_DF + par);
        sq = sv + 1;
        round = rv;
        if (sq >= kSlots) { sq -= kSlots; ++round; }
      }
      if (!ok) *abort = 1;
      umma_commit(bars + B_END);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------- decays
    const float* g = a.g_head ? a.g + u.h : a.g + vrow;
    const int gs = a.g_head ? 0 : 1;
    float4 x = load_decays(g, gs, min(len, C), lane);
    for (int c = 0; c < chunks; ++c) {
      if (c > 0 && !warp_wait(bars + B_GFREE, (c - 1) & 1, abort)) break;
      make_gates<false>(gates, x, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_G);
      if (c + 1 < chunks)
        x = load_decays(g + (size_t)(c + 1) * C * gs, gs, min(len - (c + 1) * C, C), lane);
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------- P and o
    const int w = warp - 4, i = tid - 128;
    const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
    int c = 0;
    for (; c < chunks; ++c) {
      const uint32_t par = c & 1;
      const int valid = min(len - c * C, C);
      if (a.cu_seqlens && valid < C) {  // tokens of the next sequence behind this one
        const int iv = 3 * c + 2;
        if (!warp_wait(bars + B_FULL + iv % kSlots, (iv / kSlots) & 1, abort)) break;
        if (i >= valid) zero_row(sm + L::at(iv % kSlots), i);
      }
      if (!warp_wait(bars + B_G, par, abort)) break;
      const float pre = gates->pre[i], into = gates->eL[i];
      if (!warp_wait(bars + B_S, par, abort)) break;
      tc_fence_after();
      // earlier blocks: from j to its block's end, over the blocks between, and
      // from this block's start to i
#pragma unroll 1
      for (int p = 0; p < w; ++p) {
        uint32_t s[32];
        tmem_ld32<32>(lanes + T_S + 32 * p, s);
        float x = pre;
        if (p < 1 && w > 1) x += gates->tot[1];
        if (p < 2 && w > 2) x += gates->tot[2];
        const float r = ex2(x);
        uint32_t out[16];
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 q = reinterpret_cast<const float4*>(gates->es + 32 * p)[e];
          out[2 * e] = pack_bf162(__uint_as_float(s[4 * e]) * (r * q.x),
                                  __uint_as_float(s[4 * e + 1]) * (r * q.y));
          out[2 * e + 1] = pack_bf162(__uint_as_float(s[4 * e + 2]) * (r * q.z),
                                      __uint_as_float(s[4 * e + 3]) * (r * q.w));
        }
        tmem_st32<16>(lanes + T_P + 16 * p, out);
      }
      {
        // its own block, j <= i: from the difference of short sums
        uint32_t s[32], out[16];
        tmem_ld32<32>(lanes + T_S + 32 * w, s);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 q = reinterpret_cast<const float4*>(gates->pre + 32 * w)[e];
          const float qq[4] = {q.x, q.y, q.z, q.w};
          float v[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            v[z] = 4 * e + z <= lane ? __uint_as_float(s[4 * e + z]) * ex2(pre - qq[z]) : 0.f;
          out[2 * e] = pack_bf162(v[0], v[1]);
          out[2 * e + 1] = pack_bf162(v[2], v[3]);
        }
        tmem_st32<16>(lanes + T_P + 16 * w, out);
#pragma unroll
        for (int e = 0; e < 16; ++e) out[e] = 0;
#pragma unroll 1
        for (int p = w + 1; p < 4; ++p) tmem_st32<16>(lanes + T_P + 16 * p, out);
      }
      tmem_st_wait();
      warp_publish(bars + B_P);
      if (lane == 0) mbar_arrive(bars + B_GFREE);

      if (!warp_wait(bars + B_O + par, (c >> 1) & 1, abort)) break;
      tc_fence_after();
      // o by way of the state's tile, which nothing reads any more
      char* stage = sm + kH;
      const float fo = a.scale, fi = a.scale * into;
#pragma unroll 1
      for (int p = 0; p < 4; ++p) {
        if (32 * p >= a.dv) break;
        uint32_t x[32], y[32];
        tmem_ld32<32>(lanes + T_O + 32 * p, x);
        tmem_ld32<32>(lanes + T_OI + 32 * p, y);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 8 * j + 2 * e;
            o[e] = pack_bf162(fmaf(fo, __uint_as_float(x[k]), fi * __uint_as_float(y[k])),
                              fmaf(fo, __uint_as_float(x[k + 1]), fi * __uint_as_float(y[k + 1])));
          }
          *reinterpret_cast<uint4*>(stage + sw128_chunk(128, i, 4 * p + j)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      tc_fence_before();
      fence_proxy_async_smem();
      named_sync(1, 128);
      if (a.cu_seqlens && valid < C) {
        store_rows(static_cast<__nv_bfloat16*>(a.o) + (vrow + (size_t)c * C) * a.dv, stage, valid,
                   a.dv, 0, 2, i);
        // (the last chunk of the sequence: nothing reuses the tile)
      } else if (i == 0) {
        store_tile(&mo, sb + kH, t0 + c * C, vz, 0, a.dv > 64 ? 2 : 1);
        store_read_wait();  // (this warp has the shortest rows of P)
        mbar_arrive(bars + B_HFREE);
      }
    }
    leave_group(1, 128, chunks - c);
  } else if (warp >= 8) {
    // --------------------------------------------------------------- state
    const int s = (warp - 8) >> 2, r = (tid - 256) & 127;   // half of dk, value column
    const uint32_t lanes = tmem + ((uint32_t)(r & 96) << 16);
    float H[kHalf];
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      const int d = kHalf * s + i;
      H[i] = from && r < a.dv && d < a.dk ? from[(size_t)d * a.dv + r] : 0.f;
    }
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      const uint32_t par = c & 1;
      const int ik = 3 * c + 1, valid = min(len - c * C, C);
      // the state entering the chunk, once the last chunk's queries have read
      // theirs and o has left the tile again
      if (c > 0 && !(ok = warp_wait(bars + B_HFREE, (c - 1) & 1, abort))) break;
#pragma unroll
      for (int j = 0; j < kHalf / 8; ++j)
        *reinterpret_cast<uint4*>(sm + kH + sw128_chunk(128, r, kHalf / 8 * s + j)) =
            make_uint4(pack_bf162(H[8 * j], H[8 * j + 1]), pack_bf162(H[8 * j + 2], H[8 * j + 3]),
                       pack_bf162(H[8 * j + 4], H[8 * j + 5]),
                       pack_bf162(H[8 * j + 6], H[8 * j + 7]));
      // S has read the keys.  Looked at before these warps publish: the next S waits for
      // that, and a warp that looked after it could find S two phases on and wait for a
      // third, which waits for its keys.
      if (!(ok = warp_wait(bars + B_S, par, abort))) break;
      warp_publish(bars + B_HREADY);
      // the keys, scaled
      if (!(ok = warp_wait(bars + B_G, par, abort))) break;
      const float wt = gates->w[r], all = gates->all;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_GFREE);
      if (!(ok = warp_wait(bars + B_FULL + ik % kSlots, (ik / kSlots) & 1, abort))) break;
      scale_row(sm + L::at(ik % kSlots), sm + kLo, r, kHalf / 8 * s, kHalf / 8 * (s + 1), wt,
                r < valid);
      warp_publish(bars + B_KT);
      // the chunk's contribution
      if (!(ok = warp_wait(bars + B_DF + par, (c >> 1) & 1, abort))) break;
      tc_fence_after();
#pragma unroll
      for (int p = 0; p < kHalf / 32; ++p) {
        uint32_t x[32];
        tmem_ld32<32>(lanes + T_DF + kHalf * s + 32 * p, x);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          H[32 * p + i] = fmaf(all, H[32 * p + i], __uint_as_float(x[i]));
      }
      tc_fence_before();
    }
    if (ok && a.hT && u.seg == u.segs - 1 && r < a.dv) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i) {
        const int d = kHalf * s + i;
        if (d < a.dk) a.hT[st + (size_t)d * a.dv + r] = H[i];
      }
    }
  }

  // ------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    // every commit has arrived before the memory is given back
    if (!mbar_wait(bars + B_END, 0)) *abort = 1;
    if (*abort) set_status(a.status, CKDA_ERR_TIMEOUT);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 3) tmem_dealloc(tmem, 512);
}

}  // namespace

bool linear_map(CUtensorMap* m, const void* base, uint64_t heads, uint64_t T, uint64_t width) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dim[3] = {width, T, heads};
  cuuint64_t stride[2] = {width * 2, width * T * 2};
  cuuint32_t box[3] = {64, 128, 1};
  cuuint32_t step[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dim, stride, box,
             step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t linear_chunk_fwd_bytes(int N, int B, int H, int T, int dk, int dv, bool packed) {
  return linear_split_bytes(linear_split(N, B, H, T, packed), N, H, dk, dv, packed, 1);
}

cudaError_t linear_chunk_fwd(LinearArgs a, char* ws, cudaStream_t s) {
  CUtensorMap mq{}, mk{}, mv{}, mo{};
  if (a.T > 0 && (!linear_map(&mq, a.q, (uint64_t)a.B * a.Hk, a.T, a.dk) ||
                  !linear_map(&mk, a.k, (uint64_t)a.B * a.Hk, a.T, a.dk) ||
                  !linear_map(&mv, a.v, (uint64_t)a.B * a.H, a.T, a.dv) ||
                  !linear_map(&mo, a.o, (uint64_t)a.B * a.H, a.T, a.dv)))
    return cudaErrorInvalidValue;
  Split sp = linear_split(a.N, a.B, a.H, a.T, a.cu_seqlens != nullptr);
  if (a.clear && !a.cu_seqlens && sp.per > 1) {  // more kernels than one
    if (cudaMemsetAsync(a.status, 0, sizeof(int), s) != cudaSuccess) return cudaErrorUnknown;
    a.clear = 0;
  }
  cudaError_t e = linear_split_plan(a, sp, ws, s);
  if (a.cu_seqlens) a.clear = 0;  // the plan's kernel has done it
  if (e == cudaSuccess) e = linear_segment_states(a, sp, ws, false, 0, s);
  if (e != cudaSuccess) return e;
  const bool half = a.dk <= 64;
  e = half ? allow_smem<linear_fwd_kernel<64>>(Layout<64>::kSmem)
           : allow_smem<linear_fwd_kernel<128>>(Layout<128>::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned blocks = (unsigned)sp.items * a.H;
  return half ? launch_next(!a.clear, linear_fwd_kernel<64>, blocks, kThreads, Layout<64>::kSmem, s,
                            a, sp, mq, mk, mv, mo)
              : launch_next(!a.clear, linear_fwd_kernel<128>, blocks, kThreads,
                            Layout<128>::kSmem, s, a, sp, mq, mk, mv, mo);
}

}  // namespace ckda
