// ckda_linear_bwd.cu -- chunked backward of linear attention with a scalar decay
// per head on the tensor cores (bf16 I/O, widths up to 128).
//
// With the forward's notation (chunks of 128 tokens, H the state entering a
// chunk, L the cumulative log decay inside it) and G = dL/dH at the chunk's end:
//     dQ = s e^{L_i} (dO H^T) + dS K,       dS_ij = s e^{L_i - L_j} (do_i.v_j)
//     dK = e^{L_C - L_j} (V G^T) + dS^T Q
//     dV = e^{L_C - L_j} (K G) + P^T dO,    P_ij  = s e^{L_i - L_j} (q_i.k_j)
//     G <- e^{L_C} G + sum_i s e^{L_i} q_i do_i^T      (to the chunk before)
//     dg_t = e^{L_C} <H, G> + sum_{j<t} e^{L_C-L_j} k_j.(G v_j)
//            + sum_{i>=t} [ s e^{L_i} q_i.(H do_i) + sum_{j<i} W_ij - sum_{l>i} W_li ],
//     W_ij = s e^{L_i - L_j} (q_i.k_j)(do_i.v_j)
// (s the query scale).  dg has no term that is larger than what it counts: a
// token's own product W_ii, which no decay touches, is not in it, and pairs on
// the same side of t cancel inside one chunk only.
//
// Three steps:
//   1. linear_chunk_states, forward in time: H entering every chunk;
//   2. the same, backward in time over (q, do): G at every chunk's end;
//   3. linear_grad_kernel: all gradients of a chunk.
// The states pass through HBM in two bf16 parts (hi + lo, 64 KiB a chunk and
// direction): dg and dh0 are fp32 and need more than one bf16 rounding.
// 8 x 16 heads x 2048 tokens at 128 x 128: 271 us, 42 of them the states in each direction
// and 175 the gradients, which no unit bounds (tensor pipe 29%, DRAM 49%, issue 39%): one
// chunk is in flight on an SM, a chain from product to rows of a thread to product.
// 64 x 64 channels 205 us; four query heads to a key head 288 us.
#include <type_traits>
#include "ckda_linear_chunk.cuh"

namespace ckda {
namespace {
using namespace chunk;

struct BwdWs {
  char* himg;           // [slots * H] images of H
  char* gimg;           // of G
  float* dg;            // [B, H, T] (a decay per head only)
  __nv_bfloat16* dq;    // [B, H, T, dk]: each head's part of dq and dk (shared key
  __nv_bfloat16* dk;    // heads only)
  int32_t* first;       // [N + 1] first chunk of each sequence (packed only)
  int2* table;          // [chunks] first token, tokens (packed only)
  int chunks;           // slots of a head: chunks, or a bound on them
};

// Chunks of the packed sequences before each, and the table of all.
__global__ void __launch_bounds__(1024) chunk_plan_kernel(LinearArgs a, BwdWs w, int32_t* first) {
  after_previous();
  let_next_start();
  __shared__ int32_t sum[1024];
  const int per = (a.N + 1023) / 1024, i0 = threadIdx.x * per, i1 = min(i0 + per, a.N);
  int32_t s = 0;
  for (int i = i0; i < i1; ++i) {
    int t0, len;
    seq_range(a, i, t0, len);
    s += (len + C - 1) / C;
  }
  sum[threadIdx.x] = s;
  __syncthreads();
  if (i0 >= i1) return;
  int32_t before = 0;
  for (int j = 0; j < (int)threadIdx.x; ++j) before += sum[j];
  for (int i = i0; i < i1; ++i) {
    first[i] = before;
    int t0, len;
    seq_range(a, i, t0, len);
    // (offsets that are no packing would run past the table)
    for (int c = 0; c * C < len && before < w.chunks; ++c, ++before)
      w.table[before] = make_int2(t0 + c * C, min(len - c * C, C));
  }
  if (i1 == a.N) first[a.N] = before;
}

// ------------------------------------------------------ gradients of a chunk
// A CTA of 512 threads takes chunk after chunk of all (sequence, head)s, one CTA
// an SM (a fresh CTA for each chunk cost 7 k cycles of 32 k between two of them),
// with the next chunk's loads and first products under the last results of this
// one.  Products, each 128 x 128 x 128: S, dP and their transposes (so that dS and
// dS^T, P^T are rows of a thread and go back to TMEM as operands), dO H^T, V G^T and
// K G in two parts each, dS K, dS^T Q, P^T dO: thirteen, 6.7 k cycles of the 24 k that a
// chunk takes.  The rest is the chain from product to rows of a thread to product.
//   warp 0 loads; warp 1 issues the products, each as soon as its operands are
//   there; warp 2 makes the decays
//   warps 4-7   A: thread = query row.  dS and the row sums of W; dQ; then the
//               second half of dV's columns, whose accumulator follows dQ's
//   warps 8-11  B: thread = key row.    dS^T and the column sums of W; dK
//   warps 12-15 C: thread = key row.    <H, G>; P^T; the first half of dV's columns
// Shared memory holds three of the four state tiles: Glo comes last, where Hlo
// was, once dO H^T is done.  Results are staged over the state tiles (dQ over
// Hhi, dK over Ghi, dV over Glo), so that the next chunk's q, k, v and do can be
// loaded as soon as this chunk's products have read theirs.
// An accumulator takes the state's part first; its thread scales that row in
// place and the product inside the chunk is added to it.  A token's own product
// (W_ii's factors, the largest under strong decay) stays out of the bf16 operands
// and is added there in fp32.  Results are staged in tiles that are no longer
// read and stored with TMA.
namespace gr {
constexpr int kThreads = 512;
constexpr uint32_t kQ = 0, kK = kTile, kV = 2 * kTile, kDo = 3 * kTile;
constexpr uint32_t kS0 = 4 * kTile, kS1 = 5 * kTile, kS2 = 6 * kTile;  // Hhi; Hlo, then Glo; Ghi
constexpr uint32_t kGates = 7 * kTile;
constexpr uint32_t kEp = kGates + sizeof(Gates);  // exp2(pre_t)
constexpr uint32_t kBars = kEp + C * sizeof(float);
constexpr uint32_t kSmem = kBars + 480;
static_assert(kSmem <= 232448, "shared memory of a CTA");
enum { B_QK, B_VD, B_H, B_GH, B_GL, B_G, B_TAIL, B_A, B_B, B_DSA, B_DSB, B_DSC, B_X1L, B_X1, B_X2, B_X3,
       B_X1S, B_X2S, B_X3S, B_DQ, B_DK, B_DV, B_HG,
       // free again: the columns of X1, X2, X3; the state tiles; the decays
       B_XR = B_HG + 2, B_F0 = B_XR + 3, B_F1, B_F2, B_PART, B_GFREE, B_END, B_COUNT };
// TMEM columns: S, dP, S^T, dP^T; then dS over S and P^T behind it, X1 and after
// it X3 over dP, X2 over S^T, dS^T over dP^T
constexpr uint32_t T_S = 0, T_DP = 128, T_ST = 256, T_DPT = 384;
constexpr uint32_t T_DS = 0, T_PT = 64, T_X1 = 128, T_X3 = 128, T_X2 = 256, T_DST = 384;
}  // namespace gr

// dq and dk of shared key heads from their heads' parts.  The parts are bf16: each
// is rounded once, as dq and dk would be of a head of its own, and added in fp32;
// fp32 parts would double the bytes of a pass that is bound by them.
__global__ void __launch_bounds__(256) sum_parts_kernel(LinearArgs a, BwdWs w) {
  after_previous();
  let_next_start();
  const int group = a.H / a.Hk;
  const size_t per = (size_t)a.T * a.dk / 8, total = (size_t)a.B * a.Hk * per;  // vectors of 8
  for (size_t e = (size_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (size_t)gridDim.x * 256) {
    const size_t first = e / per * group * per + e % per;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const uint4* part = reinterpret_cast<const uint4*>(which ? w.dk : w.dq);
      float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int i = 0; i < group; ++i) {
        const uint4 v = part[first + i * per];
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[2 * k] += __uint_as_float(x[k] << 16);
          s[2 * k + 1] += __uint_as_float(x[k] & 0xffff0000u);
        }
      }
      reinterpret_cast<uint4*>(which ? a.dkey : a.dq)[e] =
          make_uint4(pack_bf162(s[0], s[1]), pack_bf162(s[2], s[3]), pack_bf162(s[4], s[5]),
                     pack_bf162(s[6], s[7]));
    }
  }
}

// Chunk and head of a block.
struct Chunk {
  int h, valid;     // head; tokens
  int y, qz, vz;    // first token, rows of the key and value heads
};
__device__ __forceinline__ Chunk chunk_of(const LinearArgs& a, const BwdWs& w, unsigned block) {
  Chunk u;
  const int ci = block / a.H;
  u.h = block % a.H;
  int b = 0;
  if (w.first) {
    const int2 t = w.table[ci];
    u.y = t.x;
    u.valid = t.y;
  } else {
    const int per = (a.T + C - 1) / C;
    b = ci / per;
    u.y = ci % per * C;
    u.valid = min(a.T - u.y, C);
  }
  u.qz = b * a.Hk + u.h / (a.H / a.Hk);
  u.vz = b * a.H + u.h;
  return u;
}

// One part of an image into a tile: KP panels of 64 channels, VP x 64 value rows.
template <int KP, int VP>
__device__ __forceinline__ void load_image(uint32_t dst, const char* src, uint64_t* bar) {
#pragma unroll
  for (int p = 0; p < KP; ++p)
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
        "[%3];" ::"r"(dst + p * kPanel),
        "l"(src + p * (VP * kPanel / 2)), "r"(VP * (kPanel / 2)), "r"(smem_u32(bar))
        : "memory");
}

// A 128th of the elementwise product of two image tiles, summed.
template <int KP, int VP>
static __device__ __noinline__ float tile_dot(const char* a, const char* b, int t) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
  for (int i = t; i < KP * VP * (int)kPanel / 32; i += 128) {
    const int at = VP == 2 ? i : i / 512 * 1024 + i % 512;  // 64 rows of a panel: its first half
    const uint4 u = reinterpret_cast<const uint4*>(a)[at], v = reinterpret_cast<const uint4*>(b)[at];
    const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s0 = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), s0);
      s1 = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(y[e] & 0xffff0000u), s1);
    }
  }
  return s0 + s1;
}

// Scales columns [32 p0, 32 p1) of an accumulator's row in place, adds a multiple
// of the same row of a bf16 tile, and returns the scaled row's dot product with
// that of another.  acc: the TMEM address of column 32 p0.
static __device__ __noinline__ float scale_acc(uint32_t acc, float f, float m, const char* add,
                                               const char* tile, int row, int p0, int p1) {
  float dot = 0.f;
#pragma unroll 1
  for (int p = p0; p < p1; ++p) {
    uint32_t x[32];
    tmem_ld32<32>(acc + 32 * (p - p0), x);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t off = sw128_chunk(128, row, 4 * p + j);
      const uint4 u = *reinterpret_cast<const uint4*>(add + off);
      const uint4 v = *reinterpret_cast<const uint4*>(tile + off);
      const uint32_t t[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = f * __uint_as_float(x[8 * j + 2 * e]);
        const float b = f * __uint_as_float(x[8 * j + 2 * e + 1]);
        dot = fmaf(a, __uint_as_float(y[e] << 16), dot);
        dot = fmaf(b, __uint_as_float(y[e] & 0xffff0000u), dot);
        x[8 * j + 2 * e] = __float_as_uint(fmaf(m, __uint_as_float(t[e] << 16), a));
        x[8 * j + 2 * e + 1] = __float_as_uint(fmaf(m, __uint_as_float(t[e] & 0xffff0000u), b));
      }
    }
    tmem_st32<32>(acc + 32 * (p - p0), x);
  }
  tmem_st_wait();
  return dot;
}

// The same columns as bf16 into a tile.
static __device__ __noinline__ void stage_acc(uint32_t acc, char* tile, int row, int p0, int p1) {
#pragma unroll 1
  for (int p = p0; p < p1; ++p) {
    uint32_t x[32];
    tmem_ld32<32>(acc + 32 * (p - p0), x);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = pack_bf162(__uint_as_float(x[8 * j + 2 * e]), __uint_as_float(x[8 * j + 2 * e + 1]));
      *reinterpret_cast<uint4*>(tile + sw128_chunk(128, row, 4 * p + j)) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// KP, VP: panels of 64 key and value channels.
template <int KP, int VP>
__global__ void __launch_bounds__(gr::kThreads, 1)
linear_grad_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ BwdWs w,
                   const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                   const __grid_constant__ CUtensorMap mdq,
                   const __grid_constant__ CUtensorMap mdk,
                   const __grid_constant__ CUtensorMap mdv) {
  using namespace gr;
  constexpr uint32_t kPart = KP * VP * kPanel / 2;  // bytes of an image's hi or lo
  extern __shared__ __align__(1024) char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kBars);
  Gates* gates = reinterpret_cast<Gates*>(sm + kGates);
  float* ep = reinterpret_cast<float*>(sm + kEp);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + kBars + 400);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sm + kBars + 404);
  float* hg = reinterpret_cast<float*>(sm + kBars + 408);   // <H, G> by warp of A, C
  float* run = reinterpret_cast<float*>(sm + kBars + 440);  // sums by warp of A
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (sb & 1023u) {
    if (tid == 0) set_status(a.status, CKDA_ERR_CUDA);
    return;
  }
  // chunks times heads; the grid is no larger
  const unsigned blocks = (unsigned)(w.first ? min(w.first[a.N], w.chunks) : w.chunks) * a.H;
  const unsigned step = gridDim.x;

  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      const bool by_warps = (i >= B_DSA && i <= B_DSC) || (i >= B_X1S && i < B_DQ) ||
                            (i >= B_HG && i < B_F0) || i == B_GFREE;
      mbar_init(bars + i, i == B_TAIL                          ? 12
                          : i == B_PART                        ? 8
                          : i == B_X3S || i == B_XR + 2        ? 4 * VP
                          : by_warps                           ? 4
                          : i == B_F1                          ? VP
                                                               : 1);
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
    if (lane == 0) {
      uint32_t par = 0;
      int begun = 0;  // loads of this chunk: q and k; v and do; H and Ghi; Glo
      unsigned block = blockIdx.x;
      for (; block < blocks; block += step, par ^= 1, begun = 0) {
        const Chunk u = chunk_of(a, w, block);
        const char* himg = w.himg + (size_t)block * 2 * kPart;
        const char* gimg = w.gimg + (size_t)block * 2 * kPart;
        const bool again = block != blockIdx.x;
        bool ok = true;
        // a barrier of the chunk before, whose tile is wanted
        auto last = [&](int bar) { ok = ok && (!again || mbar_wait(bars + bar, par ^ 1)); };
        last(B_DQ); last(B_X3); last(B_DK);
        if (!ok) { *abort = 1; break; }
        mbar_arrive_expect_tx(bars + B_QK, 2 * KP * kPanel);
        for (int p = 0; p < KP; ++p) {
          tma_load_3d(sb + kQ + p * kPanel, &mq, bars + B_QK, 64 * p, u.y, u.qz);
          tma_load_3d(sb + kK + p * kPanel, &mk, bars + B_QK, 64 * p, u.y, u.qz);
        }
        begun = 1;
        last(B_X2); last(B_DV);
        if (!ok) { *abort = 1; break; }
        mbar_arrive_expect_tx(bars + B_VD, 2 * VP * kPanel);
        for (int p = 0; p < VP; ++p) {
          tma_load_3d(sb + kV + p * kPanel, &mv, bars + B_VD, 64 * p, u.y, u.vz);
          tma_load_3d(sb + kDo + p * kPanel, &mo, bars + B_VD, 64 * p, u.y, u.vz);
        }
        begun = 2;
        last(B_F0); last(B_F1); last(B_F2);
        if (!ok) { *abort = 1; break; }
        mbar_arrive_expect_tx(bars + B_H, 2 * kPart);
        load_image<KP, VP>(sb + kS0, himg, bars + B_H);
        load_image<KP, VP>(sb + kS1, himg + kPart, bars + B_H);
        mbar_arrive_expect_tx(bars + B_GH, kPart);
        load_image<KP, VP>(sb + kS2, gimg, bars + B_GH);
        begun = 3;
        if (!mbar_wait(bars + B_X1L, par) || !mbar_wait(bars + B_HG, par)) { *abort = 1; break; }
        mbar_arrive_expect_tx(bars + B_GL, kPart);  // Hlo has been read
        load_image<KP, VP>(sb + kS1, gimg + kPart, bars + B_GL);
        begun = 4;
        // What comes next, into L2 while this chunk is worked on: tiles come free
        // late, and their loads should not wait for HBM then.
        if (block + step < blocks) {
          const Chunk v = chunk_of(a, w, block + step);
          prefetch_tile(&mq, v.y, v.qz, a.dk);
          prefetch_tile(&mk, v.y, v.qz, a.dk);
          prefetch_tile(&mv, v.y, v.vz, a.dv);
          prefetch_tile(&mo, v.y, v.vz, a.dv);
          for (int z = 0; z < 2 * KP; ++z) {
            const size_t at = (size_t)(block + step) * 2 * kPart + z * (VP * kPanel / 2);
            prefetch_bytes(w.himg + at, VP * kPanel / 2);
            prefetch_bytes(w.gimg + at, VP * kPanel / 2);
          }
        }
      }
      // (none is left in flight, whatever the others do)
      const int loads[][2] = {{B_QK, 1}, {B_VD, 2}, {B_H, 3}, {B_GH, 3}, {B_GL, 4}};
      for (auto& l : loads)
        if (begun >= l[1] || block != blockIdx.x)
          mbar_wait(bars + l[0], begun >= l[1] ? par : par ^ 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t par = 0, tails = 0;
      unsigned finished = 0;
      for (unsigned block = blockIdx.x; block < blocks && !*abort; block += step, par ^= 1) {
      const Chunk u = chunk_of(a, w, block);
      const bool again = block != blockIdx.x;
      bool ok = mbar_wait(bars + B_QK, par);
      auto last = [&](int bar) { ok = ok && (!again || mbar_wait(bars + bar, par ^ 1)); };
      if (a.cu_seqlens && u.valid < C) ok = ok && mbar_wait(bars + B_TAIL, tails++ & 1);
      last(B_DV); last(B_XR + 1); last(B_XR + 2);
      if (!ok) break;
      tc_fence_after();
      mma_ss<false, false, 128, 4 * KP>(tmem + T_S, sb + kQ, sb + kK, 0);
      // A waits for dP: S^T meanwhile only where v and do are still on their way
      const bool soon = mbar_test(bars + B_VD, par);
      if (!soon) mma_ss<false, false, 128, 4 * KP>(tmem + T_ST, sb + kK, sb + kQ, 0);
      last(B_XR); last(B_DK);
      ok = ok && mbar_wait(bars + B_VD, par);
      if (!ok) break;
      tc_fence_after();
      mma_ss<false, false, 128, 4 * VP>(tmem + T_DP, sb + kDo, sb + kV, 0);
      umma_commit(bars + B_A);
      if (soon) mma_ss<false, false, 128, 4 * KP>(tmem + T_ST, sb + kK, sb + kQ, 0);
      mma_ss<false, false, 128, 4 * VP>(tmem + T_DPT, sb + kV, sb + kDo, 0);
      umma_commit(bars + B_B);
      // what is left, by readiness; `done` keeps the order that TMEM asks for
      enum { X1 = 1, X2H = 2, X2L = 4, X3 = 8, DQ = 16, DK = 32, DV = 64, ALL = 127 };
      uint32_t done = 0;
      const uint64_t start = globaltimer_ns();
      auto ready = [&](uint32_t what, uint32_t after, int bar) {
        if ((done & (what | after)) != after || !mbar_test(bars + bar, par)) return false;
        tc_fence_after();
        done |= what;
        return true;
      };
      for (uint32_t look = 1; done != ALL; ++look) {
        if (!(done & X1)) {
          if (mbar_test(bars + B_H, par) && ready(X1, 0, B_DSA)) {
            mma_ss<false, true, 64 * KP, 4 * VP>(tmem + T_X1, sb + kDo, sb + kS1, 0);
            umma_commit(bars + B_X1L);  // Glo may come
            mma_ss<false, true, 64 * KP, 4 * VP>(tmem + T_X1, sb + kDo, sb + kS0, 1);
            umma_commit(bars + B_X1);
          }
        } else if (ready(DQ, X1, B_X1S)) {
          mma_ts<true, 64 * KP>(tmem + T_X1, tmem + T_DS, sb + kK, 1);
          umma_commit(bars + B_DQ);
        }
        if (!(done & X2H)) {
          if (mbar_test(bars + B_GH, par) && mbar_test(bars + B_DSC, par) && ready(X2H, 0, B_DSB)) {
            mma_ss<false, true, 64 * KP, 4 * VP>(tmem + T_X2, sb + kV, sb + kS2, 0);
          }
        } else if (ready(X2L, X2H, B_GL)) {
          mma_ss<false, true, 64 * KP, 4 * VP>(tmem + T_X2, sb + kV, sb + kS1, 1);
          umma_commit(bars + B_X2);
        } else if (done & X2L) {
          if (ready(DK, X2L, B_X2S)) {
            mma_ts<true, 64 * KP>(tmem + T_X2, tmem + T_DST, sb + kQ, 1);
            umma_commit(bars + B_DK);
          }
          if (ready(X3, DQ, B_XR)) {  // dQ has left its columns
            mma_ss<false, false, 64 * VP, 4 * KP>(tmem + T_X3, sb + kK, sb + kS2, 0);
            mma_ss<false, false, 64 * VP, 4 * KP>(tmem + T_X3, sb + kK, sb + kS1, 1);
            umma_commit(bars + B_X3);
          }
          if (ready(DV, X3, B_X3S)) {
            mma_ts<true, 64 * VP>(tmem + T_X3, tmem + T_PT, sb + kDo, 1);
            umma_commit(bars + B_DV);
          }
        }
        if ((look & 255) == 0 && (*abort || globaltimer_ns() - start > kWaitLimitNs)) break;
      }
      if (done != ALL) break;
      ++finished;
      }
      if (finished != (blocks > blockIdx.x ? (blocks - 1 - blockIdx.x) / step + 1 : 0)) *abort = 1;
      umma_commit(bars + B_END);
    }
  } else if (warp == 2) {
    uint32_t par = 0;
    for (unsigned block = blockIdx.x; block < blocks; block += step, par ^= 1) {
      const Chunk u = chunk_of(a, w, block);
      const float* g = a.g_head ? a.g + u.h : a.g + (size_t)u.vz * a.T + u.y;
      const float4 x = load_decays(g, a.g_head ? 0 : 1, u.valid, lane);
      if (block != blockIdx.x && !warp_wait(bars + B_GFREE, par ^ 1, abort)) break;
      make_gates<true>(gates, x, lane);
      const float4 pre = reinterpret_cast<const float4*>(gates->pre)[lane];
      reinterpret_cast<float4*>(ep)[lane] = make_float4(ex2(pre.x), ex2(pre.y), ex2(pre.z), ex2(pre.w));
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_G);
    }
  } else if (warp >= 4) {
    const int wg = (warp - 4) >> 2, wq = warp & 3, row = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(32 * wq) << 16);
    const bool lead = row == 0;
    uint32_t par = 0;
    int met = 0;  // barriers of this group so far
    auto together = [&] {
      ++met;
      named_sync(1 + wg, 128);
    };
    for (unsigned block = blockIdx.x; block < blocks; block += step, par ^= 1) {
      const Chunk u = chunk_of(a, w, block);
      const int valid = u.valid;
      const size_t vrow = (size_t)u.vz * a.T + u.y, krow = (size_t)u.qz * a.T + u.y;
      const bool tail = a.cu_seqlens && valid < C;
      const bool in = row < valid;
      // a staged result to memory, by its 128 threads
      auto put = [&](const CUtensorMap* m, void* dst, size_t at, int width, uint32_t tile, int head,
                     int p0, int p1) {
        fence_proxy_async_smem();
        together();
        if (tail) {
          store_rows(static_cast<__nv_bfloat16*>(dst) + at * width, sm + tile, valid, width, p0, p1,
                     row);
          together();
        } else if (lead && 64 * p0 < width) {
          store_tile(m, sb + tile, u.y, head, p0, min(p1, (width + 63) / 64));
        }
      };
      if (tail) {  // tokens of the next sequence behind this one: out of every sum over tokens
        if (!warp_wait(bars + (wg == 2 ? B_VD : B_QK), par, abort)) break;
        if (!in) zero_row(sm + (wg == 0 ? kQ : wg == 1 ? kK : kDo), row);
        warp_publish(bars + B_TAIL);
      }
      float hgsum = 0.f;
      if (wg == 2) {
        // <H, G>, first (Hhi + Hlo, Ghi); A adds (Hhi, Glo) when Glo has come.
        // (Hlo, Glo) is 2^-18 of the rest and left out.
        if (!warp_wait(bars + B_H, par, abort) || !warp_wait(bars + B_GH, par, abort)) break;
        hgsum = tile_dot<KP, VP>(sm + kS0, sm + kS2, row) + tile_dot<KP, VP>(sm + kS1, sm + kS2, row);
        warp_arrive(bars + B_HG);
      }
      if (!warp_wait(bars + B_G, par, abort)) break;
      const float pre = gates->pre[row], pre_lo = gates->lo[row], es = gates->es[row];
      const float into = a.scale * from_start(gates, row), out = gates->w[row], s = a.scale;
      // own, own_p: s do_i.v_i (A, B) and s q_i.k_i (A; C has it in own)
      float wsum = 0.f, dot = 0.f, own = 0.f, own_p = 0.f;
      if (wg == 0) {
        // row i: j over blocks up to its own
        if (!warp_wait(bars + B_A, par, abort)) break;
        tc_fence_after();
#pragma unroll 1
        for (int p = 0; p < wq; ++p) {
          uint32_t x[32], d[32], o[16];
          tmem_ld32<32>(lanes + T_S + 32 * p, x);
          tmem_ld32<32>(lanes + T_DP + 32 * p, d);
          float f = pre;
          if (p < 1 && wq > 1) f += gates->tot[1];
          if (p < 2 && wq > 2) f += gates->tot[2];
          f = s * ex2(f);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 g = reinterpret_cast<const float4*>(gates->es + 32 * p)[e];
            const float gg[4] = {g.x, g.y, g.z, g.w};
            float v[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              v[z] = __uint_as_float(d[4 * e + z]) * (f * gg[z]);
              wsum = fmaf(v[z], __uint_as_float(x[4 * e + z]), wsum);
            }
            o[2 * e] = pack_bf162(v[0], v[1]);
            o[2 * e + 1] = pack_bf162(v[2], v[3]);
          }
          tmem_st32<16>(lanes + T_DS + 16 * p, o);
        }
        {
          uint32_t x[32], d[32], o[16];
          tmem_ld32<32>(lanes + T_S + 32 * wq, x);
          tmem_ld32<32>(lanes + T_DP + 32 * wq, d);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 g = reinterpret_cast<const float4*>(gates->pre + 32 * wq)[e];
            const float4 r = reinterpret_cast<const float4*>(gates->lo + 32 * wq)[e];
            const float2 g0 = gaps(g.x, g.y, r.x, r.y, -pre, -pre_lo);
            const float2 g1 = gaps(g.z, g.w, r.z, r.w, -pre, -pre_lo);
            const float gg[4] = {g0.x, g0.y, g1.x, g1.y};  // from this row to those
            float v[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int j = 4 * e + z;
              const float dp = s * __uint_as_float(d[j]);
              v[z] = j < lane ? dp * ex2(-gg[z]) : 0.f;
              if (j < lane) wsum = fmaf(v[z], __uint_as_float(x[j]), wsum);
              if (j == lane) {
                own = dp;
                own_p = s * __uint_as_float(x[j]);
              }
            }
            o[2 * e] = pack_bf162(v[0], v[1]);
            o[2 * e + 1] = pack_bf162(v[2], v[3]);
          }
          tmem_st32<16>(lanes + T_DS + 16 * wq, o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0;
#pragma unroll 1
          for (int p = wq + 1; p < 4; ++p) tmem_st32<16>(lanes + T_DS + 16 * p, o);
        }
        tmem_st_wait();
        warp_arrive(bars + B_DSA);
        if (!warp_wait(bars + B_X1, par, abort)) break;
        tc_fence_after();
        dot = scale_acc(lanes + T_X1, into, own, sm + kK, sm + kQ, row, 0, 2 * KP);
        warp_arrive(bars + B_X1S);
        // the rest of <H, G> meanwhile: (Hhi, Glo)
        if (!warp_wait(bars + B_H, par, abort) || !warp_wait(bars + B_GL, par, abort)) break;
        hgsum = tile_dot<KP, VP>(sm + kS0, sm + kS1, row);
        warp_arrive(bars + B_HG + 1);
        together();  // dQ goes over Hhi
        if (!warp_wait(bars + B_DQ, par, abort)) break;
        tc_fence_after();
        stage_acc(lanes + T_X1, sm + kS0, row, 0, 2 * KP);
        warp_arrive(bars + B_XR);
        put(&mdq, w.dq ? w.dq : a.dq, w.dq ? vrow : krow, a.dk, kS0, w.dq ? u.vz : u.qz, 0, KP);
      } else {
        // row j: i over blocks from its own on.  B forms dS^T (over dP^T) and the
        // sums of W, C forms P^T (behind dS, so after A).
        const bool isb = wg == 1;
        const uint32_t to = lanes + (isb ? T_DST : T_PT);
        if (!warp_wait(bars + B_B, par, abort)) break;
        if (!isb && !warp_wait(bars + B_DSA, par, abort)) break;
        tc_fence_after();
        uint32_t o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0;
#pragma unroll 1
        for (int p = 0; p < wq; ++p) tmem_st32<16>(to + 16 * p, o);
        {
          uint32_t x[32], d[32];
          tmem_ld32<32>(lanes + T_ST + 32 * wq, x);
          if (isb) {
            tmem_ld32<32>(lanes + T_DPT + 32 * wq, d);
            tmem_ld_wait();
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) d[e] = x[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 g = reinterpret_cast<const float4*>(gates->pre + 32 * wq)[e];
            const float4 r = reinterpret_cast<const float4*>(gates->lo + 32 * wq)[e];
            const float2 g0 = gaps(g.x, g.y, r.x, r.y, -pre, -pre_lo);
            const float2 g1 = gaps(g.z, g.w, r.z, r.w, -pre, -pre_lo);
            const float gg[4] = {g0.x, g0.y, g1.x, g1.y};  // from this row to those
            float v[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int i = 4 * e + z;
              const float dp = s * __uint_as_float(d[i]);
              v[z] = i > lane ? dp * ex2(gg[z]) : 0.f;
              if (i > lane) wsum = fmaf(v[z], __uint_as_float(x[i]), wsum);
              if (i == lane) own = dp;
            }
            o[2 * e] = pack_bf162(v[0], v[1]);
            o[2 * e + 1] = pack_bf162(v[2], v[3]);
          }
          tmem_st32<16>(to + 16 * wq, o);
        }
#pragma unroll 1
        for (int p = wq + 1; p < 4; ++p) {
          uint32_t x[32], d[32];
          tmem_ld32<32>(lanes + T_ST + 32 * p, x);
          float f = 0.f;
          if (wq < 1 && p > 1) f += gates->tot[1];
          if (wq < 2 && p > 2) f += gates->tot[2];
          f = s * es * ex2(f);
          if (isb) {
            tmem_ld32<32>(lanes + T_DPT + 32 * p, d);
            tmem_ld_wait();
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) d[e] = x[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 g = reinterpret_cast<const float4*>(ep + 32 * p)[e];
            const float gg[4] = {g.x, g.y, g.z, g.w};
            float v[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int i = 4 * e + z;
              v[z] = __uint_as_float(d[i]) * (f * gg[z]);
              wsum = fmaf(v[z], __uint_as_float(x[i]), wsum);
            }
            o[2 * e] = pack_bf162(v[0], v[1]);
            o[2 * e + 1] = pack_bf162(v[2], v[3]);
          }
          tmem_st32<16>(to + 16 * p, o);
        }
        tmem_st_wait();
        warp_arrive(bars + (isb ? B_DSB : B_DSC));
        if (isb) {
          if (!warp_wait(bars + B_X2, par, abort)) break;
          tc_fence_after();
          dot = scale_acc(lanes + T_X2, out, own, sm + kQ, sm + kK, row, 0, 2 * KP);
          warp_arrive(bars + B_X2S);
          if (!warp_wait(bars + B_DK, par, abort)) break;
          tc_fence_after();
          // over Ghi: the products' last reader is X3, C's dot product came before
          if (!warp_wait(bars + B_X3, par, abort) || !warp_wait(bars + B_HG, par, abort)) break;
          stage_acc(lanes + T_X2, sm + kS2, row, 0, 2 * KP);
          warp_arrive(bars + B_XR + 1);
          put(&mdk, w.dk ? w.dk : a.dkey, w.dk ? vrow : krow, a.dk, kS2, w.dk ? u.vz : u.qz, 0, KP);
        } else {
          own_p = own;
        }
      }
      if (wg == 2 || (wg == 0 && VP == 2)) {
        // dV: C the first panel, A the second
        const int half = wg == 0 ? 1 : 0;
        if (!warp_wait(bars + B_X3, par, abort)) break;
        tc_fence_after();
        scale_acc(lanes + T_X3 + 64 * half, out, own_p, sm + kDo, sm + kDo, row, 2 * half,
                  2 * half + 2);
        warp_arrive(bars + B_X3S);
        if (!warp_wait(bars + B_DV, par, abort)) break;
        tc_fence_after();
        // over Glo, which X3 and A have read
        if (!warp_wait(bars + B_HG + 1, par, abort)) break;
        stage_acc(lanes + T_X3 + 64 * half, sm + kS1, row, 2 * half, 2 * half + 2);
        warp_arrive(bars + B_XR + 2);
        put(&mdv, a.dval, vrow, a.dv, kS1, u.vz, half, half + 1);
      }
      if (lead) {
        store_read_wait();
        if (wg == 0) mbar_arrive(bars + B_F0);
        if (wg == 1) mbar_arrive(bars + B_F2);
        if (wg == 2 || (wg == 0 && VP == 2)) mbar_arrive(bars + B_F1);
      }
      // dg_t = e^{L_C} <H, G> + sum_{j<t} kd_j + sum_{i>=t} (qd_i + row_i - col_i):
      // B hands its sums by token to A, over decays that all three have read
      if (wg == 1) {
        if (!warp_wait(bars + B_DSA, par, abort) || !warp_wait(bars + B_DSC, par, abort)) break;
        gates->lo[row] = in ? wsum : 0.f;
        gates->w[row] = in ? dot : 0.f;
      }
      if (wg != 1) {
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) hgsum += __shfl_xor_sync(0xffffffffu, hgsum, m);
        if (lane == 0) hg[wg * 2 + wq] = hgsum;  // A 0 .. 3, C 4 .. 7
      }
      if (wg != 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + B_PART);
        continue;
      }
      if (!warp_wait(bars + B_PART, par, abort)) break;
      float fwd = gates->w[row];
      float back = in ? dot + wsum - gates->lo[row] : 0.f;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, fwd, m);
        const float z = __shfl_down_sync(0xffffffffu, back, m);
        if (lane >= m) fwd += x;
        if (lane + m < 32) back += z;
      }
      float excl = __shfl_up_sync(0xffffffffu, fwd, 1);
      if (lane == 0) excl = 0.f;
      if (lane == 31) run[wq] = fwd;
      if (lane == 0) run[4 + wq] = back;
      together();
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) t += hg[i];
      t = gates->all * t + excl + back;
      for (int i = 0; i < wq; ++i) t += run[i];
      for (int i = wq + 1; i < 4; ++i) t += run[4 + i];
      if (in) (w.dg ? w.dg : a.dg)[vrow + row] = t;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_GFREE);
    }
    if (*abort) {
      int all = 0;  // a put, or two and what A meets in besides; each once more in a tail
      for (unsigned block = blockIdx.x; block < blocks; block += step) {
        const bool tail = a.cu_seqlens && chunk_of(a, w, block).valid < C;
        all += (wg == 0 ? VP : 1) * (tail ? 2 : 1) + (wg == 0 ? 2 : 0);
      }
      leave_group(1 + wg, 128, all - met);
      if (lead) store_read_wait();
    }
  }

  // ------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    if (!mbar_wait(bars + B_END, 0)) *abort = 1;
    if (*abort) set_status(a.status, CKDA_ERR_TIMEOUT);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 3) tmem_dealloc(tmem, 512);
}

struct ChunkPlan {
  size_t chunks, himg, gimg, dg, dq, dk, first, table, split, total;
};
ChunkPlan chunk_plan(int N, int B, int H, int Hk, int T, int dk, int dv, bool packed) {
  ChunkPlan p;
  auto up256 = [](size_t x) { return (x + 255) / 256 * 256; };
  // packed: ceil(len / 128) over sequences that add up to T
  p.chunks = packed ? (size_t)T / C + N : (size_t)N * ((T + C - 1) / C);
  const size_t rows = (size_t)B * H * T;
  size_t at = 0;
  p.himg = at; at += p.chunks * H * image_bytes(dk, dv);
  p.gimg = at; at += p.chunks * H * image_bytes(dk, dv);
  p.dg = at; at += up256(rows * 4);
  p.dq = at; at += Hk == H ? 0 : up256(rows * dk * 2);
  p.dk = at; at += Hk == H ? 0 : up256(rows * dk * 2);
  p.first = at; at += up256(((size_t)N + 1) * 4);
  p.table = at; at += packed ? up256(p.chunks * 8) : 0;
  p.split = at; at += linear_split_bytes(linear_split(N, B, H, T, packed), N, H, dk, dv, packed, 2);
  p.total = at;
  return p;
}

}  // namespace

size_t linear_chunk_bwd_bytes(int N, int B, int H, int Hk, int T, int dk, int dv, bool packed) {
  return chunk_plan(N, B, H, Hk, T, dk, dv, packed).total;
}

cudaError_t linear_chunk_bwd(const LinearArgs& a, char* ws, cudaStream_t s) {
  const ChunkPlan p =
      chunk_plan(a.N, a.B, a.H, a.Hk, a.T, a.dk, a.dv, a.cu_seqlens != nullptr);
  BwdWs w{};
  w.himg = ws + p.himg;
  w.gimg = ws + p.gimg;
  w.dg = a.g_head ? reinterpret_cast<float*>(ws + p.dg) : nullptr;
  w.dq = a.Hk == a.H ? nullptr : reinterpret_cast<__nv_bfloat16*>(ws + p.dq);
  w.dk = a.Hk == a.H ? nullptr : reinterpret_cast<__nv_bfloat16*>(ws + p.dk);
  w.chunks = (int)p.chunks;
  cudaError_t e = cudaSuccess;
  CUtensorMap mq{}, mk{}, mv{}, mo{}, mdq{}, mdk{}, mdv{};
  const uint64_t heads = (uint64_t)a.B * (w.dq ? a.H : a.Hk);
  if (a.T > 0 && (!linear_map(&mq, a.q, (uint64_t)a.B * a.Hk, a.T, a.dk) ||
                  !linear_map(&mk, a.k, (uint64_t)a.B * a.Hk, a.T, a.dk) ||
                  !linear_map(&mv, a.v, (uint64_t)a.B * a.H, a.T, a.dv) ||
                  !linear_map(&mo, a.dout, (uint64_t)a.B * a.H, a.T, a.dv) ||
                  !linear_map(&mdq, w.dq ? w.dq : a.dq, heads, a.T, a.dk) ||
                  !linear_map(&mdk, w.dk ? w.dk : a.dkey, heads, a.T, a.dk) ||
                  !linear_map(&mdv, a.dval, (uint64_t)a.B * a.H, a.T, a.dv)))
    return cudaErrorInvalidValue;
  if (a.cu_seqlens) {
    w.first = reinterpret_cast<int32_t*>(ws + p.first);
    w.table = reinterpret_cast<int2*>(ws + p.table);
    e = launch_next(true, chunk_plan_kernel, 1, 1024, 0, s, a, w, w.first);
    if (e != cudaSuccess) return e;
  }
  Split sp = linear_split(a.N, a.B, a.H, a.T, a.cu_seqlens != nullptr);
  if ((e = linear_split_plan(a, sp, ws + p.split, s)) != cudaSuccess) return e;
  for (int back = 0; back < 2; ++back) {
    if ((e = linear_segment_states(a, sp, ws + p.split, back, back, s)) != cudaSuccess) return e;
    const ChunkImages out{back ? w.gimg : w.himg, w.first, w.chunks};
    if ((e = linear_chunk_states(a, sp, out, back, s)) != cudaSuccess) return e;
  }
  if (a.T > 0) {
    const size_t blocks = p.chunks * a.H;
    const auto grad = [&](auto kp, auto vp) {
      constexpr int KP = decltype(kp)::value, VP = decltype(vp)::value;
      const cudaError_t e = allow_smem<linear_grad_kernel<KP, VP>>(gr::kSmem);
      if (e != cudaSuccess) return e;
      return launch_next(false, linear_grad_kernel<KP, VP>,
                         (unsigned)(blocks < kLinSms ? blocks : kLinSms), gr::kThreads, gr::kSmem,
                         s, a, w, mq, mk, mv, mo, mdq, mdk, mdv);
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    e = a.dk <= 64 ? (a.dv <= 64 ? grad(one, one) : grad(one, two))
                   : (a.dv <= 64 ? grad(two, one) : grad(two, two));
    if (e != cudaSuccess) return e;
    if (w.dq) {
      const size_t n = (size_t)a.B * a.Hk * a.T * a.dk / 8, blocks = (n + 255) / 256;
      e = launch_next(true, sum_parts_kernel,
                      (unsigned)(blocks < 16 * kLinSms ? blocks : 16 * kLinSms), 256, 0, s, a, w);
      if (e != cudaSuccess) return e;
    }
  }
  return a.g_head ? linear_sum_decay(a, w.dg, s) : e;
}

}  // namespace ckda
