// ckda_linear_chunk.cuh -- what the chunked tensor-core kernels of linear
// attention share: tiles of 128 tokens by 128 channels, their loads, the decay
// factors of a chunk, and bounded waits.
#pragma once
#include "ckda_linear.cuh"
#include "sm103.cuh"

namespace ckda {
namespace chunk {

constexpr int C = 128;                 // tokens of a chunk
constexpr uint32_t kTile = 32768;      // bytes of a 128 x 128 bf16 tile, two 64-column panels
constexpr uint32_t kPanel = 16384;
constexpr uint32_t kImage = 2 * kTile; // a state: hi tile, lo tile, [dv][dk], swizzled
// In memory an image has the panels of its hi part, then of its lo part, one behind the
// other, and of a panel only the 64 value rows where there are no more.
__host__ __device__ inline uint32_t panel_bytes(int dv) { return dv > 64 ? kPanel : kPanel / 2; }
__host__ __device__ inline uint32_t image_bytes(int dk, int dv) {
  return 2 * (dk > 64 ? 2 : 1) * panel_bytes(dv);
}

// Sequences are cut into segments where there are too few (sequence, head)s for
// the SMs, or one is much longer than an SM's share.  The state entering each
// segment comes first: every segment but the last (backward, the first) runs
// from zero, and a scan joins them.
struct Split {
  int per;               // dense: segments of a sequence; packed: most chunks of a segment
  int items;             // segments of all sequences; packed: a bound on them
  const int32_t* item0;  // packed: [N + 1] first segment by rank in a.order
                         // and behind it the numbers of cut sequences and of cuts
  const int4* table;     // packed: [items] sequence, segment, segments, unused (one load
                         // for a CTA; a search through item0 takes several, one after another)
  const int2* cuts;      // packed: [cuts] rank of a cut sequence, segment before a cut
  int most_cuts;
  float* state;          // [items * H][dk][dv]: what each segment hands on
  float* decay;          // [items * H]: over the segment
  float* begin;          // [N * H][dk][dv]: h0 again, for the first segments of sequences
                         // that are cut (hT may be h0, and another CTA writes it)
};
// A segment of one (sequence, head).
struct Piece {
  int n, h, qz, vz;      // sequence, head, rows of the key and value heads
  int t0, len;           // tokens on the T axis
  int c0, chunks;        // chunks, counted inside the sequence
  int seg, segs, item;
};
__device__ __forceinline__ unsigned pieces(const LinearArgs& a, const Split& sp) {
  return (unsigned)(a.cu_seqlens ? min(sp.item0[a.N], sp.items) : sp.items) * a.H;
}
__device__ __forceinline__ Piece piece_of(const LinearArgs& a, const Split& sp, unsigned block) {
  Piece u;
  u.item = block / a.H;
  u.h = block % a.H;
  if (a.cu_seqlens) {
    const int4 t = sp.table[u.item];
    u.n = t.x;
    u.seg = t.y;
    u.segs = t.z;
  } else {
    u.n = u.item / sp.per;
    u.seg = u.item % sp.per;
    u.segs = sp.per;
  }
  int len;
  seq_range(a, u.n, u.t0, len);
  const int all = (len + C - 1) / C;
  u.c0 = (int)((long long)all * u.seg / u.segs);
  u.chunks = (int)((long long)all * (u.seg + 1) / u.segs) - u.c0;
  u.t0 += u.c0 * C;
  u.len = min(len - u.c0 * C, u.chunks * C);
  const int b = a.cu_seqlens ? 0 : u.n;
  u.qz = b * a.Hk + u.h / (a.H / a.Hk);
  u.vz = b * a.H + u.h;
  return u;
}

// ------------------------------------------------------------------- TMA
// Box of 64 channels x 128 tokens of one head; coordinates (channel, token,
// head).  Channels past the width and tokens past T are filled with zeros.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// The panels of a tile; completion counts their bytes on `bar`.
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                          int32_t token, int32_t head, int panels = 2) {
  mbar_arrive_expect_tx(bar, panels * kPanel);
  for (int p = 0; p < panels; ++p) tma_load_3d(dst + p * kPanel, map, bar, 64 * p, token, head);
}

// The same tile, and `bytes` of memory, into L2 only.
__device__ __forceinline__ void prefetch_tile(const CUtensorMap* map, int32_t token, int32_t head,
                                              int width) {
  for (int x = 0; x < width; x += 64)
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(token), "r"(head)
                 : "memory");
}
__device__ __forceinline__ void prefetch_bytes(const char* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
// Panels [p0, p1) of a tile to memory; rows past T and channels past the width
// are not written.
__device__ __forceinline__ void store_tile(const CUtensorMap* map, uint32_t src, int32_t token,
                                           int32_t head, int p0, int p1) {
  for (int p = p0; p < p1; ++p)
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src + p * kPanel), "r"(64 * p), "r"(token), "r"(head)
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// `bytes` of shared memory to memory, both 16-byte aligned.
__device__ __forceinline__ void store_bytes(char* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The first `valid` rows of panels [p0, p1) of a staged tile to memory by 128
// threads (t), 16 bytes a lane: where the rows behind belong to another sequence.
__device__ __forceinline__ void store_rows(__nv_bfloat16* dst, const char* tile, int valid,
                                           int width, int p0, int p1, int t) {
  const int per = 8 * (p1 - p0);
  for (int e = t; e < per * valid; e += 128) {
    const int row = e / per, j = 8 * p0 + e % per;
    if (8 * j < width)
      *reinterpret_cast<uint4*>(dst + (size_t)row * width + 8 * j) =
          *reinterpret_cast<const uint4*>(tile + sw128_chunk(128, row, j));
  }
}
// This thread's stores have read their shared memory.
__device__ __forceinline__ void store_read_wait() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// 2^x, zero below 2^-126.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D[tmem] (+)= A[tmem] * B[smem]: row i of A in lane i, two bf16 a column.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 128 x N products over K = 16 KS, bf16 operands, issued by one thread.  AMN,
// BMN: the operand is stored with its K index along the rows.  One copy of the
// issue code for each pair of layouts, out of line (see the note on short loops
// below), with the descriptors' steps as constants: one that is looked up costs
// the issuing thread as long as two products take.
template <bool MN>
__device__ __forceinline__ uint64_t tile_desc(uint32_t tile) {
  return MN ? mnmajor_desc(tile, 128, 0) : kmajor_desc(tile, 128, 0);
}
// Step k of 16 along K starts 2 (k % 4) + 1024 (k / 4) units of 16 bytes
// further in a K-major tile and 128 k in an MN-major one.
template <bool MN>
__device__ __forceinline__ uint64_t desc_step(int k) {
  return MN ? 128u * k : 1024u * (k >> 2) + 2u * (k & 3);
}
template <bool AMN, bool BMN, int N = 128, int KS = 8>
static __device__ __noinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t accumulate) {
  const uint64_t da = tile_desc<AMN>(a), db = tile_desc<BMN>(b);
  umma_ss(d, da, db, idesc_f16(128, N, 1, AMN, BMN), accumulate);
#pragma unroll
  for (int k = 1; k < KS; ++k)
    umma_ss(d, da + desc_step<AMN>(k), db + desc_step<BMN>(k), idesc_f16(128, N, 1, AMN, BMN), 1);
}
template <bool BMN, int N = 128>
static __device__ __noinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b,
                                           uint32_t accumulate) {
  const uint64_t db = tile_desc<BMN>(b);
  umma_ts(d, a_tmem, db, idesc_f16(128, N, 1, 0, BMN), accumulate);
#pragma unroll
  for (int k = 1; k < 8; ++k)
    umma_ts(d, a_tmem + 8 * k, db + desc_step<BMN>(k), idesc_f16(128, N, 1, 0, BMN), 1);
}

// ----------------------------------------------------------------- waiting
// Bounded (about a second), and over at once when another warp has given up.
// Called by whole warps; the answer is the same in every lane.
static __device__ __noinline__ bool warp_wait_on(uint64_t* bar, uint32_t parity,
                                                 volatile int* abort) {
  const uint64_t start = globaltimer_ns();
  for (uint32_t i = 0; i < (1u << 24); ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity, 1000000u))) return true;
    if (__any_sync(0xffffffffu, *abort || globaltimer_ns() - start > kWaitLimitNs)) break;
  }
  *abort = 1;
  return false;
}
// One thread's look at a barrier, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity, 1000000u))) return true;
  return warp_wait_on(bar, parity, abort);
}
// A named hardware barrier waits without a limit, and faster than an mbarrier would (forward
// of 4 x 32 x 8192 208 us and 212, backward of 8 x 16 x 2048 269 and 274).  So a warp that
// has given up still meets the others in the `left` ones that they may come to.
static __device__ __noinline__ void leave_group(int id, int threads, int left) {
  for (; left > 0; --left) named_sync(id, threads);
}
// Orders this warp's shared-memory writes and TMEM accesses before the tensor
// cores' next use, and arrives once for the warp.
__device__ __forceinline__ void warp_publish(uint64_t* bar) {
  fence_proxy_async_smem();
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ------------------------------------------------------------------ decays
// Factors of a chunk of 128 tokens in four blocks of 32, from log2 decays x_t
// (zero past the end).  Sums run inside a block and over whole blocks, each
// from the side it is read from, so that no factor is the exponential of a
// difference of large sums, but for the pairs inside a block:
//   pre_t  sum of x over the block's tokens up to t
//   eL_t   exp2 of the sum from the chunk's start to t; or, with LO, in its place
//   lo_t   what the roundings of pre_t left: a block of 32 may hold resets of -160 each,
//          and pre_i - pre_j alone gives the mild decays behind four of them an error of
//          1e-4, behind sixteen 4e-4.  The decay's gradient is fp32 and takes the second
//          sum; o is bf16, its P rounded by up to 2e-3, and does without (forward of
//          4 x 32 x 8192 208 us, with it 216)
//   es_t   exp2 of the sum over the block's tokens after t
//   w_t    exp2 of the sum after t to the chunk's end
//   tot_b  sum over block b;   all = exp2 of the sum over the chunk
struct Gates {
  float pre[C];
  union {
    float eL[C], lo[C];
  };
  float es[C], w[C];
  float tot[4];
  float all;
  float pad[3];
};
// eL_t where lo has its place.
__device__ __forceinline__ float from_start(const Gates* g, int t) {
  float x = 0.f;
  for (int b = 0; b < t >> 5; ++b) x += g->tot[b];
  return ex2(x + g->pre[t]);
}
// A sum and the error of its rounding, joined to those of its terms.
template <bool LO>
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) {
  if (!LO) return make_float2(a.x + b.x, 0.f);
  const float s = a.x + b.x, t = s - a.x;
  return make_float2(s, (a.x - (s - t)) + (b.x - t) + (a.y + b.y));
}
// (q + p) + (r + l) for two columns, an instruction for both.
__device__ __forceinline__ float2 gaps(float qx, float qy, float rx, float ry, float p, float l) {
  float2 d;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%6, %6};\n"
      " add.rn.f32x2 a, a, b;\n mov.b64 b, {%4, %5};\n mov.b64 c, {%7, %7};\n"
      " add.rn.f32x2 b, b, c;\n add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(qx), "f"(qy), "f"(rx), "f"(ry), "f"(p), "f"(l));
  return d;
}
// One warp: lane l brings tokens 4l .. 4l+3.
template <bool LO>
__device__ __forceinline__ void make_gates(Gates* g, float4 x, int lane) {
  const float2 p0 = make_float2(x.x, 0.f), p1 = add_pair<LO>(p0, make_float2(x.y, 0.f));
  const float2 p2 = add_pair<LO>(p1, make_float2(x.z, 0.f)), sum = add_pair<LO>(p2, make_float2(x.w, 0.f));
  const float s2 = x.w, s1 = x.z + s2, s0 = x.y + s1;
  float2 up = sum;  // inclusive scans over the block's eight lanes
  float down = sum.x;
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) {
    const float2 a = make_float2(__shfl_up_sync(0xffffffffu, up.x, m, 8),
                                 LO ? __shfl_up_sync(0xffffffffu, up.y, m, 8) : 0.f);
    const float b = __shfl_down_sync(0xffffffffu, down, m, 8);
    if ((lane & 7) >= m) up = add_pair<LO>(up, a);
    if ((lane & 7) + m < 8) down += b;
  }
  // exclusive: shifted, not subtracted
  float2 before = make_float2(__shfl_up_sync(0xffffffffu, up.x, 1, 8),
                              LO ? __shfl_up_sync(0xffffffffu, up.y, 1, 8) : 0.f);
  float after = __shfl_down_sync(0xffffffffu, down, 1, 8);
  if ((lane & 7) == 0) before = make_float2(0.f, 0.f);
  if ((lane & 7) == 7) after = 0.f;
  const float tot = __shfl_sync(0xffffffffu, up.x, 7, 8);
  const float t0 = __shfl_sync(0xffffffffu, tot, 0), t1 = __shfl_sync(0xffffffffu, tot, 8);
  const float t2 = __shfl_sync(0xffffffffu, tot, 16), t3 = __shfl_sync(0xffffffffu, tot, 24);
  const int b = lane >> 3;
  const float later = b == 3 ? 0.f : b == 2 ? t3 : b == 1 ? t3 + t2 : t3 + t2 + t1;
  const float2 q0 = add_pair<LO>(before, p0), q1 = add_pair<LO>(before, p1), q2 = add_pair<LO>(before, p2);
  const float2 q3 = add_pair<LO>(before, sum);
  const float4 suf = make_float4(after + s0, after + s1, after + s2, after);
  reinterpret_cast<float4*>(g->pre)[lane] = make_float4(q0.x, q1.x, q2.x, q3.x);
  if (LO) {
    reinterpret_cast<float4*>(g->lo)[lane] = make_float4(q0.y, q1.y, q2.y, q3.y);
  } else {
    const float earlier = b == 0 ? 0.f : b == 1 ? t0 : b == 2 ? t0 + t1 : t0 + t1 + t2;
    reinterpret_cast<float4*>(g->eL)[lane] =
        make_float4(ex2(earlier + q0.x), ex2(earlier + q1.x), ex2(earlier + q2.x),
                    ex2(earlier + q3.x));
  }
  reinterpret_cast<float4*>(g->es)[lane] =
      make_float4(ex2(suf.x), ex2(suf.y), ex2(suf.z), ex2(suf.w));
  reinterpret_cast<float4*>(g->w)[lane] =
      make_float4(ex2(later + suf.x), ex2(later + suf.y), ex2(later + suf.z),
                  ex2(later + suf.w));
  if ((lane & 7) == 0) g->tot[b] = tot;
  if (lane == 0) g->all = ex2(t0 + t1 + t2 + t3);
}
// log2 decays of tokens 4l .. 4l+3 of a chunk, `valid` of its tokens in the sequence.
__device__ __forceinline__ float4 load_decays(const float* g, int stride, int valid, int lane) {
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    x[e] = 4 * lane + e < valid ? log2_decay(g[(size_t)(4 * lane + e) * stride]) : 0.f;
  return make_float4(x[0], x[1], x[2], x[3]);
}

// Rows [valid, 128) of a tile, row by row, set to zero (by 128 threads): tokens
// of the next packed sequence, whose values must not reach a product even with
// a factor of zero.
__device__ __forceinline__ void zero_row(char* tile, int row) {
#pragma unroll
  for (int j = 0; j < 16; ++j)
    *reinterpret_cast<uint4*>(tile + sw128_chunk(128, row, j)) = make_uint4(0, 0, 0, 0);
}

// (The loops over a row's pieces here and in the kernels are kept short on
// purpose: with a dozen warps in different code, instructions that run once a
// chunk come from beyond the instruction cache, and unrolled rows took three
// times as long.)
//
// Channels 8 j0 .. 8 j1 of a token row times w, in two bf16 parts: hi in place, lo at the
// same place of another tile.  With w = wh + wl in bf16, hi = round(k wh), what
// that rounding left is exact in bf16 (k wh has 16 bits), and k wl joins it:
// hi + lo is w k to 2^-16, in three packed operations: the fp32 states that come of it err
// by 4.3e-6 of their rms.  (One part would leave 2e-3; a third, with a product of its own
// and no room for its tile, some 2e-7.)
__device__ __forceinline__ void scale_row(char* tile, char* lo, int row, int j0, int j1,
                                          float w, bool keep) {
  const __nv_bfloat16 h = __float2bfloat16_rn(w);
  const __nv_bfloat162 wh = __bfloat162bfloat162(h);
  const __nv_bfloat162 wl = __float2bfloat162_rn(w - __bfloat162float(h));
#pragma unroll 2
  for (int j = j0; j < j1; ++j) {
    const uint32_t off = sw128_chunk(128, row, j);
    const uint4 v = *reinterpret_cast<const uint4*>(tile + off);
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t hi[4], rest[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 k = *reinterpret_cast<const __nv_bfloat162*>(&in[e]);
      const __nv_bfloat162 a = __hmul2_rn(k, wh);
      const __nv_bfloat162 b = __hfma2(k, wl, __hfma2(k, wh, __hneg2(a)));
      hi[e] = keep ? *reinterpret_cast<const uint32_t*>(&a) : 0u;
      rest[e] = keep ? *reinterpret_cast<const uint32_t*>(&b) : 0u;
    }
    *reinterpret_cast<uint4*>(tile + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(lo + off) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
  }
}

}  // namespace chunk

// The cut for these sizes, its bytes after `at`, and its tables filled in from a
// workspace; the plan of packed sequences is made on the device.
chunk::Split linear_split(int N, int B, int H, int T, bool packed);
size_t linear_split_bytes(const chunk::Split& sp, int N, int H, int dk, int dv, bool packed,
                          int directions);
cudaError_t linear_split_plan(const LinearArgs& a, chunk::Split& sp, char* ws, cudaStream_t s);
// What each segment hands on, in time (back = false: over k, v from h0) or against
// it (over q, dout from dhT), joined.  `dir`: which of the workspace's tables.
cudaError_t linear_segment_states(const LinearArgs& a, chunk::Split& sp, char* ws, bool back,
                                  int dir, cudaStream_t s);

// The state entering every chunk (back: dL/dH at every chunk's end, and dh0),
// as images.
struct ChunkImages {
  char* img;             // [chunks * H] images
  const int32_t* first;  // packed: [N + 1] first chunk of each sequence
  int chunks;            // a bound on the chunks
};
cudaError_t linear_chunk_states(const LinearArgs& a, const chunk::Split& sp, const ChunkImages& out,
                                bool back, cudaStream_t s);

// Tensor map of a [heads, T, width] bf16 tensor for load_tile.
bool linear_map(CUtensorMap* m, const void* base, uint64_t heads, uint64_t T, uint64_t width);

}  // namespace ckda
