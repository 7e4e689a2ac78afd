// ckda_linear_piece.cuh -- linear attention on CUDA cores, in pieces of 64 tokens
// side by side: the tables over pieces, and products of small matrices in shared
// memory that their kernels are made of.
//
// With H the state entering a piece, D_ij the decay from token j to token i >= j,
// e_i the one from the piece's start through i and w_j the one from j to its end,
//     A_ij = scale D_ij q_i.k_j,   o_i = scale e_i H^T q_i + sum_{j <= i} A_ij v_j,
//     (state after the piece) = e H + sum_j w_j k_j v_j^T.
// D is the exponential of a sum that runs down its column, so a decay that is strong
// or -infinity somewhere leaves the others their full precision, which a difference
// of cumulative sums would not (and 64 factors multiplied lose three bits).  Masks are taken exactly: a token's values, whatever
// they are, enter no result that they do not belong to.
#pragma once
#include <type_traits>
#include "ckda_linear.cuh"

namespace ckda {

constexpr int kTok = 64;            // tokens of a piece
constexpr int kPieceThreads = 256;
constexpr int kPS = kTok + 4;       // row of a token matrix

// Pieces of a sequence, and the tables over them.  Slot p of a sequence is the
// state entering its piece p (H) or the gradient of that state (G); the slot
// after its last piece is the final state's.
struct Pieces {
  const int32_t* slot0;   // packed: [N + 1] first slot of a sequence
  size_t slots;           // of a head
  float* H;               // [slots][H][dk][dv]
  float* G;
  float* dec;             // [slots][H] decay over the piece behind a slot
};
__host__ __device__ inline int pieces_of(int len) { return (len + kTok - 1) / kTok; }

// A piece of one (sequence, head).
struct Where {
  int n, h, piece, pieces;
  int t0, len;            // its tokens on the T axis
  size_t slot;            // of the state entering it
  size_t krow, vrow;      // row of its first token in q, k and in v, do, ...
};
// Block x runs over slots times heads, final states' slots among them; false
// where there is no piece.
__device__ __forceinline__ bool where(const LinearArgs& a, const Pieces& p, size_t block, Where& u) {
  size_t s = block / a.H;
  u.h = block % a.H;
  u.slot = s;
  if (a.cu_seqlens) {
    if (s >= (size_t)p.slot0[a.N]) return false;
    int lo = 0, hi = a.N;  // slot0[lo] <= s < slot0[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((size_t)p.slot0[mid] <= s) lo = mid; else hi = mid;
    }
    u.n = lo;
    u.piece = (int)(s - p.slot0[lo]);
  } else {
    const int per = pieces_of(a.T) + 1;
    u.n = (int)(s / per);
    u.piece = (int)(s % per);
  }
  int t0, len;
  seq_range(a, u.n, t0, len);
  u.pieces = pieces_of(len);
  u.t0 = t0 + u.piece * kTok;
  u.len = min(len - u.piece * kTok, kTok);
  const int b = a.cu_seqlens ? 0 : u.n, hk = u.h / (a.H / a.Hk);
  u.krow = ((size_t)b * a.Hk + hk) * a.T + u.t0;
  u.vrow = ((size_t)b * a.H + u.h) * a.T + u.t0;
  return true;
}

inline size_t slots_of(int N, int T, bool packed) {
  // packed: ceil(len / 64) pieces of each sequence, and a final state
  return packed ? (size_t)T / kTok + 2 * (size_t)N : (size_t)N * (pieces_of(T) + 1);
}
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
// Fills slot0 of packed sequences; what each piece adds to the states and their scan
// (directions 2: and the gradients' of them).
cudaError_t linear_plan_slots(const LinearArgs& a, int32_t* slot0, cudaStream_t s);
cudaError_t linear_join_pieces(const LinearArgs& a, const Pieces& p, int directions,
                               cudaStream_t s);

__device__ __forceinline__ void copy16(float* dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                     __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}

// Rows of n values, ss apart, into rows of `cols` (a multiple of 16) floats, stride ds, zeros
// behind them and in rows [rows, total): a warp a row.  (One copy of the code: a
// block runs most of its code once, and fetching it is a third of a short launch.)
template <typename IO>
static __device__ __noinline__ void stage_rows(float* dst, int ds, const IO* src, int ss, int n,
                                           int rows, int total, int cols) {
  constexpr uintptr_t kMask = 4 * sizeof(IO) - 1;
  const bool four = ((n | ss) & 3) == 0 && (reinterpret_cast<uintptr_t>(src) & kMask) == 0;
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int r = threadIdx.x >> 5; r < total; r += kPieceThreads / 32) {
    if (four) {
      for (int c = 4 * lane; c < cols; c += 128) {
        const bool in = r < rows && c < n;
        const IO* from = in ? src + (size_t)r * ss + c : src;
        if constexpr (sizeof(IO) == 4)
          copy16(dst + r * ds + c, from, in);
        else
          *reinterpret_cast<float4*>(dst + r * ds + c) = in ? load4(from) : make_float4(0, 0, 0, 0);
      }
    } else {
      for (int c = lane; c < cols; c += 32)
        dst[r * ds + c] = r < rows && c < n ? ld_io(src + (size_t)r * ss + c) : 0.f;
    }
  }
}

// acc[i][j] += sum_{x < n} a[i][x] b[16 j][x]; a, b at this thread's first row.
template <int C>
__device__ __forceinline__ void add_nt(float (&acc)[4][C], const float* a, int sa, const float* b,
                                       int sb, int n) {
#pragma unroll 1
  for (int x = 0; x < n; x += 4) {
    float4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const float4*>(a + i * sa + x);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(b + 16 * j * sb + x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][j] = fmaf(u[i].x, v.x, acc[i][j]);
        acc[i][j] = fmaf(u[i].y, v.y, acc[i][j]);
        acc[i][j] = fmaf(u[i].z, v.z, acc[i][j]);
        acc[i][j] = fmaf(u[i].w, v.w, acc[i][j]);
      }
    }
  }
}
// acc[i][j] += sum_{x0 <= x < x1} a[i][x] b[x][16 j], or with TA a[x][i].
template <bool TA, int C>
__device__ __forceinline__ void add_nn(float (&acc)[4][C], const float* a, int sa, const float* b,
                                       int sb, int x0, int x1) {
#pragma unroll 1
  for (int x = x0; x < x1; x += 4) {
    float u[4][4];  // [i][x]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(TA ? a + (x + i) * sa : a + i * sa + x);
      (TA ? u[0][i] : u[i][0]) = t.x;
      (TA ? u[1][i] : u[i][1]) = t.y;
      (TA ? u[2][i] : u[i][2]) = t.z;
      (TA ? u[3][i] : u[i][3]) = t.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const float v = b[(x + e) * sb + 16 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = fmaf(u[i][e], v, acc[i][j]);
      }
  }
}
// The 4 x 4 block on the diagonal, x0 + e against i: only e < i, with INCL e <= i; with
// TA e > i, e >= i.  (A short loop: code that a block runs once is fetched for it.)
template <bool TA, bool INCL, int C>
__device__ __forceinline__ void add_diag(float (&acc)[4][C], const float* a, int sa, const float* b,
                                         int sb, int x0) {
#pragma unroll 1
  for (int e = 0; e < 4; ++e) {
    float u[4];
    bool in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = TA ? a[(x0 + e) * sa + i] : a[i * sa + x0 + e];
      in[i] = (INCL && e == i) || (TA ? e > i : e < i);
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const float v = b[(x0 + e) * sb + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (in[i]) acc[i][j] = fmaf(u[i], v, acc[i][j]);
    }
  }
}

// The decays of a piece of nt tokens from their log decays g (zeros behind them) by 65
// threads: e, w, and the logarithms of D.
__device__ __forceinline__ void piece_decays(float* logD, float* e, float* w, const float* g,
                                             int nt) {
  const int tid = threadIdx.x;
  if (tid < kTok) {
    float d = 0.f;
#pragma unroll 8
    for (int i = 0; i < kTok; ++i) {
      d = i > tid ? d + g[i] : 0.f;
      logD[i * kPS + tid] = d;
      if (i == nt - 1) w[tid] = tid < nt ? expf(d) : 0.f;
    }
  } else if (tid == kTok) {
    float x = 0.f;
#pragma unroll 8
    for (int i = 0; i < kTok; ++i) e[i] = expf(x += g[i]);
  }
}
__device__ __forceinline__ void copies_arrived() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}

// Floats of a row of n columns: to a multiple of 16, and four more against bank
// conflicts.  Products over more columns than that read into the next row, and what
// they make of it is not used.
__host__ __device__ inline int row_floats(int n) { return (n + 15) / 16 * 16 + 4; }

// Calls f with the number of 16-column groups, a constant, that hold n columns.
template <typename F>
cudaError_t with_columns(int n, F f) {
  return n <= 64   ? f(std::integral_constant<int, 4>())
         : n <= 96 ? f(std::integral_constant<int, 6>())
                   : f(std::integral_constant<int, 8>());
}
// The same for a slab of key channels: 48, or 64 and one or two slabs.
template <int CK>
constexpr int kMostSlabs = CK == 4 ? 2 : 1;
template <typename F>
cudaError_t with_slab(int n, F f) {
  return n <= 48 ? f(std::integral_constant<int, 3>()) : f(std::integral_constant<int, 4>());
}

}  // namespace ckda
