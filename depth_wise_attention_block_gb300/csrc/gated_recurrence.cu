// Gated linear recurrence over packed sequences, its backward, and the form
// for single tokens.  Per channel:
//
//   a_t = sigmoid(f_t),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  out_t = h_t silu(g_t)
//   (without an output gate g: out_t = h_t).
//   backward, last token first: dh_t = dy_t silu(g_t) + a_{t+1} dh_{t+1},
//   dx = (1 - a) dh,  df = dh (h_{t-1} - x) a (1 - a),  dg = dy h silu'(g).
//
// A span of tokens acts on the state as h -> A h + B, and spans compose, so
// all rows are one scan whatever sequences they belong to: at a sequence's
// first token the state behind it is cut off (its initial state enters B).
// Every element is read once and written once: the bound is HBM.
//
// A CTA owns a slab of channels, 128 bytes of a row, and walks over the rows
// in tiles of 64, 8 rows to a warp, one 32-bit word of a row to a lane.  Each
// warp copies its own rows ahead (cp.async, a ring of its own), so a tile takes
// one barrier: the warps' (A, B) meet in shared memory and each warp goes on
// from the state at its first row.  Where the slabs do not fill the GPU, a
// cluster of R CTAs shares a slab: they take R neighbouring tiles at a time and
// exchange the tiles' (A, B) through distributed shared memory.  The backward
// walks from the last tile to the first; the states ahead of each tile, which
// the forward kept, let it form h_{t-1} again without a second scan.
#include <limits.h>
#include <math.h>

#include "attnres.h"
#include "body.h"
#include "device_common.cuh"
#include "launch.h"
#include "vec16.cuh"

namespace attnres {

namespace {

constexpr int kGrChunk = ATTNRES_RECURRENCE_CHUNK;  // rows of a tile
constexpr int kGrWarps = 8;
constexpr int kGrRows = kGrChunk / kGrWarps;        // of a warp
constexpr int kGrThreads = 32 * kGrWarps;
constexpr int kGrRowBytes = 128;                    // of a slab
#ifndef GR_FS
#define GR_FS 2
#define GR_FB 3
#define GR_BS 2
#define GR_BB 2
#define GR_MAXR 8
#endif
constexpr int kGrStages = GR_FS, kGrBwdStages = GR_BS;          // tiles of a warp's ring
constexpr int kGrBlocksPerSm = GR_FB, kGrBwdBlocksPerSm = GR_BB;  // resident CTAs
constexpr int kGrMaxCluster = GR_MAXR;
constexpr int kGsThreads = 256;

__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ float rcp(float x) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
constexpr float kLog2e = 1.44269504f;

// a = 1 / (1 + e^-f) and rest = 1 - a, neither by a difference.  f below -83
// counts as -83 (a = 1e-36), where e^-f would leave fp32; NaN stays NaN.  For
// bf16 tensors the fast exponential and reciprocal (2^-22 each, far below the
// results' 2^-8), for fp32 ones the full functions.
template <typename T>
__device__ __forceinline__ void forget(float f, float* a, float* rest) {
  if constexpr (sizeof(T) == 2) {
    const float e = ex2(min_nan(-kLog2e * f, 120.f));
    *a = rcp(1.f + e);
    *rest = e * *a;
  } else {
    const float e = expf(min_nan(-f, 83.f));
    *a = 1.f / (1.f + e);
    *rest = e * *a;
  }
}
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(T) == 2) return rcp(1.f + ex2(-kLog2e * z));
  else return 1.f / (1.f + expf(-z));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {  // the rest of 16: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, const float (&v)[4]) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, const float (&v)[2]) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v[0]), "f"(v[1]) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// How the rows of a tensor lie: 16-byte vectors, 32-bit words, or elements.
enum RowAccess { kVectors = 0, kWords = 1, kElements = 2 };

struct GrParams {
  RecurrenceArgs a;
  int ranks;       // CTAs of a cluster
  int groups;      // tiles of a CTA: ceil(tiles / ranks)
  int access[4];   // of x, f, g and (backward) dout
  int words_out;   // every row tensor written lies on 32-bit words
};

// The channels of a lane: one 32-bit word of a row.
template <typename T>
struct Word {
  static constexpr int N = 4 / sizeof(T);
  static __device__ __forceinline__ void unpack(uint32_t w, float (&v)[N]) {
    if constexpr (N == 2) {
      v[0] = bf16lo(w);
      v[1] = bf16hi(w);
    } else {
      v[0] = __uint_as_float(w);
    }
  }
  static __device__ __forceinline__ uint32_t pack(const float (&v)[N]) {
    if constexpr (N == 2) return pack_bf16x2(v[0], v[1]);
    else return __float_as_uint(v[0]);
  }
  // row: the row's slab; in: how many of the lane's channels there are
  static __device__ __forceinline__ void store(T* row, int lane, int in, bool words, const float (&v)[N]) {
    if (in == N && words) {
      *reinterpret_cast<uint32_t*>(row + lane * N) = pack(v);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < in) store_elem(row + lane * N + e, v[e]);
    }
  }
};

// One warp's copy of its 8 rows from t0 on into shared memory, rows of 128
// bytes; zeros where there is no row or channel.
template <typename T>
__device__ __forceinline__ void fetch_rows(uint32_t dst, const void* src, long long stride, long long t0, long long T_, int c0, int C,
                                           int access, int lane) {
  constexpr int N = Word<T>::N;
  const T* base = static_cast<const T*>(src);
  if (access == kVectors) {
    constexpr int V = 16 / sizeof(T);
    const int v = lane & 7, left = C - c0 - v * V;
    const int bytes = left >= V ? 16 : left > 0 ? left * (int)sizeof(T) : 0;
#pragma unroll
    for (int i = 0; i < kGrRows / 4; ++i) {
      const int r = (lane >> 3) + 4 * i;
      const int n = t0 + r < T_ ? bytes : 0;
      cp_async16(dst + r * kGrRowBytes + v * 16, n > 0 ? base + (t0 + r) * stride + c0 + v * V : base, n);
    }
  } else {
    const int in = C - c0 - lane * N;
#pragma unroll
    for (int r = 0; r < kGrRows; ++r) {
      const bool row = t0 + r < T_ && in > 0;
      const T* at = base + (row ? (t0 + r) * stride + c0 + lane * N : 0);
      const uint32_t to = dst + r * kGrRowBytes + lane * 4;
      if (access == kWords) {
        cp_async4(to, row ? at : base, !row ? 0 : in >= N ? 4 : (int)sizeof(T));
      } else {  // (bf16 off the 32-bit words)
        uint32_t w = 0;
        if (row) w = *reinterpret_cast<const uint16_t*>(at);
        if (row && in >= N) w |= (uint32_t) * reinterpret_cast<const uint16_t*>(at + N - 1) << 16;
        st_shared_u32(to, w);
      }
    }
  }
}

__device__ __forceinline__ int clamp_row(int r, int T_) { return r < 0 ? 0 : r > T_ ? T_ : r; }

// Which of a warp's 8 rows begin and end a sequence, and of which sequence.
// The offsets are looked through in one direction as the tiles go by: `j` is
// the first offset not below the rows (forward) or the first one above all
// earlier-visited rows' lower end (backward starts a new search).
struct Marks {
  uint32_t starts, ends;
};
// smallest index in [lo, N + 1] whose offset is not below t (N + 1: none), given that offset lo - 1 is below
__device__ __forceinline__ int lower_bound(const int* cu, int N, int T_, int t, int lo, int lane) {
  int hi = N + 1;
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool below = at < hi && clamp_row(__ldg(cu + at), T_) < t;
    const int k = __popc(__ballot_sync(0xffffffffu, below));  // probes below: the first of them, in order
    if (k == 0) return lo;
    const int from = lo + (k - 1) * step + 1, to = lo + k * step;
    lo = from;
    hi = to < hi ? to : hi;
  }
  const bool below = lo + lane < hi && clamp_row(__ldg(cu + lo + lane), T_) < t;
  return lo + __popc(__ballot_sync(0xffffffffu, below));
}

__device__ __forceinline__ Marks find_marks(const int* cu, int N, int T_, int t0, int j, int* seqs, int lane) {
  Marks m{0, 0};
  for (int base = j; base <= N; base += 32) {
    const int i = base + lane;
    const int b = i <= N ? clamp_row(__ldg(cu + i), T_) : INT_MAX;
    uint32_t st = 0, en = 0;
    if (i < N && b >= t0 && b < t0 + kGrRows && clamp_row(__ldg(cu + i + 1), T_) > b) {
      st = 1u << (b - t0);
      seqs[b - t0] = i;
    }
    if (i >= 1 && b > t0 && b <= t0 + kGrRows && clamp_row(__ldg(cu + i - 1), T_) < b) {
      en = 1u << (b - 1 - t0);
      seqs[kGrRows + b - 1 - t0] = i - 1;
    }
    m.starts |= __reduce_or_sync(0xffffffffu, st);
    m.ends |= __reduce_or_sync(0xffffffffu, en);
    if (__shfl_sync(0xffffffffu, b, 31) > t0 + kGrRows) break;
  }
  __syncwarp();
  return m;
}

// The marks of one warp's rows, tile after tile in either direction.
struct Boundaries {
  int j, next;  // forward: the first offset not below the last rows looked at, and its value
  __device__ __forceinline__ Marks rows(const RecurrenceArgs& a, int t0, int* seqs, int lane, bool descending) {
    const int T_ = (int)a.T;
    if (!a.cu) {
      Marks m{t0 == 0 ? 1u : 0u, t0 < T_ && T_ <= t0 + kGrRows ? 1u << (T_ - 1 - t0) : 0u};
      if (lane < 2 * kGrRows) seqs[lane] = 0;
      __syncwarp();
      return m;
    }
    if (descending) {
      // `next`: the largest offset not above the last rows looked at
      if (next < t0) return {0, 0};
      j = lower_bound(a.cu, a.N, T_, t0, 0, lane);
      next = j > 0 ? clamp_row(__ldg(a.cu + j - 1), T_) : -1;
    } else if (next < t0) {
      j = lower_bound(a.cu, a.N, T_, t0, j + 1, lane);
      next = j <= a.N ? clamp_row(__ldg(a.cu + j), T_) : INT_MAX;
    }
    if (!descending && next > t0 + kGrRows) return {0, 0};
    return find_marks(a.cu, a.N, T_, t0, j, seqs, lane);
  }
};

// the state of every empty sequence goes on unchanged (from: its states or null)
__device__ __forceinline__ void pass_empty(const RecurrenceArgs& a, const float* from, float* to, int rank, int ranks, int c, int in, int warp,
                                           int lane) {
  if (!to) return;
  const int T_ = (int)a.T;
  for (int base = (rank * kGrWarps + warp) * 32; base < a.N; base += ranks * kGrWarps * 32) {
    const int i = base + lane;
    const bool none = i < a.N && (a.cu ? clamp_row(__ldg(a.cu + i + 1), T_) <= clamp_row(__ldg(a.cu + i), T_) : T_ == 0);
    for (uint32_t left = __ballot_sync(0xffffffffu, none); left; left &= left - 1) {
      const long long at = (long long)(base + __ffs(left) - 1) * a.C + c;
      for (int e = 0; e < in; ++e) to[at + e] = from ? from[at + e] : 0.f;
    }
  }
}

// (A, B) of a span followed by (A2, B2); a cut span forgets what is behind it
__device__ __forceinline__ float carry_on(float c, float A, float B, bool cut) { return cut ? B : fmaf(A, c, B); }

template <typename T>
struct GrShared {
  static constexpr int N = Word<T>::N;
  float warps[2][kGrWarps][32][2 * N];          // (A, B) per channel of the tile's warps; two tiles in turn
  int warp_cut[2][kGrWarps], rank_cut[2][kGrMaxCluster];
  int seqs[kGrWarps][2 * kGrRows];
};

// After a tile's warps have left their (A, B) in sh: the state ahead of this
// CTA's tile, for the lane's channels (state: the one ahead of the cluster's
// tiles, and then the one behind them).  of_ranks: [2][ranks], the (A, B) of the
// cluster's tiles, two sets in turn.  REV: spans follow one another from the
// last row to the first.
template <typename T, bool REV>
__device__ __forceinline__ void exchange(GrShared<T>& sh, float (*of_ranks)[32][2 * Word<T>::N], int par, int rank, int ranks, int warp, int lane, float (&state)[Word<T>::N],
                                         float (&ahead)[Word<T>::N]) {
  constexpr int N = Word<T>::N;
  auto nth = [](int i, int n) { return REV ? n - 1 - i : i; };
  if (ranks == 1) {
#pragma unroll
    for (int e = 0; e < N; ++e) ahead[e] = state[e];
#pragma unroll
    for (int i = 0; i < kGrWarps; ++i) {
      const int w = nth(i, kGrWarps);
      const bool cut = sh.warp_cut[par][w];
#pragma unroll
      for (int e = 0; e < N; ++e) state[e] = carry_on(state[e], sh.warps[par][w][lane][2 * e], sh.warps[par][w][lane][2 * e + 1], cut);
    }
    return;
  }
  if (warp == 0) {  // the tile's own (A, B), to every CTA of the cluster
    float v[2 * N];
    bool any = false;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      v[2 * e] = 1.f;
      v[2 * e + 1] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kGrWarps; ++i) {
      const int w = nth(i, kGrWarps);
      const bool cut = sh.warp_cut[par][w];
      any |= cut;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float A = sh.warps[par][w][lane][2 * e], B = sh.warps[par][w][lane][2 * e + 1];
        v[2 * e + 1] = carry_on(v[2 * e + 1], A, B, cut);
        v[2 * e] *= A;
      }
    }
    const uint32_t at = smem_addr(&of_ranks[par * ranks + rank][lane][0]), flag = smem_addr(&sh.rank_cut[par][rank]);
    for (int r = 0; r < ranks; ++r) {
      st_cluster(map_shared_rank(at, r), v);
      if (lane == 0) st_cluster(map_shared_rank(flag, r), (int)any);
    }
  }
  cluster_sync_all();
  for (int i = 0; i < ranks; ++i) {
    const int r = nth(i, ranks);
    if (r == rank) {
#pragma unroll
      for (int e = 0; e < N; ++e) ahead[e] = state[e];
    }
    const bool cut = sh.rank_cut[par][r];
#pragma unroll
    for (int e = 0; e < N; ++e) state[e] = carry_on(state[e], of_ranks[par * ranks + r][lane][2 * e], of_ranks[par * ranks + r][lane][2 * e + 1], cut);
  }
}

// the state at this warp's first row (REV: behind its last), from the one ahead of the tile
template <typename T, bool REV>
__device__ __forceinline__ void through_warps(const GrShared<T>& sh, int par, int warp, int lane, float (&c)[Word<T>::N]) {
  constexpr int N = Word<T>::N;
  const int n = REV ? kGrWarps - 1 - warp : warp;
  for (int i = 0; i < n; ++i) {
    const int w = REV ? kGrWarps - 1 - i : i;
    const bool cut = sh.warp_cut[par][w];
#pragma unroll
    for (int e = 0; e < N; ++e) c[e] = carry_on(c[e], sh.warps[par][w][lane][2 * e], sh.warps[par][w][lane][2 * e + 1], cut);
  }
}

template <typename T, bool GATE>
__global__ void __launch_bounds__(kGrThreads, kGrBlocksPerSm) gr_forward_kernel(const __grid_constant__ GrParams p) {
  constexpr int N = Word<T>::N, kArrays = GATE ? 3 : 2, kBytes = kArrays * kGrRows * kGrRowBytes;
  extern __shared__ __align__(128) unsigned char ring_mem[];  // [warp][stage][array][row], then the exchange of a cluster
  __shared__ __align__(16) GrShared<T> sh;
  const RecurrenceArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = p.ranks, rank = ranks > 1 ? (int)cluster_ctarank() : 0;
  const int c0 = blockIdx.x / ranks * (kGrRowBytes / (int)sizeof(T)), c = c0 + lane * N;
  const int in = a.C - c < 0 ? 0 : a.C - c < N ? a.C - c : N;  // channels of this lane
  const int T_ = (int)a.T;
  const uint32_t ring = smem_addr(ring_mem) + warp * (kGrStages * kBytes);
  auto of_ranks = reinterpret_cast<float (*)[32][2 * N]>(ring_mem + kGrWarps * kGrStages * kBytes);
  if (ranks > 1) cluster_sync_all();  // every CTA of the cluster is there
  pdl_wait();
  pdl_trigger();

  auto row0 = [&](int i) { return (i * ranks + rank) * kGrChunk + warp * kGrRows; };
  auto fetch = [&](int i) {
    if (i < p.groups) {
      const uint32_t to = ring + i % kGrStages * kBytes;
      fetch_rows<T>(to, a.x, a.xs, row0(i), a.T, c0, a.C, p.access[0], lane);
      fetch_rows<T>(to + kGrRows * kGrRowBytes, a.f, a.fs, row0(i), a.T, c0, a.C, p.access[1], lane);
      if constexpr (GATE) fetch_rows<T>(to + 2 * kGrRows * kGrRowBytes, a.g, a.gs, row0(i), a.T, c0, a.C, p.access[2], lane);
    }
    cp_async_commit();  // a group for every tile, there or not
  };
  for (int i = 0; i < kGrStages - 1; ++i) fetch(i);
  pass_empty(a, a.s0, a.s1, rank, ranks, c, in, warp, lane);
  const int first = a.cu ? clamp_row(__ldg(a.cu), T_) : 0, last = a.cu ? clamp_row(__ldg(a.cu + a.N), T_) : T_;
  Boundaries bounds{0, first};
  float state[N];
#pragma unroll
  for (int e = 0; e < N; ++e) state[e] = 0.f;

  for (int i = 0; i < p.groups; ++i) {
    const int t0 = row0(i), par = i & 1;
    __syncwarp();  // the slot that is filled next has been read
    fetch(i + kGrStages - 1);
    const Marks m = bounds.rows(a, t0, sh.seqs[warp], lane, false);
    cp_async_wait<kGrStages - 1>();
    __syncwarp();
    const uint32_t at = ring + i % kGrStages * kBytes + lane * 4;

    // the rows from a state of zero: h = hl + pa * (the state ahead), hl alone behind a first token
    float hl[kGrRows][N], pa[kGrRows][N], A[N], B[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      A[e] = 1.f;
      B[e] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < kGrRows; ++k) {
      float x[N], f[N], h0[N];
      Word<T>::unpack(ld_shared_u32(at + k * kGrRowBytes), x);
      Word<T>::unpack(ld_shared_u32(at + (kGrRows + k) * kGrRowBytes), f);
      const bool start = m.starts >> k & 1;
      if (start) {
        const long long s = (long long)sh.seqs[warp][k] * a.C + c;
#pragma unroll
        for (int e = 0; e < N; ++e) h0[e] = a.s0 && e < in ? a.s0[s + e] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float g, rest;
        forget<T>(f[e], &g, &rest);
        B[e] = fmaf(g, start ? h0[e] : B[e], rest * x[e]);
        A[e] *= g;
        hl[k][e] = B[e];
        pa[k][e] = A[e];
      }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      sh.warps[par][warp][lane][2 * e] = A[e];
      sh.warps[par][warp][lane][2 * e + 1] = B[e];
    }
    if (lane == 0) sh.warp_cut[par][warp] = m.starts != 0;
    __syncthreads();
    float h[N];
    exchange<T, false>(sh, of_ranks, par, rank, ranks, warp, lane, state, h);
    if (warp == 0 && a.chunk && t0 < T_) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < in) a.chunk[(long long)(t0 / kGrChunk) * a.C + c + e] = h[e];
    }
    through_warps<T, false>(sh, par, warp, lane, h);

    T* o = static_cast<T*>(a.out) + (long long)t0 * a.os + c0;
#pragma unroll
    for (int k = 0; k < kGrRows; ++k) {
      float v[N], g[N];
      const bool cut = m.starts & ((2u << k) - 1);
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = cut ? hl[k][e] : fmaf(pa[k][e], h[e], hl[k][e]);
      if (a.s1 && (m.ends >> k & 1)) {
        const long long s = (long long)sh.seqs[warp][kGrRows + k] * a.C + c;
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e < in) a.s1[s + e] = v[e];
      }
      if constexpr (GATE) {
        Word<T>::unpack(ld_shared_u32(at + (2 * kGrRows + k) * kGrRowBytes), g);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] *= g[e] * sigmoid<T>(g[e]);
      }
      if (t0 + k >= first && t0 + k < last) Word<T>::store(o + k * a.os, lane, in, p.words_out, v);
    }
  }
}

template <typename T, bool GATE>
__global__ void __launch_bounds__(kGrThreads, kGrBwdBlocksPerSm) gr_backward_kernel(const __grid_constant__ GrParams p) {
  constexpr int N = Word<T>::N, kArrays = GATE ? 4 : 3, kBytes = kArrays * kGrRows * kGrRowBytes, kArray = kGrRows * kGrRowBytes;
  extern __shared__ __align__(128) unsigned char ring_mem[];  // [warp][stage][array][row], then the exchange of a cluster
  __shared__ __align__(16) GrShared<T> sh;
  __shared__ float fwd_b[2][kGrWarps][32][N];  // the forward's B of the tile's warps
  __shared__ int fwd_cut[2][kGrWarps];
  const RecurrenceArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = p.ranks, rank = ranks > 1 ? (int)cluster_ctarank() : 0;
  const int c0 = blockIdx.x / ranks * (kGrRowBytes / (int)sizeof(T)), c = c0 + lane * N;
  const int in = a.C - c < 0 ? 0 : a.C - c < N ? a.C - c : N;
  const int T_ = (int)a.T;
  const uint32_t ring = smem_addr(ring_mem) + warp * (kGrBwdStages * kBytes);
  auto of_ranks = reinterpret_cast<float (*)[32][2 * N]>(ring_mem + kGrWarps * kGrBwdStages * kBytes);
  if (ranks > 1) cluster_sync_all();  // every CTA of the cluster is there
  pdl_wait();
  pdl_trigger();

  auto row0 = [&](int i) { return ((p.groups - 1 - i) * ranks + rank) * kGrChunk + warp * kGrRows; };
  auto fetch = [&](int i) {
    if (i < p.groups) {
      const uint32_t to = ring + i % kGrBwdStages * kBytes;
      fetch_rows<T>(to, a.x, a.xs, row0(i), a.T, c0, a.C, p.access[0], lane);
      fetch_rows<T>(to + kArray, a.f, a.fs, row0(i), a.T, c0, a.C, p.access[1], lane);
      fetch_rows<T>(to + 2 * kArray, a.dout, a.dos, row0(i), a.T, c0, a.C, p.access[3], lane);
      if constexpr (GATE) fetch_rows<T>(to + 3 * kArray, a.g, a.gs, row0(i), a.T, c0, a.C, p.access[2], lane);
    }
    cp_async_commit();
  };
  for (int i = 0; i < kGrBwdStages - 1; ++i) fetch(i);
  pass_empty(a, a.ds1, a.ds0, rank, ranks, c, in, warp, lane);
  const int first = a.cu ? clamp_row(__ldg(a.cu), T_) : 0, last = a.cu ? clamp_row(__ldg(a.cu + a.N), T_) : T_;
  Boundaries bounds{0, INT_MAX};
  float state[N];  // the gradient at the state behind the rows not yet visited
#pragma unroll
  for (int e = 0; e < N; ++e) state[e] = 0.f;

  for (int i = 0; i < p.groups; ++i) {
    const int t0 = row0(i), par = i & 1;
    __syncwarp();
    fetch(i + kGrBwdStages - 1);
    float hf[N];  // the state ahead of the tile
#pragma unroll
    for (int e = 0; e < N; ++e) hf[e] = t0 < T_ && e < in ? a.chunk[(long long)(t0 / kGrChunk) * a.C + c + e] : 0.f;
    const Marks m = bounds.rows(a, t0, sh.seqs[warp], lane, true);
    cp_async_wait<kGrBwdStages - 1>();
    __syncwarp();
    const uint32_t at = ring + i % kGrBwdStages * kBytes + lane * 4;

    float ga[kGrRows][N], rest[kGrRows][N], d[kGrRows][N], sg[GATE ? kGrRows : 1][N];
    float A[N], B[N], R[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      A[e] = 1.f;
      B[e] = R[e] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < kGrRows; ++k) {
      float x[N], f[N], h0[N];
      Word<T>::unpack(ld_shared_u32(at + k * kGrRowBytes), x);
      Word<T>::unpack(ld_shared_u32(at + kArray + k * kGrRowBytes), f);
      Word<T>::unpack(ld_shared_u32(at + 2 * kArray + k * kGrRowBytes), d[k]);
      if constexpr (GATE) {
        float g[N];
        Word<T>::unpack(ld_shared_u32(at + 3 * kArray + k * kGrRowBytes), g);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          sg[k][e] = sigmoid<T>(g[e]);
          d[k][e] *= g[e] * sg[k][e];
        }
      }
      if (a.ds1 && (m.ends >> k & 1)) {
        const long long s = (long long)sh.seqs[warp][kGrRows + k] * a.C + c;
#pragma unroll
        for (int e = 0; e < N; ++e) d[k][e] += e < in ? a.ds1[s + e] : 0.f;
      }
      const bool start = m.starts >> k & 1;
      if (start) {
        const long long s = (long long)sh.seqs[warp][k] * a.C + c;
#pragma unroll
        for (int e = 0; e < N; ++e) h0[e] = a.s0 && e < in ? a.s0[s + e] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        forget<T>(f[e], &ga[k][e], &rest[k][e]);
        B[e] = fmaf(ga[k][e], start ? h0[e] : B[e], rest[k][e] * x[e]);
        A[e] *= ga[k][e];
      }
    }
#pragma unroll
    for (int k = kGrRows - 1; k >= 0; --k) {
      const bool end = m.ends >> k & 1;
#pragma unroll
      for (int e = 0; e < N; ++e) R[e] = ga[k][e] * (end ? d[k][e] : d[k][e] + R[e]);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      sh.warps[par][warp][lane][2 * e] = A[e];
      sh.warps[par][warp][lane][2 * e + 1] = R[e];
      fwd_b[par][warp][lane][e] = B[e];
    }
    if (lane == 0) {
      sh.warp_cut[par][warp] = m.ends != 0;
      fwd_cut[par][warp] = m.starts != 0;
    }
    __syncthreads();
    float G[N];
    exchange<T, true>(sh, of_ranks, par, rank, ranks, warp, lane, state, G);
    through_warps<T, true>(sh, par, warp, lane, G);
    for (int w = 0; w < warp; ++w) {
      const bool cut = fwd_cut[par][w];
#pragma unroll
      for (int e = 0; e < N; ++e) hf[e] = carry_on(hf[e], sh.warps[par][w][lane][2 * e], fwd_b[par][w][lane][e], cut);
    }
    // the states ahead of the rows
    float hp[kGrRows][N];
#pragma unroll
    for (int k = 0; k < kGrRows; ++k) {
      float x[N];
      Word<T>::unpack(ld_shared_u32(at + k * kGrRowBytes), x);
      if (m.starts >> k & 1) {
        const long long s = (long long)sh.seqs[warp][k] * a.C + c;
#pragma unroll
        for (int e = 0; e < N; ++e) hf[e] = a.s0 && e < in ? a.s0[s + e] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        hp[k][e] = hf[e];
        hf[e] = fmaf(ga[k][e], hf[e], rest[k][e] * x[e]);
      }
    }
    T* dx = static_cast<T*>(a.dx) + (a.dx ? (long long)t0 * a.dxs + c0 : 0);
    T* df = static_cast<T*>(a.df) + (a.df ? (long long)t0 * a.dfs + c0 : 0);
    T* dg = static_cast<T*>(a.dg) + (a.dg ? (long long)t0 * a.dgs + c0 : 0);
#pragma unroll
    for (int k = kGrRows - 1; k >= 0; --k) {
      const bool end = m.ends >> k & 1, live = t0 + k >= first && t0 + k < last;
      float x[N], vx[N], vf[N], vg[N];
      Word<T>::unpack(ld_shared_u32(at + k * kGrRowBytes), x);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float dh = end ? d[k][e] : d[k][e] + G[e];
        vx[e] = rest[k][e] * dh;
        vf[e] = dh * (hp[k][e] - x[e]) * (ga[k][e] * rest[k][e]);
        G[e] = ga[k][e] * dh;
      }
      if constexpr (GATE) {
        float g[N], dy[N];
        Word<T>::unpack(ld_shared_u32(at + 3 * kArray + k * kGrRowBytes), g);
        Word<T>::unpack(ld_shared_u32(at + 2 * kArray + k * kGrRowBytes), dy);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float h = fmaf(ga[k][e], hp[k][e], rest[k][e] * x[e]), s = sg[k][e];
          vg[e] = dy[e] * h * fmaf(g[e] * s, 1.f - s, s);
        }
        if (live && a.dg) Word<T>::store(dg + k * a.dgs, lane, in, p.words_out, vg);
      }
      if (live && a.dx) Word<T>::store(dx + k * a.dxs, lane, in, p.words_out, vx);
      if (live && a.df) Word<T>::store(df + k * a.dfs, lane, in, p.words_out, vf);
      if (a.ds0 && (m.starts >> k & 1)) {
        const long long s = (long long)sh.seqs[warp][k] * a.C + c;
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e < in) a.ds0[s + e] = G[e];
      }
    }
  }
}

// One token per row: a CTA owns a row's channels, and goes on through the
// later rows of the same slot.
template <typename T>
__global__ void __launch_bounds__(kGsThreads) gr_step_kernel(const __grid_constant__ RecurrenceStepArgs p) {
  __shared__ int next_row;
  const int tid = threadIdx.x, c = blockIdx.x * kGsThreads + tid;
  int row = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const int slot = p.slots ? __ldg(p.slots + row) : row;
  if (slot < 0 || slot >= p.num_slots) return;  // a padding row
  float* st = p.state + (long long)slot * p.C + c;
  const bool in = c < p.C;
  float h = in ? *st : 0.f;
  if (p.slots) {  // rows of one slot belong to the CTA of the first of them
    bool later = false;
    for (int i = tid; i < row; i += kGsThreads) later |= __ldg(p.slots + i) == slot;
    if (__syncthreads_or(later)) return;
  }
  for (;;) {
    if (in) {
      float a, rest;
      forget<T>(load_elem(static_cast<const T*>(p.f) + row * p.fs + c), &a, &rest);
      h = fmaf(a, h, rest * load_elem(static_cast<const T*>(p.x) + row * p.xs + c));
      float o = h;
      if (p.g) {
        const float g = load_elem(static_cast<const T*>(p.g) + row * p.gs + c);
        o *= g * sigmoid<T>(g);
      }
      store_elem(static_cast<T*>(p.out) + row * p.os + c, o);
    }
    if (!p.slots) break;
    if (tid == 0) next_row = p.B;
    __syncthreads();
    for (int i = row + 1 + tid; i < p.B; i += kGsThreads)
      if (__ldg(p.slots + i) == slot) {
        atomicMin(&next_row, i);
        break;
      }
    __syncthreads();
    row = next_row;
    if (row >= p.B) break;
    __syncthreads();  // every thread has read next_row
  }
  if (in) *st = h;
}

int row_access(const void* p, int64_t stride, int es) {
  if (!p) return kVectors;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p), step = (uintptr_t)stride * es;
  return ((at | step) & 15) == 0 ? kVectors : ((at | step) & 3) == 0 ? kWords : kElements;
}

// CTAs to a slab: the GPU's slots filled as evenly as they can be, by as few
// CTAs as do it (each doubling has to take off a tenth).
int choose_ranks(int64_t tiles, int64_t slabs, int slots) {
  int best = 1;
  double least = 1e300;
  for (int r = 1; r <= kGrMaxCluster && r <= tiles; r *= 2) {
    const double cost = (double)((slabs * r + slots - 1) / slots) / r;
    if (cost < 0.9 * least) {
      least = cost;
      best = r;
    }
  }
  return best;
}

template <typename K>
cudaError_t launch_gr(K kern, SmemOptIn& opt, const RecurrenceArgs& a, int arrays, int stages, int blocks_per_sm) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const int es = a.dtype == ATTNRES_BF16 ? 2 : 4, ring = kGrWarps * stages * arrays * kGrRows * kGrRowBytes;
  const int per_rank = 2 * 32 * (8 / es) * (int)sizeof(float);  // of the exchange
  e = opt.ensure(reinterpret_cast<const void*>(kern), ring + kGrMaxCluster * per_rank);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.T + kGrChunk - 1) / kGrChunk, width = kGrRowBytes / es, slabs = (a.C + width - 1) / width;
  GrParams p{};
  p.a = a;
  p.ranks = choose_ranks(tiles, slabs, di.sm_count * blocks_per_sm);
  p.groups = (int)((tiles + p.ranks - 1) / p.ranks);
  const void* in[4] = {a.x, a.f, a.g, a.dout};
  const int64_t strides[4] = {a.xs, a.fs, a.gs, a.dos};
  for (int i = 0; i < 4; ++i) p.access[i] = row_access(in[i], strides[i], es);
  p.words_out = row_access(a.out, a.os, es) <= kWords && row_access(a.dx, a.dxs, es) <= kWords &&
                row_access(a.df, a.dfs, es) <= kWords && row_access(a.dg, a.dgs, es) <= kWords;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(slabs * p.ranks));
  cfg.blockDim = dim3(kGrThreads);
  cfg.dynamicSmemBytes = ring + (p.ranks > 1 ? p.ranks * per_rank : 0);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (p.ranks > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = p.ranks;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T, bool GATE>
cudaError_t launch_forward(const RecurrenceArgs& a) {
  static SmemOptIn opt;
  return launch_gr(gr_forward_kernel<T, GATE>, opt, a, GATE ? 3 : 2, kGrStages, kGrBlocksPerSm);
}
template <typename T, bool GATE>
cudaError_t launch_backward(const RecurrenceArgs& a) {
  static SmemOptIn opt;
  return launch_gr(gr_backward_kernel<T, GATE>, opt, a, GATE ? 4 : 3, kGrBwdStages, kGrBwdBlocksPerSm);
}

}  // namespace

cudaError_t launch_gated_recurrence(const RecurrenceArgs& a) {
  if (a.dtype == ATTNRES_BF16) return a.g ? launch_forward<bf16_t, true>(a) : launch_forward<bf16_t, false>(a);
  return a.g ? launch_forward<float, true>(a) : launch_forward<float, false>(a);
}

cudaError_t launch_gated_recurrence_backward(const RecurrenceArgs& a) {
  if (a.dtype == ATTNRES_BF16) return a.g ? launch_backward<bf16_t, true>(a) : launch_backward<bf16_t, false>(a);
  return a.g ? launch_backward<float, true>(a) : launch_backward<float, false>(a);
}

cudaError_t launch_gated_recurrence_step(const RecurrenceStepArgs& a) {
  const dim3 grid((a.C + kGsThreads - 1) / kGsThreads, a.B);
  return a.dtype == ATTNRES_BF16 ? launch_kernel(gr_step_kernel<bf16_t>, grid, dim3(kGsThreads), 0, a.stream, a)
                                 : launch_kernel(gr_step_kernel<float>, grid, dim3(kGsThreads), 0, a.stream, a);
}

}  // namespace attnres
