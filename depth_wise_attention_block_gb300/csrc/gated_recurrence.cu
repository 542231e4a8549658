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
// Every element is read once and written once: the floor is HBM's.
//
// A CTA owns a slab of 64 channels, two to a lane (one packed pair of fp32),
// and walks over the rows in tiles of 64.  Forward: 4 warps, 16 rows each, the
// rows' h from a zero state and the products of their gates in registers; the
// warps' (A, B) meet in shared memory, and each warp goes on from the state at
// its first row.  More rows to a warp leave more registers' worth of work
// between two meetings: 8 warps with 8 rows took 280 us where this takes 187.
// Backward: 8 warps, 8 rows each, from the last tile to the first; of a row
// e^-f and the state ahead of it are kept, the rest is formed again, because
// there the registers decide how many warps there are (80 a thread, 24 warps
// to an SM; 4 warps of 16 rows at 128: 248 us where forward and backward
// together took 230).  The states ahead of the tiles, which the forward kept,
// let it form h_{t-1} without a second scan over the rows.
//
// Where the slabs do not fill the GPU, a cluster of R CTAs shares a slab: they
// take R neighbouring tiles at a time and send the tiles' (A, B) through
// distributed shared memory.  With one CTA to a slab instead: 427 us where 187
// (16384 x 7168), 195 where 38 (5003 x 1000).
//
// Rows of whole 16-byte vectors move by TMA, a box to a warp, and the results
// go out the same way, which costs a lane no address: the warps' instructions
// are what bounds the kernels once every tensor passes once.  Rows on 32-bit
// words come by cp.async (8192 x 4094 bf16: 132 us where 4096 channels take
// 72), bf16 rows on single elements through registers (4095: 205); both leave
// by words.
//
// All figures here are single calls with cold caches; among other calls the
// forward of 16384 x 7168 takes 182 us and that of 5003 x 1000 30.  Gate and all
// gradients, HBM traffic of one pass over each tensor:
// 16384 x 7168 bf16 forward 187 us, 5.0 TB/s, backward 459 us, 3.6 TB/s;
// 8192 x 4096 bf16 in 5 sequences 72 us, 3.7 TB/s, and 140 us, 3.4 TB/s; the
// same of fp32 99 us, 5.4 TB/s, and 191 us, 4.9 TB/s (the copy: 6.8).  What
// bounds them: for each pair of channels some 75 instructions forward and 130
// backward, at 51 % of the issue slots (forward of 8192 x 4096: 39 %), the rest
// lost to the latency of a warp's own chain with at most 16 and 24 warps to an SM
// and to fetching instructions (a second form of the backward's stores beside the
// boxes cost a tenth without running).  And not every place on the SMs is taken:
// the CTAs of 16384 x 7168 fill 0.92 of them, those of 8192 x 4096 0.84 in both
// directions, with SMs that hold none beside full ones.
#include <limits.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "attnres.h"
#include "body.h"
#include "device_common.cuh"
#include "launch.h"
#include "tc_common.cuh"
#include "vec16.cuh"

namespace attnres {

namespace {

constexpr int kGrChunk = ATTNRES_RECURRENCE_CHUNK;  // rows of a tile
constexpr int kGrMaxCluster = 16;
constexpr int kGsThreads = 256;

// ---------------------------------------------------------- arithmetic ---

__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
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
__device__ __forceinline__ float f2_low(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo;
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) { return f2_fma(b, f2_both(-1.f), a); }
__device__ __forceinline__ uint64_t f2_neg(uint64_t a) { return f2_mul(a, f2_both(-1.f)); }
// log2 e as the sum of two fp32 numbers
constexpr float kLog2e = 1.44269504f, kLog2eLow = (float)(1.4426950408889634074 - (double)1.44269504f);

// 1 / (1 + e^-z) on both halves, and e^-z, with the hardware's power of two
// and reciprocal (2^-22 each).  For fp32 tensors the product z log2 e, whose
// rounding would cost |z| 2^-24 of e, is the unevaluated sum of two numbers
// (Dekker's product, by fma), the second entering as a factor 1 + ln 2 * it.
template <typename T>
__device__ __forceinline__ uint64_t f2_sigmoid(uint64_t z, uint64_t* e) {
  float a, b;
  if constexpr (sizeof(T) == 4) {  // (of an infinity the product has no second number; at 100 e^-z is 0 already)
    f2_unpack(z, a, b);
    z = f2_pack(min_nan(a, 100.f), min_nan(b, 100.f));
  }
  const uint64_t hi = f2_mul(z, f2_both(-kLog2e));
  f2_unpack(hi, a, b);
  *e = f2_pack(ex2(a), ex2(b));
  if constexpr (sizeof(T) == 4) {
    const uint64_t lo = f2_fma(z, f2_both(-kLog2eLow), f2_fma(z, f2_both(-kLog2e), f2_neg(hi)));
    *e = f2_fma(*e, f2_mul(lo, f2_both(0.69314718f)), *e);
  }
  f2_unpack(f2_add(*e, f2_both(1.f)), a, b);
  return f2_pack(rcp(a), rcp(b));
}

// 1 / (1 + e) on both halves: a gate's value again from its e^-z
__device__ __forceinline__ uint64_t f2_open(uint64_t e) {
  float a, b;
  f2_unpack(f2_add(e, f2_both(1.f)), a, b);
  return f2_pack(rcp(a), rcp(b));
}

// One value of it: a gate z (below -83 as -83) gives sigma and 1 - sigma.
template <typename T>
__device__ __forceinline__ float sigmoid(float z, float* rest) {
  uint64_t e;
  const float s = f2_low(f2_sigmoid<T>(f2_both(-min_nan(-z, 83.f)), &e));
  *rest = f2_low(e) * s;
  return s;
}

// -------------------------------------------------- the channels of a lane --

// N (two) channels of one row: a lane's 4 or 8 bytes in memory, N / 2 packed
// pairs of fp32 in registers.
template <typename T, int N>
struct Lane {
  static constexpr int P = N / 2;
  static constexpr int kBytes = N * (int)sizeof(T);
  static constexpr int kWords = kBytes / 4;
  struct Raw {
    uint32_t w[kWords];
  };
  static __device__ __forceinline__ Raw load(uint32_t addr) {
    Raw r;
    if constexpr (kWords == 2) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(addr));
    else asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.w[0]) : "r"(addr));
    return r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, uint64_t (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if constexpr (sizeof(T) == 2) v[i] = f2_pack(bf16lo(r.w[i]), bf16hi(r.w[i]));
      else v[i] = f2_pack(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    }
  }
  static __device__ __forceinline__ void load(uint32_t addr, uint64_t (&v)[P]) { unpack(load(addr), v); }
  // a gate: values below -83 count as -83, where e^-z would leave fp32 (NaN stays NaN)
  static __device__ __forceinline__ void load_gate(uint32_t addr, uint64_t (&v)[P]) {
    Raw r = load(addr);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 2) r.w[i] = max_nan_bf16x2(r.w[i], 0xC2A6C2A6u);  // -83
      else r.w[i] = __float_as_uint(-min_nan(-__uint_as_float(r.w[i]), 83.f));
    }
    unpack(r, v);
  }
  // the forget gate's a and 1 - a (not by a difference)
  static __device__ __forceinline__ void forgets(uint32_t addr, uint64_t (&a)[P], uint64_t (&rest)[P]) {
    uint64_t f[P];
    load_gate(addr, f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      uint64_t e;
      a[i] = f2_sigmoid<T>(f[i], &e);
      rest[i] = f2_mul(e, a[i]);
    }
  }
  // results, rounded to T, into shared memory
  static __device__ __forceinline__ void stage(uint32_t addr, const uint64_t (&v)[P]) {
    float f[N];
#pragma unroll
    for (int i = 0; i < P; ++i) f2_unpack(v[i], f[2 * i], f[2 * i + 1]);
    if constexpr (sizeof(T) == 2) {
      static_assert(N == 2, "a word");
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(pack_bf16x2(f[0], f[1])) : "memory");
    } else {
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(f[0]), "f"(f[1]) : "memory");
    }
  }
  // fp32 states in device memory, and in shared memory
  static __device__ __forceinline__ void load_state(const float* at, int in, uint64_t (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = f2_pack(2 * i < in ? at[2 * i] : 0.f, 2 * i + 1 < in ? at[2 * i + 1] : 0.f);
  }
  static __device__ __forceinline__ void store_state(float* at, int in, const uint64_t (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float a, b;
      f2_unpack(v[i], a, b);
      if (2 * i < in) at[2 * i] = a;
      if (2 * i + 1 < in) at[2 * i + 1] = b;
    }
  }
  static __device__ __forceinline__ void get(const uint64_t (&at)[P], uint64_t (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = at[i];
  }
  static __device__ __forceinline__ void put(uint64_t (&at)[P], const uint64_t (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) at[i] = v[i];
  }
  // into a CTA of the cluster, counted by its mbarrier
  static __device__ __forceinline__ void put_cluster(uint32_t addr, const uint64_t (&v)[P], uint32_t bar) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(addr + 8 * i), "l"(v[i]), "r"(bar)
                   : "memory");
  }
};

// ------------------------------------------------------------ rows ahead --

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {  // the rest of 4: zeros
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// a box of shared memory to a tensor (rows and columns outside it are left out)
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x),
               "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

struct GrParams {
  CUtensorMap in[4], out[3];  // x, f, g, dout; out or dx, df, dg (tma): boxes of a warp's rows
  RecurrenceArgs a;
  int ranks;     // CTAs of a cluster
  int groups;    // tiles of a CTA: ceil(tiles / ranks)
  int tma;       // every row is whole 16-byte vectors: boxes by TMA
  int words[4];  // otherwise: x, f, g, dout lie on 32-bit words
  unsigned long long wait_ns;  // limit of a wait
  int withhold;  // the bounded-wait test: the first tile's spans are not sent
};

constexpr int kBoxAlign = 128;  // of a box in shared memory
__device__ __forceinline__ unsigned char* aligned_box(unsigned char* dyn) { return dyn + (0u - smem_addr(dyn)) % kBoxAlign; }

// One warp's copy of its rows from t0 on (channels c0 and up, N to a lane)
// into shared memory where they do not lie on 16-byte vectors; zeros where
// there is no row or channel.
template <typename T, int N, int ROWS>
__device__ __forceinline__ void fetch_rows(uint32_t dst, const void* src, long long stride, int t0, int T_, int c0, int C, int words,
                                           int lane) {
  constexpr int kRow = 32 * Lane<T, N>::kBytes, E = 4 / sizeof(T);  // elements of a word
  const T* base = static_cast<const T*>(src);
  if (words) {
    const int c = lane * E, e = 32 * E;  // neighbouring lanes, neighbouring words
    const T* row = base + (long long)t0 * stride + c0 + c;
    dst += lane * 4;
    if (t0 + ROWS <= T_ && c0 + 32 * (int)Lane<T, N>::kWords * E <= C) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r, row += stride)
#pragma unroll
        for (int i = 0; i < Lane<T, N>::kWords; ++i) cp_async4(dst + r * kRow + i * 128, row + i * e, 4);
    } else {
      for (int r = 0; r < ROWS; ++r, row += stride)
#pragma unroll
        for (int i = 0; i < Lane<T, N>::kWords; ++i) {
          const int in = t0 + r < T_ ? C - c0 - c - i * e : 0;
          cp_async4(dst + r * kRow + i * 128, in > 0 ? row + i * e : base, in >= E ? 4 : in > 0 ? (int)sizeof(T) : 0);
        }
    }
  } else {  // bf16 off the words: by way of registers, some rows at a time
    constexpr int kBatch = 4;
    const int left = C - c0 - 2 * lane;
    const uint16_t* row = reinterpret_cast<const uint16_t*>(base) + (long long)t0 * stride + c0 + 2 * lane;
    for (int r = 0; r < ROWS; r += kBatch) {
      uint32_t w[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k, row += stride) {
        const int in = t0 + r + k < T_ ? left : 0;
        w[k] = in > 0 ? row[0] : 0;
        if (in > 1) w[k] |= (uint32_t)row[1] << 16;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) st_shared_u32(dst + (r + k) * kRow + lane * 4, w[k]);
    }
  }
}

// Rows of results from shared memory to those of from .. to - 1 among t0 ..: by
// words, whatever boundaries they lie on.  (A function of its own: in line it
// costs the rows that leave as boxes one part in a hundred.)
template <typename T, int N, int ROWS>
__device__ __noinline__ void put_rows(uint32_t src, void* dst, long long stride, int t0, int from, int to, int c0, int C, int lane) {
  constexpr int kRow = 32 * Lane<T, N>::kBytes;
  const int r0 = from > t0 ? from - t0 : 0, r1 = to - t0 < ROWS ? to - t0 : ROWS;
  src += r0 * kRow;
  T* row = static_cast<T*>(dst) + (long long)(t0 + r0) * stride + c0;
#pragma unroll 2
  for (int r = r0; r < r1; ++r, row += stride, src += kRow) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < Lane<T, N>::kWords; ++i)
        if (c0 + i * 32 + lane < C) reinterpret_cast<uint32_t*>(row)[i * 32 + lane] = ld_shared_u32(src + (i * 32 + lane) * 4);
    } else {
      const int left = C - c0 - 2 * lane;
      uint16_t* to = reinterpret_cast<uint16_t*>(row) + 2 * lane;
      const uint32_t own = ld_shared_u32(src + lane * 4);
      if (reinterpret_cast<uintptr_t>(row) & 2) {  // the words lie an element ahead of the lanes'
        const uint32_t before = __shfl_up_sync(0xffffffffu, own, 1);
        if (left > 0 && lane > 0) *reinterpret_cast<uint32_t*>(to - 1) = __funnelshift_l(before, own, 16);
        if (lane == 0) to[0] = (uint16_t)own;
        if (left > 1 && (lane == 31 || left == 2)) to[1] = (uint16_t)(own >> 16);
      } else {
        if (left > 1) *reinterpret_cast<uint32_t*>(to) = own;
        else if (left > 0) to[0] = (uint16_t)own;
      }
    }
  }
}

// A warp's boxes on their way, a phase of `bar` for each tile.  A wait that
// runs out ends the loads (an open phase takes no second arrival).
struct Boxes {
  uint32_t bar;
  bool landed;
  __device__ __forceinline__ void wait(int i, unsigned long long limit_ns) {
    if (landed) landed = __all_sync(0xffffffffu, mbar_wait_bounded(bar, (uint32_t)i & 1u, limit_ns));
  }
  // what is still on its way is not to outlive the CTA's memory
  __device__ __forceinline__ void settle() const {
    if (!landed)
      for (uint32_t parity = 0; parity < 2; ++parity) mbar_wait_bounded(bar, parity);
  }
};

// ------------------------------------------------------------- sequences --

__device__ __forceinline__ int clamp_row(int r, int T_) { return r < 0 ? 0 : r > T_ ? T_ : r; }

// The smallest index in [lo, N + 1] whose offset is not below t (N + 1: none),
// given that those before lo are below.
__device__ __forceinline__ int lower_bound(const int* cu, int N, int T_, int t, int lo, int lane) {
  int hi = N + 1;
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool below = at < hi && clamp_row(__ldg(cu + at), T_) < t;
    const int k = __popc(__ballot_sync(0xffffffffu, below));  // the first k probes
    if (k == 0) return lo;
    const int to = lo + k * step;
    lo += (k - 1) * step + 1;
    hi = to < hi ? to : hi;
  }
  const bool below = lo + lane < hi && clamp_row(__ldg(cu + lo + lane), T_) < t;
  return lo + __popc(__ballot_sync(0xffffffffu, below));
}

// Which of a warp's rows begin and end a sequence: bit k for row t0 + k, the
// sequences in seqs[k] and seqs[rows + k].
struct Marks {
  uint32_t starts, ends;
};
// j: the first offset not below t0
__device__ __noinline__ Marks find_marks(const int* cu, int N, int T_, int t0, int rows, int j, int* seqs, int lane) {
  Marks m{0, 0};
  for (int base = j; base <= N; base += 32) {
    const int i = base + lane;
    const int b = i <= N ? clamp_row(__ldg(cu + i), T_) : INT_MAX;
    uint32_t st = 0, en = 0;
    if (i < N && b >= t0 && b < t0 + rows && clamp_row(__ldg(cu + i + 1), T_) > b) {
      st = 1u << (b - t0);
      seqs[b - t0] = i;
    }
    if (i >= 1 && b > t0 && b <= t0 + rows && clamp_row(__ldg(cu + i - 1), T_) < b) {
      en = 1u << (b - 1 - t0);
      seqs[rows + b - 1 - t0] = i - 1;
    }
    m.starts |= __reduce_or_sync(0xffffffffu, st);
    m.ends |= __reduce_or_sync(0xffffffffu, en);
    if (__shfl_sync(0xffffffffu, b, 31) > t0 + rows) break;
  }
  __syncwarp();
  return m;
}

// The marks of a warp's rows, tile after tile in either direction: the offsets
// are searched only when the rows reach the next one.
template <int ROWS, bool REV>
struct Boundaries {
  int j, next;  // the first offset not below the rows last looked at, and its value (REV: that of the one before)
  __device__ __forceinline__ void begin(int first) {
    j = 0;
    next = REV ? INT_MAX : first;
  }
  __device__ __forceinline__ Marks rows(const RecurrenceArgs& a, int t0, int* seqs, int lane) {
    const int T_ = (int)a.T;
    if (!a.cu) {
      const Marks m{t0 == 0 ? 1u : 0u, t0 < T_ && T_ <= t0 + ROWS ? 1u << (T_ - 1 - t0) : 0u};
      if (m.starts | m.ends) {
        if (lane < 2 * ROWS) seqs[lane] = 0;
        __syncwarp();
      }
      return m;
    }
    if (REV ? next < t0 : next > t0 + ROWS) return {0, 0};
    if (REV) {
      j = lower_bound(a.cu, a.N, T_, t0, 0, lane);
      next = j > 0 ? clamp_row(__ldg(a.cu + j - 1), T_) : -1;
    } else if (next < t0) {
      j = lower_bound(a.cu, a.N, T_, t0, j + 1, lane);
      next = j <= a.N ? clamp_row(__ldg(a.cu + j), T_) : INT_MAX;
      if (next > t0 + ROWS) return {0, 0};
    }
    return find_marks(a.cu, a.N, T_, t0, ROWS, j, seqs, lane);
  }
};

// the states of empty sequences go on unchanged (from: or null, zeros)
__device__ __forceinline__ void pass_empty(const RecurrenceArgs& a, const float* from, float* to, int rank, int ranks, int c, int in, int warp,
                                           int warps, int lane) {
  if (!to) return;
  const int T_ = (int)a.T;
  for (int base = (rank * warps + warp) * 32; base < a.N; base += ranks * warps * 32) {
    const int i = base + lane;
    const bool none = i < a.N && (a.cu ? clamp_row(__ldg(a.cu + i + 1), T_) <= clamp_row(__ldg(a.cu + i), T_) : T_ == 0);
    for (uint32_t left = __ballot_sync(0xffffffffu, none); left; left &= left - 1) {
      const long long at = (long long)(base + __ffs(left) - 1) * a.C + c;
      for (int e = 0; e < in; ++e) to[at + e] = from ? from[at + e] : 0.f;
    }
  }
}

// ---------------------------------------------- spans: h -> A h + B ------

// What a tile's warps leave for one another, two tiles in turn.  A span that a
// sequence begins in (REV: ends in) is cut: it forgets the state behind it
// (by choice and not by A = 0: infinities do not pass).
template <int P, int W, int ROWS>
struct alignas(16) GrShared {
  uint64_t A[2][W][32][P], B[2][W][32][P];
  uint64_t state[2][32][P];  // of a CTA alone: ahead of its tile
  uint64_t loads[W][2];  // mbarriers: a warp's boxes have landed
  uint64_t before[3], after[3];  // mbarriers: a cluster's spans ahead of this CTA's tile are here; the others, its own among them
  unsigned char cut[2][8];  // a byte for each warp
  uint32_t rank_cut[3][kGrMaxCluster];
  int seqs[W][2 * ROWS];
};
// of a cluster's tiles
template <int P>
struct RankSpan {
  uint64_t A[32][P], B[32][P];
};

template <int P>
__device__ __forceinline__ void carry_on(uint64_t (&c)[P], const uint64_t (&A)[P], const uint64_t (&B)[P], bool cut) {
#pragma unroll
  for (int i = 0; i < P; ++i) c[i] = cut ? B[i] : f2_fma(A[i], c[i], B[i]);
}

// c through the spans of the warps before this one (REV: behind it); cuts: a
// byte for each warp
template <typename L, int W, bool REV>
__device__ __forceinline__ void through_warps(const uint64_t (&A)[W][32][L::P], const uint64_t (&B)[W][32][L::P],
                                              uint64_t cuts, int warp, int lane, uint64_t (&c)[L::P]) {
  const int n = REV ? W - 1 - warp : warp;
  uint64_t a[L::P], b[L::P];
  if (cuts == 0) {
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      if (i == n) break;
      const int w = REV ? W - 1 - i : i;
      L::get(A[w][lane], a);
      L::get(B[w][lane], b);
      carry_on(c, a, b, false);
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int w = REV ? W - 1 - i : i;
      L::get(A[w][lane], a);
      L::get(B[w][lane], b);
      carry_on(c, a, b, cuts >> (8 * w) & 1);
    }
  }
}

// A cluster's CTAs in the order of their tiles: `turn` (REV: the last rank
// first).  Each goes on from the spans ahead of its own tile: those of the
// earlier turns, and before them those of the tiles that the later turns had
// before this one.  So a CTA only waits for work that precedes it, and the
// later turns may fall behind the earlier ones by most of a tile.  The spans
// lie in three sets, tile i's in set i % 3: a CTA sends tile i + 3's after it
// has received for tile i + 2, for which every other has sent its tile i + 1's
// (and those of an earlier turn tile i + 2's), hence used what it got of tile i.

// Behind a barrier after the warps' spans, by one warp: the tile's span to
// every CTA of the cluster.  (Behind a wait that ran out, ok = false, the
// barriers' phases are open without an arrival to come; a second one there is
// not allowed.  The spans that the others still send are few: they stop in
// turn when these stay away.)
template <typename L, int W, int ROWS, bool REV>
__device__ __forceinline__ void send_span(GrShared<L::P, W, ROWS>& sh, RankSpan<L::P>* spans, int par, int set, int turn, int ranks,
                                          bool send, int lane) {
  constexpr int P = L::P;
  const uint64_t cuts = *reinterpret_cast<const uint64_t*>(sh.cut[par]);
  uint64_t a[P], b[P];
#pragma unroll
  for (int e = 0; e < P; ++e) {
    a[e] = f2_both(1.f);
    b[e] = 0;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int w = REV ? W - 1 - i : i;
    uint64_t wa[P], wb[P];
    L::get(sh.A[par][w][lane], wa);
    L::get(sh.B[par][w][lane], wb);
    carry_on(b, wa, wb, cuts >> (8 * w) & 1);
#pragma unroll
    for (int e = 0; e < P; ++e) a[e] = f2_mul(a[e], wa[e]);
  }
  const uint32_t at = smem_addr(&spans[set * ranks + turn].A[lane][0]), bt = smem_addr(&spans[set * ranks + turn].B[lane][0]);
  const uint32_t before = smem_addr(&sh.before[set]), after = smem_addr(&sh.after[set]), flag = smem_addr(&sh.rank_cut[set][turn]);
  if (lane == 0) {
    constexpr uint32_t kBytes = sizeof(RankSpan<P>) + 4;
    mbar_arrive_expect_tx(before, turn * kBytes + (send ? 0u : 4u));  // (the bounded-wait test: more than will come)
    mbar_arrive_expect_tx(after, (ranks - turn) * kBytes);
  }
  if (!send) return;
#pragma unroll 1
  for (int t = 0; t < ranks; ++t) {  // the receiver's turn
    const int r = REV ? ranks - 1 - t : t;
    const uint32_t bar = map_shared_rank(turn < t ? before : after, r);
    L::put_cluster(map_shared_rank(at, r), a, bar);
    L::put_cluster(map_shared_rank(bt, r), b, bar);
    if (lane == 0)
      asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(map_shared_rank(flag, r)),
                   "r"((uint32_t)(cuts != 0)), "r"(bar)
                   : "memory");
  }
}

// c through the spans of turns from .. to - 1 of a set
template <typename L, int W, int ROWS>
__device__ __forceinline__ void through_turns(const GrShared<L::P, W, ROWS>& sh, const RankSpan<L::P>* spans, int set, int from, int to,
                                              int ranks, int lane, uint64_t (&c)[L::P]) {
  const uint32_t cut = __ballot_sync(0xffffffffu, lane < ranks && sh.rank_cut[set][lane & (kGrMaxCluster - 1)] != 0);
  const RankSpan<L::P>* span = spans + set * ranks + from;
#pragma unroll 4
  for (int t = from; t < to; ++t, ++span) {
    uint64_t a[L::P], b[L::P];
    L::get(span->A[lane], a);
    L::get(span->B[lane], b);
    carry_on(c, a, b, cut >> t & 1);
  }
}

// The state at this warp's first row (REV: the gradient behind its last), h,
// and the one at the CTA's tile, ahead.  A, B: the warp's own span.  state: the
// one that was at the CTA's last tile.  ok: becomes false where the cluster's
// spans did not arrive in time (and then nothing is waited for any more).
template <typename L, int W, int ROWS, bool REV>
__device__ __forceinline__ void receive(GrShared<L::P, W, ROWS>& sh, RankSpan<L::P>* spans, int i, int turn, int ranks,
                                        unsigned long long limit_ns, bool& ok, int warp, int lane, const uint64_t (&A)[L::P],
                                        const uint64_t (&B)[L::P], uint64_t (&state)[L::P], uint64_t (&h)[L::P]) {
  constexpr int P = L::P;
  const int par = i & 1;
  const uint64_t cuts = *reinterpret_cast<const uint64_t*>(sh.cut[par]);
  if (ranks == 1) {
    L::get(sh.state[par][lane], state);
  } else {
    if (i > 0) {
      const int set = (i - 1) % 3;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_cluster_bounded(smem_addr(&sh.after[set]), (uint32_t)((i - 1) / 3) & 1u, limit_ns));
      through_turns<L, W, ROWS>(sh, spans, set, turn, ranks, ranks, lane, state);
    }
    const int set = i % 3;
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_cluster_bounded(smem_addr(&sh.before[set]), (uint32_t)(i / 3) & 1u, limit_ns));
    through_turns<L, W, ROWS>(sh, spans, set, 0, turn, ranks, lane, state);
    if (!ok) {
#pragma unroll
      for (int e = 0; e < P; ++e) state[e] = f2_both(__int_as_float(0x7fc00000));
    }
  }
#pragma unroll
  for (int e = 0; e < P; ++e) h[e] = state[e];
  through_warps<L, W, REV>(sh.A[par], sh.B[par], cuts, warp, lane, h);
  if (ranks == 1 && (REV ? warp == 0 : warp == W - 1)) {
    uint64_t c[P];
#pragma unroll
    for (int e = 0; e < P; ++e) c[e] = h[e];
    carry_on(c, A, B, cuts >> (8 * warp) & 1);
    L::put(sh.state[par ^ 1][lane], c);
  }
}

// Ahead of a kernel's end: what others still send to this CTA's last tile has
// come, and no CTA leaves while another may write into it.
template <int P, int W, int ROWS>
__device__ __forceinline__ void leave(GrShared<P, W, ROWS>& sh, int groups, int ranks, unsigned long long limit_ns, bool ok, int* dev_err,
                                      int lane) {
  if (ranks > 1 && ok && groups > 0)
    ok = mbar_wait_cluster_bounded(smem_addr(&sh.after[(groups - 1) % 3]), (uint32_t)((groups - 1) / 3) & 1u, limit_ns);
  if (!ok && lane == 0) report_error(dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
  if (lane == 0) bulk_wait_read();
  __syncwarp();
  if (ranks > 1) cluster_sync_all();
}

// --------------------------------------------------------------- forward --

constexpr int kGfWarps = 4, kGfRows = kGrChunk / kGfWarps;

template <typename T, bool GATE>
__global__ void __launch_bounds__(32 * kGfWarps, 4) gr_forward_kernel(const __grid_constant__ GrParams p) {
  constexpr int N = 2;
  using L = Lane<T, N>;
  constexpr int P = L::P, kRow = 32 * L::kBytes, kArray = kGfRows * kRow, kArrays = GATE ? 4 : 3;
  extern __shared__ unsigned char dyn[];  // [warp][x, f, out, g][row], then the spans of a cluster's tiles
  __shared__ GrShared<P, kGfWarps, kGfRows> sh;
  const RecurrenceArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = p.ranks, rank = ranks > 1 ? (int)cluster_ctarank() : 0;
  const int c0 = blockIdx.x / ranks * (32 * N), c = c0 + lane * N;
  const int in = a.C - c < 0 ? 0 : a.C - c < N ? a.C - c : N;  // channels of this lane
  const int T_ = (int)a.T;
  unsigned char* const arrays = aligned_box(dyn);
  const uint32_t ring = smem_addr(arrays) + warp * (kArrays * kArray), staged = ring + 2 * kArray;
  auto spans = reinterpret_cast<RankSpan<P>*>(arrays + kGfWarps * kArrays * kArray);
  const uint64_t zero[P] = {};
  if (warp == 0) L::put(sh.state[0][lane], zero);
  if (threadIdx.x < 2) *reinterpret_cast<uint64_t*>(sh.cut[threadIdx.x]) = 0;
  if (lane < 2) mbar_init(smem_addr(&sh.loads[warp][lane]), 1);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      mbar_init(smem_addr(&sh.before[i]), 1);
      mbar_init(smem_addr(&sh.after[i]), 1);
    }
  }
  mbar_fence_init();
  __syncthreads();
  if (ranks > 1) cluster_sync_all();  // every CTA of the cluster is there, its barriers ready
  bool ok = true;
  pdl_wait();
  pdl_trigger();

  auto row0 = [&](int i) { return (i * ranks + rank) * kGrChunk + warp * kGfRows; };
  Boxes xf{smem_addr(&sh.loads[warp][0]), true}, gs{smem_addr(&sh.loads[warp][1]), true};
  auto fetch_xf = [&](int i) {
    if (p.tma) {
      if (lane == 0 && i < p.groups && xf.landed) {
        mbar_arrive_expect_tx(xf.bar, 2 * kArray);
        tma_load_2d(ring, &p.in[0], c0, row0(i), xf.bar);
        tma_load_2d(ring + kArray, &p.in[1], c0, row0(i), xf.bar);
      }
    } else {
      if (i < p.groups) {
        fetch_rows<T, N, kGfRows>(ring, a.x, a.xs, row0(i), T_, c0, a.C, p.words[0], lane);
        fetch_rows<T, N, kGfRows>(ring + kArray, a.f, a.fs, row0(i), T_, c0, a.C, p.words[1], lane);
      }
      cp_async_commit();  // a group for every tile, there or not
    }
  };
  auto fetch_g = [&](int i) {
    if (p.tma) {
      if (lane == 0 && i < p.groups && gs.landed) {
        mbar_arrive_expect_tx(gs.bar, kArray);
        tma_load_2d(ring + 3 * kArray, &p.in[2], c0, row0(i), gs.bar);
      }
    } else {
      if (i < p.groups) fetch_rows<T, N, kGfRows>(ring + 3 * kArray, a.g, a.gs, row0(i), T_, c0, a.C, p.words[2], lane);
      cp_async_commit();
    }
  };
  auto wait = [&](Boxes& boxes, int i) {
    if (p.tma) {
      boxes.wait(i, p.wait_ns);
      ok = ok && boxes.landed;
    } else {
      cp_async_wait<GATE ? 1 : 0>();
      __syncwarp();
    }
  };
  fetch_xf(0);
  if constexpr (GATE) fetch_g(0);
  pass_empty(a, a.s0, a.s1, rank, ranks, c, in, warp, kGfWarps, lane);
  const int first = a.cu ? clamp_row(__ldg(a.cu), T_) : 0, last = a.cu ? clamp_row(__ldg(a.cu + a.N), T_) : T_;
  Boundaries<kGfRows, false> bounds;
  bounds.begin(first);
  uint64_t state[P];
#pragma unroll
  for (int e = 0; e < P; ++e) state[e] = 0;

  for (int i = 0; i < p.groups; ++i) {
    const int t0 = row0(i), par = i & 1;
    __syncwarp();  // the last rows' marks have been read
    const Marks m = bounds.rows(a, t0, sh.seqs[warp], lane);
    wait(xf, i);
    const uint32_t at = ring + lane * L::kBytes;

    // the rows from a state of zero: h = hl + pa * (the state ahead), hl alone behind a first token
    uint64_t hl[kGfRows][P], pa[kGfRows][P], A[P], B[P];
#pragma unroll
    for (int e = 0; e < P; ++e) {
      A[e] = f2_both(1.f);
      B[e] = 0;
    }
    // (the rows without a branch where no sequence begins among them)
    auto scan = [&](auto starts) {
#pragma unroll
      for (int k = 0; k < kGfRows; ++k) {
        uint64_t x[P], g[P], rest[P];
        L::load(at + k * kRow, x);
        L::forgets(at + kArray + k * kRow, g, rest);
        if constexpr (starts.value) {
          if (m.starts >> k & 1) L::load_state(a.s0 + (a.s0 ? (long long)sh.seqs[warp][k] * a.C + c : 0), a.s0 ? in : 0, B);
        }
#pragma unroll
        for (int e = 0; e < P; ++e) {
          B[e] = f2_fma(g[e], B[e], f2_mul(rest[e], x[e]));
          A[e] = f2_mul(A[e], g[e]);
          hl[k][e] = B[e];
          pa[k][e] = A[e];
        }
      }
    };
    if (m.starts == 0) scan(std::false_type{});
    else scan(std::true_type{});
    L::put(sh.A[par][warp][lane], A);
    L::put(sh.B[par][warp][lane], B);
    if (lane == 0) sh.cut[par][warp] = m.starts != 0;
    __syncwarp();  // x and f have been read
    fetch_xf(i + 1);
    __syncthreads();
    if (ranks > 1 && ok && warp == kGfWarps - 1)
      send_span<L, kGfWarps, kGfRows, false>(sh, spans, par, i % 3, rank, ranks, !(p.withhold && i == 0), lane);
    uint64_t h[P];
    receive<L, kGfWarps, kGfRows, false>(sh, spans, i, rank, ranks, p.wait_ns, ok, warp, lane, A, B, state, h);
    if (warp == 0 && a.chunk && t0 < T_) L::store_state(a.chunk + (long long)(t0 / kGrChunk) * a.C + c, in, state);
    if (m.starts == 0) {
#pragma unroll
      for (int k = 0; k < kGfRows; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e) hl[k][e] = f2_fma(pa[k][e], h[e], hl[k][e]);
    } else {
#pragma unroll
      for (int k = 0; k < kGfRows; ++k)
        if (!(m.starts & ((2u << k) - 1)))
#pragma unroll
          for (int e = 0; e < P; ++e) hl[k][e] = f2_fma(pa[k][e], h[e], hl[k][e]);
    }
    if constexpr (GATE) wait(gs, i);
    if (!ok) {
#pragma unroll
      for (int k = 0; k < kGfRows; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e) hl[k][e] = f2_both(__int_as_float(0x7fc00000));
    }
    if (m.ends && a.s1) {
#pragma unroll
      for (int k = 0; k < kGfRows; ++k)
        if (m.ends >> k & 1) L::store_state(a.s1 + (long long)sh.seqs[warp][kGfRows + k] * a.C + c, in, hl[k]);
    }
    // (twice in the code: around one copy of it the compiler holds more at once,
    // 197 us where these take 187)
    auto finish = [&]() {
#pragma unroll
      for (int k = 0; k < kGfRows; ++k) {
        if constexpr (GATE) {
          uint64_t g[P], e;
          L::load_gate(at + 3 * kArray + k * kRow, g);
#pragma unroll
          for (int q = 0; q < P; ++q) hl[k][q] = f2_mul(hl[k][q], f2_mul(g[q], f2_sigmoid<T>(g[q], &e)));
        }
        L::stage(staged + lane * L::kBytes + k * kRow, hl[k]);
      }
    };
    // (a box leaves out rows behind the tensor's end, but not those outside every sequence)
    if (p.tma && t0 >= first && (t0 + kGfRows <= last || last == T_)) {
      if (lane == 0) bulk_wait_read();  // of the last tile's box
      __syncwarp();
      finish();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && t0 < T_) {
        tma_store_2d(&p.out[0], c0, t0, staged);
        bulk_commit();
      }
    } else {
      if (lane == 0) bulk_wait_read();
      __syncwarp();
      finish();
      __syncwarp();
      put_rows<T, N, kGfRows>(staged, a.out, a.os, t0, first, last, c0, a.C, lane);
    }
    if constexpr (GATE) {
      __syncwarp();  // g has been read
      fetch_g(i + 1);
    }
  }
  xf.settle();
  gs.settle();
  leave(sh, p.groups, ranks, p.wait_ns, ok, a.dev_err, lane);
}

// -------------------------------------------------------------- backward --

constexpr int kGbWarps = 8, kGbRows = kGrChunk / kGbWarps;

template <typename T, bool GATE>
__global__ void __launch_bounds__(32 * kGbWarps, sizeof(T) == 2 ? 3 : 2) gr_backward_kernel(const __grid_constant__ GrParams p) {
  constexpr int N = 2;
  using L = Lane<T, N>;
  constexpr int P = L::P, kRow = 32 * L::kBytes, kArray = kGbRows * kRow, kArrays = GATE ? 4 : 3;
  // [warp][x, f, dy, g][row], then the spans of a cluster's tiles.  A row's
  // gradients take its places: dx that of x, df that of f, dg that of g.
  extern __shared__ unsigned char dyn[];
  __shared__ GrShared<P, kGbWarps, kGbRows> sh;
  __shared__ alignas(16) uint64_t fwd_B[2][kGbWarps][32][P];  // the forward's spans; their A is that of the gradients
  __shared__ alignas(8) unsigned char fwd_cut[2][8];
  const RecurrenceArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = p.ranks, rank = ranks > 1 ? (int)cluster_ctarank() : 0;
  const int c0 = blockIdx.x / ranks * (32 * N), c = c0 + lane * N;
  const int in = a.C - c < 0 ? 0 : a.C - c < N ? a.C - c : N;
  const int T_ = (int)a.T;
  unsigned char* const arrays = aligned_box(dyn);
  const uint32_t ring = smem_addr(arrays) + warp * (kArrays * kArray);
  auto spans = reinterpret_cast<RankSpan<P>*>(arrays + kGbWarps * kArrays * kArray);
  const uint64_t zero[P] = {};
  if (threadIdx.x < 2) *reinterpret_cast<uint64_t*>(fwd_cut[threadIdx.x]) = 0;
  if (warp == 0) L::put(sh.state[0][lane], zero);
  if (threadIdx.x < 2) *reinterpret_cast<uint64_t*>(sh.cut[threadIdx.x]) = 0;
  if (lane < 2) mbar_init(smem_addr(&sh.loads[warp][lane]), 1);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      mbar_init(smem_addr(&sh.before[i]), 1);
      mbar_init(smem_addr(&sh.after[i]), 1);
    }
  }
  mbar_fence_init();
  __syncthreads();
  if (ranks > 1) cluster_sync_all();  // every CTA of the cluster is there, its barriers ready
  bool ok = true;
  pdl_wait();
  pdl_trigger();

  auto row0 = [&](int i) { return ((p.groups - 1 - i) * ranks + rank) * kGrChunk + warp * kGbRows; };
  Boxes boxes{smem_addr(&sh.loads[warp][0]), true};
  auto fetch = [&](int i) {
    if (p.tma) {
      if (lane == 0 && i < p.groups && boxes.landed) {
        mbar_arrive_expect_tx(boxes.bar, kArrays * kArray);
        tma_load_2d(ring + 2 * kArray, &p.in[3], c0, row0(i), boxes.bar);
        bulk_wait_read();  // the gradients of the last tile have left these places
        tma_load_2d(ring, &p.in[0], c0, row0(i), boxes.bar);
        tma_load_2d(ring + kArray, &p.in[1], c0, row0(i), boxes.bar);
        if constexpr (GATE) tma_load_2d(ring + 3 * kArray, &p.in[2], c0, row0(i), boxes.bar);
      }
    } else if (i < p.groups) {
      fetch_rows<T, N, kGbRows>(ring, a.x, a.xs, row0(i), T_, c0, a.C, p.words[0], lane);
      fetch_rows<T, N, kGbRows>(ring + kArray, a.f, a.fs, row0(i), T_, c0, a.C, p.words[1], lane);
      fetch_rows<T, N, kGbRows>(ring + 2 * kArray, a.dout, a.dos, row0(i), T_, c0, a.C, p.words[3], lane);
      if constexpr (GATE) fetch_rows<T, N, kGbRows>(ring + 3 * kArray, a.g, a.gs, row0(i), T_, c0, a.C, p.words[2], lane);
      cp_async_commit();
    }
  };
  fetch(0);
  pass_empty(a, a.ds1, a.ds0, rank, ranks, c, in, warp, kGbWarps, lane);
  const int first = a.cu ? clamp_row(__ldg(a.cu), T_) : 0, last = a.cu ? clamp_row(__ldg(a.cu + a.N), T_) : T_;
  Boundaries<kGbRows, true> bounds;
  bounds.begin(first);
  uint64_t state[P];  // the gradient at the state behind the rows not yet visited
#pragma unroll
  for (int e = 0; e < P; ++e) state[e] = 0;

  for (int i = 0; i < p.groups; ++i) {
    const int t0 = row0(i), par = i & 1;
    uint64_t hf[P];  // the state ahead of the tile
    L::load_state(a.chunk + (t0 < T_ ? (long long)(t0 / kGrChunk) * a.C + c : 0), t0 < T_ ? in : 0, hf);
    __syncwarp();  // the last rows' marks have been read
    const Marks m = bounds.rows(a, t0, sh.seqs[warp], lane);
    if (p.tma) {
      boxes.wait(i, p.wait_ns);
      ok = ok && boxes.landed;
    } else {
      cp_async_wait<0>();
      __syncwarp();
    }
    const uint32_t at = ring + lane * L::kBytes;

    // The rows' span for the state (A, B) and for the gradients, R = sum of
    // (a_0 .. a_k) d_k up to the first row that ends a sequence.  Of a row
    // only e^-f is kept, from which a and 1 - a come back exactly.
    uint64_t ef[kGbRows][P], A[P], B[P], R[P];
    uint64_t final[kGbRows][P];  // the gradients at final states (read once: ds0 may lie in their place)
#pragma unroll
    for (int e = 0; e < P; ++e) {
      A[e] = f2_both(1.f);
      B[e] = R[e] = 0;
    }
    auto scan = [&](auto marks) {
#pragma unroll
      for (int k = 0; k < kGbRows; ++k) {
        uint64_t x[P], f[P], d[P], ga[P];
        L::load(at + k * kRow, x);
        L::load_gate(at + kArray + k * kRow, f);
        L::load(at + 2 * kArray + k * kRow, d);
        if constexpr (GATE) {
          uint64_t g[P], u;
          L::load_gate(at + 3 * kArray + k * kRow, g);
#pragma unroll
          for (int e = 0; e < P; ++e) d[e] = f2_mul(d[e], f2_mul(g[e], f2_sigmoid<T>(g[e], &u)));
        }
        if constexpr (marks.value) {
          if (a.ds1 && (m.ends >> k & 1)) {
            uint64_t v[P];
            L::load_state(a.ds1 + (long long)sh.seqs[warp][kGbRows + k] * a.C + c, in, v);
#pragma unroll
            for (int e = 0; e < P; ++e) {
              d[e] = f2_add(d[e], v[e]);
              final[__popc(m.ends & ((1u << k) - 1))][e] = v[e];
            }
          }
          if (m.starts >> k & 1) L::load_state(a.s0 + (a.s0 ? (long long)sh.seqs[warp][k] * a.C + c : 0), a.s0 ? in : 0, B);
        }
#pragma unroll
        for (int e = 0; e < P; ++e) {
          ga[e] = f2_sigmoid<T>(f[e], &ef[k][e]);
          const uint64_t rest = f2_mul(ef[k][e], ga[e]);
          B[e] = f2_fma(ga[e], B[e], f2_mul(rest, x[e]));
          A[e] = f2_mul(A[e], ga[e]);
          if (!marks.value || !(m.ends & ((1u << k) - 1))) R[e] = f2_fma(A[e], d[e], R[e]);
        }
      }
    };
    if ((m.starts | m.ends) == 0) scan(std::false_type{});
    else scan(std::true_type{});
    L::put(sh.A[par][warp][lane], A);
    L::put(sh.B[par][warp][lane], R);
    L::put(fwd_B[par][warp][lane], B);
    if (lane == 0) {
      sh.cut[par][warp] = m.ends != 0;
      fwd_cut[par][warp] = m.starts != 0;
    }
    __syncthreads();
    if (ranks > 1 && ok && warp == 0)
      send_span<L, kGbWarps, kGbRows, true>(sh, spans, par, i % 3, ranks - 1 - rank, ranks, !(p.withhold && i == 0), lane);
    // while the spans are on their way: the states ahead of the rows
    through_warps<L, kGbWarps, false>(sh.A[par], fwd_B[par], *reinterpret_cast<const uint64_t*>(fwd_cut[par]), warp, lane, hf);
    uint64_t hp[kGbRows][P];
    auto states = [&](auto marks) {
#pragma unroll
      for (int k = 0; k < kGbRows; ++k) {
        uint64_t x[P];
        L::load(at + k * kRow, x);
        if constexpr (marks.value) {
          if (m.starts >> k & 1) L::load_state(a.s0 + (a.s0 ? (long long)sh.seqs[warp][k] * a.C + c : 0), a.s0 ? in : 0, hf);
        }
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const uint64_t ga = f2_open(ef[k][e]);
          hp[k][e] = hf[e];
          hf[e] = f2_fma(ga, hf[e], f2_mul(f2_mul(ef[k][e], ga), x[e]));
        }
      }
    };
    if (m.starts == 0) states(std::false_type{});
    else states(std::true_type{});
    uint64_t G[P];
    receive<L, kGbWarps, kGbRows, true>(sh, spans, i, ranks - 1 - rank, ranks, p.wait_ns, ok, warp, lane, A, R, state, G);
    if (!ok) {  // every result NaN
#pragma unroll
      for (int k = 0; k < kGbRows; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e) ef[k][e] = hp[k][e] = f2_both(__int_as_float(0x7fc00000));
    }
    // marks: a sequence begins or ends among the rows.
    // (Which gradients are wanted does not choose the code: their last bits
    // must not depend on it.)
    auto finish = [&](auto marks) {
      constexpr bool kMarks = marks.value;
#pragma unroll
      for (int k = kGbRows - 1; k >= 0; --k) {
        uint64_t x[P], d[P], vx[P], vf[P];
        [[maybe_unused]] uint64_t vg[P];
        L::load(at + k * kRow, x);
        L::load(at + 2 * kArray + k * kRow, d);
        if constexpr (GATE) {
          uint64_t g[P], u;
          L::load_gate(at + 3 * kArray + k * kRow, g);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const uint64_t s = f2_sigmoid<T>(g[e], &u);
            vg[e] = f2_mul(d[e], f2_fma(f2_mul(g[e], s), f2_sub(f2_both(1.f), s), s));  // dy silu'(g)
            d[e] = f2_mul(d[e], f2_mul(g[e], s));
          }
        }
        if constexpr (kMarks) {
          if (a.ds1 && (m.ends >> k & 1)) {
#pragma unroll
            for (int e = 0; e < P; ++e) d[e] = f2_add(d[e], final[__popc(m.ends & ((1u << k) - 1))][e]);
          }
        }
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const uint64_t ga = f2_open(ef[k][e]), rest = f2_mul(ef[k][e], ga);
          G[e] = kMarks && (m.ends >> k & 1) ? d[e] : f2_add(d[e], G[e]);  // dh
          vx[e] = f2_mul(rest, G[e]);
          vf[e] = f2_mul(f2_mul(G[e], f2_sub(hp[k][e], x[e])), f2_mul(ga, rest));
          if constexpr (GATE) vg[e] = f2_mul(vg[e], f2_fma(ga, hp[k][e], f2_mul(rest, x[e])));
          G[e] = f2_mul(ga, G[e]);
        }
        L::stage(at + k * kRow, vx);
        L::stage(at + kArray + k * kRow, vf);
        if constexpr (GATE) L::stage(at + 3 * kArray + k * kRow, vg);
        if constexpr (kMarks) {
          if (a.ds0 && (m.starts >> k & 1)) L::store_state(a.ds0 + (long long)sh.seqs[warp][k] * a.C + c, in, G);
        }
      }
    };
    if ((m.starts | m.ends) == 0) finish(std::false_type{});
    else finish(std::true_type{});
    if (p.tma && t0 >= first && (t0 + kGbRows <= last || last == T_)) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && t0 < T_) {
        if (a.dx) tma_store_2d(&p.out[0], c0, t0, ring);
        if (a.df) tma_store_2d(&p.out[1], c0, t0, ring + kArray);
        if (GATE && a.dg) tma_store_2d(&p.out[2], c0, t0, ring + 3 * kArray);
        bulk_commit();
      }
    } else {
      __syncwarp();
      if (a.dx) put_rows<T, N, kGbRows>(ring, a.dx, a.dxs, t0, first, last, c0, a.C, lane);
      if (a.df) put_rows<T, N, kGbRows>(ring + kArray, a.df, a.dfs, t0, first, last, c0, a.C, lane);
      if (GATE && a.dg) put_rows<T, N, kGbRows>(ring + 3 * kArray, a.dg, a.dgs, t0, first, last, c0, a.C, lane);
      if (p.tma) fence_proxy_async_smem();  // the next boxes land where these gradients were written
    }
    __syncwarp();  // the rows have been read
    fetch(i + 1);
  }
  boxes.settle();
  leave(sh, p.groups, ranks, p.wait_ns, ok, a.dev_err, lane);
}

// V channels of a row for one thread (V = 4: on their boundaries)
template <typename T, int V>
__device__ __forceinline__ void load_channels(const void* at, long long i, float (&v)[V]) {
  const T* p = static_cast<const T*>(at) + i;
  if constexpr (V == 1) {
    v[0] = load_elem(p);
  } else if constexpr (sizeof(T) == 2) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
  } else {
    const float4 w = *reinterpret_cast<const float4*>(p);
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_channels(void* at, long long i, const float (&v)[V]) {
  T* p = static_cast<T*>(at) + i;
  if constexpr (V == 1) store_elem(p, v[0]);
  else if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  else *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// One token per row: a CTA owns V channels to a thread of a row, and goes on
// through the later rows of the same slot.  Every load of the row is on its way
// before the other rows' slots are looked at.  64 rows of 7168 bf16 channels
// with a gate move 7.3 MB, 1.1 us of HBM; in a graph of such calls one takes 2.4
// us, which is its launch and one chain of loads (128 rows in fp32: 5.5 us for
// 22 MB), a call from a program 9.5, most of it the binding's.  (Every CTA reads
// all B slots to find its row's like: nothing for hundreds of rows, 256 turns of
// its loop for 65535.)
template <typename T, int V>
__global__ void __launch_bounds__(kGsThreads) gr_step_kernel(const __grid_constant__ RecurrenceStepArgs p) {
  __shared__ int next_row;
  const int tid = threadIdx.x, c = (blockIdx.x * kGsThreads + tid) * V;
  const bool in = c < p.C;
  int row = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const int slot = p.slots ? __ldg(p.slots + row) : row;
  if (slot < 0 || slot >= p.num_slots) return;  // a padding row
  const long long at = (long long)slot * p.C + c;
  float h[V] = {}, x[V] = {}, f[V] = {}, g[V] = {};
  auto load_row = [&]() {
    if (!in) return;
    load_channels<T, V>(p.x, row * p.xs + c, x);
    load_channels<T, V>(p.f, row * p.fs + c, f);
    if (p.g) load_channels<T, V>(p.g, row * p.gs + c, g);
  };
  if (in) load_channels<float, V>(p.state, at, h);
  load_row();
  bool more = false;
  if (p.slots && p.B > 1) {  // rows of one slot belong to the CTA of the first of them
    bool earlier = false, later = false;
    for (int i = tid; i < p.B; i += kGsThreads)
      if (__ldg(p.slots + i) == slot) {
        earlier |= i < row;
        later |= i > row;
      }
    if (__syncthreads_or(earlier)) return;
    more = __syncthreads_or(later);
  }
  for (;;) {
    if (in) {
      float o[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float rest;
        const float a = sigmoid<T>(f[k], &rest);
        h[k] = fmaf(a, h[k], rest * x[k]);
        o[k] = h[k];
        if (p.g) {
          const float z = -min_nan(-g[k], 83.f);
          o[k] *= z * sigmoid<T>(z, &rest);
        }
      }
      store_channels<T, V>(p.out, row * p.os + c, o);
    }
    if (!more) break;
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
    load_row();
  }
  if (in) store_channels<float, V>(p.state, at, h);
}

// whether a row tensor (null: absent) lies on boundaries of `bytes`
bool rows_on(const void* p, int64_t stride, int es, int bytes) {
  return !p || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * es)) & (uintptr_t)(bytes - 1)) == 0;
}

// a row tensor in boxes of a warp's rows and a CTA's channels
bool make_rows_map(CUtensorMap* map, const void* p, int64_t stride, int64_t T, int C, bool bf16, int width, int rows) {
  const EncodeTiled enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)C, (cuuint64_t)T}, strides[1] = {(cuuint64_t)(stride * (bf16 ? 2 : 4))};
  const cuuint32_t box[2] = {(cuuint32_t)width, (cuuint32_t)rows}, steps[2] = {1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(p), dims, strides, box, steps,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A kernel's launch: its channels to a CTA, its shared memory without the
// cluster's, and how many clusters of each size run at once.
struct GrKernel {
  const void* kern;
  int threads, rows, width, smem, span_bytes;
  SmemOptIn opt;
  std::atomic<int> clusters[SmemOptIn::kMaxDevices][kGrMaxCluster + 1];  // and one (0: not asked yet)
};

cudaLaunchConfig_t gr_config(const GrKernel& k, int64_t slabs, int ranks, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(slabs * ranks));
  cfg.blockDim = dim3(k.threads);
  cfg.dynamicSmemBytes = k.smem + (ranks > 1 ? 3 * ranks * k.span_bytes : 0);
  cfg.stream = stream;
  int n = 0;
  if (ranks > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = ranks;
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
  return cfg;
}

// (clusters of more than 8 CTAs are asked for explicitly)
cudaError_t allow_cluster(const GrKernel& k, int ranks) {
  return ranks > 8 ? cudaFuncSetAttribute(k.kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : cudaSuccess;
}

// clusters of `ranks` CTAs that run at once (clusters do not cross the GPU's
// groups of SMs, so fewer than CTAs / ranks may fit)
cudaError_t clusters_at_once(GrKernel& k, int ranks, int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>* slot = dev >= 0 && dev < SmemOptIn::kMaxDevices ? &k.clusters[dev][ranks] : nullptr;
  if (slot && (*n = slot->load() - 1) >= 0) return cudaSuccess;
  e = allow_cluster(k, ranks);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = gr_config(k, 1, ranks, nullptr, attr);
  if (ranks > 1) {
    e = cudaOccupancyMaxActiveClusters(n, k.kern, &cfg);
  } else {
    DeviceInfo di;
    e = device_info(&di);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, k.kern, k.threads, cfg.dynamicSmemBytes);
    *n *= di.sm_count;
  }
  if (e == cudaSuccess && slot) slot->store(*n + 1);
  return e;
}

template <typename... A>
cudaError_t launch_gr(GrKernel& k, void (*kern)(A...), const RecurrenceArgs& a) {
  cudaError_t e = k.opt.ensure(k.kern, k.smem + 3 * kGrMaxCluster * k.span_bytes);
  if (e != cudaSuccess) return e;
  const int es = a.dtype == ATTNRES_BF16 ? 2 : 4;
  const int64_t tiles = (a.T + kGrChunk - 1) / kGrChunk, slabs = (a.C + k.width - 1) / k.width;
  // CTAs to a slab: the smallest cluster that takes off a tenth of the time
  // (rounds of clusters x tiles of a CTA) against each smaller one.  (5003 x
  // 1000, fp32: 38 us with up to 16 CTAs, 48 with up to 8; 16384 x 7168 takes
  // few and is the same with either limit.)
  GrParams p{};
  double least = 1e300;
  for (int r = 1; r <= kGrMaxCluster && r <= (tiles > 1 ? tiles : 1); ++r) {
    int n = 0;
    e = clusters_at_once(k, r, &n);
    if (e != cudaSuccess) return e;
    if (n < 1 && r > 1) continue;  // not to be had here
    if (n < 1) n = 1;
    const double cost = (double)((slabs + n - 1) / n) * (double)((tiles + r - 1) / r);
    if (r == 1 || cost < 0.9 * least) {
      least = cost;
      p.ranks = r;
    }
  }
  p.a = a;
  p.wait_ns = wait_limit_ns();
  p.withhold = debug_withhold_row1() > 0;
  p.groups = (int)((tiles + p.ranks - 1) / p.ranks);
  const bool backward = a.dout != nullptr;
  const void* in[4] = {a.x, a.f, a.g, a.dout};
  const int64_t in_strides[4] = {a.xs, a.fs, a.gs, a.dos};
  void* const out[3] = {backward ? a.dx : a.out, a.df, a.dg};
  const int64_t out_strides[3] = {backward ? a.dxs : a.os, a.dfs, a.dgs};
  p.tma = a.T > 0 && (int64_t)a.C * es % 16 == 0;  // (a box is cut off at 16 bytes, not at an element)
  for (int i = 0; i < 4; ++i) {
    p.tma = p.tma && rows_on(in[i], in_strides[i], es, 16);
    p.words[i] = rows_on(in[i], in_strides[i], es, 4);
  }
  for (int i = 0; i < 3; ++i) p.tma = p.tma && rows_on(out[i], out_strides[i], es, 16);
  for (int i = 0; i < 4 && p.tma; ++i)
    if (in[i]) p.tma = make_rows_map(&p.in[i], in[i], in_strides[i], a.T, a.C, es == 2, k.width, k.rows);
  for (int i = 0; i < 3 && p.tma; ++i)
    if (out[i]) p.tma = make_rows_map(&p.out[i], out[i], out_strides[i], a.T, a.C, es == 2, k.width, k.rows);
  e = allow_cluster(k, p.ranks);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = gr_config(k, slabs, p.ranks, a.stream, attr);
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T, bool GATE>
cudaError_t launch_forward(const RecurrenceArgs& a) {
  using L = Lane<T, 2>;
  static GrKernel k{reinterpret_cast<const void*>(gr_forward_kernel<T, GATE>), 32 * kGfWarps, kGfRows, 32 * 2 * L::P,
                    kBoxAlign + kGrChunk * 32 * L::kBytes * (GATE ? 4 : 3), (int)sizeof(RankSpan<L::P>), {}, {}};
  return launch_gr(k, gr_forward_kernel<T, GATE>, a);
}
template <typename T, bool GATE>
cudaError_t launch_backward(const RecurrenceArgs& a) {
  using L = Lane<T, 2>;
  static GrKernel k{reinterpret_cast<const void*>(gr_backward_kernel<T, GATE>), 32 * kGbWarps, kGbRows, 32 * 2 * L::P,
                    kBoxAlign + kGrChunk * 32 * L::kBytes * (GATE ? 4 : 3), (int)sizeof(RankSpan<L::P>), {}, {}};
  return launch_gr(k, gr_backward_kernel<T, GATE>, a);
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
  // four channels to a thread where all rows lie on those boundaries (64 x
  // 7168 bf16: 2.4 us, one to a thread 3.7; 128 x 7168 fp32: 5.5 and 7.9)
  const int es = a.dtype == ATTNRES_BF16 ? 2 : 4;
  const bool four = a.C % 4 == 0 && rows_on(a.state, 4, 4, 16) && rows_on(a.x, a.xs, es, 4 * es) && rows_on(a.f, a.fs, es, 4 * es) &&
                    rows_on(a.g, a.gs, es, 4 * es) && rows_on(a.out, a.os, es, 4 * es);
  const int channels = kGsThreads * (four ? 4 : 1);
  const dim3 grid((a.C + channels - 1) / channels, a.B), block(kGsThreads);
  if (es == 2)
    return four ? launch_kernel(gr_step_kernel<bf16_t, 4>, grid, block, 0, a.stream, a)
                : launch_kernel(gr_step_kernel<bf16_t, 1>, grid, block, 0, a.stream, a);
  return four ? launch_kernel(gr_step_kernel<float, 4>, grid, block, 0, a.stream, a)
              : launch_kernel(gr_step_kernel<float, 1>, grid, block, 0, a.stream, a);
}

}  // namespace attnres
