// Layer norm of whole rows, and its backward.
//
//   h = (x - m) / sqrt(mean_c (x_c - m)^2 + eps),  y = gain * h + bias.
//   backward: n = gain * dy,  dx = (n - mean(n) - h mean(n h)) / sigma,
//   dgain = sum_t dy h,  dbias = sum_t dy.
//
// The mean is held as the sum of two fp32 numbers: m, the rounded mean, and
// delta, the mean of the differences x - m (exact where m is near x), so rows
// whose mean is far from zero keep their digits.
//
// The floor is HBM's: x once in and once out, backward x and dy in, dx out.
// A row therefore stays on the SM between its passes (mean, squares, result):
// forward in registers, backward in shared memory, since there the registers
// hold a lane's sums of the gain and bias gradients.  Rows wider than that are
// read once per pass by ln_any_kernel; what this saves, 16384 x 7168 bf16: 228
// us there, 81 here (5.8 TB/s, the copy runs at 6.8); backward of 8192 x 7168:
// 426 and 76 us (4.7 TB/s; 69 without the gain and bias gradients, whose
// partial rows a second launch adds).  What bounds them now is latency at the
// warps that the registers leave: forward 16 to an SM, 48 % of the issue slots
// and 64 % of DRAM's cycles, backward 14, 50 % and 55 %.  They wait for their own
// chains, for one another at the barriers of the rows' sums (forward two a row,
// backward one for two rows) and for arithmetic that comes in bursts: every pass
// unpacks x, and backward dy, again.  64 rows take the launch and one row's chain
// of load, sums and store: 6.5 us between the calls of a program.
#include <math.h>

#include "attnres.h"
#include "body.h"
#include "device_common.cuh"
#include "launch.h"
#include "vec16.cuh"

namespace attnres {

namespace {

constexpr int kLnThreads = 256;
constexpr int kLnBlocksPerSm = 4;   // ln_any_kernel
constexpr int kLnMaxWarps = 16;     // of a row in registers

struct LnParams {
  const void* x;
  const void* dy;
  void* out;
  long long xs, dys, os;
  const float *gain, *bias;
  long long T;
  int d;
  float eps, inv_d;
  float* part;  // backward: [grid][2][d] partial gain and bias gradients, or null
  int warps;    // rows in registers: warps of a row
};

// sums of N values over the CTA, the same in every thread
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*red)[N]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  __syncthreads();  // the last sums have been read
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[warp][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < (int)blockDim.x >> 5; ++w) v[i] += red[w][i];
  }
}

// Any width, alignment and stride: one CTA per row, read three times.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kLnThreads) ln_any_kernel(const __grid_constant__ LnParams p) {
  __shared__ float red2[32][2], red3[32][3];
  pdl_wait();
  pdl_trigger();
  float* dg = BWD && p.part ? p.part + (long long)blockIdx.x * 2 * p.d : nullptr;
  float* db = dg ? dg + p.d : nullptr;
  for (int c = threadIdx.x; dg && c < p.d; c += kLnThreads) dg[c] = db[c] = 0.f;
  auto gain = [&](int c) { return p.gain ? __ldg(p.gain + c) : 1.f; };
  for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + t * p.xs;
    const T* dy = BWD ? static_cast<const T*>(p.dy) + t * p.dys : nullptr;
    T* o = static_cast<T*>(p.out) + (p.out ? t * p.os : 0);
    float s1[2] = {0.f, 0.f};  // sum x, sum n
    for (int c = threadIdx.x; c < p.d; c += kLnThreads) {
      s1[0] += load_elem(x + c);
      if (BWD) s1[1] = fmaf(load_elem(dy + c), gain(c), s1[1]);
    }
    block_sums(s1, red2);
    const float m = s1[0] * p.inv_d;
    float s2[3] = {0.f, 0.f, 0.f};  // sum x - m, its squares, sum n (x - m)
    for (int c = threadIdx.x; c < p.d; c += kLnThreads) {
      const float z = load_elem(x + c) - m;
      s2[0] += z;
      s2[1] = fmaf(z, z, s2[1]);
      if (BWD) s2[2] = fmaf(load_elem(dy + c) * gain(c), z, s2[2]);
    }
    block_sums(s2, red3);
    const float delta = s2[0] * p.inv_d;
    const float rstd = rsqrtf(fmaxf(fmaf(-delta, delta, s2[1] * p.inv_d), 0.f) + p.eps);
    if (!BWD) {
      for (int c = threadIdx.x; c < p.d; c += kLnThreads) {
        const float h = ((load_elem(x + c) - m) - delta) * rstd;
        store_elem(o + c, fmaf(h, gain(c), p.bias ? __ldg(p.bias + c) : 0.f));
      }
    } else {
      const float mn = s1[1] * p.inv_d;
      const float mh = (s2[2] * p.inv_d - delta * mn) * rstd;  // mean(n h)
      for (int c = threadIdx.x; c < p.d; c += kLnThreads) {
        const float h = ((load_elem(x + c) - m) - delta) * rstd, g = load_elem(dy + c);
        if (p.out) store_elem(o + c, (fmaf(-h, mh, g * gain(c)) - mn) * rstd);
        if (dg) {
          dg[c] = fmaf(g, h, dg[c]);
          db[c] += g;
        }
      }
    }
  }
}

// ------------------------------------------------------- rows in registers --

__device__ __forceinline__ void st_shared_zero(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

// What a lane holds of a row: up to VPL vectors' worth of channels, as they lie
// in memory (16 bits a channel for bf16).  A row's warps own segments of it,
// `held` vectors to a lane: vector i of a lane is vector lane + 32 i of the
// segment (VEC), or its channel k of vector i is channel lane + 32 (i V + k).
// Everything is at a fixed distance from the segment's first address.
template <typename T, bool VEC>
struct Segment {
  static constexpr int V = Vec16<T>::kElems, P = V / 2;  // channels and packed pairs of a vector
  int at;    // the lane's first channel
  int left;  // channels of the segment from there on
  int held;

  __device__ __forceinline__ Segment(int warp, int warps, int lane, int d) {
    held = (d + 32 * V * warps - 1) / (32 * V * warps);
    at = warp * held * 32 * V + lane * (VEC ? V : 1);
    const int end = (warp + 1) * held * 32 * V;
    left = (end < d ? end : d) - at;
  }
  static __device__ __forceinline__ constexpr int offset(int i, int k) { return VEC ? i * 32 * V + k : (i * V + k) * 32; }
  __device__ __forceinline__ bool has(int i, int k = 0) const { return offset(i, VEC ? 0 : k) < left; }
  __device__ __forceinline__ uint4 load(const T* x, int i) const {
    uint4 v = make_uint4(0, 0, 0, 0);
    if constexpr (VEC) {
      if (has(i)) v = __ldcs(reinterpret_cast<const uint4*>(x + offset(i, 0)));
    } else {
      float f[V];
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] = has(i, k) ? load_elem(x + offset(i, k)) : 0.f;
      v = Vec16<T>::pack(f);  // (exact: the values are of this type)
    }
    return v;
  }
  static __device__ __forceinline__ void unpack(const uint4& v, uint64_t (&f)[P]) {
    float t[V];
    Vec16<T>::unpack(v, t);
#pragma unroll
    for (int k = 0; k < P; ++k) f[k] = f2_pack(t[2 * k], t[2 * k + 1]);
  }
  template <bool MASK>
  __device__ __forceinline__ void store(T* y, int i, const uint64_t (&f)[P]) const {
    float t[V];
#pragma unroll
    for (int k = 0; k < P; ++k) f2_unpack(f[k], t[2 * k], t[2 * k + 1]);
    if constexpr (VEC) {
      if (!MASK || has(i)) __stcs(reinterpret_cast<uint4*>(y + offset(i, 0)), Vec16<T>::pack(t));
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (!MASK || has(i, k)) store_elem(y + offset(i, k), t[k]);
    }
  }
  // A vector of fp32 in shared memory, as the lanes read it without conflicts:
  // the first four channels of every vector, then the other four (V = 8).
  static __device__ __forceinline__ int place(int c, int d) { return VEC && V == 8 ? (c >> 2 & 1) * (d >> 1) + (c >> 3) * 4 + (c & 3) : c; }
  // the lane's channels of it; `first`: at place(at).  (VEC: only where the lane
  // has channels, something else lies behind them.)
  __device__ __forceinline__ void load_f32(const float* first, int i, int d, uint64_t (&f)[P]) const {
    if constexpr (VEC) {
#pragma unroll
      for (int h = 0; h < P / 2; ++h) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(first + i * 128 + (h ? d >> 1 : 0));
        f[2 * h] = w.x;
        f[2 * h + 1] = w.y;
      }
    } else {
#pragma unroll
      for (int k = 0; k < P; ++k) f[k] = f2_pack(has(i, 2 * k) ? first[offset(i, 2 * k)] : 0.f, has(i, 2 * k + 1) ? first[offset(i, 2 * k + 1)] : 0.f);
    }
  }
  // x - m where there is a channel, else 0 (MASK: some lanes have none here)
  template <bool MASK>
  __device__ __forceinline__ void center(const uint4& v, uint64_t minus_m, int i, uint64_t (&z)[P]) const {
    unpack(v, z);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      z[k] = f2_add(z[k], minus_m);
      if constexpr (MASK) {
        float t[2];
        f2_unpack(z[k], t[0], t[1]);
        z[k] = f2_pack(has(i, 2 * k) ? t[0] : 0.f, has(i, 2 * k + 1) ? t[1] : 0.f);
      }
    }
  }
};

// Sums of N values (up to W) over a row's warps, the same in every thread of
// the row, in a fixed order.  Several values are summed over a warp by halves:
// after the first exchanges each lane carries one of them.  One barrier: the
// caller alternates between two buffers.
template <int N, int W>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[W], int warps, int group, int warp, int lane) {
  constexpr uint32_t kAll = 0xffffffffu;
  constexpr int kValues = N == 1 ? 1 : N == 2 ? 2 : N <= 4 ? 4 : N <= 8 ? 8 : 16, kLanes = 32 / kValues;  // lanes that end up with the same value
  float a[kValues];
#pragma unroll
  for (int i = 0; i < kValues; ++i) a[i] = i < N ? v[i < N ? i : 0] : 0.f;
#pragma unroll
  for (int n = kValues / 2, o = 16; n > 0; n /= 2, o /= 2) {
    const bool hi = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) a[i] = (hi ? a[i + n] : a[i]) + __shfl_xor_sync(kAll, hi ? a[i] : a[i + n], o);
  }
  float s = a[0];
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  if (warps > 1) {
    const int which = lane / kLanes, w = lane % kLanes;
    if (w == 0) red[warp][which] = s;
    named_barrier_sync(1 + group, 32 * warps);
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kLnMaxWarps; i += kLanes)
      if (w + i < warps) s += red[w + i][which];
#pragma unroll
    for (int o = (kLanes < kLnMaxWarps ? kLanes : kLnMaxWarps) / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(kAll, s, i * kLanes);
}

// a vector of fp32 into shared memory by the whole CTA (null: `none`); VEC: on
// its way, in the caller's next group of copies
template <typename S, bool VEC>
__device__ __forceinline__ void stage(float* to, const float* v, float none, int d) {
  if (VEC && v) {
    for (int c = 4 * threadIdx.x; c < d; c += 4 * blockDim.x) cp_async16(smem_addr(to + S::place(c, d)), v + c);
  } else {
    for (int c = threadIdx.x; c < d; c += blockDim.x) to[S::place(c, d)] = v ? __ldg(v + c) : none;
  }
}

// Rows that fit registers, read once and then taken from there three times.  A
// CTA's warps form groups, each with a row at a time; gain and bias lie in
// shared memory.  VEC: the next rows are on their way by cp.async, in shared
// memory that each thread keeps to itself.
template <typename T, int VPL, bool VEC>
__global__ void __launch_bounds__(32 * kLnMaxWarps, VPL > 8 ? 1 : 2) ln_row_kernel(const __grid_constant__ LnParams p) {
  using S = Segment<T, VEC>;
  constexpr int P = S::P;
  extern __shared__ __align__(16) unsigned char dyn[];  // gain, bias; VEC: [held][threads] vectors
  __shared__ __align__(16) float red[2][kLnMaxWarps][8];
  const int warps = p.warps, lane = threadIdx.x & 31, nthreads = (int)blockDim.x;
  const int group = (threadIdx.x >> 5) / warps, groups = (nthreads >> 5) / warps, warp = (threadIdx.x >> 5) % warps;
  const S seg(warp, warps, lane, p.d);
  float* gains = reinterpret_cast<float*>(dyn);
  float* biases = gains + (p.d + 3 & ~3);
  pdl_wait();
  pdl_trigger();
  const T* X = static_cast<const T*>(p.x) + seg.at;
  const long long step = (long long)gridDim.x * groups;
  long long t = (long long)blockIdx.x * groups + group;
  const uint32_t vec = nthreads * 16, ring = smem_addr(biases + (p.d + 3 & ~3)) + threadIdx.x * 16;
  auto fetch = [&](long long t) {
    if (t < p.T) {
      const T* row = X + t * p.xs;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i < seg.held) cp_async16(ring + i * vec, seg.has(i) ? row + S::offset(i, 0) : static_cast<const T*>(p.x), seg.has(i));
    }
    cp_async_commit();
  };
  stage<S, VEC>(gains, p.gain, 1.f, p.d);
  stage<S, VEC>(biases, p.bias, 0.f, p.d);
  if constexpr (VEC) {
    fetch(t);
    cp_async_wait<0>();
  }
  __syncthreads();
  gains += S::place(seg.at, p.d);
  biases += S::place(seg.at, p.d);
  for (; t < p.T; t += step) {
    uint4 x[VPL];
    if constexpr (VEC) {
      cp_async_wait<0>();
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i < seg.held) x[i] = ld_shared_v4(ring + i * vec);
      fetch(t + step);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i < seg.held) x[i] = seg.load(X + t * p.xs, i);
    }
    uint64_t s = 0, f[P];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < seg.held) {
        S::unpack(x[i], f);
#pragma unroll
        for (int k = 0; k < P; ++k) s = f2_add(s, f[k]);
      }
    float s1[1] = {f2_hsum(s)};
    row_sums<1>(s1, red[0] + group * warps, warps, group, warp, lane);
    const float m = s1[0] * p.inv_d;
    uint64_t sz = 0, sq = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < seg.held && (!VEC || seg.has(i))) {
        seg.template center<!VEC>(x[i], f2_both(-m), i, f);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          sz = f2_add(sz, f[k]);
          sq = f2_fma(f[k], f[k], sq);
        }
      }
    float s2[2] = {f2_hsum(sz), f2_hsum(sq)};
    row_sums<2>(s2, red[1] + group * warps, warps, group, warp, lane);
    const float delta = s2[0] * p.inv_d;
    const float rstd = rsqrtf(fmaxf(fmaf(-delta, delta, s2[1] * p.inv_d), 0.f) + p.eps);
    const uint64_t minus_m = f2_both(-m), r2 = f2_both(rstd), shift = f2_both(-delta * rstd);
    T* out = static_cast<T*>(p.out) + t * p.os + seg.at;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < seg.held && (!VEC || seg.has(i))) {
        uint64_t gain[P], bias[P];
        seg.load_f32(gains, i, p.d, gain);
        seg.load_f32(biases, i, p.d, bias);
        S::unpack(x[i], f);
#pragma unroll
        for (int k = 0; k < P; ++k) f[k] = f2_fma(f2_fma(f2_add(f[k], minus_m), r2, shift), gain[k], bias[k]);
        seg.template store<!VEC>(out, i, f);
      }
  }
}

// Its backward: a lane also keeps its channels' sums of dy h and dy over its
// group's rows, which are taken ROWS at a time (their sums cross the warps
// together).
constexpr int kLnTakes = 3;  // of the ring: one at work, the next, and one on its way
template <typename T, int VPL, int ROWS, bool VEC>
__global__ void __launch_bounds__(32 * kLnMaxWarps) ln_row_backward_kernel(const __grid_constant__ LnParams p) {
  using S = Segment<T, VEC>;
  constexpr int P = S::P;
  constexpr uint32_t kRow = 2 * VPL * 512, kTake = ROWS * kRow;  // of a warp's ring
  extern __shared__ __align__(16) unsigned char dyn[];  // gain; VEC: [warp][kLnTakes][ROWS][x, dy][VPL][lane] vectors; at the end: sums
  __shared__ __align__(16) float red[2][kLnMaxWarps][16];
  const int warps = p.warps, lane = threadIdx.x & 31, nthreads = (int)blockDim.x;
  const int group = (threadIdx.x >> 5) / warps, groups = (nthreads >> 5) / warps, warp = (threadIdx.x >> 5) % warps;
  const S seg(warp, warps, lane, p.d);
  float* gains = reinterpret_cast<float*>(dyn);
  pdl_wait();
  pdl_trigger();
  const long long step = (long long)gridDim.x * groups;
  long long t = (long long)blockIdx.x * groups + group, ahead_t = t;
  // the next rows to load and to write
  const T* xr = static_cast<const T*>(p.x) + t * p.xs + seg.at;
  const T* dr = static_cast<const T*>(p.dy) + t * p.dys + seg.at;
  T* out = static_cast<T*>(p.out) + (p.out ? t * p.os + seg.at : 0);
  const long long x_step = step * p.xs, d_step = step * p.dys, out_step = p.out ? step * p.os : 0;
  const uint32_t ring = smem_addr(gains + (p.d + 3 & ~3)) + (threadIdx.x >> 5) * (kLnTakes * kTake) + lane * 16;
  uint32_t ahead_slot = 0, slot = 0;
  if constexpr (VEC) {  // what no copy fills stays zero
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!seg.has(i))
        for (int r = 0; r < kLnTakes * ROWS; ++r) {
          st_shared_zero(ring + r * kRow + i * 512);
          st_shared_zero(ring + r * kRow + (VPL + i) * 512);
        }
  }
  auto fetch = [&] {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (ahead_t < p.T) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (seg.has(i)) {
            cp_async16(ring + ahead_slot + r * kRow + i * 512, xr + S::offset(i, 0));
            cp_async16(ring + ahead_slot + r * kRow + (VPL + i) * 512, dr + S::offset(i, 0));
          }
      }
      ahead_t += step;
      xr += x_step;
      dr += d_step;
    }
    ahead_slot = ahead_slot + kTake == kLnTakes * kTake ? 0 : ahead_slot + kTake;
    cp_async_commit();
  };
  stage<S, VEC>(gains, p.gain, 1.f, p.d);
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < kLnTakes - 1; ++i) fetch();
    cp_async_wait<kLnTakes - 2>();  // gain and the first rows
  }
  __syncthreads();
  gains += S::place(seg.at, p.d);
  uint64_t dg[VPL][P], db[VPL][P];
#pragma unroll
  for (int i = 0; i < VPL; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) dg[i][k] = db[i][k] = 0;
  // sums of a take's x, behind its other sums
  auto add_x = [&](auto x, float (&s)[5 * ROWS]) {
    uint64_t f[P], sx[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) sx[r] = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        S::unpack(x(r, i), f);
#pragma unroll
        for (int k = 0; k < P; ++k) sx[r] = f2_add(sx[r], f[k]);
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) s[4 * ROWS + r] = f2_hsum(sx[r]);
  };
  float m[ROWS];  // the take's means
  [[maybe_unused]] int turn = 0;
  if constexpr (VEC) {
    float s[5 * ROWS], s1[ROWS];
    add_x([&](int r, int i) { return ld_shared_v4(ring + r * kRow + i * 512); }, s);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) s1[r] = s[4 * ROWS + r];
    row_sums<ROWS>(s1, red[1] + group * warps, warps, group, warp, lane);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) m[r] = s1[r] * p.inv_d;
  }
  for (; t < p.T; t += ROWS * step) {
    // rows are read from the ring again for every pass (their registers are the sums'); single channels stay in registers
    uint4 held_x[VEC ? 1 : ROWS][VEC ? 1 : VPL] = {}, held_dy[VEC ? 1 : ROWS][VEC ? 1 : VPL] = {};
    auto x = [&](int r, int i) {
      if constexpr (VEC) return ld_shared_v4(ring + slot + r * kRow + i * 512);
      else return held_x[r][i];
    };
    auto dy = [&](int r, int i) {
      if constexpr (VEC) return ld_shared_v4(ring + slot + r * kRow + (VPL + i) * 512);
      else return held_dy[r][i];
    };
    if constexpr (VEC) {
      fetch();  // into the slot of the last take
    } else {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const bool row = ROWS == 1 || t + r * step < p.T;
          held_x[r][i] = row ? seg.load(xr, i) : make_uint4(0, 0, 0, 0);
          held_dy[r][i] = row ? seg.load(dr, i) : make_uint4(0, 0, 0, 0);
        }
        xr += x_step;
        dr += d_step;
      }
    }
    uint64_t f[P], g[P], gain[P];
    float s[5 * ROWS];  // of the take (behind the last row it goes through the motions with what its slot held), and sums of the next one's x
    if constexpr (!VEC) {
      add_x(x, s);
      float s1[ROWS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) s1[r] = s[4 * ROWS + r];
      row_sums<ROWS>(s1, red[1] + group * warps, warps, group, warp, lane);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) m[r] = s1[r] * p.inv_d;
    }
    {
      uint64_t sz[ROWS], sq[ROWS], sn[ROWS], sw[ROWS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) sz[r] = sq[r] = sn[r] = sw[r] = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (VPL > 1 && i >= seg.held) break;
        // (where a lane has no channel there is no gain either: behind the gains
        // lies another row's x, whose infinities a product with zero would keep)
        if (VEC && !seg.has(i)) break;
        seg.load_f32(gains, i, p.d, gain);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          seg.template center<!VEC>(x(r, i), f2_both(-m[r]), i, f);
          S::unpack(dy(r, i), g);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            const uint64_t n = f2_mul(g[k], gain[k]);
            sz[r] = f2_add(sz[r], f[k]);
            sq[r] = f2_fma(f[k], f[k], sq[r]);
            sn[r] = f2_add(sn[r], n);
            sw[r] = f2_fma(n, f[k], sw[r]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        s[4 * r] = f2_hsum(sz[r]);
        s[4 * r + 1] = f2_hsum(sq[r]);
        s[4 * r + 2] = f2_hsum(sw[r]);
        s[4 * r + 3] = f2_hsum(sn[r]);
      }
    }
    if constexpr (VEC) {  // the next take's means come by the same barrier (by one of their own: 79 us where 76)
      cp_async_wait<kLnTakes - 2>();
      const uint32_t next = slot + kTake == kLnTakes * kTake ? 0 : slot + kTake;
      add_x([&](int r, int i) { return ld_shared_v4(ring + next + r * kRow + i * 512); }, s);
      row_sums<5 * ROWS>(s, red[turn] + group * warps, warps, group, warp, lane);
      turn ^= 1;
    } else {
      float s2[4 * ROWS];
#pragma unroll
      for (int k = 0; k < 4 * ROWS; ++k) s2[k] = s[k];
      row_sums<4 * ROWS>(s2, red[0] + group * warps, warps, group, warp, lane);
#pragma unroll
      for (int k = 0; k < 4 * ROWS; ++k) s[k] = s2[k];
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (r > 0 && t + r * step >= p.T) break;
      const float delta = s[4 * r] * p.inv_d;
      const float rstd = rsqrtf(fmaxf(fmaf(-delta, delta, s[4 * r + 1] * p.inv_d), 0.f) + p.eps);
      const float mn = s[4 * r + 3] * p.inv_d;
      const float mh = (s[4 * r + 2] * p.inv_d - delta * mn) * rstd;  // mean(n h)
      // h = (x - m) r - delta r,  dx = (n r - mn r) - h mh r
      const uint64_t minus_m = f2_both(-m[r]), r2 = f2_both(rstd), shift = f2_both(-delta * rstd), n0 = f2_both(-mn * rstd), h0 = f2_both(-mh * rstd);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (VPL > 1 && i >= seg.held) break;
        if (VEC && !seg.has(i)) break;
        seg.load_f32(gains, i, p.d, gain);
        S::unpack(x(r, i), f);
        S::unpack(dy(r, i), g);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const uint64_t h = f2_fma(f2_add(f[k], minus_m), r2, shift);
          dg[i][k] = f2_fma(g[k], h, dg[i][k]);
          db[i][k] = f2_add(db[i][k], g[k]);
          f[k] = f2_fma(h, h0, f2_fma(f2_mul(g[k], gain[k]), r2, n0));
        }
        if (p.out) seg.template store<!VEC>(out, i, f);
      }
      out += out_step;
    }
    if constexpr (VEC) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) m[r] = s[4 * ROWS + r] * p.inv_d;
    }
    slot = slot + kTake == kLnTakes * kTake ? 0 : slot + kTake;
  }
  if (!p.part) return;
  float* part = p.part + (long long)blockIdx.x * 2 * p.d;
  float* sums = reinterpret_cast<float*>(dyn);  // [groups][2][d]
  if constexpr (VEC) cp_async_wait<0>();
  __syncthreads();  // gain and ring are done with
  float* own = groups > 1 ? sums + group * 2 * p.d : part;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    float a[S::V], b[S::V];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      f2_unpack(dg[i][k], a[2 * k], a[2 * k + 1]);
      f2_unpack(db[i][k], b[2 * k], b[2 * k + 1]);
    }
    if constexpr (VEC) {  // (a row of sums is whole vectors too)
      if (seg.has(i)) {
        float* at = own + seg.at + S::offset(i, 0);
#pragma unroll
        for (int k = 0; k < S::V; k += 4) {
          *reinterpret_cast<float4*>(at + k) = make_float4(a[k], a[k + 1], a[k + 2], a[k + 3]);
          *reinterpret_cast<float4*>(at + p.d + k) = make_float4(b[k], b[k + 1], b[k + 2], b[k + 3]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < S::V; ++k)
        if (seg.has(i, k)) {
          own[seg.at + S::offset(i, k)] = a[k];
          own[p.d + seg.at + S::offset(i, k)] = b[k];
        }
    }
  }
  if (groups > 1) {  // in order: the sums do not depend on timing
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.d; c += nthreads) {
      float s = 0.f;
      for (int g = 0; g < groups; ++g) s += sums[g * 2 * p.d + c];
      part[c] = s;
    }
  }
}

// gain and bias gradients: the CTAs' partial rows, summed in order (32
// channels x 16 interleaved runs of rows per CTA, whose loads do not wait for
// one another; blockIdx.y: gain or bias)
constexpr int kLnRuns = 16;
__global__ void __launch_bounds__(32 * kLnRuns) ln_dgain_kernel(const float* part, int blocks, int d, float* dgain, float* dbias) {
  __shared__ float sums[kLnRuns][33];
  const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, r = threadIdx.x >> 5;
  float* out = blockIdx.y ? dbias : dgain;
  pdl_wait();
  pdl_trigger();
  if (!out) return;
  float s = 0.f;
  if (c < d) {
    const float* at = part + blockIdx.y * (long long)d + c;
#pragma unroll 10
    for (int b = r; b < blocks; b += kLnRuns) s += at[b * 2LL * d];
  }
  sums[r][lane] = s;
  __syncthreads();
  if (r == 0 && c < d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kLnRuns; ++i) s += sums[i][lane];
    out[c] = s;
  }
}

// How a call's rows are held: vectors to a lane, warps to a row, rows of a CTA
// at a time, dynamic shared memory, CTAs to an SM (vpl 0: a row does not fit,
// ln_any_kernel).  The partial rows of the gain gradients follow the grid that
// this gives: layer_norm_backward_workspace_bytes asks for the most of any plan.
struct LnPlan {
  int vpl, warps, groups, smem, per_sm;
};
int ln_fixed_smem(bool backward) { return backward ? 2048 : 1024; }  // the sums' buffers
LnPlan ln_plan(int64_t T, int d, int es, bool vec, bool backward, const DeviceInfo& di) {
  constexpr int kForwardVec[3] = {2, 8, 16}, kForward[3] = {1, 2, 4}, kBackward[3] = {1, 2, 4};
  const int V = 16 / es, n = 3;
  const int* vpl = backward ? kBackward : vec ? kForwardVec : kForward;
  // few rows (one to an SM): each over as many warps as it feeds, a lane's
  // channels few; many: a row in as few warps as hold it, so that its sums cross
  // few of them.  Forward of 7168 bf16, with caches cold and the launch: 64 rows
  // 10.9 us over many warps, 13.0 over few; 304 rows 17.0 and 15.0; 16384 rows
  // 111 and 87; 2047 rows of 1003 fp32 19.1 and 12.9.
  const bool few = T <= di.sm_count;
  for (int i = 0; i < n; ++i) {
    const int per_warp = 32 * vpl[i] * V, warps = (d + per_warp - 1) / per_warp;
    // (backward, two vectors to a lane may take several warps: they take two rows
    // at a time, 97 us where single rows over fewer warps took 108)
    if (warps > kLnMaxWarps || (!few && i + 1 < n && warps > 1 && !(backward && vpl[i] == 2))) continue;
    const int held = (d + 32 * V * warps - 1) / (32 * V * warps);
    for (int groups = few ? 1 : kLnMaxWarps / warps; groups >= 1; --groups) {
      const int64_t vectors = (int64_t)((d + 3) / 4) * 16 * (backward ? 1 : 2);
      const int64_t vectors_of_warp = backward ? (vpl[i] == 2 ? 2 : 1) * 2 * vpl[i] * kLnTakes : held;
      const int64_t ring = vec ? warps * groups * vectors_of_warp * 512 : 0;
      const int64_t sums = backward && groups > 1 ? (int64_t)groups * 2 * d * 4 : 0;
      const int64_t smem = vectors + ring > sums ? vectors + ring : sums;
      if (smem + ln_fixed_smem(backward) > di.max_smem_optin) continue;
      // the variants with most registers to a thread run as one CTA to an SM
      const bool one = vpl[i] >= (backward ? 2 : 16) || 2 * (smem + 512 + ln_fixed_smem(backward)) > di.max_smem_optin + 1024;
      return {vpl[i], warps, groups, (int)smem, one ? 1 : 2};
    }
  }
  return {0, 0, 0, 0, 0};
}

template <typename T, int VPL, bool VEC>
cudaError_t launch_forward(const LayerNormArgs& a, const LnParams& p, const LnPlan& k, int grid, int most) {
  static SmemOptIn opt;
  const cudaError_t e = opt.ensure(reinterpret_cast<const void*>(ln_row_kernel<T, VPL, VEC>), most);
  if (e != cudaSuccess) return e;
  return launch_kernel(ln_row_kernel<T, VPL, VEC>, dim3(grid), dim3(32 * k.warps * k.groups), k.smem, a.stream, p);
}
template <typename T, int VPL, bool VEC>
cudaError_t launch_backward(const LayerNormArgs& a, const LnParams& p, const LnPlan& k, int grid, int most) {
  static SmemOptIn opt;
  const cudaError_t e = opt.ensure(reinterpret_cast<const void*>(ln_row_backward_kernel<T, VPL, VPL == 2 ? 2 : 1, VEC>), most);
  if (e != cudaSuccess) return e;
  return launch_kernel(ln_row_backward_kernel<T, VPL, VPL == 2 ? 2 : 1, VEC>, dim3(grid), dim3(32 * k.warps * k.groups), k.smem, a.stream, p);
}

template <typename T>
cudaError_t launch_rows(const LayerNormArgs& a, const LnParams& p, const LnPlan& k, bool vec, int grid, int most) {
  if (a.backward) {
    if (vec)
      return k.vpl == 1   ? launch_backward<T, 1, true>(a, p, k, grid, most)
             : k.vpl == 2 ? launch_backward<T, 2, true>(a, p, k, grid, most)
                          : launch_backward<T, 4, true>(a, p, k, grid, most);
    return k.vpl == 1   ? launch_backward<T, 1, false>(a, p, k, grid, most)
           : k.vpl == 2 ? launch_backward<T, 2, false>(a, p, k, grid, most)
                        : launch_backward<T, 4, false>(a, p, k, grid, most);
  }
  switch (k.vpl) {
    case 1: return launch_forward<T, 1, false>(a, p, k, grid, most);
    case 2: return vec ? launch_forward<T, 2, true>(a, p, k, grid, most) : launch_forward<T, 2, false>(a, p, k, grid, most);
    case 4: return launch_forward<T, 4, false>(a, p, k, grid, most);
    case 8: return launch_forward<T, 8, true>(a, p, k, grid, most);
    default: return launch_forward<T, 16, true>(a, p, k, grid, most);
  }
}

bool vec_rows(const void* ptr, int64_t stride, int V) { return (reinterpret_cast<uintptr_t>(ptr) & 15) == 0 && stride % V == 0; }

}  // namespace

int64_t layer_norm_backward_workspace_bytes(int64_t T, int d) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return -1;
  // the most CTAs that up to T rows of this width take, of any type and alignment
  int64_t grid = T < di.sm_count ? T : di.sm_count;  // few rows: one to a CTA
  for (int es = 2; es <= 4; es *= 2)
    for (int vec = 0; vec < 2; ++vec) {
      const LnPlan k = ln_plan(INT64_MAX, d, es, vec != 0, true, di);
      const int64_t cap = (int64_t)di.sm_count * (k.vpl ? k.per_sm : kLnBlocksPerSm);
      const int64_t n = T < cap ? T : cap;
      grid = n > grid ? n : grid;
    }
  return grid * 2 * d * 4;
}

cudaError_t launch_layer_norm(const LayerNormArgs& a) {
  const bool dgain = a.backward && (a.dgain || a.dbias);
  if (a.T == 0) {
    for (float* g : {a.dgain, a.dbias})
      if (dgain && g) {
        const cudaError_t e = cudaMemsetAsync(g, 0, (size_t)a.d * 4, a.stream);
        if (e != cudaSuccess) return e;
      }
    return cudaSuccess;
  }
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  LnParams p{a.x, a.dy, a.out, a.xs, a.dys, a.os, a.gain, a.bias, a.T, a.d, a.eps, 1.f / (float)a.d, dgain ? a.workspace : nullptr, 0};
  const bool bf16 = a.dtype == ATTNRES_BF16;
  const int es = bf16 ? 2 : 4, V = 16 / es;
  const bool vec = a.d % V == 0 && vec_rows(a.x, a.xs, V) && (!a.out || vec_rows(a.out, a.os, V)) && (!a.backward || vec_rows(a.dy, a.dys, V)) &&
                   ((reinterpret_cast<uintptr_t>(a.gain) | reinterpret_cast<uintptr_t>(a.bias)) & 15) == 0;
  const LnPlan k = ln_plan(a.T, a.d, es, vec, a.backward, di);
  int grid;
  if (k.vpl) {
    p.warps = k.warps;
    const int64_t need = (a.T + k.groups - 1) / k.groups, cap = (int64_t)di.sm_count * k.per_sm;
    grid = (int)(need < cap ? need : cap);
    const int most = di.max_smem_optin - ln_fixed_smem(a.backward);
    e = bf16 ? launch_rows<bf16_t>(a, p, k, vec, grid, most) : launch_rows<float>(a, p, k, vec, grid, most);
  } else {
    const int64_t cap = (int64_t)di.sm_count * kLnBlocksPerSm;
    grid = (int)(a.T < cap ? a.T : cap);
    if (bf16)
      e = a.backward ? launch_kernel(ln_any_kernel<bf16_t, true>, dim3(grid), dim3(kLnThreads), 0, a.stream, p)
                     : launch_kernel(ln_any_kernel<bf16_t, false>, dim3(grid), dim3(kLnThreads), 0, a.stream, p);
    else
      e = a.backward ? launch_kernel(ln_any_kernel<float, true>, dim3(grid), dim3(kLnThreads), 0, a.stream, p)
                     : launch_kernel(ln_any_kernel<float, false>, dim3(grid), dim3(kLnThreads), 0, a.stream, p);
  }
  if (e != cudaSuccess || !dgain) return e;
  return launch_kernel(ln_dgain_kernel, dim3((a.d + 31) / 32, 2), dim3(32 * kLnRuns), 0, a.stream, (const float*)p.part, grid, a.d,
                       a.dgain, a.dbias);
}

}  // namespace attnres
