// Layer norm of whole rows, and its backward.
//
//   h = (x - m) / sqrt(mean_c (x_c - m)^2 + eps),  y = gain * h + bias.
//   backward: n = gain * dy,  dx = (n - mean(n) - h mean(n h)) / sigma,
//   dgain = sum_t dy h,  dbias = sum_t dy.
//
// The mean is held as the sum of two fp32 numbers: m, the rounded mean, and
// delta, the mean of the differences x - m (exact where m is near x), so rows
// whose mean is far from zero keep their digits.
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
constexpr int kLnMaxWarps = 16;     // of a row (ln_row_kernel)

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
  int warps;    // ln_row_kernel: warps of a row
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

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(v, v); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  const int bytes = in ? 16 : 0;  // none: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// rows on their way: as many as shared memory holds at the widest, up to four
template <int VPT, bool BWD>
constexpr int kLnAhead = BWD && VPT > 2 ? 3 : 4;

// What a thread holds of a row: E channels, as packed pairs of fp32.  VEC: VPT
// 16-byte vectors, vector tid + i G of the row; otherwise single channels,
// channel tid + j G (G threads to a row).
template <typename T, int VPT, bool VEC>
struct Hold {
  static constexpr int V = Vec16<T>::kElems, E = VPT * V, P = E / 2;
  static __device__ __forceinline__ int channel(int j, int tid, int G) { return VEC ? (tid + j / V * G) * V + j % V : tid + j * G; }
  static __device__ __forceinline__ bool has(int j, int tid, int G, int d) { return channel(j, tid, G) < d; }
  static __device__ __forceinline__ void unpack(const uint4& v, uint64_t* f) {
    float t[V];
    Vec16<T>::unpack(v, t);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[i] = f2_pack(t[2 * i], t[2 * i + 1]);
  }
  // a row of single channels
  static __device__ __forceinline__ void load(const T* row, int tid, int G, int d, uint64_t (&f)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float t[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) t[k] = has(2 * i + k, tid, G, d) ? load_elem(row + channel(2 * i + k, tid, G)) : 0.f;
      f[i] = f2_pack(t[0], t[1]);
    }
  }
  static __device__ __forceinline__ void store(T* row, int tid, int G, int d, const uint64_t (&f)[P]) {
    float t[E];
#pragma unroll
    for (int i = 0; i < P; ++i) f2_unpack(f[i], t[2 * i], t[2 * i + 1]);
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (has(i * V, tid, G, d)) __stcs(reinterpret_cast<uint4*>(row) + tid + i * G, Vec16<T>::pack(t + i * V));
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (has(j, tid, G, d)) store_elem(row + channel(j, tid, G), t[j]);
    }
  }
  // a vector of fp32 (null: `none`); zero where there is no channel
  static __device__ __forceinline__ void load_f32(const float* v, float none, int tid, int G, int d, uint64_t (&f)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float t[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) t[k] = !has(2 * i + k, tid, G, d) ? 0.f : v ? __ldg(v + channel(2 * i + k, tid, G)) : none;
      f[i] = f2_pack(t[0], t[1]);
    }
  }
  // f where there is a channel, else 0
  static __device__ __forceinline__ void mask(int tid, int G, int d, uint64_t (&f)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if constexpr (VEC) {
        if (!has(2 * i / V * V, tid, G, d)) f[i] = 0;
      } else {
        float t[2];
        f2_unpack(f[i], t[0], t[1]);
        f[i] = f2_pack(has(2 * i, tid, G, d) ? t[0] : 0.f, has(2 * i + 1, tid, G, d) ? t[1] : 0.f);
      }
    }
  }
};

// sums of N values over a row's warps, the same in every thread of the row
// (one barrier: the caller alternates between two buffers)
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[4], int warps, int warp, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (warps == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[warp][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < warps ? red[lane & (kLnMaxWarps - 1)][i] : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
}

// Rows that fit the registers of up to 16 warps: read once, with the next ones
// on their way (VEC: cp.async into shared memory that each thread keeps to
// itself).  A row belongs to one warp of eight in a CTA, or to a whole CTA.
template <typename T, int VPT, bool BWD, bool VEC>
__global__ void __launch_bounds__(32 * kLnMaxWarps, BWD || VPT > 2 ? 1 : 2) ln_row_kernel(const __grid_constant__ LnParams p) {
  using H = Hold<T, VPT, VEC>;
  constexpr int P = H::P, kAhead = kLnAhead<VPT, BWD>, kArrays = BWD ? 2 : 1;
  extern __shared__ __align__(16) unsigned char ring_mem[];  // VEC: [kAhead][kArrays][VPT][threads] vectors; at the end, BWD: sums
  __shared__ __align__(16) float red[2][kLnMaxWarps][4];
  const int warps = p.warps, G = 32 * warps, lane = threadIdx.x & 31;
  const int groups = warps == 1 ? (int)blockDim.x >> 5 : 1, group = warps == 1 ? (int)threadIdx.x >> 5 : 0;
  const int tid = warps == 1 ? lane : (int)threadIdx.x, warp = warps == 1 ? 0 : (int)threadIdx.x >> 5;
  const int d = p.d;
  pdl_wait();
  pdl_trigger();
  const T* X = static_cast<const T*>(p.x);
  const T* DY = static_cast<const T*>(p.dy);
  T* O = static_cast<T*>(p.out);
  const long long step = (long long)gridDim.x * groups;
  long long t = (long long)blockIdx.x * groups + group, ahead_t = t;
  const uint32_t ring = smem_addr(ring_mem) + threadIdx.x * 16;
  const int slot_bytes = kArrays * VPT * (int)blockDim.x * 16;
  int ahead_slot = 0, slot = 0;
  auto fetch = [&] {
    if constexpr (VEC) {
      if (ahead_t < p.T) {
        const uint32_t to = ring + ahead_slot * slot_bytes;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const bool in = H::has(i * H::V, tid, G, d);
          const int at = in ? H::channel(i * H::V, tid, G) : 0;
          cp_async16(to + i * blockDim.x * 16, X + ahead_t * p.xs + at, in);
          if constexpr (BWD) cp_async16(to + (VPT + i) * blockDim.x * 16, DY + ahead_t * p.dys + at, in);
        }
      }
      ahead_t += step;
      ahead_slot = ahead_slot + 1 == kAhead ? 0 : ahead_slot + 1;
      cp_async_commit();  // a group for every row, there or not
    }
  };
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch();
  }
  uint64_t gain[P], bias[BWD ? 1 : P], dg[BWD ? P : 1], db[BWD ? P : 1], x[P], dy[BWD ? P : 1], next_x[VEC ? 1 : P], next_dy[!VEC && BWD ? P : 1];
  H::load_f32(p.gain, 1.f, tid, G, d, gain);
  if constexpr (!BWD) H::load_f32(p.bias, 0.f, tid, G, d, bias);
  if constexpr (BWD) {
#pragma unroll
    for (int i = 0; i < P; ++i) dg[i] = db[i] = 0;
  }
  if constexpr (!VEC) {
    if (t < p.T) {
      H::load(X + t * p.xs, tid, G, d, next_x);
      if constexpr (BWD) H::load(DY + t * p.dys, tid, G, d, next_dy);
    }
  }
  for (; t < p.T; t += step) {
    if constexpr (VEC) {
      cp_async_wait<kAhead - 1>();
      const uint32_t at = ring + slot * slot_bytes;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        H::unpack(ld_shared_v4(at + i * blockDim.x * 16), x + i * H::V / 2);
        if constexpr (BWD) H::unpack(ld_shared_v4(at + (VPT + i) * blockDim.x * 16), dy + i * H::V / 2);
      }
      slot = slot + 1 == kAhead ? 0 : slot + 1;
      fetch();  // into the slot just read
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        x[i] = next_x[i];
        if constexpr (BWD) dy[i] = next_dy[i];
      }
      if (t + step < p.T) {
        H::load(X + (t + step) * p.xs, tid, G, d, next_x);
        if constexpr (BWD) H::load(DY + (t + step) * p.dys, tid, G, d, next_dy);
      }
    }
    uint64_t sx = 0, sn = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      sx = f2_add(sx, x[i]);
      if constexpr (BWD) sn = f2_fma(dy[i], gain[i], sn);
    }
    float s1[2] = {f2_hsum(sx), f2_hsum(sn)};
    if constexpr (BWD) {
      row_sums<2>(s1, red[0], warps, warp, lane);
    } else {
      float s[1] = {s1[0]};
      row_sums<1>(s, red[0], warps, warp, lane);
      s1[0] = s[0];
    }
    const float m = s1[0] * p.inv_d;
    const uint64_t minus_m = f2_both(-m);
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = f2_add(x[i], minus_m);
    H::mask(tid, G, d, x);
    uint64_t sz = 0, sq = 0, sw = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      sz = f2_add(sz, x[i]);
      sq = f2_fma(x[i], x[i], sq);
      if constexpr (BWD) sw = f2_fma(f2_mul(dy[i], gain[i]), x[i], sw);
    }
    float s2[3] = {f2_hsum(sz), f2_hsum(sq), f2_hsum(sw)};
    if constexpr (BWD) {
      row_sums<3>(s2, red[1], warps, warp, lane);
    } else {
      float s[2] = {s2[0], s2[1]};
      row_sums<2>(s, red[1], warps, warp, lane);
      s2[0] = s[0];
      s2[1] = s[1];
    }
    const float delta = s2[0] * p.inv_d;
    const float rstd = rsqrtf(fmaxf(fmaf(-delta, delta, s2[1] * p.inv_d), 0.f) + p.eps);
    const uint64_t minus_delta = f2_both(-delta), r2 = f2_both(rstd);
    if constexpr (!BWD) {
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = f2_fma(f2_mul(f2_add(x[i], minus_delta), r2), gain[i], bias[i]);
      H::store(O + t * p.os, tid, G, d, x);
    } else {
      const float mn = s1[1] * p.inv_d;
      const float mh = (s2[2] * p.inv_d - delta * mn) * rstd;  // mean(n h)
      const uint64_t minus_mh = f2_both(-mh), minus_mn = f2_both(-mn);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint64_t h = f2_mul(f2_add(x[i], minus_delta), r2);
        dg[i] = f2_fma(dy[i], h, dg[i]);
        db[i] = f2_add(db[i], dy[i]);
        x[i] = f2_mul(f2_add(f2_fma(h, minus_mh, f2_mul(dy[i], gain[i])), minus_mn), r2);
      }
      if (O) H::store(O + t * p.os, tid, G, d, x);
    }
  }
  if constexpr (BWD) {
    if (!p.part) return;
    float* part = p.part + (long long)blockIdx.x * 2 * d;
    float* sums = reinterpret_cast<float*>(ring_mem);  // [groups][2][d]
    cp_async_wait<0>();
    __syncthreads();  // the ring is done with
#pragma unroll
    for (int j = 0; j < H::E; ++j) {
      float a[2], b[2];
      f2_unpack(dg[j / 2], a[0], a[1]);
      f2_unpack(db[j / 2], b[0], b[1]);
      if (H::has(j, tid, G, d)) {
        const int c = H::channel(j, tid, G);
        float* at = groups > 1 ? sums + group * 2 * d : part;
        at[c] = a[j & 1];
        at[d + c] = b[j & 1];
      }
    }
    if (groups > 1) {  // in order: the sums do not depend on timing
      __syncthreads();
      for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) {
        float s = 0.f;
        for (int g = 0; g < groups; ++g) s += sums[g * 2 * d + c];
        part[c] = s;
      }
    }
  }
}

// gain and bias gradients: the CTAs' partial rows, summed in order (32
// channels x 32 interleaved runs of rows per CTA, whose loads do not wait for
// one another; blockIdx.y: gain or bias)
constexpr int kLnRuns = 32;
__global__ void __launch_bounds__(32 * kLnRuns) ln_dgain_kernel(const float* part, int blocks, int d, float* dgain, float* dbias) {
  __shared__ float sums[kLnRuns][33];
  const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, r = threadIdx.x >> 5;
  float* out = blockIdx.y ? dbias : dgain;
  pdl_wait();
  pdl_trigger();
  if (!out) return;
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int b = r; b < blocks; b += kLnRuns) s += part[((long long)b * 2 + blockIdx.y) * d + c];
  }
  sums[r][lane] = s;
  __syncthreads();
  s = warp_sum(sums[lane][r]);  // warp r: channel r of the CTA's
  if (lane == 0 && blockIdx.x * 32 + r < d) out[blockIdx.x * 32 + r] = s;
}

// How a call's rows are held: vectors or channels to a thread, warps to a row
// (0: a row does not fit, ln_any_kernel).
struct LnPlan {
  int vpt, warps, threads;
};
LnPlan ln_plan(int d, int es, bool vec) {
  const int V = 16 / es;
  for (int vpt = vec ? 2 : 1; vpt <= (vec ? 4 : 2); vpt *= 2) {
    const int per_warp = 32 * vpt * (vec ? 1 : V), items = vec ? d / V : d;
    const int warps = (items + per_warp - 1) / per_warp;
    if (warps <= kLnMaxWarps) return {vpt, warps, warps == 1 ? 256 : 32 * warps};
  }
  return {0, 0, 0};
}
// CTAs to an SM: the forward's registers allow 32 warps, the backward's 16
int ln_blocks_per_sm(const LnPlan& k, bool backward) {
  const int n = (backward || k.vpt > 2 ? 512 : 1024) / k.threads;
  return n < 1 ? 1 : n > 8 ? 8 : n;
}

template <typename T, int VPT, bool VEC>
cudaError_t launch_rows(const LayerNormArgs& a, const LnParams& p, const LnPlan& k, int grid) {
  const int ring = VEC ? (a.backward ? kLnAhead<VPT, true> : kLnAhead<VPT, false>) * (a.backward ? 2 : 1) * VPT * k.threads * 16 : 0;
  const int sums = a.backward && k.warps == 1 ? k.threads / 32 * 2 * a.d * 4 : 0;
  const int smem = ring > sums ? ring : sums;
  if (a.backward) {
    static SmemOptIn opt;
    const cudaError_t e = opt.ensure(reinterpret_cast<const void*>(ln_row_kernel<T, VPT, true, VEC>), kLnAhead<VPT, true> * 2 * VPT * 32 * kLnMaxWarps * 16);
    if (e != cudaSuccess) return e;
    return launch_kernel(ln_row_kernel<T, VPT, true, VEC>, dim3(grid), dim3(k.threads), smem, a.stream, p);
  }
  static SmemOptIn opt;
  const cudaError_t e = opt.ensure(reinterpret_cast<const void*>(ln_row_kernel<T, VPT, false, VEC>), kLnAhead<VPT, false> * VPT * 32 * kLnMaxWarps * 16);
  if (e != cudaSuccess) return e;
  return launch_kernel(ln_row_kernel<T, VPT, false, VEC>, dim3(grid), dim3(k.threads), smem, a.stream, p);
}

template <typename T>
cudaError_t launch_rows(const LayerNormArgs& a, const LnParams& p, const LnPlan& k, bool vec, int grid) {
  if (vec) return k.vpt == 2 ? launch_rows<T, 2, true>(a, p, k, grid) : launch_rows<T, 4, true>(a, p, k, grid);
  return k.vpt == 1 ? launch_rows<T, 1, false>(a, p, k, grid) : launch_rows<T, 2, false>(a, p, k, grid);
}

bool vec_rows(const void* ptr, int64_t stride, int V) { return (reinterpret_cast<uintptr_t>(ptr) & 15) == 0 && stride % V == 0; }

}  // namespace

int64_t layer_norm_backward_workspace_bytes(int64_t T, int d) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return -1;
  // the most CTAs that any type or alignment of rows of this width takes
  int blocks = 0;
  for (int es = 2; es <= 4; es *= 2)
    for (int vec = 0; vec < 2; ++vec) {
      const LnPlan k = ln_plan(d, es, vec != 0);
      const int n = k.vpt ? ln_blocks_per_sm(k, true) : kLnBlocksPerSm;
      blocks = n > blocks ? n : blocks;
    }
  int64_t grid = (int64_t)di.sm_count * blocks;
  if (T < grid) grid = T;
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
  const bool vec = a.d % V == 0 && vec_rows(a.x, a.xs, V) && (!a.out || vec_rows(a.out, a.os, V)) && (!a.backward || vec_rows(a.dy, a.dys, V));
  const LnPlan k = ln_plan(a.d, es, vec);
  int grid;
  if (k.vpt) {
    p.warps = k.warps;
    const int64_t rows = k.warps == 1 ? k.threads / 32 : 1, need = (a.T + rows - 1) / rows;  // of a CTA at a time
    const int64_t cap = (int64_t)di.sm_count * ln_blocks_per_sm(k, a.backward);
    grid = (int)(need < cap ? need : cap);
    e = bf16 ? launch_rows<bf16_t>(a, p, k, vec, grid) : launch_rows<float>(a, p, k, vec, grid);
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
