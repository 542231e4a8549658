// RMSNorm of every head of q and k with the rotation by position in the same
// pass, and its backward.
//
//   y = gain * x / rho,  rho = sqrt(mean_c x_c^2 + eps);  pair i of the first
//   `rot` channels turns by positions[t] * inv_freq[i].
//   backward: dy = the incoming gradient turned back, n = gain * dy,
//   dx = (n - h mean(n h)) / rho with h = x / rho,  dgain = sum dy h.
//
// Every element is read once and written once: the bound is HBM.  A group of
// L lanes owns one token and runs through a range of its heads: the cosines
// and sines of the token's position are computed once per group and stay in
// registers, the two 16-byte vectors that a lane holds of a head contain both
// members of its pairs (no exchange between lanes but the row sums), and the
// next head's vectors load while this one is computed.
//
// Angles: p inv_freq is reduced modulo a full turn before it is rounded to
// fp32.  inv_freq / (2 pi) is held as an unevaluated sum of two fp32 numbers
// (2^-48 relative), its product with the position is split exactly by fma,
// and whole turns are dropped from both parts; positions of 2^24 and more,
// which fp32 does not hold, take one fp64 product instead.
#include <math.h>

#include "attnres.h"
#include "body.h"
#include "device_common.cuh"
#include "launch.h"
#include "vec16.cuh"

namespace attnres {

namespace {

constexpr int kQkThreads = 256;
constexpr int kQkBlocksPerSm = 4;  // resident CTAs the grid is sized for
constexpr int kQkMaxD = 1024;

struct QkParams {
  QkHead h[2];
  int blocks0;      // CTAs 0 .. blocks0 - 1 work on h[0], the others on h[1]
  int hc[2];        // heads per group and pass
  long long units[2];  // T * ceil(H / hc)
  long long T;
  int D, rot;
  float eps, inv_d;
  const long long* pos;
  const float* freq;
  float* part;  // [grid][D] partial gain gradients
};

// 1 / (2 pi) as the sum of two fp32 numbers
constexpr float kTurnHi = 0.15915494f;
constexpr float kTurnLo = (float)(0.15915494309189533577 - (double)0.15915494f);

__device__ __forceinline__ void turn(long long pos, float freq, float* c, float* s) {
  float frac;
  if (pos > -(1 << 24) && pos < (1 << 24)) {
    const float p = (float)(int)pos;  // exact
    const float rh = freq * kTurnHi;
    const float rl = fmaf(freq, kTurnHi, -rh) + freq * kTurnLo;
    const float th = p * rh;
    const float tl = fmaf(p, rh, -th) + p * rl;
    frac = (th - rintf(th)) + (tl - rintf(tl));
  } else {
    const double t = (double)pos * (double)freq * 0.15915494309189533577;
    frac = (float)(t - rint(t));
  }
  sincospif(2.f * frac, s, c);
}

// sum over the L lanes of a group (L a power of two)
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// (a, b) turned by (c, s)
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = a * c - b * s;
  b = fmaf(b, c, a * s);
  a = x;
}

// INTER pairs channels (2i, 2i + 1), otherwise (i, i + rot/2).
template <typename T, int L, bool INTER, bool BWD>
__global__ void __launch_bounds__(kQkThreads) qk_vec_kernel(const __grid_constant__ QkParams p) {
  constexpr int V = Vec16<T>::kElems;
  constexpr int kGroups = kQkThreads / L;
  extern __shared__ float smem[];  // BWD: [kGroups][D]
  const int which = blockIdx.x >= p.blocks0 ? 1 : 0;
  const QkHead& hd = p.h[which];
  const int block = blockIdx.x - (which ? p.blocks0 : 0);
  const int nblocks = which ? gridDim.x - p.blocks0 : p.blocks0;
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int nv = p.D / V;

  // the two vectors of this lane, and which of their pairs turn
  int va, vb;
  bool rot_half = false;
  if constexpr (INTER) {
    const int n2 = (nv + 1) / 2;
    va = lane < n2 ? lane : nv;
    vb = lane < n2 ? lane + n2 : nv;
  } else {
    const int r2 = p.rot / (2 * V);
    rot_half = lane < r2;
    va = rot_half ? lane : 2 * lane;            // the unrotated vectors start at 2 r2
    vb = rot_half ? lane + r2 : 2 * lane + 1;
  }
  const bool ha = va < nv, hb = vb < nv;

  pdl_wait();
  pdl_trigger();

  float ga[V], gb[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    ga[e] = hd.gain && ha ? __ldg(hd.gain + va * V + e) : 1.f;
    gb[e] = hd.gain && hb ? __ldg(hd.gain + vb * V + e) : 1.f;
  }
  float dga[BWD ? V : 1], dgb[BWD ? V : 1];
  if constexpr (BWD) {
#pragma unroll
    for (int e = 0; e < V; ++e) dga[e] = dgb[e] = 0.f;
  }

  const int hc = p.hc[which];
  const int nch = (hd.H + hc - 1) / hc;
  const T* X = static_cast<const T*>(hd.x);
  const T* DY = static_cast<const T*>(hd.dy);
  T* O = static_cast<T*>(hd.out);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // the loop is uniform over a warp (its groups share the shuffles): a group
  // past the end works on nothing
  const long long stride = (long long)nblocks * kGroups;
  const long long warp_unit = (long long)block * kGroups + (threadIdx.x / 32) * (32 / L);
  for (long long u0 = warp_unit; u0 < p.units[which]; u0 += stride) {
    const long long u = u0 + group % (32 / L);
    const bool live = u < p.units[which];
    const long long t = live ? u / nch : 0;
    const int h0 = live ? (int)(u % nch) * hc : 0;
    const int h1 = live ? (h0 + hc < hd.H ? h0 + hc : hd.H) : 0;

    float cs[V], sn[V];
    if (p.rot > 0) {
      const long long pos = __ldg(p.pos + t);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        int i;  // frequency of the lane's pair e
        if constexpr (INTER)
          i = e < V / 2 ? va * (V / 2) + e : vb * (V / 2) + e - V / 2;
        else
          i = rot_half ? lane * V + e : p.rot;
        cs[e] = 1.f;
        sn[e] = 0.f;
        if (i < p.rot / 2) turn(pos, __ldg(p.freq + i), &cs[e], &sn[e]);
      }
    }

    const T* x = X + t * hd.xs;
    const T* dy = BWD ? DY + t * hd.dys : nullptr;
    T* o = O + t * hd.os;
    const bool la = ha && live, lb = hb && live;
    uint4 xa = zero, xb = zero, ya = zero, yb = zero;
    auto load = [&](int h) {
      const bool in = h < h1;
      xa = in && la ? __ldcs(reinterpret_cast<const uint4*>(x + (long long)h * p.D) + va) : zero;
      xb = in && lb ? __ldcs(reinterpret_cast<const uint4*>(x + (long long)h * p.D) + vb) : zero;
      if constexpr (BWD) {
        ya = in && la ? __ldcs(reinterpret_cast<const uint4*>(dy + (long long)h * p.D) + va) : zero;
        yb = in && lb ? __ldcs(reinterpret_cast<const uint4*>(dy + (long long)h * p.D) + vb) : zero;
      }
    };
    load(h0);
    for (int k = 0; k < hc; ++k) {  // the same count for every group of the warp
      const int h = h0 + k;
      float a[V], b[V], da[BWD ? V : 1], db[BWD ? V : 1];
      Vec16<T>::unpack(xa, a);
      Vec16<T>::unpack(xb, b);
      if constexpr (BWD) {
        Vec16<T>::unpack(ya, da);
        Vec16<T>::unpack(yb, db);
      }
      load(h + 1);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
      if constexpr (!BWD) {
        const float inv = 1.f / sqrtf(group_sum<L>(ss) * p.inv_d + p.eps);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          a[e] *= inv * ga[e];
          b[e] *= inv * gb[e];
        }
        if (p.rot > 0) {
          if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
              rotate(a[2 * e], a[2 * e + 1], cs[e], sn[e]);
              rotate(b[2 * e], b[2 * e + 1], cs[V / 2 + e], sn[V / 2 + e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) rotate(a[e], b[e], cs[e], sn[e]);
          }
        }
      } else {
        if (p.rot > 0) {
          if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
              rotate(da[2 * e], da[2 * e + 1], cs[e], -sn[e]);
              rotate(db[2 * e], db[2 * e + 1], cs[V / 2 + e], -sn[V / 2 + e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) rotate(da[e], db[e], cs[e], -sn[e]);
          }
        }
        float nx = 0.f;  // sum n x
#pragma unroll
        for (int e = 0; e < V; ++e) nx = fmaf(da[e] * ga[e], a[e], fmaf(db[e] * gb[e], b[e], nx));
        const float inv = 1.f / sqrtf(group_sum<L>(ss) * p.inv_d + p.eps);
        const float mh = group_sum<L>(nx) * p.inv_d * inv;  // mean(n h)
        const bool in = h < h1;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float hx = a[e] * inv, hy = b[e] * inv;
          if (in) {  // a head past the group's range holds zeros, and 0 / rho may be NaN (eps = 0)
            dga[e] = fmaf(da[e], hx, dga[e]);
            dgb[e] = fmaf(db[e], hy, dgb[e]);
          }
          a[e] = (da[e] * ga[e] - hx * mh) * inv;
          b[e] = (db[e] * gb[e] - hy * mh) * inv;
        }
      }
      if (h < h1) {
        if (la) __stcs(reinterpret_cast<uint4*>(o + (long long)h * p.D) + va, Vec16<T>::pack(a));
        if (lb) __stcs(reinterpret_cast<uint4*>(o + (long long)h * p.D) + vb, Vec16<T>::pack(b));
      }
    }
  }
  if constexpr (BWD) {
    if (p.part) {  // groups in order: the sums do not depend on timing
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (ha) smem[group * p.D + va * V + e] = dga[e];
        if (hb) smem[group * p.D + vb * V + e] = dgb[e];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < p.D; c += kQkThreads) {
        float s = 0.f;
        for (int g = 0; g < kGroups; ++g) s += smem[g * p.D + c];
        p.part[(long long)blockIdx.x * p.D + c] = s;
      }
    }
  }
}

// Any head size, alignment and stride: one warp per head row.  A lane reads
// and writes both members of its pairs, so a row may be its own result.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kQkThreads) qk_any_kernel(const __grid_constant__ QkParams p, bool inter) {
  constexpr int kWarps = kQkThreads / 32;
  extern __shared__ float smem[];  // BWD: [kWarps][D]
  const int which = blockIdx.x >= p.blocks0 ? 1 : 0;
  const QkHead& hd = p.h[which];
  const int block = blockIdx.x - (which ? p.blocks0 : 0);
  const int nblocks = which ? gridDim.x - p.blocks0 : p.blocks0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int items = p.D - p.rot / 2;  // rotated pairs, then single channels
  const int half = p.rot / 2;
  float* dg = smem + warp * p.D;
  if (BWD && p.part)
    for (int c = lane; c < p.D; c += 32) dg[c] = 0.f;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  auto gain = [&](int c) { return hd.gain ? __ldg(hd.gain + c) : 1.f; };
  for (long long u = (long long)block * kWarps + warp; u < p.units[which]; u += (long long)nblocks * kWarps) {
    const long long t = u / hd.H;
    const int h = (int)(u % hd.H);
    const T* x = static_cast<const T*>(hd.x) + t * hd.xs + (long long)h * p.D;
    const T* dy = BWD ? static_cast<const T*>(hd.dy) + t * hd.dys + (long long)h * p.D : nullptr;
    T* o = static_cast<T*>(hd.out) + t * hd.os + (long long)h * p.D;
    const long long pos = p.rot > 0 ? __ldg(p.pos + t) : 0;
    float ss = 0.f, nx = 0.f;
    for (int c = lane; c < p.D; c += 32) {
      const float v = load_elem(x + c);
      ss = fmaf(v, v, ss);
    }
    const float inv = 1.f / sqrtf(warp_sum(ss) * p.inv_d + p.eps);
    if (BWD) {
      for (int i = lane; i < items; i += 32) {
        const int a = i < half ? (inter ? 2 * i : i) : half + i, b = inter ? a + 1 : a + half;
        float da = load_elem(dy + a);
        if (i < half) {
          float db = load_elem(dy + b), c, s;
          turn(pos, __ldg(p.freq + i), &c, &s);
          rotate(da, db, c, -s);
          const float xb = load_elem(x + b);
          nx = fmaf(db * gain(b), xb, nx);
          if (p.part) dg[b] = fmaf(db, xb * inv, dg[b]);
        }
        const float xa = load_elem(x + a);
        nx = fmaf(da * gain(a), xa, nx);
        if (p.part) dg[a] = fmaf(da, xa * inv, dg[a]);
      }
    }
    const float mh = BWD ? warp_sum(nx) * p.inv_d * inv : 0.f;
    __syncwarp();  // every lane has read the row before any lane writes (in place)
    for (int i = lane; i < items; i += 32) {
      const int a = i < half ? (inter ? 2 * i : i) : half + i, b = inter ? a + 1 : a + half;
      float c = 1.f, s = 0.f;
      if (i < half) turn(pos, __ldg(p.freq + i), &c, &s);
      const float xa = load_elem(x + a) * inv, xb = i < half ? load_elem(x + b) * inv : 0.f;
      if (!BWD) {
        float ya = xa * gain(a), yb = i < half ? xb * gain(b) : 0.f;
        if (i < half) rotate(ya, yb, c, s);
        store_elem(o + a, ya);
        if (i < half) store_elem(o + b, yb);
      } else {
        float da = load_elem(dy + a), db = i < half ? load_elem(dy + b) : 0.f;
        if (i < half) rotate(da, db, c, -s);
        store_elem(o + a, (da * gain(a) - xa * mh) * inv);
        if (i < half) store_elem(o + b, (db * gain(b) - xb * mh) * inv);
      }
    }
  }
  if (BWD && p.part) {
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += kQkThreads) {
      float s = 0.f;
      for (int g = 0; g < kWarps; ++g) s += smem[g * p.D + c];
      p.part[(long long)blockIdx.x * p.D + c] = s;
    }
  }
}

// gain gradients: the CTAs' partial rows, summed in order (32 channels x 8
// interleaved runs of rows per CTA; blockIdx.y: q or k)
__global__ void __launch_bounds__(256) qk_dgain_kernel(const float* part, int blocks0, int blocks, int D, float* dq,
                                                       float* dk) {
  __shared__ float sums[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  const int b0 = blockIdx.y ? blocks0 : 0, b1 = blockIdx.y ? blocks : blocks0;
  float* out = blockIdx.y ? dk : dq;
  pdl_wait();
  pdl_trigger();
  float s = 0.f;
  if (c < D && out)
    for (int b = b0 + r; b < b1; b += 8) s += part[(long long)b * D + c];
  sums[r][threadIdx.x & 31] = s;
  __syncthreads();
  if (r == 0 && c < D && out) {
    for (int k = 1; k < 8; ++k) s += sums[k][threadIdx.x & 31];
    out[c] = s;
  }
}

template <typename T, int L, bool BWD>
cudaError_t launch_vec(const QkArgs& a, const QkParams& p, int grid) {
  const int smem = BWD && p.part ? kQkThreads / L * p.D * 4 : 0;
  return a.interleaved ? launch_kernel(qk_vec_kernel<T, L, true, BWD>, dim3(grid), dim3(kQkThreads), smem, a.stream, p)
                       : launch_kernel(qk_vec_kernel<T, L, false, BWD>, dim3(grid), dim3(kQkThreads), smem, a.stream, p);
}

template <typename T, bool BWD>
cudaError_t launch_lanes(const QkArgs& a, const QkParams& p, int L, int grid) {
  switch (L) {
    case 4: return launch_vec<T, 4, BWD>(a, p, grid);
    case 8: return launch_vec<T, 8, BWD>(a, p, grid);
    case 16: return launch_vec<T, 16, BWD>(a, p, grid);
    default: return launch_vec<T, 32, BWD>(a, p, grid);
  }
}

bool vec_rows(const void* ptr, int64_t stride, int V) {
  return (reinterpret_cast<uintptr_t>(ptr) & 15) == 0 && stride % V == 0;
}

}  // namespace

int64_t qk_backward_workspace_bytes(int64_t T, int Hq, int Hk, int D) {
  (void)T, (void)Hq, (void)Hk;
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return -1;
  return (int64_t)di.sm_count * kQkBlocksPerSm * D * 4;
}

cudaError_t launch_qk_norm_rope(const QkArgs& a) {
  const bool dgain = a.backward && (a.h[0].dgain || a.h[1].dgain);
  if (a.T == 0) {
    for (const QkHead& h : a.h)
      if (dgain && h.dgain) {
        const cudaError_t e = cudaMemsetAsync(h.dgain, 0, (size_t)a.D * 4, a.stream);
        if (e != cudaSuccess) return e;
      }
    return cudaSuccess;
  }
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const int es = a.dtype == ATTNRES_BF16 ? 2 : 4, V = 16 / es;

  // 16-byte vectors: whole vectors per head, at most two per lane, and pairs
  // of rotate-halves in two vectors of one lane
  const int nv = a.D / V;
  bool vec = a.D % V == 0 && nv <= 64 && (a.interleaved || a.rot % (2 * V) == 0);
  for (const QkHead& h : a.h)
    if (h.H > 0)
      vec = vec && vec_rows(h.x, h.xs, V) && vec_rows(h.out, h.os, V) && (!a.backward || vec_rows(h.dy, h.dys, V));
  int L = 4;
  while (L < (nv + 1) / 2) L *= 2;
  const int groups = vec ? kQkThreads / L : kQkThreads / 32;  // per CTA

  QkParams p{};
  p.h[0] = a.h[0];
  p.h[1] = a.h[1];
  p.T = a.T;
  p.D = a.D;
  p.rot = a.rot;
  p.eps = a.eps;
  p.inv_d = 1.f / (float)a.D;
  p.pos = reinterpret_cast<const long long*>(a.pos);
  p.freq = a.freq;
  p.part = dgain ? a.workspace : nullptr;
  // heads per group and pass: all of them when there are tokens enough to
  // fill the GPU, fewer (each group then computes its angles again) when not
  const long long slots = (long long)di.sm_count * kQkBlocksPerSm * groups;
  const long long rows = a.T * (a.h[0].H + a.h[1].H);
  int hc = (int)(vec ? (rows + slots - 1) / slots : 1);
  if (hc > 16) hc = 16;
  for (int i = 0; i < 2; ++i) {
    const int H = a.h[i].H;
    p.hc[i] = H < 1 ? 1 : (hc < H ? hc : H);
    p.units[i] = H > 0 ? a.T * ((H + p.hc[i] - 1) / p.hc[i]) : 0;
  }
  // CTAs to q and k by their share of the units, at least one each
  const long long need0 = (p.units[0] + groups - 1) / groups, need1 = (p.units[1] + groups - 1) / groups;
  const long long cap = (long long)di.sm_count * kQkBlocksPerSm;
  long long b0 = need0, b1 = need1;
  if (b0 + b1 > cap) {
    b0 = need0 * cap / (need0 + need1);
    if (b0 < 1 && need0 > 0) b0 = 1;
    if (b0 > cap - 1 && need1 > 0) b0 = cap - 1;
    b1 = need1 > 0 ? cap - b0 : 0;
  }
  p.blocks0 = (int)b0;
  const int grid = (int)(b0 + b1);
  if (vec) {
    if (a.dtype == ATTNRES_BF16)
      e = a.backward ? launch_lanes<bf16_t, true>(a, p, L, grid) : launch_lanes<bf16_t, false>(a, p, L, grid);
    else
      e = a.backward ? launch_lanes<float, true>(a, p, L, grid) : launch_lanes<float, false>(a, p, L, grid);
  } else {
    const int smem = p.part ? kQkThreads / 32 * a.D * 4 : 0;
    if (a.dtype == ATTNRES_BF16)
      e = a.backward ? launch_kernel(qk_any_kernel<bf16_t, true>, dim3(grid), dim3(kQkThreads), smem, a.stream, p, a.interleaved)
                     : launch_kernel(qk_any_kernel<bf16_t, false>, dim3(grid), dim3(kQkThreads), smem, a.stream, p, a.interleaved);
    else
      e = a.backward ? launch_kernel(qk_any_kernel<float, true>, dim3(grid), dim3(kQkThreads), smem, a.stream, p, a.interleaved)
                     : launch_kernel(qk_any_kernel<float, false>, dim3(grid), dim3(kQkThreads), smem, a.stream, p, a.interleaved);
  }
  if (e != cudaSuccess || !dgain) return e;
  return launch_kernel(qk_dgain_kernel, dim3((a.D + 31) / 32, 2), dim3(256), 0, a.stream, (const float*)p.part, p.blocks0, grid, a.D,
                       a.h[0].dgain, a.h[1].dgain);
}

}  // namespace attnres
