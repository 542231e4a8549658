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
// vectors of the next rows are on their way (cp.async into shared memory that
// each thread keeps to itself: four rows ahead, two in the backward, where a
// register prefetch of one row left HBM at 57 % on 16384 tokens x 112 heads:
// 169 us, 5.6 TB/s; backward of 2047 tokens x 30 heads of 96 in fp32: 25 us).
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
constexpr int kQkBlocksPerSm = 3;     // resident CTAs of the forward (2 or 4 are slower: rows in flight against registers)
constexpr int kQkBwdBlocksPerSm = 2;  // of the backward

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

// A lane's two vectors as packed fp32: X the first members of its pairs, Y
// the second ones, two pairs to a register pair.  INTER: the pairs are
// neighbours inside a vector (X[0 .. V/4) of vector a, the rest of b);
// otherwise X is vector a and Y vector b.
template <typename T, bool INTER>
struct Pairs;
template <bool INTER>
struct Pairs<bf16_t, INTER> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const uint4& a, const uint4& b, uint64_t* X, uint64_t* Y) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      X[i] = INTER ? f2_pack(bf16lo(w[2 * i]), bf16lo(w[2 * i + 1])) : f2_pack(bf16lo(w[i]), bf16hi(w[i]));
      Y[i] = INTER ? f2_pack(bf16hi(w[2 * i]), bf16hi(w[2 * i + 1])) : f2_pack(bf16lo(w[4 + i]), bf16hi(w[4 + i]));
    }
  }
  static __device__ __forceinline__ void store(const uint64_t* X, const uint64_t* Y, uint4* a, uint4* b) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x0, x1, y0, y1;
      f2_unpack(X[i], x0, x1);
      f2_unpack(Y[i], y0, y1);
      w[INTER ? 2 * i : i] = INTER ? pack_bf16x2(x0, y0) : pack_bf16x2(x0, x1);
      w[INTER ? 2 * i + 1 : 4 + i] = INTER ? pack_bf16x2(x1, y1) : pack_bf16x2(y0, y1);
    }
    *a = make_uint4(w[0], w[1], w[2], w[3]);
    *b = make_uint4(w[4], w[5], w[6], w[7]);
  }
};
template <bool INTER>
struct Pairs<float, INTER> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void load(const uint4& a, const uint4& b, uint64_t* X, uint64_t* Y) {
    auto f = [](uint32_t u) { return __uint_as_float(u); };
    X[0] = INTER ? f2_pack(f(a.x), f(a.z)) : f2_pack(f(a.x), f(a.y));
    Y[0] = INTER ? f2_pack(f(a.y), f(a.w)) : f2_pack(f(b.x), f(b.y));
    X[1] = INTER ? f2_pack(f(b.x), f(b.z)) : f2_pack(f(a.z), f(a.w));
    Y[1] = INTER ? f2_pack(f(b.y), f(b.w)) : f2_pack(f(b.z), f(b.w));
  }
  static __device__ __forceinline__ void store(const uint64_t* X, const uint64_t* Y, uint4* a, uint4* b) {
    float x[4], y[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f2_unpack(X[i], x[2 * i], x[2 * i + 1]);
      f2_unpack(Y[i], y[2 * i], y[2 * i + 1]);
    }
    auto u = [](float v) { return __float_as_uint(v); };
    *a = INTER ? make_uint4(u(x[0]), u(y[0]), u(x[1]), u(y[1])) : make_uint4(u(x[0]), u(x[1]), u(x[2]), u(x[3]));
    *b = INTER ? make_uint4(u(x[2]), u(y[2]), u(x[3]), u(y[3])) : make_uint4(u(y[0]), u(y[1]), u(y[2]), u(y[3]));
  }
};

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// each pair (x, y) turned by (c, s)
__device__ __forceinline__ void rotate2(uint64_t& x, uint64_t& y, uint64_t c, uint64_t s) {
  const uint64_t minus = f2_pack(-1.f, -1.f);
  const uint64_t ys = f2_mul(f2_mul(y, s), minus), xs = f2_mul(x, s);
  x = f2_fma(x, c, ys);
  y = f2_fma(y, c, xs);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  const int bytes = in ? 16 : 0;  // none: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// INTER pairs channels (2i, 2i + 1), otherwise (i, i + rot/2).
template <typename T, int L, bool INTER, bool BWD>
__global__ void __launch_bounds__(kQkThreads, BWD ? kQkBwdBlocksPerSm : kQkBlocksPerSm) qk_vec_kernel(const __grid_constant__ QkParams p) {
  constexpr int V = Vec16<T>::kElems, NP = Pairs<T, INTER>::N;
  constexpr int kGroups = kQkThreads / L;
  constexpr int kAhead = BWD ? 2 : 4, kVecs = BWD ? 4 : 2;  // rows on their way; vectors of a row per thread
  extern __shared__ __align__(16) float smem[];  // [kAhead][kVecs][threads] vectors; at the end, BWD: [kGroups][D]
  // this head's gains, a vector's first members before its second ones
  // (INTER), read again for every row: the registers go to loads in flight
  __shared__ __align__(16) float gains[64 * V];
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

  for (int c = threadIdx.x; c < p.D; c += kQkThreads)
    gains[INTER ? c / V * V + c % 2 * (V / 2) + c % V / 2 : c] = hd.gain ? __ldg(hd.gain + c) : 1.f;
  __syncthreads();
  // the lane's gains in the order of X and Y (vector 0's where it has none)
  auto gain = [&](uint64_t* GX, uint64_t* GY) {
    const ulonglong2* ga = reinterpret_cast<const ulonglong2*>(gains + (ha ? va : 0) * V);
    const ulonglong2* gb = reinterpret_cast<const ulonglong2*>(gains + (hb ? vb : 0) * V);
    if constexpr (V == 8) {
      const ulonglong2 a0 = ga[0], a1 = ga[1], b0 = gb[0], b1 = gb[1];
      GX[0] = a0.x, GX[1] = a0.y;
      GX[2] = INTER ? b0.x : a1.x, GX[3] = INTER ? b0.y : a1.y;
      GY[0] = INTER ? a1.x : b0.x, GY[1] = INTER ? a1.y : b0.y;
      GY[2] = b1.x, GY[3] = b1.y;
    } else {
      const ulonglong2 a0 = ga[0], b0 = gb[0];
      GX[0] = a0.x, GX[1] = INTER ? b0.x : a0.y;
      GY[0] = INTER ? a0.y : b0.x, GY[1] = b0.y;
    }
  };
  uint64_t dgx[BWD ? NP : 1], dgy[BWD ? NP : 1];
  if constexpr (BWD) {
#pragma unroll
    for (int e = 0; e < NP; ++e) dgx[e] = dgy[e] = 0;
  }

  const int hc = p.hc[which];
  const int nch = (hd.H + hc - 1) / hc;
  const T* X0 = static_cast<const T*>(hd.x);
  const T* DY = static_cast<const T*>(hd.dy);
  T* O = static_cast<T*>(hd.out);
  // the loop is uniform over a warp (its groups share the shuffles): a group
  // past the end works on nothing
  const long long stride = (long long)nblocks * kGroups;
  const long long warp_unit = (long long)block * kGroups + (threadIdx.x / 32) * (32 / L), units = p.units[which];
  struct Unit {
    long long t;
    int h0, h1;
  };
  auto unit = [&](long long u0) {
    const long long u = u0 + group % (32 / L);
    Unit r{0, 0, 0};
    if (u < units) {
      r.t = u / nch;
      r.h0 = (int)(u % nch) * hc;
      r.h1 = r.h0 + hc < hd.H ? r.h0 + hc : hd.H;
    }
    return r;
  };
  // the rows ahead: row `ahead_k` of unit `ahead_u`, in ring order
  const uint32_t ring = smem_addr(smem) + threadIdx.x * 16;
  long long ahead_u = warp_unit;
  int ahead_k = 0, ahead_slot = 0;
  Unit au = unit(ahead_u);
  auto fetch = [&] {
    if (ahead_u < units) {
      const int h = au.h0 + ahead_k;
      const bool in = h < au.h1;
      const long long xo = in ? au.t * hd.xs + (long long)h * p.D : 0;
      const uint32_t to = ring + ahead_slot * (kVecs * kQkThreads * 16);
      cp_async16(to, X0 + xo + (ha ? va * V : 0), in && ha);
      cp_async16(to + kQkThreads * 16, X0 + xo + (hb ? vb * V : 0), in && hb);
      if constexpr (BWD) {
        const long long yo = in ? au.t * hd.dys + (long long)h * p.D : 0;
        cp_async16(to + 2 * kQkThreads * 16, DY + yo + (ha ? va * V : 0), in && ha);
        cp_async16(to + 3 * kQkThreads * 16, DY + yo + (hb ? vb * V : 0), in && hb);
      }
      if (++ahead_k == hc) {
        ahead_k = 0;
        ahead_u += stride;
        au = unit(ahead_u);
      }
      ahead_slot = ahead_slot + 1 == kAhead ? 0 : ahead_slot + 1;
    }
    cp_async_commit();  // a group for every row, empty or not
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch();
  int slot = 0;
  for (long long u0 = warp_unit; u0 < units; u0 += stride) {
    const Unit cu = unit(u0);
    const long long t = cu.t;
    const int h0 = cu.h0, h1 = cu.h1;

    // cosines and sines of the lane's 2 NP pairs, in the order of X
    uint64_t cs[NP], sn[NP];
    if (p.rot > 0) {
      const long long pos = __ldg(p.pos + t);
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        float c[2] = {1.f, 1.f}, sv[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int pair = 2 * e + k;
          int i;  // its frequency
          if constexpr (INTER)
            i = pair < NP ? va * NP + pair : vb * NP + pair - NP;
          else
            i = rot_half ? lane * V + pair : p.rot;
          if (i < p.rot / 2) turn(pos, __ldg(p.freq + i), &c[k], &sv[k]);
          if (BWD) sv[k] = -sv[k];  // gradients turn back
        }
        cs[e] = f2_pack(c[0], c[1]);
        sn[e] = f2_pack(sv[0], sv[1]);
      }
    }

    T* o = O + t * hd.os;
    for (int k = 0; k < hc; ++k) {  // the same count for every group of the warp
      const int h = h0 + k;
      uint64_t X[NP], Y[NP], GX[NP], GY[NP], dX[BWD ? NP : 1], dY[BWD ? NP : 1];
      cp_async_wait<kAhead - 1>();
      const uint32_t at = ring + slot * (kVecs * kQkThreads * 16);
      Pairs<T, INTER>::load(ld_shared_v4(at), ld_shared_v4(at + kQkThreads * 16), X, Y);
      if constexpr (BWD) Pairs<T, INTER>::load(ld_shared_v4(at + 2 * kQkThreads * 16), ld_shared_v4(at + 3 * kQkThreads * 16), dX, dY);
      slot = slot + 1 == kAhead ? 0 : slot + 1;
      fetch();  // into the slot just read
      uint64_t sq = 0;
#pragma unroll
      for (int e = 0; e < NP; ++e) sq = f2_fma(X[e], X[e], f2_fma(Y[e], Y[e], sq));
      const float inv = rsqrtf(group_sum<L>(f2_hsum(sq)) * p.inv_d + p.eps);
      const uint64_t inv2 = f2_pack(inv, inv);
      gain(GX, GY);
      if constexpr (!BWD) {
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          X[e] = f2_mul(X[e], f2_mul(GX[e], inv2));
          Y[e] = f2_mul(Y[e], f2_mul(GY[e], inv2));
          if (p.rot > 0) rotate2(X[e], Y[e], cs[e], sn[e]);
        }
      } else {
        uint64_t nx = 0;  // sum n x
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          if (p.rot > 0) rotate2(dX[e], dY[e], cs[e], sn[e]);
          nx = f2_fma(f2_mul(dX[e], GX[e]), X[e], f2_fma(f2_mul(dY[e], GY[e]), Y[e], nx));
        }
        const float mh = group_sum<L>(f2_hsum(nx)) * p.inv_d * inv;  // mean(n h)
        const uint64_t mh2 = f2_pack(-mh, -mh);
        const bool in = h < h1;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          X[e] = f2_mul(X[e], inv2);
          Y[e] = f2_mul(Y[e], inv2);
          if (in) {  // a head past the group's range holds zeros, and 0 / rho may be NaN (eps = 0)
            dgx[e] = f2_fma(dX[e], X[e], dgx[e]);
            dgy[e] = f2_fma(dY[e], Y[e], dgy[e]);
          }
          X[e] = f2_mul(f2_fma(X[e], mh2, f2_mul(dX[e], GX[e])), inv2);
          Y[e] = f2_mul(f2_fma(Y[e], mh2, f2_mul(dY[e], GY[e])), inv2);
        }
      }
      if (h < h1) {
        uint4 oa, ob;
        Pairs<T, INTER>::store(X, Y, &oa, &ob);
        if (ha) __stcs(reinterpret_cast<uint4*>(o + (long long)h * p.D) + va, oa);
        if (hb) __stcs(reinterpret_cast<uint4*>(o + (long long)h * p.D) + vb, ob);
      }
    }
  }
  if constexpr (BWD) {
    cp_async_wait<0>();
    __syncthreads();  // the ring is done with
    if (p.part) {  // groups in order: the sums do not depend on timing
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        float x[2], y[2];
        f2_unpack(dgx[e], x[0], x[1]);
        f2_unpack(dgy[e], y[0], y[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int pair = 2 * e + k;
          // the channels of pair `pair`, and whether the lane has its vector
          const bool second = INTER && pair >= NP;
          const int at = INTER ? (second ? vb : va) * V + 2 * (pair - (second ? NP : 0)) : va * V + pair;
          const int bt = INTER ? at + 1 : vb * V + pair;
          if (second ? hb : ha) smem[group * p.D + at] = x[k];
          if (INTER ? (second ? hb : ha) : hb) smem[group * p.D + bt] = y[k];
        }
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
    const float inv = rsqrtf(warp_sum(ss) * p.inv_d + p.eps);
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

// gain gradients: the CTAs' partial rows, summed in order (32 channels x 32
// interleaved runs of rows per CTA, whose loads do not wait for one another;
// blockIdx.y: q or k)
constexpr int kGainRuns = 32;
__global__ void __launch_bounds__(32 * kGainRuns) qk_dgain_kernel(const float* part, int blocks0, int blocks, int D, float* dq, float* dk) {
  __shared__ float sums[kGainRuns][33];
  const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, r = threadIdx.x >> 5;
  const int b0 = blockIdx.y ? blocks0 : 0, b1 = blockIdx.y ? blocks : blocks0;
  float* out = blockIdx.y ? dk : dq;
  pdl_wait();
  pdl_trigger();
  if (!out) return;
  float s = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int b = b0 + r; b < b1; b += kGainRuns) s += part[(long long)b * D + c];
  }
  sums[r][lane] = s;
  __syncthreads();
  // warp r: channel r of the CTA's
  s = warp_sum(sums[lane][r]);
  if (lane == 0 && blockIdx.x * 32 + r < D) out[blockIdx.x * 32 + r] = s;
}

template <typename T, int L, bool BWD>
cudaError_t launch_vec(const QkArgs& a, const QkParams& p, int grid) {
  const int smem = 8 * kQkThreads * 16;  // the ring; the gain gradients' sums need at most half of it
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
  return (int64_t)di.sm_count * kQkBwdBlocksPerSm * D * 4;
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
  // heads per group: few enough that every resident group has a unit, many
  // enough that its angles (about three rows' worth of work) are shared
  const long long cap = (long long)di.sm_count * (a.backward ? kQkBwdBlocksPerSm : kQkBlocksPerSm);
  const long long slots = cap * groups;
  auto plan = [&](int hc) {
    for (int i = 0; i < 2; ++i) {
      const int H = a.h[i].H;
      const int parts = H < 1 ? 1 : (H + hc - 1) / hc;
      p.hc[i] = H < 1 ? 1 : (H + parts - 1) / parts;  // as even as they come
      p.units[i] = H > 0 ? a.T * parts : 0;
    }
    const int most = p.hc[0] > p.hc[1] ? p.hc[0] : p.hc[1];
    return (p.units[0] + p.units[1] + slots - 1) / slots * (most + (a.rot > 0 ? 3 : 0));
  };
  int hc = 1;
  if (vec) {
    long long best = plan(1);
    for (int c = 2; c <= 32; ++c) {
      const long long cost = plan(c);
      if (cost < best) {
        best = cost;
        hc = c;
      }
    }
  }
  plan(hc);
  // CTAs to q and k by their share of the units, at least one each
  const long long need0 = (p.units[0] + groups - 1) / groups, need1 = (p.units[1] + groups - 1) / groups;
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
  return launch_kernel(qk_dgain_kernel, dim3((a.D + 31) / 32, 2), dim3(32 * kGainRuns), 0, a.stream, (const float*)p.part, p.blocks0, grid, a.D,
                       a.h[0].dgain, a.h[1].dgain);
}

}  // namespace attnres
