// Causal linear attention with one decay per head: the scan on the CUDA
// cores (any head size, type and alignment), the recurrent step, and the
// dispatch of the forward and backward.
//
// The scan.  With U_i = l U_{i-1} + b_i c_i^T (l = exp(log_decay)) it gives
//   out_i = a_i U_i = l^{i+1} a_i U_{-1} + sum_{j <= i} l^{i-j} (a_i.b_j) c_j
// over a chunk of tokens: a decayed triangle of products inside the chunk,
// and one product with the state before it.  The forward is scan(q, k, v);
// the gradients are the same scan three times,
//   dq = scan(do, v, k) on S^T,
//   dk = scan(v, do, q) and dv = scan(k, q, do) from the last token to the first,
// where the reversed scans carry the state already decayed for the next
// token (W = l U), since the gradient that arrives at the final state does
// not decay before the last token: out_i = l^i a_i W + ..., and W ends as the
// initial state's gradient.
#include <math.h>

#include "attnres.h"
#include "body.h"
#include "device_common.cuh"
#include "launch.h"
#include "linear_attention.cuh"

namespace attnres {

namespace {

constexpr int kSC = 64;        // tokens per chunk
constexpr int kSMaxD = 256;  // of the step's rows
constexpr int kSPitchP = kSC + 4;

// The scan on the CUDA cores: a CTA takes a sequence and head, or the pieces
// of a range of the heads' chunks one after the other, and NG groups of
// 32 columns of c for each of W groups of 256 threads (STATE: the pieces'
// own states only, without scores and outputs; the combine kernel then leaves
// the state before each).  Every product runs from shared memory in register tiles,
// four rows by 2 NG columns per thread (16 x 16 threads), four steps of its
// contraction per 16-byte load of the rows, column pairs in packed fp32.
// Rows lie 16 bytes further apart than their length (no bank conflicts
// between a tile's rows).  The bound is the FMA rate, of which shared-memory
// loads leave about half (8192 tokens of 3 sequences, 24 heads of 128 in fp32:
// 875 us; 999 with one vector per thread on its way, 1157 with the sequences
// cut into lengths of one size).
__host__ __device__ constexpr int scan_rows(int Da) { return (Da + 3) / 4 * 4 + 4; }  // pitch of a and b
__host__ constexpr int scan_smem(int Da, int nc) {  // nc columns of c
  const int d = (Da + 63) / 64 * 64;  // the state's rows, whole tiles
  return (2 * kSC * scan_rows(Da) + kSC * nc + kSC * kSPitchP + d * nc + kSC + 8) * 4;
}

// rows 0 .. kSC - 1 (zero from len on) of `width` channels to dst, columns up
// to `cols` zero-filled; four vectors per thread are on their way at a time
template <typename T, int THREADS>
__device__ __forceinline__ void scan_load(float* dst, int pitch, const void* src, long long stride, int off, int width, int cols, int len,
                                          const SeqRange& sr, long long i0, bool reverse, bool vec) {
  constexpr int kBatch = 4;
  const T* p = static_cast<const T*>(src) + off + sr.row(i0, reverse) * stride;
  const long long step = reverse ? -stride : stride;
  const int q = cols / 4, total = kSC * q;
  for (int i = threadIdx.x; i < total; i += kBatch * THREADS) {
    float4 v[kBatch];
    int to[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int at_i = i + u * THREADS, r = at_i / q, c = (at_i - r * q) * 4;
      to[u] = at_i < total ? r * pitch + c : -1;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < len) {  // (rows past the tile are past len)
        const T* at = p + r * step + c;
        if (vec && c + 4 <= width) {
          if constexpr (sizeof(T) == 4) {
            v[u] = __ldg(reinterpret_cast<const float4*>(at));
          } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(at));
            v[u] = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
          }
        } else {
          if (c < width) v[u].x = load_elem(at);
          if (c + 1 < width) v[u].y = load_elem(at + 1);
          if (c + 2 < width) v[u].z = load_elem(at + 2);
          if (c + 3 < width) v[u].w = load_elem(at + 3);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (to[u] >= 0) *reinterpret_cast<float4*>(dst + to[u]) = v[u];
  }
}

// acc[r][s] += sum_k A[ty + 16 r][k] B[k][32 s + 2 tx ..], k < K (a multiple of 4), rows of B NC long
template <int NG, int NC>
__device__ __forceinline__ void scan_mma(uint64_t (&acc)[4][NG], const float* A, int pitch, const float* B, int K, int tx, int ty) {
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float4 a[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const float4*>(A + (ty + 16 * r) * pitch + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint64_t b[NG];
#pragma unroll
      for (int s = 0; s < NG; ++s) b[s] = *reinterpret_cast<const uint64_t*>(B + (k + e) * NC + 32 * s + 2 * tx);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = e == 0 ? a[r].x : e == 1 ? a[r].y : e == 2 ? a[r].z : a[r].w;
        const uint64_t xx = f2_pack(x, x);
#pragma unroll
        for (int s = 0; s < NG; ++s) acc[r][s] = f2_fma(xx, b[s], acc[r][s]);
      }
    }
  }
}

// Row i of P c in two columns over the rows that the mask leaves alone: where
// the product, in which a masked row counts as 0 times its values, met an
// infinity or a NaN.
__device__ __noinline__ uint64_t masked_pair(const float* P, const float* c, int pitch, int i) {
  float x = 0.f, y = 0.f;
  for (int j = 0; j <= i; ++j) {
    x = fmaf(P[j], c[j * pitch], x);
    y = fmaf(P[j], c[j * pitch + 1], y);
  }
  return f2_pack(x, y);
}

template <typename T, int NG, int W, bool STATE>
__global__ void __launch_bounds__(256 * W, 2 / W) scan_any_kernel(const __grid_constant__ ScanArgs p) {
  extern __shared__ __align__(16) float sm[];
  const int Da = p.Da, Dc = p.Dc, pitch = scan_rows(Da), K = pitch - 4, Dr = (Da + 63) / 64 * 64;
  constexpr int NC = 32 * NG * W, kThreads = 256 * W;
  float* a = sm;                        // [kSC][pitch]
  float* b = a + kSC * pitch;           // [kSC][pitch]
  float* c = b + kSC * pitch;           // [kSC][NC]
  float* P = c + kSC * NC;              // [kSC][kSPitchP]
  float* S = P + kSC * kSPitchP;        // [Dr][NC]
  float* pw = S + Dr * NC;              // l^0 .. l^kSC
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16 % 16, group = tid / 256;
  const int own = group * 32 * NG;  // the group's first column
  const int c0 = blockIdx.x * NC, wc = Dc - c0 < NC ? Dc - c0 : NC;
  pdl_wait();
  pdl_trigger();
  PieceWalk walk;
  if (p.parts > 0) walk = PieceWalk(p, blockIdx.y);
  Piece pc;
  for (bool first = true;; first = false) {
    if (p.parts > 0) {
      if (!walk.next(p, blockIdx.y, &pc)) return;
      if (STATE && pc.last) continue;  // its own state is part of the final one only, which the scan writes
    } else {
      if (!first) return;
      pc = whole_sequence(p, blockIdx.z, blockIdx.y);
    }
    const int h = pc.head;
    const float g = p.log_decay[h];
    __syncthreads();  // the piece before is done with
    if (tid <= kSC) pw[tid] = decay_pow(g, tid);
    const SeqRange sr{pc.first, pc.len};
    const long long of_seq = ((long long)pc.seq * p.H + h) * Da * Dc, of_piece = (long long)pc.id * Da * Dc;
    const float* before = STATE ? nullptr : pc.whole ? p.s_in : p.piece_state;
    if (before) before += pc.whole ? of_seq : of_piece;
    for (int i0 = tid; i0 < Dr * NC; i0 += 8 * kThreads) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kThreads, da = i / NC, dc = c0 + i % NC;
        v[u] = before && da < Da && dc < Dc ? before[p.state_at(da, dc)] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u * kThreads < Dr * NC) S[i0 + u * kThreads] = v[u];
    }
    for (long long i0 = 0; i0 < sr.len; i0 += kSC) {
      const int len = (int)(sr.len - i0 < kSC ? sr.len - i0 : kSC);
      __syncthreads();
      if constexpr (!STATE) scan_load<T, kThreads>(a, pitch, p.a, p.as, h * Da, Da, K, len, sr, i0, p.reverse, p.vec_a);
      scan_load<T, kThreads>(b, pitch, p.b, p.bs, h * Da, Da, K, len, sr, i0, p.reverse, p.vec_b);
      scan_load<T, kThreads>(c, NC, p.c, p.cs, h * Dc + c0, wc, NC, len, sr, i0, p.reverse, p.vec_c);
      __syncthreads();
      if constexpr (!STATE) {
        {  // the triangle: rows ty + 16 r of the group's, columns tx + 16 s, sums over even and odd channels packed
          constexpr int R = 4 / W;
          const float* ag = a + group * 16 * R * pitch;
          uint64_t acc[R][4];
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int s = 0; s < 4; ++s) acc[r][s] = 0;
#pragma unroll 2
          for (int k = 0; k < K; k += 4) {
            ulonglong2 x[R], y[4];
#pragma unroll
            for (int r = 0; r < R; ++r) x[r] = *reinterpret_cast<const ulonglong2*>(ag + (ty + 16 * r) * pitch + k);
#pragma unroll
            for (int s = 0; s < 4; ++s) y[s] = *reinterpret_cast<const ulonglong2*>(b + (tx + 16 * s) * pitch + k);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int s = 0; s < 4; ++s) acc[r][s] = f2_fma(x[r].y, y[s].y, f2_fma(x[r].x, y[s].x, acc[r][s]));
          }
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const int i = group * 16 * R + ty + 16 * r, j = tx + 16 * s;
              P[i * kSPitchP + j] = j <= i ? f2_hsum(acc[r][s]) * pw[i - j] * p.p_scale : 0.f;
            }
        }
        __syncthreads();
        {
          uint64_t in[4][NG], from[4][NG];
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int s = 0; s < NG; ++s) in[r][s] = from[r][s] = 0;
          scan_mma<NG, NC>(in, P, kSPitchP, c + own, (len + 3) / 4 * 4, tx, ty);
          scan_mma<NG, NC>(from, a, pitch, S + own, K, tx, ty);
          uint64_t sum = 0;  // 0, or NaN where a value is not finite
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int s = 0; s < NG; ++s) sum = f2_fma(in[r][s], 0ull, sum);
          if (f2_hsum(sum) != 0.f) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int s = 0; s < NG; ++s) in[r][s] = masked_pair(P + (ty + 16 * r) * kSPitchP, c + own + 32 * s + 2 * tx, NC, ty + 16 * r);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = ty + 16 * r;
            if (i < len) {
              const float coef = pw[i + 1 - p.shift] * p.in_scale;
              T* out = static_cast<T*>(p.out) + sr.row(i0 + i, p.reverse) * p.os + (long long)h * Dc + c0;
#pragma unroll
              for (int s = 0; s < NG; ++s) {
                float x0, x1, y0, y1;
                f2_unpack(in[r][s], x0, x1);
                f2_unpack(from[r][s], y0, y1);
                const int d = own + 32 * s + 2 * tx;
                if (d < wc) store_elem(out + d, fmaf(y0, coef, x0));
                if (d + 1 < wc) store_elem(out + d + 1, fmaf(y1, coef, x1));
              }
            }
          }
        }
        __syncthreads();
      }
      // the state: rows d0 + 4 ty .. + 3
      const uint64_t decay = f2_pack(pw[len], pw[len]), zero = f2_pack(0.f, 0.f);
      for (int d0 = 0; d0 < Dr; d0 += 64) {
        const int d = d0 + 4 * ty;
        if (d >= K) continue;
        uint64_t u[4][NG];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int s = 0; s < NG; ++s) u[r][s] = zero;
#pragma unroll 4
        for (int j = 0; j < len; ++j) {
          const float f = pw[len - 1 - j + p.shift] * p.up_scale;
          const float4 x = *reinterpret_cast<const float4*>(b + j * pitch + d);
          const uint64_t w[4] = {f2_pack(x.x * f, x.x * f), f2_pack(x.y * f, x.y * f), f2_pack(x.z * f, x.z * f), f2_pack(x.w * f, x.w * f)};
#pragma unroll
          for (int s = 0; s < NG; ++s) {
            const uint64_t y = *reinterpret_cast<const uint64_t*>(c + j * NC + own + 32 * s + 2 * tx);
#pragma unroll
            for (int r = 0; r < 4; ++r) u[r][s] = f2_fma(w[r], y, u[r][s]);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int s = 0; s < NG; ++s) {
            uint64_t* at = reinterpret_cast<uint64_t*>(S + (d + r) * NC + own + 32 * s + 2 * tx);
            *at = f2_fma(*at, decay, u[r][s]);
          }
      }
    }
    __syncthreads();
    float* to = STATE ? p.piece_state + of_piece : p.s_out && pc.last && !p.keep_final ? p.s_out + of_seq : nullptr;
    if (to)
      for (int i = tid; i < Da * NC; i += kThreads) {
        const int da = i / NC, dc = c0 + i % NC;
        if (dc < Dc) to[p.state_at(da, dc)] = S[i];
      }
  }
}

// Columns per CTA: all of them (every CTA of a head forms the chunk's scores
// again) up to 128, in one group of 32, 64 or 96, or two of 64; fewer where
// shared memory does not hold them.
int scan_columns(int Da, int Dc, int smem_max) {
  int nc = Dc > 96 ? 128 : (Dc + 31) / 32 * 32;
  while (nc > 32 && scan_smem(Da, nc) > smem_max) nc -= 32;
  return nc;
}

template <typename T, int NG, int W, bool STATE>
cudaError_t launch_scan_any(const ScanArgs& s, cudaStream_t stream) {
  static SmemOptIn optin;
  constexpr int nc = 32 * NG * W;
  const auto kern = scan_any_kernel<T, NG, W, STATE>;
  const cudaError_t e = optin.ensure(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return e;
  const dim3 grid((s.Dc + nc - 1) / nc, s.parts > 0 ? s.parts * s.gang : s.H, s.parts > 0 ? 1 : s.N);
  return launch_kernel(kern, grid, dim3(256 * W), scan_smem(s.Da, nc), stream, s);
}

template <typename T, bool STATE>
cudaError_t launch_scan_groups(const ScanArgs& s, int nc, cudaStream_t stream) {
  switch (nc) {
    case 32: return launch_scan_any<T, 1, 1, STATE>(s, stream);
    case 64: return launch_scan_any<T, 2, 1, STATE>(s, stream);
    case 96: return launch_scan_any<T, 3, 1, STATE>(s, stream);
    default: return launch_scan_any<T, 2, 2, STATE>(s, stream);
  }
}

// Ranges on the CUDA cores: a chunk's products at the 110 FMA per ns that an
// SM gives them, shared by the CTAs of an SM.
CutRule scan_any_rule(int Da, int Dc, const DeviceInfo& di) {
  const int nc = scan_columns(Da, Dc, di.max_smem_optin);
  const int per_sm = 2 * scan_smem(Da, nc) + 2048 <= di.max_smem_optin ? 2 : 1;
  const double chunk_ns = per_sm * (double)kSC * (kSC * (Da + nc) + 2 * Da * nc) / 110;
  return {kSC, (Dc + nc - 1) / nc, per_sm * di.sm_count, 0.4, chunk_ns};
}
Cut scan_any_cut(int64_t T, int H, int Da, int Dc, int N, const DeviceInfo& di) {
  return choose_cut(T, H, Da, Dc, N, scan_any_rule(Da, Dc, di));
}

template <typename T>
cudaError_t launch_scan_type(const ScanArgs& in, void* workspace, int64_t workspace_bytes, ScanReady ready, cudaStream_t stream) {
  ScanArgs s = in;
  auto vec = [](const void* p, long long stride, int D) {
    return (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(T) - 1)) == 0 && stride % 4 == 0 && D % 4 == 0;
  };
  s.vec_a = vec(s.a, s.as, s.Da);
  s.vec_b = vec(s.b, s.bs, s.Da);
  s.vec_c = vec(s.c, s.cs, s.Dc);
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  s.chunk = kSC;
  s.final_in_scan = true;
  // one cut for both orders of the two head sizes: the gradients' scans share states
  const Cut cut = scan_any_cut(s.T, s.H, s.transposed ? s.Dc : s.Da, s.transposed ? s.Da : s.Dc, s.N, di);
  const PieceLayout L = piece_layout(s.H, s.Da, s.Dc, s.N, cut);
  s.gang = cut.gang;
  s.parts = L.total > workspace_bytes ? 0 : cut.parts;  // tensors that the tensor cores would have taken but for their alignment
  const int nc = scan_columns(s.Da, s.Dc, di.max_smem_optin);
  if (s.parts > 0) piece_place(s, L, workspace);
  if (s.parts > 0 && ready < kStates) {
    if (ready < kTables) e = launch_piece_plan(s, stream);
    if (e == cudaSuccess) e = launch_scan_groups<T, true>(s, nc, stream);
    if (e == cudaSuccess) e = launch_piece_combine(s, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_scan_groups<T, false>(s, nc, stream);
}

// The tables of a ragged batch.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) la_plan_kernel(const __grid_constant__ ScanArgs p) {
  const int N = p.N, chunk = p.chunk;
  const int32_t* cu = p.cu;
  const long long T = p.T;
  int* first = const_cast<int*>(p.first);
  // 64 bits: offsets that decrease can ask for any number of chunks
  __shared__ long long sums[32], carry;
  __shared__ int near[kPlanThreads + 1];  // first, of up to 1024 sequences
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long cap = (T + chunk - 1) / chunk + N;  // what offsets that do not decrease stay below
  pdl_wait();
  pdl_trigger();
  if (tid == 0) carry = 0;
  for (int n0 = 0; n0 < N; n0 += kPlanThreads) {
    const int n = n0 + tid;
    const long long cnt = n < N ? (seq_range(cu, n, T).len + chunk - 1) / chunk : 0;
    long long x = cnt;
    for (int o = 1; o < 32; o *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
      long long y = sums[lane];
      for (int o = 1; o < 32; o *= 2) {
        const long long z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      sums[lane] = y;
    }
    __syncthreads();
    const long long at = carry + (warp ? sums[warp - 1] : 0) + x - cnt;
    if (n < N) first[n] = near[tid] = (int)(at < cap ? at : cap);
    const long long total = sums[31];
    __syncthreads();
    if (tid == 0) carry += total;
    __syncthreads();
  }
  if (tid == 0) first[N] = near[N < kPlanThreads ? N : kPlanThreads] = (int)(carry < cap ? carry : cap);
  __syncthreads();
  const Ranges r(p);
  const int* const from = N <= kPlanThreads ? near : first;
  for (int i = tid; i <= p.parts; i += kPlanThreads) {
    const int u = r.begin(i), gang = r.per_head > 0 ? u / r.per_head : 0;
    const_cast<int4*>(p.starts)[i] = make_int4(u, gang, sequence_of(from, N, u - gang * r.per_head), r.per_head);
  }
}

// Per sequence and head: the state before each piece, from the pieces' own
// states, in place and in order, and the final state.  VEC floats per thread
// of [H][Da Dc].
template <int VEC>
__global__ void __launch_bounds__(256) la_combine_kernel(const __grid_constant__ ScanArgs p, int per_head) {
  const long long e = (blockIdx.x * 256LL + threadIdx.x) * VEC;
  const int n = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const long long all = (long long)p.H * per_head;
  if (e >= all) return;
  const int h = (int)(e / per_head);
  const float g = __ldg(p.log_decay + h);
  const Ranges r(p);
  // the sequence's chunks of this head, and the ranges that have them
  const int gang = h / p.gang, at_gang = gang * r.per_head;
  const int u0 = at_gang + (p.first ? p.first[n] : 0), u1 = at_gang + (p.first ? p.first[n + 1] : r.per_head);
  const int i0 = u0 < u1 ? r.owner(u0) : 0, i1 = u0 < u1 ? r.owner(u1 - 1) + 1 : 0;
  const long long step = (long long)p.gang * per_head;  // from a piece's state to the next one's
  if (p.final_in_scan && i1 - i0 == 1) return;  // a whole sequence
  float* const at0 = p.piece_state + ((long long)gang * p.N + n) * step + (h - gang * p.gang) * (long long)per_head + (e - (long long)h * per_head);
  float w[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) w[k] = p.s_in ? p.s_in[n * all + e + k] : 0.f;
  // several pieces' states are loaded before the first of them is replaced
  constexpr int kAhead = VEC == 4 ? 4 : 16;
  for (int i = i0; i < i1; i += kAhead) {
    float u[kAhead][VEC], d[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      d[j] = 1.f;
#pragma unroll
      for (int k = 0; k < VEC; ++k) u[j][k] = 0.f;
      if (i + j < i1) {
        const int b = r.begin(i + j) > u0 ? r.begin(i + j) : u0, f = r.begin(i + j + 1) < u1 ? r.begin(i + j + 1) : u1;
        const Piece pc = cut_piece(p, n, h, b - u0, f - b);
        d[j] = decay_pow(g, pc.len);
        const float* at = at0 + (i + j) * step;
        if (!pc.last || (p.s_out && !p.final_in_scan)) {
          if constexpr (VEC == 4) {
            const float4 x = *reinterpret_cast<const float4*>(at);
            u[j][0] = x.x, u[j][1] = x.y, u[j][2] = x.z, u[j][3] = x.w;
          } else {
            u[j][0] = *at;
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j < i1) {
        float* at = at0 + (i + j) * step;
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(at) = make_float4(w[0], w[1], w[2], w[3]);
        else
          *at = w[0];
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) w[k] = fmaf(w[k], d[j], u[j][k]);
    }
  }
  if (p.s_out && (!p.final_in_scan || i0 == i1)) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) p.s_out[n * all + e + k] = w[k];
  }
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// ------------------------------------------------------------------ step --

// One token of one head: S = l S + k v^T, out = scale q S.  The state is read
// and written once: the bound is HBM (or, for few rows, one round trip to
// it).  A CTA takes all Dk rows of 8 vectors of columns, so that a row of
// threads reads whole 32-byte sectors and small batches still fill the GPU;
// its state loads are issued before it knows anything but its slot.  64 rows x
// 56 heads of 128 x 128: 72.5 us (6.5 TB/s); one row: 2.8 us.
constexpr int kStThreads = 256;
constexpr int kStX = 8;                    // vectors of columns per CTA
constexpr int kStY = kStThreads / kStX;    // rows of the state in flight

template <int VEC>
struct StVec;
template <>
struct StVec<4> {
  float4 v;
  __device__ void load(const float* p) { v = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ void store(float* p) const { __stcs(reinterpret_cast<float4*>(p), v); }
  __device__ float& operator[](int i) { return reinterpret_cast<float*>(&v)[i]; }
};
template <>
struct StVec<1> {
  float v;
  __device__ void load(const float* p) { v = __ldcs(p); }
  __device__ void store(float* p) const { __stcs(p, v); }
  __device__ float& operator[](int) { return v; }
};

template <typename T, int VEC, int ROWS>  // ROWS: Dk / kStY, rounded up
__global__ void __launch_bounds__(kStThreads) step_kernel(const __grid_constant__ LinAttnStepArgs p) {
  __shared__ float sq[kSMaxD], sk[kSMaxD];
  __shared__ float red[kStThreads / 32][kStX * VEC];
  __shared__ int next_row;
  const int tid = threadIdx.x, x = tid % kStX, y = tid / kStX;
  const int h = blockIdx.x;
  const int col = (blockIdx.y * kStX + x) * VEC;
  int row = blockIdx.z;
  const bool in = col < p.Dv;
  pdl_wait();
  pdl_trigger();
  const int slot = p.slots ? __ldg(p.slots + row) : row;
  if (slot < 0 || slot >= p.num_slots) return;  // a padding row
  float* st = p.state + (((long long)slot * p.H + h) * p.Dk) * p.Dv + col;
  StVec<VEC> S[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    if (in && y + r * kStY < p.Dk) S[r].load(st + (long long)(y + r * kStY) * p.Dv);
  const float l = expf(p.log_decay[h]);
  if (p.slots) {  // rows of one slot belong to the CTA of the first of them
    bool later = false;
    for (int i = tid; i < row; i += kStThreads) later |= __ldg(p.slots + i) == slot;
    if (__syncthreads_or(later)) return;
  }
  for (;;) {
    if (tid == 0) next_row = p.B;
    for (int d = tid; d < p.Dk; d += kStThreads) {
      sq[d] = load_elem(static_cast<const T*>(p.q) + row * p.qs + (long long)h * p.Dk + d);
      sk[d] = load_elem(static_cast<const T*>(p.k) + row * p.ks + (long long)h * p.Dk + d);
    }
    float v[VEC], o[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      v[e] = in ? load_elem(static_cast<const T*>(p.v) + row * p.vs + (long long)h * p.Dv + col + e) : 0.f;
      o[e] = 0.f;
    }
    __syncthreads();
    if (p.slots)
      for (int i = row + 1 + tid; i < p.B; i += kStThreads)
        if (__ldg(p.slots + i) == slot) {
          atomicMin(&next_row, i);
          break;
        }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int d = y + r * kStY;
      if (in && d < p.Dk) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          S[r][e] = fmaf(S[r][e], l, sk[d] * v[e]);
          o[e] = fmaf(sq[d], S[r][e], o[e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      o[e] += __shfl_xor_sync(0xffffffffu, o[e], 8);
      o[e] += __shfl_xor_sync(0xffffffffu, o[e], 16);
      if (tid % 32 < kStX) red[tid / 32][x * VEC + e] = o[e];
    }
    __syncthreads();
    if (tid < kStX * VEC) {
      const int c = blockIdx.y * kStX * VEC + tid;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kStThreads / 32; ++w) s += red[w][tid];
      if (c < p.Dv) store_elem(static_cast<T*>(p.out) + row * p.os + (long long)h * p.Dv + c, p.scale * s);
    }
    row = next_row;
    if (row >= p.B) break;
    __syncthreads();  // every thread has read next_row and red
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    if (in && y + r * kStY < p.Dk) S[r].store(st + (long long)(y + r * kStY) * p.Dv);
}

template <typename T, int VEC>
cudaError_t launch_step(const LinAttnStepArgs& a) {
  const dim3 grid(a.H, (a.Dv + kStX * VEC - 1) / (kStX * VEC), a.B);
  const int rows = (a.Dk + kStY - 1) / kStY;
  if (rows <= 2) return launch_kernel(step_kernel<T, VEC, 2>, grid, dim3(kStThreads), 0, a.stream, a);
  if (rows <= 4) return launch_kernel(step_kernel<T, VEC, 4>, grid, dim3(kStThreads), 0, a.stream, a);
  return launch_kernel(step_kernel<T, VEC, 8>, grid, dim3(kStThreads), 0, a.stream, a);
}

// scan(a, b, c) over a's and b's Da channels and c's Dc
ScanArgs scan_args(const LinAttnArgs& a, const void* x, int64_t xs, const void* y, int64_t ys, int Da, const void* z,
                   int64_t zs, int Dc, void* out, int64_t os) {
  ScanArgs s{};
  s.a = x;
  s.as = xs;
  s.b = y;
  s.bs = ys;
  s.c = z;
  s.cs = zs;
  s.out = out;
  s.os = os;
  s.Da = Da;
  s.Dc = Dc;
  s.T = a.T;
  s.H = a.H;
  s.N = a.N;
  s.cu = a.cu;
  s.log_decay = a.log_decay;
  s.p_scale = s.in_scale = s.up_scale = 1.f;
  return s;
}

}  // namespace

PieceLayout piece_layout(int H, int Da, int Dc, int N, Cut cut) {
  PieceLayout L{};
  if (cut.parts == 0) return L;
  L.first = round_up((N + 1) * 4LL, 256);
  L.starts = round_up((cut.parts + 1) * (int64_t)sizeof(int4), 256);
  L.states = round_up(((int64_t)cut.parts * cut.gang + (int64_t)H * N) * Da * Dc * 4, 256);
  L.total = L.first + L.starts + L.states;
  return L;
}

void piece_place(ScanArgs& s, const PieceLayout& L, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  s.first = s.cu ? reinterpret_cast<const int*>(ws) : nullptr;
  s.starts = reinterpret_cast<const int4*>(ws + L.first);
  s.piece_state = reinterpret_cast<float*>(ws + L.first + L.starts);
}

Cut choose_cut(int64_t T, int H, int Da, int Dc, int N, const CutRule& r) {
  const int64_t chunks = round_up(T, r.chunk) / r.chunk, units = H * (chunks + N);
  const int groups = r.groups, slots = r.slots;
  if (T == 0 || units >= INT32_MAX / 2) return {0, 1};  // a chunk's index is an int
  const double even = (double)groups * (double)units / slots;  // chunks per slot if all were equal
  // Neighbouring heads lie side by side in memory: the largest gang, unless a
  // smaller one divides the work better (8192 tokens of 5 sequences, 32 heads
  // of 128, backward: 334 us in gangs of 8, 344 in gangs of 1, before the state entered
  // its products as two terms).
  Cut cut{0, 1};
  double best = 1e300;
  for (int gang = 8; gang >= 1; --gang) {
    if (H % gang || gang > slots / groups) continue;
    const int64_t gangs = H / gang;
    for (int least = 1; least <= 4; ++least) {  // chunks of a range
      int64_t parts = slots / groups / gang;
      if (parts > gangs * chunks / least) parts = gangs * chunks / least;
      if (parts == 0) break;
      const double pieces = (double)(parts + gangs * N);  // of a gang's head
      const double bytes = pieces * gang * Da * Dc * 16;  // written, read, replaced and read
      const double join = bytes / 6500 + 250. * (double)parts / (double)gangs + 12000;
      const double cost = ((double)(gangs * chunks) + pieces) / (double)parts * (1 + r.extra) + join / r.chunk_ns;
      if (cost < 0.95 * best) {
        best = cost;
        cut = {(int)parts, gang};
      }
    }
  }
  const double whole = (double)(chunks > even ? chunks : even) + 2;  // every sequence in one piece
  if (best >= whole) cut.parts = 0;
  return cut;
}

// A cut's cost is at least even (1 + extra) + (1 + extra) + join (no more
// ranges than CTAs at once) and at least (2 + N / chunks) (1 + extra) + join
// (no more than chunks), with join no less than the sequences' own states and
// the launches; it has to be below chunks + 2 (where `even` is the larger part
// of `whole`, the first bound alone exceeds it).  Both leave a largest N, which
// grows with T; more sequences than that are never cut.
int64_t piece_bytes(int64_t T, int H, int Da, int Dc, int N, const CutRule& r) {
  const int64_t chunks = round_up(T, r.chunk) / r.chunk;
  if (chunks == 0) return 0;
  const double m = (double)chunks, x = r.extra, fixed = 12000 / r.chunk_ns, state = (double)H * Da * Dc * 16 / 6500 / r.chunk_ns;
  const double share = (double)r.groups * H / r.slots * (1 + x);  // of `even` (1 + extra), per chunk
  const double n1 = (m * (1 - share) + 1 - x - fixed) / (share + state), n2 = (m - 2 * x - fixed) / ((1 + x) / m + state);
  const double most = n1 < n2 ? n1 : n2;
  if (most <= 1) return 0;
  const Cut widest{r.slots / r.groups, 1};
  return piece_layout(H, Da, Dc, most < N ? (int)most : N, widest).total;
}

cudaError_t launch_piece_plan(const ScanArgs& s, cudaStream_t stream) {
  if (!s.first) return cudaSuccess;
  return launch_kernel(la_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, s);
}

cudaError_t launch_piece_combine(const ScanArgs& s, cudaStream_t stream) {
  const int per_head = s.Da * s.Dc;
  const int64_t all = (int64_t)s.H * per_head;
  // four values per thread where that gives every SM a CTA; else one, with
  // more of a sequence's pieces at a time (8192 tokens of 4 heads of 128 in
  // fp32: the whole call 190 us with four, 182 with one)
  DeviceInfo di;
  const cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  if (per_head % 4 == 0 && all * s.N >= 4 * 256 * (int64_t)di.sm_count)
    return launch_kernel(la_combine_kernel<4>, dim3((unsigned)((all / 4 + 255) / 256), s.N), dim3(256), 0, stream, s, per_head);
  return launch_kernel(la_combine_kernel<1>, dim3((unsigned)((all + 255) / 256), s.N), dim3(256), 0, stream, s, per_head);
}

int64_t linear_attention_workspace_bytes(int64_t T, int H, int Dk, int Dv, int dtype, int N) {
  if (scan_tc_dims(Dk, Dv, dtype)) return scan_tc_workspace(T, H, Dk, Dv, N);
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return -1;
  return piece_bytes(T, H, Dk, Dv, N, scan_any_rule(Dk, Dv, di));
}

namespace {

cudaError_t launch_scan(const LinAttnArgs& a, const ScanArgs& s, bool tc, ScanReady ready) {
  if (tc) return launch_scan_tc(s, a.workspace, a.workspace_bytes, ready, a.dev_err, a.stream);
  return a.dtype == ATTNRES_BF16 ? launch_scan_type<bf16_t>(s, a.workspace, a.workspace_bytes, ready, a.stream)
                                 : launch_scan_type<float>(s, a.workspace, a.workspace_bytes, ready, a.stream);
}

// whether the scan runs in pieces on the CUDA cores
bool scan_any_in_pieces(const LinAttnArgs& a) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return false;
  const Cut cut = scan_any_cut(a.T, a.H, a.Dk, a.Dv, a.N, di);
  return cut.parts > 0 && piece_layout(a.H, a.Dk, a.Dv, a.N, cut).total <= a.workspace_bytes;
}

}  // namespace

cudaError_t launch_linear_attention(const LinAttnArgs& a) {
  ScanArgs s = scan_args(a, a.q, a.qs, a.k, a.ks, a.Dk, a.v, a.vs, a.Dv, a.out, a.os);
  s.s_in = a.s0;
  s.s_out = a.s1;
  s.p_scale = s.in_scale = a.scale;
  return launch_scan(a, s, scan_tc_dims(a.Dk, a.Dv, a.dtype) && scan_tc_ok(s), kNothing);
}

cudaError_t launch_linear_attention_backward(const LinAttnArgs& a) {
  const int64_t rk = (int64_t)a.H * a.Dk, rv = (int64_t)a.H * a.Dv;
  ScanArgs q = scan_args(a, a.dout, a.dos, a.v, a.vs, a.Dv, a.k, a.ks, a.Dk, a.dq, rk);
  q.s_in = a.s0;
  q.transposed = true;
  q.p_scale = q.in_scale = a.scale;
  ScanArgs k = scan_args(a, a.v, a.vs, a.dout, a.dos, a.Dv, a.q, a.qs, a.Dk, a.dk, rk);
  k.s_in = a.ds1;
  k.transposed = true;
  k.reverse = true;
  k.shift = 1;
  k.p_scale = k.up_scale = a.scale;
  ScanArgs v = scan_args(a, a.k, a.ks, a.q, a.qs, a.Dk, a.dout, a.dos, a.Dv, a.dv, rv);
  v.s_in = a.ds1;
  v.reverse = true;
  v.shift = 1;
  v.p_scale = v.up_scale = a.scale;
  const bool tc = scan_tc_dims(a.Dk, a.Dv, a.dtype) && scan_tc_ok(q) && scan_tc_ok(k) && scan_tc_ok(v);
  // dk and dv carry the same reversed state ([Dk, Dv] in memory for both): in
  // pieces it is formed once.  grad_initial_state may lie over
  // grad_final_state, so it is written after the last read of that: where
  // the pieces' states are joined, or by dv's scan (on the CUDA cores: by
  // both, the former for empty sequences).  It comes with dv, whose scan runs
  // for it alone where there are no rows.
  const bool cut = tc ? scan_tc_in_pieces(a.T, a.H, a.Dk, a.Dv, a.N) : scan_any_in_pieces(a);
  if (cut && a.dk) k.s_out = a.ds0;
  if (!cut || !tc || !a.dk) v.s_out = a.ds0;
  k.keep_final = true;
  cudaError_t e = cudaSuccess;
  if (a.dq) e = launch_scan(a, q, tc, kNothing);
  if (a.dk && e == cudaSuccess) e = launch_scan(a, k, tc, a.dq ? kTables : kNothing);
  if ((a.dv || a.ds0) && e == cudaSuccess) e = launch_scan(a, v, tc, a.dk ? kStates : a.dq ? kTables : kNothing);
  return e;
}

cudaError_t launch_linear_attention_step(const LinAttnStepArgs& a) {
  const bool vec = a.Dv % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
  if (a.dtype == ATTNRES_BF16) return vec ? launch_step<bf16_t, 4>(a) : launch_step<bf16_t, 1>(a);
  return vec ? launch_step<float, 4>(a) : launch_step<float, 1>(a);
}

}  // namespace attnres
