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

constexpr int kSC = 32;        // tokens per chunk
constexpr int kSD = 32;        // columns of c per CTA
constexpr int kSThreads = 256;
constexpr int kSMaxD = 256;

// rows of a and b in shared memory: one word of padding against bank conflicts
__host__ __device__ constexpr int scan_pitch(int Da) { return Da + 1; }
__host__ constexpr int scan_smem(int Da) {
  return (2 * kSC * scan_pitch(Da) + kSC * kSD + kSC * (kSC + 1) + Da * kSD + 2 * kSC) * 4;
}

template <typename T>
__global__ void __launch_bounds__(kSThreads) scan_any_kernel(const __grid_constant__ ScanArgs p) {
  extern __shared__ float sm[];
  const int Da = p.Da, Dc = p.Dc, pitch = scan_pitch(Da);
  float* a = sm;                        // [kSC][pitch]
  float* b = a + kSC * pitch;           // [kSC][pitch]
  float* c = b + kSC * pitch;           // [kSC][kSD]
  float* P = c + kSC * kSD;             // [kSC][kSC + 1]
  float* S = P + kSC * (kSC + 1);       // [Da][kSD]
  float* pw = S + Da * kSD;             // l^0 .. l^kSC
  const int tid = threadIdx.x;
  const int c0 = blockIdx.x * kSD, h = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const float g = p.log_decay[h];
  if (tid <= kSC) pw[tid] = expf(g * (float)tid);
  for (int n = blockIdx.z; n < p.N; n += gridDim.z) {
    const SeqRange sr = seq_range(p.cu, n, p.T);
    const long long st = ((long long)n * p.H + h) * Da * Dc;
    __syncthreads();
    for (int i = tid; i < Da * kSD; i += kSThreads) {
      const int da = i / kSD, dc = c0 + i % kSD;
      S[i] = p.s_in && dc < Dc ? p.s_in[st + p.state_at(da, dc)] : 0.f;
    }
    for (long long i0 = 0; i0 < sr.len; i0 += kSC) {
      const int len = (int)(sr.len - i0 < kSC ? sr.len - i0 : kSC);
      __syncthreads();
      for (int i = tid; i < kSC * Da; i += kSThreads) {
        const int r = i / Da, d = i % Da;
        const long long row = sr.row(i0 + r, p.reverse);
        a[r * pitch + d] = r < len ? load_elem(static_cast<const T*>(p.a) + row * p.as + (long long)h * Da + d) : 0.f;
        b[r * pitch + d] = r < len ? load_elem(static_cast<const T*>(p.b) + row * p.bs + (long long)h * Da + d) : 0.f;
      }
      for (int i = tid; i < kSC * kSD; i += kSThreads) {
        const int r = i / kSD, d = c0 + i % kSD;
        const long long row = sr.row(i0 + r, p.reverse);
        c[i] = r < len && d < Dc ? load_elem(static_cast<const T*>(p.c) + row * p.cs + (long long)h * Dc + d) : 0.f;
      }
      __syncthreads();
      {  // the triangle: rows i, i + 16; columns j, j + 16
        const int i = tid / 16, j = tid % 16;
        float s00 = 0.f, s01 = 0.f, s10 = 0.f, s11 = 0.f;
        for (int d = 0; d < Da; ++d) {
          const float x0 = a[i * pitch + d], x1 = a[(i + 16) * pitch + d];
          const float y0 = b[j * pitch + d], y1 = b[(j + 16) * pitch + d];
          s00 = fmaf(x0, y0, s00);
          s01 = fmaf(x0, y1, s01);
          s10 = fmaf(x1, y0, s10);
          s11 = fmaf(x1, y1, s11);
        }
        auto put = [&](int r, int q, float v) { P[r * (kSC + 1) + q] = q <= r ? v * pw[r - q] * p.p_scale : 0.f; };
        put(i, j, s00);
        put(i, j + 16, s01);
        put(i + 16, j, s10);
        put(i + 16, j + 16, s11);
      }
      __syncthreads();
      {  // out rows ty, ty + 8, ..; column tx
        const int tx = tid % 32, ty = tid / 32;
        float in[4] = {}, from[4] = {};
        for (int j = 0; j < kSC; ++j) {
          const float y = c[j * kSD + tx];
#pragma unroll
          for (int r = 0; r < 4; ++r) in[r] = fmaf(P[(ty + 8 * r) * (kSC + 1) + j], y, in[r]);
        }
        for (int d = 0; d < Da; ++d) {
          const float y = S[d * kSD + tx];
#pragma unroll
          for (int r = 0; r < 4; ++r) from[r] = fmaf(a[(ty + 8 * r) * pitch + d], y, from[r]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = ty + 8 * r;
          if (i < len && c0 + tx < Dc)
            store_elem(static_cast<T*>(p.out) + sr.row(i0 + i, p.reverse) * p.os + (long long)h * Dc + c0 + tx,
                       fmaf(from[r], pw[i + 1 - p.shift] * p.in_scale, in[r]));
        }
      }
      __syncthreads();
      {  // the state: rows ty, ty + 8, ..; column tx
        const int tx = tid % 32, ty = tid / 32;
        float u[kSMaxD / 8];
#pragma unroll
        for (int r = 0; r < kSMaxD / 8; ++r) u[r] = 0.f;
        for (int j = 0; j < len; ++j) {
          const float y = c[j * kSD + tx] * pw[len - 1 - j + p.shift] * p.up_scale;
#pragma unroll
          for (int r = 0; r < kSMaxD / 8; ++r)
            if (ty + 8 * r < Da) u[r] = fmaf(b[j * pitch + ty + 8 * r], y, u[r]);
        }
#pragma unroll
        for (int r = 0; r < kSMaxD / 8; ++r)
          if (ty + 8 * r < Da) S[(ty + 8 * r) * kSD + tx] = fmaf(S[(ty + 8 * r) * kSD + tx], pw[len], u[r]);
      }
    }
    __syncthreads();
    if (p.s_out)
      for (int i = tid; i < Da * kSD; i += kSThreads) {
        const int da = i / kSD, dc = c0 + i % kSD;
        if (dc < Dc) p.s_out[st + p.state_at(da, dc)] = S[i];
      }
  }
}

template <typename T>
cudaError_t launch_scan_any(const ScanArgs& s, cudaStream_t stream) {
  static SmemOptIn optin;
  const cudaError_t e = optin.ensure(reinterpret_cast<const void*>(scan_any_kernel<T>), scan_smem(kSMaxD));
  if (e != cudaSuccess) return e;
  return launch_kernel(scan_any_kernel<T>, dim3((s.Dc + kSD - 1) / kSD, s.H, s.N), dim3(kSThreads), scan_smem(s.Da), stream, s);
}

cudaError_t launch_scan(const ScanArgs& s, int dtype, cudaStream_t stream) {
  return dtype == ATTNRES_BF16 ? launch_scan_any<bf16_t>(s, stream) : launch_scan_any<float>(s, stream);
}

// ------------------------------------------------------------------ step --

// One token of one head: S = l S + k v^T, out = scale q S.  The state is read
// and written once: the bound is HBM (or, for few rows, one round trip to
// it).  A CTA takes all Dk rows of 8 vectors of columns, so that a row of
// threads reads whole 32-byte sectors and small batches still fill the GPU;
// its state loads are issued before it knows anything but its slot.
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

int64_t linear_attention_workspace_bytes(int64_t T, int H, int Dk, int Dv, int dtype, int N) {
  return scan_tc_dims(Dk, Dv, dtype) ? scan_tc_workspace(T, H, Dk, Dv, N) : 0;
}

cudaError_t launch_linear_attention(const LinAttnArgs& a) {
  ScanArgs s = scan_args(a, a.q, a.qs, a.k, a.ks, a.Dk, a.v, a.vs, a.Dv, a.out, a.os);
  s.s_in = a.s0;
  s.s_out = a.s1;
  s.p_scale = s.in_scale = a.scale;
  if (scan_tc_dims(a.Dk, a.Dv, a.dtype) && scan_tc_ok(s)) return launch_scan_tc(s, a.workspace, false, a.dev_err, a.stream);
  return launch_scan(s, a.dtype, a.stream);
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
  v.s_out = a.ds0;
  v.reverse = true;
  v.shift = 1;
  v.p_scale = v.up_scale = a.scale;
  // grad_initial_state may lie over grad_final_state: it is written after
  // the last read, by dv's scan or where the segments' states are joined
  if (scan_tc_dims(a.Dk, a.Dv, a.dtype) && scan_tc_ok(q) && scan_tc_ok(k) && scan_tc_ok(v)) {
    if (scan_tc_segmented(a.T, a.H, a.N)) {
      k.s_out = a.ds0;
      v.s_out = nullptr;
    }
    cudaError_t e = launch_scan_tc(q, a.workspace, false, a.dev_err, a.stream);
    if (e == cudaSuccess) e = launch_scan_tc(k, a.workspace, false, a.dev_err, a.stream);
    // the same reversed state, [Dk, Dv] in both
    if (e == cudaSuccess) e = launch_scan_tc(v, a.workspace, true, a.dev_err, a.stream);
    return e;
  }
  cudaError_t e = launch_scan(q, a.dtype, a.stream);
  if (e == cudaSuccess) e = launch_scan(k, a.dtype, a.stream);
  if (e == cudaSuccess) e = launch_scan(v, a.dtype, a.stream);
  return e;
}

cudaError_t launch_linear_attention_step(const LinAttnStepArgs& a) {
  const bool vec = a.Dv % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
  if (a.dtype == ATTNRES_BF16) return vec ? launch_step<bf16_t, 4>(a) : launch_step<bf16_t, 1>(a);
  return vec ? launch_step<float, 4>(a) : launch_step<float, 1>(a);
}

}  // namespace attnres
