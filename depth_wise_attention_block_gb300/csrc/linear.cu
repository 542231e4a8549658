// Matrix product with bias, activation and residual in its epilogue, and its
// gradients: dispatch, and the CUDA-core kernel that takes any size, type,
// alignment and operand order.
//
//   z = x w^T + bias,  out = round(act(z) + residual)
//   dz = grad_out act'(z),  dx = dz w,  dw = dz^T x,  dbias = column sums of dz
#include <math.h>

#include "attnres.h"
#include "body.h"
#include "device_common.cuh"
#include "launch.h"
#include "linear_epilogue.cuh"

namespace attnres {

namespace {

constexpr int kGT = 64;        // rows and columns of a tile
constexpr int kGK = 16;        // depth of a stage
constexpr int kGThreads = 256;

// C(m, n) = sum_k A(m, k) B(n, k) with A(m, k) = a[m am + k ak], B(n, k) =
// b[n bn + k bk], one of each operand's strides 1 (AK: ak = 1, BK: bk = 1).
template <typename T>
struct AnyParams {
  const T* a;
  long long am, ak;
  const T* b;
  long long bn, bk;
  int M, N, K;
  LinearEpilogue epi;
};

template <typename T, bool AK, bool BK, int MODE>
__global__ void __launch_bounds__(kGThreads) gemm_any_kernel(const __grid_constant__ AnyParams<T> p) {
  __shared__ float as[kGK][kGT + 4], bs[kGK][kGT + 4];
  __shared__ float cols[kGThreads / 16][kGT];
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const long long m0 = (long long)blockIdx.y * kGT;
  const int n0 = blockIdx.x * kGT;
  pdl_wait();
  pdl_trigger();
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += kGK) {
#pragma unroll
    for (int r = 0; r < kGT * kGK / kGThreads; ++r) {
      const int i = r * kGThreads + tid;
      const int ka = AK ? i % kGK : i / kGT, ma = AK ? i / kGK : i % kGT;
      const int kb = BK ? i % kGK : i / kGT, nb = BK ? i / kGK : i % kGT;
      as[ka][ma] = m0 + ma < p.M && k0 + ka < p.K ? load_elem(p.a + (m0 + ma) * p.am + (long long)(k0 + ka) * p.ak) : 0.f;
      bs[kb][nb] = n0 + nb < p.N && k0 + kb < p.K ? load_elem(p.b + (long long)(n0 + nb) * p.bn + (long long)(k0 + kb) * p.bk) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kGK; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = as[k][ty * 4 + i];
        b[i] = bs[k][tx * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  float sum[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long m = m0 + ty * 4 + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (m < p.M && n < p.N) sum[j] += epilogue_one<T, MODE>(p.epi, m, n, acc[i][j]);
    }
  }
  if (MODE == kEpiDz && p.epi.part) {
#pragma unroll
    for (int j = 0; j < 4; ++j) cols[ty][tx * 4 + j] = sum[j];
    __syncthreads();
    if (tid < kGT && n0 + tid < p.N) {
      float s = 0.f;
      for (int r = 0; r < kGThreads / 16; ++r) s += cols[r][tid];
      p.epi.part[(long long)blockIdx.y * p.N + n0 + tid] = s;
    }
  }
}

template <typename T, bool AK, bool BK, int MODE>
cudaError_t launch_any(const T* a, long long am, long long ak, const T* b, long long bn, long long bk, long long M, int N,
                       int K, const LinearEpilogue& epi, cudaStream_t stream) {
  // tiles of 64 rows over blockIdx.y: at most 65535 of them per launch
  constexpr long long kRows = 65535LL * kGT;
  for (long long r0 = 0; r0 < M; r0 += kRows) {
    const long long m = M - r0 < kRows ? M - r0 : kRows;
    AnyParams<T> p{a + r0 * am, am, ak, b, bn, bk, (int)m, N, K, epi.rows_from<T>(r0, r0 / kGT, N)};
    const cudaError_t e = launch_kernel(gemm_any_kernel<T, AK, BK, MODE>, dim3((N + kGT - 1) / kGT, (unsigned)((m + kGT - 1) / kGT)),
                                        dim3(kGThreads), 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Column sums of a [M, N] row tensor, 64 rows per CTA, as partial rows.
template <typename T>
__global__ void __launch_bounds__(256) colsum_kernel(const T* g, long long ldg, int M, int N, float* part) {
  __shared__ float sums[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  for (long long y = blockIdx.y; y * kGT < M; y += gridDim.y) {
    float s = 0.f;
    if (c < N)
      for (int k = r; k < kGT && y * kGT + k < M; k += 8) s += load_elem(g + (y * kGT + k) * ldg + c);
    sums[r][threadIdx.x & 31] = s;
    __syncthreads();
    if (r == 0 && c < N) {
      for (int k = 1; k < 8; ++k) s += sums[k][threadIdx.x & 31];
      part[y * N + c] = s;
    }
    __syncthreads();
  }
}

// dbias[c] = sum of the partial rows, in order (8 interleaved runs)
__global__ void __launch_bounds__(256) rowsum_kernel(const float* part, int rows, int N, float* out) {
  __shared__ float sums[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  float s = 0.f;
  if (c < N)
    for (int k = r; k < rows; k += 8) s += part[(long long)k * N + c];
  sums[r][threadIdx.x & 31] = s;
  __syncthreads();
  if (r == 0 && c < N) {
    for (int k = 1; k < 8; ++k) s += sums[k][threadIdx.x & 31];
    out[c] = s;
  }
}

int64_t align_up(int64_t x) { return (x + 255) & ~int64_t(255); }

template <typename T>
cudaError_t linear_any(const LinearArgs& a) {
  LinearEpilogue epi{};
  epi.bias = a.bias;
  epi.res = a.residual;
  epi.ldr = a.ldr;
  epi.out = a.out;
  epi.ldo = a.ldo;
  epi.act = a.act;
  return launch_any<T, true, true, kEpiForward>(static_cast<const T*>(a.x), a.ldx, 1, static_cast<const T*>(a.w), a.K, 1,
                                                a.M, a.N, a.K, epi, a.stream);
}

// Workspace of the backward: dz [M, N] (with an activation), then the
// partial rows of the bias gradient (one per 32 tokens at most).
struct BwdLayout {
  int64_t dz, part, total;
};
BwdLayout bwd_layout(int64_t M, int N, int dtype, int act) {
  BwdLayout L;
  L.dz = act != ATTNRES_ACT_NONE ? align_up(M * N * (dtype == ATTNRES_BF16 ? 2 : 4)) : 0;
  L.part = align_up((M + 31) / 32 * N * 4);
  L.total = L.dz + L.part;
  return L;
}

template <typename T>
cudaError_t linear_backward_any(const LinearBwdArgs& a) {
  const T *x = static_cast<const T*>(a.x), *w = static_cast<const T*>(a.w), *g = static_cast<const T*>(a.grad_out);
  const BwdLayout L = bwd_layout(a.M, a.N, a.dtype, a.act);
  char* ws = static_cast<char*>(a.workspace);
  float* part = reinterpret_cast<float*>(ws + L.dz);
  const T* dz = g;
  long long ldz = a.ldg;
  cudaError_t e;
  const int tiles = (int)((a.M + kGT - 1) / kGT);
  if (a.act != ATTNRES_ACT_NONE) {
    LinearEpilogue epi{};
    epi.bias = a.bias;
    epi.res = a.grad_out;
    epi.ldr = a.ldg;
    epi.out = ws;
    epi.ldo = a.N;
    epi.act = a.act;
    epi.part = a.grad_bias ? part : nullptr;
    e = launch_any<T, true, true, kEpiDz>(x, a.ldx, 1, w, a.K, 1, a.M, a.N, a.K, epi, a.stream);
    if (e != cudaSuccess) return e;
    dz = reinterpret_cast<const T*>(ws);
    ldz = a.N;
  } else if (a.grad_bias) {
    e = launch_kernel(colsum_kernel<T>, dim3((a.N + 31) / 32, tiles < 65535 ? tiles : 65535), dim3(256), 0, a.stream, g,
                      (long long)a.ldg, (int)a.M, a.N, part);
    if (e != cudaSuccess) return e;
  }
  if (a.grad_bias) {
    e = launch_kernel(rowsum_kernel, dim3((a.N + 31) / 32), dim3(256), 0, a.stream, (const float*)part, tiles, a.N, a.grad_bias);
    if (e != cudaSuccess) return e;
  }
  if (a.grad_x) {
    LinearEpilogue epi{};
    epi.out = a.grad_x;
    epi.ldo = a.K;
    e = launch_any<T, true, false, kEpiForward>(dz, ldz, 1, w, 1, a.K, a.M, a.K, a.N, epi, a.stream);
    if (e != cudaSuccess) return e;
  }
  if (a.grad_w) {
    LinearEpilogue epi{};
    epi.out = a.grad_w;
    epi.ldo = a.K;
    e = launch_any<T, false, false, kEpiForward>(dz, 1, ldz, x, 1, a.ldx, a.N, a.K, (int)a.M, epi, a.stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

int64_t linear_workspace_bytes(int64_t M, int N, int K, int dtype) {
  (void)M, (void)N, (void)K, (void)dtype;
  return 0;
}

int64_t linear_backward_workspace_bytes(int64_t M, int N, int K, int dtype, int act) {
  (void)K;
  return bwd_layout(M, N, dtype, act).total;
}

cudaError_t launch_linear(const LinearArgs& a) {
  return a.dtype == ATTNRES_BF16 ? linear_any<bf16_t>(a) : linear_any<float>(a);
}

cudaError_t launch_linear_backward(const LinearBwdArgs& a) {
  if (a.M == 0) {
    cudaError_t e = cudaSuccess;
    if (a.grad_w) e = cudaMemsetAsync(a.grad_w, 0, (size_t)a.N * a.K * (a.dtype == ATTNRES_BF16 ? 2 : 4), a.stream);
    if (e == cudaSuccess && a.grad_bias) e = cudaMemsetAsync(a.grad_bias, 0, (size_t)a.N * 4, a.stream);
    return e;
  }
  return a.dtype == ATTNRES_BF16 ? linear_backward_any<bf16_t>(a) : linear_backward_any<float>(a);
}

}  // namespace attnres
