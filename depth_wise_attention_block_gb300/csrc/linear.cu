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
#include "linear_tc.h"

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

LinearEpilogue forward_epilogue(const LinearArgs& a) {
  LinearEpilogue epi{};
  epi.bias = a.bias;
  epi.res = a.residual;
  epi.ldr = a.ldr;
  epi.out = a.out;
  epi.ldo = a.ldo;
  epi.act = a.act;
  return epi;
}

template <typename T>
cudaError_t linear_any(const LinearArgs& a) {
  return launch_any<T, true, true, kEpiForward>(static_cast<const T*>(a.x), a.ldx, 1, static_cast<const T*>(a.w), a.K, 1,
                                                a.M, a.N, a.K, forward_epilogue(a), a.stream);
}

// Workspace of the backward: dz [M, N rounded up to 8] (with an activation),
// the partial rows of the bias gradient, and the operands' copies for the
// tensor cores.
int64_t dz_pitch(int N) { return ((int64_t)N + 7) / 8 * 8; }
struct BwdLayout {
  int64_t dz, part, x, w, g, total;
};
BwdLayout bwd_layout(int64_t M, int N, int K, int dtype, int act, LinearUneven u) {
  const bool bf16 = dtype == ATTNRES_BF16;
  const int np = bf16 ? 1 : 3;
  BwdLayout L;
  L.dz = act != ATTNRES_ACT_NONE ? align_up(M * dz_pitch(N) * (bf16 ? 2 : 4)) : 0;
  // rows of 64 tokens (CUDA cores, column sums), of 32 (wide tiles and
  // pairs), or the clusters' of up to 1024 tokens (16 per tile of 128)
  const int64_t rows = M <= 1024 ? (M + 127) / 128 * 16 : (M + 255) / 256 * 8;
  L.part = align_up(rows * N * 4);
  L.x = !bf16 || u.x ? tc_prep_bytes(M, K, np) : 0;
  L.w = !bf16 || u.w ? tc_prep_bytes(N, K, np) : 0;
  L.g = !bf16 || (act == ATTNRES_ACT_NONE && u.g) ? tc_prep_bytes(M, N, np) : 0;
  L.total = L.dz + L.part + L.x + L.w + L.g;
  return L;
}

template <typename T>
cudaError_t launch_colsum(const T* g, const LinearBwdArgs& a, float* part) {
  const int64_t tiles = (a.M + kGT - 1) / kGT;
  return launch_kernel(colsum_kernel<T>, dim3((a.N + 31) / 32, (unsigned)(tiles < 65535 ? tiles : 65535)), dim3(256), 0, a.stream, g,
                       (long long)a.ldg, (int)a.M, a.N, part);
}

cudaError_t launch_rowsum(const float* part, int rows, const LinearBwdArgs& a) {
  return launch_kernel(rowsum_kernel, dim3((a.N + 31) / 32), dim3(256), 0, a.stream, part, rows, a.N, a.grad_bias);
}

template <typename T>
cudaError_t linear_backward_any(const LinearBwdArgs& a) {
  const T *x = static_cast<const T*>(a.x), *w = static_cast<const T*>(a.w), *g = static_cast<const T*>(a.grad_out);
  const BwdLayout L = bwd_layout(a.M, a.N, a.K, a.dtype, a.act, {});
  char* ws = static_cast<char*>(a.workspace);
  float* part = reinterpret_cast<float*>(ws + L.dz);
  const T* dz = g;
  long long ldz = a.ldg;
  cudaError_t e;
  if (a.act != ATTNRES_ACT_NONE) {
    LinearEpilogue epi{};
    epi.bias = a.bias;
    epi.res = a.grad_out;
    epi.ldr = a.ldg;
    epi.out = ws;
    epi.ldo = dz_pitch(a.N);
    epi.act = a.act;
    epi.part = a.grad_bias ? part : nullptr;
    e = launch_any<T, true, true, kEpiDz>(x, a.ldx, 1, w, a.K, 1, a.M, a.N, a.K, epi, a.stream);
    if (e != cudaSuccess) return e;
    dz = reinterpret_cast<const T*>(ws);
    ldz = dz_pitch(a.N);
  } else if (a.grad_bias) {
    e = launch_colsum(g, a, part);
    if (e != cudaSuccess) return e;
  }
  if (a.grad_bias) {
    e = launch_rowsum(part, (int)((a.M + kGT - 1) / kGT), a);
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

// Short fp32 products below this many multiply-adds stay on the CUDA cores:
// the tensor cores need one more launch, which splits the operands (about 9 us
// together), a stage of 16 steps here about 1.2 us (100 x 100 x 100: 11 us).
constexpr int64_t kSmallFp32 = int64_t(1) << 24;

bool small_fp32(int64_t M, int N, int K, int dtype) { return dtype == ATTNRES_F32 && K <= 96 && M * N < kSmallFp32 / K; }

// Takes the next `bytes` of the workspace, or null where they do not fit.
struct Arena {
  char* at;
  int64_t left;
  void* take(int64_t bytes) {
    if (bytes > left) return nullptr;
    void* r = at;
    at += bytes;
    left -= bytes;
    return r;
  }
};

// On the tensor cores; *done says whether the workspace sufficed.
cudaError_t linear_tc(const LinearArgs& a, bool* done) {
  const bool bf16 = a.dtype == ATTNRES_BF16;
  const int np = bf16 ? 1 : 3;
  *done = false;
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const TcPlan plan = tc_plan(a.M, a.N, a.K, np, di.sm_count);
  TcOperand op[2] = {{a.x, a.ldx, a.M, a.K, false, nullptr}, {a.w, a.K, a.N, a.K, false, nullptr}};
  Arena ws{static_cast<char*>(a.workspace), a.workspace_bytes};
  TcOperand prep[2];
  int nprep = 0;
  for (TcOperand& o : op) {
    if ((bf16 && tc_rows_ok(o.ptr, o.ld)) || (plan.fused && &o == &op[1])) continue;
    o.prep = ws.take(tc_prep_bytes(o.rows, o.cols, np));
    if (!o.prep) return cudaSuccess;
    prep[nprep++] = o;
  }
  *done = true;
  if (nprep) e = launch_tc_prep(prep, nprep, np, a.stream);
  if (e != cudaSuccess) return e;
  return launch_tc_gemm(plan, op[0], op[1], a.M, a.N, a.K, np, kEpiForward, forward_epilogue(a), a.dev_err, a.stream);
}

// bf16: dz enters grad_x's and grad_w's products rounded once (their error in
// the 2-norm is then 0.0023, 0.0017 with an exact dz).  A second term would
// double both products, 85 of the 141 us of 2048 x 7168 x 2048, for less than
// one more rounding of the result.
cudaError_t linear_backward_tc(const LinearBwdArgs& a, bool* done) {
  const bool bf16 = a.dtype == ATTNRES_BF16, act = a.act != ATTNRES_ACT_NONE;
  const int np = bf16 ? 1 : 3;
  const BwdLayout L = bwd_layout(a.M, a.N, a.K, a.dtype, a.act, {});
  Arena ws{static_cast<char*>(a.workspace), a.workspace_bytes};
  void* dz_buf = L.dz ? ws.take(L.dz) : nullptr;
  float* part = static_cast<float*>(ws.take(L.part));
  TcOperand x{a.x, a.ldx, a.M, a.K, false, nullptr}, w{a.w, a.K, a.N, a.K, false, nullptr};
  TcOperand dz{act ? dz_buf : a.grad_out, act ? dz_pitch(a.N) : a.ldg, a.M, a.N, false, nullptr};
  *done = false;
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const TcPlan plan_z = tc_plan(a.M, a.N, a.K, np, di.sm_count), plan_x = tc_plan(a.M, a.K, a.N, np, di.sm_count);
  TcPlan plan_w = tc_plan(a.N, a.K, a.M, np, di.sm_count);
  // (dw's second operand is x, whose terms the first product needs anyway)
  if (plan_w.fused) plan_w = tc_plan_unfused(plan_w);
  const bool use_x = act || a.grad_w, use_dz = a.grad_x || a.grad_w;
  const bool use_w = (act && !plan_z.fused) || (a.grad_x && !plan_x.fused);
  TcOperand prep[3];
  int nprep = 0;
  for (TcOperand* o : {&x, &w, &dz}) {
    if (!(o == &x ? use_x : o == &w ? use_w : use_dz) || (bf16 && tc_rows_ok(o->ptr, o->ld))) continue;
    o->prep = ws.take(tc_prep_bytes(o->rows, o->cols, np));
    if (!o->prep) return cudaSuccess;
    if (o != &dz || !act) prep[nprep++] = *o;  // dz's copy comes after dz
  }
  *done = true;
  for (int i = 0; i < nprep && e == cudaSuccess; i += 2) e = launch_tc_prep(prep + i, nprep - i < 2 ? 1 : 2, np, a.stream);
  if (e != cudaSuccess) return e;
  int part_rows = 0;
  if (act) {
    LinearEpilogue epi{};
    epi.bias = a.bias;
    epi.res = a.grad_out;
    epi.ldr = a.ldg;
    epi.out = dz_buf;
    epi.ldo = dz_pitch(a.N);
    epi.act = a.act;
    epi.part = a.grad_bias ? part : nullptr;
    part_rows = plan_z.part_rows;
    e = launch_tc_gemm(plan_z, x, w, a.M, a.N, a.K, np, kEpiDz, epi, a.dev_err, a.stream);
    if (e == cudaSuccess && dz.prep) e = launch_tc_prep(&dz, 1, np, a.stream);
  } else if (a.grad_bias) {
    part_rows = (int)((a.M + kGT - 1) / kGT);
    e = bf16 ? launch_colsum(static_cast<const bf16_t*>(a.grad_out), a, part) : launch_colsum(static_cast<const float*>(a.grad_out), a, part);
  }
  if (e == cudaSuccess && a.grad_bias) e = launch_rowsum(part, part_rows, a);
  if (e == cudaSuccess && a.grad_x) {
    LinearEpilogue epi{};
    epi.out = a.grad_x;
    epi.ldo = a.K;
    TcOperand wt = w;
    wt.mn = true;
    e = launch_tc_gemm(plan_x, dz, wt, a.M, a.K, a.N, np, kEpiForward, epi, a.dev_err, a.stream);
  }
  if (e == cudaSuccess && a.grad_w) {
    LinearEpilogue epi{};
    epi.out = a.grad_w;
    epi.ldo = a.K;
    TcOperand zt = dz, xt = x;
    zt.mn = xt.mn = true;
    e = launch_tc_gemm(plan_w, zt, xt, a.N, a.K, a.M, np, kEpiForward, epi, a.dev_err, a.stream);
  }
  return e;
}

}  // namespace

LinearUneven linear_uneven(const void* x, int64_t ldx, const void* w, const void* g, int64_t ldg, int N, int K) {
  LinearUneven u = linear_uneven_sizes(N, K);
  u.x |= !tc_rows_ok(x, ldx);
  u.w |= !tc_rows_ok(w, K);
  u.g |= !tc_rows_ok(g, ldg);
  return u;
}

int64_t linear_workspace_bytes(int64_t M, int N, int K, int dtype, LinearUneven u) {
  if (small_fp32(M, N, K, dtype) || M == 0) return 0;
  if (dtype == ATTNRES_BF16) return (u.x ? tc_prep_bytes(M, K, 1) : 0) + (u.w ? tc_prep_bytes(N, K, 1) : 0);
  DeviceInfo di;
  // (without a device: enough for any plan)
  const bool fused = device_info(&di) == cudaSuccess && tc_plan(M, N, K, 3, di.sm_count).fused;
  return tc_prep_bytes(M, K, 3) + (fused ? 0 : tc_prep_bytes(N, K, 3));
}

int64_t linear_backward_workspace_bytes(int64_t M, int N, int K, int dtype, int act, LinearUneven u) {
  return bwd_layout(M, N, K, dtype, act, u).total;
}

cudaError_t launch_linear(const LinearArgs& a) {
  if (!small_fp32(a.M, a.N, a.K, a.dtype)) {
    bool done;
    const cudaError_t e = linear_tc(a, &done);
    if (done || e != cudaSuccess) return e;
  }
  return a.dtype == ATTNRES_BF16 ? linear_any<bf16_t>(a) : linear_any<float>(a);
}

cudaError_t launch_linear_backward(const LinearBwdArgs& a) {
  if (a.M == 0) {
    cudaError_t e = cudaSuccess;
    if (a.grad_w) e = cudaMemsetAsync(a.grad_w, 0, (size_t)a.N * a.K * (a.dtype == ATTNRES_BF16 ? 2 : 4), a.stream);
    if (e == cudaSuccess && a.grad_bias) e = cudaMemsetAsync(a.grad_bias, 0, (size_t)a.N * 4, a.stream);
    return e;
  }
  // its products run over each of the three sizes
  if (!small_fp32(a.M, a.N, a.K, a.dtype) || a.M > 96 || a.N > 96) {
    bool done;
    const cudaError_t e = linear_backward_tc(a, &done);
    if (done || e != cudaSuccess) return e;
  }
  return a.dtype == ATTNRES_BF16 ? linear_backward_any<bf16_t>(a) : linear_backward_any<float>(a);
}

}  // namespace attnres
