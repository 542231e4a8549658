// Host-side launch interface between the C ABI (body_api.cu) and the kernels
// of a layer body: matrix products with a fused epilogue, head norms with
// rotation, and linear attention with a decay per head.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace attnres {

// ---------------------------------------------------------- linear -------

struct LinearArgs {
  const void* x;
  int64_t ldx;
  const void* w;
  const float* bias;
  const void* residual;
  int64_t ldr;
  void* out;
  int64_t ldo;
  int64_t M;
  int N, K;
  int dtype;
  int act;
  void* workspace;
  int64_t workspace_bytes;
  int* dev_err;
  cudaStream_t stream;
};
cudaError_t launch_linear(const LinearArgs& a);
// bf16 operands that TMA does not take as they are (rows off the 16-byte
// boundaries), whose copies the workspace has room for.
struct LinearUneven {
  bool x, w, g;
};
// of contiguous aligned operands: by the length of a row
inline LinearUneven linear_uneven_sizes(int N, int K) { return {K % 8 != 0, K % 8 != 0, N % 8 != 0}; }
// of these ones (and no fewer than by the sizes)
LinearUneven linear_uneven(const void* x, int64_t ldx, const void* w, const void* g, int64_t ldg, int N, int K);
int64_t linear_workspace_bytes(int64_t M, int N, int K, int dtype, LinearUneven u);

struct LinearBwdArgs {
  const void* x;
  int64_t ldx;
  const void* w;
  const float* bias;
  const void* grad_out;
  int64_t ldg;
  void* grad_x;
  void* grad_w;
  float* grad_bias;
  int64_t M;
  int N, K;
  int dtype;
  int act;
  void* workspace;
  int64_t workspace_bytes;
  int* dev_err;
  cudaStream_t stream;
};
cudaError_t launch_linear_backward(const LinearBwdArgs& a);
int64_t linear_backward_workspace_bytes(int64_t M, int N, int K, int dtype, int act, LinearUneven u);

// ----------------------------------------------------- qk norm + rope ----

// One of q and k.
struct QkHead {
  const void* x;
  int64_t xs;  // token stride, elements
  const void* dy;
  int64_t dys;  // backward: the incoming gradient
  void* out;
  int64_t os;  // forward: the result; backward: the input's gradient
  const float* gain;
  float* dgain;
  int H;
};
struct QkArgs {
  QkHead h[2];
  int64_t T;
  int D;
  int dtype;
  float eps;
  const int64_t* pos;
  const float* freq;
  int rot;
  bool interleaved;
  bool backward;
  float* workspace;  // gain gradients' partial rows
  cudaStream_t stream;
};
cudaError_t launch_qk_norm_rope(const QkArgs& a);
int64_t qk_backward_workspace_bytes(int64_t T, int Hq, int Hk, int D);

// --------------------------------------------------- linear attention ----

struct LinAttnArgs {
  const void *q, *k, *v;
  int64_t qs, ks, vs;
  int64_t T;
  int H, Dk, Dv;
  int dtype;
  const float* log_decay;
  const int32_t* cu;  // null: one sequence of T rows
  int N;
  const float* s0;
  float* s1;
  float scale;
  void* out;
  int64_t os;
  // backward
  const void* dout;
  int64_t dos;
  const float* ds1;
  void *dq, *dk, *dv;
  float* ds0;
  void* workspace;
  int64_t workspace_bytes;
  int* dev_err;
  cudaStream_t stream;
};
cudaError_t launch_linear_attention(const LinAttnArgs& a);
cudaError_t launch_linear_attention_backward(const LinAttnArgs& a);
int64_t linear_attention_workspace_bytes(int64_t T, int H, int Dk, int Dv, int dtype, int N);

struct LinAttnStepArgs {
  const void *q, *k, *v;
  int64_t qs, ks, vs;
  int B, H, Dk, Dv;
  int dtype;
  const float* log_decay;
  float* state;
  int num_slots;
  const int32_t* slots;
  float scale;
  void* out;
  int64_t os;
  cudaStream_t stream;
};
cudaError_t launch_linear_attention_step(const LinAttnStepArgs& a);

}  // namespace attnres
