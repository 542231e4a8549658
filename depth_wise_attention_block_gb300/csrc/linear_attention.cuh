// The scan behind linear attention and its gradients (linear_attention.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace attnres {

// Sequence n's rows: cu[n] .. cu[n+1] - 1, clamped to 0 .. T.
struct SeqRange {
  long long start, len;
  // row of its i-th token, counted from the end when reversed
  __host__ __device__ long long row(long long i, bool reverse) const { return reverse ? start + len - 1 - i : start + i; }
};

__device__ __forceinline__ SeqRange seq_range(const int32_t* cu, int n, long long T) {
  if (!cu) return {0, T};
  long long s = cu[n], e = cu[n + 1];
  s = s < 0 ? 0 : s > T ? T : s;
  e = e < s ? s : e > T ? T : e;
  return {s, e - s};
}

struct ScanArgs {
  const void *a, *b, *c;   // [T, H, Da], [T, H, Da], [T, H, Dc]; token strides
  long long as, bs, cs;
  void* out;               // [T, H, Dc]
  long long os;
  int Da, Dc, H, N;
  long long T;
  const int32_t* cu;
  const float* log_decay;  // [H]
  const float* s_in;       // [N, H, Da, Dc] (transposed: [N, H, Dc, Da]) or null
  float* s_out;
  bool transposed, reverse;
  int shift;               // 1: the carried state is already decayed for the next token
  bool wide_out;           // out's rows start on 32-byte boundaries (set by the launch)
  bool vec_a, vec_b, vec_c;  // rows in vectors of 4 elements (set by the launch)
  float p_scale, in_scale, up_scale;  // factors of the triangle, of the carried state's part, of what enters the state

  __host__ __device__ int state_at(int da, int dc) const { return transposed ? dc * Da + da : da * Dc + dc; }
};

// The scan on the tensor cores (linear_attention_tc.cu).
constexpr int kScanChunk = 128;  // tokens per chunk
bool scan_tc_dims(int Dk, int Dv, int dtype);
bool scan_tc_ok(const ScanArgs& s);  // alignment, sizes
bool scan_tc_segmented(int64_t T, int H, int N);  // whether long sequences are cut into segments
int64_t scan_tc_workspace(int64_t T, int H, int Dk, int Dv, int N);
// states_ready: the workspace holds the states before the segments already,
// left there by a scan of the same direction, states and sums b c^T (which
// wrote the final state, if any)
cudaError_t launch_scan_tc(const ScanArgs& s, void* workspace, bool states_ready, int* dev_err, cudaStream_t stream);

}  // namespace attnres
