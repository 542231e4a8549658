// The scan behind linear attention and its gradients (linear_attention.cu).
#pragma once

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
  float p_scale, in_scale, up_scale;  // factors of the triangle, of the carried state's part, of what enters the state

  __host__ __device__ int state_at(int da, int dc) const { return transposed ? dc * Da + da : da * Dc + dc; }
};

}  // namespace attnres
