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

// l^n = exp(n log_decay), and l^0 = 1 for a decay that leaves nothing (-inf) too
__device__ __forceinline__ float decay_pow(float log_decay, int n) { return n == 0 ? 1.f : expf(log_decay * (float)n); }

struct Segment {
  int seq, first, len, last;  // sequence, first token, tokens, whether the sequence ends with it
};

// segment `i` of a sequence, in the direction of the scan
__device__ __forceinline__ Segment cut(int n, const SeqRange& r, int i, int seg_len, bool reverse) {
  Segment g;
  g.seq = n;
  const long long i0 = (long long)i * seg_len;
  const long long len = seg_len > 0 && r.len - i0 > seg_len ? seg_len : r.len - i0;
  g.len = (int)len;
  g.first = (int)(reverse ? r.start + r.len - i0 - len : r.start + i0);
  g.last = i0 + len >= r.len;
  return g;
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

  // segments: null, and a segment is a sequence, or arithmetic over the one
  // there is
  const Segment* segs;
  const int* nsegs;
  int seg_len;             // tokens per segment (0: a sequence is one segment)
  float* seg_state;        // [segment][H][..]: each segment's own state, then the state before it

  __host__ __device__ int state_at(int da, int dc) const { return transposed ? dc * Da + da : da * Dc + dc; }
};

__device__ __forceinline__ Segment segment_of(const ScanArgs& s, int i) {
  if (s.segs) return s.segs[i];
  if (s.cu) return cut(i, seq_range(s.cu, i, s.T), 0, 0, s.reverse);
  return cut(0, {0, s.T}, i, s.seg_len, s.reverse);
}

// Workspace of a scan in segments: at most `segs` of them; bytes of the table,
// of the sequences' first segments and of the states.
struct SegLayout {
  int64_t segs, table, first, states, total;
};
SegLayout seg_layout(int64_t T, int H, int Da, int Dc, int N, int seg_len);
// Points s at the workspace; *segs: the CTAs' segments.
void seg_place(ScanArgs& s, const SegLayout& L, void* workspace, int64_t* segs);
// Tokens per segment (0: every sequence in one piece): a wave of `slots` CTAs
// (per_seg of them to a segment) takes a segment's chunks and about two more
// to start and end; the segments' own states cost `extra` of a scan, and the
// launches about 4 chunks.  The lengths are on the device, so the longest
// sequence is taken to be all T tokens.
int seg_tokens(int64_t T, int N, int chunk, int64_t per_seg, int slots, double extra);
cudaError_t launch_seg_plan(const ScanArgs& s, cudaStream_t stream);      // the table of a ragged batch
cudaError_t launch_seg_combine(const ScanArgs& s, cudaStream_t stream);   // own states -> the states before, and the final ones

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
