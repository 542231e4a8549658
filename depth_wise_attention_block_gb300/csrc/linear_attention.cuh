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

// What a CTA scans in one go: tokens of one sequence and head.
struct Piece {
  int seq, head, first, len;  // first: the lowest row
  int id;                     // of its state
  int last, whole;            // whether the sequence ends with it, in the direction of the scan; and begins, too
};

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

  // parts > 0: the heads in gangs of neighbours, the gangs' chunks (gang by
  // gang, the sequences in order) in `parts` even ranges, a CTA to each range
  // and head of its gang; a piece is what a range holds of a sequence.  0: a
  // CTA per sequence and head
  int chunk, parts, gang;  // tokens per chunk; heads per gang, which divides H
  const int* first;        // of a ragged batch: [N + 1] a head's chunks before each sequence,
  const int4* starts;      // [parts + 1] each range's first chunk, its gang and sequence, and a head's chunks
  float* piece_state;      // [piece][..]: each piece's own state, then the state before it
  // where the scan itself is exact enough: the last pieces' own states are not
  // formed, it writes the final states (but for empty sequences), and whole
  // sequences are not joined
  bool final_in_scan;
  bool keep_final;         // the final states are another scan's to write, after this one

  __host__ __device__ int state_at(int da, int dc) const { return transposed ? dc * Da + da : da * Dc + dc; }
};

// The ranges: range i's first chunk, and the range that has chunk u.
struct Ranges {
  int per_head, q, rem;
  __device__ explicit Ranges(const ScanArgs& s) {
    per_head = s.first ? s.first[s.N] : (int)((s.T + s.chunk - 1) / s.chunk);
    const int units = per_head * (s.H / s.gang);
    q = units / s.parts;
    rem = units - q * s.parts;
  }
  __device__ int begin(int i) const { return q * i + (i < rem ? i : rem); }
  __device__ int owner(int u) const { return u < rem * (q + 1) ? u / (q + 1) : rem + (u - rem * (q + 1)) / q; }
};
// Chunks c0 .. c0 + n - 1 of a sequence as a piece.
__device__ __forceinline__ Piece cut_piece(const ScanArgs& s, int seq, int head, int c0, int n) {
  const SeqRange r = seq_range(s.cu, seq, s.T);
  const long long i0 = (long long)c0 * s.chunk, all = (long long)n * s.chunk, len = r.len - i0 < all ? r.len - i0 : all;
  return {seq, head, (int)(s.reverse ? r.start + r.len - i0 - len : r.start + i0), (int)len, 0, i0 + len >= r.len, i0 == 0 && len >= r.len};
}
__device__ __forceinline__ Piece whole_sequence(const ScanArgs& s, int seq, int head) {
  const SeqRange r = seq_range(s.cu, seq, s.T);
  return {seq, head, (int)r.start, (int)r.len, 0, 1, 1};
}
// The sequence with a head's chunk c: the last one that starts at c or before.
__device__ __forceinline__ int sequence_of(const int* first, int N, int c) {
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}
// The pieces of CTA `cta`, one after the other.
struct PieceWalk {
  int u = 0, end = 0, gang = 0, seq = 0, per_head = 0;
  __device__ PieceWalk() {}
  __device__ PieceWalk(const ScanArgs& s, int cta) {
    const int part = cta / s.gang;
    if (s.first) {
      const int4 a = s.starts[part];
      u = a.x, gang = a.y, seq = a.z, per_head = a.w;
      end = s.starts[part + 1].x;
    } else {
      const Ranges r(s);
      u = r.begin(part), end = r.begin(part + 1), per_head = r.per_head;
      gang = u / per_head;
    }
  }
  __device__ bool next(const ScanArgs& s, int cta, Piece* p) {
    if (u >= end) return false;
    if (u == (gang + 1) * per_head) ++gang, seq = 0;
    const int c = u - gang * per_head;
    int f0 = 0, f1 = per_head;
    if (s.first) {
      f0 = s.first[seq], f1 = s.first[seq + 1];
      while (f1 <= c) f0 = f1, f1 = s.first[++seq + 1];
    }
    const int n = f1 - c < end - u ? f1 - c : end - u, part = cta / s.gang, member = cta - part * s.gang;
    *p = cut_piece(s, seq, gang * s.gang + member, c - f0, n);
    p->id = (part + gang * s.N + seq) * s.gang + member;  // part + gang N + seq grows from piece to piece
    u += n;
    return true;
  }
};

// Workspace of a scan in pieces: bytes of the tables and of the states.
struct PieceLayout {
  int64_t first, starts, states, total;
};
struct Cut {
  int parts, gang;
};
PieceLayout piece_layout(int H, int Da, int Dc, int N, Cut cut);
void piece_place(ScanArgs& s, const PieceLayout& L, void* workspace);  // points s at the workspace
// Ranges to cut the chunks into (0: every sequence in one piece).  A range
// takes its chunks and about one more per piece; the pieces' own states cost
// `extra` of a scan, then there are their bytes, 250 ns for each of a
// sequence's pieces that are joined, and three launches.  `slots`
// CTAs run at once, `groups` of them to a range and head, a chunk takes
// chunk_ns.  The lengths are on the device, so the longest sequence is taken
// to be all T tokens.
struct CutRule {
  int chunk, groups, slots;  // tokens per chunk
  double extra, chunk_ns;
};
Cut choose_cut(int64_t T, int H, int Da, int Dc, int N, const CutRule& r);
// Bytes that suffice for every cut of up to T tokens in up to N sequences: a
// buffer kept for the largest batch serves the smaller ones, which may be cut
// where that is not.
int64_t piece_bytes(int64_t T, int H, int Da, int Dc, int N, const CutRule& r);
cudaError_t launch_piece_plan(const ScanArgs& s, cudaStream_t stream);     // the tables of a ragged batch
cudaError_t launch_piece_combine(const ScanArgs& s, cudaStream_t stream);  // own states -> the states before, and the final ones

// The scan on the tensor cores (linear_attention_tc.cu).
constexpr int kScanChunk = 128;  // tokens per chunk
bool scan_tc_dims(int Dk, int Dv, int dtype);
bool scan_tc_ok(const ScanArgs& s);  // alignment, sizes
bool scan_tc_in_pieces(int64_t T, int H, int Dk, int Dv, int N);  // whether the scan runs in pieces
int64_t scan_tc_workspace(int64_t T, int H, int Dk, int Dv, int N);
// What the workspace holds already: the tables of pieces, left by a scan of the
// same sequences; and the states before the pieces, left by one of the same
// direction, states and sums b c^T (which wrote the final state, if any).
enum ScanReady { kNothing = 0, kTables = 1, kStates = 2 };
cudaError_t launch_scan_tc(const ScanArgs& s, void* workspace, int64_t workspace_bytes, ScanReady ready, int* dev_err,
                           cudaStream_t stream);

}  // namespace attnres
