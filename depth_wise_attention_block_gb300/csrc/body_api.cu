// The C ABI of a layer body's operators and of gradient clipping (declared in
// include/attnres.h): argument checks and dispatch to the kernels (linear.cu,
// qk_norm_rope.cu, linear_attention.cu, layer_norm.cu, gated_recurrence.cu,
// grad_clip.cu).
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <memory>
#include <new>

#include "api_common.h"
#include "body.h"
#include "launch.h"

using namespace attnres;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 42;  // element offsets stay far inside int64
constexpr int kMaxWidth = 1 << 30;               // of a projection: tiles past its end stay inside int
constexpr int64_t kMaxRows = INT32_MAX - 64;     // of a projection (grad_w's contraction): a step past its end, too

// `rows` rows of `width` bytes, `pitch` bytes apart
struct Rows {
  const void* p;
  int64_t rows, width, pitch;
  int64_t span() const { return rows > 0 ? (rows - 1) * pitch + width : 0; }
};

// Whether two row tensors share a byte.  Of equal pitch, slices of one wider
// buffer are told apart; of different pitches, any overlap of their spans
// counts.
bool rows_overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || !overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.pitch != b.pitch) return true;
  const int64_t pa = (int64_t)reinterpret_cast<uintptr_t>(a.p), pb = (int64_t)reinterpret_cast<uintptr_t>(b.p);
  const int64_t off = ((pb - pa) % a.pitch + a.pitch) % a.pitch;  // b's column in a's rows
  return off < a.width || off + b.width > a.pitch;
}

bool same_rows(const Rows& a, const Rows& b) { return a.p == b.p && a.pitch == b.pitch && a.width == b.width; }

// every output apart from every input and from each other; `in_place[o]` is
// the input output o may be itself (or -1)
int check_apart(const Rows* in, int nin, const Rows* out, int nout, const int* in_place) {
  for (int o = 0; o < nout; ++o) {
    for (int i = 0; i < nin; ++i)
      if (rows_overlap(out[o], in[i]) && !(in_place && in_place[o] == i && same_rows(out[o], in[i])))
        return fail(ATTNRES_EINVAL, "output %d overlaps input %d", o, i);
    for (int j = 0; j < o; ++j)
      if (rows_overlap(out[o], out[j])) return fail(ATTNRES_EINVAL, "outputs %d and %d overlap", o, j);
  }
  return ATTNRES_OK;
}

int check_linear_sizes(int64_t M, int N, int K, int dtype, int act) {
  if (!valid_dtype(dtype)) return fail(ATTNRES_EDTYPE, "dtype %d", dtype);
  if (M < 0 || N < 1 || K < 1) return fail(ATTNRES_EINVAL, "M=%lld N=%d K=%d", (long long)M, N, K);
  if (M > kMaxRows) return fail(ATTNRES_ERANGE, "M=%lld", (long long)M);
  if (N > kMaxWidth || K > kMaxWidth) return fail(ATTNRES_ERANGE, "N=%d K=%d", N, K);
  if (M > kMaxElems / N || M > kMaxElems / K || N > kMaxElems / K) return fail(ATTNRES_ERANGE, "M*N, M*K or N*K too large");
  if (act < ATTNRES_ACT_NONE || act > ATTNRES_ACT_SILU) return fail(ATTNRES_EINVAL, "activation %d", act);
  return ATTNRES_OK;
}

bool stride_ok(int64_t ld, int64_t width) { return ld >= width && ld <= kMaxElems; }
bool span_ok(int64_t rows, int64_t ld) { return rows <= 0 || ld <= kMaxElems / rows; }
bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(n - 1)) == 0; }

int check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (bytes < 0) return fail(ATTNRES_EINVAL, "workspace_bytes=%lld", (long long)bytes);
  if (need <= 0) return ATTNRES_OK;
  if (!ws) return fail(ATTNRES_EINVAL, "workspace is NULL, %lld bytes needed", (long long)need);
  if (bytes < need)
    return fail(ATTNRES_EINVAL, "workspace of %lld bytes, %lld needed", (long long)bytes, (long long)need);
  if (!aligned(ws, 256)) return fail(ATTNRES_EINVAL, "workspace is not 256-byte aligned");
  return ATTNRES_OK;
}

int check_qk(const void* q, int64_t qs, int Hq, const void* k, int64_t ks, int Hk, int64_t T, int D, int dtype,
             float eps, const int64_t* pos, const float* freq, int rot, int interleaved) {
  if (!valid_dtype(dtype)) return fail(ATTNRES_EDTYPE, "dtype %d", dtype);
  if (T < 0 || D < 1 || Hq < 0 || Hk < 0 || Hq + (int64_t)Hk < 1)
    return fail(ATTNRES_EINVAL, "T=%lld D=%d Hq=%d Hk=%d", (long long)T, D, Hq, Hk);
  if (D > 1024 || Hq > 65535 || Hk > 65535) return fail(ATTNRES_ERANGE, "D=%d Hq=%d Hk=%d", D, Hq, Hk);
  if (rot < 0 || rot > D || (rot & 1)) return fail(ATTNRES_EINVAL, "rot=%d (even, 0..D)", rot);
  if (interleaved != 0 && interleaved != 1) return fail(ATTNRES_EINVAL, "interleaved must be 0 or 1");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(ATTNRES_EINVAL, "eps must be finite and >= 0");
  if ((Hq > 0 && !stride_ok(qs, (int64_t)Hq * D)) || (Hk > 0 && !stride_ok(ks, (int64_t)Hk * D)))
    return fail(ATTNRES_EINVAL, "a token stride is shorter than its row");
  if (!span_ok(T, Hq > 0 ? qs : 1) || !span_ok(T, Hk > 0 ? ks : 1)) return fail(ATTNRES_ERANGE, "T*stride too large");
  if (T == 0) return ATTNRES_OK;
  if ((Hq > 0 && !q) || (Hk > 0 && !k)) return fail(ATTNRES_EINVAL, "q/k is NULL");
  if (rot > 0 && (!pos || !freq)) return fail(ATTNRES_EINVAL, "positions/inv_freq is NULL");
  return ATTNRES_OK;
}

int check_la_sizes(int64_t T, int H, int Dk, int Dv, int dtype, int N) {
  if (!valid_dtype(dtype)) return fail(ATTNRES_EDTYPE, "dtype %d", dtype);
  if (T < 0 || H < 1 || Dk < 1 || Dv < 1 || N < 1)
    return fail(ATTNRES_EINVAL, "T=%lld H=%d Dk=%d Dv=%d num_seqs=%d", (long long)T, H, Dk, Dv, N);
  if (H > 65535 || Dk > 256 || Dv > 256 || N > 65535)
    return fail(ATTNRES_ERANGE, "H=%d Dk=%d Dv=%d num_seqs=%d", H, Dk, Dv, N);
  if (T > INT32_MAX) return fail(ATTNRES_ERANGE, "T=%lld", (long long)T);
  return ATTNRES_OK;
}

int check_la(const void* q, int64_t qs, const void* k, int64_t ks, const void* v, int64_t vs, int64_t T, int H, int Dk,
             int Dv, int dtype, const float* log_decay, const int32_t* cu, int N, float scale) {
  const int rc = check_la_sizes(T, H, Dk, Dv, dtype, N);
  if (rc != ATTNRES_OK) return rc;
  if (!cu && N != 1) return fail(ATTNRES_EINVAL, "num_seqs=%d without cu_seqlens", N);
  if (!std::isfinite(scale)) return fail(ATTNRES_EINVAL, "scale is not finite");
  if (!stride_ok(qs, (int64_t)H * Dk) || !stride_ok(ks, (int64_t)H * Dk) || !stride_ok(vs, (int64_t)H * Dv))
    return fail(ATTNRES_EINVAL, "a token stride is shorter than its row");
  if (!span_ok(T, qs) || !span_ok(T, ks) || !span_ok(T, vs)) return fail(ATTNRES_ERANGE, "T*stride too large");
  if (!log_decay) return fail(ATTNRES_EINVAL, "log_decay is NULL");
  if (T > 0 && (!q || !k || !v)) return fail(ATTNRES_EINVAL, "q/k/v is NULL");
  return ATTNRES_OK;
}

// fp32 and int32 arrays (null: absent)
int check_words(std::initializer_list<const void*> arrays) {
  for (const void* p : arrays)
    if (!aligned(p, 4)) return fail(ATTNRES_EINVAL, "a float or int32 array is not 4-byte aligned");
  return ATTNRES_OK;
}

constexpr int kMaxNormWidth = 1 << 24;   // of a layer norm's row
constexpr int kMaxChannels = 1 << 24;    // of a recurrence
constexpr int kMaxTensors = 65535;       // of a list of gradients

int check_ln(const void* x, int64_t xs, int64_t T, int d, int dtype, float eps) {
  if (!valid_dtype(dtype)) return fail(ATTNRES_EDTYPE, "dtype %d", dtype);
  if (T < 0 || d < 1) return fail(ATTNRES_EINVAL, "T=%lld d=%d", (long long)T, d);
  if (d > kMaxNormWidth) return fail(ATTNRES_ERANGE, "d=%d", d);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(ATTNRES_EINVAL, "eps must be finite and >= 0");
  if (!stride_ok(xs, d)) return fail(ATTNRES_EINVAL, "a row stride is shorter than its row");
  if (!span_ok(T, xs)) return fail(ATTNRES_ERANGE, "T*stride too large");
  if (T > 0 && !x) return fail(ATTNRES_EINVAL, "x is NULL");
  if (!aligned(x, (int)dtype_bytes(dtype))) return fail(ATTNRES_EINVAL, "a tensor is not aligned to its elements");
  return ATTNRES_OK;
}

// a row tensor [T, C] that an operator reads or writes (null: absent)
int check_gr_rows(const void* p, int64_t stride, int64_t T, int C, int dtype) {
  if (!p) return ATTNRES_OK;
  if (!aligned(p, (int)dtype_bytes(dtype))) return fail(ATTNRES_EINVAL, "a tensor is not aligned to its elements");
  if (!stride_ok(stride, C)) return fail(ATTNRES_EINVAL, "a row stride is shorter than its row");
  if (!span_ok(T, stride)) return fail(ATTNRES_ERANGE, "T*stride too large");
  return ATTNRES_OK;
}

int check_gr(const void* x, int64_t xs, const void* f, int64_t fs, const void* g, int64_t gs, int64_t T, int C, int dtype,
             const int32_t* cu, int N) {
  if (!valid_dtype(dtype)) return fail(ATTNRES_EDTYPE, "dtype %d", dtype);
  if (T < 0 || C < 1 || N < 1) return fail(ATTNRES_EINVAL, "T=%lld C=%d num_seqs=%d", (long long)T, C, N);
  if (T > INT32_MAX - 65536 || C > kMaxChannels || N > 65535)
    return fail(ATTNRES_ERANGE, "T=%lld C=%d num_seqs=%d", (long long)T, C, N);
  if (!cu && N != 1) return fail(ATTNRES_EINVAL, "num_seqs=%d without cu_seqlens", N);
  if (T > 0 && (!x || !f)) return fail(ATTNRES_EINVAL, "x/forget is NULL");
  int rc = check_gr_rows(x, xs, T, C, dtype);
  if (rc == ATTNRES_OK) rc = check_gr_rows(f, fs, T, C, dtype);
  if (rc == ATTNRES_OK) rc = check_gr_rows(g, gs, T, C, dtype);
  return rc;
}

// [begin, end) of a tensor of a list, and whether it is written
struct Interval {
  uintptr_t begin, end;
  bool out;
};

// Every output apart from every other output and from every input but its
// own (which is left out of the list where they are the same).
bool intervals_apart(Interval* v, int n) {
  std::sort(v, v + n, [](const Interval& a, const Interval& b) { return a.begin < b.begin; });
  uintptr_t read_to = 0, written_to = 0;
  for (int i = 0; i < n; ++i) {
    if (v[i].begin < written_to || (v[i].out && v[i].begin < read_to)) return false;
    uintptr_t& to = v[i].out ? written_to : read_to;
    if (v[i].end > to) to = v[i].end;
  }
  return true;
}

}  // namespace

extern "C" {

int64_t attnres_linear_workspace_size(int64_t M, int N, int K, int dtype) {
  const int rc = check_linear_sizes(M, N, K, dtype, ATTNRES_ACT_NONE);
  if (rc != ATTNRES_OK) return rc;
  ok();
  return linear_workspace_bytes(M, N, K, dtype, linear_uneven_sizes(N, K));
}

int64_t attnres_linear_operands_workspace_size(const void* x, int64_t ldx, const void* w, int64_t M, int N, int K, int dtype) {
  const int rc = check_linear_sizes(M, N, K, dtype, ATTNRES_ACT_NONE);
  if (rc != ATTNRES_OK) return rc;
  if (!stride_ok(ldx, K)) return fail(ATTNRES_EINVAL, "a row stride is shorter than its row");
  ok();
  return linear_workspace_bytes(M, N, K, dtype, linear_uneven(x, ldx, w, nullptr, 0, N, K));
}

int attnres_linear(const void* x, int64_t ldx, const void* w, const float* bias, const void* residual, int64_t ldr,
                   void* out, int64_t ldo, int64_t M, int N, int K, int dtype, int act, void* workspace,
                   int64_t workspace_bytes, int* dev_err, void* stream) {
  const int rc = check_linear_sizes(M, N, K, dtype, act);
  if (rc != ATTNRES_OK) return rc;
  if (M == 0) return ok();
  if (!x || !w || !out) return fail(ATTNRES_EINVAL, "x/w/out is NULL");
  if (!stride_ok(ldx, K) || !stride_ok(ldo, N) || (residual && !stride_ok(ldr, N)))
    return fail(ATTNRES_EINVAL, "a row stride is shorter than its row");
  if (!span_ok(M, ldx) || !span_ok(M, ldo) || (residual && !span_ok(M, ldr)))
    return fail(ATTNRES_ERANGE, "M*stride too large");
  if (workspace_bytes < 0) return fail(ATTNRES_EINVAL, "workspace_bytes=%lld", (long long)workspace_bytes);
  if (workspace && !aligned(workspace, 256)) return fail(ATTNRES_EINVAL, "workspace is not 256-byte aligned");
  const int64_t es = dtype_bytes(dtype);
  {
    const Rows in[4] = {{x, M, K * es, ldx * es},
                        {w, 1, (int64_t)N * K * es, (int64_t)N * K * es},
                        {bias, 1, (int64_t)N * 4, (int64_t)N * 4},
                        {residual, M, N * es, ldr * es}};
    const int64_t wsb = workspace ? workspace_bytes : 0;
    const Rows out_rows[2] = {{out, M, N * es, ldo * es}, {workspace, 1, wsb, wsb}};
    const int in_place[2] = {3, -1};
    const int ra = check_apart(in, 4, out_rows, 2, in_place);
    if (ra != ATTNRES_OK) return ra;
  }
  LinearArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.ldr = ldr;
  a.out = out;
  a.ldo = ldo;
  a.M = M;
  a.N = N;
  a.K = K;
  a.dtype = dtype;
  a.act = act;
  a.workspace = workspace;
  a.workspace_bytes = workspace ? workspace_bytes : 0;
  a.dev_err = dev_err;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_linear(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_linear launch");
  return ok();
}

int64_t attnres_linear_backward_workspace_size(int64_t M, int N, int K, int dtype, int act) {
  const int rc = check_linear_sizes(M, N, K, dtype, act);
  if (rc != ATTNRES_OK) return rc;
  ok();
  return linear_backward_workspace_bytes(M, N, K, dtype, act, linear_uneven_sizes(N, K));
}

int64_t attnres_linear_backward_operands_workspace_size(const void* x, int64_t ldx, const void* w, const void* grad_out, int64_t ldg,
                                                        int64_t M, int N, int K, int dtype, int act) {
  const int rc = check_linear_sizes(M, N, K, dtype, act);
  if (rc != ATTNRES_OK) return rc;
  if (!stride_ok(ldx, K) || !stride_ok(ldg, N)) return fail(ATTNRES_EINVAL, "a row stride is shorter than its row");
  ok();
  return linear_backward_workspace_bytes(M, N, K, dtype, act, linear_uneven(x, ldx, w, grad_out, ldg, N, K));
}

int attnres_linear_backward(const void* x, int64_t ldx, const void* w, const float* bias, const void* grad_out,
                            int64_t ldg, void* grad_x, void* grad_w, float* grad_bias, int64_t M, int N, int K,
                            int dtype, int act, void* workspace, int64_t workspace_bytes, int* dev_err, void* stream) {
  int rc = check_linear_sizes(M, N, K, dtype, act);
  if (rc != ATTNRES_OK) return rc;
  if (!grad_x && !grad_w && !grad_bias) return ok();
  const int64_t es = dtype_bytes(dtype);
  if (M > 0) {
    if (!grad_out) return fail(ATTNRES_EINVAL, "grad_out is NULL");
    if ((!x && (grad_w || act != ATTNRES_ACT_NONE)) || (!w && (grad_x || act != ATTNRES_ACT_NONE)))
      return fail(ATTNRES_EINVAL, "x/w is NULL");
    if ((x && !stride_ok(ldx, K)) || !stride_ok(ldg, N))
      return fail(ATTNRES_EINVAL, "a row stride is shorter than its row");
    if ((x && !span_ok(M, ldx)) || !span_ok(M, ldg)) return fail(ATTNRES_ERANGE, "M*stride too large");
    rc = check_workspace(workspace, workspace_bytes,
                         linear_backward_workspace_bytes(M, N, K, dtype, act, linear_uneven_sizes(N, K)));
    if (rc != ATTNRES_OK) return rc;
  }
  {
    const int64_t wsb = workspace ? workspace_bytes : 0;
    const Rows in[4] = {{x, M, K * es, ldx * es},
                        {w, 1, (int64_t)N * K * es, (int64_t)N * K * es},
                        {bias, 1, (int64_t)N * 4, (int64_t)N * 4},
                        {grad_out, M, N * es, ldg * es}};
    const Rows out[4] = {{grad_x, 1, M * K * es, M * K * es},
                         {grad_w, 1, (int64_t)N * K * es, (int64_t)N * K * es},
                         {grad_bias, 1, (int64_t)N * 4, (int64_t)N * 4},
                         {workspace, 1, wsb, wsb}};
    rc = check_apart(in, M > 0 ? 4 : 0, out, 4, nullptr);
    if (rc != ATTNRES_OK) return rc;
  }
  LinearBwdArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.bias = bias;
  a.grad_out = grad_out;
  a.ldg = ldg;
  a.grad_x = M > 0 ? grad_x : nullptr;
  a.grad_w = grad_w;
  a.grad_bias = grad_bias;
  a.M = M;
  a.N = N;
  a.K = K;
  a.dtype = dtype;
  a.act = act;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.dev_err = dev_err;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_linear_backward(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_linear_backward launch");
  return ok();
}

int attnres_qk_norm_rope(const void* q, int64_t q_stride, int Hq, const void* k, int64_t k_stride, int Hk, int64_t T,
                         int D, int dtype, const float* q_gain, const float* k_gain, float eps,
                         const int64_t* positions, const float* inv_freq, int rot, int interleaved, void* q_out,
                         int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  const int rc = check_qk(q, q_stride, Hq, k, k_stride, Hk, T, D, dtype, eps, positions, inv_freq, rot, interleaved);
  if (rc != ATTNRES_OK) return rc;
  if (T == 0) return ok();
  if ((Hq > 0 && !q_out) || (Hk > 0 && !k_out)) return fail(ATTNRES_EINVAL, "q_out/k_out is NULL");
  const int64_t wq = (int64_t)Hq * D, wk = (int64_t)Hk * D, es = dtype_bytes(dtype);
  if ((Hq > 0 && !stride_ok(q_out_stride, wq)) || (Hk > 0 && !stride_ok(k_out_stride, wk)))
    return fail(ATTNRES_EINVAL, "a token stride is shorter than its row");
  if (!span_ok(T, Hq > 0 ? q_out_stride : 1) || !span_ok(T, Hk > 0 ? k_out_stride : 1))
    return fail(ATTNRES_ERANGE, "T*stride too large");
  {
    const Rows in[6] = {{Hq > 0 ? q : nullptr, T, wq * es, q_stride * es},
                        {Hk > 0 ? k : nullptr, T, wk * es, k_stride * es},
                        {q_gain, 1, D * 4, D * 4},
                        {k_gain, 1, D * 4, D * 4},
                        {rot > 0 ? positions : nullptr, 1, T * 8, T * 8},
                        {rot > 0 ? inv_freq : nullptr, 1, rot * 2, rot * 2}};
    const Rows out[2] = {{Hq > 0 ? q_out : nullptr, T, wq * es, q_out_stride * es},
                         {Hk > 0 ? k_out : nullptr, T, wk * es, k_out_stride * es}};
    const int in_place[2] = {0, 1};
    const int ra = check_apart(in, 6, out, 2, in_place);
    if (ra != ATTNRES_OK) return ra;
  }
  QkArgs a{};
  a.h[0] = {q, q_stride, nullptr, 0, q_out, q_out_stride, q_gain, nullptr, Hq};
  a.h[1] = {k, k_stride, nullptr, 0, k_out, k_out_stride, k_gain, nullptr, Hk};
  a.T = T;
  a.D = D;
  a.dtype = dtype;
  a.eps = eps;
  a.pos = positions;
  a.freq = inv_freq;
  a.rot = rot;
  a.interleaved = interleaved != 0;
  a.backward = false;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_qk_norm_rope(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_qk_norm_rope launch");
  return ok();
}

int64_t attnres_qk_norm_rope_backward_workspace_size(int64_t T, int Hq, int Hk, int D) {
  if (T < 0 || D < 1 || Hq < 0 || Hk < 0 || Hq + (int64_t)Hk < 1)
    return fail(ATTNRES_EINVAL, "T=%lld D=%d Hq=%d Hk=%d", (long long)T, D, Hq, Hk);
  if (D > 1024 || Hq > 65535 || Hk > 65535) return fail(ATTNRES_ERANGE, "D=%d Hq=%d Hk=%d", D, Hq, Hk);
  const int64_t n = qk_backward_workspace_bytes(T, Hq, Hk, D);
  if (n < 0) return fail(ATTNRES_ECUDA, "device query");
  ok();
  return n;
}

int attnres_qk_norm_rope_backward(const void* q, int64_t q_stride, int Hq, const void* k, int64_t k_stride, int Hk,
                                  int64_t T, int D, int dtype, const float* q_gain, const float* k_gain, float eps,
                                  const int64_t* positions, const float* inv_freq, int rot, int interleaved,
                                  const void* grad_q_out, int64_t gqo_stride, const void* grad_k_out,
                                  int64_t gko_stride, void* grad_q, int64_t gq_stride, void* grad_k,
                                  int64_t gk_stride, float* grad_q_gain, float* grad_k_gain, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  int rc = check_qk(q, q_stride, Hq, k, k_stride, Hk, T, D, dtype, eps, positions, inv_freq, rot, interleaved);
  if (rc != ATTNRES_OK) return rc;
  const int64_t wq = (int64_t)Hq * D, wk = (int64_t)Hk * D, es = dtype_bytes(dtype);
  if (T > 0) {
    if ((Hq > 0 && (!grad_q_out || !grad_q)) || (Hk > 0 && (!grad_k_out || !grad_k)))
      return fail(ATTNRES_EINVAL, "a gradient of q/k is NULL");
    if ((Hq > 0 && (!stride_ok(gqo_stride, wq) || !stride_ok(gq_stride, wq))) ||
        (Hk > 0 && (!stride_ok(gko_stride, wk) || !stride_ok(gk_stride, wk))))
      return fail(ATTNRES_EINVAL, "a token stride is shorter than its row");
    if ((Hq > 0 && (!span_ok(T, gqo_stride) || !span_ok(T, gq_stride))) ||
        (Hk > 0 && (!span_ok(T, gko_stride) || !span_ok(T, gk_stride))))
      return fail(ATTNRES_ERANGE, "T*stride too large");
    const int64_t wsb = workspace && workspace_bytes > 0 ? workspace_bytes : 0;
    const Rows in[8] = {{Hq > 0 ? grad_q_out : nullptr, T, wq * es, gqo_stride * es},
                        {Hk > 0 ? grad_k_out : nullptr, T, wk * es, gko_stride * es},
                        {Hq > 0 ? q : nullptr, T, wq * es, q_stride * es},
                        {Hk > 0 ? k : nullptr, T, wk * es, k_stride * es},
                        {q_gain, 1, D * 4, D * 4},
                        {k_gain, 1, D * 4, D * 4},
                        {rot > 0 ? positions : nullptr, 1, T * 8, T * 8},
                        {rot > 0 ? inv_freq : nullptr, 1, rot * 2, rot * 2}};
    const Rows out[5] = {{Hq > 0 ? grad_q : nullptr, T, wq * es, gq_stride * es},
                         {Hk > 0 ? grad_k : nullptr, T, wk * es, gk_stride * es},
                         {grad_q_gain, 1, D * 4, D * 4},
                         {grad_k_gain, 1, D * 4, D * 4},
                         {workspace, 1, wsb, wsb}};
    const int in_place[5] = {0, 1, -1, -1, -1};
    rc = check_apart(in, 8, out, 5, in_place);
    if (rc != ATTNRES_OK) return rc;
    if (grad_q_gain || grad_k_gain) {
      if (!workspace) return fail(ATTNRES_EINVAL, "the gain gradients need a workspace");
      const int64_t need = qk_backward_workspace_bytes(T, Hq, Hk, D);
      if (need < 0) return fail(ATTNRES_ECUDA, "device query");
      if (workspace_bytes < need)
        return fail(ATTNRES_EINVAL, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)need);
      if (!aligned(workspace, 4)) return fail(ATTNRES_EINVAL, "workspace is not 4-byte aligned");
    }
  }
  QkArgs a{};
  a.h[0] = {q, q_stride, grad_q_out, gqo_stride, grad_q, gq_stride, q_gain, grad_q_gain, Hq};
  a.h[1] = {k, k_stride, grad_k_out, gko_stride, grad_k, gk_stride, k_gain, grad_k_gain, Hk};
  a.T = T;
  a.D = D;
  a.dtype = dtype;
  a.eps = eps;
  a.pos = positions;
  a.freq = inv_freq;
  a.rot = rot;
  a.interleaved = interleaved != 0;
  a.backward = true;
  a.workspace = static_cast<float*>(workspace);
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_qk_norm_rope(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_qk_norm_rope_backward launch");
  return ok();
}

int64_t attnres_linear_attention_workspace_size(int64_t T, int H, int Dk, int Dv, int dtype, int num_seqs) {
  const int rc = check_la_sizes(T, H, Dk, Dv, dtype, num_seqs);
  if (rc != ATTNRES_OK) return rc;
  const int64_t n = linear_attention_workspace_bytes(T, H, Dk, Dv, dtype, num_seqs);
  if (n < 0) return fail(ATTNRES_ECUDA, "device query");
  ok();
  return n;
}

int64_t attnres_linear_attention_backward_workspace_size(int64_t T, int H, int Dk, int Dv, int dtype, int num_seqs) {
  const int rc = check_la_sizes(T, H, Dk, Dv, dtype, num_seqs);
  if (rc != ATTNRES_OK) return rc;
  const int64_t n = linear_attention_workspace_bytes(T, H, Dk, Dv, dtype, num_seqs);
  if (n < 0) return fail(ATTNRES_ECUDA, "device query");
  ok();
  return n;
}

int attnres_linear_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, int64_t T, int H, int Dk, int Dv, int dtype, const float* log_decay,
                             const int32_t* cu_seqlens, int num_seqs, const float* initial_state, float* final_state,
                             float scale, void* out, int64_t out_stride, void* workspace, int64_t workspace_bytes,
                             int* dev_err, void* stream) {
  int rc = check_la(q, q_stride, k, k_stride, v, v_stride, T, H, Dk, Dv, dtype, log_decay, cu_seqlens, num_seqs, scale);
  if (rc != ATTNRES_OK) return rc;
  if (T > 0 && !out) return fail(ATTNRES_EINVAL, "out is NULL");
  if (!stride_ok(out_stride, (int64_t)H * Dv)) return fail(ATTNRES_EINVAL, "out_stride is shorter than its row");
  if (!span_ok(T, out_stride)) return fail(ATTNRES_ERANGE, "T*stride too large");
  if (T == 0 && !final_state) return ok();
  {
    const int64_t es = dtype_bytes(dtype), st = (int64_t)num_seqs * H * Dk * Dv * 4, cub = (num_seqs + 1) * 4LL;
    const int64_t wsb = workspace ? workspace_bytes : 0;
    const Rows in[6] = {{q, T, (int64_t)H * Dk * es, q_stride * es}, {k, T, (int64_t)H * Dk * es, k_stride * es},
                        {v, T, (int64_t)H * Dv * es, v_stride * es}, {log_decay, 1, H * 4LL, H * 4LL},
                        {cu_seqlens, 1, cub, cub},                   {initial_state, 1, st, st}};
    const Rows outs[3] = {{T > 0 ? out : nullptr, T, (int64_t)H * Dv * es, out_stride * es},
                          {final_state, 1, st, st},
                          {workspace, 1, wsb, wsb}};
    const int in_place[3] = {-1, 5, -1};
    rc = check_apart(in, 6, outs, 3, in_place);
    if (rc != ATTNRES_OK) return rc;
  }
  if (workspace && !aligned(workspace, 256)) return fail(ATTNRES_EINVAL, "workspace is not 256-byte aligned");
  const int64_t need = linear_attention_workspace_bytes(T, H, Dk, Dv, dtype, num_seqs);
  if (need < 0) return fail(ATTNRES_ECUDA, "device query");
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != ATTNRES_OK) return rc;
  LinAttnArgs a{};
  a.q = q;
  a.qs = q_stride;
  a.k = k;
  a.ks = k_stride;
  a.v = v;
  a.vs = v_stride;
  a.T = T;
  a.H = H;
  a.Dk = Dk;
  a.Dv = Dv;
  a.dtype = dtype;
  a.log_decay = log_decay;
  a.cu = cu_seqlens;
  a.N = num_seqs;
  a.s0 = initial_state;
  a.s1 = final_state;
  a.scale = scale;
  a.out = out;
  a.os = out_stride;
  a.workspace = workspace;
  a.workspace_bytes = workspace ? workspace_bytes : 0;
  a.dev_err = dev_err;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_linear_attention(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_linear_attention launch");
  return ok();
}

int attnres_linear_attention_backward(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                      int64_t v_stride, int64_t T, int H, int Dk, int Dv, int dtype,
                                      const float* log_decay, const int32_t* cu_seqlens, int num_seqs,
                                      const float* initial_state, float scale, const void* grad_out,
                                      int64_t grad_out_stride, const float* grad_final_state, void* grad_q,
                                      void* grad_k, void* grad_v, float* grad_initial_state, void* workspace,
                                      int64_t workspace_bytes, int* dev_err, void* stream) {
  int rc = check_la(q, q_stride, k, k_stride, v, v_stride, T, H, Dk, Dv, dtype, log_decay, cu_seqlens, num_seqs, scale);
  if (rc != ATTNRES_OK) return rc;
  if (!grad_q && !grad_k && !grad_v && !grad_initial_state) return ok();
  if (T > 0 && !grad_out) return fail(ATTNRES_EINVAL, "grad_out is NULL");
  if (T > 0 && grad_initial_state && !grad_v) return fail(ATTNRES_EINVAL, "grad_initial_state comes with grad_v");
  if (!stride_ok(grad_out_stride, (int64_t)H * Dv))
    return fail(ATTNRES_EINVAL, "grad_out_stride is shorter than its row");
  if (!span_ok(T, grad_out_stride)) return fail(ATTNRES_ERANGE, "T*stride too large");
  if (T == 0 && !grad_initial_state) return ok();
  {
    const int64_t es = dtype_bytes(dtype), st = (int64_t)num_seqs * H * Dk * Dv * 4, cub = (num_seqs + 1) * 4LL;
    const int64_t bk = (int64_t)H * Dk * es, bv = (int64_t)H * Dv * es, wsb = workspace ? workspace_bytes : 0;
    const Rows in[8] = {{q, T, bk, q_stride * es},
                        {k, T, bk, k_stride * es},
                        {v, T, bv, v_stride * es},
                        {log_decay, 1, H * 4LL, H * 4LL},
                        {cu_seqlens, 1, cub, cub},
                        {initial_state, 1, st, st},
                        {grad_out, T, bv, grad_out_stride * es},
                        {grad_final_state, 1, st, st}};
    const Rows outs[5] = {{T > 0 ? grad_q : nullptr, 1, T * bk, T * bk},
                          {T > 0 ? grad_k : nullptr, 1, T * bk, T * bk},
                          {T > 0 ? grad_v : nullptr, 1, T * bv, T * bv},
                          {grad_initial_state, 1, st, st},
                          {workspace, 1, wsb, wsb}};
    const int in_place[5] = {-1, -1, -1, 7, -1};
    rc = check_apart(in, 8, outs, 5, in_place);
    if (rc != ATTNRES_OK) return rc;
  }
  if (workspace && !aligned(workspace, 256)) return fail(ATTNRES_EINVAL, "workspace is not 256-byte aligned");
  const int64_t need = linear_attention_workspace_bytes(T, H, Dk, Dv, dtype, num_seqs);
  if (need < 0) return fail(ATTNRES_ECUDA, "device query");
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != ATTNRES_OK) return rc;
  LinAttnArgs a{};
  a.q = q;
  a.qs = q_stride;
  a.k = k;
  a.ks = k_stride;
  a.v = v;
  a.vs = v_stride;
  a.T = T;
  a.H = H;
  a.Dk = Dk;
  a.Dv = Dv;
  a.dtype = dtype;
  a.log_decay = log_decay;
  a.cu = cu_seqlens;
  a.N = num_seqs;
  a.s0 = initial_state;
  a.scale = scale;
  a.dout = grad_out;
  a.dos = grad_out_stride;
  a.ds1 = grad_final_state;
  a.dq = grad_q;
  a.dk = grad_k;
  a.dv = grad_v;
  a.ds0 = grad_initial_state;
  a.workspace = workspace;
  a.workspace_bytes = workspace ? workspace_bytes : 0;
  a.dev_err = dev_err;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_linear_attention_backward(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_linear_attention_backward launch");
  return ok();
}

int attnres_linear_attention_step(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, int B, int H, int Dk, int Dv, int dtype, const float* log_decay,
                                  float* state, int num_slots, const int32_t* slots, float scale, void* out,
                                  int64_t out_stride, void* stream) {
  if (B < 0 || num_slots < 0) return fail(ATTNRES_EINVAL, "B=%d num_slots=%d", B, num_slots);
  if (B > 65535) return fail(ATTNRES_ERANGE, "B=%d", B);
  int rc = check_la(q, q_stride, k, k_stride, v, v_stride, B, H, Dk, Dv, dtype, log_decay, slots, 1, scale);
  if (rc != ATTNRES_OK) return rc;
  if (!stride_ok(out_stride, (int64_t)H * Dv)) return fail(ATTNRES_EINVAL, "out_stride is shorter than its row");
  if (!span_ok(B, out_stride)) return fail(ATTNRES_ERANGE, "B*stride too large");
  if (!slots && B > num_slots) return fail(ATTNRES_EINVAL, "B=%d rows for %d slots", B, num_slots);
  if (B == 0 || num_slots == 0) return ok();
  if (!state || !out) return fail(ATTNRES_EINVAL, "state/out is NULL");
  {
    const int64_t es = dtype_bytes(dtype), st = (int64_t)num_slots * H * Dk * Dv * 4;
    const Rows in[5] = {{q, B, (int64_t)H * Dk * es, q_stride * es},
                        {k, B, (int64_t)H * Dk * es, k_stride * es},
                        {v, B, (int64_t)H * Dv * es, v_stride * es},
                        {log_decay, 1, H * 4LL, H * 4LL},
                        {slots, 1, B * 4LL, B * 4LL}};
    const Rows outs[2] = {{out, B, (int64_t)H * Dv * es, out_stride * es}, {state, 1, st, st}};
    rc = check_apart(in, 5, outs, 2, nullptr);
    if (rc != ATTNRES_OK) return rc;
  }
  LinAttnStepArgs a{};
  a.q = q;
  a.qs = q_stride;
  a.k = k;
  a.ks = k_stride;
  a.v = v;
  a.vs = v_stride;
  a.B = B;
  a.H = H;
  a.Dk = Dk;
  a.Dv = Dv;
  a.dtype = dtype;
  a.log_decay = log_decay;
  a.state = state;
  a.num_slots = num_slots;
  a.slots = slots;
  a.scale = scale;
  a.out = out;
  a.os = out_stride;
  const cudaError_t e = (a.stream = static_cast<cudaStream_t>(stream), launch_linear_attention_step(a));
  if (e != cudaSuccess) return cuda_fail(e, "attnres_linear_attention_step launch");
  return ok();
}

int attnres_layer_norm(const void* x, int64_t x_stride, int64_t T, int d, int dtype, const float* gain, const float* bias,
                       float eps, void* out, int64_t out_stride, void* stream) {
  int rc = check_ln(x, x_stride, T, d, dtype, eps);
  if (rc == ATTNRES_OK) rc = check_words({gain, bias});
  if (rc != ATTNRES_OK) return rc;
  if (!stride_ok(out_stride, d)) return fail(ATTNRES_EINVAL, "a row stride is shorter than its row");
  if (!span_ok(T, out_stride)) return fail(ATTNRES_ERANGE, "T*stride too large");
  if (T == 0) return ok();
  if (!out) return fail(ATTNRES_EINVAL, "out is NULL");
  const int64_t es = dtype_bytes(dtype), w = d * es;
  if (!aligned(out, (int)es)) return fail(ATTNRES_EINVAL, "a tensor is not aligned to its elements");
  {
    const Rows in[3] = {{x, T, w, x_stride * es}, {gain, 1, d * 4LL, d * 4LL}, {bias, 1, d * 4LL, d * 4LL}};
    const Rows outs[1] = {{out, T, w, out_stride * es}};
    const int in_place[1] = {0};
    const int ra = check_apart(in, 3, outs, 1, in_place);
    if (ra != ATTNRES_OK) return ra;
  }
  LayerNormArgs a{};
  a.x = x;
  a.xs = x_stride;
  a.out = out;
  a.os = out_stride;
  a.gain = gain;
  a.bias = bias;
  a.T = T;
  a.d = d;
  a.dtype = dtype;
  a.eps = eps;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_layer_norm(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_layer_norm launch");
  return ok();
}

int64_t attnres_layer_norm_backward_workspace_size(int64_t T, int d) {
  if (T < 0 || d < 1) return fail(ATTNRES_EINVAL, "T=%lld d=%d", (long long)T, d);
  if (d > kMaxNormWidth) return fail(ATTNRES_ERANGE, "d=%d", d);
  const int64_t n = layer_norm_backward_workspace_bytes(T, d);
  if (n < 0) return fail(ATTNRES_ECUDA, "device query");
  ok();
  return n;
}

int attnres_layer_norm_backward(const void* x, int64_t x_stride, int64_t T, int d, int dtype, const float* gain, float eps,
                                const void* grad_out, int64_t grad_out_stride, void* grad_x, int64_t grad_x_stride,
                                float* grad_gain, float* grad_bias, void* workspace, int64_t workspace_bytes, void* stream) {
  int rc = check_ln(x, x_stride, T, d, dtype, eps);
  if (rc == ATTNRES_OK) rc = check_words({gain, grad_gain, grad_bias});
  if (rc != ATTNRES_OK) return rc;
  const int64_t es = dtype_bytes(dtype), w = d * es, vec = d * 4LL;
  if (!stride_ok(grad_out_stride, d) || !stride_ok(grad_x_stride, d))
    return fail(ATTNRES_EINVAL, "a row stride is shorter than its row");
  if (!span_ok(T, grad_out_stride) || !span_ok(T, grad_x_stride)) return fail(ATTNRES_ERANGE, "T*stride too large");
  if (!grad_x && !grad_gain && !grad_bias) return ok();
  if (T > 0 && !grad_out) return fail(ATTNRES_EINVAL, "grad_out is NULL");
  if (!aligned(grad_out, (int)es) || !aligned(grad_x, (int)es)) return fail(ATTNRES_EINVAL, "a tensor is not aligned to its elements");
  {
    const int64_t wsb = workspace && workspace_bytes > 0 ? workspace_bytes : 0;
    const Rows in[3] = {{grad_out, T, w, grad_out_stride * es}, {x, T, w, x_stride * es}, {gain, 1, vec, vec}};
    const Rows out[4] = {{grad_x, T, w, grad_x_stride * es}, {grad_gain, 1, vec, vec}, {grad_bias, 1, vec, vec}, {workspace, 1, wsb, wsb}};
    const int in_place[4] = {0, -1, -1, -1};
    rc = check_apart(in, 3, out, 4, in_place);
    if (rc != ATTNRES_OK) return rc;
  }
  if (T > 0 && (grad_gain || grad_bias)) {
    if (!workspace) return fail(ATTNRES_EINVAL, "the gain and bias gradients need a workspace");
    const int64_t need = layer_norm_backward_workspace_bytes(T, d);
    if (need < 0) return fail(ATTNRES_ECUDA, "device query");
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != ATTNRES_OK) return rc;
  }
  LayerNormArgs a{};
  a.x = x;
  a.xs = x_stride;
  a.dy = grad_out;
  a.dys = grad_out_stride;
  a.out = grad_x;
  a.os = grad_x_stride;
  a.gain = gain;
  a.dgain = grad_gain;
  a.dbias = grad_bias;
  a.T = T;
  a.d = d;
  a.dtype = dtype;
  a.eps = eps;
  a.backward = true;
  a.workspace = static_cast<float*>(workspace);
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_layer_norm(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_layer_norm_backward launch");
  return ok();
}

int attnres_gated_recurrence(const void* x, int64_t x_stride, const void* forget, int64_t forget_stride, const void* gate,
                             int64_t gate_stride, int64_t T, int C, int dtype, const int32_t* cu_seqlens, int num_seqs,
                             const float* initial_state, float* final_state, void* out, int64_t out_stride,
                             float* chunk_states, int* dev_err, void* stream) {
  int rc = check_gr(x, x_stride, forget, forget_stride, gate, gate_stride, T, C, dtype, cu_seqlens, num_seqs);
  if (rc != ATTNRES_OK) return rc;
  if (T > 0 && !out) return fail(ATTNRES_EINVAL, "out is NULL");
  rc = check_gr_rows(out, out_stride, T, C, dtype);
  if (rc == ATTNRES_OK) rc = check_words({cu_seqlens, initial_state, final_state, chunk_states, dev_err});
  if (rc != ATTNRES_OK) return rc;
  if (T == 0 && !final_state) return ok();
  {
    const int64_t es = dtype_bytes(dtype), w = C * es, st = (int64_t)num_seqs * C * 4, cub = (num_seqs + 1) * 4LL;
    const int64_t ch = (T + ATTNRES_RECURRENCE_CHUNK - 1) / ATTNRES_RECURRENCE_CHUNK * C * 4;
    const Rows in[5] = {{x, T, w, x_stride * es}, {forget, T, w, forget_stride * es}, {gate, T, w, gate_stride * es},
                        {cu_seqlens, 1, cub, cub}, {initial_state, 1, st, st}};
    const Rows outs[3] = {{out, T, w, out_stride * es}, {final_state, 1, st, st}, {chunk_states, 1, ch, ch}};
    const int in_place[3] = {-1, 4, -1};
    rc = check_apart(in, 5, outs, 3, in_place);
    if (rc != ATTNRES_OK) return rc;
  }
  RecurrenceArgs a{};
  a.x = x;
  a.xs = x_stride;
  a.f = forget;
  a.fs = forget_stride;
  a.g = gate;
  a.gs = gate_stride;
  a.T = T;
  a.C = C;
  a.dtype = dtype;
  a.cu = cu_seqlens;
  a.N = num_seqs;
  a.s0 = initial_state;
  a.s1 = final_state;
  a.out = out;
  a.os = out_stride;
  a.chunk = T > 0 ? chunk_states : nullptr;
  a.dev_err = dev_err;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_gated_recurrence(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_gated_recurrence launch");
  return ok();
}

int attnres_gated_recurrence_backward(const void* x, int64_t x_stride, const void* forget, int64_t forget_stride,
                                      const void* gate, int64_t gate_stride, int64_t T, int C, int dtype,
                                      const int32_t* cu_seqlens, int num_seqs, const float* initial_state,
                                      const float* chunk_states, const void* grad_out, int64_t grad_out_stride,
                                      const float* grad_final_state, void* grad_x, int64_t grad_x_stride, void* grad_forget,
                                      int64_t grad_forget_stride, void* grad_gate, int64_t grad_gate_stride,
                                      float* grad_initial_state, int* dev_err, void* stream) {
  int rc = check_gr(x, x_stride, forget, forget_stride, gate, gate_stride, T, C, dtype, cu_seqlens, num_seqs);
  if (rc != ATTNRES_OK) return rc;
  if (grad_gate && !gate) return fail(ATTNRES_EINVAL, "grad_gate without gate");
  if (!grad_x && !grad_forget && !grad_gate && !grad_initial_state) return ok();
  if (T == 0 && !grad_initial_state) return ok();
  if (T > 0 && (!grad_out || !chunk_states)) return fail(ATTNRES_EINVAL, "grad_out/chunk_states is NULL");
  rc = check_gr_rows(grad_out, grad_out_stride, T, C, dtype);
  if (rc == ATTNRES_OK) rc = check_gr_rows(grad_x, grad_x_stride, T, C, dtype);
  if (rc == ATTNRES_OK) rc = check_gr_rows(grad_forget, grad_forget_stride, T, C, dtype);
  if (rc == ATTNRES_OK) rc = check_gr_rows(grad_gate, grad_gate_stride, T, C, dtype);
  if (rc == ATTNRES_OK)
    rc = check_words({cu_seqlens, initial_state, chunk_states, grad_final_state, grad_initial_state, dev_err});
  if (rc != ATTNRES_OK) return rc;
  {
    const int64_t es = dtype_bytes(dtype), w = C * es, st = (int64_t)num_seqs * C * 4, cub = (num_seqs + 1) * 4LL;
    const int64_t ch = (T + ATTNRES_RECURRENCE_CHUNK - 1) / ATTNRES_RECURRENCE_CHUNK * C * 4;
    const Rows in[8] = {{x, T, w, x_stride * es}, {forget, T, w, forget_stride * es}, {gate, T, w, gate_stride * es},
                        {cu_seqlens, 1, cub, cub}, {initial_state, 1, st, st}, {chunk_states, 1, ch, ch},
                        {grad_out, T, w, grad_out_stride * es}, {grad_final_state, 1, st, st}};
    const Rows outs[4] = {{grad_x, T, w, grad_x_stride * es}, {grad_forget, T, w, grad_forget_stride * es},
                          {grad_gate, T, w, grad_gate_stride * es}, {grad_initial_state, 1, st, st}};
    const int in_place[4] = {-1, -1, -1, 7};
    rc = check_apart(in, 8, outs, 4, in_place);
    if (rc != ATTNRES_OK) return rc;
  }
  RecurrenceArgs a{};
  a.x = x;
  a.xs = x_stride;
  a.f = forget;
  a.fs = forget_stride;
  a.g = gate;
  a.gs = gate_stride;
  a.T = T;
  a.C = C;
  a.dtype = dtype;
  a.cu = cu_seqlens;
  a.N = num_seqs;
  a.s0 = initial_state;
  a.chunk = const_cast<float*>(chunk_states);
  a.dout = grad_out;
  a.dos = grad_out_stride;
  a.ds1 = grad_final_state;
  a.dx = grad_x;
  a.dxs = grad_x_stride;
  a.df = grad_forget;
  a.dfs = grad_forget_stride;
  a.dg = grad_gate;
  a.dgs = grad_gate_stride;
  a.ds0 = grad_initial_state;
  a.dev_err = dev_err;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_gated_recurrence_backward(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_gated_recurrence_backward launch");
  return ok();
}

int attnres_gated_recurrence_step(const void* x, int64_t x_stride, const void* forget, int64_t forget_stride, const void* gate,
                                  int64_t gate_stride, int B, int C, int dtype, float* state, int num_slots,
                                  const int32_t* slots, void* out, int64_t out_stride, void* stream) {
  if (B < 0 || num_slots < 0) return fail(ATTNRES_EINVAL, "B=%d num_slots=%d", B, num_slots);
  if (B > 65535) return fail(ATTNRES_ERANGE, "B=%d", B);
  int rc = check_gr(x, x_stride, forget, forget_stride, gate, gate_stride, B, C, dtype, nullptr, 1);
  if (rc == ATTNRES_OK) rc = check_gr_rows(out, out_stride, B, C, dtype);
  if (rc == ATTNRES_OK) rc = check_words({state, slots});
  if (rc != ATTNRES_OK) return rc;
  if (!slots && B > num_slots) return fail(ATTNRES_EINVAL, "B=%d rows for %d slots", B, num_slots);
  if (B == 0 || num_slots == 0) return ok();
  if (!state || !out) return fail(ATTNRES_EINVAL, "state/out is NULL");
  {
    const int64_t es = dtype_bytes(dtype), w = C * es, st = (int64_t)num_slots * C * 4;
    const Rows in[4] = {{x, B, w, x_stride * es}, {forget, B, w, forget_stride * es}, {gate, B, w, gate_stride * es},
                        {slots, 1, B * 4LL, B * 4LL}};
    const Rows outs[2] = {{out, B, w, out_stride * es}, {state, 1, st, st}};
    rc = check_apart(in, 4, outs, 2, nullptr);
    if (rc != ATTNRES_OK) return rc;
  }
  RecurrenceStepArgs a{};
  a.x = x;
  a.xs = x_stride;
  a.f = forget;
  a.fs = forget_stride;
  a.g = gate;
  a.gs = gate_stride;
  a.B = B;
  a.C = C;
  a.dtype = dtype;
  a.state = state;
  a.num_slots = num_slots;
  a.slots = slots;
  a.out = out;
  a.os = out_stride;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_gated_recurrence_step(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_gated_recurrence_step launch");
  return ok();
}

int64_t attnres_grad_clip_workspace_size(void) {
  const int64_t n = grad_clip_workspace_bytes();
  if (n < 0) return fail(ATTNRES_ECUDA, "device query");
  ok();
  return n;
}

int attnres_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes, int n,
                      float max_norm, float* out_norm, void* workspace, int64_t workspace_bytes, void* stream) {
  if (n < 0) return fail(ATTNRES_EINVAL, "n=%d", n);
  if (n > kMaxTensors) return fail(ATTNRES_ERANGE, "n=%d", n);
  if (n > 0 && (!grads || !numels || !dtypes)) return fail(ATTNRES_EINVAL, "grads/numels/dtypes is NULL");
  if (outs && !(max_norm >= 0.f)) return fail(ATTNRES_EINVAL, "max_norm must be >= 0");
  if (!out_norm) return fail(ATTNRES_EINVAL, "out_norm is NULL");
  if (!aligned(out_norm, 4)) return fail(ATTNRES_EINVAL, "out_norm is not 4-byte aligned");
  std::unique_ptr<Interval[]> v(new (std::nothrow) Interval[2 * (size_t)n + 2]);
  if (!v) return fail(ATTNRES_ERANGE, "no host memory for a list of %d tensors", n);
  int m = 0;
  auto add = [&](const void* p, int64_t bytes, bool out) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    if (p && bytes > 0) v[m++] = {b, b + (uintptr_t)bytes, out};
  };
  for (int i = 0; i < n; ++i) {
    if (!valid_dtype(dtypes[i])) return fail(ATTNRES_EDTYPE, "tensor %d: dtype %d", i, dtypes[i]);
    if (numels[i] < 0) return fail(ATTNRES_EINVAL, "tensor %d: %lld elements", i, (long long)numels[i]);
    if (numels[i] > kMaxElems) return fail(ATTNRES_ERANGE, "tensor %d: %lld elements", i, (long long)numels[i]);
    if (numels[i] == 0) continue;
    const int es = (int)dtype_bytes(dtypes[i]);
    if (!grads[i] || (outs && !outs[i])) return fail(ATTNRES_EINVAL, "tensor %d is NULL", i);
    if (!aligned(grads[i], es) || (outs && !aligned(outs[i], es)))
      return fail(ATTNRES_EINVAL, "tensor %d is not aligned to its elements", i);
    const bool same = outs && outs[i] == grads[i];
    if (!same) add(grads[i], numels[i] * es, false);
    if (outs) add(outs[i], numels[i] * es, true);
  }
  add(out_norm, 4, true);
  if (workspace && workspace_bytes > 0) add(workspace, workspace_bytes, true);
  if (!intervals_apart(v.get(), m)) return fail(ATTNRES_EINVAL, "an output overlaps another tensor of the call");
  const int64_t need = grad_clip_workspace_bytes();
  if (need < 0) return fail(ATTNRES_ECUDA, "device query");
  const int rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != ATTNRES_OK) return rc;
  GradClipArgs a{};
  a.grads = grads;
  a.outs = outs;
  a.numels = numels;
  a.dtypes = dtypes;
  a.n = n;
  a.max_norm = max_norm;
  a.norm = out_norm;
  a.workspace = static_cast<double*>(workspace);
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_grad_clip(a);
  if (e != cudaSuccess) return cuda_fail(e, "attnres_grad_clip launch");
  return ok();
}

}  // extern "C"
