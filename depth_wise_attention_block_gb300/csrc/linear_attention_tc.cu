// The scan of linear attention (linear_attention.cu) on the tensor cores:
// bf16 tensors with head sizes of 64 or 128, in chunks of 128 tokens.
//
//   P    = a b^T, masked and decayed       scores of the chunk   [128 x 128]
//   out  = P c + l^{i+1} (a S)             S: the state before it
//   U    = sum_j l^{C-1-j} b_j c_j^T,      S <- l^C S + U
//
// Every product is a tcgen05.mma with its accumulator in TMEM.  a, b and c
// arrive by TMA in the 128-byte swizzle and serve K-major (a b^T, a S) or
// MN-major (P c, the token sums) from the same tile.  Four warps turn the
// scores into P (bf16, back into TMEM as the next product's operand) and
// write the outputs; four warps hold the state in fp32 registers (one row of
// Da per thread), give it to the products rounded to bf16, and weigh b with
// the decays: the weighted rows enter as three bf16 terms (24 bits), so that
// the state keeps fp32 precision over any number of chunks; each chunk's U
// starts from zero in TMEM and is added in fp32 round-to-nearest.
//
// A reversed scan (gradients of k and v) takes the chunks from the end and
// mirrors the mask and the powers; nothing is reordered in memory.
//
// Few heads and sequences do not fill the GPU.  A long sequence is then cut
// into segments: scan_tc_kernel<STATE> forms every segment's own state (it
// reads b and c only), la_combine_kernel runs through the segments and
// leaves the state before each, and the scan runs over all segments at once.
//
// Bound: HBM.  A chunk of 128 x 128 heads takes 6 x 512 cycles of the tensor
// cores against about 5500 cycles of HBM time per SM.
#include <math.h>

#include "attnres.h"
#include "body.h"
#include "device_common.cuh"
#include "launch.h"
#include "linear_attention.cuh"
#include "tc_common.cuh"

namespace attnres {

namespace {

constexpr int kC = kScanChunk;         // tokens per chunk
constexpr int kTileThreads = 320;      // 4 warps scores and outputs, 4 state, TMA, MMA
constexpr int kMaxSlots = 8;
constexpr int kPanel = kC * 128;       // bytes of 64 channels of a tile

struct Segment {
  int seq, first, len, last;  // sequence, first token, tokens, whether the sequence ends with it
};

struct ScanTcParams {
  CUtensorMap ma, mb, mc;
  ScanArgs s;
  const Segment* segs;   // null: segment = sequence, or arithmetic over one sequence
  const int* nsegs;
  int seg_len;           // tokens per segment (0: a sequence is one segment)
  float* seg_state;      // [segment][H][..]: STATE writes each segment's own, the scan reads the state before it
  int slots;
  int* dev_err;
  unsigned long long wait_ns;
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

__device__ __forceinline__ Segment segment_of(const ScanTcParams& p, int i) {
  if (p.segs) return p.segs[i];
  if (p.s.cu) return cut(i, seq_range(p.s.cu, i, p.s.T), 0, 0, p.s.reverse);
  return cut(0, {0, p.s.T}, i, p.seg_len, p.s.reverse);
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] x B[smem]^T
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 32 bytes: a whole sector per thread
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
               "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// STATE: the segments' own states only (b and c; no scores, no outputs).
template <int DA, int DC, bool STATE>
__global__ void __launch_bounds__(kTileThreads, 1) scan_tc_kernel(const __grid_constant__ ScanTcParams p) {
  constexpr int kTile = kC * (DA > DC ? DA : DC) * 2;  // bytes of a slot
  constexpr int kTiles = STATE ? 2 : 3;                // tiles per chunk: (a,) b, c
  constexpr int kSplitWarps = STATE ? 8 : 4;
  constexpr uint32_t kColP = 0, kColO1 = 128, kColO2 = 256, kColU = 384;  // TMEM columns
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxSlots], empty[kMaxSlots], p_full, p_ready, o_full, o_free, s_ready, b_ready, u_full, u_free;
  __shared__ uint32_t tmem_base;
  __shared__ float tab[kC], pw[kC + 2];  // p_scale l^k; l^k
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t s_buf = base + p.slots * kTile, mid = s_buf + (STATE ? 0 : DC * DA * 2), lo = mid + kC * DA * 2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.s.H, seg_i = blockIdx.x / p.s.H;

  if (tid == 0) {
    for (int s = 0; s < p.slots; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), 1);
    }
    mbar_init(smem_addr(&p_full), 1);
    mbar_init(smem_addr(&p_ready), 4);
    mbar_init(smem_addr(&o_full), 1);
    mbar_init(smem_addr(&o_free), 4);
    mbar_init(smem_addr(&s_ready), 4);
    mbar_init(smem_addr(&b_ready), kSplitWarps);
    mbar_init(smem_addr(&u_full), 1);
    mbar_init(smem_addr(&u_free), 4);
    mbar_fence_init();
  }
  if (warp == 9) tmem_alloc(smem_addr(&tmem_base), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_wait();
  pdl_trigger();
  const float g = __ldg(p.s.log_decay + h);
  if (tid < kC + 2) {
    const float l = expf(g * (float)tid);
    pw[tid] = l;
    if (tid < kC) tab[tid] = p.s.p_scale * l;
  }
  __syncthreads();
  const bool live = !p.nsegs || seg_i < *p.nsegs;
  Segment sg{0, 0, 0, 0};
  if (live) sg = segment_of(p, seg_i);
  const bool work = live && !(STATE && sg.last);  // nothing needs the state behind the last segment but its own scan
  const int nchunk = work ? (sg.len + kC - 1) / kC : 0;
  const bool rev = p.s.reverse;
  // chunk n's first token and length (a reversed scan's short chunk is its last)
  auto chunk_len = [&](int n) { return sg.len - n * kC < kC ? sg.len - n * kC : kC; };
  auto chunk_at = [&](int n) { return rev ? sg.first + sg.len - n * kC - chunk_len(n) : sg.first + n * kC; };
  // once a wait runs out, the others of this thread return at once
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_wait_bounded(smem_addr(bar), parity & 1u, p.wait_ns)) {
      report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
      ok = false;
    }
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    wait(bar, parity);
    ok = __all_sync(0xffffffffu, ok);
  };

  if (warp == 8) {
    if (lane == 0) {
      int it = 0;
      for (int n = 0; n < nchunk && ok; ++n) {
        const int t = chunk_at(n);
        for (int k = 0; k < kTiles; ++k, ++it) {
          const int st = it % p.slots;
          wait(&empty[st], (uint32_t)(it / p.slots) + 1u);
          if (!ok) break;
          const int which = STATE ? k + 1 : k;
          const int D = which == 2 ? DC : DA;
          const CUtensorMap* m = which == 0 ? &p.ma : which == 1 ? &p.mb : &p.mc;
          const uint32_t fb = smem_addr(&full[st]);
          mbar_arrive_expect_tx(fb, D * kC * 2);
          for (int x = 0; x < D; x += 64) tma_load_2d(base + st * kTile + x / 64 * kPanel, m, h * D + x, t, fb);
        }
      }
      // the CTA never exits under a copy
      const int armed = it < p.slots ? it : p.slots;
      for (int st = 0; st < armed; ++st) mbar_wait_bounded(smem_addr(&full[st]), (uint32_t)((it - 1 - st) / p.slots) & 1u);
    }
    __syncwarp();
  } else if (warp == 9) {
    if (lane == 0) {
      constexpr uint32_t kI1 = tc_idesc_bf16(128, 128), kI2 = tc_idesc_bf16(128, DC, false, true), kI3 = tc_idesc_bf16(128, DC),
                         kI4 = tc_idesc_bf16(128, DA, true, true);
      for (int n = 0; n < nchunk && ok; ++n) {
        const int it = n * kTiles;
        const int sa = it % p.slots, sb = (it + kTiles - 2) % p.slots, sc = (it + kTiles - 1) % p.slots;
        const uint32_t A = base + sa * kTile, B = base + sb * kTile, Ct = base + sc * kTile;
        auto lap = [&](int i) { return (uint32_t)(i / p.slots); };
        const uint32_t ph = (uint32_t)n;
        if constexpr (!STATE) {
          // P's columns are free once the last chunk's P c is done
          if (n > 0) wait(&o_full, ph - 1);
          wait(&full[sa], lap(it));
          wait(&full[sb], lap(it + 1));
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < DA / 16; ++kk) {
            const uint32_t off = kk / 4 * kPanel + kk % 4 * 32;
            tc_mma_bf16(tmem + kColP, smem_desc_k128(A + off), smem_desc_k128(B + off), kI1, kk > 0);
          }
          tc_commit(smem_addr(&p_full));
          wait(&s_ready, ph);
          wait(&o_free, ph + 1);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < DA / 16; ++kk)
            tc_mma_bf16(tmem + kColO2, smem_desc_k128(A + kk / 4 * kPanel + kk % 4 * 32),
                        smem_desc_k128(s_buf + kk / 4 * (DC * 128) + kk % 4 * 32), kI3, kk > 0);
          tc_commit(smem_addr(&empty[sa]));
          wait(&full[sc], lap(it + 2));
          // rows behind a short chunk's end are cleared with the weighted rows
          if (chunk_len(n) < kC) wait(&b_ready, ph);
          wait(&p_ready, ph);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kC / 16; ++kk)
            tc_mma_bf16_ts(tmem + kColO1, tmem + kColP + kk * 8, smem_desc_mn128(Ct + kk * 2048, kPanel), kI2, kk > 0);
          tc_commit(smem_addr(&o_full));
        } else {
          wait(&full[sc], lap(it + 1));
        }
        wait(&b_ready, ph);
        wait(&u_free, ph + 1);
        tc_fence_after();
        // c's channels as the 128 rows (64 channels: the other 64 rows are
        // whatever lies behind, and are not read)
#pragma unroll
        for (int term = 0; term < 3; ++term) {
          const uint32_t bt = term == 0 ? B : term == 1 ? mid : lo;
#pragma unroll
          for (int kk = 0; kk < kC / 16; ++kk)
            tc_mma_bf16(tmem + kColU, smem_desc_mn128(Ct + kk * 2048, kPanel), smem_desc_mn128(bt + kk * 2048, kPanel), kI4,
                        term > 0 || kk > 0);
        }
        tc_commit(smem_addr(&empty[sb]));
        tc_commit(smem_addr(&empty[sc]));
        tc_commit(smem_addr(&u_full));
      }
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes_at = tmem + ((uint32_t)(32 * quarter) << 16);
    // b's rows times their decay, as three bf16 terms (hi over b itself)
    auto split = [&](int n, int threads, int t0) {
      const int len = chunk_len(n);
      const uint32_t B = base + (n * kTiles + kTiles - 2) % p.slots * kTile, Ct = base + (n * kTiles + kTiles - 1) % p.slots * kTile;
#pragma unroll 2
      for (int v = t0; v < kC * DA / 8; v += threads) {
        const int j = (v / 8) % kC;
        const uint32_t at = v * 16;
        if (j < len) {
          const float f = p.s.up_scale * pw[rev ? j + p.s.shift : len - 1 - j + p.s.shift];
          const uint4 w = ld_shared_v4(B + at);
          const uint32_t in[4] = {w.x, w.y, w.z, w.w};
          uint32_t th[4], tm[4], tl[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x = bf16lo(in[k]) * f, y = bf16hi(in[k]) * f;
            th[k] = pack_bf16x2(x, y);
            const float x1 = x - bf16lo(th[k]), y1 = y - bf16hi(th[k]);
            tm[k] = pack_bf16x2(x1, y1);
            tl[k] = pack_bf16x2(x1 - bf16lo(tm[k]), y1 - bf16hi(tm[k]));
          }
          st_shared_v4(B + at, th[0], th[1], th[2], th[3]);
          st_shared_v4(mid + at, tm[0], tm[1], tm[2], tm[3]);
          st_shared_v4(lo + at, tl[0], tl[1], tl[2], tl[3]);
        } else {  // behind the chunk's end: another chunk's or sequence's rows
          st_shared_v4(B + at, 0, 0, 0, 0);
          st_shared_v4(mid + at, 0, 0, 0, 0);
          st_shared_v4(lo + at, 0, 0, 0, 0);
        }
      }
      for (int v = t0 + len * 8; v < kC * 8; v += threads)
        for (int x = 0; x < DC / 64; ++x) st_shared_v4(Ct + x * kPanel + v * 16, 0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&b_ready));
    };

    if (warp < 4) {
      if constexpr (STATE) {
        for (int n = 0; n < nchunk; ++n) {
          if (n > 0) warp_wait(&u_full, n - 1);
          const int i1 = n * 2;
          warp_wait(&full[i1 % p.slots], (uint32_t)(i1 / p.slots));
          warp_wait(&full[(i1 + 1) % p.slots], (uint32_t)((i1 + 1) / p.slots));
          split(n, 256, tid);
        }
      } else {
        for (int n = 0; n < nchunk; ++n) {
          const int len = chunk_len(n);
          warp_wait(&p_full, n);
          tc_fence_after();
#pragma unroll 2
          for (int j0 = 0; j0 < kC; j0 += 16) {
            uint32_t w[8];
            // blocks that the mask leaves empty for all of the warp's rows
            if (rev ? j0 + 15 < 32 * quarter || j0 >= len : j0 > 32 * quarter + 31) {
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = 0;
            } else {
              uint32_t v[16];
              tmem_ld16(lanes_at + kColP + j0, v);
              tmem_ld_wait();
              float f[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const int j = j0 + k, d = rev ? j - row : row - j;
                f[k] = d >= 0 && (!rev || j < len) ? __uint_as_float(v[k]) * tab[d & (kC - 1)] : 0.f;
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
            }
            tmem_st8(lanes_at + kColP + j0 / 2, w);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&p_ready));

          warp_wait(&o_full, n);
          tc_fence_after();
          const bool in = row < len;
          const int e = rev ? len - row - p.s.shift : row + 1 - p.s.shift;
          const float coef = in ? p.s.in_scale * pw[e] : 0.f;
          bf16_t* out = static_cast<bf16_t*>(p.s.out) + (long long)(chunk_at(n) + row) * p.s.os + (long long)h * DC;
#pragma unroll 2
          for (int c0 = 0; c0 < DC; c0 += 16) {
            uint32_t x[16], y[16];
            tmem_ld16(lanes_at + kColO1 + c0, x);
            tmem_ld16(lanes_at + kColO2 + c0, y);
            tmem_ld_wait();
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              w[k] = ok ? pack_bf16x2(fmaf(coef, __uint_as_float(y[2 * k]), __uint_as_float(x[2 * k])),
                                      fmaf(coef, __uint_as_float(y[2 * k + 1]), __uint_as_float(x[2 * k + 1])))
                        : 0x7fc07fc0u;
            if (in) {
              if (p.s.wide_out) {
                st_global_v8(out + c0, w);
              } else {
                *reinterpret_cast<uint4*>(out + c0) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4*>(out + c0 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&o_free));
        }
      }
    } else {
      // the state: thread `row` holds S[0 .. DA)[row]
      float S[DA];
      const long long st = ((long long)(p.seg_state ? seg_i : sg.seq) * p.s.H + h) * DA * DC;
      const float* from = STATE ? nullptr : p.seg_state ? p.seg_state : p.s.s_in;
      const bool mine = row < DC && live;
      if (from && mine) {
        if (p.s.transposed) {
#pragma unroll
          for (int d = 0; d < DA; d += 4) {
            const float4 v = *reinterpret_cast<const float4*>(from + st + (long long)row * DA + d);
            S[d] = v.x, S[d + 1] = v.y, S[d + 2] = v.z, S[d + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int d = 0; d < DA; ++d) S[d] = from[st + d * DC + row];
        }
      } else {
#pragma unroll
        for (int d = 0; d < DA; ++d) S[d] = 0.f;
      }
      for (int n = 0; n < nchunk; ++n) {
        if constexpr (!STATE) {
          // rounded to bf16 for a S, [DC rows][DA] in the 128-byte swizzle
          // (chunk n - 1's a S was done before its U, waited for below)
          if (row < DC) {
#pragma unroll
            for (int d = 0; d < DA; d += 8)
              st_shared_v4(s_buf + d / 64 * (DC * 128) + row * 128 + (((d / 8) ^ row) & 7) * 16, pack_bf16x2(S[d], S[d + 1]),
                           pack_bf16x2(S[d + 2], S[d + 3]), pack_bf16x2(S[d + 4], S[d + 5]), pack_bf16x2(S[d + 6], S[d + 7]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&s_ready));
        }
        const int ib = n * kTiles + kTiles - 2;
        warp_wait(&full[ib % p.slots], (uint32_t)(ib / p.slots));
        if (STATE || chunk_len(n) < kC) warp_wait(&full[(ib + 1) % p.slots], (uint32_t)((ib + 1) / p.slots));
        if constexpr (!STATE) warp_wait(&p_full, n);  // a b^T has read b
        split(n, 32 * kSplitWarps, STATE ? tid : tid - 128);
        warp_wait(&u_full, n);
        tc_fence_after();
        const float decay = expf(g * (float)chunk_len(n));
#pragma unroll
        for (int d = 0; d < DA; d += 16) {
          uint32_t v[16];
          tmem_ld16(lanes_at + kColU + d, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) S[d + k] = fmaf(S[d + k], decay, __uint_as_float(v[k]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&u_free));
      }
      // STATE: the segment's own state; the scan: behind a sequence's end
      const bool emit = STATE ? work : live && sg.last && p.s.s_out;
      if (emit && mine) {
        float* to = STATE ? p.seg_state : p.s.s_out;
        const long long at = STATE ? st : ((long long)sg.seq * p.s.H + h) * DA * DC;
        const float nan = __int_as_float(0x7fc00000);
        if (p.s.transposed) {
#pragma unroll
          for (int d = 0; d < DA; d += 4)
            *reinterpret_cast<float4*>(to + at + (long long)row * DA + d) =
                ok ? make_float4(S[d], S[d + 1], S[d + 2], S[d + 3]) : make_float4(nan, nan, nan, nan);
        } else {
#pragma unroll
          for (int d = 0; d < DA; ++d) to[at + d * DC + row] = ok ? S[d] : nan;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The segments of a ragged batch, in order: one thread per sequence counts,
// a prefix sum places them.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) la_plan_kernel(const int32_t* cu, int N, long long T, int seg_len, bool reverse, Segment* segs,
                                                               int* first_of, int* nsegs) {
  __shared__ int sums[32];
  __shared__ int carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if (tid == 0) carry = 0;
  for (int n0 = 0; n0 < N; n0 += kPlanThreads) {
    const int n = n0 + tid;
    SeqRange r{0, 0};
    int cnt = 0;
    if (n < N) {
      r = seq_range(cu, n, T);
      cnt = r.len > seg_len ? (int)((r.len + seg_len - 1) / seg_len) : 1;
    }
    int x = cnt;
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int y = sums[lane];
      for (int o = 1; o < 32; o *= 2) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      sums[lane] = y;
    }
    __syncthreads();
    const int at = carry + (warp ? sums[warp - 1] : 0) + x - cnt;
    // offsets that decrease could ask for more segments than there are rows: none past the table
    const long long cap = (T + seg_len - 1) / seg_len + N;
    if (n < N) first_of[n] = (int)(at < cap ? at : cap);
    for (int i = 0; i < cnt && at + i < cap; ++i) segs[at + i] = cut(n, r, i, seg_len, reverse);
    const int total = sums[31];
    __syncthreads();
    if (tid == 0) carry += total;
    __syncthreads();
  }
  if (tid == 0) {
    const long long cap = (T + seg_len - 1) / seg_len + N;
    const int total = (int)(carry < cap ? carry : cap);
    first_of[N] = total;
    *nsegs = total;
  }
}

// Per sequence and head: the state before each segment, from the segments'
// own states, in place (and in order).
__global__ void __launch_bounds__(256) la_combine_kernel(const __grid_constant__ ScanTcParams p, const int* first_of, int per_head) {
  const long long e = (blockIdx.x * 256LL + threadIdx.x) * 4;  // over [H][Da Dc]
  const int n = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const long long all = (long long)p.s.H * per_head;
  if (e >= all) return;
  const float g = __ldg(p.s.log_decay + (int)(e / per_head));
  const int s0 = first_of ? first_of[n] : 0;
  const int s1 = first_of ? first_of[n + 1] : (int)((p.s.T + p.seg_len - 1) / p.seg_len);
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.s.s_in) {
    const float* in = p.s.s_in + n * all + e;
    w = make_float4(in[0], in[1], in[2], in[3]);
  }
  for (int s = s0; s < s1; ++s) {
    float4* at = reinterpret_cast<float4*>(p.seg_state + s * all + e);
    const Segment sg = segment_of(p, s);
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!sg.last) u = *at;
    *at = w;
    const float d = expf(g * (float)sg.len);
    w = make_float4(fmaf(w.x, d, u.x), fmaf(w.y, d, u.y), fmaf(w.z, d, u.z), fmaf(w.w, d, u.w));
  }
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

struct Layout {
  int64_t segs, table, first, states, total;  // segments at most; bytes
};
Layout layout(int64_t T, int H, int Dk, int Dv, int N, int seg_len) {
  Layout L{};
  if (seg_len == 0) return L;
  L.segs = up(T, seg_len) / seg_len + N;
  L.table = up(L.segs * (int64_t)sizeof(Segment), 256);
  L.first = up((N + 2) * 4, 256);
  L.states = up(L.segs * H * (int64_t)Dk * Dv * 4, 256);
  L.total = L.table + L.first + L.states;
  return L;
}

template <int DA, int DC, bool STATE>
cudaError_t launch_tile(ScanTcParams& p, int64_t segs, const DeviceInfo& di, cudaStream_t stream) {
  constexpr int kTile = kC * (DA > DC ? DA : DC) * 2;
  const int fixed = (STATE ? 0 : DC * DA * 2) + 2 * kC * DA * 2 + 1024;
  const int smem_max = di.max_smem_optin - 2560;  // barriers and power tables are static
  p.slots = (smem_max - fixed) / kTile;
  if (p.slots > kMaxSlots) p.slots = kMaxSlots;
  if (p.slots < (STATE ? 2 : 3)) return cudaErrorInvalidValue;
  static SmemOptIn optin;
  const cudaError_t e = optin.ensure(reinterpret_cast<const void*>(scan_tc_kernel<DA, DC, STATE>), smem_max);
  if (e != cudaSuccess) return e;
  return launch_kernel(scan_tc_kernel<DA, DC, STATE>, dim3((unsigned)(segs * p.s.H)), dim3(kTileThreads), (size_t)(fixed + p.slots * kTile),
                       stream, p);
}

template <bool STATE>
cudaError_t launch_dims(ScanTcParams& p, int64_t segs, const DeviceInfo& di, cudaStream_t stream) {
  if (p.s.Da == 128) return p.s.Dc == 128 ? launch_tile<128, 128, STATE>(p, segs, di, stream) : launch_tile<128, 64, STATE>(p, segs, di, stream);
  return p.s.Dc == 128 ? launch_tile<64, 128, STATE>(p, segs, di, stream) : launch_tile<64, 64, STATE>(p, segs, di, stream);
}

bool token_map(CUtensorMap* m, const void* ptr, int64_t T, int64_t width, int64_t stride) {
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)T};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, kC};
  return make_tensor_map(m, ptr, 2, dims, strides, box);
}

}  // namespace

bool scan_tc_dims(int Dk, int Dv, int dtype) { return dtype == ATTNRES_BF16 && (Dk == 64 || Dk == 128) && (Dv == 64 || Dv == 128); }

// Tokens per segment (0: every sequence in one piece), by a count of chunks:
// a wave of segments takes their chunks and about two more to start and end;
// the segments' own states cost half of a scan, and the launches about 4
// chunks.  The lengths are on the device, so the longest sequence is taken
// to be all T tokens.
int scan_tc_segment(int64_t T, int H, int N, int sm_count) {
  const int64_t chunks = up(T, kC) / kC;
  const double even = (double)H * (double)(chunks + N) / sm_count;  // chunks per SM if all were equal
  double best = (double)(chunks > even ? chunks : even) + 2;
  int seg = 0;
  for (int64_t c = 2; c < chunks; c += c < 16 ? 1 : c / 8) {
    const int64_t ctas = H * (up(chunks, c) / c + N - 1);
    const double cost = (double)((ctas + sm_count - 1) / sm_count) * ((double)c + 2) * 1.5 + 4;
    if (cost < best) {
      best = cost;
      seg = (int)(c * kC);
    }
  }
  return seg;
}

int64_t scan_tc_workspace(int64_t T, int H, int Dk, int Dv, int N) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return -1;
  return layout(T, H, Dk, Dv, N, scan_tc_segment(T, H, N, di.sm_count)).total;
}

bool scan_tc_ok(const ScanArgs& s) {
  auto rows = [](const void* p, long long stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; };
  auto state = [](const float* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  return rows(s.a, s.as) && rows(s.b, s.bs) && rows(s.c, s.cs) && rows(s.out, s.os) && state(s.s_in) && state(s.s_out) && s.T > 0 &&
         s.T * 2 < INT32_MAX && ((s.T + kC - 1) / kC + s.N) * s.H < INT32_MAX;
}

cudaError_t launch_scan_tc(const ScanArgs& s, void* workspace, bool states_ready, int* dev_err, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  ScanTcParams p{};
  p.s = s;
  p.s.wide_out = (reinterpret_cast<uintptr_t>(s.out) & 31) == 0 && s.os % 16 == 0;
  if (!token_map(&p.ma, s.a, s.T, (int64_t)s.H * s.Da, s.as) || !token_map(&p.mb, s.b, s.T, (int64_t)s.H * s.Da, s.bs) ||
      !token_map(&p.mc, s.c, s.T, (int64_t)s.H * s.Dc, s.cs))
    return cudaErrorInvalidValue;
  p.dev_err = dev_err;
  p.wait_ns = wait_limit_ns();
  p.seg_len = scan_tc_segment(s.T, s.H, s.N, di.sm_count);
  const Layout L = layout(s.T, s.H, s.Da, s.Dc, s.N, p.seg_len);
  int64_t segs = s.N;
  if (p.seg_len > 0) {
    char* ws = static_cast<char*>(workspace);
    Segment* table = reinterpret_cast<Segment*>(ws);
    int* first_of = reinterpret_cast<int*>(ws + L.table);  // [N + 1], then the count
    p.seg_state = reinterpret_cast<float*>(ws + L.table + L.first);
    segs = s.cu ? L.segs : up(s.T, p.seg_len) / p.seg_len;
    if (s.cu) {
      p.segs = table;
      p.nsegs = first_of + s.N + 1;
    }
    if (!states_ready) {
      if (s.cu) {
        e = launch_kernel(la_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, s.cu, s.N, s.T, p.seg_len, s.reverse, table, first_of,
                          first_of + s.N + 1);
        if (e != cudaSuccess) return e;
      }
      e = launch_dims<true>(p, segs, di, stream);
      if (e != cudaSuccess) return e;
      const int per_head = s.Da * s.Dc;
      e = launch_kernel(la_combine_kernel, dim3((unsigned)(((int64_t)s.H * per_head / 4 + 255) / 256), s.N), dim3(256), 0, stream, p,
                        (const int*)(s.cu ? first_of : nullptr), per_head);
      if (e != cudaSuccess) return e;
    }
  }
  return launch_dims<false>(p, segs, di, stream);
}

}  // namespace attnres
