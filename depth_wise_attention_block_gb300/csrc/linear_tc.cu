// The matrix products of attnres_linear and its backward on the tensor cores.
//
//   C(m, n) = sum_k A(m, k) B(n, k), then an epilogue (linear_epilogue.cuh)
//
// Operands come in by TMA, 64 steps of the contraction at a time, in the
// 128-byte swizzle, either K-major (rows of the contraction: x, w, dz in
// dz w) or MN-major (columns of it: w in dz w, both operands of dz^T x), so
// that no operand is ever transposed in memory.  One warp issues
// tcgen05.mma (M = 128 rows, fp32 accumulators in TMEM); eight warps run the
// epilogue while the next tile's products are formed in the other half of
// TMEM.
//
// Three shapes of launch:
//  - pairs: two CTAs of a cluster form one 256 x 256 tile
//    (tcgen05.mma.cta_group::2): each loads 128 rows of A and 128 rows of B,
//    half the L2 traffic per product of a 128 x 256 tile, whose 94 bytes per
//    cycle and SM are more than L2 delivers (2048 x 7168 x 7168: 175 us with
//    single tiles, 117 with pairs: 1.80 PFLOP/s).  Persistent, the bound is
//    the tensor cores.
//  - wide: persistent single CTAs over tiles of 128 x bn, where there are too
//    few 256 x 256 tiles, for fp32 operands, and for few rows of x where so
//    many columns to a tile as make one wave read the weights at HBM's rate
//    (64 x 21504 x 7168: 51 us, 6.1 TB/s).
//  - narrow (SWAP): few rows of one operand (decode).  The wide operand's
//    rows become the 128 lanes and the few rows the columns, so the weights
//    are read once; the contraction is split over a cluster of `ksplit` CTAs
//    whose partial tiles are joined through distributed shared memory in rank
//    order (no atomics, no workspace).  Two CTAs share an SM.  The bound is
//    HBM.
//
// fp32 operands (NP = 3) enter as three bf16 terms each (hi + mid + lo, 24
// bits).  The product hi hi goes to one accumulator and the five others that
// matter (hi mid, mid hi, mid mid, hi lo, lo hi) to a second one 2^-8
// smaller; both are drained into fp32 registers every kDrain blocks, so that
// the tensor cores' truncating accumulation never runs over more than 256
// steps of the contraction.  Up to 64 columns, the terms of B lie one behind
// the other as one operand and a term of A meets all it needs of them in one
// instruction (three instead of six: issuing one takes about as long as 128
// columns take to execute), each order of magnitude in columns of its own.
// Operands are split by a kernel of their own (prep_kernel) but for the wide
// operand of a narrow product of up to 128 rows: there the eight epilogue
// warps read it in fp32, two blocks ahead in registers, and write the terms
// where TMA would (FUSED), since reading the weights once is the bound
// (64 x 7168 x 7168: 101 us, with the terms made in memory first 191).
#include <math.h>

#include "attnres.h"
#include "body.h"
#include "launch.h"
#include "linear_epilogue.cuh"
#include "linear_tc.h"
#include "tc_common.cuh"

namespace attnres {

namespace {

constexpr int kLanes = 128;            // M of the instruction
constexpr int kKB = 64;                // contraction steps per block: one 128-byte swizzle row
constexpr int kThreads = 320;          // TMA warp, MMA warp, 8 epilogue warps
constexpr int kEpiWarps = 8;
constexpr int kMaxStages = 8;
constexpr int kDrain = 4;              // NP = 3: blocks between two drains
constexpr int kMaxKsplit = 8;
constexpr int kNarrowSmem = 100 * 1024;  // two CTAs per SM

struct TcParams {
  CUtensorMap ma, mb;    // lanes' operand, columns' operand
  bool a_mn, b_mn;
  int lanes, cols;       // size of the product along lanes and columns
  int kblocks;
  int bn;                // columns per tile, a multiple of 16
  int tiles_l, tiles_c;
  int ksplit, stages;
  uint32_t stage_bytes, plane_a, plane_b;  // bytes of a stage, of one plane of A and of B
  uint32_t tmem_cols, acc_cols;            // allocated columns, columns of one accumulator buffer
  uint32_t idesc, idesc2, idesc3;          // of one, two and three times bn columns (stacked)
  bool stacked;
  const float* raw;      // FUSED: the lanes' operand in fp32, row stride raw_ld
  long long raw_ld;
  int depth;             // steps of the contraction
  bool raw_vec;
  LinearEpilogue epi;
  int* dev_err;
  unsigned long long wait_ns;
  int withhold1;         // bounded-wait test: 1 + the block that each CTA arms without its copies
};

// A place in the ring of stages and the parity of its lap, without the
// divisions (the thread that issues the MMAs has 128 cycles for each).
struct RingPos {
  int st = 0;
  uint32_t lap = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++st == stages) {
      st = 0;
      lap ^= 1u;
    }
  }
};
// waits for the last phase of every stage that a producer armed: the CTA
// never exits under a copy (`r` is the place after the last armed one, `lap0`
// whether it is still in the first lap; a block armed without copies is its
// stage's last and never completes)
__device__ __forceinline__ void drain_stages(const uint64_t* full, const RingPos& r, bool lap0, int stages, int issued, int withhold1) {
  const int skip = withhold1 > 0 && issued >= withhold1 ? (withhold1 - 1) % stages : -1;
  for (int st = 0; st < (lap0 ? r.st : stages); ++st)
    if (st != skip) mbar_wait_bounded(smem_addr(&full[st]), st < r.st ? r.lap : r.lap ^ 1u);
}

// One plane of an operand's tile, block kb of the contraction, rows from r0.
__device__ __forceinline__ void load_plane(uint32_t dst, const CUtensorMap* map, bool mn, int r0, int rows, int kb, int plane,
                                           uint32_t bar) {
  if (!mn) {
    tma_load_3d(dst, map, kb * kKB, r0, plane, bar);
  } else {
    for (int j = 0; j < rows; j += 64) tma_load_3d(dst + j * 128, map, r0 + j, kb * kKB, plane, bar);  // 8 KB panels
  }
}

// descriptor of the 16 contraction steps from 16 kk of a plane
__device__ __forceinline__ uint64_t plane_desc(uint32_t addr, bool mn, int kk) {
  return mn ? smem_desc_mn128(addr + kk * 2048, 8192) : smem_desc_k128(addr + kk * 32);
}

// 16 values of a row as they lie in memory
template <typename T>
struct Raw16;
template <>
struct Raw16<bf16_t> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const bf16_t* p, bool vec) {
    if (vec) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = (uint32_t)p[2 * i].bits | (uint32_t)p[2 * i + 1].bits << 16;
    }
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    }
  }
};
template <>
struct Raw16<float> {
  float w[16];
  __device__ __forceinline__ void load(const float* p, bool vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (vec) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p) + i);
        w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = __ldg(p + 4 * i + j);
      }
    }
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = w[i];
  }
};
template <typename T>
__device__ __forceinline__ void store16(T* p, const float* v);
template <>
__device__ __forceinline__ void store16<bf16_t>(bf16_t* p, const float* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    st_global_v8(p, w);
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
template <>
__device__ __forceinline__ void store16<float>(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// Sums of 16 columns over the warp's 32 lanes: lane l returns column l / 2's
// (both lanes of a pair the same), in a fixed order, by halving exchanges.
__device__ __forceinline__ float column_sums16(float* v, int lane) {
#pragma unroll
  for (int half = 8; half > 0; half >>= 1) {
    const bool up = lane & (2 * half);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[i + half] : v[i], give = up ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * half);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// The epilogue of 16 columns n0 .. of row m (lanes: rows), and (kEpiDz with
// partial rows) their columns' sums over the warp.  `ahead` loads the
// residual's values, which a caller does before it waits for the product.
template <typename T, int MODE>
struct RowEpilogue {
  const TcParams& p;
  bool vec_out, vec_res, vec_bias;
  __device__ __forceinline__ explicit RowEpilogue(const TcParams& q) : p(q) {
    vec_out = q.epi.ldo % 8 == 0 && (reinterpret_cast<uintptr_t>(q.epi.out) & 15) == 0;
    vec_res = q.epi.ldr % 8 == 0 && (reinterpret_cast<uintptr_t>(q.epi.res) & 15) == 0;
    vec_bias = (reinterpret_cast<uintptr_t>(q.epi.bias) & 15) == 0;
  }
  __device__ __forceinline__ void ahead(Raw16<T>& r, long long m, int n0) const {
    if (p.epi.res && n0 + 16 <= p.cols)
      r.load(static_cast<const T*>(p.epi.res) + (m < p.lanes ? m : 0) * p.epi.ldr + n0, vec_res);
  }
  __device__ __forceinline__ void run(float* v, const Raw16<T>& res, long long m, int n0, int lane, int part_row) const {
    const LinearEpilogue& e = p.epi;
    const bool row = m < p.lanes;
    if (n0 + 16 <= p.cols) {
      if (e.bias) {
        Raw16<float> b;
        b.load(e.bias + n0, vec_bias);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += b.w[i];
      }
      float r[16];
      if (e.res) {
        res.get(r);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = 0.f;
      }
      act_apply<T, MODE, 16>(e.act, v, r);
      if (row) {
        T* dst = static_cast<T*>(e.out) + m * e.ldo + n0;
        if (vec_out) {
          store16<T>(dst, v);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) store_elem(dst + i, v[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = row && n0 + i < p.cols ? epilogue_one<T, MODE>(e, m, n0 + i, v[i]) : 0.f;
    }
    if (MODE == kEpiDz && e.part) {
      if (!row) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.f;
      }
      const float s = column_sums16(v, lane);
      const int n = n0 + lane / 2;
      if ((lane & 1) == 0 && n < p.cols) e.part[(long long)part_row * p.cols + n] = s;
    }
  }
};

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// FUSED: thread t's four vectors of 8 fp32 values of a block of 128 lanes x 64
// steps, K-major (lane t / 8 + 32 i, steps 8 (t mod 8) ..) or MN-major (step
// t / 16 + 16 i, lanes 8 (t mod 16) ..), zero outside the matrix.
__device__ __forceinline__ void fused_load(const TcParams& p, float (&v)[4][8], int l0, int kb, int t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = p.a_mn ? kb * kKB + t / 16 + 16 * i : l0 + t / 8 + 32 * i;
    const int col = p.a_mn ? l0 + t % 16 * 8 : kb * kKB + t % 8 * 8;
    const int rows = p.a_mn ? p.depth : p.lanes, cols = p.a_mn ? p.lanes : p.depth;
    const float* at = p.raw + (long long)row * p.raw_ld + col;
    if (row < rows && col + 8 <= cols && p.raw_vec) {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(at)), b = __ldcs(reinterpret_cast<const float4*>(at) + 1);
      v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
      v[i][4] = b.x, v[i][5] = b.y, v[i][6] = b.z, v[i][7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = row < rows && col + e < cols ? __ldcs(at + e) : 0.f;
    }
  }
}

// Three bf16 terms of two values: the first cut (a finite value stays finite),
// the others rounded, 2^-25 of the value left behind; the subtractions are
// exact.
__device__ __forceinline__ void three_terms(float x, float y, uint32_t (&w)[3]) {
  w[0] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  x -= bf16lo(w[0]);
  y -= bf16hi(w[0]);
  w[1] = pack_bf16x2(x, y);
  w[2] = pack_bf16x2(x - bf16lo(w[1]), y - bf16hi(w[1]));
}

// Those values' three terms into a stage's planes, in the 128-byte swizzle.
__device__ __forceinline__ void fused_store(const TcParams& p, const float (&v)[4][8], uint32_t stage, int t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = p.a_mn ? t / 16 + 16 * i : t / 8 + 32 * i, chunk = t % 8;
    const uint32_t at = stage + (p.a_mn ? t % 16 / 8 * 8192 : 0) + row * 128 + ((chunk ^ (row & 7)) << 4);
    uint32_t w[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) three_terms(v[i][2 * e], v[i][2 * e + 1], w[e]);
#pragma unroll
    for (int pl = 0; pl < 3; ++pl)
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + pl * p.plane_a), "r"(w[0][pl]), "r"(w[1][pl]), "r"(w[2][pl]), "r"(w[3][pl])
                   : "memory");
  }
}

// FUSED: 0, or the lanes' operand in fp32 and tiles of up to 64 (1) or 128 (2)
// columns, whose sums the epilogue warps hold beside the values on their way.
template <int NP, int MODE, bool SWAP, int FUSED>
__global__ void __launch_bounds__(kThreads) tc_gemm_kernel(const __grid_constant__ TcParams p) {
  using T = typename std::conditional<NP == 3, float, bf16_t>::type;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], split[FUSED ? kMaxStages : 1], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_base;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = warp_value(tid >> 5), lane = tid & 31;
  const int rank = SWAP && p.ksplit > 1 ? (int)cluster_ctarank() : 0;
  const int ntiles = p.tiles_l * p.tiles_c;
  const int tile0 = SWAP ? blockIdx.x / p.ksplit : blockIdx.x, tstep = SWAP ? ntiles : gridDim.x;
  const int kb0 = (int)((long long)rank * p.kblocks / p.ksplit), kb1 = (int)((long long)(rank + 1) * p.kblocks / p.ksplit);
  const int group = NP == 3 ? kDrain : p.kblocks;  // blocks per accumulator drain

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), 1);
      if (FUSED) mbar_init(smem_addr(&split[s]), kEpiWarps);
    }
    mbar_init(smem_addr(&drained), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&acc_full[b]), 1);
      mbar_init(smem_addr(&acc_empty[b]), kEpiWarps);
    }
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_base), p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_value(tmem_base);
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      const int brows = p.b_mn ? (p.bn + 63) / 64 * 64 : p.bn;
      RingPos r;
      int issued = 0;
      bool ok = true, lap0 = true;
      for (int tile = tile0; tile < ntiles && ok; tile += tstep) {
        const int l0 = tile % p.tiles_l * kLanes, c0 = tile / p.tiles_l * p.bn;
        for (int kb = kb0; kb < kb1; ++kb) {
          const int st = r.st;
          if (!mbar_wait_bounded(smem_addr(&empty[st]), r.lap ^ 1u, p.wait_ns)) {
            report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
            ok = false;
            break;
          }
          const uint32_t fb = smem_addr(&full[st]), a = base + st * p.stage_bytes, b = a + NP * p.plane_a;
          mbar_arrive_expect_tx(fb, NP * ((FUSED ? 0 : kLanes * 128) + brows * 128));
          ++issued;
#pragma unroll
          for (int pl = 0; pl < NP; ++pl) {
            if (issued == p.withhold1) break;
            if (!FUSED) load_plane(a + pl * p.plane_a, &p.ma, p.a_mn, l0, kLanes, kb, pl, fb);
            load_plane(b + pl * p.plane_b, &p.mb, p.b_mn, c0, brows, kb, pl, fb);
          }
          r.next(p.stages);
          lap0 = lap0 && r.st > 0;
        }
      }
      drain_stages(full, r, lap0, p.stages, issued, p.withhold1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // descriptors of the first stage; a stage, a plane and 16 steps further
    // are additions to the address field (units of 16 bytes)
    const uint64_t da0 = plane_desc(base, p.a_mn, 0), db0 = plane_desc(base + NP * p.plane_a, p.b_mn, 0);
    const uint32_t sa = p.a_mn ? 128 : 2, sb = p.b_mn ? 128 : 2, pa = p.plane_a / 16, pb = p.plane_b / 16;
    RingPos r;
    int g = 0;
    bool ok = true;
    for (int tile = tile0; tile < ntiles && ok; tile += tstep) {
      for (int kb = kb0; kb < kb1 && ok; ++g) {
        const int end = kb + group < kb1 ? kb + group : kb1;
        const int buf = g & 1;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&acc_empty[buf]), ((uint32_t)(g >> 1) & 1u) ^ 1u, p.wait_ns))) {
          report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + buf * p.acc_cols, d1 = d + p.acc_cols / 2;
        uint32_t acc = 0;
        for (; kb < end; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&full[r.st]), r.lap, p.wait_ns) &&
                                           (!FUSED || mbar_wait_bounded(smem_addr(&split[r.st]), r.lap, p.wait_ns)))) {
            report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = r.st * (p.stage_bytes / 16);
          const uint64_t da = da0 + at, db = db0 + at;
          if (NP == 3 && p.stacked) {
#pragma unroll
            for (int kk = 0; kk < kKB / 16; ++kk) {
              const uint64_t a = da + kk * sa, b = db + kk * sb;
              tc_mma_bf16_warp(d, a, b, p.idesc3, acc);                    // hi (hi, mid, lo)
              tc_mma_bf16_warp(d + p.bn, a + pa, b, p.idesc2, 1u);         // mid (hi, mid)
              tc_mma_bf16_warp(d + 2 * p.bn, a + 2 * pa, b, p.idesc, 1u);  // lo hi
              acc = 1;
            }
          } else {
#pragma unroll
            for (int kk = 0; kk < kKB / 16; ++kk) {
              const uint64_t a = da + kk * sa, b = db + kk * sb;
              tc_mma_bf16_warp(d, a, b, p.idesc, acc);
              if constexpr (NP == 3) {
                tc_mma_bf16_warp(d1, a, b + 2 * pb, p.idesc, acc);
                tc_mma_bf16_warp(d1, a + 2 * pa, b, p.idesc, 1u);
                tc_mma_bf16_warp(d1, a + pa, b + pb, p.idesc, 1u);
                tc_mma_bf16_warp(d1, a, b + pb, p.idesc, 1u);
                tc_mma_bf16_warp(d1, a + pa, b, p.idesc, 1u);
              }
              acc = 1;
            }
          }
          tc_commit_warp(smem_addr(&empty[r.st]));
          r.next(p.stages);
        }
        if (ok) tc_commit_warp(smem_addr(&acc_full[buf]));  // (else the epilogue's wait runs out, too, and it writes NaN)
      }
    }
    if (!ok) {  // no product is under way when shared memory and TMEM are given back
      tc_commit_warp(smem_addr(&drained));
      mbar_wait_bounded(smem_addr(&drained), 0);
    }
    __syncwarp();
  } else {
    // warp w reads TMEM lanes 32 (w mod 4) .. + 31; two warps share a quarter
    // and take the 16-column chunks in turn
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes_at = tmem + ((uint32_t)(32 * quarter) << 16);
    const int nchunk = (p.bn + 15) / 16;
    constexpr int kRegChunks = FUSED == 1 ? 2 : NP == 3 ? 4 : 1;  // NP = 3: bn <= 128
    const RowEpilogue<T, MODE> epi(p);
    const float nan = __int_as_float(0x7fc00000);
    bool ok = true;
    int g = 0;
    for (int tile = tile0; tile < ntiles; tile += tstep) {
      const int l0 = tile % p.tiles_l * kLanes, c0 = tile / p.tiles_l * p.bn;
      const long long m = l0 + 32 * quarter + lane;
      float acc[kRegChunks][16];
      if constexpr (NP == 3) {
#pragma unroll
        for (int c = 0; c < kRegChunks; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c][i] = 0.f;
      }
      Raw16<T> res[2];
      if constexpr (!SWAP && NP == 1) epi.ahead(res[0], m, c0 + half * 16);
      // one drain of an accumulator: into registers (NP = 3), or on its way out
      auto drain = [&] {
        const int buf = g & 1;
        if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&acc_full[buf]), (uint32_t)(g >> 1) & 1u, p.wait_ns))) {
          if (lane == 0) report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
          ok = false;
        }
        tc_fence_after();
        const uint32_t at = lanes_at + buf * p.acc_cols;
        if constexpr (NP == 3) {
#pragma unroll
          for (int c = 0; c < kRegChunks; ++c) {
            const int ch = 2 * c + half;
            if (ch < nchunk) {
              uint32_t v[16], w[16];
              tmem_ld16(at + ch * 16, v);
              tmem_ld16(at + (p.stacked ? p.bn : p.acc_cols / 2) + ch * 16, w);
              tmem_ld_wait();
              float small[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) small[i] = __uint_as_float(w[i]);
              if (p.stacked) {
                tmem_ld16(at + 2 * p.bn + ch * 16, w);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) small[i] += __uint_as_float(w[i]);
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[c][i] += __uint_as_float(v[i]) + small[i];
            }
          }
        } else {
#pragma unroll 2
          for (int ch = half; ch < nchunk; ch += 2) {
            uint32_t v[16];
            tmem_ld16(at + ch * 16, v);
            if constexpr (!SWAP) epi.ahead(res[1], m, c0 + (ch + 2) * 16);
            tmem_ld_wait();
            float f[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = ok ? __uint_as_float(v[i]) : nan;
            if constexpr (SWAP) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((ch * 16 + i) * kLanes + 32 * quarter + lane) * 4), "f"(f[i]) : "memory");
            } else if (c0 + ch * 16 < p.cols) {
              epi.run(f, res[0], m, c0 + ch * 16, lane, l0 / 32 + quarter);
              res[0] = res[1];
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&acc_empty[buf]));
        ++g;
      };
      if constexpr (FUSED) {
        // split block after block, two of them on their way in registers; a
        // group's sums are drained once the next group's terms are written
        const int t = tid - 64;
        float raw[2][4][8];
        fused_load(p, raw[0], l0, kb0, t);
        fused_load(p, raw[1], l0, kb0 + 1, t);
        RingPos r;
        for (int kb = kb0; kb < kb1; kb += 2) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int k = kb + u;
            if (k < kb1) {
              if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&empty[r.st]), r.lap ^ 1u, p.wait_ns))) {
                if (lane == 0) report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
                ok = false;
              }
              fused_store(p, raw[u], base + r.st * p.stage_bytes, t);
              if (k + 2 < kb1) fused_load(p, raw[u], l0, k + 2, t);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&split[r.st]));
              r.next(p.stages);
              if ((k - kb0) % kDrain == kDrain - 1 && k - kb0 >= kDrain) drain();
            }
          }
        }
        while (g * kDrain < kb1 - kb0) drain();
      } else {
        for (int kb = kb0; kb < kb1; kb += group) drain();
      }
      if constexpr (NP == 3) {
#pragma unroll
        for (int c = 0; c < kRegChunks; ++c) {
          const int ch = 2 * c + half;
          if (ch < nchunk) {
            if (!ok) {
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[c][i] = nan;
            }
            if constexpr (SWAP) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((ch * 16 + i) * kLanes + 32 * quarter + lane) * 4), "f"(acc[c][i]) : "memory");
            } else if (c0 + ch * 16 < p.cols) {
              epi.ahead(res[0], m, c0 + ch * 16);
              epi.run(acc[c], res[0], m, c0 + ch * 16, lane, l0 / 32 + quarter);
            }
          }
        }
      }
    }
  }
  if constexpr (SWAP) {
    // the cluster's partial tiles [column][lane], joined in rank order; each
    // rank takes a range of the columns
    if (p.ksplit > 1) {
      __syncwarp();
      cluster_sync_all();
    } else {
      __syncthreads();
    }
    if (warp >= 2) {
      const int e = tid - 64, row = e % kLanes, g = e / kLanes;
      const int l0 = tile0 % p.tiles_l * kLanes, c0 = tile0 / p.tiles_l * p.bn;
      const int cl0 = rank * p.bn / p.ksplit, cl1 = (rank + 1) * p.bn / p.ksplit;
      const int n = l0 + row;
      const uint32_t mine = base + row * 4;
      uint32_t at[kMaxKsplit];
#pragma unroll
      for (int r = 0; r < kMaxKsplit; ++r) at[r] = r < p.ksplit && p.ksplit > 1 ? map_shared_rank(mine, r) : mine;
      float sum = 0.f;
      for (int c = cl0 + g; c < cl1; c += 2) {
        float v = 0.f;
        if (p.ksplit > 1) {
#pragma unroll
          for (int r = 0; r < kMaxKsplit; ++r)
            if (r < p.ksplit) v += ld_shared_cluster(at[r] + c * kLanes * 4);
        } else {
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(mine + c * kLanes * 4) : "memory");
        }
        if (n < p.lanes && c0 + c < p.cols) sum += epilogue_one<T, MODE>(p.epi, c0 + c, n, v);
      }
      if (MODE == kEpiDz && p.epi.part && n < p.lanes)
        p.epi.part[(long long)((tile0 / p.tiles_l * p.ksplit + rank) * 2 + g) * p.lanes + n] = sum;
    }
    if (p.ksplit > 1) {
      __syncwarp();
      cluster_sync_all();  // no CTA leaves while another reads its tile
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// ------------------------------------------------------------- pairs -------

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// (by a whole warp)
__device__ __forceinline__ void tc_mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// one arrival at `bar` of both CTAs once the MMAs issued so far are done
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

constexpr int kPairN = 256;                              // columns of a pair's tile
constexpr int kPairBlock = 2 * kLanes * 128;             // bytes of a block in one CTA: 128 rows of A, 128 of B
// Two blocks to a stage: waiting, committing and stepping on take the issuing
// thread about 300 cycles, an instruction's issue 64 and its execution 128;
// with one block (four instructions) to a stage the issue was the bound.
constexpr int kPairStage = 2 * kPairBlock;
constexpr int kPairTmem = 512;                           // two accumulators of 256 columns

// Rank r of a cluster of two holds rows 128 r .. + 127 of the tile (in its
// TMEM) and rows 128 r .. + 127 of B.  Rank 0 issues the MMAs for both; its
// `full` barriers count the bytes of both, and its commits free the stages of
// both.
template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) tc_pair_kernel(const __grid_constant__ TcParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_base;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = warp_value(tid >> 5), lane = tid & 31;
  const int rank = warp_value((int)cluster_ctarank());
  const int ntiles = p.tiles_l * p.tiles_c, tile0 = blockIdx.x / 2, tstep = gridDim.x / 2;

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), 1);
    }
    mbar_init(smem_addr(&drained), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&acc_full[b]), 1);
      mbar_init(smem_addr(&acc_empty[b]), 2 * kEpiWarps);
    }
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_addr(&tmem_base), kPairTmem);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem = warp_value(tmem_base);
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      RingPos r;
      int issued = 0;
      bool ok = true, lap0 = true;
      for (int tile = tile0; tile < ntiles && ok; tile += tstep) {
        const int l0 = tile % p.tiles_l * (2 * kLanes) + rank * kLanes, c0 = tile / p.tiles_l * kPairN + rank * kLanes;
        for (int kb = 0; kb < p.kblocks; kb += 2) {
          if (!mbar_wait_bounded(smem_addr(&empty[r.st]), r.lap ^ 1u, p.wait_ns)) {
            report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
            ok = false;
            break;
          }
          const int blocks = kb + 1 < p.kblocks ? 2 : 1;
          const uint32_t fb = smem_addr(&full[r.st]);
          if (rank == 0) mbar_arrive_expect_tx(fb, 2 * kPairBlock * blocks);
          const uint32_t bar = map_shared_rank(fb, 0);
          ++issued;
          for (int i = 0; i < blocks && issued != p.withhold1; ++i) {
            const uint32_t a = base + r.st * kPairStage + i * kPairBlock, b = a + kPairBlock / 2;
            const int k = (kb + i) * kKB;
            if (p.a_mn) {
              tma_load_3d_pair(a, &p.ma, l0, k, 0, bar);
              tma_load_3d_pair(a + 8192, &p.ma, l0 + 64, k, 0, bar);
            } else {
              tma_load_3d_pair(a, &p.ma, k, l0, 0, bar);
            }
            if (p.b_mn) {
              tma_load_3d_pair(b, &p.mb, c0, k, 0, bar);
              tma_load_3d_pair(b + 8192, &p.mb, c0 + 64, k, 0, bar);
            } else {
              tma_load_3d_pair(b, &p.mb, k, c0, 0, bar);
            }
          }
          r.next(p.stages);
          lap0 = lap0 && r.st > 0;
        }
      }
      // no CTA exits under a copy: rank 0 sees the bytes of both
      if (rank == 0) drain_stages(full, r, lap0, p.stages, issued, p.withhold1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const uint64_t da0 = plane_desc(base, p.a_mn, 0), db0 = plane_desc(base + kPairBlock / 2, p.b_mn, 0);
      const uint32_t sa = p.a_mn ? 128 : 2, sb = p.b_mn ? 128 : 2;  // 16 contraction steps, in units of 16 bytes
      RingPos r;
      int g = 0;
      bool ok = true;
      for (int tile = tile0; tile < ntiles && ok; tile += tstep, ++g) {
        const int buf = g & 1;
        if (!__all_sync(0xffffffffu, mbar_wait_cluster_bounded(smem_addr(&acc_empty[buf]), ((uint32_t)(g >> 1) & 1u) ^ 1u, p.wait_ns))) {
          report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + buf * kPairN;
        uint32_t acc = 0;
        for (int kb = 0; kb < p.kblocks; kb += 2) {
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&full[r.st]), r.lap, p.wait_ns))) {
            report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = da0 + r.st * (kPairStage / 16), db = db0 + r.st * (kPairStage / 16);
#pragma unroll
          for (int kk = 0; kk < kKB / 16; ++kk) {
            tc_mma_bf16_pair(d, da + kk * sa, db + kk * sb, p.idesc, acc);
            acc = 1;
          }
          if (kb + 1 < p.kblocks) {
#pragma unroll
            for (int kk = 0; kk < kKB / 16; ++kk)
              tc_mma_bf16_pair(d, da + kPairBlock / 16 + kk * sa, db + kPairBlock / 16 + kk * sb, p.idesc, 1u);
          }
          tc_commit_pair(smem_addr(&empty[r.st]));
          r.next(p.stages);
        }
        if (ok) tc_commit_pair(smem_addr(&acc_full[buf]));
      }
      if (!ok) {
        tc_commit_pair(smem_addr(&drained));
        mbar_wait_bounded(smem_addr(&drained), 0);
      }
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes_at = tmem + ((uint32_t)(32 * quarter) << 16);
    const RowEpilogue<bf16_t, MODE> epi(p);
    const float nan = __int_as_float(0x7fc00000);
    bool ok = true;
    int g = 0;
    for (int tile = tile0; tile < ntiles; tile += tstep, ++g) {
      const int l0 = tile % p.tiles_l * (2 * kLanes) + rank * kLanes, c0 = tile / p.tiles_l * kPairN;
      const long long m = l0 + 32 * quarter + lane;
      const int buf = g & 1;
      Raw16<bf16_t> res[2];
      epi.ahead(res[0], m, c0 + half * (kPairN / 2));
      if (ok && !__all_sync(0xffffffffu, mbar_wait_cluster_bounded(smem_addr(&acc_full[buf]), (uint32_t)(g >> 1) & 1u, p.wait_ns))) {
        if (lane == 0) report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
        ok = false;
      }
      tc_fence_after();
#pragma unroll 2
      for (int ch = half * (kPairN / 32); ch < (half + 1) * (kPairN / 32); ++ch) {
        uint32_t v[16];
        tmem_ld16(lanes_at + buf * kPairN + ch * 16, v);
        if (ch + 1 < (half + 1) * (kPairN / 32)) epi.ahead(res[1], m, c0 + (ch + 1) * 16);
        tmem_ld_wait();
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = ok ? __uint_as_float(v[i]) : nan;
        if (c0 + ch * 16 < p.cols) epi.run(f, res[0], m, c0 + ch * 16, lane, l0 / 32 + quarter);
        res[0] = res[1];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_shared_rank(smem_addr(&acc_empty[buf]), 0));
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA's shared memory or TMEM is in use by the other
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kPairTmem);
  }
}

// ----------------------------------------------------------- operands ------

// Copies of operands TMA cannot take as they are: rows on 16-byte boundaries
// (bf16), or the three bf16 terms of fp32 values.
struct PrepJob {
  const void* src;
  long long ld, rows;
  int cols;
  long long pitch;  // elements per destination row, a multiple of 8
  bf16_t* dst;      // NP planes of rows x pitch
};
struct PrepParams {
  PrepJob job[2];
};

template <int NP>
__global__ void __launch_bounds__(256) prep_kernel(const __grid_constant__ PrepParams p) {
  const PrepJob& j = p.job[blockIdx.y];
  pdl_wait();
  pdl_trigger();
  const long long plane = j.rows * j.pitch;
  for (long long r = blockIdx.x; r < j.rows; r += gridDim.x) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(j.dst + r * j.pitch);
#pragma unroll 2
    for (int c = threadIdx.x * 2; c < j.pitch; c += 512) {
      if constexpr (NP == 1) {
        const uint16_t* s = static_cast<const uint16_t*>(j.src) + r * j.ld + c;
        const uint32_t lo = c < j.cols ? s[0] : 0, hi = c + 1 < j.cols ? s[1] : 0;
        dst[c / 2] = lo | hi << 16;
      } else {
        const float* s = static_cast<const float*>(j.src) + r * j.ld + c;
        uint32_t w[3];
        three_terms(c < j.cols ? s[0] : 0.f, c + 1 < j.cols ? s[1] : 0.f, w);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) dst[(pl * plane + c) / 2] = w[pl];
      }
    }
  }
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// The operand's tensor map: element (row, contraction step) at ptr[row ld +
// step] (K-major) or ptr[step ld + row] (MN-major), `np` planes apart.
bool operand_map(CUtensorMap* map, const void* ptr, int64_t outer, int64_t inner, int64_t ld, int np, bool mn, int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)np};
  if (outer == 1) ld = up(inner, 8);  // a stride that no address depends on
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)((np == 1 ? 1 : outer) * ld * 2)};
  const cuuint32_t box[3] = {64, (cuuint32_t)(mn ? kKB : box_rows), 1};
  return make_tensor_map(map, ptr, 3, dims, strides, box);
}

// A kernel's launch attributes: clusters of `cluster` CTAs (0: none), and
// programmatic dependent launch.
template <typename K>
cudaError_t launch_tc(K kern, const TcParams& p, int grid, int cluster, int smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 0) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int NP, int MODE, bool SWAP, int FUSED>
cudaError_t launch_gemm(const TcParams& p, int grid, int smem, int smem_max, cudaStream_t stream) {
  static SmemOptIn optin;
  const auto kern = tc_gemm_kernel<NP, MODE, SWAP, FUSED>;
  const cudaError_t e = optin.ensure(reinterpret_cast<const void*>(kern), smem_max);
  return e != cudaSuccess ? e : launch_tc(kern, p, grid, SWAP ? p.ksplit : 0, smem, stream);
}

template <int MODE>
cudaError_t launch_mode(const TcParams& p, int np, bool swap, bool fused, int grid, int smem, int smem_max, cudaStream_t stream) {
  if (np == 1)
    return swap ? launch_gemm<1, MODE, true, 0>(p, grid, smem, smem_max, stream)
                : launch_gemm<1, MODE, false, 0>(p, grid, smem, smem_max, stream);
  if (fused)
    return p.bn <= 64 ? launch_gemm<3, MODE, true, 1>(p, grid, smem, smem_max, stream)
                      : launch_gemm<3, MODE, true, 2>(p, grid, smem, smem_max, stream);
  return swap ? launch_gemm<3, MODE, true, 0>(p, grid, smem, smem_max, stream)
              : launch_gemm<3, MODE, false, 0>(p, grid, smem, smem_max, stream);
}

template <int MODE>
cudaError_t launch_pair(const TcParams& p, int grid, int smem, int smem_max, cudaStream_t stream) {
  static SmemOptIn optin;
  const cudaError_t e = optin.ensure(reinterpret_cast<const void*>(tc_pair_kernel<MODE>), smem_max);
  return e != cudaSuccess ? e : launch_tc(tc_pair_kernel<MODE>, p, grid, 2, smem, stream);
}

}  // namespace

bool tc_rows_ok(const void* ptr, int64_t ld) { return (reinterpret_cast<uintptr_t>(ptr) & 15) == 0 && ld % 8 == 0; }

int64_t tc_prep_bytes(int64_t rows, int64_t cols, int np) { return np * up(rows * up(cols, 8) * 2, 256); }

TcPlan tc_plan(int64_t M, int N, int64_t K, int np, int sm_count) {
  // fp32: making the terms in memory reads 4 bytes and writes 6 per value
  const double prep = np == 3 ? (double)(M + N) * K * 10 / 6000 : 0;
  TcPlan best{};
  const int64_t kblocks = up(K, kKB) / kKB;
  const int bn_max = np == 3 ? 128 : 256;
  double cost = 1e300;
  // All in nanoseconds.  Whole waves of tiles, of as many columns as make the
  // waves even: an instruction of a single tile of 256 columns takes about 130
  // (L2), of 128 or fewer about 68, of a pair's tile 70; then the start and
  // end of a tile's pipeline.  With few rows the loads are the bound: an SM
  // gets 80 bytes per ns with the 192 KB it keeps in flight, all of them 6500
  // (64 x 21504 x 7168: 57 us in 84 tiles of 256 columns, 51 in 150 of 144).
  constexpr double kTileNs = 800, kLaunchNs = 800;
  for (int bn = 64; bn <= bn_max; bn += 16) {
    const int64_t rows = up(M, kLanes) / kLanes, tiles = rows * (up(N, bn) / bn);
    const double instr = bn <= 128 ? 68 : 68 + 62. * (bn - 128) / 128;
    const double mma = (double)kblocks * (np == 3 ? (bn <= 64 ? 16 : 24) * 68 : 4 * instr);
    const double load = (double)kblocks * np * 128 * ((rows > 1 ? kLanes : M) + bn) / 80;
    const double waves = (double)((tiles + sm_count - 1) / sm_count), hbm = (double)(M + N) * (double)kblocks * np * 128 / 6500;
    double c = waves * (mma > load ? mma : load);
    if (c < hbm) c = hbm;
    c += waves * kTileNs + kLaunchNs + prep;
    if (c < cost) {
      cost = c;
      best = {TcPlan::kWide, bn, 1, 0, false};
    }
  }
  if (np == 1) {
    const int64_t tiles = up(M, 2 * kLanes) / (2 * kLanes) * (up(N, kPairN) / kPairN);
    const double c = (double)((tiles + sm_count / 2 - 1) / (sm_count / 2)) * ((double)kblocks * 4 * 70 + kTileNs) + kLaunchNs + 500;
    if (c < cost) {
      cost = c;
      best = {TcPlan::kPairs, kPairN, 1, 0, false};
    }
  }
  // narrow: M's rows as columns, N's as lanes, the contraction over a
  // cluster.  The CTAs of a wave share HBM (6.5 bytes per ps); alone one gets
  // about 40 bytes per ns with the 96 KB it keeps in flight (two per SM), 80
  // with the 192 KB of fp32's terms; starting, joining and ending a wave takes
  // about 5500.  64 x 21504 x 7168, clusters of 1, 2, 3, 5, 7: 59, 75, 62, 65,
  // 75 us; 64 x 7168 x 7168, clusters of 2, 3, 4, 5, 8: 29, 25, 23, 22, 29 us.
  if (M <= 1024) {
    const int bn = M >= 128 ? 128 : (int)up(M, 16);
    const int64_t slots = (int64_t)sm_count * (np == 3 ? 1 : 2);
    for (int ks = 1; ks <= kMaxKsplit && ks <= kblocks; ++ks) {
      const int64_t tiles = up(N, kLanes) / kLanes * (up(M, bn) / bn);
      const int64_t ctas = tiles * ks, blocks = (kblocks + ks - 1) / ks;
      const double mma = (double)blocks * (np == 1 ? 4 : bn <= 64 ? 12 : 24) * 68;
      // bytes of the lanes' operand per CTA (fused: fp32, else np terms), and
      // the bytes per ns that a CTA alone gets
      auto price = [&](double bytes, double rate) {
        const double alone = (bytes + (double)blocks * np * bn * 128) / rate;
        auto wave = [&](int64_t n) {
          const double share = (double)n * bytes / 6500;
          const double t = share > alone ? share : alone;
          return (t > mma ? t : mma) + 5500;
        };
        return (double)(ctas / slots) * wave(slots) + (ctas % slots ? wave(ctas % slots) : 0);
      };
      const double c = price((double)blocks * np * kLanes * 128, np == 3 ? 80 : 40) + prep;
      if (c < cost) {
        cost = c;
        best = {TcPlan::kNarrow, bn, ks, 0, false};
      }
      if (np == 3 && M <= 128) {
        const double f = price((double)blocks * kLanes * 256, 40) + (double)M * K * 10 / 6000;
        if (f < cost) {
          cost = f;
          best = {TcPlan::kNarrow, bn, ks, 0, true};
        }
      }
    }
  }
  best.part_rows = best.shape == TcPlan::kNarrow ? (int)(up(M, best.bn) / best.bn * best.ksplit * 2)
                   : best.shape == TcPlan::kPairs ? (int)(up(M, 2 * kLanes) / 32)
                                                  : (int)(up(M, kLanes) / 32);
  return best;
}

cudaError_t launch_tc_prep(const TcOperand* ops, int n, int np, cudaStream_t stream) {
  PrepParams pp{};
  int64_t most = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t pitch = up(ops[i].cols, 8);
    pp.job[i] = {ops[i].ptr, ops[i].ld, ops[i].rows, (int)ops[i].cols, pitch, static_cast<bf16_t*>(ops[i].prep)};
    if (ops[i].rows > most) most = ops[i].rows;
  }
  const dim3 grid((unsigned)(most < 2432 ? most : 2432), n);
  return np == 3 ? launch_kernel(prep_kernel<3>, grid, dim3(256), 0, stream, pp)
                 : launch_kernel(prep_kernel<1>, grid, dim3(256), 0, stream, pp);
}

cudaError_t launch_tc_gemm(const TcPlan& plan, const TcOperand& A, const TcOperand& B, int64_t M, int N, int64_t K, int np,
                           int mode, const LinearEpilogue& epi, int* dev_err, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const bool swap = plan.shape == TcPlan::kNarrow, pairs = plan.shape == TcPlan::kPairs;
  const TcOperand &lo = swap ? B : A, &co = swap ? A : B;
  TcParams p{};
  auto map = [&](CUtensorMap* m, const TcOperand& o, int box) {
    const void* ptr = o.prep ? o.prep : o.ptr;
    const int64_t ld = o.prep ? up(o.cols, 8) : o.ld;
    return operand_map(m, ptr, o.rows, o.cols, ld, np, o.mn, box);
  };
  if ((!plan.fused && !map(&p.ma, lo, kLanes)) || !map(&p.mb, co, pairs ? kLanes : plan.bn)) return cudaErrorInvalidValue;
  if (plan.fused) {
    p.raw = static_cast<const float*>(lo.ptr);
    p.raw_ld = lo.ld;
    p.raw_vec = (reinterpret_cast<uintptr_t>(lo.ptr) & 15) == 0 && lo.ld % 4 == 0;
  }
  p.depth = (int)K;
  p.a_mn = lo.mn;
  p.b_mn = co.mn;
  p.lanes = swap ? N : (int)M;
  p.cols = swap ? (int)M : N;
  p.kblocks = (int)(up(K, kKB) / kKB);
  p.bn = plan.bn;
  const int tile_l = pairs ? 2 * kLanes : kLanes;
  p.tiles_l = (int)(up(p.lanes, tile_l) / tile_l);
  p.tiles_c = (int)(up(p.cols, p.bn) / p.bn);
  p.ksplit = plan.ksplit;
  p.plane_a = kLanes * 128;
  p.plane_b = (uint32_t)((p.b_mn ? up(p.bn, 64) : up(p.bn, 8)) * 128);
  p.stage_bytes = np * (p.plane_a + p.plane_b);
  p.stacked = np == 3 && !p.b_mn && p.bn <= 64;
  const int nacc = p.stacked ? 3 : np == 3 ? 2 : 1;
  const int nbuf = swap && np == 1 ? 1 : 2;
  p.acc_cols = nacc * (uint32_t)p.bn;
  p.tmem_cols = 32;
  while (p.tmem_cols < nbuf * p.acc_cols) p.tmem_cols *= 2;
  p.idesc = tc_idesc_bf16(kLanes, p.bn, p.a_mn, p.b_mn);
  if (p.stacked) {
    p.idesc2 = tc_idesc_bf16(kLanes, 2 * p.bn, p.a_mn, p.b_mn);
    p.idesc3 = tc_idesc_bf16(kLanes, 3 * p.bn, p.a_mn, p.b_mn);
  }
  p.epi = epi;
  p.dev_err = dev_err;
  p.wait_ns = wait_limit_ns();
  p.withhold1 = debug_withhold_row1();
  // shared memory: the stages; narrow tiles also park their partial sums there
  const int smem_max = di.max_smem_optin - 1024;  // the kernels' static shared memory fits in the rest
  const int budget = (swap && np == 1 ? kNarrowSmem : smem_max) - 1024;
  int stages = budget / (int)p.stage_bytes;
  if (stages > kMaxStages) stages = kMaxStages;
  if (stages < 2) return cudaErrorInvalidValue;
  p.stages = stages;
  int smem = stages * (int)p.stage_bytes;
  if (swap && smem < p.bn * kLanes * 4) smem = p.bn * kLanes * 4;
  smem += 1024;
  const int64_t tiles = (int64_t)p.tiles_l * p.tiles_c;
  if (tiles > INT32_MAX / kMaxKsplit) return cudaErrorInvalidValue;
  if (pairs) {
    p.stages = (smem_max - 1024) / kPairStage;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    p.idesc = tc_idesc_bf16(2 * kLanes, kPairN, p.a_mn, p.b_mn);
    const int64_t pr = di.sm_count / 2;
    const int grid = (int)(2 * (tiles < pr ? tiles : pr)), smem = p.stages * kPairStage + 1024;
    return mode == kEpiDz ? launch_pair<kEpiDz>(p, grid, smem, smem_max, stream) : launch_pair<kEpiForward>(p, grid, smem, smem_max, stream);
  }
  const int64_t grid = swap ? tiles * p.ksplit : (tiles < di.sm_count ? tiles : di.sm_count);
  return mode == kEpiDz ? launch_mode<kEpiDz>(p, np, swap, plan.fused, (int)grid, smem, smem_max, stream)
                        : launch_mode<kEpiForward>(p, np, swap, plan.fused, (int)grid, smem, smem_max, stream);
}

}  // namespace attnres
