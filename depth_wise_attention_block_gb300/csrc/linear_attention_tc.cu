// The scan of linear attention (linear_attention.cu) on the tensor cores:
// bf16 tensors with head sizes of up to 128, multiples of 16, in chunks of 128
// tokens.  DA and DC are the sizes rounded up to 64 or 128: the loads fill the
// channels behind a head's last with zeros.
//
//   P    = a b^T, masked and decayed       scores of the chunk   [128 x 128]
//   out  = P c + l^{i+1} (a S)             S: the state before it
//   U    = sum_j l^{C-1-j} b_j c_j^T,      S <- l^C S + U
//
// Every product is a tcgen05.mma with its accumulator in TMEM.  a, b and c
// arrive by TMA in the 128-byte swizzle and serve K-major (a b^T, a S) or
// MN-major (P c, the token sums) from the same tile.  Eight warps turn the
// scores into P (two bf16 terms, back into TMEM as the next product's operand)
// and write the outputs; eight warps hold the state in fp32 registers (half a
// row of Da per thread) and give it to the products as two bf16 terms (one
// term, whose error is the output's own rounding once more, is 5 % faster: 288
// us instead of 304 for the prompt below); all of them weigh b with the decays.
// The weighted rows enter as three bf16 terms (24 bits) where the state is a
// result, so that it keeps fp32 precision over any number of chunks; each
// chunk's U starts from zero in TMEM and is added in fp32 round-to-nearest.
//
// A reversed scan (gradients of k and v) takes the chunks from the end and
// mirrors the mask and the powers; nothing is reordered in memory.
//
// Few heads and sequences do not fill the GPU, and many of unequal lengths
// fill it badly.  The chunks of all heads are then cut into even ranges, one
// to an SM: state_tc_kernel forms the state of every piece of a sequence in a
// range (it reads b and c only), la_combine_kernel runs through a sequence's
// pieces and leaves the state before each, and the scan runs over the ranges.
// The loads run ahead from piece to piece; a table in shared memory tells the
// other warps of each.  Code and registers are kept small: the roles share the
// instruction cache (unrolling the scores' loop twice cost 4 %), and pieces
// held in registers 8 %.
//
// Bound: HBM, with the arithmetic warps close behind.  A chunk of 128 x 128
// heads takes about 5500 cycles of HBM time per SM, its products 3800 of
// the tensor cores, and the warps that turn scores into P and write outputs
// about 6000.  16384 tokens x 56 heads of 128: the scan 199 us (4.7 TB/s), the
// pieces' states 92 us (5.2 TB/s), joining them 10.6 us (each by itself, cold;
// the whole call in a graph 304).
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
constexpr int kTileThreads = 576;      // the states' kernel: 16 warps of arithmetic, TMA, MMA
constexpr int kScanThreads = 608;      // the scan: 8 warps scores and outputs, 8 state, TMA, two MMA
constexpr int kMaxSlots = 8;
constexpr int kPieces = 8;  // of the table of pieces; the loads are at most four pieces ahead
// Dynamic shared memory of sm_103a's 227 KB per CTA beside 2 KB of barriers
// and tables.  The rings' lengths are constants: a division by a length read
// from a parameter costs the issuing threads more than a product.
constexpr int kDynSmem = 232448 - 2048;

// ring slots of the scan, of the states' kernel
template <int DA, int DC, int TERMS>
struct ScanSmem {
  static constexpr int kTile = kC * (DA > DC ? DA : DC) * 2;
  static constexpr int kState = DC * DA * 2, kTerms = (TERMS - 1) * kC * DA * 2;
  // the state's second term: a place of its own where that leaves enough slots
  static constexpr bool kOwnLow = kDynSmem - 2 * kState - kTerms - 1024 >= 4 * kTile;
  static constexpr int kFixed = (kOwnLow ? 2 : 1) * kState + kTerms + 1024;
  static constexpr int kFit = (kDynSmem - kFixed) / kTile, kSlots = kFit < kMaxSlots ? kFit : kMaxSlots;
  static constexpr int kBytes = kFixed + kSlots * kTile;
  static_assert(kSlots >= 4, "a chunk's tiles and the next chunk's first");
};
constexpr int kHalf = kC / 2;
template <int DA, int DC>
struct StateSmem {
  static constexpr int kStage = kHalf * (DA + DC) * 2;
  static constexpr int kFixed = 6 * kHalf * DA * 2 + 1024;
  static constexpr int kFit = (kDynSmem - kFixed) / kStage, kSlots = kFit < kMaxSlots ? kFit : kMaxSlots;
  static constexpr int kBytes = kFixed + kSlots * kStage;
  static_assert(kSlots >= 4, "a half's barrier is read before its stage's next use");
};
constexpr int kPanel = kC * 128;       // bytes of 64 channels of a tile

struct ScanTcParams {
  CUtensorMap ma, mb, mc;
  ScanArgs s;
  int* dev_err;
  unsigned long long wait_ns;
  int withhold1;  // bounded-wait test: 1 + the tile that each CTA arms without its copies
};

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] x B[smem]^T, by a whole warp
__device__ __forceinline__ void tc_mma_bf16_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// two bf16 values, 1e30 in the place of a NaN (and of what is larger)
__device__ __forceinline__ uint32_t finite_or_large(uint32_t v) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x714A714Au));
  return r;
}

// The outputs of one row from the tensors in memory, over the rows that the
// mask leaves alone, channels c0 .. c1 - 1: where the products, in which a
// masked row counts as 0 times its values, met an infinity or a NaN.  o2: the
// row's a S in TMEM, which a whole warp reads; `bad`: this lane's row is
// redone; l: the table of p_scale l^distance.
__device__ __noinline__ void masked_row(const ScanArgs& s, const float* l, uint32_t o2, long long t0, int h, int row, int len, int c0, int c1,
                                        float coef, bool bad) {
  for (; c0 < c1; c0 += 16) {
    uint32_t y[16];
    tmem_ld16(o2 + c0, y);
    tmem_ld_wait();
    if (!bad || c0 >= s.Dc) continue;
    const bf16_t* a = static_cast<const bf16_t*>(s.a) + (t0 + row) * s.as + (long long)h * s.Da;
    float x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = coef * __uint_as_float(y[k]);
    for (int j = s.reverse ? row : 0; j < (s.reverse ? len : row + 1); ++j) {
      const bf16_t* b = static_cast<const bf16_t*>(s.b) + (t0 + j) * s.bs + (long long)h * s.Da;
      const bf16_t* c = static_cast<const bf16_t*>(s.c) + (t0 + j) * s.cs + (long long)h * s.Dc + c0;
      float dot = 0.f;
      for (int d = 0; d < s.Da; ++d) dot = fmaf(load_elem(a + d), load_elem(b + d), dot);
      const float f = dot * l[s.reverse ? j - row : kC - 1 - row + j];
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = fmaf(f, load_elem(c + k), x[k]);
    }
    bf16_t* out = static_cast<bf16_t*>(s.out) + (t0 + row) * s.os + (long long)h * s.Dc + c0;
#pragma unroll
    for (int k = 0; k < 16; ++k) store_elem(out + k, x[k]);
  }
}

// After a wait that ran out, by a warp: NaN to the outputs of a CTA's whole
// range (STATES: to its pieces' own states).
template <bool STATES>
__device__ __noinline__ void poison_range(const ScanArgs& s, int cta, int lane) {
  PieceWalk walk(s, cta);
  Piece q;
  const float nan = __int_as_float(0x7fc00000);
  while (walk.next(s, cta, &q)) {
    if constexpr (STATES) {
      if (q.last && !s.s_out) continue;
      const long long n = (long long)s.Da * s.Dc;
      for (long long i = lane; i < n; i += 32) s.piece_state[q.id * n + i] = nan;
    } else {
      for (int r = 0; r < q.len; ++r)
        for (int c = lane; c < s.Dc; c += 32)
          store_elem(static_cast<bf16_t*>(s.out) + (long long)(q.first + r) * s.os + (long long)q.head * s.Dc + c, nan);
    }
  }
}

// mbar_wait_bounded with one try in the code: the roles' waits are many, and
// they share the instruction cache.
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t it = 0; it < kWaitMaxPolls; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0) {
      const uint64_t t = global_timer_ns();
      if (it == 0)
        t0 = t;
      else if (t - t0 > limit_ns)
        return false;
    }
  }
  return false;
}

// FULL: the head sizes are DA and DC.  TERMS: bf16 terms of b's weighted rows, 3 where the state is a result, 2
// where only bf16 outputs follow from it.
template <int DA, int DC, int TERMS, bool FULL>
__global__ void __launch_bounds__(kScanThreads, 1) scan_tc_kernel(const __grid_constant__ ScanTcParams p) {
  constexpr int kTile = ScanSmem<DA, DC, TERMS>::kTile, kSlots = ScanSmem<DA, DC, TERMS>::kSlots;
  constexpr int kTiles = 3;                            // tiles per chunk: a, b, c
  constexpr uint32_t kColP = 0, kColO1 = 128, kColO2 = 256, kColU = 384;  // TMEM columns
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxSlots], empty[kMaxSlots], p_full, p_ready, o_full, o_free, s_ready, s_read, b_ready, u_full, u_free;
  __shared__ __align__(8) uint64_t t_ready, drained[2];
  __shared__ uint32_t tmem_base;
  // l^i; and p_scale l^distance in the order of a row's columns: distances
  // below 0, which the mask covers, read up to 46 places before it (reversed)
  // or behind it
  __shared__ float pw[2 * kC + 4 + 48];
  float* const tab = pw + kC + 4;
  __shared__ Piece pieces[kPieces];
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t s_buf = base + kSlots * kTile, rest = s_buf + DC * DA * 2;  // the terms behind the first
  // the state's second term lies behind them, or (not kOwnLow) where the last
  // of them does: it is written once the chunk before has summed that up, and
  // read by a S before split writes the chunk's own
  constexpr bool kOwnLow = ScanSmem<DA, DC, TERMS>::kOwnLow;
  const uint32_t s_low = rest + (TERMS - (kOwnLow ? 1 : 2)) * (kC * DA * 2);
  const int tid = threadIdx.x, warp = warp_value(tid >> 5), lane = tid & 31;
  const int Da = FULL ? DA : p.s.Da, Dc = FULL ? DC : p.s.Dc;

  if (tid == 0) {
    mbar_init(smem_addr(&t_ready), 16);
    mbar_init(smem_addr(&drained[0]), 1);
    mbar_init(smem_addr(&drained[1]), 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), 2);  // two arrivals free a slot: each MMA warp's (c), or one warp's two (a, b)
    }
    mbar_init(smem_addr(&p_full), 1);
    mbar_init(smem_addr(&p_ready), 8);
    mbar_init(smem_addr(&o_full), 1);
    mbar_init(smem_addr(&o_free), 8);
    mbar_init(smem_addr(&s_ready), 8);
    mbar_init(smem_addr(&s_read), 1);
    mbar_init(smem_addr(&b_ready), 16);
    mbar_init(smem_addr(&u_full), 1);
    mbar_init(smem_addr(&u_free), 8);
    mbar_fence_init();
  }
  if (warp == 17) tmem_alloc(smem_addr(&tmem_base), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_value(tmem_base);
  pdl_wait();
  pdl_trigger();
  const bool cut = p.s.parts > 0, rev = p.s.reverse;
  // the table of pieces: its first one, then what the loads publish
  PieceWalk walk;
  if (warp == 16 && lane == 0) {
    Piece pc{0, 0, 0, 0, 0, 0};
    if (cut) {
      walk = PieceWalk(p.s, blockIdx.x);
      walk.next(p.s, blockIdx.x, &pc);
    } else {
      pc = whole_sequence(p.s, blockIdx.x / p.s.H, blockIdx.x % p.s.H);
    }
    pieces[0] = pc;
  }
  __syncthreads();
  const bool live = !cut || pieces[0].len > 0;
  // first token of the chunk that begins `left` tokens before a piece's end
  // (a reversed scan's short chunk is its last)
  auto chunk_at = [&](const Piece& q, int left) { return rev ? q.first + (left > kC ? left - kC : 0) : q.first + q.len - left; };
  // once a wait runs out, the others of this thread return at once
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !poll(smem_addr(bar), parity & 1u, p.wait_ns)) {
      report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
      ok = false;
    }
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    wait(bar, parity);
    ok = __all_sync(0xffffffffu, ok);
  };
  // Nothing is passed on once a wait has run out: the other roles' waits run
  // out, too, and the results are NaN.
  auto commit = [&](uint64_t* bar) {
    if (ok) tc_commit_warp(smem_addr(bar));
  };
  // no product of this warp is under way when shared memory and TMEM are given back
  auto drain = [&](uint64_t* bar) {
    if (!ok) {
      tc_commit_warp(smem_addr(bar));
      mbar_wait_bounded(smem_addr(bar), 0);
    }
  };

  if (warp == 16) {
    if (lane == 0) {
      int it = 0;
      Piece pc = pieces[0];
      for (int k = 1; ok; ++k) {
        for (int left = pc.len; left > 0 && ok; left -= kC) {
          const int t = chunk_at(pc, left);
          for (int x = 0; x < kTiles; ++x, ++it) {
            const int st = it % kSlots;
            wait(&empty[st], (uint32_t)(it / kSlots) + 1u);
            if (!ok) break;
            const int D = x == 2 ? DC : DA;
            const CUtensorMap* m = x == 0 ? &p.ma : x == 1 ? &p.mb : &p.mc;
            const uint32_t fb = smem_addr(&full[st]);
            mbar_arrive_expect_tx(fb, D * kC * 2);
            for (int y = 0; y < D && it + 1 != p.withhold1; y += 64) tma_load_3d(base + st * kTile + y / 64 * kPanel, m, y, pc.head, t, fb);
          }
        }
        if (!cut || !live || !ok) break;
        // the next piece, which its first tile's barrier publishes; behind the
        // last a barrier of no bytes
        const bool more = walk.next(p.s, blockIdx.x, &pc);
        if (!more) pc.len = 0;
        pieces[k % kPieces] = pc;
        if (!more) {
          wait(&empty[it % kSlots], (uint32_t)(it / kSlots) + 1u);
          if (ok) mbar_arrive(smem_addr(&full[it++ % kSlots]));
          break;
        }
      }
      // the CTA never exits under a copy
      // (a tile armed without copies is its slot's last and never completes)
      const int armed = it < kSlots ? it : kSlots, skip = p.withhold1 > 0 && it >= p.withhold1 ? (p.withhold1 - 1) % kSlots : -1;
      for (int st = 0; st < armed; ++st)
        if (st != skip) mbar_wait_bounded(smem_addr(&full[st]), (uint32_t)((it - 1 - st) / kSlots) & 1u);
    }
    __syncwarp();
  } else if (warp == 17) {
    constexpr uint32_t kI1 = tc_idesc_bf16(128, 128), kI2 = tc_idesc_bf16(128, DC, false, true), kI3 = tc_idesc_bf16(128, DC);
    auto slot = [&](int i) { return base + i % kSlots * kTile; };
    auto wait_tile = [&](int i) { warp_wait(&full[i % kSlots], (uint32_t)(i / kSlots)); };
    // scores of chunk m, over those of m - 1 (whose P c is done)
    auto before = [&](int m) {
      if (m > 0) warp_wait(&o_full, (uint32_t)m - 1u);
      wait_tile(m * kTiles);
    };
    auto scores = [&](int m) {
      const int it = m * kTiles;
      wait_tile(it + 1);
      tc_fence_after();
      const uint64_t da = smem_desc_k128(slot(it)), db = smem_desc_k128(slot(it + 1));
#pragma unroll 4
      for (int kk = 0; kk < DA / 16; ++kk) {
        const uint32_t off = (kk / 4 * kPanel + kk % 4 * 32) / 16;
        tc_mma_bf16_warp(tmem + kColP, da + off, db + off, kI1, kk > 0);
      }
      commit(&p_full);
    };
    int m = 0, left = warp_value(pieces[0].len);  // chunk of all pieces; tokens to go in this one
    if (left > 0) {
      before(0);
      scores(0);
    }
    for (int k = 1; left > 0 && ok; ++k) {
      for (; left > 0 && ok; left -= kC, ++m) {
        const int it = m * kTiles, ic = it + 2;
        const uint32_t ph = (uint32_t)m;
        const uint64_t dc = smem_desc_mn128(slot(ic), kPanel);
        warp_wait(&s_ready, ph);
        warp_wait(&o_free, ph + 1);
        tc_fence_after();
        const uint64_t da = smem_desc_k128(slot(it)), ds = smem_desc_k128(s_buf), dl = smem_desc_k128(s_low);
#pragma unroll 4
        for (int kk = 0; kk < DA / 16; ++kk) {
          const uint32_t at = (kk / 4 * (DC * 128) + kk % 4 * 32) / 16;
          const uint64_t a = da + (kk / 4 * kPanel + kk % 4 * 32) / 16;
          tc_mma_bf16_warp(tmem + kColO2, a, ds + at, kI3, kk > 0);
          tc_mma_bf16_warp(tmem + kColO2, a, dl + at, kI3, 1u);
        }
        if constexpr (!kOwnLow) commit(&s_read);
        commit(&empty[it % kSlots]);
        commit(&empty[it % kSlots]);
        wait_tile(ic);
        // rows behind a short chunk's end are cleared with the weighted rows
        if (left < kC) warp_wait(&b_ready, ph);
        warp_wait(&p_ready, ph);
        tc_fence_after();
#pragma unroll 4
        for (int kk = 0; kk < kC / 16; ++kk)
          for (int lo = 0; lo < 2; ++lo) tc_mma_bf16_ts_warp(tmem + kColO1, tmem + kColP + kk * 16 + lo * 8, dc + kk * 128, kI2, lo > 0 || kk > 0);
        commit(&o_full);
        commit(&empty[ic % kSlots]);
        if (left > kC) {
          before(m + 1);
          scores(m + 1);
        }
      }
      if (!cut || !ok) break;
      before(m);
      left = ok ? warp_value(pieces[k % kPieces].len) : 0;
      if (left > 0)
        scores(m);
      else if (ok && lane == 0)
        mbar_arrive(smem_addr(&p_full));  // the others read of the end behind it
    }
    drain(&drained[0]);
    __syncwarp();
  } else if (warp == 18) {
    // a warp of its own, since these products wait for other things
    constexpr uint32_t kI4 = tc_idesc_bf16(128, DA, true, true);
    int m = 0, left = warp_value(pieces[0].len);
    for (int k = 1; left > 0 && ok; ++k) {
      for (; left > 0 && ok; left -= kC, ++m) {
        const int ib = m * kTiles + 1, ic = ib + 1;
        const uint32_t ph = (uint32_t)m, b0 = base + ib % kSlots * kTile;
        const uint64_t dc = smem_desc_mn128(base + ic % kSlots * kTile, kPanel);
        warp_wait(&b_ready, ph);
        warp_wait(&full[ic % kSlots], (uint32_t)(ic / kSlots));
        warp_wait(&u_free, ph + 1);
        tc_fence_after();
        // c's channels as the 128 rows (64 channels: the other 64 rows are
        // whatever lies behind, and are not read)
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
          const uint64_t dt = smem_desc_mn128(term == 0 ? b0 : rest + (term - 1) * (kC * DA * 2), kPanel);
#pragma unroll 4
          for (int kk = 0; kk < kC / 16; ++kk) tc_mma_bf16_warp(tmem + kColU, dc + kk * 128, dt + kk * 128, kI4, term > 0 || kk > 0);
        }
        commit(&u_full);
        commit(&empty[ib % kSlots]);
        commit(&empty[ib % kSlots]);
        commit(&empty[ic % kSlots]);
      }
      if (!cut || !ok) break;
      warp_wait(&b_ready, (uint32_t)m);  // of the next piece's first chunk, or of the end
      left = ok ? warp_value(pieces[k % kPieces].len) : 0;
    }
    drain(&drained[1]);
    __syncwarp();
  } else {
    // warp w reads TMEM lanes 32 (w mod 4) .. + 31; two warps of a group share
    // a quarter, each with half of the columns
    const int quarter = warp & 3, half = warp >> 2 & 1, row = 32 * quarter + lane;
    const uint32_t lanes_at = tmem + ((uint32_t)(32 * quarter) << 16);
    // the powers of piece k's head, where it is not the last piece's (all
    // sixteen warps: once they are done with the old ones, each its part)
    int meets = 0;
    auto meet = [&] {
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(smem_addr(&t_ready));
      warp_wait(&t_ready, meets++);
    };
    auto powers = [&](int k) {
      const int head = pieces[k % kPieces].head;
      if (k > 0) {
        if (pieces[(k - 1) % kPieces].head == head) return;
        meet();
      }
      const float g = __ldg(p.s.log_decay + head);
      if (tid < kC + 4) {
        const float l = decay_pow(g, tid);
        pw[tid] = l;
        if (tid < kC) tab[rev ? tid : kC - 1 - tid] = p.s.p_scale * l;
      }
      meet();
    };
    // whether there is a piece k, which chunk m begins
    auto more = [&](int k, int m) {
      if (!cut || !ok) return false;
      warp_wait(&p_full, m);
      if (!ok) return false;
      if (pieces[k % kPieces].len > 0) return true;
      if (ok && lane == 0) mbar_arrive(smem_addr(&b_ready));  // the token sums' warp reads of the end behind it
      return false;
    };
    // b's rows times their decay, as three bf16 terms (hi over b itself)
    auto split = [&](int len, int m, int t0) {
      const uint32_t B = base + (m * kTiles + 1) % kSlots * kTile, Ct = base + (m * kTiles + 2) % kSlots * kTile;
      if constexpr (!kOwnLow) warp_wait(&s_read, m);
      // thread t0's vectors of 8 channels lie in rows t0 / 8 + kStep i of each
      // panel, i < kBatch; a panel's are loaded before the first is stored
      constexpr int kStep = 512 / 8, kBatch = kC / kStep;
      static_assert(kBatch >= 1 && kBatch * kStep == kC, "the batches cover a panel's rows once");
      float f[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int j = t0 / 8 + i * kStep;
        f[i] = p.s.up_scale * pw[p.s.shift + (rev ? j : j < len ? len - 1 - j : 0)];
      }
#pragma unroll 1
      for (int x = 0; x < DA / 64; ++x) {
        const int j0 = t0 / 8;
        const uint32_t at = x * kPanel + j0 * 128 + t0 % 8 * 16;
        uint4 w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int j = j0 + i * kStep;
          w[i] = ld_shared_v4(B + at + i * kStep * 128);
          if (j >= len) w[i] = make_uint4(0, 0, 0, 0);  // behind the chunk's end: another chunk's or sequence's row
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          const uint64_t ff = f2_pack(f[i], f[i]), zero = f2_pack(0.f, 0.f), minus = f2_pack(-1.f, -1.f);
          uint64_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = f2_fma(f2_pack(bf16lo(in[k]), bf16hi(in[k])), ff, zero);
#pragma unroll
          for (int term = 0; term < TERMS; ++term) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float a, b;
              f2_unpack(v[k], a, b);
              h[k] = pack_bf16x2(a, b);
              if (term + 1 < TERMS) v[k] = f2_fma(f2_pack(bf16lo(h[k]), bf16hi(h[k])), minus, v[k]);
            }
            st_shared_v4((term == 0 ? B : rest + (term - 1) * (kC * DA * 2)) + at + i * kStep * 128, h[0], h[1], h[2], h[3]);
          }
        }
      }
      for (int v = t0 + len * 8; v < kC * 8; v += 512)
        for (int x = 0; x < DC / 64; ++x) st_shared_v4(Ct + x * kPanel + v * 16, 0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(smem_addr(&b_ready));
    };

    if (warp < 8) {
      int m = 0, k = 0;  // chunk of all pieces, piece
      if (live) do {
        powers(k);
        const Piece& q = pieces[k % kPieces];
        for (int left = q.len; left > 0; left -= kC, ++m) {
          const int len = left < kC ? left : kC;
          warp_wait(&p_full, m);
          tc_fence_after();
          // 16 columns at a time (a short loop: the warps of the roles share
          // the instruction cache); P's two bf16 terms lie over their scores
          // (one term, rounded once more than the output, gives 1.4 times the
          // error of the output's rounding alone)
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            const int j0 = half * 64 + b * 16, lo_row = 32 * quarter;
            uint32_t w[16];
            if (rev ? j0 + 15 < lo_row || j0 >= len : j0 > lo_row + 31) {  // empty for all of the warp's rows
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = 0;
            } else {
              uint32_t v[16];
              tmem_ld16(lanes_at + kColP + j0, v);
              // the powers of 16 columns' distances (masked ones: whatever lies there)
              const float* t = tab + (rev ? j0 - row : kC - 1 - row + j0);
              float f[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) f[k] = t[k];
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) f[k] *= __uint_as_float(v[k]);
              if (rev ? j0 < lo_row + 31 || j0 + 16 > len : j0 + 15 > lo_row) {  // a masked score may be infinite or NaN
                const int last = rev ? len : row + 1, first = rev ? row : 0;
#pragma unroll
                for (int k = 0; k < 16; ++k) f[k] = j0 + k >= first && j0 + k < last ? f[k] : 0.f;
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                w[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
                w[8 + k] = pack_bf16x2(f[2 * k] - bf16lo(w[k]), f[2 * k + 1] - bf16hi(w[k]));
              }
            }
            tmem_st8(lanes_at + kColP + j0, w);
            tmem_st8(lanes_at + kColP + j0 + 8, w + 8);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(smem_addr(&p_ready));

          // b's weighted rows: a b^T has read b, and the last chunk's sums
          // have read its terms
          if (m > 0) warp_wait(&u_full, m - 1);
          const int ib = m * kTiles + 1;
          warp_wait(&full[ib % kSlots], (uint32_t)(ib / kSlots));
          if (len < kC) warp_wait(&full[(ib + 1) % kSlots], (uint32_t)((ib + 1) / kSlots));
          split(len, m, tid);

          warp_wait(&o_full, m);
          tc_fence_after();
          const bool in = row < len;
          const int e = rev ? len - row - p.s.shift : row + 1 - p.s.shift;
          const float coef = in ? p.s.in_scale * pw[e] : 0.f;
          bf16_t* out = static_cast<bf16_t*>(p.s.out) + (long long)(chunk_at(q, left) + row) * p.s.os + (long long)q.head * Dc;
          uint64_t sum = 0;  // 0, or NaN where a value is not finite
#pragma unroll 1
          for (int c0 = half * (DC / 2); c0 < (half + 1) * (DC / 2); c0 += 32) {
            uint32_t x[32], y[32];
            tmem_ld16(lanes_at + kColO1 + c0, x);
            tmem_ld16(lanes_at + kColO2 + c0, y);
            tmem_ld16(lanes_at + kColO1 + c0 + 16, x + 16);
            tmem_ld16(lanes_at + kColO2 + c0 + 16, y + 16);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) sum = f2_fma(f2_pack(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), 0ull, sum);
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              w[k] = ok ? pack_bf16x2(fmaf(coef, __uint_as_float(y[2 * k]), __uint_as_float(x[2 * k])),
                                      fmaf(coef, __uint_as_float(y[2 * k + 1]), __uint_as_float(x[2 * k + 1])))
                        : 0x7fc07fc0u;
            if (in) {
              if (p.s.wide_out) {
                if (FULL || c0 < Dc) st_global_v8(out + c0, w);
                if (FULL || c0 + 16 < Dc) st_global_v8(out + c0 + 16, w + 8);
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (FULL || c0 + 8 * k < Dc) reinterpret_cast<uint4*>(out + c0)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
              }
            }
          }
          const bool bad = in && ok && f2_hsum(sum) != 0.f;
          if (__any_sync(0xffffffffu, bad))
            masked_row(p.s, tab, lanes_at + kColO2, chunk_at(q, left), q.head, row, len, half * (DC / 2), (half + 1) * (DC / 2), coef, bad);
          tc_fence_before();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(smem_addr(&o_free));
        }
      } while (more(++k, m));
      if (cut && !ok) poison_range<false>(p.s, blockIdx.x, lane);
    } else {
      // the state: a thread holds S[d0 .. d0 + DH)[row]
      constexpr int DH = DA / 2;
      const int d0 = half * DH;
      float S[DH];
      const float* from = cut ? p.s.piece_state : p.s.s_in;
      int m = 0, k = 0;
      if (live) do {
        powers(k);
        const Piece& q = pieces[k % kPieces];
        const long long st = (cut ? q.id : (long long)q.seq * p.s.H + q.head) * Da * Dc;
        if (from && row < Dc) {
          if (p.s.transposed) {
#pragma unroll
            for (int d = 0; d < DH; d += 4) {
              float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
              if (FULL || d0 + d < Da) v = *reinterpret_cast<const float4*>(from + st + (long long)row * Da + d0 + d);
              S[d] = v.x, S[d + 1] = v.y, S[d + 2] = v.z, S[d + 3] = v.w;
            }
          } else {
#pragma unroll
            for (int d = 0; d < DH; ++d) S[d] = FULL || d0 + d < Da ? from[st + (d0 + d) * Dc + row] : 0.f;
          }
        } else {
#pragma unroll
          for (int d = 0; d < DH; ++d) S[d] = 0.f;
        }
        // S as two bf16 terms for a S: 8 values of this thread's row, [DC
        // rows][DA] in the 128-byte swizzle
        auto put = [&](int d) {
          const int at = d0 + d;
          const uint32_t to = at / 64 * (DC * 128) + row * 128 + (((at / 8) ^ row) & 7) * 16;
          if (row < DC) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              h[k] = pack_bf16x2(S[d + 2 * k], S[d + 2 * k + 1]);
              float x, y;
              f2_unpack(f2_fma(f2_pack(bf16lo(h[k]), bf16hi(h[k])), f2_pack(-1.f, -1.f), f2_pack(S[d + 2 * k], S[d + 2 * k + 1])), x, y);
              l[k] = finite_or_large(pack_bf16x2(x, y));  // (NaN behind an infinity, which keeps its sign so)
            }
            st_shared_v4(s_buf + to, h[0], h[1], h[2], h[3]);
            st_shared_v4(s_low + to, l[0], l[1], l[2], l[3]);
          }
        };
        // ready for chunk m, whose scores this warp sees first: the next ones
        // follow on this, so that it cannot miss a phase of p_full
        auto put_done = [&](int m) {
          fence_proxy_async_smem();
          warp_wait(&p_full, m);
          if (ok && lane == 0) mbar_arrive(smem_addr(&s_ready));
        };
        if (q.len > 0) {
#pragma unroll
          for (int d = 0; d < DH; d += 8) put(d);
          put_done(m);
        }
        for (int left = q.len; left > 0; left -= kC, ++m) {
          // this group's half of b's weighted rows
          const int ib = m * kTiles + 1, len = left < kC ? left : kC;
          warp_wait(&full[ib % kSlots], (uint32_t)(ib / kSlots));
          if (len < kC) warp_wait(&full[(ib + 1) % kSlots], (uint32_t)((ib + 1) / kSlots));
          split(len, m, tid);
          const float decay = pw[len];
          warp_wait(&u_full, m);
          warp_wait(&o_full, m);  // a S has read the state before
          tc_fence_after();
          const bool next = left > kC;
#pragma unroll
          for (int d = 0; d < DH; d += 16) {
            uint32_t v[16];
            tmem_ld16(lanes_at + kColU + d0 + d, v);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) S[d + k] = fmaf(S[d + k], decay, __uint_as_float(v[k]));
            if (next) {
              put(d);
              put(d + 8);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(smem_addr(&u_free));
          if (next) put_done(m + 1);
        }
        // the state behind a sequence in one piece (others: joined before)
        if (row < Dc && p.s.s_out && !cut) {
          float* to = p.s.s_out + st;
          const float nan = __int_as_float(0x7fc00000);
          if (p.s.transposed) {
#pragma unroll
            for (int d = 0; d < DH; d += 4)
              if (FULL || d0 + d < Da) *reinterpret_cast<float4*>(to + (long long)row * Da + d0 + d) =
                  ok ? make_float4(S[d], S[d + 1], S[d + 2], S[d + 3]) : make_float4(nan, nan, nan, nan);
          } else {
#pragma unroll
            for (int d = 0; d < DH; ++d)
              if (FULL || d0 + d < Da) to[(d0 + d) * Dc + row] = ok ? S[d] : nan;
          }
        }
      } while (more(++k, m));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Every piece's own state, sum_j l^{len-1-j} b_j c_j^T over its tokens, in
// half chunks of 64 tokens: while the tensor cores take one half, eight warps
// weigh the rows of the next and eight others those of the one behind it
// (each group has its buffer of terms, and its latencies fall into the
// other's arithmetic), and all sixteen add the last whole chunk's sums, from
// one of two accumulators in TMEM, to the state (a quarter of a row of DA per
// thread).  The first two terms lie one behind the other and form one operand
// of 2 DA columns with sums of their own, to which the third term's are
// added: two instructions per 16 tokens instead of three (an operand of 128
// channels of b is read from shared memory once for both).  One
// barrier per stage says that a half's products are done: to the loads, to
// the terms' next writers and to the sums' readers.  The bound is HBM.
constexpr int kHalfPanel = kHalf * 128;  // bytes of 64 channels of a half chunk

template <int DA, int DC, bool FULL>
__global__ void __launch_bounds__(kTileThreads, 1) state_tc_kernel(const __grid_constant__ ScanTcParams p) {
  constexpr int kTileB = kHalf * DA * 2, kStage = StateSmem<DA, DC>::kStage, kSlots = StateSmem<DA, DC>::kSlots;
  constexpr uint32_t kColU = 2 * DA;  // columns between the accumulators: first terms' sums, then the others'
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxSlots], done[kMaxSlots], b_ready[2], u_free[2], drained;
  __shared__ uint32_t tmem_base;
  __shared__ Piece pieces[kPieces];
  // stages (b, c), then two buffers of three terms (which an operand of 64
  // channels reads into behind the last stage: rows of its product not used)
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u, rest = base + kSlots * kStage;
  const int tid = threadIdx.x, warp = warp_value(tid >> 5), lane = tid & 31;
  const int Da = FULL ? DA : p.s.Da, Dc = FULL ? DC : p.s.Dc;

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&done[s]), 1);
    }
    mbar_init(smem_addr(&drained), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&b_ready[b]), 8);
      mbar_init(smem_addr(&u_free[b]), 16);
    }
    mbar_fence_init();
  }
  if (warp == 17) tmem_alloc(smem_addr(&tmem_base), 4 * DA);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_value(tmem_base);
  pdl_wait();
  pdl_trigger();
  const bool rev = p.s.reverse;
  PieceWalk walk(p.s, blockIdx.x);
  Piece pc;
  // the next piece that has a state of its own: a last one's is part of the
  // final state only
  auto step = [&] {
    do {
      if (!walk.next(p.s, blockIdx.x, &pc)) return false;
    } while (pc.last && !p.s.s_out);
    return true;
  };
  bool live = step();
  int nchunk = live ? (pc.len + kC - 1) / kC : 0;
  auto chunk_len = [&](int n) { return pc.len - n * kC < kC ? pc.len - n * kC : kC; };
  auto chunk_at = [&](int n) { return rev ? pc.first + pc.len - n * kC - chunk_len(n) : pc.first + n * kC; };
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !poll(smem_addr(bar), parity & 1u, p.wait_ns)) {
      report_error(p.dev_err, ATTNRES_DEVERR_WAIT_TIMEOUT);
      ok = false;
    }
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    wait(bar, parity);
    ok = __all_sync(0xffffffffu, ok);
  };
  // Nothing is passed on once a wait has run out: the other roles' waits run
  // out, too, and the results are NaN.
  auto commit = [&](uint64_t* bar) {
    if (ok) tc_commit_warp(smem_addr(bar));
  };
  // no product of this warp is under way when shared memory and TMEM are given back
  auto drain = [&](uint64_t* bar) {
    if (!ok) {
      tc_commit_warp(smem_addr(bar));
      mbar_wait_bounded(smem_addr(bar), 0);
    }
  };

  if (warp == 16) {
    if (lane == 0) {
      int i = 0;  // half of all pieces
      for (int k = 1; ok; ++k) {
        for (int n = 0; n < 2 * nchunk; ++n, ++i) {
          const int st = i % kSlots, t = chunk_at(n / 2) + n % 2 * kHalf;
          wait(&done[st], (uint32_t)(i / kSlots) + 1u);
          if (!ok) break;
          const uint32_t fb = smem_addr(&full[st]), to = base + st * kStage;
          mbar_arrive_expect_tx(fb, kStage);
          if (i + 1 == p.withhold1) continue;
#pragma unroll
          for (int x = 0; x < DA; x += 64) tma_load_3d(to + x / 64 * kHalfPanel, &p.mb, x, pc.head, t, fb);
#pragma unroll
          for (int x = 0; x < DC; x += 64) tma_load_3d(to + kTileB + x / 64 * kHalfPanel, &p.mc, x, pc.head, t, fb);
        }
        if (!live || !ok) break;
        // the next piece, which its first halves' barriers publish; behind
        // the last two barriers of no bytes
        live = step();
        if (!live) pc.len = 0;
        nchunk = (pc.len + kC - 1) / kC;
        pieces[k % kPieces] = pc;
        if (!live) {
          for (int e = 0; e < 2; ++e, ++i) {
            wait(&done[i % kSlots], (uint32_t)(i / kSlots) + 1u);
            if (!ok) break;
            mbar_arrive(smem_addr(&full[i % kSlots]));
          }
          break;
        }
      }
      // the CTA never exits under a copy
      const int armed = i < kSlots ? i : kSlots, skip = p.withhold1 > 0 && i >= p.withhold1 ? (p.withhold1 - 1) % kSlots : -1;
      for (int st = 0; st < armed; ++st)
        if (st != skip) mbar_wait_bounded(smem_addr(&full[st]), (uint32_t)((i - 1 - st) / kSlots) & 1u);
    }
    __syncwarp();
  } else if (warp == 17) {
    constexpr uint32_t kI2 = tc_idesc_bf16(128, 2 * DA, true, true), kI1 = tc_idesc_bf16(128, DA, true, true);
    nchunk = warp_value(nchunk);
    int i = 0;
    for (int k = 1; nchunk > 0 && ok; ++k) {
      for (int end = i + 2 * nchunk; i < end && ok; ++i) {
        const int st = i % kSlots, n = i / 2;
        const uint32_t d = tmem + (n & 1) * kColU, more = i % 2;
        const uint64_t dc = smem_desc_mn128(base + st * kStage + kTileB, kHalfPanel);
        const uint64_t dt = smem_desc_mn128(rest + (i & 1) * 3 * kTileB, kHalfPanel);
        warp_wait(&b_ready[i & 1], (uint32_t)(i / 2));
        if (i % 2 == 0) warp_wait(&u_free[n & 1], (uint32_t)(n / 2) + 1u);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kHalf / 16; ++kk) {
          tc_mma_bf16_warp(d, dc + kk * 128, dt + kk * 128, kI2, kk > 0 ? 1u : more);
          tc_mma_bf16_warp(d + DA, dc + kk * 128, dt + 2 * kTileB / 16 + kk * 128, kI1, 1u);
        }
        commit(&done[st]);
      }
      warp_wait(&b_ready[0], (uint32_t)(i / 2));  // of the next piece's first half, or of the end
      pc.len = warp_value(pieces[k % kPieces].len);
      nchunk = ok ? (pc.len + kC - 1) / kC : 0;
    }
    drain(&drained);
    __syncwarp();
  } else {
    // thread: row `row` of the state, DA / 4 of its values from d0
    constexpr int DQ = DA / 4;
    const int row = 32 * (warp & 3) + lane, d0 = (warp >> 2) * DQ;
    const uint32_t from = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + d0;
    float S[DQ];
#pragma unroll
    for (int d = 0; d < DQ; ++d) S[d] = 0.f;
    float g = 0.f;
    // chunk n of the piece, m of all
    auto add = [&](int n, int m) {
      const float decay = decay_pow(g, chunk_len(n));
      const int i = 2 * m + 1;  // its last half
      warp_wait(&done[i % kSlots], (uint32_t)(i / kSlots));
      tc_fence_after();
#pragma unroll
      for (int d = 0; d < DQ; d += 16) {
        uint32_t v[16], w[16];
        tmem_ld16(from + (m & 1) * kColU + d, v);
        tmem_ld16(from + (m & 1) * kColU + DA + d, w);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) S[d + k] = fmaf(S[d + k], decay, __uint_as_float(v[k]) + __uint_as_float(w[k]));
      }
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(smem_addr(&u_free[m & 1]));
    };
    const int group = warp >> 3, tg = tid & 255;
    int m = 0;  // chunk of all pieces
    for (int k = 1; nchunk > 0 && ok; ++k) {
      g = __ldg(p.s.log_decay + pc.head);
#pragma unroll
      for (int d = 0; d < DQ; ++d) S[d] = 0.f;
      for (int n = 0; n < nchunk; ++n, ++m) {
        const int i = 2 * m + group, st = i % kSlots, len = chunk_len(n), j0 = group * kHalf;  // rows j0 .. of the chunk
        const uint32_t B = base + st * kStage, Ct = B + kTileB, T = rest + group * 3 * kTileB;
        warp_wait(&full[st], (uint32_t)(i / kSlots));
        if (i >= 2) warp_wait(&done[(i - 2) % kSlots], (uint32_t)((i - 2) / kSlots));  // the terms' last readers
        // vectors of 8 channels: rows tg / 8 and 32 further of every panel of 64
        constexpr int kVecs = 2 * DA / 64;
        float f[2];
        uint4 w[kVecs];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int j = j0 + tg / 8 + 32 * r;
          f[r] = j < len ? p.s.up_scale * decay_pow(g, p.s.shift + (rev ? j : len - 1 - j)) : 0.f;
#pragma unroll
          for (int x = 0; x < DA / 64; ++x) {
            const int v = r * (DA / 64) + x;
            w[v] = ld_shared_v4(B + x * kHalfPanel + r * 4096 + tg * 16);
            if (j >= len) w[v] = make_uint4(0, 0, 0, 0);  // behind the chunk's end: another chunk's or sequence's row
          }
          if (j >= len) {
#pragma unroll
            for (int x = 0; x < DC / 64; ++x) st_shared_v4(Ct + x * kHalfPanel + r * 4096 + tg * 16, 0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          const uint32_t at = v % (DA / 64) * kHalfPanel + v / (DA / 64) * 4096 + tg * 16, in[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
          const float fv = f[v / (DA / 64)];
          uint32_t th[4], tm[4], tl[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = bf16lo(in[k]) * fv, b = bf16hi(in[k]) * fv;
            th[k] = pack_bf16x2(a, b);
            const float a1 = a - bf16lo(th[k]), b1 = b - bf16hi(th[k]);
            tm[k] = pack_bf16x2(a1, b1);
            tl[k] = pack_bf16x2(a1 - bf16lo(tm[k]), b1 - bf16hi(tm[k]));
          }
          st_shared_v4(T + at, th[0], th[1], th[2], th[3]);
          st_shared_v4(T + kTileB + at, tm[0], tm[1], tm[2], tm[3]);
          st_shared_v4(T + 2 * kTileB + at, tl[0], tl[1], tl[2], tl[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(smem_addr(&b_ready[group]));
        if (n > 0) add(n - 1, m - 1);
      }
      add(nchunk - 1, m - 1);
      if (row < Dc) {
        float* to = p.s.piece_state + (long long)pc.id * Da * Dc;
        const float nan = __int_as_float(0x7fc00000);
        if (p.s.transposed) {
#pragma unroll
          for (int d = 0; d < DQ; d += 4)
            if (FULL || d0 + d < Da) *reinterpret_cast<float4*>(to + (long long)row * Da + d0 + d) =
                ok ? make_float4(S[d], S[d + 1], S[d + 2], S[d + 3]) : make_float4(nan, nan, nan, nan);
        } else {
#pragma unroll
          for (int d = 0; d < DQ; ++d)
            if (FULL || d0 + d < Da) to[(d0 + d) * Dc + row] = ok ? S[d] : nan;
        }
      }
      // the next piece, in its first chunk's half of this group
      const int i = 2 * m + group;
      warp_wait(&full[i % kSlots], (uint32_t)(i / kSlots));
      pc = pieces[k % kPieces];
      nchunk = ok ? (pc.len + kC - 1) / kC : 0;
      if (ok && nchunk == 0 && lane == 0) mbar_arrive(smem_addr(&b_ready[group]));  // the products' warp reads of the end behind it
    }
    if (!ok) poison_range<true>(p.s, blockIdx.x, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 4 * DA);
  }
}

template <typename K>
cudaError_t launch_tile(K kern, SmemOptIn& optin, int bytes, int threads, int64_t ctas, const ScanTcParams& p, const DeviceInfo& di,
                        cudaStream_t stream) {
  if (bytes + 2048 > di.max_smem_optin) return cudaErrorInvalidValue;
  const cudaError_t e = optin.ensure(reinterpret_cast<const void*>(kern), bytes);
  return e != cudaSuccess ? e : launch_kernel(kern, dim3((unsigned)ctas), dim3(threads), (size_t)bytes, stream, p);
}

template <int DA, int DC, int TERMS, bool FULL>
cudaError_t launch_scan_tile(const ScanTcParams& p, const DeviceInfo& di, cudaStream_t stream) {
  static SmemOptIn optin;
  return launch_tile(scan_tc_kernel<DA, DC, TERMS, FULL>, optin, ScanSmem<DA, DC, TERMS>::kBytes, kScanThreads,
                     p.s.parts > 0 ? p.s.parts * p.s.gang : (int64_t)p.s.N * p.s.H, p, di, stream);
}
template <int DA, int DC>
cudaError_t launch_scan_size(const ScanTcParams& p, bool three, const DeviceInfo& di, cudaStream_t stream) {
  const bool full = p.s.Da == DA && p.s.Dc == DC;
  if (three) return full ? launch_scan_tile<DA, DC, 3, true>(p, di, stream) : launch_scan_tile<DA, DC, 3, false>(p, di, stream);
  return full ? launch_scan_tile<DA, DC, 2, true>(p, di, stream) : launch_scan_tile<DA, DC, 2, false>(p, di, stream);
}
cudaError_t launch_scan_dims(const ScanTcParams& p, bool three, const DeviceInfo& di, cudaStream_t stream) {
  if (p.s.Da > 64) return p.s.Dc > 64 ? launch_scan_size<128, 128>(p, three, di, stream) : launch_scan_size<128, 64>(p, three, di, stream);
  return p.s.Dc > 64 ? launch_scan_size<64, 128>(p, three, di, stream) : launch_scan_size<64, 64>(p, three, di, stream);
}

template <int DA, int DC, bool FULL>
cudaError_t launch_state_tile(const ScanTcParams& p, const DeviceInfo& di, cudaStream_t stream) {
  static SmemOptIn optin;
  return launch_tile(state_tc_kernel<DA, DC, FULL>, optin, StateSmem<DA, DC>::kBytes, kTileThreads, (int64_t)p.s.parts * p.s.gang, p, di, stream);
}
template <int DA, int DC>
cudaError_t launch_state_size(const ScanTcParams& p, const DeviceInfo& di, cudaStream_t stream) {
  return p.s.Da == DA && p.s.Dc == DC ? launch_state_tile<DA, DC, true>(p, di, stream) : launch_state_tile<DA, DC, false>(p, di, stream);
}
cudaError_t launch_state_dims(const ScanTcParams& p, const DeviceInfo& di, cudaStream_t stream) {
  if (p.s.Da > 64) return p.s.Dc > 64 ? launch_state_size<128, 128>(p, di, stream) : launch_state_size<128, 64>(p, di, stream);
  return p.s.Dc > 64 ? launch_state_size<64, 128>(p, di, stream) : launch_state_size<64, 64>(p, di, stream);
}

// [T, H, D] with tokens `stride` elements apart, boxes of 64 channels of a head
bool token_map(CUtensorMap* m, const void* ptr, int64_t T, int H, int D, int64_t stride, int tokens = kC) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)tokens};
  return make_tensor_map(m, ptr, 3, dims, strides, box);
}

}  // namespace

bool scan_tc_dims(int Dk, int Dv, int dtype) { return dtype == ATTNRES_BF16 && Dk <= 128 && Dv <= 128 && Dk % 16 == 0 && Dv % 16 == 0; }

// (a chunk's HBM time on one of 152 SMs is 23 ns per channel)
static CutRule scan_tc_rule(int Dk, int Dv, int sm_count) {
  return {kC, 1, sm_count, 0.55, 23. * (Dk > 64 || Dv > 64 ? 128 : 64)};
}
static Cut scan_tc_cut(int64_t T, int H, int Dk, int Dv, int N, int sm_count) {
  return choose_cut(T, H, Dk, Dv, N, scan_tc_rule(Dk, Dv, sm_count));
}

bool scan_tc_in_pieces(int64_t T, int H, int Dk, int Dv, int N) {
  DeviceInfo di;
  return device_info(&di) == cudaSuccess && scan_tc_cut(T, H, Dk, Dv, N, di.sm_count).parts > 0;
}

int64_t scan_tc_workspace(int64_t T, int H, int Dk, int Dv, int N) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return -1;
  return piece_bytes(T, H, Dk, Dv, N, scan_tc_rule(Dk, Dv, di.sm_count));
}

bool scan_tc_ok(const ScanArgs& s) {
  auto rows = [](const void* p, long long stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; };
  auto state = [](const float* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  return rows(s.a, s.as) && rows(s.b, s.bs) && rows(s.c, s.cs) && rows(s.out, s.os) && state(s.s_in) && state(s.s_out) && s.T > 0 &&
         s.T * 2 < INT32_MAX && (int64_t)s.N * s.H < INT32_MAX;
}

cudaError_t launch_scan_tc(const ScanArgs& s, void* workspace, int64_t workspace_bytes, ScanReady ready, int* dev_err, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  ScanTcParams p{};
  p.s = s;
  p.s.wide_out = (reinterpret_cast<uintptr_t>(s.out) & 31) == 0 && s.os % 16 == 0;
  if (!token_map(&p.ma, s.a, s.T, s.H, s.Da, s.as) || !token_map(&p.mb, s.b, s.T, s.H, s.Da, s.bs) ||
      !token_map(&p.mc, s.c, s.T, s.H, s.Dc, s.cs))
    return cudaErrorInvalidValue;
  p.dev_err = dev_err;
  p.wait_ns = wait_limit_ns();
  p.withhold1 = debug_withhold_row1();
  p.s.chunk = kC;
  const Cut cut = scan_tc_cut(s.T, s.H, s.Da, s.Dc, s.N, di.sm_count);
  p.s.parts = cut.parts;
  p.s.gang = cut.gang;
  if (p.s.parts > 0) {
    const PieceLayout L = piece_layout(s.H, s.Da, s.Dc, s.N, cut);
    if (L.total > workspace_bytes) return cudaErrorInvalidValue;
    piece_place(p.s, L, workspace);
  }
  if (p.s.parts > 0 && ready < kStates) {
    if (ready < kTables) e = launch_piece_plan(p.s, stream);
    if (e != cudaSuccess) return e;
    ScanTcParams ps = p;
    if (!token_map(&ps.mb, s.b, s.T, s.H, s.Da, s.bs, kHalf) || !token_map(&ps.mc, s.c, s.T, s.H, s.Dc, s.cs, kHalf))
      return cudaErrorInvalidValue;
    e = launch_state_dims(ps, di, stream);
    if (e == cudaSuccess) e = launch_piece_combine(p.s, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_scan_dims(p, s.s_out && p.s.parts == 0, di, stream);
}

}  // namespace attnres
