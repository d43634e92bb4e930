// attn_bwd.cu -- gradient of the block-sparse attention (vsa_sparse_attn_bwd) for sm_100a.
//
// With P = exp(scale * Q K^T - lse) on the kept block pairs (0 elsewhere, and on rows whose lse
// is -inf) and delta_i = sum_d dO_id O_id - dlse_i:
//
//   dV = P^T dO     dP = dO V^T     dS = P o (dP - delta)     dQ = scale dS K     dK = scale dS^T Q
//
// P is recomputed from the forward call's log-sum-exp; nothing of size N x N is stored.
//
// Two launches.  bwd_prep_kernel turns each row's lse and delta into the two terms the main
// kernel adds (-lse * log2 e and -delta, -inf and 0 for rows that see nothing) and validates the
// key lists into one bitset per query block.  sparse_attn_bwd_kernel then runs two kinds of CTA:
//
//   key CTAs    own one key block: they walk the query blocks that keep it (its column of the
//               bitset) and accumulate dV and dK in TMEM.  S^T = K Q^T and dP^T = V dO^T have the
//               keys as TMEM lanes, so that P^T and dS^T are written over them as packed bf16 and
//               read from TMEM as the A operands of dV += P^T dO and dK += dS^T Q.
//   query CTAs  own one query block: they walk its kept key blocks and accumulate dQ += dS K and the
//               row's mean key m += P K; S = Q K^T and dP = dO V^T have the queries as lanes.
//
// S and dP are computed twice so that every gradient has one owner: no atomics, no fp32 copy of dQ in
// memory, the same bits on every run.
//
// Why the mean key.  The sum of dS over a row is known (d_lse; 0 without one), and what all of a row's keys
// have in common drops out of dQ.  It does not drop out of errors: rounding dS to bf16, and a delta that is
// off, leave a sum e that adds e m to dQ.  The query CTA adds up e in fp32 and takes e m off again.  Without
// it dQ measured 0.0043 (2-norm, relative) from the gradient of the given O in 64 bits on keys with a common part
// twice their own size, against 0.0024 with it; the eighth product costs 0.4 of 3.7 ms (12 heads x 32760 rows, d 128,
// 21% kept).  A block's unweighted mean key instead, one K = 16 step, was faster by 0.1 ms but left 0.0036 to 0.0041.
// With a bf16 O alone the sum of a row is not known so well, and dQ was 0.0093 from the gradient of the unrounded
// attention; with O's rounding errors beside it 0.0025.  dK takes delta as it is, in which the forward call's rounding
// of P is left: 0.0025 to 0.0027.  Rounding P, dS and the result to bf16 alone comes to 0.0024.
//
// What bounds it.  3.66 ms there after a pause: executed products at 1480 TFLOP/s (0.89 of cuBLAS's burst); back to
// back 4.04 ms under the power cap, 1340 (0.96 of the sustained rate).  A key block's loop takes 2500 cycles for 2048 of
// tensor time: the threads' chain S -> exponentials (MUFU, 1024) -> dP -> dS is the longer one.  What made it so short:
// S is freed as soon as it has been read, so that the next block's S runs under the exponentials; P and dS go over
// dP; barriers are tested ahead; the issuing lane is elected, which lets tcgen05.mma run ahead of it (8 products
// 770 -> 560 cycles against a branch on lane 0).
//
// Each CTA: 384 threads in three warpgroups (registers rebalanced as in the forward kernel).
//   warps 0-3 / 4-7  one lane (row of S) per thread, the first / second half of its columns:
//                    p = exp2(s * scale * log2 e - lse * log2 e) in fp32, packed to bf16 for its
//                    product, kept in registers in fp32 for dS = p * (dP - delta)
//   warp 8 / 10      TMA producers of the two rings (X: Q or K; Y: dO or V)
//   warp 11          bulk copies of the rows' terms (key CTAs)
//   warp 9           the tcgen05 issuer (one lane); owns TMEM
// P and dS are rounded to bf16 because both operands of the tensor product have one type; every
// sum (S, dP, dV, dK, dQ) is held in fp32.
//
// Operand tiles use the 128-byte swizzle as in the forward kernel; every wait is bounded, and on a
// timeout the CTA drains its copies and MMAs, frees TMEM and returns.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace vsa {

namespace {

constexpr int kBwdThreads = 384;
constexpr int kWarpX = 8, kWarpMma = 9, kWarpY = 10, kWarpT = 11;
constexpr int kBM = 128;
constexpr int kRegsSoftmax = 208, kRegsCtl = 88;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsCtl == 384 * 168, "register split must equal the launch total");

template <int D, int BN>
struct BwdCfg {
  // Ring stages of X (Q or K) and Y (dO or V) and of the rows' terms.  A tile takes about 1500 cycles to
  // arrive; with a spare stage of each no product waits for it.  The spare X stage is given up where the
  // bitset of a very long head needs its place.
  static constexpr int NX_MOST = 3, NY = 2, NT = 2;
  static constexpr int A_BYTES = kBM * D * 2;             // a resident tile (M = 128 lanes, BN rows loaded)
  static constexpr int T_BYTES = BN * D * 2;              // a ring tile
  static constexpr int ST_BYTES = 2 * BN * 4;             // the rows' two terms of a block
  static constexpr int PANELS = D / 64;
  static constexpr int OFF_A0 = 0;                        // K (key CTA) or Q (query CTA)
  static constexpr int OFF_A1 = OFF_A0 + A_BYTES;         // V or dO
  // X is the last ring, behind it the small things: its number of stages moves only those.
  static constexpr int OFF_Y = OFF_A1 + A_BYTES;
  static constexpr int OFF_X = OFF_Y + NY * T_BYTES;
  static constexpr int NBAR = 28;
  // behind the nx stages of X: the rows' terms of NT blocks, barriers, TMEM base and abort flag, bitset
  static constexpr int OFF_BAR = NT * ST_BYTES;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int OFF_BITS = OFF_MISC + 16;
  // TMEM columns.  S; dP with P and dS (packed bf16) written over it once it has been read: each half
  // of the columns holds its threads' dP, then P and dS.  Behind them the products with P (dV, or the mean
  // key) and with dS (dK or dQ).
  static constexpr int TM_S = 0, TM_DP = BN, TM_P = TM_DP, TM_DS = TM_DP + BN / 4, TM_ACC_P = 2 * BN, TM_ACC_DS = 2 * BN + D;
  static constexpr int TM_COLS = 2 * BN + 2 * D <= 256 ? 256 : 512;
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(kBM, BN, false, false);
  static constexpr uint32_t IDESC_G = idesc_bf16_f32(kBM, D, false, true);
  static int smem_bytes(int nx, int nwords) { return OFF_X + nx * T_BYTES + OFF_BITS + 4 * nwords; }
  static int stages(int nwords) { return smem_bytes(NX_MOST, nwords) <= kMaxSmem ? NX_MOST : NX_MOST - 1; }
};

enum {
  B_A0 = 0,
  B_A1 = 1,
  B_FULL_X = 2,    // +stage
  B_REL_X = 5,     // +stage
  B_FULL_Y = 8,    // +stage
  B_REL_Y = 10,    // +stage
  B_FULL_T = 12,   // +stage of the rows' terms
  B_S = 14,        // S (dP) is in TMEM
  B_DP = 15,
  B_SREAD = 16,    // S has been read into registers
  B_P = 17,        // P is written
  B_DS = 18,       // dS is written
  B_FINAL = 19,
};
constexpr int kSoftmaxWarps = 8;  // arrivals on B_SREAD, B_P and B_DS: one per warp

// The set bits of a bitset in ascending order.
struct BitWalk {
  const uint32_t* w;
  int at;
  uint32_t cur;
  __device__ explicit BitWalk(const uint32_t* words) : w(words), at(0), cur(words[0]) {}
  __device__ int next() {  // only called while a bit is left
    while (cur == 0u) cur = w[++at];
    const int b = at * 32 + __ffs(cur) - 1;
    cur &= cur - 1u;
    return b;
  }
};

// 2^x of a packed pair.  All on the hardware exponential: moving one pair in 8 (2, 3) to the FMA pipe, as
// the forward kernel does, measured 0.7% (1.2%, 1.7%) slower on 12 x 32760 rows.
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x) {
  float x0, x1;
  f2_split(x, x0, x1);
  return f2_make(fast_exp2(x0), fast_exp2(x1));
}

__device__ __forceinline__ uint32_t pack_pair(uint64_t x) {
  float x0, x1;
  f2_split(x, x0, x1);
  return pack_bf16x2(x0, x1);
}

__device__ __forceinline__ uint64_t unpack_pair(uint32_t x) {
  return f2_make(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// N consecutive TMEM columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t* r) {
#pragma unroll
  for (int c = 0; c < N / 32; ++c) tmem_ld32_async(taddr + c * 32, r + c * 32);
  tmem_wait_ld();
  reg_fence<N>(r);
}

// One lane's COLS accumulator columns (less `off` times those at `other`) -> a bf16 row of the swizzled staging
// tile.
template <int BN, int COLS, bool kOther>
__device__ __forceinline__ void stage_rows(uint8_t* stage, uint32_t taddr, uint32_t other, float off, int col0, int row,
                                           bool live, bool have, float scale) {
#pragma unroll 1
  for (int c = 0; c < COLS / 32; ++c) {
    float o[32];
    tmem_ld32(taddr + c * 32, o);
    if constexpr (kOther) {
      float m[32];
      tmem_ld32(other + c * 32, m);
#pragma unroll
      for (int x = 0; x < 32; ++x) o[x] = fmaf(-off, m[x], o[x]);
    }
#pragma unroll
    for (int x = 0; x < 32; ++x) o[x] = have && live ? o[x] * scale : 0.f;
    if (row < BN) {
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        uint4 v4;
        v4.x = pack_bf16x2(o[q4 * 8 + 0], o[q4 * 8 + 1]);
        v4.y = pack_bf16x2(o[q4 * 8 + 2], o[q4 * 8 + 3]);
        v4.z = pack_bf16x2(o[q4 * 8 + 4], o[q4 * 8 + 5]);
        v4.w = pack_bf16x2(o[q4 * 8 + 6], o[q4 * 8 + 7]);
        const int col = col0 + c * 32 + q4 * 8;
        const int dc = col >> 6, cc = (col & 63) >> 3;
        *reinterpret_cast<uint4*>(stage + dc * (BN * 128) + row * 128 + ((cc ^ (row & 7)) << 4)) = v4;
      }
    }
  }
}

// kKey: a key CTA (dK, dV of block `blk`); else a query CTA (dQ of block `blk`).
template <int D, int BN, bool kKey>
__device__ __forceinline__ void bwd_cta(const BwdMaps* mn, const BwdMaps* mp, const BwdArgs& a, int bh, int blk,
                                        uint8_t* smem) {
  using C = BwdCfg<D, BN>;
  constexpr int H = BN / 2;  // columns per thread
  const uint32_t sbase = smem_u32(smem);
  const int nx = a.nx;
  const uint32_t rest = C::OFF_X + nx * C::T_BYTES;
  auto bar = [&](int i) -> uint32_t { return sbase + rest + C::OFF_BAR + 8u * i; };
  volatile int* misc = reinterpret_cast<volatile int*>(smem + rest + C::OFF_MISC);  // [0] TMEM base, [1] abort flag
  volatile int* abort_flag = misc + 1;
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + rest + C::OFF_BITS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Geom& g = a.g;
  const int nwords = (g.nblk + 31) >> 5;
  const int kind = a.kinds[bh];

  if (!known_kind(g, kind)) {
    // unknown layout: this block's rows of the natural-order gradients become zeros
    pdl_wait();
    if (tid == 0 && blk == 0) atomicOr(a.err, kDevErrKind);
    const int r0 = blk * BN, r1 = min(r0 + BN, a.nat_rows);
    for (int x = tid; x < (r1 - r0) * (D / 8); x += kBwdThreads) {
      const size_t at = (static_cast<size_t>(bh) * a.nat_rows + r0) * (D / 8) + x;
      if (kKey) {
        static_cast<uint4*>(a.nat_dk)[at] = make_uint4(0, 0, 0, 0);
        static_cast<uint4*>(a.nat_dv)[at] = make_uint4(0, 0, 0, 0);
      } else {
        static_cast<uint4*>(a.nat_dq)[at] = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  const int rows = layout_rows(g, kind);
  const int nb_head = (rows + BN - 1) / BN;
  if (blk >= nb_head) {
    pdl_wait();  // no CTA ends before the kernel in front has
    return;
  }
  const BwdMaps* m = a.has_perm && kind != kSpatial ? mp : mn;

  // ---- barriers, the resident tiles, the blocks this CTA walks, TMEM ----
  bool stop = false;
  if (tid == kWarpX * 32) {
    stop = (*reinterpret_cast<volatile int*>(a.err) & kDevErrTimeout) != 0;
    mbar_init(bar(B_A0), 1);
    mbar_init(bar(B_A1), 1);
    for (int s = 0; s < C::NX_MOST; ++s) {
      mbar_init(bar(B_FULL_X + s), 1);
      mbar_init(bar(B_REL_X + s), 1);
    }
    for (int s = 0; s < C::NY; ++s) {
      mbar_init(bar(B_FULL_Y + s), 1);
      mbar_init(bar(B_REL_Y + s), 1);
    }
    for (int s = 0; s < C::NT; ++s) mbar_init(bar(B_FULL_T + s), 1);
    mbar_init(bar(B_S), 1);
    mbar_init(bar(B_DP), 1);
    mbar_init(bar(B_SREAD), kSoftmaxWarps);
    mbar_init(bar(B_P), kSoftmaxWarps);
    mbar_init(bar(B_DS), kSoftmaxWarps);
    mbar_init(bar(B_FINAL), 1);
    misc[1] = 0;
    mbar_init_fence();
    if (!stop) {  // K and V, or Q and dO, land while the list is built
      mbar_arrive_expect_tx(bar(B_A0), C::T_BYTES);
      mbar_arrive_expect_tx(bar(B_A1), C::T_BYTES);
#pragma unroll
      for (int c = 0; c < C::PANELS; ++c) {
        tma_load_3d(sbase + C::OFF_A0 + c * kBM * 128, kKey ? &m->k : &m->q, bar(B_A0), c * 64, blk * BN, bh);
        tma_load_3d(sbase + C::OFF_A1 + c * kBM * 128, kKey ? &m->v : &m->g, bar(B_A1), c * 64, blk * BN, bh);
      }
      tma_prefetch_desc(kKey ? &m->q : &m->k);
      tma_prefetch_desc(kKey ? &m->g : &m->v);
    }
  }
  if (warp == kWarpMma) {
    tmem_alloc(sbase + rest + C::OFF_MISC, C::TM_COLS);
    tmem_relinquish();
  }
  pdl_wait();  // from here the bitsets and the rows' terms
  const uint32_t* rbits = a.rbits + static_cast<size_t>(bh) * g.nblk * nwords;
  if (kKey) {
    for (int w = warp; w < nwords; w += kSoftmaxWarps) {
      if (warp >= kSoftmaxWarps) break;
      const int r = w * 32 + lane;
      const bool keeps = r < nb_head && ((rbits[static_cast<size_t>(r) * nwords + (blk >> 5)] >> (blk & 31)) & 1u);
      const uint32_t word = __ballot_sync(0xffffffffu, keeps);
      if (lane == 0) bits[w] = word;
    }
  } else if (warp < kSoftmaxWarps) {
    for (int w = tid; w < nwords; w += kSoftmaxWarps * 32) bits[w] = rbits[static_cast<size_t>(blk) * nwords + w];
  }
  tc_fence_before();
  stop = __syncthreads_or(stop);
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  if (stop) {  // another CTA gave up waiting: nothing is in flight here
    if (warp == kWarpMma) tmem_dealloc(tmem, C::TM_COLS);
    return;
  }
  int U = 0;
  for (int w = lane; w < nwords; w += 32) U += __popc(bits[w]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) U += __shfl_xor_sync(0xffffffffu, U, off);

  if (warp >= 8) {
    setmaxnreg_dec<kRegsCtl>();
    const bool one = elect_one();
    if (warp == kWarpX || warp == kWarpY) {
      // ================= TMA producers =================
      if (one) {
        const bool isx = warp == kWarpX;
        const CUtensorMap* tr = kKey ? (isx ? &m->q : &m->g) : (isx ? &m->k : &m->v);
        const int ns = isx ? nx : C::NY;
        const int full0 = isx ? B_FULL_X : B_FULL_Y, rel0 = isx ? B_REL_X : B_REL_Y;
        const uint32_t dst_r = sbase + (isx ? C::OFF_X : C::OFF_Y);
        BitWalk walk(bits);
        int st = 0, ph = 1, issued = 0;  // ph: parity of the release to wait for
        for (int n = 0; n < U; ++n) {
          const int b = walk.next();
          if (n >= ns && !mbar_wait(bar(rel0 + st), ph, abort_flag, a.err)) break;
          mbar_arrive_expect_tx(bar(full0 + st), C::T_BYTES);
#pragma unroll
          for (int c = 0; c < C::PANELS; ++c)
            tma_load_3d(dst_r + st * C::T_BYTES + c * BN * 128, tr, bar(full0 + st), c * 64, b * BN, bh);
          issued = n + 1;
          if (++st == ns) {
            st = 0;
            ph ^= 1;
          }
        }
        // every copy lands before the CTA exits; without an abort the products have waited for all but
        // the resident tiles of an empty list
        if (*abort_flag || U == 0) {
          mbar_wait_drain(bar(isx ? B_A0 : B_A1), 0, a.err);
          for (int s = 0; s < ns; ++s) {
            int last = -1;
            for (int n = s; n < issued; n += ns) last = n;
            if (last >= 0) mbar_wait_drain(bar(full0 + s), (last / ns) & 1, a.err);
          }
        }
      }
      __syncwarp();
    } else if (kKey && warp == kWarpT) {
      // ================= the rows' terms, two blocks ahead =================
      if (one && U > 0) {
        BitWalk walk(bits);
        int rs = 0, rp = 0, issued = 0;  // X stage and parity of the release two blocks back
        for (int n = 0; n < U; ++n) {
          const int b = walk.next(), st = n % C::NT;
          if (n >= C::NT) {  // block n - NT's dS is written once its dK product has been issued
            if (!mbar_wait(bar(B_REL_X + rs), rp, abort_flag, a.err)) break;
            if (++rs == nx) {
              rs = 0;
              rp ^= 1;
            }
          }
          mbar_arrive_expect_tx(bar(B_FULL_T + st), C::ST_BYTES);
          bulk_load(sbase + rest + st * C::ST_BYTES, a.terms + (static_cast<size_t>(bh) * g.nblk + b) * (2 * BN),
                    C::ST_BYTES, bar(B_FULL_T + st));
          issued = n + 1;
        }
        if (*abort_flag)
          for (int n = max(0, issued - C::NT); n < issued; ++n)
            mbar_wait_drain(bar(B_FULL_T + n % C::NT), (n / C::NT) & 1, a.err);
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      // ================= tcgen05 issuer =================
      if (one && U > 0) {
        const uint64_t da0 = sdesc_sw128(sbase + C::OFF_A0, 16, 1024), da1 = sdesc_sw128(sbase + C::OFF_A1, 16, 1024);
        // ring tiles as K-major (S, dP) and MN-major (gradient) B operands
        const uint64_t dxk = sdesc_sw128(sbase + C::OFF_X, 16, 1024);
        const uint64_t dyk = sdesc_sw128(sbase + C::OFF_Y, 16, 1024);
        const uint64_t dxm = sdesc_sw128(sbase + C::OFF_X, BN * 128, 1024);
        const uint64_t dym = sdesc_sw128(sbase + C::OFF_Y, BN * 128, 1024);
        constexpr uint64_t kStage = C::T_BYTES / 16;
        bool ok = true;
        int xs = 0, xp = 0, ys = 0, yp = 0;  // next X and Y stage to be read by S and dP
        int xr = 0, yr = 0;                  // stage of the gradient product
        int ts = 0, tp = 0;                  // stage of the rows' terms
        static_assert(C::NT == 2, "ts alternates");
        auto wait = [&](int b, int parity) {
          if (ok && !mbar_wait(bar(b), parity, abort_flag, a.err)) ok = false;
          return ok;
        };
        // D[lanes, BN] = resident tile * ring tile^T
        auto product = [&](uint32_t d_tm, uint64_t da, uint64_t db) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc_mma_ss(d_tm, da + static_cast<uint64_t>(((kk >> 2) * (kBM * 128) + (kk & 3) * 32) / 16),
                      db + static_cast<uint64_t>(((kk >> 2) * (BN * 128) + (kk & 3) * 32) / 16), C::IDESC_S,
                      kk > 0 ? 1u : 0u);
        };
        // acc[lanes, D] += packed bf16 (TMEM, two halves) * ring tile
        auto accumulate = [&](uint32_t d_tm, uint32_t a_tm, uint64_t db, bool first) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            tc_mma_ts(d_tm, a_tm + (kk < BN / 32 ? kk * 8 : H + (kk - BN / 32) * 8),
                      db + static_cast<uint64_t>(kk * 16 * 128 / 16), C::IDESC_G, first && kk == 0 ? 0u : 1u);
        };
        auto next_s = [&](bool first, int parity) {
          if (!wait(B_FULL_X + xs, xp)) return;
          if (kKey) {  // the threads' terms of the block: S says that they are there
            if (!wait(B_FULL_T + ts, tp)) return;
            ts ^= 1;
            tp ^= ts == 0;
          }
          if (!first && !wait(B_SREAD, parity)) return;
          product(tmem + C::TM_S, da0, dxk + xs * kStage);
          tc_commit(bar(B_S));
          if (++xs == nx) {
            xs = 0;
            xp ^= 1;
          }
        };
        auto next_dp = [&]() {
          if (!wait(B_FULL_Y + ys, yp)) return;
          product(tmem + C::TM_DP, da1, dyk + ys * kStage);
          tc_commit(bar(B_DP));
          if (!kKey) tc_commit(bar(B_REL_Y + ys));
          if (++ys == C::NY) {
            ys = 0;
            yp ^= 1;
          }
        };
        // S of the next block is issued as soon as S has been read, and runs under the exponentials.
        // Products of one thread complete in order, so B_DP of a block says that the products of the
        // block before have read P and dS, which then may be written over dP.
        wait(B_A0, 0);
        wait(B_A1, 0);
        if (ok) next_s(true, 0);
        if (ok) next_dp();
        for (int n = 0; ok && n < U; ++n) {
          if (n + 1 < U) next_s(false, n & 1);
          if (!wait(B_P, n & 1)) break;
          accumulate(tmem + C::TM_ACC_P, tmem + C::TM_P, kKey ? dym + yr * kStage : dxm + xr * kStage, n == 0);
          if (kKey) {
            tc_commit(bar(B_REL_Y + yr));
            if (++yr == C::NY) yr = 0;
          }
          if (!wait(B_DS, n & 1)) break;
          accumulate(tmem + C::TM_ACC_DS, tmem + C::TM_DS, dxm + xr * kStage, n == 0);
          tc_commit(bar(B_REL_X + xr));
          if (++xr == nx) xr = 0;
          if (n + 1 < U) next_dp();
        }
        // all MMAs of this thread complete before the accumulators are read or TMEM is released
        tc_commit(bar(B_FINAL));
        mbar_wait_drain(bar(B_FINAL), 0, a.err);
      }
      __syncwarp();
    }
  } else {
    // ================= probabilities and dS: one lane per thread, half of the columns =================
    setmaxnreg_inc<kRegsSoftmax>();
    const int half = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int slot = blk * BN + row;
    const bool live = row < BN && slot < rows && token_of_slot(g, kind, slot) >= 0;
    const uint64_t sl2 = f2_make(a.scale_log2, a.scale_log2);
    uint64_t nl_row = 0, nd_row = 0;  // query CTA: this row's terms
    if (!kKey) {
      const float* t = a.terms + (static_cast<size_t>(bh) * g.nblk + blk) * (2 * BN);
      const float nl = row < BN ? t[row] : -INFINITY, nd = row < BN ? t[BN + row] : 0.f;
      nl_row = f2_make(nl, nl);
      nd_row = f2_make(nd, nd);
    }
    const uint32_t t_s = t_lane + C::TM_S + half * H, t_dp = t_lane + C::TM_DP + half * H;
    bool ok = true;
    auto wait = [&](int b, int parity) {
      ok = mbar_wait(bar(b), parity, abort_flag, a.err) && ok;
      __syncwarp();
    };
    auto arrive = [&](int b) {  // this warp's TMEM loads or stores are done
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    BitWalk walk(bits);
    // A wait costs 100 to 200 cycles even when its barrier has completed (the tensor core keeps the
    // shared memory busy), so the barriers are tested ahead, under arithmetic.
    bool s_in = false, dp_in = false;
    // query CTA: the sum of the row's rounded dS, less that of the unrounded (or, with an exact delta, than
    // what it has to be)
    uint64_t off = 0ull;
    const uint64_t minus = a.exact ? f2_make(0.f, 0.f) : f2_make(-1.f, -1.f);
    for (int n = 0; n < U; ++n) {
      const int b = walk.next();
      if (!__all_sync(0xffffffffu, ok)) break;  // after a wait that gave up the rest runs on without waiting
      // (the issuer waits for the block's terms before it issues S)
      if (!__all_sync(0xffffffffu, s_in)) wait(B_S, n & 1);
      tc_fence_after();
      // -lse * log2 e and, BN floats on, -delta of this thread's columns: the same address for a warp
      const ulonglong2* terms =
          reinterpret_cast<const ulonglong2*>(smem + rest + (n % C::NT) * C::ST_BYTES) + half * (H / 4);
      uint64_t p[H / 2];
      {
        uint32_t r[H];
        tmem_ld_cols<H>(t_s, r);
        arrive(B_SREAD);
        if (!kKey && !block_full(g, kind, b)) {  // key columns that hold no token (ragged tail, cube padding)
#pragma unroll
          for (int w = 0; w < H / 32; ++w) {
            const uint32_t vb =
                __ballot_sync(0xffffffffu, token_of_slot(g, kind, b * BN + half * H + w * 32 + lane) >= 0);
#pragma unroll
            for (int x = 0; x < 32; ++x) r[w * 32 + x] = ((vb >> x) & 1u) ? r[w * 32 + x] : 0xff800000u;
          }
        }
#pragma unroll
        for (int c = 0; c < H / 2; c += 2) {
          if (c == H / 8 * 3) dp_in = mbar_test(bar(B_DP), n & 1);
          const ulonglong2 nl = kKey ? terms[c / 2] : make_ulonglong2(nl_row, nl_row);
          p[c] = exp2_pair(f2_fma(f2_make(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1])), sl2, nl.x));
          p[c + 1] =
              exp2_pair(f2_fma(f2_make(__uint_as_float(r[2 * c + 2]), __uint_as_float(r[2 * c + 3])), sl2, nl.y));
        }
      }
      uint32_t pp[H / 2];  // packed under the exponentials, which leave the issue slots free
#pragma unroll
      for (int c = 0; c < H / 2; ++c) pp[c] = pack_pair(p[c]);
      if (!__all_sync(0xffffffffu, dp_in)) wait(B_DP, n & 1);
      tc_fence_after();
      uint32_t r[H];
      tmem_ld_cols<H>(t_dp, r);
      tmem_st_cols<H / 2>(t_dp, pp);
      arrive(B_P);
      s_in = n + 1 < U && mbar_test(bar(B_S), (n + 1) & 1);
      uint32_t pk[H / 2];
#pragma unroll
      for (int c = 0; c < H / 2; c += 2) {
        const ulonglong2 nd = kKey ? terms[BN / 4 + c / 2] : make_ulonglong2(nd_row, nd_row);
        const uint64_t d0 = f2_mul(p[c], f2_add(f2_make(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1])), nd.x));
        const uint64_t d1 =
            f2_mul(p[c + 1], f2_add(f2_make(__uint_as_float(r[2 * c + 2]), __uint_as_float(r[2 * c + 3])), nd.y));
        pk[c] = pack_pair(d0);
        pk[c + 1] = pack_pair(d1);
        if constexpr (!kKey) {
          off = f2_add(off, f2_fma(d0, minus, unpack_pair(pk[c])));
          off = f2_add(off, f2_fma(d1, minus, unpack_pair(pk[c + 1])));
        }
      }
      tmem_st_cols<H / 2>(t_dp + H / 2, pk);
      arrive(B_DS);
    }
    ok = __all_sync(0xffffffffu, ok);
    // ---- epilogue: accumulators -> bf16 -> swizzled shared memory (over the resident tiles) -> TMA store ----
    if (ok && U > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(B_FINAL), 0, abort_flag, a.err));
      tc_fence_after();
    }
    if (U == 0) {  // the staging below reuses tiles that nothing has waited for
      wait(B_A0, 0);
      wait(B_A1, 0);
    }
    const bool have = ok && U > 0;
    if constexpr (kKey) {
      // warps 0-3 write dV over V's tile, warps 4-7 dK over K's
      const int tile = half ? C::OFF_A0 : C::OFF_A1;
      stage_rows<BN, D, false>(smem + tile, t_lane + (half ? C::TM_ACC_DS : C::TM_ACC_P), 0, 0.f, 0, row, live, have,
                               half ? a.scale : 1.f);
      fence_proxy_async_smem();
      named_barrier_sync(1 + half, 128);
      if (quad == 2 && lane == 0) {
#pragma unroll
        for (int c = 0; c < C::PANELS; ++c)
          tma_store_3d(half ? &m->dk : &m->dv, sbase + tile + c * BN * 128, c * 64, blk * BN, bh);
        tma_store_commit();
        tma_store_wait_read();
      }
    } else {
      // the row's two threads add up how far its sum of dS is off
      float* both = reinterpret_cast<float*>(smem + rest);  // the terms' ring, which only key CTAs use
      float o0, o1;
      f2_split(off, o0, o1);
      both[half * kBM + row] = o0 + o1;
      named_barrier_sync(1, 256);
      float sum = both[row] + both[kBM + row];
      if (a.exact && row < BN) sum -= a.target[(static_cast<size_t>(bh) * g.nblk + blk) * BN + row];
      stage_rows<BN, D / 2, true>(smem + C::OFF_A0, t_lane + C::TM_ACC_DS + half * (D / 2),
                                  t_lane + C::TM_ACC_P + half * (D / 2), sum, half * (D / 2), row, live, have, a.scale);
      fence_proxy_async_smem();
      named_barrier_sync(1, 256);
      if (warp == 2 && lane == 0) {
#pragma unroll
        for (int c = 0; c < C::PANELS; ++c)
          tma_store_3d(&m->dq, sbase + C::OFF_A0 + c * BN * 128, c * 64, blk * BN, bh);
        tma_store_commit();
        tma_store_wait_read();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, C::TM_COLS);
}

template <int D, int BN>
__global__ void __launch_bounds__(kBwdThreads, 1)
    sparse_attn_bwd_kernel(const __grid_constant__ BwdMaps mn, const __grid_constant__ BwdMaps mp,
                           const __grid_constant__ BwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int per = a.BH * a.g.nblk;
  const int at = static_cast<int>(blockIdx.x);
  const int i = at < per ? at : at - per;
  const int bh = i / a.g.nblk, blk = i - bh * a.g.nblk;
  if (at < per) bwd_cta<D, BN, true>(&mn, &mp, a, bh, blk, smem);
  else bwd_cta<D, BN, false>(&mn, &mp, a, bh, blk, smem);
}

// ---------------------------------------------------------------------------------------
// Row terms and row bitsets
// ---------------------------------------------------------------------------------------
constexpr int kPrepThreads = 256, kPrepRows = 2;

__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
    s = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), s);
  }
  return s;
}

// Eight values of a row as bf16 (fp32 rows round to nearest even, as the permuted copies do).
__device__ __forceinline__ uint4 load8(const void* p, size_t at, bool f32) {
  if (!f32) return *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
  const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
  const float4 a = q[0], b = q[1];
  return make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
}

// CTAs [0, mask_ctas): one warp per query block checks its list (ascending, in range, count within
// max_kv) and writes it as bits; a bad list sets the error bit and becomes empty.
// The others: d / 16 threads per slot of a head's padded rows, kPrepRows slots at a time so that every thread has
// eight 16-byte loads in flight; the two terms of each slot's row.  kLo: O has its rounding errors beside it.
template <bool kLo>
__global__ void __launch_bounds__(kPrepThreads) bwd_prep_kernel(const BwdPrep a) {
  const Geom& g = a.g;
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) < a.mask_ctas) {
    const int nwords = (g.nblk + 31) >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * (kPrepThreads / 32) + warp;
    if (row >= static_cast<long long>(a.BH) * g.nblk) return;
    const int bh = static_cast<int>(row / g.nblk), i = static_cast<int>(row - static_cast<long long>(bh) * g.nblk);
    const int kind = a.kinds[bh];
    const int nb = known_kind(g, kind) ? (layout_rows(g, kind) + g.block - 1) / g.block : 0;
    const int32_t* list = a.kv_idx + row * a.max_kv;
    uint32_t* out = a.rbits + row * nwords;
    const int cnt = i < nb ? a.kv_cnt[row] : 0;
    bool bad = cnt < 0 || cnt > a.max_kv;
    if (!bad)
      for (int j = lane; j < cnt; j += 32) {
        const int kb = list[j];
        if (kb < 0 || kb >= nb || (j > 0 && list[j - 1] >= kb)) bad = true;
      }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0) atomicOr(a.err, kDevErrKvRange);
    const int n = bad ? 0 : cnt;
    // word w holds the listed blocks in [32 w, 32 w + 32): each lane finds them by binary search
    for (int w = lane; w < nwords; w += 32) {
      int lo = 0, hi = n;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (list[mid] < w * 32) lo = mid + 1;
        else hi = mid;
      }
      uint32_t word = 0u;
      for (int j = lo; j < n && list[j] < w * 32 + 32; ++j) word |= 1u << (list[j] & 31);
      out[w] = word;
    }
    return;
  }
  const int tpr = a.d / 16, groups = kPrepThreads / tpr;
  const int slots = g.nblk * g.block;
  const long long first = static_cast<long long>(blockIdx.x - a.mask_ctas) * (groups * kPrepRows) + threadIdx.x / tpr;
  const long long all = static_cast<long long>(a.BH) * slots;
  const int c = threadIdx.x % tpr;
  uint4 o[kPrepRows][2], go[kPrepRows][2], lo[kLo ? kPrepRows : 1][2];
  float lse[kPrepRows], dlse[kPrepRows];
  bool has[kPrepRows];
#pragma unroll
  for (int r = 0; r < kPrepRows; ++r) {
    const long long at = min(first + r * groups, all - 1);
    const int bh = static_cast<int>(at / slots), slot = static_cast<int>(at - static_cast<long long>(bh) * slots);
    const int kind = a.kinds[bh];
    const int token = known_kind(g, kind) ? token_of_slot(g, kind, slot) : -1;
    has[r] = token >= 0;
    // whole call: O, dO and LSE in natural order; lists: each head's own layout and set.  A slot without a
    // token loads row 0 of its head.
    const bool perm = !a.by_token && a.has_perm && kind != kSpatial;
    const int stride = a.by_token ? g.N : (perm ? g.R : a.nat_rows);
    const size_t row = static_cast<size_t>(bh) * stride + (has[r] ? (a.by_token ? token : slot) : 0);
    const void* po = perm ? a.o_perm : a.o_nat;
    const void* pg = perm ? a.do_perm : a.do_nat;
    const void* pl = perm ? a.lo_perm : a.lo_nat;
    const float* dl = perm ? a.dlse_perm : a.dlse_nat;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      o[r][j] = load8(po, row * a.d + (j * tpr + c) * 8, a.f32);
      go[r][j] = load8(pg, row * a.d + (j * tpr + c) * 8, a.f32);
      if constexpr (kLo) lo[r][j] = load8(pl, row * a.d + (j * tpr + c) * 8, a.f32);
    }
    lse[r] = (perm ? a.lse_perm : a.lse_nat)[row];
    dlse[r] = 0.f;
    if (dl != nullptr) dlse[r] = dl[row];
  }
#pragma unroll
  for (int r = 0; r < kPrepRows; ++r) {
    float delta = dot8(o[r][0], go[r][0]) + dot8(o[r][1], go[r][1]);
    if constexpr (kLo) delta += dot8(lo[r][0], go[r][0]) + dot8(lo[r][1], go[r][1]);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1)
      if (off < tpr) delta += __shfl_xor_sync(0xffffffffu, delta, off);
    const long long at = first + r * groups;
    if (c == 0 && at < all) {
      const bool sees = has[r] && lse[r] != -INFINITY;
      float* t = a.terms + (at / g.block) * (2 * g.block) + at % g.block;  // slots are whole blocks
      t[0] = sees ? -lse[r] * 1.4426950408889634f : -INFINITY;
      t[g.block] = sees ? dlse[r] - delta : 0.f;
      if constexpr (kLo) a.target[at] = sees ? dlse[r] : 0.f;
    }
  }
}

template <int D, int BN>
cudaError_t launch_bwd_t(const BwdMaps& nat, const BwdMaps& perm, BwdArgs a, cudaStream_t stream) {
  auto kern = sparse_attn_bwd_kernel<D, BN>;
  const int nwords = (a.g.nblk + 31) / 32;
  using C = BwdCfg<D, BN>;
  a.nx = C::stages(nwords);
  const int smem = C::smem_bytes(a.nx, nwords);
  if (smem > kMaxSmem) return cudaErrorInvalidConfiguration;
  cudaError_t e = allow_smem(kern, kMaxSmem);
  if (e != cudaSuccess) return e;
  // may start while the last prep CTAs still run (programmatic dependent launch): everything up to
  // pdl_wait() in the kernel needs only what was there before prep
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * a.BH * a.g.nblk));
  cfg.blockDim = dim3(kBwdThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, nat, perm, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool sparse_attn_bwd_fits(const Geom& g, int BH) {
  using C = BwdCfg<128, 128>;
  return C::smem_bytes(C::NX_MOST - 1, (g.nblk + 31) / 32) <= kMaxSmem &&
         2LL * BH * g.nblk <= 0x7fffffffLL && static_cast<long long>(BH) * g.nblk * g.block / 8 <= 0x7fffffffLL;
}

cudaError_t launch_sparse_attn_bwd(const BwdMaps& nat, const BwdMaps& perm, BwdPrep prep, const BwdArgs& a, int d,
                                   cudaStream_t stream) {
  const long long lists = static_cast<long long>(a.BH) * a.g.nblk;
  const long long slots = lists * a.g.block;
  const int rows_per_cta = kPrepThreads / (d / 16) * kPrepRows;
  prep.mask_ctas = static_cast<int>((lists + kPrepThreads / 32 - 1) / (kPrepThreads / 32));
  const long long grid = prep.mask_ctas + (slots + rows_per_cta - 1) / rows_per_cta;
  if (a.exact) bwd_prep_kernel<true><<<static_cast<unsigned>(grid), kPrepThreads, 0, stream>>>(prep);
  else bwd_prep_kernel<false><<<static_cast<unsigned>(grid), kPrepThreads, 0, stream>>>(prep);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int bn = a.g.block;
  if (d == 128 && bn == 128) return launch_bwd_t<128, 128>(nat, perm, a, stream);
  if (d == 64 && bn == 128) return launch_bwd_t<64, 128>(nat, perm, a, stream);
  if (d == 128 && bn == 64) return launch_bwd_t<128, 64>(nat, perm, a, stream);
  if (d == 64 && bn == 64) return launch_bwd_t<64, 64>(nat, perm, a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace vsa
