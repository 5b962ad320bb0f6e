// Tree-verify attention over the 8-bit cache on the sm_100a tensor cores (tcgen05 + TMEM + TMA): bf16
// queries, d = 128, groups of up to 128 heads.  The operation, the work decomposition, the split shares and the
// merge are those of attn_umma.cu ("EAGLE-Pangu", technical summary sec. 2: a tree token attends to the
// committed prefix and to its own ancestors only); what differs is how 8-bit keys and values become
// operands.  At half the bytes a 64-key tile (16 KB) arrives every ~700 cycles per SM, so shared-memory
// traffic and instructions per tile decide the design.
//   * Scores: K tiles are the tensor cores' B operand as they arrive (kind::f8f6f4).  The bf16 query
//     row, scaled by a power of two to a maximum in (224, 448], is the sum of two e4m3 pieces, q1 = rne(q),
//     q2 = rne(q - q1): bf16 has 8 significant bits, a piece 4, and the residue's fit the second piece, so
//     q1 + q2 = q exactly down to 2^-9 of the row's maximum and within 2^-17 of the maximum below it.
//     Both pieces live in TMEM and accumulate into one S tile: two 8-bit products cost what one bf16
//     product does (a probe: 307 cycles per 128 x 64 x 128 tile against 346), and K is never expanded.
//   * K's scales (one per block of tokens) multiply groups of keys: they ride in the constant of the
//     exponent's FFMA.  V's scales are powers of two: p * 2^e is the same exponential with e added to
//     its argument, and the running reference M is the maximum of (score + e), so P' = 2^(s + e - M)
//     is what the exponential gives, and the row sum takes each group's sum times 2^-e.  Scales thus cost
//     no instruction per score.
//   * Values: four converter warps expand V's codes to f16 (exact, one instruction for two codes) from the
//     TMA ring into the operand ring; P' is f16 too (11 significant bits; at most 2^8, and what falls
//     below 2^-24 of the largest contribution is lost).
//   * Few query rows (a decode step has G of them): when all rows fit 64 or 32 TMEM lanes they are
//     repeated 2 or 4 times over the 128 lanes of the S tile, which the tensor cores compute anyway, and
//     each repetition's thread takes its own half or quarter of the tile's keys (its P' is zero
//     elsewhere).  The epilogue merges the repetitions by log-sum-exp.  All four sub-partitions then
//     share the exponentials that would otherwise sit on one or two.
//   * The tree's own K/V are bf16; their tiles (the last of a sequence) use the bf16 query from shared
//     memory and a bf16 P.
// Warps: 0 K producer, 1 ancestor bits, then P V issue, 2 V producer, 3 S issue, 4-11 softmax (two
// warpgroups), 12-15 converters (few query rows: and 16-19).  Every mbarrier wait is bounded as in attn_umma.cu.
// What bounds it: one query tile, the hand-over between the roles (~820 cycles per 64-key tile, its products
// ~560, its bytes ~700 with all SMs streaming); two, the chain S -> exponentials -> P V (~2400 cycles; four
// softmax warpgroups, two per tile: 9-14% slower).  Measured: 64 x 6 nodes, 64/8 heads, 8192 keys 279 us
// (1.09 GB, 3.9 TB/s) in the first few ms of a loop and 330 us (3.3 TB/s) once it runs at the power cap; 512 nodes, 32/8
// heads, 32768 keys 367 us (275 GFLOP, 749 TFLOP/s); 16 x 60 nodes, up to 8192 keys 136 us; one token over 1000 keys
// 11.7 us, 26 nodes over 2048 keys 15.5 us with the merge kernel.
#include <climits>
#include <cstdlib>

#include "attn_umma_common.cuh"
#include "common.cuh"
#include "kernels.h"
#include "q8.cuh"

namespace tsd {

namespace {

using namespace attn;
using namespace umma;

constexpr int kBM = 128, kBN = 64;
// Threads: 512, and 128 more where a second group of converter warps takes every other tile (few query rows:
// the softmax of a repetition needs few registers, and the expansion of V would be the slowest role).
constexpr int threads_of(int rep) { return rep > 1 ? 640 : 512; }
constexpr uint32_t kTmemCols = 512;
// One query tile (warpgroup w takes key tiles i = w mod 2): O_w at 128 w, S_w at 256 + 64 w, P_w at
// 384 + 32 w, the query pieces at 448 (32 columns each).  Two query tiles (warpgroup w has tile w): O_w at
// 128 w, S_w at 256 + 64 w with P_w over it, the pieces of Q_w at 384 + 64 w.  (Measured for two: pieces in
// shared memory and P beside S, so that S of the next tile overlaps the softmax: 3-7% slower, the products
// with both operands in shared memory take 385 cycles against 307.)
constexpr uint32_t kColO = 0, kColS = 256;
constexpr uint32_t kSlot8 = kBN * kD;          // one 8-bit K or V tile: 8 KB
constexpr uint32_t kHalf = kBN * 128;          // one 64-column half of a bf16 tile: 8 KB
constexpr uint32_t kSlot = 2 * kHalf;          // one bf16 tile: 16 KB
constexpr uint32_t kQBytes = kBM * 256;        // one bf16 query tile: 32 KB
constexpr int kMaxRing = 8, kVB = 3;
constexpr float kRescaleLog2 = 8.0f;           // lazy max: rescale only past a 2^8 growth

struct QParams {
  int splits, Rmax, mtiles;
  int whole;           // row blocks (sequences longest first) that one CTA takes whole; the others are split
  uint32_t wait;       // cycles after which an mbarrier wait gives up
  int withhold;        // test hook: the K producer never issues this tile (-1: off)
  int lpt;
  int ks, vs;          // 8-bit K and V ring depths
  int box_rows;
  int npt;             // nodes per query tile (a repetition's lanes hold npt * G rows)
  int W;
  int* tickets;
  int evict_first;
  uint32_t kt_off, k_off, v_off, vb_off, mask_off, ps_off;
};

// The scale bytes of a group of keys in one word: K's in bits 0-7, V's in bits 16-23.
__device__ __forceinline__ float k_factor(uint32_t w) { return __uint_as_float(w << 23); }   // 2^(byte - 127)
// byte - 127 as a float: 2^23 + byte is exact and so is the difference
__device__ __forceinline__ float v_exponent(uint32_t w) {
  return __uint_as_float((w >> 16) | 0x4b000000u) - 8388735.f;
}
__device__ __forceinline__ float v_inverse(uint32_t w) {                                     // 2^(127 - byte)
  return __uint_as_float(0x7f000000u - ((w & 0x00ff0000u) << 7));
}

struct __align__(8) Bars {
  uint64_t q_full;                                    // bf16 query tile(s) in shared memory
  uint64_t q8_full;                                   // query pieces in TMEM
  uint64_t k_full[kMaxRing], k_empty[kMaxRing];       // 8-bit K ring
  uint64_t v_full[kMaxRing], v_empty[kMaxRing];       // 8-bit V ring
  uint64_t kt_full, kt_empty, vt_full[kVB];           // the tree's bf16 K tile, its V tile's arrival in an operand slot
  uint64_t vb_full[kVB], vb_empty[kVB];               // bf16 V operand ring
  uint64_t s_full[2], s_empty[2];                     // S_w in TMEM; read (one query tile)
  uint64_t p_full[2], pv_done[2];
  uint64_t mask_full;
  uint64_t fin[2];                                    // time-out: the issuing warps' MMAs
};

// Bounded wait as umma::mbar_wait, without its suspend-time hint (measured 3% faster here: every role is
// on some tile's critical path) and with a 32-bit clock (shorter).
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, uint32_t limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = clock();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((uint32_t)clock() - t0 > limit) return false;
  }
}

// Place in a ring of n slots: the slot and the parity of its current use (a division by the ring's depth
// would sit on every role's critical path).
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) slot = 0, parity ^= 1u;
  }
};

// Block ids of the boxes of prefix tile t (paged caches), loaded a tile ahead by the producers.
struct TileBlocks {
  int blk[8];
};
__device__ __forceinline__ void fetch_blocks(const AttnArgs& a, const SeqView& v, const QParams& u, int b, int t,
                                             TileBlocks& tb) {
  if (a.block_table == nullptr || t >= v.nPT) return;
  const int pos0 = t * kBN;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int seg = k * u.box_rows;
    if (seg < kBN) tb.blk[k] = a.block_table[(size_t)b * a.max_blocks + min((pos0 + seg) >> a.block_shift,
                                                                            a.max_blocks - 1)];
  }
}
// TMA loads of one 64-key tile of 8-bit codes: rows of 128 bytes, one box (contiguous) or one per page.
__device__ __forceinline__ void load_codes(const AttnArgs& a, const SeqView& v, const QParams& u, int b, int g, int t,
                                           uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int* s_err,
                                           const TileBlocks& tb, uint64_t pol) {
  const int pos0 = t * kBN;
  if (a.block_table == nullptr) {
    tma_load_2d_hint(dst, map, 0, (b * a.Hkv + g) * a.Lcap + pos0, bar, pol);
    return;
  }
  const int bs_mask = (1 << a.block_shift) - 1;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int seg = k * u.box_rows;
    if (seg >= kBN) break;
    const int pos = pos0 + seg;
    int blk = tb.blk[k];
    if (blk < 0 || blk >= a.num_blocks) {
      if (pos < v.L) *s_err = 1;
      blk = 0;
    }
    tma_load_2d_hint(dst + (uint32_t)seg * 128, map, 0, (blk * a.Hkv + g) * (1 << a.block_shift) + (pos & bs_mask), bar,
                     pol);
  }
}

// Two codes to two f16 values (exact; NaN stays NaN).
__device__ __forceinline__ uint32_t expand2(uint32_t two) {
  uint32_t r;
  asm("{\n.reg .b16 h, x;\nmov.b32 {h, x}, %1;\ncvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(two));
  return r;
}

// Exponent of a query row's scale: smallest 2^k with amax <= 448 * 2^k, k >= -100 (as q8::scale_byte,
// without its floor at 2^-40).
__device__ __forceinline__ int row_byte(float amax) {
  const uint32_t w = __float_as_uint(amax);
  return min(max((int)(w >> 23) - 8 + ((w & 0x7fffffu) > 0x600000u ? 1 : 0), 27), 247);   // (247: infinities, NaN)
}

// kDual: two query tiles per CTA (more than 128 rows per KV head), warpgroup w owns tile w; else one, whose
// rows are repeated kRep times.  kG: scale groups per key tile (block sizes 8: 8, 16 and 32: 4, 64 up: 1).
template <bool kDual, int kRep, int kG>
__global__ void __launch_bounds__(threads_of(kRep), 1)
    attn_q8_umma_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKt,
                        const __grid_constant__ CUtensorMap tmVt, const AttnArgs a, const QParams u) {
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_err;
  __shared__ int s_ticket;
  __shared__ volatile int s_abort;
  __shared__ int s_q_issued, s_k_issued, s_kt_issued, s_v_issued, s_vt_issued[kVB];
  __shared__ int s_poison;   // the tree's V held infinities or NaN
  __shared__ float2 s_ml1[kBM], s_ml[kDual ? 2 * kBM : kBM];
  constexpr uint32_t kColQ = kDual ? 384 : 448, kColP = kDual ? 256 : 384, kPW = kDual ? 64 : 32;   // P_w at kColP + kPW w
  constexpr int kRows = kDual ? 2 * kBM : kBM / kRep;   // most query rows of this CTA
  constexpr int kThreadsQ = threads_of(kRep), kCG = kRep > 1 ? 2 : 1;   // threads, groups of converter warps
  constexpr int kLanes = kBM / kRep;                    // TMEM lanes of one repetition
  constexpr int kNC = kBN / kRep;                       // keys of a tile per thread
  constexpr int kGW = kBN / kG;                         // keys per scale group
  constexpr int kTG = kGW >= kNC ? 1 : kNC / kGW;       // scale groups per thread
  constexpr int kTW = kNC / kTG;                        // keys per scale group and thread

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---------------------------------------------------------------- set-up (before the wait on the
  // previous launch: nothing here reads what an earlier kernel writes)
  if (tid == 0) {
    mbar_init(&bars.q_full, 1);
    mbar_init(&bars.q8_full, 8);
    for (int s = 0; s < u.ks; ++s) mbar_init(&bars.k_full[s], 1), mbar_init(&bars.k_empty[s], 1);
    for (int s = 0; s < u.vs; ++s) mbar_init(&bars.v_full[s], 1), mbar_init(&bars.v_empty[s], 4);
    mbar_init(&bars.kt_full, 1), mbar_init(&bars.kt_empty, 1);
    for (int s = 0; s < kVB; ++s) {
      mbar_init(&bars.vb_full[s], 4), mbar_init(&bars.vb_empty[s], 1), mbar_init(&bars.vt_full[s], 1);
      s_vt_issued[s] = 0;
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bars.s_full[w], 1), mbar_init(&bars.s_empty[w], 4);
      mbar_init(&bars.p_full[w], 4), mbar_init(&bars.pv_done[w], 1);
    }
    mbar_init(&bars.mask_full, 1);
    mbar_init(&bars.fin[0], 1), mbar_init(&bars.fin[1], 1);
    s_err = 0;
    s_abort = 0;
    s_q_issued = s_k_issued = s_kt_issued = s_v_issued = s_poison = 0;
    fence_barrier_init();
    fence_proxy_async();
    prefetch_tmap(&tmQ), prefetch_tmap(&tmK), prefetch_tmap(&tmV), prefetch_tmap(&tmKt), prefetch_tmap(&tmVt);
  }
  if (warp == 3) {
    tmem_alloc(&s_tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  auto leave = [&]() {
    if (warp == 3) tmem_dealloc(tmem, kTmemCols);
  };

  const int item = (int)blockIdx.x - u.whole, unit = item < 0 ? blockIdx.x : u.whole + item / u.splits;
  const int ns = item < 0 ? 1 : u.splits, split = item < 0 ? 0 : item % u.splits;
  const int mt = unit % u.mtiles, g = unit / u.mtiles % a.Hkv, zb = unit / u.mtiles / a.Hkv;
  int b = zb;
  if (u.lpt) {   // sequences longest prefix first (ties by index)
    __shared__ int s_b;
    __shared__ int s_len[512];
    if (tid < a.B) s_len[tid] = a.prefix_len[tid];
    __syncthreads();
    if (tid < a.B) {
      const int L = s_len[tid];
      int rank = 0;
      for (int o = 0; o < a.B; ++o) {
        const int Lo = s_len[o];
        rank += (Lo > L) || (Lo == L && o < tid);
      }
      if (rank == zb) s_b = tid;
    }
    __syncthreads();
    b = s_b;
  }
  const int G = a.Hq / a.Hkv;
  __shared__ int s_status;   // one read, so that the CTA takes one branch
  if (tid == 0) s_status = __ldcg(a.status + b);
  SeqView v = seq_view(a, b, G, kBN, 1 << 30);
  __syncthreads();
  v.zero = v.cap || s_status != 0;
  const int rows_tile = u.npt * G, rows_cta = kDual ? 2 * rows_tile : rows_tile;
  const int r0 = mt * rows_cta;
  if (v.skip || r0 >= v.R) {
    leave();
    return;
  }
  const int r_hi = min(r0 + rows_cta, v.R);
  // where this CTA's partial and its ticket word are: all pairs have theirs, or only the split ones
  const int pairs = u.whole > 0 ? a.B * a.Hkv - u.whole : a.B * a.Hkv, pair = u.whole > 0 ? unit - u.whole : b * a.Hkv + g;
  const size_t word = (size_t)pair * u.mtiles + mt;
  if (v.zero) {
    if (split == 0 && mt == 0 && g == 0 && tid == 0 && s_status == 0 && v.cap)
      flag_status(a.status, b, TSD_ERR_CAPACITY);
    if (ns > 1 && u.tickets != nullptr) {
      const int t = take_ticket(u.tickets + word, ns, &s_ticket);
      if (t == 1) zero_rows<__nv_bfloat16>(a, b, g, G, r0, r_hi);
      else if (t == 2 && tid == 0) flag_status(a.status, b, TSD_ERR_WORKSPACE);
    } else if (split == 0) {
      zero_rows<__nv_bfloat16>(a, b, g, G, r0, r_hi);
    }
    leave();
    return;
  }
  const bool direct = (ns == 1);
  // (T <= 2^25 tiles and at most 64 splits: no overflow)
  const int t_begin = (int)((uint32_t)split * (uint32_t)v.T / (uint32_t)ns);
  const int nt = (int)((uint32_t)(split + 1) * (uint32_t)v.T / (uint32_t)ns) - t_begin;   // 0 when T < splits
  const int np = max(0, min(nt, v.nPT - t_begin));                           // prefix tiles, then nt - np tree tiles
  const int cta_nodes = kDual ? 2 * u.npt : u.npt;
  const int node0 = mt * cta_nodes;

  uint8_t* sQ = smem;
  uint8_t* sKt = smem + u.kt_off;
  uint8_t* sK = smem + u.k_off;
  uint8_t* sV = smem + u.v_off;
  uint8_t* sVB = smem + u.vb_off;
  uint32_t* sMask = reinterpret_cast<uint32_t*>(smem + u.mask_off);

  // P V of key tile i for warpgroup w (its tile k), V in operand slot st (warp-collective)
  auto issue_pv = [&](int i, int w, int k, int st) {
    const uint64_t bv = sdesc_sw128(smem_u32(sVB), kHalf, 1024) + (uint64_t)((st * kSlot) >> 4);
    const uint32_t idesc = i < np ? idesc_f16(kBM, kD, true) : idesc_bf16(kBM, kD, true);   // the tree's P and V are bf16
    tc_fence_after();
    mma_f16_pv_warp(tmem + kColO + (uint32_t)w * kD, tmem + kColP + (uint32_t)w * kPW, bv, idesc, k > 0 ? 1u : 0u);
    if (!kDual || w == 1) tc_commit2_warp(&bars.pv_done[w], &bars.vb_empty[st]);
    else tc_commit_warp(&bars.pv_done[w]);
  };

  float row_m = -INFINITY, row_l = 0.f;

  if (warp == 0) {
    // ------------------------------------------------------------ K producer (one thread)
    if (lane == 0) {
      const uint64_t pol = u.evict_first ? l2_evict_first_policy() : l2_evict_normal_policy();
      if (nt > 0) {   // the query tile(s), or the repetitions of one
        mbar_expect_tx(&bars.q_full, (uint32_t)rows_tile * 256 * (kDual ? 2 : kRep));
#pragma unroll
        for (int w = 0; w < (kDual ? 2 : kRep); ++w) {
          const int zq = b * a.Nmax + node0 + (kDual ? w * u.npt : 0);
          uint8_t* dq = sQ + (kDual ? (uint32_t)w * kQBytes : (uint32_t)w * kLanes * 128);
          tma_load_3d(dq, &tmQ, 0, g * G, zq, &bars.q_full);
          tma_load_3d(dq + kQBytes / 2, &tmQ, 64, g * G, zq, &bars.q_full);
        }
        s_q_issued = 1;
      }
      int issued = 0;
      bool ok = true;
      Ring ring;
      TileBlocks nxt;
      fetch_blocks(a, v, u, b, t_begin, nxt);
      for (int i = 0; i < np && !s_abort; ++i) {
        if (t_begin + i == u.withhold) {   // test hook: this tile (and every later one) never arrives
          ok = false;
          break;
        }
        const TileBlocks cur = nxt;
        if (i + 1 < np) fetch_blocks(a, v, u, b, t_begin + i + 1, nxt);
        const int st = ring.slot;
        if (i >= u.ks && !mbar_wait(&bars.k_empty[st], ring.parity ^ 1u, u.wait)) {
          abort_cta(a, b, &s_abort);
          ok = false;
          break;
        }
        mbar_expect_tx(&bars.k_full[st], kSlot8);
        load_codes(a, v, u, b, g, t_begin + i, sK + (size_t)st * kSlot8, &tmK, &bars.k_full[st], &s_err, cur, pol);
        ring.next(u.ks);
        ++issued;
      }
      s_k_issued = issued;
      if (ok && np < nt) {   // the tree's K tiles
        int kt = 0;
        for (int j = 0; j < nt - np && !s_abort; ++j) {
          if (t_begin + np + j == u.withhold) break;
          if (j > 0 && !mbar_wait(&bars.kt_empty, (j - 1) & 1, u.wait)) {
            abort_cta(a, b, &s_abort);
            break;
          }
          mbar_expect_tx(&bars.kt_full, kSlot);
          const int z = b * a.Nmax + (t_begin + np + j - v.nPT) * kBN;
          tma_load_3d(sKt, &tmKt, 0, g, z, &bars.kt_full);
          tma_load_3d(sKt + kHalf, &tmKt, 64, g, z, &bars.kt_full);
          ++kt;
        }
        s_kt_issued = kt;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ ancestor bits of the tree tiles
    // built while the prefix tiles stream in; the softmax waits for them at its first tree tile
    if (np < nt) {
      build_mask_staged(a, b, node0, cta_nodes, u.W, sMask, v.N, reinterpret_cast<int32_t*>(smem + u.ps_off), lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.mask_full);
    }
    if constexpr (!kDual) {
      // ---------------------------------------------------------- P V issue of one query tile, by a second warp: a
      // warp issues an MMA every ~40 cycles, so the products of a tile would take one warp the time of the tile
      bool ok = true;
      Ring vr;
      for (int i = 0; ok && i < nt; ++i, vr.next(kVB)) {
        const bool got = mbar_wait(&bars.vb_full[vr.slot], vr.parity, u.wait) &&
                         mbar_wait(&bars.p_full[i & 1], (i >> 1) & 1, u.wait);
        ok = __all_sync(0xffffffffu, got) != 0;
        if (ok) issue_pv(i, i & 1, i >> 1, vr.slot);
      }
      if (!ok) abort_cta(a, b, &s_abort);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ V producer (one thread)
    if (lane == 0) {
      const uint64_t pol = u.evict_first ? l2_evict_first_policy() : l2_evict_normal_policy();
      int issued = 0;
      Ring ring;
      TileBlocks nxt;
      fetch_blocks(a, v, u, b, t_begin, nxt);
      for (int i = 0; i < np && !s_abort; ++i) {
        const TileBlocks cur = nxt;
        if (i + 1 < np) fetch_blocks(a, v, u, b, t_begin + i + 1, nxt);
        const int st = ring.slot;
        if (i >= u.vs && !mbar_wait(&bars.v_empty[st], ring.parity ^ 1u, u.wait)) {
          abort_cta(a, b, &s_abort);
          break;
        }
        mbar_expect_tx(&bars.v_full[st], kSlot8);
        load_codes(a, v, u, b, g, t_begin + i, sV + (size_t)st * kSlot8, &tmV, &bars.v_full[st], &s_err, cur, pol);
        ring.next(u.vs);
        ++issued;
      }
      s_v_issued = issued;
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ S issue (warp-collective), and with two query
    // tiles P V in the same order
    const uint32_t idesc_8 = idesc_e4m3(kBM, kBN);
    const uint32_t idesc_s = idesc_bf16(kBM, kBN, false);
    const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dkt = sdesc_sw128(smem_u32(sKt), 16, 1024);
    const uint64_t dk = sdesc_sw128(smem_u32(sK), 16, 1024);
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, u.wait)) != 0;
    };
    // S of tile j for query tile w into TMEM columns d; frees the K slot with the last query tile
    Ring kr;
    auto issue_s = [&](int j, int w) -> bool {
      const bool last = !kDual || w == 1;
      const int sw = kDual ? w : j & 1;
      const uint32_t d = tmem + kColS + (uint32_t)sw * kBN;
      uint64_t* empty;
      if (j < np) {
        const int st = kr.slot;
        if (w == 0 && !wait_all(&bars.k_full[st], kr.parity)) return false;
        tc_fence_after();
        mma_e4m3_pieces_warp(d, tmem + kColQ + (uint32_t)w * 64, dk + (uint64_t)((st * kSlot8) >> 4), idesc_8);
        empty = &bars.k_empty[st];
        if (last) kr.next(u.ks);
      } else {
        if (w == 0 && !wait_all(&bars.kt_full, (j - np) & 1)) return false;
        tc_fence_after();
        const uint64_t aq = dq + (uint64_t)((w * kQBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off_q = ((kk >> 2) * (kQBytes / 2) + (kk & 3) * 32) >> 4;
          const uint32_t off_k = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          mma_bf16_ss_warp(d, aq + off_q, dkt + off_k, idesc_s, kk > 0 ? 1u : 0u);
        }
        empty = &bars.kt_empty;
      }
      if (last) tc_commit2_warp(&bars.s_full[sw], empty);
      else tc_commit_warp(&bars.s_full[sw]);
      return true;
    };
    bool ok = true;
    if (nt > 0) ok = wait_all(&bars.q_full, 0) && wait_all(&bars.q8_full, 0);
    if constexpr (kDual) {
      for (int w = 0; ok && w < 2 && nt > 0; ++w) ok = issue_s(0, w);
      Ring vr;
      for (int i = 0; ok && i < nt; ++i, vr.next(kVB)) {
        ok = wait_all(&bars.vb_full[vr.slot], vr.parity);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          ok = ok && wait_all(&bars.p_full[w], i & 1);
          if (!ok) break;
          issue_pv(i, w, i, vr.slot);
          // S_w(i+1) overwrites P_w(i), which the product just issued reads first (issue order)
          if (i + 1 < nt) ok = issue_s(i + 1, w);
        }
      }
    } else {
      // S_w(i + 2) goes out as soon as warpgroup w has S_w(i) in registers
      for (int i = 0; ok && i < nt; ++i)
        ok = (i < 2 || wait_all(&bars.s_empty[i & 1], ((i >> 1) - 1) & 1)) && issue_s(i, 0);
    }
    if (!ok) abort_cta(a, b, &s_abort);
  } else if (warp >= 12) {
    // ------------------------------------------------------------ converters: V codes -> f16 operand tiles
    // A warp takes 16 rows.  Eight lanes read 64 bytes of rows r and r ^ 5 and write their expansion:
    // with both tiles in the 128-byte swizzle, neither side meets a bank conflict.
    const int cw = warp & 3, cg = (warp - 12) >> 2;      // warp of the group, group (tiles i = cg mod kCG)
    const int row8 = (lane >> 3) ^ ((lane & 4) ? 5 : 0), c4 = lane & 3;
    bool ok = true;
    Ring vr, br;
    if (kCG == 2 && cg == 1) vr.next(u.vs), br.next(kVB);
    auto slot_free = [&](int i) -> bool {
      const bool got = i < kVB || mbar_wait(&bars.vb_empty[br.slot], br.parity ^ 1u, u.wait);
      return __all_sync(0xffffffffu, got) != 0;
    };
    int i = cg;
    for (; ok && i < np; i += kCG) {
      const int st = vr.slot, vb = br.slot;
      uint8_t* dst = sVB + (size_t)vb * kSlot;
      const int t = t_begin + i;
      ok = slot_free(i) && __all_sync(0xffffffffu, mbar_wait(&bars.v_full[st], vr.parity, u.wait)) != 0;
      if (!ok) break;
      const uint8_t* src = sV + (size_t)st * kSlot8;
      const int nv = v.L - t * kBN;     // rows at or past nv are not of the sequence: zero
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = cw * 16 + (q >> 1) * 8 + row8, c = (q & 1) * 4 + c4;   // c: 16-code piece of the row
        w[q] = *reinterpret_cast<const uint4*>(src + row * 128 + ((c ^ (row & 7)) << 4));
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = cw * 16 + (q >> 1) * 8 + row8;
        if (row >= nv) w[q] = make_uint4(0, 0, 0, 0);
        uint8_t* drow = dst + (q & 1) * kHalf + row * 128;
        *reinterpret_cast<uint4*>(drow + (((2 * c4) ^ (row & 7)) << 4)) =
            make_uint4(expand2(w[q].x), expand2(w[q].x >> 16), expand2(w[q].y), expand2(w[q].y >> 16));
        *reinterpret_cast<uint4*>(drow + (((2 * c4 + 1) ^ (row & 7)) << 4)) =
            make_uint4(expand2(w[q].z), expand2(w[q].z >> 16), expand2(w[q].w), expand2(w[q].w >> 16));
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.v_empty[st]), mbar_arrive(&bars.vb_full[vb]);
#pragma unroll
      for (int q = 0; q < kCG; ++q) vr.next(u.vs), br.next(kVB);
    }
    for (; ok && i < nt; i += kCG) {
      const int vb = br.slot;
      uint8_t* dst = sVB + (size_t)vb * kSlot;
      ok = slot_free(i);
      if (!ok) break;
      // the tree's V tile is bf16 already: TMA into the operand slot, rows past the nodes and what is not
      // finite zeroed, 16 rows per warp.  (A barrier per slot: a warp cannot fall two of its uses behind.)
      const int tn = (t_begin + i - v.nPT) * kBN, nv = v.N - tn, use = (i - np) / kVB;
      if (cw == 0 && lane == 0) {
        mbar_expect_tx(&bars.vt_full[vb], kSlot);
        const int z = b * a.Nmax + tn;
        tma_load_3d(dst, &tmVt, 0, g, z, &bars.vt_full[vb]);
        tma_load_3d(dst + kHalf, &tmVt, 64, g, z, &bars.vt_full[vb]);
        s_vt_issued[vb] = use + 1;
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, mbar_wait(&bars.vt_full[vb], use & 1, u.wait)) != 0;
      if (!ok) break;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int row = cw * 16 + (q & 3) * 4 + (lane >> 3);
        uint4* piece = reinterpret_cast<uint4*>(dst + (q >> 2) * kHalf + row * 128 + (lane & 7) * 16);
        *piece = row < nv ? finite_bf16(*piece, &s_poison) : make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.vb_full[vb]);
#pragma unroll
      for (int q = 0; q < kCG; ++q) br.next(kVB);
    }
    if (!ok) abort_cta(a, b, &s_abort);
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int wg = (warp - 4) >> 2;
    const int q4 = warp & 3;
    const int row = q4 * 32 + lane;                  // TMEM lane
    const int key0 = kRep == 1 ? 0 : (row / kLanes) * kNC;   // this repetition's first key of a tile
    const int in_tile = kDual ? row : row % kLanes;   // (lanes behind a tile's last whole node hold no row)
    const int qrow = kDual ? wg * rows_tile + in_tile : in_tile;
    const bool row_ok = in_tile < rows_tile && r0 + qrow < r_hi;
    const bool warp_live = in_tile - lane < rows_tile && r0 + qrow - lane < r_hi;   // a warp of padding rows skips the arithmetic
    const int nl = min(qrow / G, cta_nodes - 1);
    const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t o_col = kColO + (uint32_t)wg * kD;
    const float sl2 = a.scale * kLog2e;
    float c_row = sl2;                                // sl2 * 2^(scale exponent of the query row)
    bool ok = true;
    if (nt > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars.q_full, 0, u.wait)) != 0;
    if (np > 0 && ok) {
      const uint8_t* qs = sQ + (kDual ? (uint32_t)wg * kQBytes : 0u) + row * 128;
      auto q16 = [&](int c) -> uint4 {     // 8 elements of the row (rows past the sequence's are zero)
        const uint4 x = *reinterpret_cast<const uint4*>(qs + (c >> 3) * (kQBytes / 2) + (((c & 7) ^ (row & 7)) << 4));
        return row_ok ? x : make_uint4(0, 0, 0, 0);
      };
      uint32_t m2 = 0;                     // the largest |q| of the even and of the odd elements, as bf16 bits
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint4 y = q16(c);
        m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu), __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu)));
      }
      const float amax = __uint_as_float(max(m2 << 16, m2 & 0xffff0000u));
      const int byte = row_byte(amax);
      const float inv = q8::inv_pow2_byte(byte);
      // (the pieces saturate: an infinite query's row is NaN through its scale)
      c_row = amax < INFINITY ? sl2 * q8::pow2_byte(byte) : __uint_as_float(0x7fc00000u);
      // 16 elements to 4 words of each piece
      auto split16 = [&](const uint4& lo, const uint4& hi, uint32_t* q1, uint32_t* q2) {
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f0 = bf16_lo(w[2 * e]) * inv, f1 = bf16_hi(w[2 * e]) * inv;
          const float f2 = bf16_lo(w[2 * e + 1]) * inv, f3 = bf16_hi(w[2 * e + 1]) * inv;
          const uint32_t code = q8::encode4(f0, f1, f2, f3);
          const float2 d0 = q8::decode2(code), d1 = q8::decode2(code >> 16);
          q1[e] = code;
          q2[e] = q8::encode4(f0 - d0.x, f1 - d0.y, f2 - d1.x, f3 - d1.y);
        }
      };
      // one query tile: each warpgroup half of the shared rows' elements; two: all of its own rows'
#pragma unroll 1
      for (int ch = kDual ? 0 : 2 * wg; ch < (kDual ? 4 : 2 * wg + 2); ++ch) {
        uint32_t q1[8], q2[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) split16(q16(ch * 4 + 2 * h), q16(ch * 4 + 2 * h + 1), q1 + 4 * h, q2 + 4 * h);
        const uint32_t col = lane_addr + kColQ + (uint32_t)(kDual ? wg : 0) * 64 + (uint32_t)ch * 8;
        tmem_st8(col, q1);
        tmem_st8(col + 32, q2);
      }
    }
    if (nt > 0 && ok) {
      if (kRep > 1) {                      // P is zero at the other repetitions' keys, for good
        const uint32_t z[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
        for (int c = 0; c < 32; c += 8) tmem_st8(lane_addr + kColP + (uint32_t)wg * kPW + c, z);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q8_full);
    }
    // Scales: a lane holds the word of one (own tile, group) of a batch of 32 / kTG tiles; a tile's words
    // are handed out by shuffles.  The next batch's bytes are loaded a batch ahead and the block ids they
    // need two ahead, so neither latency is waited for.
    constexpr int kSB = 32 / kTG;
    const int first = kDual ? 0 : wg, step = kDual ? 1 : 2;
    auto scale_pos = [&](int batch) -> int {     // first position of this lane's group, or none
      const int i = first + step * (batch * kSB + lane / kTG);
      const int pos = (t_begin + i) * kBN + key0 + (lane % kTG) * kTW;
      return i < np && pos < v.L ? pos : -1;
    };
    auto scale_blk = [&](int batch) -> int {
      const int pos = scale_pos(batch);
      if (a.block_table == nullptr || pos < 0) return 0;
      const int blk = a.block_table[(size_t)b * a.max_blocks + (pos >> a.block_shift)];
      return blk < 0 || blk >= a.num_blocks ? 0 : blk;
    };
    auto scale_word = [&](int batch, int blk) -> uint32_t {
      const int pos = scale_pos(batch);
      if (pos < 0) return 0x007f007fu;           // groups behind the prefix: 2^0
      const size_t at = a.block_table == nullptr ? ((size_t)b * a.Hkv + g) * a.scale_cols + (pos >> a.scale_shift)
                                                 : (size_t)blk * a.Hkv + g;
      return (uint32_t)q8::clean_byte(a.k_scale[at]) | ((uint32_t)q8::clean_byte(a.v_scale[at]) << 16);
    };
    uint32_t sc_cur = 0, sc_nxt = scale_word(0, scale_blk(0));
    int blk_nxt = scale_blk(1), batch = 0;
    auto scales_at = [&](int k) -> int {         // first lane of own tile k's words; turns to the next batch
      const int j = k % kSB;
      if (j == 0) {
        sc_cur = sc_nxt;
        ++batch;
        sc_nxt = scale_word(batch, blk_nxt);
        blk_nxt = scale_blk(batch + 1);
      }
      return j * kTG;
    };

    float m_used = -INFINITY, l = 0.f, alpha = 1.f;
    bool resc = false;
    const uint32_t s_col = kColS + (uint32_t)wg * kBN;
    const uint32_t p_col = kColP + (uint32_t)wg * kPW;
    // a new maximum (in the units of the exponent): the reference is raised only past a 2^8 growth
    auto raise = [&](float mx) -> float {
      if (!row_ok) mx = -INFINITY;
      alpha = 1.f;
      resc = false;
      if (mx != -INFINITY && (m_used == -INFINITY || mx > m_used + kRescaleLog2)) {
        if (m_used != -INFINITY) {
          alpha = fast_exp2(m_used - mx);
          resc = true;
        }
        m_used = mx;
      }
      return m_used == -INFINITY ? 0.f : -m_used;
    };
    auto wait_s = [&](int k) -> bool {
      const bool got = mbar_wait(&bars.s_full[wg], k & 1, u.wait);
      if (!__all_sync(0xffffffffu, got)) return false;
      tc_fence_after();
      return true;
    };
    auto s_read = [&]() {                        // S_w is in registers: the tensor cores may write the next
      if (!kDual) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.s_empty[wg]);
      }
    };
    // this warpgroup's previous P V is done: O may be rescaled and (one query tile) P written
    auto wait_pv = [&](int k) -> bool {
      const bool got = k < 1 || mbar_wait(&bars.pv_done[wg], (k - 1) & 1, u.wait);
      if (!__all_sync(0xffffffffu, got)) return false;
      if (warp_live && __any_sync(0xffffffffu, resc)) {
        tc_fence_after();
#pragma unroll 1
        for (int ch = 0; ch < kD; ch += 16) {
          uint32_t o[16];
          tmem_ld16(lane_addr + o_col + ch, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st8(lane_addr + o_col + ch, *reinterpret_cast<uint32_t(*)[8]>(o));
          tmem_st8(lane_addr + o_col + ch + 8, *reinterpret_cast<uint32_t(*)[8]>(o + 8));
        }
      }
      return true;
    };
    auto p_written = [&]() {
      if (warp_live) tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full[wg]);
    };

    // full prefix tiles, then the masked ones (the end of a ragged prefix, the tree's)
    const int nfull = max(0, min(np, v.L / kBN - t_begin));
    int i = first, k = 0;
    for (; ok && i < nfull; i += step, ++k) {
      const int j0 = scales_at(k);
      if (!(ok = wait_s(k))) break;
      uint32_t s[kNC];
      if (warp_live) {
#pragma unroll
        for (int c = 0; c < kNC; c += 16) tmem_ld16(lane_addr + s_col + key0 + c, *reinterpret_cast<uint32_t(*)[16]>(s + c));
        uint32_t sc[kTG];
#pragma unroll
        for (int gr = 0; gr < kTG; ++gr) sc[gr] = __shfl_sync(0xffffffffu, sc_cur, j0 + gr);
        tmem_wait_ld();
        s_read();
        float mx = -INFINITY;
#pragma unroll
        for (int gr = 0; gr < kTG; ++gr) {
          const uint32_t* q = s + kTW * gr;
          float m0 = fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
          float m1 = fmaxf(__uint_as_float(q[2]), __uint_as_float(q[3]));
#pragma unroll
          for (int c = 4; c < kTW; c += 4) {
            m0 = max3f(m0, __uint_as_float(q[c]), __uint_as_float(q[c + 1]));
            m1 = max3f(m1, __uint_as_float(q[c + 2]), __uint_as_float(q[c + 3]));
          }
          mx = fmaxf(mx, fmaf(fmaxf(m0, m1), c_row * k_factor(sc[gr]), v_exponent(sc[gr])));
        }
        const float nmu = raise(mx);
        float lsum = 0.f;
#pragma unroll
        for (int gr = 0; gr < kTG; ++gr) {
          const uint32_t* q = s + kTW * gr;
          // P' = 2^(s c + e - M); the row sum takes 2^e back
          const float cg = c_row * k_factor(sc[gr]), nb = nmu + v_exponent(sc[gr]);
          float g0 = 0.f, g1 = 0.f;
#pragma unroll
          for (int c = 0; c < kTW; c += 2) {
            float x0, x1;
            fma2(x0, x1, __uint_as_float(q[c]), __uint_as_float(q[c + 1]), cg, cg, nb, nb);
            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
            add2(g0, g1, g0, g1, p0, p1);
            s[(gr * kTW + c) / 2] = pack_f16x2(p0, p1);   // over scores that have been used
          }
          lsum = fmaf(g0 + g1, v_inverse(sc[gr]), lsum);
        }
        l = l * alpha + lsum;
      } else {
        s_read();
      }
      if (!(ok = wait_pv(k))) break;
      if (warp_live) {
#pragma unroll
        for (int c = 0; c < kNC / 2; c += 8) tmem_st8(lane_addr + p_col + key0 / 2 + c, *reinterpret_cast<uint32_t(*)[8]>(s + c));
      }
      p_written();
    }
    bool mask_ready = false;
    for (; ok && i < nt; i += step, ++k) {
      const bool tree = i >= np;
      const int t = t_begin + i, kbase = tree ? (t - v.nPT) * kBN : t * kBN;
      const int j0 = scales_at(k);
      if (!(ok = wait_s(k))) break;
      if (tree && !mask_ready) {
        const bool got = mbar_wait(&bars.mask_full, 0, u.wait);
        if (!(ok = __all_sync(0xffffffffu, got) != 0)) break;
        mask_ready = true;
      }
      uint32_t pk[kNC / 2];
      if (warp_live) {
        // 16 keys at a time, read from TMEM for the maximum and again for the exponentials
        const int n0 = (tree ? v.N : v.L) - kbase;
        uint32_t w0 = 0xffffffffu, w1 = 0xffffffffu;
        if (tree) {
          const int wi = kbase >> 5;
          w0 = sMask[nl * u.W + wi];
          w1 = (wi + 1 < u.W) ? sMask[nl * u.W + wi + 1] : 0u;
        }
        if (n0 < 32) w0 &= n0 <= 0 ? 0u : ((1u << n0) - 1u);
        if (n0 < 64) w1 &= n0 <= 32 ? 0u : ((1u << (n0 - 32)) - 1u);
        auto chunk = [&](int c, uint32_t (&s)[16]) {
          const int c0 = key0 + c;
          tmem_ld16(lane_addr + s_col + c0, s);
          const uint32_t bits = (c0 < 32 ? w0 : w1) >> (c0 & 31);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) s[e] = ((bits >> e) & 1u) ? s[e] : 0xff800000u;
        };
        auto scale_of = [&](int c) -> uint32_t {   // (2^0 for the tree's keys)
          return __shfl_sync(0xffffffffu, sc_cur, j0 + c / kTW);
        };
        // (a factor that underflows, all-zero rows over all-zero blocks at a small scale: never 0, a masked score is -inf)
        auto factor = [&](uint32_t sc) -> float {
          const float f = (tree ? sl2 : c_row) * k_factor(sc);
          return f == 0.f ? 1.17549435e-38f : f;
        };
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < kNC; c += 16) {
          uint32_t s[16];
          chunk(c, s);
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
            const uint32_t sc = scale_of(c + h);
            float m0 = __uint_as_float(s[h]);
#pragma unroll
            for (int e = 1; e < 8; ++e) m0 = fmaxf(m0, __uint_as_float(s[h + e]));
            mx = fmaxf(mx, fmaf(m0, factor(sc), v_exponent(sc)));
          }
        }
        const float nmu = raise(mx);
        float lsum = 0.f;
#pragma unroll
        for (int c = 0; c < kNC; c += 16) {
          uint32_t s[16];
          chunk(c, s);
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
            const uint32_t sc = scale_of(c + h);
            const float cg = factor(sc), nb = nmu + v_exponent(sc);
            float gs = 0.f;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float p0 = fast_exp2(fmaf(__uint_as_float(s[h + e]), cg, nb));
              const float p1 = fast_exp2(fmaf(__uint_as_float(s[h + e + 1]), cg, nb));
              gs += p0 + p1;
              pk[(c + h + e) / 2] = tree ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
            }
            lsum = fmaf(gs, v_inverse(sc), lsum);
          }
        }
        l = l * alpha + lsum;
      }
      s_read();
      if (!(ok = wait_pv(k))) break;
      if (warp_live) {
#pragma unroll
        for (int c = 0; c < kNC / 2; c += 8) tmem_st8(lane_addr + p_col + key0 / 2 + c, *reinterpret_cast<uint32_t(*)[8]>(pk + c));
      }
      p_written();
    }
    const int kn = kDual ? nt : (nt - wg + 1) >> 1;
    if (ok && kn > 0 && !mbar_wait(&bars.pv_done[wg], (kn - 1) & 1, u.wait)) ok = false;
    if (!ok) abort_cta(a, b, &s_abort);
    row_m = m_used;
    row_l = l;
    if (!kDual && wg == 1) s_ml1[row] = make_float2(m_used, l);
  }

  // ---------------------------------------------------------------- epilogue / teardown
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint8_t* sStage = smem;             // the query tiles and the rings, idle once every product is done
  if (!s_abort) {
    fence_proxy_async();
    if (kDual ? (warp >= 4 && warp < 12) : (warp >= 4 && warp < 8)) {
      const int wg = (warp - 4) >> 2;
      const int q4 = warp & 3;
      const int row = q4 * 32 + lane;
      const int in_tile = kDual ? row : row % kLanes;
      const int crow = kDual ? wg * rows_tile + row : row;   // staged row: one per row of the tiles, or per TMEM lane
      const bool row_ok = in_tile < rows_tile && r0 + (kDual ? crow : in_tile) < r_hi;
      const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16);
      const uint32_t o_first = kColO + (kDual ? (uint32_t)wg * kD : 0u);
      const bool two = !kDual && nt > 1;   // a second accumulator (warpgroup 1's) to merge
      const float2 ml1 = two ? s_ml1[row] : make_float2(-INFINITY, 0.f);
      const float M = fmaxf(row_m, ml1.x);
      const float Mu = M == -INFINITY ? 0.f : M;
      const float a0 = exp2f(row_m - Mu);
      const float a1 = two ? exp2f(ml1.x - Mu) : 0.f;
      const float l = row_l * a0 + ml1.y * a1;
      // M = -inf: no keys (or no mass), its O is not read (a NaN sum is kept: its row is NaN)
      if (!kDual || row < rows_tile) s_ml[crow] = make_float2(l == 0.f ? -INFINITY : Mu, l);
#pragma unroll
      for (int ch = 0; ch < kD / 32; ++ch) {
        uint32_t o0[32], o1[32];
        tmem_ld32(lane_addr + o_first + ch * 32, o0);
        if (two) tmem_ld32(lane_addr + kColO + kD + ch * 32, o1);
        tmem_wait_ld();
        if (row_ok) {
          float4* dst = reinterpret_cast<float4*>(sStage + (size_t)crow * kStageF + ch * 128);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              f[e] = __uint_as_float(o0[4 * q + e]) * a0 + (two ? __uint_as_float(o1[4 * q + e]) * a1 : 0.f);
            dst[q] = make_float4(f[0], f[1], f[2], f[3]);
          }
        }
      }
    }
    __syncthreads();
    if (s_err != 0 && tid == 0) flag_status(a.status, b, TSD_ERR_CAPACITY);
    // every thread merges the repetitions of its pieces of rows and writes them out coalesced: the finished
    // row, or the split partial (relative to its M, with (M, l))
    const int nrows = r_hi - r0;
    const bool err = s_err != 0;
    float* wo = reinterpret_cast<float*>(a.workspace);
    float* wml = wo + (size_t)pairs * ns * u.Rmax * kD;
    const size_t base = ((size_t)pair * ns + split) * u.Rmax + r0;
    for (int idx = tid; idx < nrows * (kD / 4); idx += kThreadsQ) {
      const int cr = idx / (kD / 4), c = idx % (kD / 4);
      float M = -INFINITY, l = 0.f, w[kRep];
#pragma unroll
      for (int q = 0; q < kRep; ++q) M = fmaxf(M, s_ml[cr + q * kLanes].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kRep; ++q) {
        const float2 ml = s_ml[cr + q * kLanes];
        w[q] = kRep == 1 ? 1.f : exp2f(ml.x - (M == -INFINITY ? 0.f : M));
        l += ml.y * w[q];
        if (kRep == 1 || w[q] != 0.f) {
          const float4 x = *reinterpret_cast<const float4*>(sStage + (size_t)(cr + q * kLanes) * kStageF + c * 16);
          o.x = fmaf(w[q], x.x, o.x), o.y = fmaf(w[q], x.y, o.y), o.z = fmaf(w[q], x.z, o.z), o.w = fmaf(w[q], x.w, o.w);
        }
      }
      const int rr = r0 + cr, node = rr / G, hh = rr % G;
      const bool poison = s_poison != 0;
      if (poison) {
        const uint32_t* bits = sMask + (size_t)(node - node0) * u.W;
        const int n0 = max(t_begin - v.nPT, 0) * kBN, n1 = min(v.N, max(t_begin + nt - v.nPT, 0) * kBN);
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
          const float x = visible_nonfinite<__nv_bfloat16>(a, b, g, bits, n0, n1, 4 * c + e);
          if (e == 0) o.x += x;
          else if (e == 1) o.y += x;
          else if (e == 2) o.z += x;
          else o.w += x;
        }
      }
      const size_t orow = ((size_t)b * a.Nmax + node) * a.Hq + g * G + hh;
      if (direct) {
        const float inv = (l == 0.f || err) ? 0.f : 1.f / l;
        if (err) o = make_float4(0.f, 0.f, 0.f, 0.f);
        reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + orow * kD)[c] =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (c == 0 && a.lse) a.lse[orow] = err ? 0.f : (M + __log2f(l)) * kLn2;
      } else {
        reinterpret_cast<float4*>(wo + (base + cr) * kD)[c] = o;
        if ((kRep > 1 || poison) && u.tickets != nullptr)   // the merge below takes this split's rows from here
          *reinterpret_cast<float4*>(sStage + (size_t)cr * kStageF + c * 16) = o;
        if (c == 0) *reinterpret_cast<float2*>(wml + (base + cr) * 2) = make_float2(M, l);
      }
    }
  } else {
    // time-out: let this CTA's own TMA copies and MMAs land (bounded) before freeing TMEM
    if (tid == 0) {
      if (s_q_issued) mbar_wait(&bars.q_full, 0, u.wait);
      for (int i = max(0, s_k_issued - u.ks); i < s_k_issued; ++i) mbar_wait(&bars.k_full[i % u.ks], (i / u.ks) & 1, u.wait);
      for (int i = max(0, s_v_issued - u.vs); i < s_v_issued; ++i) mbar_wait(&bars.v_full[i % u.vs], (i / u.vs) & 1, u.wait);
      if (s_kt_issued > 0) mbar_wait(&bars.kt_full, (s_kt_issued - 1) & 1, u.wait);
      for (int c = 0; c < kVB; ++c)
        if (s_vt_issued[c] > 0) mbar_wait(&bars.vt_full[c], (s_vt_issued[c] - 1) & 1, u.wait);
    }
    if ((warp == 3 || warp == 1) && lane == 0) {
      uint64_t* fin = &bars.fin[warp == 3 ? 0 : 1];
      tc_commit(fin);
      mbar_wait(fin, 0, u.wait);
    }
    if (direct) {
      zero_rows<__nv_bfloat16>(a, b, g, G, r0, r_hi);
    } else {   // an unusable partial: the merge skips it (and zeroes the rows: status is flagged)
      float* wml = reinterpret_cast<float*>(a.workspace) + (size_t)pairs * ns * u.Rmax * kD;
      const size_t base = ((size_t)pair * ns + split) * u.Rmax;
      for (int r = r0 + tid; r < r_hi; r += kThreadsQ)
        *reinterpret_cast<float2*>(wml + (base + r) * 2) = make_float2(-INFINITY, 0.f);
    }
  }
  if (!direct && u.tickets != nullptr) {
    const int t = take_ticket(u.tickets + word, ns, &s_ticket);
    if (t == 1) {
      __threadfence();
      if (tid == 0) s_status = __ldcg(a.status + b);
      __syncthreads();
      merge_splits<true>(a, u, b, g, G, r0, r_hi, split, s_abort != 0 || s_status != 0, sStage,
                   reinterpret_cast<float*>(sStage + (size_t)kRows * kStageF), kRows, pair, pairs);
    } else if (t == 2 && tid == 0) {
      flag_status(a.status, b, TSD_ERR_WORKSPACE);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Shared-memory layout: query tile(s), the tree's K tile, K and V code rings, the V operand ring, ancestor
// bits, parent slots.  Rings shrink when a large tree's ancestor bits need the room; false when even
// the smallest do not fit.
struct QLayout {
  int rows, W, ks, vs;
  uint32_t kt_off, k_off, v_off, vb_off, mask_off, ps_off;
  size_t smem;
};
constexpr uint32_t kSmemLimit = 227 * 1024 - 6144;   // leave room for the static shared variables
bool q8_layout(bool dual, int G, int Nmax, QLayout& L) {
  L.rows = dual ? 2 * kBM : kBM;
  L.W = (Nmax + 31) / 32;
  const uint32_t q_bytes = kQBytes * (dual ? 2 : 1);
  const uint32_t mask_bytes = ((uint32_t)(L.rows / G) * L.W * 4 + 15) & ~15u;
  const uint32_t ps_bytes = (uint32_t)(Nmax + 1) * 4;
  auto total = [&](int ks, int vs) {
    return 1024 + q_bytes + kSlot + (uint32_t)(ks + vs) * kSlot8 + kVB * kSlot + mask_bytes + ps_bytes;
  };
  L.ks = kMaxRing, L.vs = kMaxRing - 1;
  while (total(L.ks, L.vs) > kSmemLimit && L.vs > 2) {
    if (L.ks > L.vs) --L.ks; else --L.vs;
  }
  if (total(L.ks, L.vs) > kSmemLimit) return false;
  L.kt_off = q_bytes;
  L.k_off = L.kt_off + kSlot;
  L.v_off = L.k_off + (uint32_t)L.ks * kSlot8;
  L.vb_off = L.v_off + (uint32_t)L.vs * kSlot8;
  L.mask_off = L.vb_off + kVB * kSlot;
  L.ps_off = L.mask_off + mask_bytes;
  L.smem = total(L.ks, L.vs);
  return L.mask_off >= (uint32_t)L.rows * kStageF;   // the staged rows fit below the ancestor bits
}

// Splits are merged by the last CTA of each row block (attn_umma.cu) where only the last blocks are split,
// and in the two-tile kernel for two splits of 32 or more blocks: one CTA reads a block's partials at ~64
// bytes a clock, the merge kernel takes all SMs to it (in the kernel / merge kernel: 16 x 8 blocks of 240
// rows, two splits 131 / 141 us; 4 blocks, two splits 19.2 / 14.5 us; 8 blocks, 18 splits 77 / 35 us).
bool q8_merges_in_kernel(const AttnPlan& p, const QLayout& L, int B, int Hkv) {
  const char* merge_env = getenv("TSD_ATTN_MERGE");
  const long long groups = (long long)B * Hkv * p.umtiles;
  const bool want = p.whole > 0 || (merge_env != nullptr ? merge_env[0] == 'f' : p.dual && p.usplits <= 2 && groups >= 32);
  return want && p.usplits > 1 && (size_t)L.mask_off >= (size_t)L.rows * kStageF + (size_t)p.usplits * L.rows * 12 &&
         groups * 4 <= (long long)kAttnTicketBytes;
}

typedef void (*Q8Kernel)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap,
                         const AttnArgs, const QParams);
template <bool kDual, int kRep>
Q8Kernel pick_groups(int groups) {
  return groups == 1 ? attn_q8_umma_kernel<kDual, kRep, 1>
                     : (groups == 4 ? attn_q8_umma_kernel<kDual, kRep, 4> : attn_q8_umma_kernel<kDual, kRep, 8>);
}
Q8Kernel pick_kernel(bool dual, int rep, int groups) {
  if (dual) return pick_groups<true, 1>(groups);
  return rep == 1 ? pick_groups<false, 1>(groups) : (rep == 2 ? pick_groups<false, 2>(groups) : pick_groups<false, 4>(groups));
}

}  // namespace

bool q8_umma_eligible(const AttnArgs& a, const AttnPlan& p, tsd_dtype dtype) {
  const int G = a.Hq / a.Hkv;
  if (dtype != TSD_BF16 || a.d != kD || a.k_tree == nullptr || a.Lcap <= 0) return false;
  if (G < 1 || G > 128) return false;
  // TMA row coordinates are 32-bit
  const long long rows = a.block_table == nullptr ? (long long)a.B * a.Hkv * a.Lcap
                                                  : ((long long)a.num_blocks * a.Hkv) << a.block_shift;
  if (rows <= 0 || rows > 0x7fffffffLL || (long long)a.B * a.Nmax > 0x7fffffffLL) return false;
  QLayout L;
  return q8_layout(p.dual, G, a.Nmax, L) && encoder() != nullptr;
}

bool q8_umma_merges(const AttnPlan& p, int G, int Nmax, int B, int Hkv) {
  QLayout L;
  return q8_layout(p.dual, G, Nmax, L) && q8_merges_in_kernel(p, L, B, Hkv);
}

tsd_status launch_attention_q8_umma(const AttnArgs& a, const AttnPlan& p, int* tickets, bool* merged,
                                    cudaStream_t stream) {
  const int G = a.Hq / a.Hkv;
  QLayout L;
  if (!q8_layout(p.dual, G, a.Nmax, L)) return TSD_ERR_INVALID_ARG;
  QParams u{};
  u.splits = p.usplits, u.Rmax = p.Rmax, u.mtiles = p.umtiles, u.whole = p.whole;
  u.wait = (uint32_t)kWaitCycles;
  u.withhold = -1;
  u.lpt = a.B > 1 && a.B <= 512 ? 1 : 0;
  const char* l2_env = getenv("TSD_ATTN_L2HINT");
  u.evict_first = (p.umtiles == 1 && !(l2_env != nullptr && l2_env[0] == '0')) ? 1 : 0;
  if (const char* w = getenv("TSD_TEST_WITHHOLD_TILE")) {   // test hook, as in attn_umma.cu
    u.withhold = atoi(w);
    u.wait = 100000;
  }
  u.W = L.W, u.ks = L.ks, u.vs = L.vs;
  u.kt_off = L.kt_off, u.k_off = L.k_off, u.v_off = L.v_off, u.vb_off = L.vb_off;
  u.mask_off = L.mask_off, u.ps_off = L.ps_off;
  const bool fuse = tickets != nullptr && q8_merges_in_kernel(p, L, a.B, a.Hkv);
  u.tickets = fuse ? tickets : nullptr;
  *merged = fuse;
  const int blocks = a.B * a.Hkv * u.mtiles;
  if (u.whole > 0 && !fuse) {   // (no ticket words, or no room for the merge: no block is split)
    u.whole = blocks, u.splits = 1;
    *merged = true;
  }

  // the rows of one query tile are repeated while they fit
  const int rep = p.dual || p.Rmax > 64 ? 1 : (p.Rmax > 32 ? 2 : 4);
  u.npt = kBM / rep / G;
  const int groups = a.scale_shift >= 6 ? 1 : (a.scale_shift >= 4 ? 4 : 8);
  auto kernel = pick_kernel(p.dual, rep, groups);
  // (before the tensor maps: their encoding is a driver call, which needs the context that a host thread's first
  // runtime call binds)
  allow_smem(kernel);
  CUtensorMap mq, mk, mv, mkt, mvt;
  {  // Q [B*Nmax rows][Hq][128] -> box (64, G, npt)
    uint64_t dims[3] = {(uint64_t)kD, (uint64_t)a.Hq, (uint64_t)a.B * a.Nmax};
    uint64_t str[2] = {(uint64_t)kD * 2, (uint64_t)a.Hq * kD * 2};
    uint32_t box[3] = {64, (uint32_t)G, (uint32_t)u.npt};
    if (!make_map(&mq, a.q, 3, dims, str, box)) return TSD_ERR_CUDA;
  }
  {  // codes [rows][128 bytes]
    const int bs = 1 << a.block_shift;
    u.box_rows = a.block_table == nullptr ? kBN : (bs < kBN ? bs : kBN);
    const uint64_t rows = a.block_table == nullptr ? (uint64_t)a.B * a.Hkv * a.Lcap : (uint64_t)a.num_blocks * a.Hkv * bs;
    uint64_t dims[2] = {(uint64_t)kD, rows};
    uint64_t str[1] = {(uint64_t)kD};
    uint32_t box[2] = {(uint32_t)kD, (uint32_t)u.box_rows};
    if (!make_map(&mk, a.k_cache, 2, dims, str, box, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
        !make_map(&mv, a.v_cache, 2, dims, str, box, CU_TENSOR_MAP_DATA_TYPE_UINT8))
      return TSD_ERR_CUDA;
  }
  {  // tree K/V [B*Nmax][Hkv][128] -> box (64, 1, 64)
    uint64_t dims[3] = {(uint64_t)kD, (uint64_t)a.Hkv, (uint64_t)a.B * a.Nmax};
    uint64_t str[2] = {(uint64_t)kD * 2, (uint64_t)a.Hkv * kD * 2};
    uint32_t box[3] = {64, 1, (uint32_t)kBN};
    if (!make_map(&mkt, a.k_tree, 3, dims, str, box) || !make_map(&mvt, a.v_tree, 3, dims, str, box))
      return TSD_ERR_CUDA;
  }
  const dim3 grid((unsigned)(u.whole + (blocks - u.whole) * u.splits));
  if (launch_pdl(kernel, grid, dim3(threads_of(rep)), L.smem, stream, mq, mk, mv, mkt, mvt, a, u) != cudaSuccess)
    return TSD_ERR_CUDA;
  return TSD_OK;
}

}  // namespace tsd
