// tsd_sample_rows: one token per row of logits under temperature, top-k, top-p and min-p.
//
// The target's own token ("Acelerando Sonar a traves de la especulacion", sections "Decodificacion
// especulativa" and "Objetivo-Borrador": the target's logits are sampled for the token after the accepted
// run) and the draft's tokens come from filtered distributions in serving; the acceptance kernels test
// tokens that are already drawn, this one draws them.
//
// Mathematics: with M = max z and w_v = exp((z_v - M) / T), tokens ordered by (z desc, id asc):
//   top-k keeps the first k; top-p keeps a token while the mass before it is < P * (mass of those k);
//   min-p keeps w >= m; all three are prefixes of that order.  The token is the smallest id t with
//   sum_{kept v <= t} w_v > u * Z, Z the kept mass.
// A border between two tokens decides an integer, and with 10^5 tokens the borders are ~10^-5 Z apart,
// so weights are computed in fp64 (2^x by a 128-entry table and a degree-4 polynomial, error < 2^-49) and
// held as integers in units of 2^-sh, sh = min(51, 62 - ceil(log2 V)): sums are then exact and the same in
// any order.
//
// Layout: a row is one cluster of 1 to 8 CTAs, each holding its share of the tokens in shared memory (one
// read of the row from HBM), each of its 16 warps a contiguous piece of them, 128 tokens at a time (four independent
// chains per thread: the fp64 latency, not its rate, bounds a small batch).  The k-th largest and the border
// of top-p are found by radix selection on order-preserving keys (8-bit digits, histograms of counts or
// masses summed over the cluster through distributed shared memory); top-p first counts tokens in 1024
// equal bins of (M - z) / T, which bound the mass so well that the border lies in a window of a few bins,
// and the mass histograms (whose 64-bit atomics collide) see those bins' tokens alone.  Ties at a border go
// to the lowest ids.  A small top-k (up to 2048 tokens) leaves the cluster early: every warp knows, from
// counts, where its kept tokens stand in the row's list, writes them there in the first CTA's shared memory,
// and that CTA does top-p, min-p and the draw on the list alone; a small vocabulary is such a list at once.
// What bounds it: ~11 fp64 and ~30 other operations per token and pass over the weights; a single row is a
// chain of passes and cluster barriers.  Measured, bf16 rows of 128256 normal logits of deviation 2.5 at T 0.8 (1 row /
// 64 rows, graph replays; the bytes of 64 take 2.5 us): greedy 4.9 / 14 us, temperature 13 / 47 us, top-k 50 18 / 56 us,
// with P 0.9 21 / 62 us, P 0.9 alone 39 / 115 us (at T 1.6, where it keeps a flat tenth of the row: 62 / 189 us).
#include <cooperative_groups.h>

#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace tsd {

namespace {

constexpr int kCS = 8;          // most CTAs per row
constexpr int kSmall = 2048;    // a top-k up to here is finished by one CTA
constexpr int kTR = 512;
constexpr int kWR = kTR / 32;
constexpr int kBins = 1024;     // first bins of top-p
constexpr int kList = 1024;     // tokens of a warp's list
typedef unsigned long long u64;

// Order-preserving unsigned keys (larger value -> larger key); NaN -> 0, below -inf.
__device__ __forceinline__ uint32_t skey(__nv_bfloat16 x) {
  const uint32_t b = __bfloat16_as_ushort(x);
  if ((b & 0x7fffu) > 0x7f80u) return 0u;
  return (b & 0x8000u) ? 0x10000u - b : (b | 0x8000u);
}
__device__ __forceinline__ uint32_t skey(float x) {
  const uint32_t b = __float_as_uint(x);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0u;
  return (b & 0x80000000u) ? 0u - b : (b | 0x80000000u);
}
// (+0 added: -0 becomes +0, whose weight it has)
__device__ __forceinline__ float sval(__nv_bfloat16 x) { return __bfloat162float(x) + 0.f; }
__device__ __forceinline__ float sval(float x) { return x + 0.f; }
// the value of a key (not of NaN's)
__device__ __forceinline__ float key_value(uint32_t k, __nv_bfloat16) {
  const uint32_t b = (k & 0x8000u) ? (k & 0x7fffu) : 0x10000u - k;
  return __uint_as_float(b << 16);
}
__device__ __forceinline__ float key_value(uint32_t k, float) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : 0u - k);
}

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// fp32 bits as a double by shifts (the conversion instruction runs at an eighth of the integer rate).
// Zeros and subnormals come out as +-2^-127 (1 + f): M and z alike, so that differences stay right.
__device__ __forceinline__ double as_double(float z) {
  const uint32_t b = __float_as_uint(z), mag = b & 0x7fffffffu;
  return __hiloint2double((int)((mag >> 3) + (896u << 20) | (b & 0x80000000u)), (int)(mag << 29));
}

// Weights in units of 2^-sh.
constexpr int kTab = 128;
struct Weigher {
  const double* tab;   // 2^(j / kTab)
  double c;            // kTab log2(e) / T
  double Md;
  float Mh, ts2;       // half the maximum, and 2 / T (halves, so that no difference of logits overflows)
  int sh;
  __device__ __forceinline__ u64 operator()(float z) const {
    const bool live = fmaf(z, -0.5f, Mh) * ts2 <= 100.f;     // e^-100 rounds to 0; false for -inf and NaN
    // t = kTab x rounded to an integer n (kept in the low mantissa bits), f = kTab x - n in [-1/2, 1/2]
    const double dz = as_double(z) - Md;
    const double magic = 6755399441055744.0;     // 1.5 * 2^52
    const double t = fma(dz, c, magic);
    const int n = __double2loint(t);
    const double f = fma(dz, c, -(t - magic));
    // 2^(f / kTab) = exp(g f), g = ln 2 / kTab: Taylor terms to f^4 (the next is < 2e-15)
    constexpr double g = 0.69314718055994530942 / kTab;
    double p = fma(f, g * g * g * g / 24.0, g * g * g / 6.0);
    p = fma(f, p, g * g / 2.0);
    p = fma(f, p, g);
    p = fma(f, p, 1.0);
    // round(2^(n / kTab) p 2^sh): below 2^52, so adding 2^52 leaves the integer in the mantissa
    const double y = p * tab[n & (kTab - 1)] * __hiloint2double((1023 + sh + (n >> 7)) << 20, 0);
    const u64 w = (u64)__double_as_longlong(y + 4503599627370496.0) & 0xfffffffffffffull;
    return live ? w : 0;
  }
};

template <typename T>
__global__ void __launch_bounds__(kTR, 2) sample_rows_kernel(const SampleArgs a) {
  pdl_trigger();
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), cs = a.cs;
  const int row = blockIdx.x / cs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  extern __shared__ __align__(16) uint8_t smem[];
  T* sZ = reinterpret_cast<T*>(smem);
  __shared__ double s_tab[kTab];
  __shared__ uint32_t s_cnt[256], s_lo[256], s_hi[256];
  __shared__ uint32_t x_cnt[2][256];      // exchange slots, double buffered by phase
  __shared__ u64 x_mass[2][256];
  __shared__ u64 x_u[2];
  __shared__ int s_bin, s_win[2];
  __shared__ uint32_t s_bins[kBins];      // top-p's first bins
  __shared__ double2 s_dsum[kWR];
  // top-p: a warp's tokens down to the window, by position (s_idx, s_listed); a small top-k: its tokens' (key,
  // id) in id order (s_list)
  __shared__ __align__(16) uint8_t s_lists[kWR * kList * 2];
  static_assert(kSmall * sizeof(uint2) <= sizeof(s_lists), "the small top-k's list shares the room");
  uint16_t (*s_idx)[kList] = reinterpret_cast<uint16_t (*)[kList]>(s_lists);
  uint2* s_list = reinterpret_cast<uint2*>(s_lists);
  __shared__ int s_listed[kWR];
  __shared__ uint32_t s_above_c;
  __shared__ u64 s_above_m;
  __shared__ u64 s_red[kWR];
  __shared__ int s_redi[kWR];
  __shared__ u64 s_each[kCS];
  __shared__ int s_pos;
  const int V = a.V;
  const int lo = rank * a.slice;
  const int cnt = max(0, min(V, lo + a.slice) - lo);
  int ph = 0;

  if (tid < kTab) s_tab[tid] = exp2((double)tid * (1.0 / kTab));
  pdl_wait();
  // (2^-100: below it 64 / T and differences of subnormal logits leave the range of floats)
  float T_in = a.temperature ? a.temperature[row] : 1.f;
  if (T_in > 0.f) T_in = fmaxf(T_in, 0x1p-100f);
  const int k_in = a.top_k ? a.top_k[row] : 0;
  const float P = a.top_p ? a.top_p[row] : 1.f;
  const float m_in = a.min_p ? a.min_p[row] : 0.f;
  float u = a.u[row];
  u = u >= 0.f ? fminf(u, 0.99999994f) : 0.f;    // NaN -> 0

  constexpr int kBits = sizeof(T) * 8;
  const bool topk = k_in > 0 && k_in < V;
  for (int i = tid; i < 256; i += kTR) s_cnt[i] = s_lo[i] = s_hi[i] = 0u;
  __syncthreads();
  // this CTA's slice of the row, read once; its largest key and the lowest id that has it, and for top-k the
  // counts of the keys' first digit
  uint32_t kmax = 0;
  int kpos = INT_MAX;
  {
    const T* g = reinterpret_cast<const T*>(a.logits) + (size_t)row * V + lo;
    if (a.vec) {
      constexpr int E = 16 / sizeof(T);
      for (int i = tid; i < cnt / E; i += kTR) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(g) + i);
        reinterpret_cast<uint4*>(sZ)[i] = w;
        const T* x = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t k = skey(x[e]);
          if (k > kmax) kmax = k, kpos = i * E + e;
          if (topk) atomicAdd(&s_cnt[k >> (kBits - 8)], 1u);
        }
      }
    } else {
      for (int i = tid; i < cnt; i += kTR) {
        const T x = g[i];
        sZ[i] = x;
        const uint32_t k = skey(x);
        if (k > kmax) kmax = k, kpos = i;
        if (topk) atomicAdd(&s_cnt[k >> (kBits - 8)], 1u);
      }
    }
  }
  // (key, ~id) as one 64-bit number: the largest is the largest key at the lowest id
  u64 best = kpos == INT_MAX ? 0 : ((u64)kmax << 32) | (uint32_t)~(uint32_t)(lo + kpos);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) s_red[warp] = best;
  __syncthreads();
  if (tid < 32) {
    best = lane < kWR ? s_red[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) x_u[ph] = best;
  }
  cl.sync();
  best = 0;
  for (int r = 0; r < cs; ++r) best = max(best, *cl.map_shared_rank(&x_u[ph], r));
  ph ^= 1;
  const uint32_t key_max = (uint32_t)(best >> 32);
  const float Mraw = key_value(key_max, T());
  const bool dead = key_max == 0u || Mraw == -INFINITY;
  // (every CTA of the row takes this branch, and none reads a peer's memory after the loop above,
  // which the last barrier of this path keeps alive)
  if (dead || !(T_in > 0.f)) {
    if (rank == 0 && tid == 0) {
      a.tokens[row] = dead ? 0 : (int)~(uint32_t)best;
      if (a.probs) a.probs[row] = dead ? 0.f : 1.f;
    }
    cl.sync();
    return;
  }
  // a row whose maximum is +inf spreads its mass over its infinities
  const bool inf_row = Mraw == INFINITY;
  const float M = inf_row ? 0.f : Mraw;
  auto value = [&](int i) -> float {
    const float z = sval(sZ[i]);
    return inf_row ? (z == INFINITY ? 0.f : -INFINITY) : z;
  };
  Weigher weigh;
  weigh.tab = s_tab;
  weigh.c = kTab * 1.4426950408889634074 / (double)T_in;
  weigh.Md = as_double(M);
  weigh.Mh = 0.5f * M;
  weigh.ts2 = 2.f / T_in;
  weigh.sh = min(51, 62 - (32 - __clz(V - 1)));
  const int sh = weigh.sh;

  // this warp's piece of the slice, and a loop over it by 128 tokens: body(position, inside)
  const int seg = ((cnt + kWR - 1) / kWR + 31) & ~31;
  const int sa = min(cnt, warp * seg), se = min(cnt, sa + seg);
  int listed = -1;                          // tokens in this warp's list, or -1: sweep the piece itself
  auto sweep = [&](auto&& body) {
    if (listed >= 0) {
      for (int n = lane; n < listed; n += 32) body((int)s_idx[warp][n], true);
      return;
    }
    for (int i0 = sa + lane; i0 < se; i0 += 128)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + 32 * j;
        body(min(i, cnt - 1), i < se);
      }
  };

  // kept so far: key > kth, or key == kth at a position below tie_cut
  uint32_t kth = 0;
  int tie_cut = INT_MAX;
  auto kept = [&](uint32_t k, int i) -> bool { return k > kth || (k == kth && i < tie_cut); };

  // ties of key kk: keep the first `keep` of the cluster in id order; returns the local position bound
  auto resolve_ties = [&](uint32_t kk, uint32_t keep) -> int {
    int eq = 0;
    sweep([&](int i, bool in) { eq += in && skey(sZ[i]) == kk; });
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) s_redi[warp] = eq;
    __syncthreads();
    int all = 0, mine = 0;                    // ties of the CTA, and of the warps before this one
    for (int w = 0; w < kWR; ++w) {
      if (w < warp) mine += s_redi[w];
      all += s_redi[w];
    }
    if (tid == 0) x_u[ph] = (u64)all;
    cl.sync();
    long long before = 0;
    for (int r = 0; r < rank; ++r) before += (long long)*cl.map_shared_rank(&x_u[ph], r);
    ph ^= 1;
    const long long take = (long long)keep - before;
    if (take <= 0) return 0;
    if (take >= all) return INT_MAX;
    // the warp that holds the take-th tie finds its position
    if (take > mine && take <= mine + eq) {
      int seen = mine;
      const int n_all = listed >= 0 ? listed : se - sa;
      for (int n0 = 0; n0 < n_all; n0 += 32) {
        const bool in = n0 + lane < n_all;
        const int i = !in ? 0 : (listed >= 0 ? (int)s_idx[warp][n0 + lane] : sa + n0 + lane);
        const unsigned bal = __ballot_sync(0xffffffffu, in && skey(sZ[i]) == kk);
        const int n = __popc(bal);
        if (seen + n >= take) {
          if (((bal >> lane) & 1u) && seen + __popc(bal & ((1u << lane) - 1u)) == take - 1) s_pos = i + 1;
          break;
        }
        seen += n;
      }
    }
    __syncthreads();
    return s_pos;
  };
  // where this warp's tokens above kk and its ties stand in the row: counts before them, in id order
  auto counts_before = [&](uint32_t kk, uint32_t& gt, uint32_t& eq) {
    uint32_t g = 0, e = 0;
    sweep([&](int i, bool in) {
      const uint32_t k = skey(sZ[i]);
      g += in && k > kk;
      e += in && k == kk;
    });
    g = __reduce_add_sync(0xffffffffu, g), e = __reduce_add_sync(0xffffffffu, e);
    if (lane == 0) s_red[warp] = (u64)g << 32 | e;
    __syncthreads();
    u64 all = 0, mine = 0;
    for (int w = 0; w < kWR; ++w) {
      if (w < warp) mine += s_red[w];
      all += s_red[w];
    }
    if (tid == 0) x_u[ph] = all;
    cl.sync();
    for (int r = 0; r < rank; ++r) mine += *cl.map_shared_rank(&x_u[ph], r);
    ph ^= 1;
    gt = (uint32_t)(mine >> 32), eq = (uint32_t)mine;
  };
  auto clear_hist = [&]() {
    for (int i = tid; i < 256; i += kTR) s_cnt[i] = s_lo[i] = s_hi[i] = 0u;
    __syncthreads();
  };
  // a 64-bit shared-memory sum in two native 32-bit atomics: the low word's carry goes with the high word
  auto add_mass = [&](int bin, u64 w) {
    const uint32_t wl = (uint32_t)w, old = atomicAdd(&s_lo[bin], wl);
    const uint32_t up = (uint32_t)(w >> 32) + (old + wl < old ? 1u : 0u);
    if (up) atomicAdd(&s_hi[bin], up);
  };
  // cluster sums of the histogram, then (warp 0) from bin 255 down the first bin where the running count
  // reaches want_c (mass == 0) or the running mass reaches want_m; s_bin, s_above_c, s_above_m
  auto gather_hist = [&](bool mass) {
    __syncthreads();
    for (int i = tid; i < 256; i += kTR) {
      x_cnt[ph][i] = s_cnt[i];
      if (mass) x_mass[ph][i] = ((u64)s_hi[i] << 32) + s_lo[i];
    }
    cl.sync();
    if (tid < 256) {
      uint32_t c = 0;
      for (int r = 0; r < cs; ++r) c += cl.map_shared_rank(&x_cnt[ph][0], r)[tid];
      s_cnt[tid] = c;
    } else if (mass) {
      u64 m = 0;
      for (int r = 0; r < cs; ++r) m += cl.map_shared_rank(&x_mass[ph][0], r)[tid - 256];
      s_lo[tid - 256] = (uint32_t)m, s_hi[tid - 256] = (uint32_t)(m >> 32);
    }
    ph ^= 1;
    __syncthreads();
  };
  auto bin_mass = [&](int bin) -> u64 { return ((u64)s_hi[bin] << 32) + s_lo[bin]; };
  auto find_bin = [&](bool mass, uint32_t want_c, u64 want_m) {
    if (warp == 0) {
      uint32_t c = 0;
      u64 m = 0;
      for (int j = 0; j < 8; ++j) {
        const int bin = 255 - (lane * 8 + j);
        c += s_cnt[bin];
        if (mass) m += bin_mass(bin);
      }
      uint32_t ci = c;
      u64 mi = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t cy = __shfl_up_sync(0xffffffffu, ci, o);
        const u64 my = __shfl_up_sync(0xffffffffu, mi, o);
        if (lane >= o) ci += cy, mi += my;
      }
      const bool hit = mass ? mi >= want_m : ci >= want_c;
      const unsigned bal = __ballot_sync(0xffffffffu, hit);
      const int src = bal ? __ffs(bal) - 1 : 31;
      if (lane == src) {
        uint32_t ac = ci - c;
        u64 am = mi - m;
        int bin = 255 - lane * 8;
        for (int j = 0; j < 8; ++j, --bin) {
          const uint32_t bc = s_cnt[bin];
          const u64 bm = mass ? bin_mass(bin) : 0;
          if ((mass ? am + bm >= want_m : ac + bc >= want_c) || j == 7) break;
          ac += bc, am += bm;
        }
        s_bin = bin, s_above_c = ac, s_above_m = am;
      }
    }
    __syncthreads();
  };

  // sum over the threads before this one (and over all, in total)
  auto block_scan = [&](u64 v, u64& total) -> u64 {
    u64 inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) s_red[warp] = inc;
    __syncthreads();
    u64 before = inc - v;
    total = 0;
    for (int w = 0; w < kWR; ++w) {
      if (w < warp) before += s_red[w];
      total += s_red[w];
    }
    return before;
  };
  const u64 wmin = m_in > 0.f ? (u64)ceil((double)fminf(m_in, 1.f) * __hiloint2double((1023 + sh) << 20, 0)) : 0;
  const u64 u64u = (u64)((double)u * 9223372036854775808.0) << 1;    // u in units of 2^-64
  const double Pd = fmax((double)P, 0.0);

  // The row's n tokens above kk or among the first `want` ties, at most kSmall: listed in id order in the
  // first CTA, which does the rest alone.
  auto finish_small = [&](uint32_t kk, uint32_t want, int n) {
    uint32_t gt, eq;
    counts_before(kk, gt, eq);
    uint2* list = cl.map_shared_rank(s_list, 0);
    for (int i0 = sa; i0 < se; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = skey(sZ[min(i, cnt - 1)]);
      const bool in = i < se;
      const unsigned bg = __ballot_sync(0xffffffffu, in && k > kk), be = __ballot_sync(0xffffffffu, in && k == kk);
      if (bg | be) {
        const unsigned lower = (1u << lane) - 1u;
        const uint32_t g = gt + __popc(bg & lower), e = eq + __popc(be & lower);
        if (((bg >> lane) & 1u) || (((be >> lane) & 1u) && e < want)) list[g + min(e, want)] = make_uint2(k, (uint32_t)(lo + i));
        gt += __popc(bg), eq += __popc(be);
      }
    }
    cl.sync();
    if (rank != 0) return;
    constexpr int kPer = kSmall / kTR;
    const int per = (n + kTR - 1) / kTR;
    uint32_t key[kPer], id[kPer];
    u64 w[kPer], mine = 0, Zk;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * per + j;
      const bool in = j < per && i < n;
      const uint2 x = s_list[in ? i : 0];
      key[j] = in ? x.x : 0u, id[j] = x.y;
      float z = key_value(key[j], T());
      if (inf_row) z = z == INFINITY ? 0.f : -INFINITY;
      w[j] = key[j] != 0u ? weigh(z) : 0;
      mine += w[j];
    }
    block_scan(mine, Zk);
    if (P < 1.f) {
      u64 left = (u64)ceil(Pd * (double)Zk);
      if (left < 1) left = 1;
      uint32_t prefix = 0, ties = 0;
      for (int shift = kBits - 8; shift >= 0; shift -= 8) {
        clear_hist();
        const uint32_t hm = shift + 8 >= 32 ? 0u : (0xffffffffu << (shift + 8));
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (w[j] && (key[j] & hm) == (prefix & hm)) {
            const int bin = (key[j] >> shift) & 0xffu;
            atomicAdd(&s_cnt[bin], 1u);
            add_mass(bin, w[j]);
          }
        __syncthreads();
        find_bin(true, 0, left);
        prefix |= (uint32_t)s_bin << shift;
        left -= min(left, s_above_m);
        ties = s_cnt[s_bin];
        __syncthreads();
      }
      const u64 wb = weigh(inf_row ? 0.f : key_value(prefix, T()));
      const u64 c = wb ? (left + wb - 1) / wb : ties;
      const u64 keep = max((u64)1, min(c, (u64)ties));
      u64 eqs = 0, all;
#pragma unroll
      for (int j = 0; j < kPer; ++j) eqs += w[j] && key[j] == prefix;
      u64 e = block_scan(eqs, all);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (key[j] < prefix) w[j] = 0;
        else if (w[j] && key[j] == prefix && e++ >= keep) w[j] = 0;
      }
    }
    mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (w[j] < wmin) w[j] = 0;
      mine += w[j];
    }
    u64 Z;
    u64 at = block_scan(mine, Z);
    const u64 thr = __umul64hi(u64u, Z);
    if (at <= thr && thr < at + mine) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (w[j] && at <= thr && thr < at + w[j]) {
          a.tokens[row] = (int)id[j];
          if (a.probs) a.probs[row] = (float)((double)w[j] / (double)Z);
        }
        at += w[j];
      }
    }
  };

  // ---------------------------------------------------------------- top-k: the k-th largest key
  if (topk || V <= kSmall) {
    uint32_t prefix = 0, want = (uint32_t)(topk ? k_in : V);
    for (int shift = kBits - 8; topk && shift >= 0; shift -= 8) {
      if (shift < kBits - 8) {     // (the first digit was counted with the load)
        clear_hist();
        const uint32_t hm = 0xffffffffu << (shift + 8);
        sweep([&](int i, bool in) {
          const uint32_t k = skey(sZ[i]);
          if (in && (k & hm) == (prefix & hm)) atomicAdd(&s_cnt[(k >> shift) & 0xffu], 1u);
        });
      }
      gather_hist(false);
      find_bin(false, want, 0);
      prefix |= (uint32_t)s_bin << shift;
      want -= s_above_c;
      if (shift > 0) __syncthreads();
    }
    if (!topk || k_in <= kSmall) {      // (a small vocabulary is such a list without a top-k)
      finish_small(prefix, want, topk ? k_in : V);
      return;
    }
    const uint32_t ties = s_cnt[prefix & 0xffu];
    __syncthreads();
    kth = prefix;
    tie_cut = want >= ties ? INT_MAX : resolve_ties(kth, want);
  }

  // ---------------------------------------------------------------- top-p: the border of the mass
  if (P < 1.f) {
    // Tokens are counted in kBins equal bins of (M - z) / T over 32 (2^-46 of the largest weight), bin 0 the
    // most likely, and the exact mass of all is taken.  A bin's mass lies between its count times the weights
    // of its ends, so the border lies in a window of few bins; a second level divides the window again when
    // it still holds many tokens.  Only what is left goes through the digits with its exact masses.
    const float bscale2 = (float)(2 * kBins / 32) / T_in;
    float off = 0.f, mul = 1.f, end = INFINITY;      // the current window: x in [off, end), kBins bins of 1 / mul
    // -1: above the window, kBins: below it.  (x is kept finite: a vocabulary masked with its type's lowest value
    // passes the largest float here, and the first window has to hold it, as every token, in its last bin.)
    auto bin_of = [&](float z) -> int {
      const float x = fminf(fmaf(z, -0.5f, weigh.Mh) * bscale2, 3.0e38f);
      return x < off ? -1 : (x < end ? (int)fminf((x - off) * mul, (float)(kBins - 1)) : kBins);
    };
    u64 sum = 0, Zk = 0, all = 0, want = 0;
    for (int level = 0; level < 2; ++level) {
      for (int i = tid; i < kBins; i += kTR) s_bins[i] = 0u;
      __syncthreads();
      if (level == 0) {
        sweep([&](int i, bool in) {
          const uint32_t k = skey(sZ[i]);
          const float z = value(i);
          const bool use = in && k != 0u && kept(k, i) && z > -INFINITY;
          const u64 w = weigh(z);                    // (not under the condition: the four chains interleave)
          sum += use ? w : 0;
          if (use) atomicAdd(&s_bins[bin_of(z)], 1u);
        });
        block_scan(sum, all);
        if (tid == 0) x_u[ph] = all;
      } else {
        sweep([&](int i, bool in) {
          const uint32_t k = skey(sZ[i]);
          const float z = value(i);
          const int bin = in && k != 0u && kept(k, i) && z > -INFINITY ? bin_of(z) : -1;
          if (bin >= 0 && bin < kBins) atomicAdd(&s_bins[bin], 1u);
        });
        __syncthreads();
      }
      cl.sync();
      if (level == 0) {
        for (int r = 0; r < cs; ++r) Zk += *cl.map_shared_rank(&x_u[ph], r);
        ph ^= 1;
        // a token is kept while the mass before it is < P * Zk: the border token is the first whose
        // inclusive mass reaches it
        want = (u64)ceil(Pd * (double)Zk);
        if (want < 1) want = 1;
      }
      constexpr int kPB = kBins / kTR;
      double lo_m[kPB], hi_m[kPB], lo_s = 0.0, hi_s = 0.0;
      uint32_t count[kPB];
      const double unit = __hiloint2double((1023 + sh) << 20, 0);
#pragma unroll
      for (int j = 0; j < kPB; ++j) {
        const int bin = tid * kPB + j;
        uint32_t c = 0;
        for (int r = 0; r < cs; ++r) c += cl.map_shared_rank(s_bins, r)[bin];
        count[j] = c;
        // the bin's ends in first-level bins, widened for the fp32 rounding of bin_of (at most 2^-13 of a
        // first-level bin), and a unit for the weights' own
        const double x0 = (double)off + (double)bin / (double)mul - 0.001, x1 = (double)off + (double)(bin + 1) / (double)mul + 0.001;
        const double w_hi = c ? exp(-x0 * (32.0 / kBins)) * unit + 1.0 : 0.0;
        const double w_lo = c && !(end == INFINITY && bin == kBins - 1) ? exp(-x1 * (32.0 / kBins)) * unit - 1.0 : 0.0;
        hi_s += (double)c * w_hi, lo_s += (double)c * fmax(w_lo, 0.0);
        hi_m[j] = hi_s, lo_m[j] = lo_s;
      }
      // inclusive sums over the bins before this thread's; then the first bin that can and the first that
      // must hold the border (sums of doubles, with a relative 1e-9 for their rounding)
      const double target = (double)want;
      double hb = hi_s, lb = lo_s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, hb, o), y = __shfl_up_sync(0xffffffffu, lb, o);
        if (lane >= o) hb += x, lb += y;
      }
      if (lane == 31) s_dsum[warp] = make_double2(hb, lb);
      if (tid == 0) s_win[0] = s_win[1] = kBins - 1;
      __syncthreads();
      hb -= hi_s, lb -= lo_s;
      for (int w = 0; w < warp; ++w) hb += s_dsum[w].x, lb += s_dsum[w].y;
#pragma unroll
      for (int j = 0; j < kPB; ++j) {
        if ((hb + hi_m[j]) * (1.0 + 1e-9) >= target) atomicMin(&s_win[0], tid * kPB + j);
        if ((lb + lo_m[j]) * (1.0 - 1e-9) >= target) atomicMin(&s_win[1], tid * kPB + j);
      }
      __syncthreads();
      // (a bin more on either side: the next level's edges are rounded)
      const int b_lo = max(min(s_win[0], s_win[1]) - level, 0), b_hi = min(max(s_win[0], s_win[1]) + level, kBins - 1);
      u64 inside = 0;
#pragma unroll
      for (int j = 0; j < kPB; ++j) inside += tid * kPB + j >= b_lo && tid * kPB + j <= b_hi ? count[j] : 0;
      block_scan(inside, all);
      inside = all;
      const float off0 = off;
      off = off0 + (float)b_lo / mul;
      if (b_hi < kBins - 1) end = off0 + (float)(b_hi + 1) / mul;
      mul = (float)kBins / ((float)(b_hi - b_lo + 1) / mul);
      // From here on only the tokens down to the window's end matter: each warp lists its own, unless they
      // are too many, and the sweeps that follow run over the lists.
      if (level == 0 && cnt <= 65536) {
        int n = 0;
        for (int i0 = sa; i0 < se; i0 += 128) {
          unsigned bal[4];
          bool use[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = i0 + 32 * j + lane, i = min(at, cnt - 1);
            const uint32_t k = skey(sZ[i]);
            const float z = value(i);
            use[j] = at < se && k != 0u && kept(k, i) && z > -INFINITY && bin_of(z) < kBins;
            bal[j] = __ballot_sync(0xffffffffu, use[j]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = n + __popc(bal[j] & ((1u << lane) - 1u));
            if (use[j] && at < kList) s_idx[warp][at] = (uint16_t)(i0 + 32 * j + lane);
            n += __popc(bal[j]);
          }
        }
        __syncwarp();
        if (n <= kList) listed = n;
      }
      // the exact mass above the window
      sum = 0;
      sweep([&](int i, bool in) {
        const uint32_t k = skey(sZ[i]);
        const float z = value(i);
        const u64 w = weigh(z);
        sum += in && k != 0u && kept(k, i) && z > -INFINITY && bin_of(z) < 0 ? w : 0;
      });
      block_scan(sum, all);
      if (tid == 0) x_u[ph] = all;
      cl.sync();
      u64 above = 0;
      for (int r = 0; r < cs; ++r) above += *cl.map_shared_rank(&x_u[ph], r);
      ph ^= 1;
      want = (u64)ceil(Pd * (double)Zk);
      want = want > above ? want - above : 1;
      __syncthreads();
      if (inside <= 4096) break;                     // (every CTA of the row has the same counts)
    }
    uint32_t prefix = 0;
    uint32_t ties = 0;
    for (int shift = kBits - 8; shift >= 0; shift -= 8) {
      clear_hist();
      const uint32_t hm = shift + 8 >= 32 ? 0u : (0xffffffffu << (shift + 8));
      sweep([&](int i, bool in) {
        const uint32_t k = skey(sZ[i]);
        if (!in || k == 0u || (k & hm) != (prefix & hm) || !kept(k, i)) return;
        const float z = value(i);
        if (!(z > -INFINITY)) return;
        const int zb = bin_of(z);
        if (zb < 0 || zb >= kBins) return;
        const int bin = (k >> shift) & 0xffu;
        atomicAdd(&s_cnt[bin], 1u);
        const u64 w = weigh(z);
        if (w) add_mass(bin, w);
      });
      gather_hist(true);
      find_bin(true, 0, want);
      prefix |= (uint32_t)s_bin << shift;
      want -= min(want, s_above_m);
      ties = s_cnt[s_bin];
      __syncthreads();
    }
    // tokens of the border key kept: the fewest whose mass reaches what is left
    const float zb = inf_row ? 0.f : key_value(prefix, T());
    const u64 wb = weigh(zb);
    const u64 c = wb ? (want + wb - 1) / wb : ties;
    const uint32_t keep = (uint32_t)max((u64)1, min(c, (u64)ties));
    const bool every = keep >= ties && prefix != kth;
    const int cut = every ? INT_MAX : (prefix == kth && keep >= ties ? tie_cut : resolve_ties(prefix, keep));
    kth = prefix;
    tie_cut = cut;
  }

  // ---------------------------------------------------------------- the draw
  auto mass_of = [&](int i, bool in) -> u64 {
    const uint32_t k = skey(sZ[i]);
    const u64 w = weigh(value(i));
    return in && k != 0u && kept(k, i) && w >= wmin ? w : 0;
  };
  u64 mine = 0;
  sweep([&](int i, bool in) { mine += mass_of(i, in); });
  mine = warp_sum_u64(mine);
  if (lane == 0) s_red[warp] = mine, s_listed[warp] = listed;
  __syncthreads();
  u64 total = 0;
  for (int w = 0; w < kWR; ++w) total += s_red[w];
  if (tid == 0) x_u[ph] = total;
  cl.sync();
  if (tid < cs) s_each[tid] = *cl.map_shared_rank(&x_u[ph], tid);
  __syncthreads();
  u64 Z = 0, base = 0;
  for (int r = 0; r < cs; ++r) {
    if (r < rank) base += s_each[r];
    Z += s_each[r];
  }
  // floor(u Z): a token's inclusive integer mass exceeds u Z iff it exceeds the floor
  const u64 thr = __umul64hi(u64u, Z);
  if (thr >= base && thr < base + total) {      // (the same verdict for the whole CTA)
    // the piece that holds the threshold, its tokens spread over all threads in order
    u64 before = base;
    int ow = 0;
    for (; ow < kWR - 1 && before + s_red[ow] <= thr; ++ow) before += s_red[ow];
    const int oa = min(cnt, ow * seg), ol = s_listed[ow], on = ol >= 0 ? ol : min(cnt, oa + seg) - oa;
    const int per = (on + kTR - 1) / kTR;
    const int ia = min(on, tid * per), ie = min(on, ia + per);
    auto token = [&](int n) -> int { return ol >= 0 ? (int)s_idx[ow][n] : oa + n; };
    u64 run = 0;
    for (int n = ia; n < ie; ++n) run += mass_of(token(n), true);
    u64 all;
    u64 at = before + block_scan(run, all);    // mass before this thread's tokens
    if (at <= thr && thr < at + run) {         // one thread of the cluster
      for (int n = ia; n < ie; ++n) {
        const u64 w = mass_of(token(n), true);
        at += w;
        if (at > thr) {
          a.tokens[row] = lo + token(n);
          if (a.probs) a.probs[row] = (float)((double)w / (double)Z);
          break;
        }
      }
    }
  }
  cl.sync();   // no CTA leaves while a peer may still read its shared memory
}

}  // namespace

namespace {
int slice_tokens(int V, int cs) { return ((V + cs - 1) / cs + 7) / 8 * 8; }
// CTAs per row: 8 unless they are more than two waves (two CTAs on each of 148 SMs), where fewer per row
// pay fewer barriers (512 rows of 16000: 8 / 2 per row 119 / 43 us; rows of unlike parameters, 64 of 128256,
// balance better with 8).  Two CTAs have to share an SM: of its 228 KB each has 47 KB of static variables and 1 KB of
// the system's, which leaves 66 KB for a slice (600 bf16 rows of 35328, one / two CTAs a row, which share an SM only
// as two: temperature alone 110 / 98 us, P 0.9 283 / 231 us; fp32 rows of 34304, two / four: 118 / 121, 348 / 327 us;
// at 65 KB a slice one CTA a row takes 90 and 202 us for bf16 rows of 33280).  A slice stays at least 4096 tokens.
constexpr size_t kSliceRoom = 66 * 1024;
int row_ctas(int R, int V, tsd_dtype dtype) {
  const size_t es = dtype == TSD_BF16 ? 2 : 4;
  int cs = kCS;
  while (cs > 1 && (size_t)slice_tokens(V, cs / 2) * es <= kSliceRoom && ((long long)R * cs > 4 * 148 || V / cs < 4096)) cs /= 2;
  return cs;
}
}  // namespace

size_t sample_rows_smem(int V, tsd_dtype dtype) { return (size_t)slice_tokens(V, kCS) * (dtype == TSD_BF16 ? 2 : 4); }

tsd_status launch_sample_rows(const SampleArgs& a_in, tsd_dtype dtype, cudaStream_t stream) {
  SampleArgs a = a_in;
  a.cs = row_ctas(a.R, a.V, dtype);
  a.slice = slice_tokens(a.V, a.cs);
  a.vec = vec16_rows(a.logits, a.V) ? 1 : 0;
  const size_t smem = (size_t)a.slice * (dtype == TSD_BF16 ? 2 : 4);
  auto kernel = dtype == TSD_BF16 ? sample_rows_kernel<__nv_bfloat16> : sample_rows_kernel<float>;
  if (allow_smem(kernel) != cudaSuccess)
    return TSD_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.R * a.cs);
  cfg.blockDim = dim3(kTR);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.cs, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return TSD_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
}

}  // namespace tsd
