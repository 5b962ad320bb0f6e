// Tree-verify attention over the 8-bit cache with fp32 queries (FFMA; the fp32 tolerance excludes the tensor
// cores' formats).  Operation, decomposition and split partials are those of attn_f32_kernel (attn.cu): a
// CTA has 16 query rows of one KV head, four per warp, and a range of 32-key tiles.
//
// What bounds it: the FMA pipes (4 d operations per row and key) for many rows, the latency of its tiles for
// few.  A tile's codes (16 per thread and load, with one block-table look-up) are fetched into registers
// while the tile before is computed.  Scores: lane = key, the four rows of a warp share every K load and read
// their queries as broadcasts; P V: lane = columns, the rows share every V load and read P as broadcasts.
// (3 sequences of 7 nodes, 12/4 heads of 64, prefixes up to 777: 62 us with one element per load and
// look-up, 20 us so, 15.7 us with its splits planned for four CTAs per SM.)
#include "attn_common.cuh"
#include "common.cuh"
#include "kernels.h"
#include "q8.cuh"

namespace tsd {

namespace {

using namespace attn;

constexpr int kBN = 32, kBM = 16, kRPW = 4, kThreadsF = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
  static constexpr int LD = D + 4;      // row stride: 16-byte rows, no bank conflict between neighbours
  float q[kBM][D];
  float k[kBN][LD];
  float v[kBN][LD];
  float p[kThreadsF / 32][kRPW][kBN];
};

template <int D>
__global__ void __launch_bounds__(kThreadsF)
    attn_q8_f32_kernel(const AttnArgs a, int mtiles, int tps, int splits, int Rmax) {
  pdl_trigger();
  pdl_wait();
  constexpr int E = D / 32, CH = D / 16, NC = kBN * CH / kThreadsF;   // columns per lane, chunks per row, per thread
  extern __shared__ __align__(128) uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  uint32_t* sMask = reinterpret_cast<uint32_t*>(raw + sizeof(Smem<D>));
  __shared__ int s_err, s_status, s_poison;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mt = blockIdx.x % mtiles, split = blockIdx.x / mtiles;
  const int g = blockIdx.y, b = blockIdx.z;
  const int G = a.Hq / a.Hkv;
  if (tid == 0) s_err = s_poison = 0, s_status = __ldcg(a.status + b);
  SeqView v = seq_view(a, b, G, kBN, tps);
  __syncthreads();
  v.zero = v.cap || s_status != 0;       // one read of the status word for the CTA
  const int r0 = mt * kBM;
  if (v.skip || r0 >= v.R) return;
  const int r_hi = min(r0 + kBM, v.R);
  if (v.zero) {
    if (split == 0) zero_rows<float>(a, b, g, G, r0, r_hi);
    if (split == 0 && mt == 0 && g == 0 && tid == 0 && s_status == 0) flag_status(a.status, b, TSD_ERR_CAPACITY);
    return;
  }
  if (split >= v.nsplit) return;
  const bool direct = v.nsplit == 1;
  const int t_begin = split * tps, t_end = min(v.T, t_begin + tps);
  const int W = (a.Nmax + 31) >> 5;
  const int i_lo = r0 / G, i_cnt = (r_hi - 1) / G - i_lo + 1;
  const uint8_t* kc = reinterpret_cast<const uint8_t*>(a.k_cache);
  const uint8_t* vc = reinterpret_cast<const uint8_t*>(a.v_cache);

  // codes and scales of a prefix tile into registers
  uint4 ck[NC], cv[NC];
  int bk[NC], bv[NC];
  auto fetch = [&](int t) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = tid + j * kThreadsF, pos = t * kBN + c / CH;
      ck[j] = cv[j] = make_uint4(0, 0, 0, 0);
      bk[j] = bv[j] = 127;
      if (t < v.nPT && t < t_end && pos < v.L) {
        bool ok = true;
        const size_t off = cache_row(a, b, g, pos, ok) + (c % CH) * 16, sc = scale_at(a, b, g, pos);
        if (!ok) {
          s_err = 1;
        } else {
          ck[j] = *reinterpret_cast<const uint4*>(kc + off), cv[j] = *reinterpret_cast<const uint4*>(vc + off);
          bk[j] = a.k_scale[sc], bv[j] = a.v_scale[sc];
        }
      }
    }
  };
  fetch(t_begin);
  const float* q = reinterpret_cast<const float*>(a.q);
  for (int idx = tid; idx < kBM * (D / 4); idx += kThreadsF) {
    const int row = idx / (D / 4), c = idx % (D / 4), r = r0 + row;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < v.R) x = reinterpret_cast<const float4*>(q + (((size_t)b * a.Nmax + r / G) * a.Hq + g * G + r % G) * D)[c];
    reinterpret_cast<float4*>(sm.q[row])[c] = x;
  }
  if (t_end > v.nPT) build_mask(a, b, i_lo, i_cnt, W, sMask, v.N);
  const float sl2 = a.scale * kLog2e;
  float m[kRPW], l[kRPW], o[kRPW][E];
#pragma unroll
  for (int rr = 0; rr < kRPW; ++rr) {
    m[rr] = -INFINITY, l[rr] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[rr][e] = 0.f;
  }
  const int lr0 = warp * kRPW;
  const bool warp_on = r0 + lr0 < r_hi;
  for (int t = t_begin; t < t_end; ++t) {
    const bool tree = t >= v.nPT;
    __syncthreads();                     // the tile before has been read
    if (!tree) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = tid + j * kThreadsF, row = c / CH, col = (c % CH) * 16;
        const float sk = q8::pow2_byte(q8::clean_byte(bk[j])), sv = q8::pow2_byte(q8::clean_byte(bv[j]));
        const uint32_t wk[4] = {ck[j].x, ck[j].y, ck[j].z, ck[j].w}, wv[4] = {cv[j].x, cv[j].y, cv[j].z, cv[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 k0 = q8::decode2(wk[i]), k1 = q8::decode2(wk[i] >> 16);
          const float2 v0 = q8::decode2(wv[i]), v1 = q8::decode2(wv[i] >> 16);
          reinterpret_cast<float4*>(&sm.k[row][col])[i] = make_float4(k0.x * sk, k0.y * sk, k1.x * sk, k1.y * sk);
          reinterpret_cast<float4*>(&sm.v[row][col])[i] = make_float4(v0.x * sv, v0.y * sv, v1.x * sv, v1.y * sv);
        }
      }
      fetch(t + 1);
    } else {
      for (int c = tid; c < kBN * (D / 4); c += kThreadsF) {
        const int row = c / (D / 4), col = c % (D / 4), j = (t - v.nPT) * kBN + row;
        float4 xk = make_float4(0.f, 0.f, 0.f, 0.f), xv = xk;
        if (j < v.N) {
          const size_t off = (((size_t)b * a.Nmax + j) * a.Hkv + g) * D;
          xk = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.k_tree) + off)[col];
          xv = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.v_tree) + off)[col];
        }
        reinterpret_cast<float4*>(sm.k[row])[col] = xk;
        auto finite = [&](float x) -> float {   // (visible_nonfinite adds the others)
          if (fabsf(x) < INFINITY) return x;
          s_poison = 1;
          return 0.f;
        };
        reinterpret_cast<float4*>(sm.v[row])[col] = make_float4(finite(xv.x), finite(xv.y), finite(xv.z), finite(xv.w));
      }
    }
    __syncthreads();
    if (!warp_on) continue;
    const int kbase = tree ? (t - v.nPT) * kBN : t * kBN;
    const bool key_in = kbase + lane < (tree ? v.N : v.L);
    float s[kRPW] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < D / 4; ++c) {
      const float4 k4 = reinterpret_cast<const float4*>(sm.k[lane])[c];
#pragma unroll
      for (int rr = 0; rr < kRPW; ++rr) {
        const float4 q4 = reinterpret_cast<const float4*>(sm.q[lr0 + rr])[c];
        s[rr] = fmaf(q4.x, k4.x, s[rr]), s[rr] = fmaf(q4.y, k4.y, s[rr]);
        s[rr] = fmaf(q4.z, k4.z, s[rr]), s[rr] = fmaf(q4.w, k4.w, s[rr]);
      }
    }
#pragma unroll
    for (int rr = 0; rr < kRPW; ++rr) {
      const int r = r0 + lr0 + rr;
      bool valid = key_in && r < r_hi;
      if (tree && valid) {
        const int node = r / G - i_lo, j = kbase + lane;
        valid = (sMask[node * W + (j >> 5)] >> (j & 31)) & 1u;
      }
      const float x = valid ? s[rr] * sl2 : -INFINITY;
      const float nm = fmaxf(m[rr], warp_max(x));
      const float use = nm == -INFINITY ? 0.f : nm;
      const float al = exp2f(m[rr] - use), p = exp2f(x - use);
      l[rr] = l[rr] * al + warp_sum(p);
      m[rr] = nm;
#pragma unroll
      for (int e = 0; e < E; ++e) o[rr][e] *= al;
      sm.p[warp][rr][lane] = p;
    }
    __syncwarp();
#pragma unroll 2
    for (int k4 = 0; k4 < kBN / 4; ++k4) {
      float vv[4][E];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if constexpr (E == 2) {
          const float2 x = reinterpret_cast<const float2*>(sm.v[4 * k4 + kk])[lane];
          vv[kk][0] = x.x, vv[kk][1] = x.y;
        } else {
          const float4 x = reinterpret_cast<const float4*>(sm.v[4 * k4 + kk])[lane];
          vv[kk][0] = x.x, vv[kk][1] = x.y, vv[kk][2] = x.z, vv[kk][3] = x.w;
        }
      }
#pragma unroll
      for (int rr = 0; rr < kRPW; ++rr) {
        const float4 p = reinterpret_cast<const float4*>(sm.p[warp][rr])[k4];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          o[rr][e] = fmaf(p.x, vv[0][e], o[rr][e]), o[rr][e] = fmaf(p.y, vv[1][e], o[rr][e]);
          o[rr][e] = fmaf(p.z, vv[2][e], o[rr][e]), o[rr][e] = fmaf(p.w, vv[3][e], o[rr][e]);
        }
      }
    }
    __syncwarp();
  }
  __syncthreads();
  const bool err = s_err != 0;
  if (err && tid == 0) flag_status(a.status, b, TSD_ERR_CAPACITY);
#pragma unroll
  for (int rr = 0; rr < kRPW; ++rr) {
    const int r = r0 + lr0 + rr;
    if (r >= r_hi) continue;
    if (s_poison != 0) {
      const uint32_t* bits = sMask + (size_t)(r / G - i_lo) * W;
      const int n0 = max(t_begin - v.nPT, 0) * kBN, n1 = min(v.N, max(t_end - v.nPT, 0) * kBN);
#pragma unroll
      for (int e = 0; e < E; ++e) o[rr][e] += visible_nonfinite<float>(a, b, g, bits, n0, n1, lane * E + e);
    }
    const size_t orow = ((size_t)b * a.Nmax + r / G) * a.Hq + g * G + r % G;
    const size_t prow = (((size_t)b * a.Hkv + g) * splits + split) * Rmax + r;
    float* wo = reinterpret_cast<float*>(a.workspace);
    float* dst = direct ? reinterpret_cast<float*>(a.out) + orow * D : wo + prow * D;
    const float w = direct ? ((l[rr] == 0.f || err) ? 0.f : 1.f / l[rr]) : 1.f;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[lane * E + e] = direct && err ? 0.f : o[rr][e] * w;
    if (lane == 0) {
      if (!direct) *reinterpret_cast<float2*>(wo + (size_t)a.B * a.Hkv * splits * Rmax * D + prow * 2) =
          make_float2(l[rr] != 0.f && m[rr] == -INFINITY ? 0.f : m[rr], l[rr]);   // (a NaN sum is merged, not skipped)
      else if (a.lse) a.lse[orow] = err ? 0.f : (m[rr] + __log2f(l[rr])) * kLn2;
    }
  }
}

}  // namespace

tsd_status launch_attention_q8_f32(const AttnArgs& a, const AttnPlan& p, cudaStream_t stream) {
  const int W = (a.Nmax + 31) / 32;
  const size_t mask = (size_t)(kBM / p.G + 2) * W * 4;
  const dim3 grid(p.mtiles * p.splits, a.Hkv, a.B);
  const size_t smem = (a.d == 128 ? sizeof(Smem<128>) : sizeof(Smem<64>)) + mask;
  auto kernel = a.d == 128 ? attn_q8_f32_kernel<128> : attn_q8_f32_kernel<64>;
  allow_smem(kernel);
  return launch_pdl(kernel, grid, dim3(kThreadsF), smem, stream, a, p.mtiles, p.tps, p.splits, p.Rmax) == cudaSuccess
             ? TSD_OK : TSD_ERR_CUDA;
}

}  // namespace tsd
