// Pieces shared by the two tcgen05 attention kernels (attn_umma.cu: bf16 cache; attn_q8_umma.cu: 8-bit
// cache): softmax arithmetic, time-out flagging, the split merge inside the kernel, tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "attn_common.cuh"
#include "umma.cuh"

namespace tsd {
namespace attn {

constexpr int kD = 128;                      // head size of the tcgen05 kernels
constexpr uint32_t kStageF = kD * 4 + 16;    // staged fp32 split-partial row, padded over the banks
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x with the hardware approximation (flush-to-zero; 2^-inf = 0).  P is rounded to bf16 or f16 anyway.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// Paired fp32 arithmetic of sm_100 (one instruction for two lanes of work) and the three-input
// maximum: the lean full-tile softmax issues a third fewer instructions with them.
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n"
      ".reg .b64 ra, rb, rc, rd;\n"
      "mov.b64 ra, {%2, %3};\n"
      "mov.b64 rb, {%4, %5};\n"
      "mov.b64 rc, {%6, %7};\n"
      "fma.rn.f32x2 rd, ra, rb, rc;\n"
      "mov.b64 {%0, %1}, rd;\n"
      "}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n"
      ".reg .b64 ra, rb, rd;\n"
      "mov.b64 ra, {%2, %3};\n"
      "mov.b64 rb, {%4, %5};\n"
      "add.rn.f32x2 rd, ra, rb;\n"
      "mov.b64 {%0, %1}, rd;\n"
      "}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ void abort_cta(const AttnArgs& a, int b, volatile int* s_abort) {
  if (*s_abort == 0) {
    *s_abort = 1;
    flag_status(a.status, b, TSD_ERR_TIMEOUT);
  }
}

// Split merge inside the kernel.  Every CTA of a (sequence, KV head, row block) publishes its
// partial, then takes a ticket from the row block's word; the CTA that draws the last ticket merges
// the partials and writes the output, and returns the word to zero for the next call.  No CTA
// waits for another.  Returns 1 to the last CTA, 2 when the word held a count no call leaves
// behind (the workspace was not zeroed before its first use), else 0.
__device__ __forceinline__ int take_ticket(int* word, int splits, int* s_flag) {
  __threadfence();   // this thread's partial stores, before the ticket
  __syncthreads();
  if (threadIdx.x == 0) {
    const int old = atomicAdd(word, 1);
    const int r = old == splits - 1 ? 1 : ((old < 0 || old >= splits) ? 2 : 0);
    if (r == 1) atomicExch(word, 0);
    __threadfence();
    *s_flag = r;
  }
  __syncthreads();
  return *s_flag;
}

// The last CTA's merge (all threads).  (1) Every split's (max, sum) of every row into shared memory
// with independent loads; (2) per row the largest split maximum, the splits' weights
// 2^(M_s - M) / sum (s_w[s][row]) and the log-sum-exp; (3) every (row, 8 columns) the weighted sum
// of the partial rows, two such pieces per thread and two splits per round so that several loads are
// in flight, written as bf16.  This CTA's own partial is read from its staged rows in shared memory,
// the others' from L2 (.cg: written by other SMs); the sum goes by split index, whichever CTA came last, so
// that a call repeats itself bit for bit.  A split with no mass (M = -inf) has weight 0 and
// its rows are never read.  Zero rows when the sequence is flagged or out of capacity.  kKeepNan: a row
// whose sum is NaN comes out NaN (else zero).  pair, pairs: which of how many (sequence, KV head) pairs the
// partials are laid out for (-1: all of them, in order).
template <bool kKeepNan = false, typename Params>
__device__ void merge_splits(const AttnArgs& a, const Params& u, int b, int g, int G, int r0, int r_hi, int own,
                             bool zero, const uint8_t* sStage, float* s_w, int rows_cap, int pair = -1, int pairs = 0) {
  if (zero) {
    zero_rows<__nv_bfloat16>(a, b, g, G, r0, r_hi);
    return;
  }
  const int nrows = r_hi - r0, ns = u.splits, bd = blockDim.x;
  const float* wo = reinterpret_cast<const float*>(a.workspace);
  const float* wml = wo + (pair >= 0 ? (size_t)pairs : (size_t)a.B * a.Hkv) * ns * u.Rmax * kD;
  const size_t base = (pair >= 0 ? (size_t)pair : (size_t)b * a.Hkv + g) * ns * u.Rmax + r0;   // + s * Rmax + row
  float2* s_ml = reinterpret_cast<float2*>(s_w + ns * rows_cap);      // [s][row]
  const int npairs = ns * nrows;
  for (int i0 = threadIdx.x; i0 < npairs; i0 += 4 * bd) {
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int idx = i0 + j * bd, sp = idx / nrows, cr = idx - sp * nrows;
      if (idx < npairs) v[j] = __ldcg(reinterpret_cast<const float2*>(wml + (base + (size_t)sp * u.Rmax + cr) * 2));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int idx = i0 + j * bd, sp = idx / nrows, cr = idx - sp * nrows;
      if (idx < npairs) s_ml[sp * rows_cap + cr] = v[j];
    }
  }
  __syncthreads();
  for (int cr = threadIdx.x; cr < nrows; cr += bd) {
    float M = -INFINITY;
    for (int sp = 0; sp < ns; ++sp) M = fmaxf(M, s_ml[sp * rows_cap + cr].x);
    const float Mu = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    for (int sp = 0; sp < ns; ++sp) {
      const float2 ml = s_ml[sp * rows_cap + cr];
      const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - Mu);
      l += ml.y * w;
      s_w[sp * rows_cap + cr] = w;
    }
    const float inv = l > 0.f || (kKeepNan && l != 0.f) ? 1.f / l : 0.f;
    for (int sp = 0; sp < ns; ++sp) s_w[sp * rows_cap + cr] *= inv;
    if (a.lse) {
      const int r = r0 + cr;
      a.lse[((size_t)b * a.Nmax + r / G) * a.Hq + g * G + r % G] = (M + __log2f(l)) * kLn2;
    }
  }
  __syncthreads();
  const int ntask = nrows * (kD / 8);
  constexpr int kT = 2;   // pieces per thread per round (registers stay near the main loop's count)
  for (int t0 = threadIdx.x; t0 < ntask; t0 += kT * bd) {
    float acc[kT][8];
#pragma unroll
    for (int j = 0; j < kT; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[j][e] = 0.f;
    for (int s0 = 0; s0 < ns; s0 += 2) {
      float4 x[2][kT][2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int sp = s0 + q;
#pragma unroll
        for (int j = 0; j < kT; ++j) {
          const int t = t0 + j * bd, cr = t / (kD / 8), c8 = t % (kD / 8);
          if (sp < ns && sp != own && t < ntask) {
            const float4* p4 = reinterpret_cast<const float4*>(wo + (base + (size_t)sp * u.Rmax + cr) * kD + c8 * 8);
            x[q][j][0] = __ldcg(p4), x[q][j][1] = __ldcg(p4 + 1);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int sp = s0 + q;
#pragma unroll
        for (int j = 0; j < kT; ++j) {
          const int t = t0 + j * bd, cr = t / (kD / 8), c8 = t % (kD / 8);
          if (sp < ns && t < ntask) {
            const float w = s_w[sp * rows_cap + cr];
            if (w != 0.f) {
              float4 a0 = x[q][j][0], a1 = x[q][j][1];
              if (sp == own) {
                const float4* p4 = reinterpret_cast<const float4*>(sStage + (size_t)cr * kStageF + c8 * 32);
                a0 = p4[0], a1 = p4[1];
              }
              acc[j][0] = fmaf(w, a0.x, acc[j][0]), acc[j][1] = fmaf(w, a0.y, acc[j][1]);
              acc[j][2] = fmaf(w, a0.z, acc[j][2]), acc[j][3] = fmaf(w, a0.w, acc[j][3]);
              acc[j][4] = fmaf(w, a1.x, acc[j][4]), acc[j][5] = fmaf(w, a1.y, acc[j][5]);
              acc[j][6] = fmaf(w, a1.z, acc[j][6]), acc[j][7] = fmaf(w, a1.w, acc[j][7]);
            }
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kT; ++j) {
      const int t = t0 + j * bd, cr = t / (kD / 8), c8 = t % (kD / 8);
      if (t < ntask) {
        const int r = r0 + cr;
        __nv_bfloat16* orow = reinterpret_cast<__nv_bfloat16*>(a.out) +
                              (((size_t)b * a.Nmax + r / G) * a.Hq + g * G + r % G) * kD;
        *reinterpret_cast<uint4*>(orow + c8 * 8) =
            make_uint4(pack_bf16x2(acc[j][0], acc[j][1]), pack_bf16x2(acc[j][2], acc[j][3]),
                       pack_bf16x2(acc[j][4], acc[j][5]), pack_bf16x2(acc[j][6], acc[j][7]));
      }
    }
  }
}

// -------------------------------------------------------------------------------- host side
inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Tensor map with 128-byte swizzle; dims/box innermost first; strides in bytes for dims 1..
inline bool make_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box, CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  auto fn = encoder();
  if (!fn) return false;
  uint32_t es[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(m, type, rank, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace attn
}  // namespace tsd
