// tsd_kv_q8_append / tsd_kv_q8_commit / tsd_kv_q8_read: the 8-bit KV cache is quantised as it is
// written and read back as bf16 or fp32.
//
// A commit moves only the accepted path's rows ("EAGLE-Pangu", technical summary sec. 2, branchable
// KV cache); here they are quantised on the way.  For every block of tokens a call touches and every
// KV head, K and V apart:
//   k = the smallest exponent >= -40 with max|new rows| <= 448 * 2^k, and >= the block's own exponent
//       when the block already holds committed rows;
//   committed rows of the block: code <- rne(code * 2^(k_old - k)), only when k grew (an exponent
//       shift: exact above the subnormal step);   new rows: code <- rne(x * 2^-k).
//
// What bounds it: bytes (rows * Hkv * d * (es + 1) for K and for V).  One item = one (block, head, K
// or V); a warp (or a whole CTA for large blocks) holds the item's rows in registers between the
// maximum and the rounding, so the source is read once; a thread moves 16 elements, so a warp stores
// 512 contiguous bytes of codes.
#include "kernels.h"
#include "q8.cuh"

namespace tsd {

namespace {

constexpr int kThreadsW = 256;
constexpr int kHold = 4;      // 16-element units a thread keeps in registers between the two steps

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]);
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + h);
    x[8 * h] = bf16_lo(w.x), x[8 * h + 1] = bf16_hi(w.x), x[8 * h + 2] = bf16_lo(w.y), x[8 * h + 3] = bf16_hi(w.y);
    x[8 * h + 4] = bf16_lo(w.z), x[8 * h + 5] = bf16_hi(w.z), x[8 * h + 6] = bf16_lo(w.w), x[8 * h + 7] = bf16_hi(w.w);
  }
}
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const float4 w = __ldg(reinterpret_cast<const float4*>(p) + h);
    x[4 * h] = w.x, x[4 * h + 1] = w.y, x[4 * h + 2] = w.z, x[4 * h + 3] = w.w;
  }
}
__device__ __forceinline__ float amax16(const float (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, q8::finite_abs(x[i]));
  return m;
}
__device__ __forceinline__ uint4 encode16(const float (&x)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = q8::encode4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint32_t shift4(uint32_t w, float r) {
  const float2 a = q8::decode2(w), b = q8::decode2(w >> 16);
  return q8::encode4(a.x * r, a.y * r, b.x * r, b.y * r);
}

// First code of (sequence b, head h, logical block j) and the index of its scale byte.
__device__ __forceinline__ void block_at(const Q8CacheArgs& c, int b, int h, int j, size_t& row, size_t& sc) {
  if (c.block_table == nullptr) {
    row = ((size_t)b * c.Hkv + h) * c.Lcap + ((size_t)j << c.shift);
    sc = ((size_t)b * c.Hkv + h) * c.scale_cols + j;
  } else {
    const int blk = c.block_table[(size_t)b * c.max_blocks + j];
    row = ((size_t)blk * c.Hkv + h) << c.shift;
    sc = (size_t)blk * c.Hkv + h;
  }
}

// Rows a call writes to sequence b: n (0: nothing to do), or -1 after flagging status[b].  Every
// thread of the CTA calls it; all CTAs of a sequence reach the same verdict before any write.
__device__ int rows_to_write(const Q8WriteArgs& a, int b, int L) {
  const Q8CacheArgs& c = a.c;
  int n;
  if (a.accept_len != nullptr) {
    const int A = a.accept_len[b];
    if (A < 0) return 0;
    n = A + 1;
  } else {
    n = a.num_rows ? a.num_rows[b] : a.rows_max;
  }
  const int N = a.num_nodes ? a.num_nodes[b] : a.src_rows;
  int code = 0;
  if (n < 0 || n > a.rows_max || (a.accept_len != nullptr && (n > N || N > a.src_rows))) code = TSD_ERR_INVALID_ARG;
  else if (L < 0 || (long long)L + n > c.Lcap) code = TSD_ERR_CAPACITY;
  if (code == 0 && n > 0) {
    int bad = 0;
    if (a.path != nullptr)
      for (int j = threadIdx.x; j < n; j += blockDim.x) {
        const int s = a.path[(size_t)b * a.rows_max + j];
        bad |= s < 1 || s > N;
      }
    if (__syncthreads_or(bad)) code = TSD_ERR_INVALID_ARG;
    if (code == 0 && c.block_table != nullptr) {
      bad = 0;
      for (int j = (L >> c.shift) + threadIdx.x; j <= ((L + n - 1) >> c.shift); j += blockDim.x) {
        const int blk = c.block_table[(size_t)b * c.max_blocks + j];
        bad |= blk < 0 || blk >= c.num_blocks;
      }
      if (__syncthreads_or(bad)) code = TSD_ERR_CAPACITY;
    }
  }
  if (code != 0) {
    if (threadIdx.x == 0 && blockIdx.x == 0) flag_status(a.status, b, code);
    return -1;
  }
  return n;
}

// P threads work on one item: 32 (a warp) or the whole CTA.
template <typename T, int P>
__global__ void __launch_bounds__(kThreadsW) q8_write_kernel(const Q8WriteArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float s_max[kThreadsW / 32];
  const Q8CacheArgs& c = a.c;
  const int b = blockIdx.y;
  // one read for the CTA: another CTA may flag the sequence meanwhile (with this CTA's own verdict)
  __shared__ int s_st;
  if (threadIdx.x == 0) s_st = a.status[b];
  __syncthreads();
  if (s_st != 0) return;
  const int L = c.prefix_len[b];
  const int n = rows_to_write(a, b, L);
  if (n <= 0) return;
  const int bs = 1 << c.shift, d = c.d, upr = d / 16;    // upr: 16-element units per row
  const int j0 = L >> c.shift, nblk = ((L + n - 1) >> c.shift) - j0 + 1;
  const int items = nblk * c.Hkv * 2;
  const int t = threadIdx.x % P, sub = threadIdx.x / P;
  constexpr int kPer = kThreadsW / P;
  for (int it = blockIdx.x * kPer + sub; it < items; it += gridDim.x * kPer) {
    const int kv = it & 1, h = (it >> 1) % c.Hkv, j = j0 + (it >> 1) / c.Hkv;
    uint8_t* code = kv ? c.v : c.k;
    uint8_t* scale = kv ? c.v_scale : c.k_scale;
    const T* src = reinterpret_cast<const T*>(kv ? a.v_src : a.k_src) + (size_t)b * a.src_rows * c.Hkv * d + (size_t)h * d;
    size_t row0, sc;
    block_at(c, b, h, j, row0, sc);
    const int p0 = j << c.shift;
    const int r_lo = max(L - p0, 0), r_hi = min(L + n - p0, bs);     // new rows of this block
    const int units = (r_hi - r_lo) * upr;
    auto src_unit = [&](int u) -> const T* {
      const int rel = p0 + r_lo + u / upr - L;
      const int node = a.path ? a.path[(size_t)b * a.rows_max + rel] - 1 : rel;
      return src + (size_t)node * c.Hkv * d + (u % upr) * 16;
    };
    float x[kHold][16];
    float m = 0.f;
#pragma unroll
    for (int q = 0; q < kHold; ++q) {
      const int u = t + q * P;
      if (u < units) load16<T>(src_unit(u), x[q]);
    }
#pragma unroll
    for (int q = 0; q < kHold; ++q)
      if (t + q * P < units) m = fmaxf(m, amax16(x[q]));
    for (int u = t + kHold * P; u < units; u += P) {
      float y[16];
      load16<T>(src_unit(u), y);
      m = fmaxf(m, amax16(y));
    }
    m = warp_max(m);
    if (P > 32) {
      if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreadsW / 32; ++w) m = fmaxf(m, s_max[w]);
    }
    int byte = q8::scale_byte(m);
    int old = 0;
    if (r_lo > 0) {                     // committed rows share the block: its scale never shrinks
      old = q8::clean_byte(scale[sc]);
      byte = max(byte, old);
    }
    if (P > 32) __syncthreads();        // every thread has read the old byte and s_max
    else __syncwarp();
    const float inv = q8::inv_pow2_byte(byte);
    uint8_t* dst = code + row0 * d;
    if (r_lo > 0 && byte > old) {
      const float r = q8::pow2_byte(max(127 + old - byte, 1));
      for (int u = t; u < r_lo * upr; u += P) {
        uint4* p = reinterpret_cast<uint4*>(dst) + u;
        const uint4 w = *p;
        *p = make_uint4(shift4(w.x, r), shift4(w.y, r), shift4(w.z, r), shift4(w.w, r));
      }
    }
    uint4* out = reinterpret_cast<uint4*>(dst + (size_t)r_lo * d);
#pragma unroll
    for (int q = 0; q < kHold; ++q) {
      const int u = t + q * P;
      if (u < units) out[u] = encode16(x[q], inv);
    }
    for (int u = t + kHold * P; u < units; u += P) {
      float y[16];
      load16<T>(src_unit(u), y);
      out[u] = encode16(y, inv);
    }
    if (t == 0) scale[sc] = (uint8_t)byte;
  }
}

// prefix_len[b] += rows, once every row is written (a launch of its own: other CTAs of the write
// still read the old length while it runs).
__global__ void q8_advance_kernel(const Q8WriteArgs a) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= a.B || a.status[b] != 0) return;
  const int n = a.accept_len ? a.accept_len[b] + 1 : (a.num_rows ? a.num_rows[b] : a.rows_max);
  if (n > 0) a.c.prefix_len[b] += n;
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const uint4& w, float s);
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const uint4& w, float s) {
  const uint2 a = q8::decode4_bf16(w.x, s), b = q8::decode4_bf16(w.y, s);
  const uint2 c = q8::decode4_bf16(w.z, s), e = q8::decode4_bf16(w.w, s);
  reinterpret_cast<uint4*>(p)[0] = make_uint4(a.x, a.y, b.x, b.y);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(c.x, c.y, e.x, e.y);
}
template <>
__device__ __forceinline__ void store16<float>(float* p, const uint4& w, float s) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = q8::decode2(v[i]), b = q8::decode2(v[i] >> 16);
    reinterpret_cast<float4*>(p)[i] = make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
  }
}

// One thread per 16 elements of an output row (K and V together): consecutive threads read a head's
// row and write it contiguously.
template <typename T>
__global__ void __launch_bounds__(256) q8_read_kernel(const Q8ReadArgs a) {
  pdl_trigger();
  pdl_wait();
  const Q8CacheArgs& c = a.c;
  const int b = blockIdx.y, d = c.d, upr = d / 16;
  __shared__ int s_st;
  if (threadIdx.x == 0) s_st = a.status[b];
  __syncthreads();
  const int n = a.num_rows ? a.num_rows[b] : a.S;
  const int s0 = a.start ? a.start[b] : 0;
  int code = 0;
  if (n < 0 || n > a.S || s0 < 0) code = TSD_ERR_INVALID_ARG;
  else if ((long long)s0 + n > c.prefix_len[b] || (long long)s0 + n > c.Lcap) code = TSD_ERR_CAPACITY;
  else if (c.block_table != nullptr && n > 0) {
    int bad = 0;
    for (int j = (s0 >> c.shift) + threadIdx.x; j <= ((s0 + n - 1) >> c.shift); j += blockDim.x) {
      const int blk = c.block_table[(size_t)b * c.max_blocks + j];
      bad |= blk < 0 || blk >= c.num_blocks;
    }
    if (__syncthreads_or(bad)) code = TSD_ERR_CAPACITY;
  }
  if (code != 0 && s_st == 0 && blockIdx.x == 0 && threadIdx.x == 0) flag_status(a.status, b, code);
  const bool zero = code != 0 || s_st != 0;
  const long long total = (long long)min(max(n, 0), a.S) * c.Hkv * upr;
  for (long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x; u < total; u += (long long)gridDim.x * blockDim.x) {
    const int ch = (int)(u % upr), h = (int)(u / upr % c.Hkv), i = (int)(u / upr / c.Hkv);
    uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
    float ks = 1.f, vs = 1.f;
    if (!zero) {
      const int pos = s0 + i;
      size_t row, sc;
      block_at(c, b, h, pos >> c.shift, row, sc);
      const size_t off = (row + (pos & ((1 << c.shift) - 1))) * d + ch * 16;
      kw = __ldg(reinterpret_cast<const uint4*>(c.k + off));
      vw = __ldg(reinterpret_cast<const uint4*>(c.v + off));
      ks = q8::pow2_byte(q8::clean_byte(c.k_scale[sc])), vs = q8::pow2_byte(q8::clean_byte(c.v_scale[sc]));
    }
    const size_t o = (((size_t)b * a.S + i) * c.Hkv + h) * d + ch * 16;
    store16<T>(reinterpret_cast<T*>(a.k_out) + o, kw, ks);
    store16<T>(reinterpret_cast<T*>(a.v_out) + o, vw, vs);
  }
}

}  // namespace

tsd_status launch_q8_write(const Q8WriteArgs& a, tsd_dtype dtype, bool advance, cudaStream_t stream) {
  const int bs = 1 << a.c.shift;
  const long long nblk = ((long long)a.rows_max + bs - 2) / bs + 1;    // blocks rows_max rows can touch
  const long long items = nblk * a.c.Hkv * 2;
  // a warp holds an item of up to 4 * 32 * 16 elements (16 rows of 128); larger blocks take a CTA
  const bool warp = bs * a.c.d <= kHold * 32 * 16;
  const int per = warp ? kThreadsW / 32 : 1;
  long long gx = (items + per - 1) / per;
  if (gx > 0x7fffffffLL) gx = 0x7fffffffLL;
  const dim3 grid((unsigned)gx, a.B);
  cudaError_t e;
  if (dtype == TSD_BF16)
    e = warp ? launch_pdl(q8_write_kernel<__nv_bfloat16, 32>, grid, dim3(kThreadsW), 0, stream, a)
             : launch_pdl(q8_write_kernel<__nv_bfloat16, kThreadsW>, grid, dim3(kThreadsW), 0, stream, a);
  else
    e = warp ? launch_pdl(q8_write_kernel<float, 32>, grid, dim3(kThreadsW), 0, stream, a)
             : launch_pdl(q8_write_kernel<float, kThreadsW>, grid, dim3(kThreadsW), 0, stream, a);
  if (e != cudaSuccess) return TSD_ERR_CUDA;
  if (advance && launch_pdl(q8_advance_kernel, dim3((a.B + 127) / 128), dim3(128), 0, stream, a) != cudaSuccess)
    return TSD_ERR_CUDA;
  return TSD_OK;
}

tsd_status launch_q8_read(const Q8ReadArgs& a, tsd_dtype dtype, cudaStream_t stream) {
  const long long units = (long long)a.S * a.c.Hkv * (a.c.d / 16);
  long long gx = (units + 255) / 256;
  if (gx > 65535) gx = 65535;
  const dim3 grid((unsigned)gx, a.B);
  const cudaError_t e = dtype == TSD_BF16 ? launch_pdl(q8_read_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, a)
                                          : launch_pdl(q8_read_kernel<float>, grid, dim3(256), 0, stream, a);
  return e == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
}

}  // namespace tsd
