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
// 512 contiguous bytes of codes.  The scale's byte, not its inverse, is carried to the rounding: 80 registers in
// bf16, three CTAs per SM (95 and two: 36 us for the prompts below).  Measured: 8 prompts of up to 4096 rows (8 heads of 128, bf16, pages of 16,
// 159 MB) 32 us, 4.9 TB/s; 8 x 2048 rows 17.6 us in bf16, 30.8 us in fp32 (5.4 TB/s); one token of 64 sequences 3.1 us
// and 64 paths of up to 7 rows 4.0 us, 4.0 and 4.6 us with the launch that advances; 8 x 8192 rows read back
// (317 MB) 59 us, 5.4 TB/s.
#include "kernels.h"
#include "q8.cuh"

namespace tsd {

namespace {

constexpr int kThreadsW = 256;
constexpr int kHold = 4;      // 16-element units a thread keeps in registers between the two steps

// 16 elements as they lie in memory (bf16: two 16-byte words, fp32: four).
template <typename T>
struct Unit {
  static constexpr int kWords = sizeof(T);
  uint4 w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void values(float (&x)[16]) const;
};
template <>
__device__ __forceinline__ void Unit<__nv_bfloat16>::values(float (&x)[16]) const {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t v[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[8 * h + 2 * i] = bf16_lo(v[i]), x[8 * h + 2 * i + 1] = bf16_hi(v[i]);
  }
}
template <>
__device__ __forceinline__ void Unit<float>::values(float (&x)[16]) const {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    x[4 * h] = __uint_as_float(w[h].x), x[4 * h + 1] = __uint_as_float(w[h].y);
    x[4 * h + 2] = __uint_as_float(w[h].z), x[4 * h + 3] = __uint_as_float(w[h].w);
  }
}
// Largest finite magnitude.
template <typename T>
__device__ __forceinline__ float amax_finite(const Unit<T>& u) {
  float x[16], m = 0.f;
  u.values(x);
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, q8::finite_abs(x[i]));
  return m;
}
template <typename T>
__device__ __forceinline__ float amax16(const Unit<T>& u) { return amax_finite(u); }
// bf16 magnitudes compare as integers, two at a time; a unit with an infinity or NaN (rare) is looked at again
template <>
__device__ __forceinline__ float amax16(const Unit<__nv_bfloat16>& u) {
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(u.w[h].x & 0x7fff7fffu, u.w[h].y & 0x7fff7fffu),
                             __vmaxu2(u.w[h].z & 0x7fff7fffu, u.w[h].w & 0x7fff7fffu)));
  const float r = __uint_as_float(max(m << 16, m & 0xffff0000u));
  return r < INFINITY ? r : amax_finite(u);
}
template <typename T>
__device__ __forceinline__ uint4 encode16(const Unit<T>& u, int byte) {
  const float inv = q8::inv_pow2_byte(byte);
  float x[16];
  u.values(x);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = q8::encode4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
  if (byte == q8::kByteMax)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = q8::saturate240(w[i]);
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
  const int bs = 1 << c.shift, d = c.d, upr = d / 16, ush = d == 128 ? 3 : 2;    // upr: 16-element units per row
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
      const int rel = p0 + r_lo + (u >> ush) - L;
      const int node = a.path ? a.path[(size_t)b * a.rows_max + rel] - 1 : rel;
      return src + (size_t)node * c.Hkv * d + (u & (upr - 1)) * 16;
    };
    Unit<T> x[kHold];
    float m = 0.f;
#pragma unroll
    for (int q = 0; q < kHold; ++q) {
      const int u = t + q * P;
      if (u < units) x[q].load(src_unit(u));
    }
#pragma unroll
    for (int q = 0; q < kHold; ++q)
      if (t + q * P < units) m = fmaxf(m, amax16(x[q]));
    for (int u = t + kHold * P; u < units; u += P) {
      Unit<T> y;
      y.load(src_unit(u));
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
      if (u < units) out[u] = encode16(x[q], byte);
    }
    for (int u = t + kHold * P; u < units; u += P) {
      Unit<T> y;
      y.load(src_unit(u));
      out[u] = encode16(y, byte);
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

// The codes behind 16 bytes of output (8 bf16 or 4 fp32), loaded and as values.
template <typename T>
struct Codes;
template <>
struct Codes<__nv_bfloat16> {
  uint2 c;
  __device__ __forceinline__ void load(const uint8_t* p) { c = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ uint4 values(float s) const {
    const uint2 a = q8::decode4_bf16(c.x, s), b = q8::decode4_bf16(c.y, s);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Codes<float> {
  uint32_t c;
  __device__ __forceinline__ void load(const uint8_t* p) { c = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ uint4 values(float s) const {
    const float2 a = q8::decode2(c), b = q8::decode2(c >> 16);
    return make_uint4(__float_as_uint(a.x * s), __float_as_uint(a.y * s), __float_as_uint(b.x * s), __float_as_uint(b.y * s));
  }
};

template <typename T>
__global__ void __launch_bounds__(256) q8_read_kernel(const Q8ReadArgs a) {
  pdl_trigger();
  pdl_wait();
  const Q8CacheArgs& c = a.c;
  const int b = blockIdx.y, d = c.d;
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
  // a thread takes kUnits pieces of 16 output bytes of K and of V a grid's width apart, all loads before any
  // store; neighbouring threads read and write neighbouring pieces
  constexpr int kUnits = 4, E = 16 / sizeof(T);
  const int psh = (d == 128 ? 7 : 6) - (E == 8 ? 3 : 2);                 // log2 of the pieces per row
  const uint32_t total = (uint32_t)min(max(n, 0), a.S) * c.Hkv;          // rows of a head (S * Hkv < 2^31)
  const long long pieces = (long long)total << psh, width = (long long)gridDim.x * blockDim.x;
  const size_t base = (size_t)b * a.S * c.Hkv * d;
  for (long long u0 = (long long)blockIdx.x * blockDim.x + threadIdx.x; u0 < pieces; u0 += kUnits * width) {
    Codes<T> kw[kUnits], vw[kUnits];
    int kb[kUnits], vb[kUnits];
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
      const long long u = u0 + q * width;
      kw[q].c = vw[q].c = {};
      kb[q] = vb[q] = 127;
      if (u < pieces && !zero) {
        const uint32_t rh = (uint32_t)(u >> psh), h = rh % (uint32_t)c.Hkv;
        const int pos = s0 + (int)(rh / (uint32_t)c.Hkv), ch = (int)(u & ((1 << psh) - 1));
        size_t row, sc;
        block_at(c, b, h, pos >> c.shift, row, sc);
        const size_t off = (row + (pos & ((1 << c.shift) - 1))) * d + ch * E;
        kw[q].load(c.k + off), vw[q].load(c.v + off);
        kb[q] = c.k_scale[sc], vb[q] = c.v_scale[sc];
      }
    }
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
      const long long u = u0 + q * width;
      if (u < pieces) {                                                  // pieces are in the output's order
        reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.k_out) + base)[u] = kw[q].values(q8::pow2_byte(q8::clean_byte(kb[q])));
        reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.v_out) + base)[u] = vw[q].values(q8::pow2_byte(q8::clean_byte(vb[q])));
      }
    }
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
  // about six CTAs per SM over the batch: a CTA checks its sequence once, then takes items in turn
  const long long most = (6 * 148 + a.B - 1) / a.B;
  long long gx = (items + per - 1) / per;
  if (gx > most) gx = most;
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
  const long long pieces = (long long)a.S * a.c.Hkv * a.c.d * (dtype == TSD_BF16 ? 2 : 4) / 16;
  // about eight CTAs per SM over the batch: a CTA checks its sequence's block ids once, so few large ones
  // beat many small ones
  const long long most = (8 * 148 + a.B - 1) / a.B;
  long long gx = (pieces + 255) / 256;
  if (gx > most) gx = most;
  const dim3 grid((unsigned)gx, a.B);
  const cudaError_t e = dtype == TSD_BF16 ? launch_pdl(q8_read_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, a)
                                          : launch_pdl(q8_read_kernel<float>, grid, dim3(256), 0, stream, a);
  return e == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
}

}  // namespace tsd
