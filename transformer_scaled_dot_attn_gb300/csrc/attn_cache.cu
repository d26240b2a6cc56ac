// Writing new keys and values into a decoding cache, quantised as they are
// written, and reading a quantised cache back.
//
// A quantised row (one position of one head) is d e4m3 codes and one exponent
// byte: e is the least integer with max|x| <= 448 2^e (448 is e4m3's largest
// value), kept in [-117, 119], and 0 for a row of zeros; code = x 2^-e rounded
// to e4m3 (nearest even, saturating); byte = e + 127. A power of two as the
// scale costs a floating-point code no precision (every code keeps its four
// significant bits; at most one of e4m3's fifteen binades is given away) and
// makes both directions exact but for the one rounding to e4m3: the division is
// exact, and code 2^e is a bf16 number, so reading back rounds nothing.
//
// Both kernels stream each byte once (HBM bound). A thread owns 16 columns of
// one row of K and the same of V, so that a step's few rows spread over many
// SMs; the row maximum takes log2(d / 16) shuffles. Its columns are two chunks of
// eight half a row apart, so that every access of a warp takes whole 32-byte sectors:
// reading 16 caches of 4096, 16 heads, d = 128, takes 105 us (the copy bandwidth gives
// 104), and took 130 with the chunks side by side. Writing 16 prompts of up to 1000: 24
// us (22).
#include "attn_kernels.cuh"

namespace attn {
namespace {

using namespace sm103;

constexpr int kCacheThreads = 128;  // (256: one step's new rows 2.3 us instead of 2.1)

struct Row16 {
  uint4 a, b;  // 8 bf16 each, half a row apart
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Largest finite |x| of the 16 values, as bf16 bits (0 when there is none). Magnitudes
// are ordered as their bits are, so two at a time are compared as 16-bit integers; only
// a row with infinities or NaN among them is looked at value by value.
__device__ __forceinline__ uint32_t finite_max(const Row16& r) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  uint32_t two = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) two = max_u16x2(two, w[i] & 0x7fff7fffu);
  uint32_t m = max(two & 0xffffu, two >> 16);
  if (m >= 0x7f80u) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
      m = max(m, lo < 0x7f80u ? lo : 0u);
      m = max(m, hi < 0x7f80u ? hi : 0u);
    }
  }
  return m;
}

// The scale exponent of a row whose largest finite magnitude has these bf16
// bits: 448 = 1.75 2^8, so e = exponent - 8, one more where the significand
// is above 1.75 (its 7 stored bits above 0x60).
__device__ __forceinline__ int scale_exponent(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = static_cast<int>(amax >> 7) - 127 - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0);
  return min(max(e, -117), 119);
}

__device__ __forceinline__ uint16_t quantise2(uint32_t two, uint64_t inv) {
  const float2 x = unpack_bf16x2(two);
  float lo, hi;
  f2_unpack(mul2(f2_pack(x.x, x.y), inv), lo, hi);
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t quantise4(uint32_t lo, uint32_t hi, uint64_t inv) {
  const uint16_t a = quantise2(lo, inv), b = quantise2(hi, inv);
  return static_cast<uint32_t>(a) | (static_cast<uint32_t>(b) << 16);
}

template <int D>
__device__ __forceinline__ void write_row(const Row16& r, unsigned char* cache, unsigned char* exps, size_t row,
                                          int tau, bool live) {
  constexpr int T = D / 16;
  uint32_t m = finite_max(r);
#pragma unroll
  for (int o = T / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int e = scale_exponent(m);
  const float back = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, a normal number
  const uint64_t inv = f2_pack(back, back);
  if (!live) return;
  unsigned char* dst = cache + row * D + tau * 8;
  *reinterpret_cast<uint2*>(dst) = make_uint2(quantise4(r.a.x, r.a.y, inv), quantise4(r.a.z, r.a.w, inv));
  *reinterpret_cast<uint2*>(dst + D / 2) = make_uint2(quantise4(r.b.x, r.b.y, inv), quantise4(r.b.z, r.b.w, inv));
  if (tau == 0) exps[row] = static_cast<unsigned char>(e + 127);
}

// New row i of sequence b goes to position L_b - new_b + i; rows past new_b and
// positions outside the cache are left alone.
template <int D, bool QUANT>
__global__ void __launch_bounds__(kCacheThreads) attn_cache_write_kernel(const CacheParams p) {
  constexpr int T = D / 16;
  grid_follow();
  const int tau = threadIdx.x % T;
  const unsigned long long row64 = static_cast<unsigned long long>(blockIdx.x) * (kCacheThreads / T) + threadIdx.x / T;
  bool live = row64 < p.rows;
  const unsigned row = live ? static_cast<unsigned>(row64) : 0u, n = p.n;
  const unsigned bg = row / n, b = bg / static_cast<unsigned>(p.h_kv);
  const int i = static_cast<int>(row - bg * n);
  const int L = p.kv_len == nullptr ? p.m : min(max(__ldg(p.kv_len + b), 0), p.m);
  const int nn = p.new_len == nullptr ? p.n : min(max(__ldg(p.new_len + b), 0), p.n);
  const int at = L - nn + i;
  live = live && i < nn && at >= 0;  // at < L <= m since i < nn
  Row16 k = {}, v = {};
  if (live) {
    const size_t src = static_cast<size_t>(row) * D + tau * 8;
    k.a = *reinterpret_cast<const uint4*>(p.k + src);
    k.b = *reinterpret_cast<const uint4*>(p.k + src + D / 2);
    v.a = *reinterpret_cast<const uint4*>(p.v + src);
    v.b = *reinterpret_cast<const uint4*>(p.v + src + D / 2);
  }
  const size_t dst = static_cast<size_t>(bg) * p.m + (live ? at : 0);
  if constexpr (QUANT) {
    write_row<D>(k, static_cast<unsigned char*>(p.k_cache), p.k_exp, dst, tau, live);
    write_row<D>(v, static_cast<unsigned char*>(p.v_cache), p.v_exp, dst, tau, live);
  } else if (live) {
    __nv_bfloat16* kc = static_cast<__nv_bfloat16*>(p.k_cache) + dst * D + tau * 8;
    __nv_bfloat16* vc = static_cast<__nv_bfloat16*>(p.v_cache) + dst * D + tau * 8;
    *reinterpret_cast<uint4*>(kc) = k.a;
    *reinterpret_cast<uint4*>(kc + D / 2) = k.b;
    *reinterpret_cast<uint4*>(vc) = v.a;
    *reinterpret_cast<uint4*>(vc + D / 2) = v.b;
  }
}

// Two codes times 2^e as a bf16 pair (exact: see above).
__device__ __forceinline__ uint32_t dequantise2(uint32_t two, float scale) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(two)));
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h2));
  return pack_bf16x2(lo * scale, hi * scale);
}

template <int D>
__device__ __forceinline__ void read_row(const unsigned char* cache, const unsigned char* exps, __nv_bfloat16* out,
                                         size_t row, size_t at, bool real) {
  uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
  if (real) {
    const uint2 c = __ldg(reinterpret_cast<const uint2*>(cache + at));
    const uint2 e = __ldg(reinterpret_cast<const uint2*>(cache + at + D / 2));
    const int byte = __ldg(exps + row);
    // 2^(byte - 127); byte 0 is 2^-127, a subnormal number; 255 (never written) reads as infinity
    const float s = byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(byte) << 23);
    lo = make_uint4(dequantise2(c.x & 0xffffu, s), dequantise2(c.x >> 16, s), dequantise2(c.y & 0xffffu, s),
                    dequantise2(c.y >> 16, s));
    hi = make_uint4(dequantise2(e.x & 0xffffu, s), dequantise2(e.x >> 16, s), dequantise2(e.y & 0xffffu, s),
                    dequantise2(e.y >> 16, s));
  }
  *reinterpret_cast<uint4*>(out + at) = lo;
  *reinterpret_cast<uint4*>(out + at + D / 2) = hi;
}

// Rows at or past the sequence's length come back as zeros (their cache bytes are not read).
template <int D>
__global__ void __launch_bounds__(kCacheThreads) attn_cache_read_kernel(const CacheParams p) {
  constexpr int T = D / 16;
  grid_follow();
  const int tau = threadIdx.x % T;
  const unsigned long long row64 = static_cast<unsigned long long>(blockIdx.x) * (kCacheThreads / T) + threadIdx.x / T;
  if (row64 >= p.rows) return;
  const unsigned row = static_cast<unsigned>(row64), m = p.m, bg = row / m;
  const int j = static_cast<int>(row - bg * m);
  const int L = p.kv_len == nullptr ? p.m : __ldg(p.kv_len + bg / static_cast<unsigned>(p.h_kv));
  const size_t at = static_cast<size_t>(row) * D + tau * 8;
  read_row<D>(static_cast<const unsigned char*>(p.k_cache), p.k_exp, p.k_out, row, at, j < L);
  read_row<D>(static_cast<const unsigned char*>(p.v_cache), p.v_exp, p.v_out, row, at, j < L);
}

template <int D>
cudaError_t launch_write_d(bool quantised, const CacheParams& p, cudaStream_t stream) {
  constexpr int RB = kCacheThreads / (D / 16);
  const unsigned blocks = static_cast<unsigned>((p.rows + RB - 1) / RB);
  prof_begin(kKindCache, stream);
  const auto kernel = quantised ? attn_cache_write_kernel<D, true> : attn_cache_write_kernel<D, false>;
  const cudaError_t e = launch_dependent(kernel, dim3(blocks), dim3(kCacheThreads), 0, stream, p);
  prof_end(kKindCache, stream);
  return e;
}

template <int D>
cudaError_t launch_read_d(const CacheParams& p, cudaStream_t stream) {
  constexpr int RB = kCacheThreads / (D / 16);
  prof_begin(kKindCache, stream);
  const dim3 grid(static_cast<unsigned>((p.rows + RB - 1) / RB));
  const cudaError_t e = launch_dependent(attn_cache_read_kernel<D>, grid, dim3(kCacheThreads), 0, stream, p);
  prof_end(kKindCache, stream);
  return e;
}

}  // namespace

cudaError_t launch_cache_write(int d, bool quantised, const CacheParams& p, cudaStream_t stream) {
  switch (d) {
    case 32: return launch_write_d<32>(quantised, p, stream);
    case 64: return launch_write_d<64>(quantised, p, stream);
    case 128: return launch_write_d<128>(quantised, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_cache_read(int d, const CacheParams& p, cudaStream_t stream) {
  switch (d) {
    case 32: return launch_read_d<32>(p, stream);
    case 64: return launch_read_d<64>(p, stream);
    case 128: return launch_read_d<128>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
