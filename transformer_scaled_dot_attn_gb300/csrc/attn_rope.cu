// Per-head RMS norm of queries and keys and the rotation by their positions,
// in one pass between the QKV projection and the attention:
//
//   r = (mean_c x_c^2 + eps)^(-1/2),   y_c = x_c r w_c,
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_a sin t + y_b cos t),  t = position * frequency,
//
// for each of the rot/2 column pairs (a, b) of the head's first rot columns.
// Backward: u = the upstream gradient turned by -t,
//   dx = r (w u - x r mean(w u x r)),   dw_c = sum over rows of u_c x_c r_c.
//
// Both directions are bound by HBM (each element is read and written once).
// A thread owns 16 columns of a row as two 16-byte chunks that hold whole
// column pairs, so the rotation needs no exchange between threads; d / 16
// neighbouring lanes make a row, and the row sums take log2(d / 16) shuffles.
// It keeps one token and loops over a chunk of its heads: the angles (position
// reduction, sin, cos) are computed once per token and head chunk.
#include "attn_kernels.cuh"

namespace attn {
namespace {

using namespace sm103;

constexpr int kNrThreads = 256;

// The fixed-point turn rate of a frequency: frequency / (2 pi) turns per
// position in units of 2^-64 turn, modulo one turn. The frequency is M 2^e
// with a 24-bit M, and M times floor(2^66 / (2 pi)) shifted by 2 - e is exact to
// a unit, so a position p (|p| < 2^31) times the rate wraps by itself and
// leaves the angle's fraction of a turn to 2^-32: a far position needs no
// 64-bit floating point.
__device__ __forceinline__ unsigned long long turn_rate(float f) {
  const unsigned int b = __float_as_uint(f);
  const int ex = static_cast<int>((b >> 23) & 0xff);
  if (ex == 0 || ex == 0xff) return 0ull;  // zero (and subnormal) frequencies turn nothing; not finite: no turn
  const unsigned long long m = (b & 0x7fffffu) | 0x800000u;
  const unsigned long long inv2pi = 0xA2F9836E4E441529ull;  // floor(2^66 / (2 pi))
  const unsigned long long lo = m * inv2pi, hi = __umul64hi(m, inv2pi);
  const int s = 2 - (ex - 150);  // right shift of the 128-bit product (f = m 2^(ex - 150))
  unsigned long long r;
  if (s >= 128) r = 0ull;
  else if (s >= 64) r = hi >> (s - 64);
  else if (s > 0) r = (lo >> s) | (hi << (64 - s));
  else if (s > -64) r = lo << (-s);
  else r = 0ull;
  return (b >> 31) ? 0ull - r : r;
}

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16x2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Turns the thread's 8 column pairs. Interleaved: the pairs are neighbouring
// columns of both chunks; else pair i is column i of each chunk.
__device__ __forceinline__ void turn16(float* x, const float* cs, const float* sn, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * cs[i] - b * sn[i];
      x[2 * i + 1] = a * sn[i] + b * cs[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = x[8 + i];
      x[i] = a * cs[i] - b * sn[i];
      x[8 + i] = a * sn[i] + b * cs[i];
    }
  }
}

template <int T>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int o = T / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// What a thread keeps for its columns: chunk offsets, turn rates and axes.
template <int D>
struct Columns {
  int c0, c1;                    // first columns of its two chunks
  bool turned;
  unsigned long long rate[8];
  int axis[8];

  __device__ __forceinline__ void init(const NormRopeParams& p, int tau) {
    const int tr = p.rot / 16;   // threads of a row whose columns are turned
    turned = tau < tr;
    if (!turned) {
      c0 = p.rot + (tau - tr) * 16;
      c1 = c0 + 8;
    } else if (p.interleaved) {
      c0 = tau * 16;
      c1 = c0 + 8;
    } else {
      c0 = tau * 8;
      c1 = c0 + p.rot / 2;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = tau * 8 + i;
      rate[i] = turned ? turn_rate(__ldg(p.freq + pair)) : 0ull;
      axis[i] = (pair >= p.sec0 ? 1 : 0) + (pair >= p.sec1 ? 1 : 0);
    }
  }

  // cos and sin of the thread's pairs at token `tok`
  __device__ __forceinline__ void angles(const NormRopeParams& p, long long tok, float* cs, float* sn) const {
    if (!turned) return;
    int pos[3];
    pos[0] = __ldg(p.pos + tok);
    pos[1] = p.axes > 1 ? __ldg(p.pos + p.tokens + tok) : 0;
    pos[2] = p.axes > 2 ? __ldg(p.pos + 2 * p.tokens + tok) : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = axis[i] == 0 ? pos[0] : axis[i] == 1 ? pos[1] : pos[2];
      const unsigned long long t = rate[i] * static_cast<unsigned long long>(static_cast<long long>(at));
      const int q = static_cast<int>((t + 0x80000000ull) >> 32);  // nearest 2^-32 of a turn, in [-1/2, 1/2)
      sincospif(static_cast<float>(q) * 4.656612873077393e-10f, &sn[i], &cs[i]);  // 2^-31: half turns
    }
  }
};

template <int D>
__device__ __forceinline__ void load_weight(const __nv_bfloat16* w, const Columns<D>& c, float* out) {
  unpack8(__ldg(reinterpret_cast<const uint4*>(w + c.c0)), out);
  unpack8(__ldg(reinterpret_cast<const uint4*>(w + c.c1)), out + 8);
}

// Grid: x = blocks of 256 / (d / 16) tokens, y = chunks of p.heads_per of the
// h + h_kv heads (queries first).
template <int D>
__global__ void __launch_bounds__(kNrThreads) attn_norm_rope_kernel(const NormRopeParams p) {
  constexpr int T = D / 16, RB = kNrThreads / T;
  const int tau = threadIdx.x % T;
  const long long tok = static_cast<long long>(blockIdx.x) * RB + threadIdx.x / T;
  const bool live = tok < p.tokens;
  const long long tk = live ? tok : p.tokens - 1;  // every lane takes part in the shuffles
  const int b = static_cast<int>(tk / p.n), i = static_cast<int>(tk - static_cast<long long>(b) * p.n);
  Columns<D> col;
  col.init(p, tau);
  float cs[8], sn[8];
  col.angles(p, tk, cs, sn);
  const int h0 = blockIdx.y * p.heads_per, h1 = min(h0 + p.heads_per, p.h + p.h_kv);
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int lo = part == 0 ? min(h0, p.h) : max(h0, p.h) - p.h;
    const int hi = part == 0 ? min(h1, p.h) : max(h1, p.h) - p.h;
    if (lo >= hi) continue;
    const int heads = part == 0 ? p.h : p.h_kv;
    const __nv_bfloat16* src = part == 0 ? p.q : p.k;
    __nv_bfloat16* dst = part == 0 ? p.q_out : p.k_out;
    float w[16];
    load_weight<D>(part == 0 ? p.w_q : p.w_k, col, w);
    const size_t step = static_cast<size_t>(p.n) * D;
    size_t at = ((static_cast<size_t>(b) * heads + lo) * p.n + i) * D;
    uint4 va = *reinterpret_cast<const uint4*>(src + at + col.c0);
    uint4 vb = *reinterpret_cast<const uint4*>(src + at + col.c1);
    for (int hd = lo; hd < hi; ++hd, at += step) {
      uint4 na = va, nb = vb;
      if (hd + 1 < hi) {  // the next head's row while this one is computed
        na = *reinterpret_cast<const uint4*>(src + at + step + col.c0);
        nb = *reinterpret_cast<const uint4*>(src + at + step + col.c1);
      }
      float x[16];
      unpack8(va, x);
      unpack8(vb, x + 8);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
      const float r = rsqrtf(row_sum<T>(ss) * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[e];
      if (col.turned) turn16(x, cs, sn, p.interleaved);
      if (live) {
        *reinterpret_cast<uint4*>(dst + at + col.c0) = pack8(x);
        *reinterpret_cast<uint4*>(dst + at + col.c1) = pack8(x + 8);
      }
      va = na;
      vb = nb;
    }
  }
}

// Backward. Persistent: block x takes token blocks x, x + gridDim.x, ...; its
// threads keep their columns, so the weight gradients of all its rows add up in
// registers, then over the block's row groups in shared memory, and leave as
// one fp32 partial a block (added in block order by the reduction below: the
// same sizes on the same GPU give the same bits).
template <int D>
__global__ void __launch_bounds__(kNrThreads) attn_norm_rope_bwd_kernel(const NormRopeParams p) {
  constexpr int T = D / 16, RB = kNrThreads / T;
  __shared__ float red[RB][D + 1];
  const int tau = threadIdx.x % T, grp = threadIdx.x / T;
  Columns<D> col;
  col.init(p, tau);
  const int h0 = blockIdx.y * p.heads_per, h1 = min(h0 + p.heads_per, p.h + p.h_kv);
  const size_t part_id = static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int lo = part == 0 ? min(h0, p.h) : max(h0, p.h) - p.h;
    const int hi = part == 0 ? min(h1, p.h) : max(h1, p.h) - p.h;
    const int heads = part == 0 ? p.h : p.h_kv;
    const __nv_bfloat16* src = part == 0 ? p.q : p.k;
    const __nv_bfloat16* up = part == 0 ? p.dq_out : p.dk_out;
    __nv_bfloat16* dst = part == 0 ? p.dq : p.dk;
    float dw[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) dw[e] = 0.f;
    if (lo < hi) {
      float w[16];
      load_weight<D>(part == 0 ? p.w_q : p.w_k, col, w);
      for (long long blk = blockIdx.x; blk < p.token_blocks; blk += gridDim.x) {
        const long long tok = blk * RB + grp;
        const bool live = tok < p.tokens;
        const long long tk = live ? tok : p.tokens - 1;
        const int b = static_cast<int>(tk / p.n), i = static_cast<int>(tk - static_cast<long long>(b) * p.n);
        float cs[8], sn[8];
        col.angles(p, tk, cs, sn);
#pragma unroll
        for (int e = 0; e < 8; ++e) sn[e] = -sn[e];
        const size_t step = static_cast<size_t>(p.n) * D;
        size_t at = ((static_cast<size_t>(b) * heads + lo) * p.n + i) * D;
        for (int hd = lo; hd < hi; ++hd, at += step) {
          float x[16], u[16];
          unpack8(*reinterpret_cast<const uint4*>(src + at + col.c0), x);
          unpack8(*reinterpret_cast<const uint4*>(src + at + col.c1), x + 8);
          unpack8(*reinterpret_cast<const uint4*>(up + at + col.c0), u);
          unpack8(*reinterpret_cast<const uint4*>(up + at + col.c1), u + 8);
          if (col.turned) turn16(u, cs, sn, p.interleaved);
          float ss = 0.f, sw = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            ss = fmaf(x[e], x[e], ss);
            sw = fmaf(w[e] * u[e], x[e], sw);
          }
          const float r = rsqrtf(row_sum<T>(ss) * (1.f / D) + p.eps);
          const float mean = row_sum<T>(sw) * r * (1.f / D);  // mean of w u x r
          if (live) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float xr = x[e] * r;
              dw[e] = fmaf(u[e], xr, dw[e]);
              x[e] = r * (w[e] * u[e] - xr * mean);
            }
            *reinterpret_cast<uint4*>(dst + at + col.c0) = pack8(x);
            *reinterpret_cast<uint4*>(dst + at + col.c1) = pack8(x + 8);
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      red[grp][col.c0 + e] = dw[e];
      red[grp][col.c1 + e] = dw[8 + e];
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll 8
      for (int g = 0; g < RB; ++g) s += red[g][threadIdx.x];
      p.part[(part_id * 2 + part) * D + threadIdx.x] = s;
    }
  }
}

// dw (bf16) of column c: the blocks' partials, 32 interleaved running sums
// joined in a fixed order. Grid: 2 d / 8 blocks of 8 columns x 32 lanes.
template <int D>
__global__ void __launch_bounds__(256) attn_norm_rope_dw_kernel(const float* part, int blocks, __nv_bfloat16* dw_q,
                                                                __nv_bfloat16* dw_k) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x / 8, cc = blockIdx.x * 8 + threadIdx.x % 8;  // cc: column of q | k
  float s = 0.f;
  for (int i = lane; i < blocks; i += 32) s += part[static_cast<size_t>(i) * 2 * D + cc];
  red[threadIdx.x % 8][lane] = s;
  __syncthreads();
  if (threadIdx.x < 8) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[threadIdx.x][i];
    __nv_bfloat16* dst = cc < D ? dw_q : dw_k;
    if (dst != nullptr) dst[cc % D] = __float2bfloat16_rn(t);
  }
}

template <int D>
cudaError_t launch_fwd_d(NormRopeParams p, cudaStream_t stream) {
  constexpr int RB = kNrThreads / (D / 16);
  const long long blocks = (p.tokens + RB - 1) / RB;
  const int heads = p.h + p.h_kv;
  // all heads of a token in one thread (one angle computation), unless that
  // leaves fewer than four blocks per SM: then the heads are split
  int per = heads;
  while (per > 1 && blocks * ((heads + per - 1) / per) < 4ll * kSms) per = (per + 1) / 2;
  while ((heads + per - 1) / per > 65535) ++per;
  p.heads_per = per;
  prof_begin(kKindNormRope, stream);
  attn_norm_rope_kernel<D><<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + per - 1) / per)),
                             kNrThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  prof_end(kKindNormRope, stream);
  return e;
}

template <int D>
cudaError_t launch_bwd_d(NormRopeParams p, cudaStream_t stream) {
  int gx, gy;
  norm_rope_bwd_grid(D, p.tokens, p.h + p.h_kv, &gx, &gy, &p.heads_per);
  p.token_blocks = (p.tokens + kNrThreads / (D / 16) - 1) / (kNrThreads / (D / 16));
  prof_begin(kKindNormRope, stream);
  attn_norm_rope_bwd_kernel<D><<<dim3(gx, gy), kNrThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  prof_end(kKindNormRope, stream);
  if (e != cudaSuccess) return e;
  prof_begin(kKindNormRope, stream);
  attn_norm_rope_dw_kernel<D><<<2 * D / 8, 256, 0, stream>>>(p.part, gx * gy, p.dw_q, p.dw_k);
  e = cudaGetLastError();
  prof_end(kKindNormRope, stream);
  return e;
}

}  // namespace

// Backward grid: at most four blocks per SM (a partial each), heads split only
// where the tokens alone do not fill them.
void norm_rope_bwd_grid(int d, long long tokens, int heads, int* gx, int* gy, int* heads_per) {
  const int rb = kNrThreads / (d / 16);
  const long long blocks = (tokens + rb - 1) / rb;
  const long long room = 4ll * kSms;
  *gx = static_cast<int>(blocks < room ? blocks : room);
  int per = heads;
  while (per > 1 && static_cast<long long>(*gx) * ((heads + per - 1) / per) * 2 <= room) per = (per + 1) / 2;
  *heads_per = per;
  *gy = (heads + per - 1) / per;
}

cudaError_t launch_norm_rope(int d, const NormRopeParams& p, cudaStream_t stream) {
  switch (d) {
    case 32: return launch_fwd_d<32>(p, stream);
    case 64: return launch_fwd_d<64>(p, stream);
    case 128: return launch_fwd_d<128>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_norm_rope_bwd(int d, const NormRopeParams& p, cudaStream_t stream) {
  switch (d) {
    case 32: return launch_bwd_d<32>(p, stream);
    case 64: return launch_bwd_d<64>(p, stream);
    case 128: return launch_bwd_d<128>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
