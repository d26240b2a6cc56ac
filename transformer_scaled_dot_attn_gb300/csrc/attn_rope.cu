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
// reduction, sin, cos) are computed once per token and head chunk. The rows of
// the next heads are on their way meanwhile: two rows in registers (forward), or
// four pairs of rows in slots of shared memory that are the thread's own, so
// without barriers (backward, whose sums need the registers). Measured, 4 x 16384
// tokens of 20 heads, d = 128: two rows ahead 105 us, one 116, shared memory 138;
// backward of 3 x 4093 tokens of 18 heads: shared memory 31 us, registers 40.
#include "attn_kernels.cuh"

#include <atomic>

namespace attn {
namespace {

using namespace sm103;

constexpr int kNrThreads = 256;
constexpr int kFwdAhead = 2;  // heads whose rows are on their way, forward
constexpr int kBwdAhead = 4;  // rows on their way into shared memory, backward (16 KB each a block)

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

// The thread's 8 column pairs (a_i, b_i) as packed fp32 pairs: a[j] holds
// a_2j, a_2j+1. The two chunks hold the a's and the b's, or (interleaved)
// a_i b_i side by side; only loading and storing differ.
struct Pairs {
  uint64_t a[4], b[4];
};

__device__ __forceinline__ uint64_t lo_pair(uint32_t w0, uint32_t w1) {
  return f2_pack(__uint_as_float(w0 << 16), __uint_as_float(w1 << 16));
}
__device__ __forceinline__ uint64_t hi_pair(uint32_t w0, uint32_t w1) {
  return f2_pack(__uint_as_float(w0 & 0xffff0000u), __uint_as_float(w1 & 0xffff0000u));
}
__device__ __forceinline__ uint64_t both(uint32_t w) {
  const float2 f = unpack_bf16x2(w);
  return f2_pack(f.x, f.y);
}

template <bool INTER>
__device__ __forceinline__ void unpack(const uint4& u, const uint4& v, Pairs& x) {
  if (INTER) {
    x.a[0] = lo_pair(u.x, u.y), x.b[0] = hi_pair(u.x, u.y);
    x.a[1] = lo_pair(u.z, u.w), x.b[1] = hi_pair(u.z, u.w);
    x.a[2] = lo_pair(v.x, v.y), x.b[2] = hi_pair(v.x, v.y);
    x.a[3] = lo_pair(v.z, v.w), x.b[3] = hi_pair(v.z, v.w);
  } else {
    x.a[0] = both(u.x), x.a[1] = both(u.y), x.a[2] = both(u.z), x.a[3] = both(u.w);
    x.b[0] = both(v.x), x.b[1] = both(v.y), x.b[2] = both(v.z), x.b[3] = both(v.w);
  }
}

template <bool INTER>
__device__ __forceinline__ void pack(const Pairs& x, uint4& u, uint4& v) {
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (INTER) {
      float a0, a1, b0, b1;
      f2_unpack(x.a[j], a0, a1);
      f2_unpack(x.b[j], b0, b1);
      o[2 * j] = pack_bf16x2(a0, b0);
      o[2 * j + 1] = pack_bf16x2(a1, b1);
    } else {
      o[j] = pack_bf16x2_pair(x.a[j]);
      o[4 + j] = pack_bf16x2_pair(x.b[j]);
    }
  }
  u = make_uint4(o[0], o[1], o[2], o[3]);
  v = make_uint4(o[4], o[5], o[6], o[7]);
}

// (a, b) -> (a c - b s, a s + b c)
__device__ __forceinline__ void turn(Pairs& x, const uint64_t* c, const uint64_t* s, const uint64_t* ns) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t a = x.a[j], b = x.b[j];
    x.a[j] = fma2(a, c[j], mul2(b, ns[j]));
    x.b[j] = fma2(a, s[j], mul2(b, c[j]));
  }
}

// sum of the products of two vectors of the thread's columns
__device__ __forceinline__ float dot(const Pairs& x, const Pairs& y) {
  uint64_t u = mul2(x.a[0], y.a[0]), v = mul2(x.b[0], y.b[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) {
    u = fma2(x.a[j], y.a[j], u);
    v = fma2(x.b[j], y.b[j], v);
  }
  float a, b;
  f2_unpack(add2(u, v), a, b);
  return a + b;
}

// Copies 16 bytes into the thread's own slot of shared memory, asynchronously.
__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of the thread's latest groups are still on their way.
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int T>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int o = T / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// A thread's columns: two chunks of eight, one in each half of the turned columns,
// or of the others. (Neighbouring threads' chunks are neighbours, so that a warp's
// access takes whole 32-byte sectors: with chunks side by side in the threads of columns
// that are not turned, the gradients of 96 x 256 tokens, 8 + 8 heads, half of 64 columns
// turned, took 38 us instead of 32.)
struct Columns {
  int c0, c1;                    // first columns of the chunks
  int pair0, pair1;              // first column pair of the first four, of the other four
  bool turned;

  __device__ __forceinline__ void init(const NormRopeParams& p, int d, int tau) {
    const int tr = p.rot / 16;   // threads of a row whose columns are turned
    turned = tau < tr;
    c0 = turned ? tau * 8 : p.rot + (tau - tr) * 8;
    c1 = c0 + (turned ? p.rot : d - p.rot) / 2;
    pair0 = p.interleaved ? c0 / 2 : c0;
    pair1 = p.interleaved ? c1 / 2 : c0 + 4;
  }
};

// The turn rates of all pairs, once a block, in shared memory.
__device__ __forceinline__ void fill_rates(const NormRopeParams& p, unsigned long long* rates) {
  for (int i = threadIdx.x; i < p.rot / 2; i += kNrThreads) rates[i] = turn_rate(__ldg(p.freq + i));
  __syncthreads();
}

// cos, sin and -sin of the thread's pairs at token `tok`. The fixed-point
// reduction leaves an angle in [-pi, pi), where the hardware's sine and cosine
// are within 2^-21 (the results are rounded to bf16, 2^-9 of their value).
__device__ __forceinline__ void angles(const NormRopeParams& p, const Columns& c, const unsigned long long* rates,
                                       long long tok, uint64_t* cs, uint64_t* sn, uint64_t* ns) {
  if (!c.turned) return;
  int pos[3];
  pos[0] = __ldg(p.pos + tok);
  pos[1] = p.axes > 1 ? __ldg(p.pos + p.tokens + tok) : 0;
  pos[2] = p.axes > 2 ? __ldg(p.pos + 2 * p.tokens + tok) : 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int pair = (j < 2 ? c.pair0 : c.pair1) + 2 * (j & 1) + e;
      const int at = pair < p.sec0 ? pos[0] : pair < p.sec1 ? pos[1] : pos[2];
      const unsigned long long t = rates[pair] * static_cast<unsigned long long>(static_cast<long long>(at));
      const int q = static_cast<int>((t + 0x80000000ull) >> 32);  // nearest 2^-32 of a turn, in [-1/2, 1/2)
      x[e] = static_cast<float>(q) * 1.46291807926715968e-9f;     // 2 pi 2^-32
    }
    const float s0 = __sinf(x[0]), s1 = __sinf(x[1]);
    cs[j] = f2_pack(__cosf(x[0]), __cosf(x[1]));
    sn[j] = f2_pack(s0, s1);
    ns[j] = f2_pack(-s0, -s1);
  }
}

// Grid: x = blocks of 256 / (d / 16) tokens, y = chunks of p.heads_per of the
// h + h_kv heads (queries first).
template <int D, bool INTER>
__global__ void __launch_bounds__(kNrThreads, 3) attn_norm_rope_kernel(const NormRopeParams p) {
  constexpr int T = D / 16, RB = kNrThreads / T;
  __shared__ unsigned long long rates[D / 2];
  grid_follow();
  const int tau = threadIdx.x % T;
  const long long tok = static_cast<long long>(blockIdx.x) * RB + threadIdx.x / T;
  const bool live = tok < p.tokens;
  const long long tk = live ? tok : p.tokens - 1;  // every lane takes part in the shuffles
  const unsigned b = static_cast<unsigned>(tk) / static_cast<unsigned>(p.n);  // (B n < 2^31)
  const unsigned i = static_cast<unsigned>(tk) - b * static_cast<unsigned>(p.n);
  Columns col;
  col.init(p, D, tau);
  fill_rates(p, rates);
  uint64_t cs[4], sn[4], ns[4];
  angles(p, col, rates, tk, cs, sn, ns);
  const int h0 = blockIdx.y * p.heads_per, h1 = min(h0 + p.heads_per, p.h + p.h_kv);
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int lo = part == 0 ? min(h0, p.h) : max(h0, p.h) - p.h;
    const int hi = part == 0 ? min(h1, p.h) : max(h1, p.h) - p.h;
    if (lo >= hi) continue;
    const int heads = part == 0 ? p.h : p.h_kv;
    const __nv_bfloat16* src = part == 0 ? p.q : p.k;
    __nv_bfloat16* dst = part == 0 ? p.q_out : p.k_out;
    const __nv_bfloat16* wp = part == 0 ? p.w_q : p.w_k;
    Pairs w;
    unpack<INTER>(__ldg(reinterpret_cast<const uint4*>(wp + col.c0)),
                  __ldg(reinterpret_cast<const uint4*>(wp + col.c1)), w);
    const size_t step = static_cast<size_t>(p.n) * D;
    const size_t at = ((static_cast<size_t>(b) * heads + lo) * p.n + i) * D;
    uint4 va[kFwdAhead], vb[kFwdAhead];
#pragma unroll
    for (int k = 0; k < kFwdAhead; ++k)
      if (lo + k < hi) {
        va[k] = *reinterpret_cast<const uint4*>(src + at + k * step + col.c0);
        vb[k] = *reinterpret_cast<const uint4*>(src + at + k * step + col.c1);
      }
#pragma unroll 1
    for (int k0 = 0; k0 < hi - lo; k0 += kFwdAhead) {
#pragma unroll
      for (int j = 0; j < kFwdAhead; ++j) {
        const int k = k0 + j;
        if (lo + k >= hi) break;
        Pairs x;
        unpack<INTER>(va[j], vb[j], x);
        if (lo + k + kFwdAhead < hi) {
          va[j] = *reinterpret_cast<const uint4*>(src + at + (k + kFwdAhead) * step + col.c0);
          vb[j] = *reinterpret_cast<const uint4*>(src + at + (k + kFwdAhead) * step + col.c1);
        }
        const float r = rsqrtf(row_sum<T>(dot(x, x)) * (1.f / D) + p.eps);
        const uint64_t r2 = f2_pack(r, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x.a[e] = mul2(mul2(x.a[e], r2), w.a[e]);
          x.b[e] = mul2(mul2(x.b[e], r2), w.b[e]);
        }
        if (col.turned) turn(x, cs, sn, ns);
        if (live) {
          uint4 u, v;
          pack<INTER>(x, u, v);
          *reinterpret_cast<uint4*>(dst + at + k * step + col.c0) = u;
          *reinterpret_cast<uint4*>(dst + at + k * step + col.c1) = v;
        }
      }
    }
  }
}

// Backward. Persistent: block x takes token blocks x, x + gridDim.x, ...; its
// threads keep their columns, so the weight gradients of all its rows add up in
// registers, then over the block's row groups in shared memory, and leave as
// one fp32 partial a block (added in block order by the reduction below: the
// same sizes give the same bits). Block y: a chunk of p.heads_per of the query
// heads, or of the key heads (p.q_chunks chunks are the queries').
template <int D, bool INTER>
__global__ void __launch_bounds__(kNrThreads, 2) attn_norm_rope_bwd_kernel(const NormRopeParams p) {
  constexpr int T = D / 16, RB = kNrThreads / T;
  __shared__ unsigned long long rates[D / 2];
  extern __shared__ uint4 slots[];  // [kBwdAhead][4][kNrThreads]; in the end the rows' dw
  const int tau = threadIdx.x % T, grp = threadIdx.x / T;
  grid_follow();
  Columns col;
  col.init(p, D, tau);
  fill_rates(p, rates);
  const bool is_q = static_cast<int>(blockIdx.y) < p.q_chunks;
  const int heads = is_q ? p.h : p.h_kv;
  const int lo = (static_cast<int>(blockIdx.y) - (is_q ? 0 : p.q_chunks)) * p.heads_per;
  const int count = min(p.heads_per, heads - lo);  // heads of this block
  const __nv_bfloat16* src = is_q ? p.q : p.k;
  const __nv_bfloat16* up = is_q ? p.dq_out : p.dk_out;
  __nv_bfloat16* dst = is_q ? p.dq : p.dk;
  const __nv_bfloat16* wp = is_q ? p.w_q : p.w_k;
  Pairs w, dw;
  unpack<INTER>(__ldg(reinterpret_cast<const uint4*>(wp + col.c0)),
                __ldg(reinterpret_cast<const uint4*>(wp + col.c1)), w);
#pragma unroll
  for (int j = 0; j < 4; ++j) dw.a[j] = dw.b[j] = 0;
  const size_t step = static_cast<size_t>(p.n) * D;
  // the thread's row in token block blk at the chunk's first head
  auto row_of = [&](long long blk) {
    const unsigned tok = static_cast<unsigned>(min(blk * RB + grp, p.tokens - 1));
    const unsigned b = tok / static_cast<unsigned>(p.n), i = tok - b * static_cast<unsigned>(p.n);
    return ((static_cast<size_t>(b) * heads + lo) * p.n + i) * D;
  };
  // what is fetched next: head f_hd of token block f_blk
  long long f_blk = blockIdx.x;
  int f_hd = 0, f_slot = 0;
  size_t f_at = f_blk < p.token_blocks ? row_of(f_blk) : 0;
  auto fetch = [&]() {
    if (f_blk < p.token_blocks) {
      uint4* s = slots + f_slot * 4 * kNrThreads + threadIdx.x;
      copy16(s, src + f_at + col.c0);
      copy16(s + kNrThreads, src + f_at + col.c1);
      copy16(s + 2 * kNrThreads, up + f_at + col.c0);
      copy16(s + 3 * kNrThreads, up + f_at + col.c1);
      f_at += step;
      if (++f_hd == count) {
        f_hd = 0;
        f_blk += gridDim.x;
        if (f_blk < p.token_blocks) f_at = row_of(f_blk);
      }
    }
    f_slot = f_slot + 1 == kBwdAhead ? 0 : f_slot + 1;
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < kBwdAhead; ++k) fetch();
  int use = 0;
#pragma unroll 1
  for (long long blk = blockIdx.x; blk < p.token_blocks; blk += gridDim.x) {
    const long long tok = blk * RB + grp;
    const bool live = tok < p.tokens;
    uint64_t cs[4], sn[4], ns[4];
    angles(p, col, rates, live ? tok : p.tokens - 1, cs, sn, ns);
    size_t at = row_of(blk);
#pragma unroll 1
    for (int hd = 0; hd < count; ++hd, at += step) {
      copy_wait<kBwdAhead - 1>();
      const uint4* s = slots + use * 4 * kNrThreads + threadIdx.x;
      use = use + 1 == kBwdAhead ? 0 : use + 1;
      Pairs x, u;
      unpack<INTER>(s[0], s[kNrThreads], x);
      unpack<INTER>(s[2 * kNrThreads], s[3 * kNrThreads], u);
      fetch();
      if (col.turned) turn(u, cs, ns, sn);  // back by the angle
      Pairs wu;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        wu.a[j] = mul2(w.a[j], u.a[j]);
        wu.b[j] = mul2(w.b[j], u.b[j]);
      }
      const float ss = row_sum<T>(dot(x, x)), sw = row_sum<T>(dot(wu, x));
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      if (live) {
        // dx = r wu - x r^3 mean(wu x)
        const float back = -(r * r) * (r * (sw * (1.f / D)));
        const uint64_t r2 = f2_pack(r, r), back2 = f2_pack(back, back);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dw.a[j] = fma2(u.a[j], mul2(x.a[j], r2), dw.a[j]);
          dw.b[j] = fma2(u.b[j], mul2(x.b[j], r2), dw.b[j]);
          x.a[j] = fma2(x.a[j], back2, mul2(wu.a[j], r2));
          x.b[j] = fma2(x.b[j], back2, mul2(wu.b[j], r2));
        }
        uint4 o, v;
        pack<INTER>(x, o, v);
        *reinterpret_cast<uint4*>(dst + at + col.c0) = o;
        *reinterpret_cast<uint4*>(dst + at + col.c1) = v;
      }
    }
  }
  copy_wait<0>();
  __syncthreads();
  float (*red)[D + 1] = reinterpret_cast<float (*)[D + 1]>(slots);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a0, a1, b0, b1;
    f2_unpack(dw.a[j], a0, a1);
    f2_unpack(dw.b[j], b0, b1);
    if (INTER) {
      float* at = &red[grp][(j < 2 ? col.c0 : col.c1) + (j & 1) * 4];
      at[0] = a0, at[1] = b0, at[2] = a1, at[3] = b1;
    } else {
      red[grp][col.c0 + 2 * j] = a0, red[grp][col.c0 + 2 * j + 1] = a1;
      red[grp][col.c1 + 2 * j] = b0, red[grp][col.c1 + 2 * j + 1] = b1;
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll 8
    for (int g = 0; g < RB; ++g) s += red[g][threadIdx.x];
    p.part[(static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * D + threadIdx.x] = s;
  }
}

// dw (bf16) of a column: the blocks' partials, 128 interleaved running sums
// joined in a fixed order. Grid: x = 8 columns, y = queries, keys; 8 columns x 128 lanes a block.
template <int D>
__global__ void __launch_bounds__(1024) attn_norm_rope_dw_kernel(const float* part, int q_parts, int k_parts,
                                                                 __nv_bfloat16* dw_q, __nv_bfloat16* dw_k) {
  __shared__ float red[8][129];
  const int lane = threadIdx.x / 8, c = blockIdx.x * 8 + threadIdx.x % 8;
  const bool is_q = blockIdx.y == 0;
  const float* src = part + (is_q ? 0 : static_cast<size_t>(q_parts) * D);
  const int count = is_q ? q_parts : k_parts;
  grid_follow();  // the partials are written
  float s = 0.f;
#pragma unroll 8
  for (int i = lane; i < count; i += 128) s += src[static_cast<size_t>(i) * D + c];
  red[threadIdx.x % 8][lane] = s;
  __syncthreads();
  if (threadIdx.x < 256) {  // a warp a column
    const int col = threadIdx.x / 32, x = threadIdx.x % 32;
    float t = (red[col][x] + red[col][x + 32]) + (red[col][x + 64] + red[col][x + 96]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    __nv_bfloat16* dst = is_q ? dw_q : dw_k;
    if (x == 0 && dst != nullptr) dst[blockIdx.x * 8 + col] = __float2bfloat16_rn(t);
  }
}

template <int D>
cudaError_t launch_fwd_d(NormRopeParams p, cudaStream_t stream) {
  constexpr int RB = kNrThreads / (D / 16);
  const long long blocks = (p.tokens + RB - 1) / RB;
  const int heads = p.h + p.h_kv;
  // A token's angles are worth several heads: all of them in one thread, unless
  // the grid is then less than three times what the SMs hold (three blocks
  // each); down to one head a thread where the tokens leave SMs empty. (4 x 16384
  // tokens, 20 heads, d = 128: 20 heads a thread 105 us, 10: 106, 5: 117.)
  int per = heads;
  while (per > 4 && blocks * ((heads + per - 1) / per) < 9ll * kSms) per = (per + 1) / 2;
  while (per > 1 && blocks * ((heads + per - 1) / per) < 3ll * kSms) per = (per + 1) / 2;
  p.heads_per = per;
  prof_begin(kKindNormRope, stream);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + per - 1) / per));
  const auto kernel = p.interleaved ? attn_norm_rope_kernel<D, true> : attn_norm_rope_kernel<D, false>;
  const cudaError_t e = launch_dependent(kernel, grid, dim3(kNrThreads), 0, stream, p);
  prof_end(kKindNormRope, stream);
  return e;
}

template <int D>
cudaError_t launch_bwd_d(NormRopeParams p, cudaStream_t stream) {
  constexpr int kSmem = kBwdAhead * 4 * kNrThreads * 16;
  static_assert(kSmem >= kNrThreads / (D / 16) * (D + 1) * 4, "the rows' dw fit");
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!set[dev & 63].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(attn_norm_rope_bwd_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attn_norm_rope_bwd_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    set[dev & 63].store(true, std::memory_order_relaxed);
  }
  int gx, gy;
  norm_rope_bwd_grid(D, p.tokens, p.h, p.h_kv, &gx, &gy, &p.heads_per);
  p.q_chunks = (p.h + p.heads_per - 1) / p.heads_per;
  p.token_blocks = (p.tokens + kNrThreads / (D / 16) - 1) / (kNrThreads / (D / 16));
  prof_begin(kKindNormRope, stream);
  const auto kernel = p.interleaved ? attn_norm_rope_bwd_kernel<D, true> : attn_norm_rope_bwd_kernel<D, false>;
  e = launch_dependent(kernel, dim3(gx, gy), dim3(kNrThreads), kSmem, stream, p);
  prof_end(kKindNormRope, stream);
  if (e != cudaSuccess) return e;
  prof_begin(kKindNormRope, stream);
  e = launch_dependent(attn_norm_rope_dw_kernel<D>, dim3(D / 8, 2), dim3(1024), 0, stream, p.part, gx * p.q_chunks,
                       gx * (gy - p.q_chunks), p.dw_q, p.dw_k);
  prof_end(kKindNormRope, stream);
  return e;
}

}  // namespace

// Backward grid: x = token blocks, y = chunks of query or key heads: all heads in
// a chunk while that gives four blocks per SM (two run at a time), down to
// one head a chunk where the tokens leave SMs empty (3 x 4093 tokens, 16 + 2
// heads, d = 128: 16 heads a chunk 31 us, 8: 34, 4: 40). With more than 32 token
// blocks per SM the blocks walk over several, so the partials of dw stay few.
void norm_rope_bwd_grid(int d, long long tokens, int h, int h_kv, int* gx, int* gy, int* heads_per) {
  const int rb = kNrThreads / (d / 16);
  const long long blocks = (tokens + rb - 1) / rb;
  auto chunks = [&](int per) { return static_cast<long long>((h + per - 1) / per) + (h_kv + per - 1) / per; };
  int per = h > h_kv ? h : h_kv;
  while (per > 1 && blocks * chunks(per) < 4ll * kSms) per = (per + 1) / 2;
  *gx = static_cast<int>(blocks < 32ll * kSms ? blocks : 32ll * kSms);
  *gy = static_cast<int>(chunks(per));
  *heads_per = per;
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
