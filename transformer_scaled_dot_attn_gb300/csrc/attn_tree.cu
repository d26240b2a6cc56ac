// Decoding of drafted tokens over a cache: the n newest positions of each
// sequence (n <= 64) are queries, hanging on one another as a tree. Every query
// sees all positions before the newest n and, of the newest n, those whose bit
// is set in its mask word (its ancestors and itself; without masks: the
// positions up to its own). h / h_kv query heads share a key head, and their
// queries of one sequence are neighbours in memory, so a key head faces one
// matrix of rows = (h / h_kv) n queries:
//
//   x_rj = scale q_r . k_j over the visible j,  O_r = sum_j softmax(x_r)_j v_j,  lse_r = ln sum_j exp(x_rj).
//
// The caches are bf16, or e4m3 codes with a power-of-two scale a row.
//
// With few rows a step is bound by reading the cache once. The keys of a head
// are split over CTAs by the sequence's own length (every CTA of a sequence
// gets the same number of tiles, whatever the capacity), and over the four warps
// of a CTA: each warp streams its own tiles through its own TMA ring and keeps
// its own running maximum, so the loop has no CTA barrier. The products run on
// mma.sync with 16 query rows (a tcgen05 tile has 128 rows, most of them idle
// here, and its operands would have to be written out in 16 bits first). The
// warps' results are joined in shared memory, the CTAs' by a second kernel.
// Many rows take the tcgen05 kernel (attn_tree_tc.cu).
#include "attn_tree.cuh"

#include <algorithm>
#include <atomic>

namespace attn {
namespace {

using namespace sm103;

constexpr int kTreeWarps = 4;
constexpr int kTreeThreads = kTreeWarps * 32;
constexpr int kTreeRows = 16;     // query rows of a CTA (one mma.sync tile)
// Tiles' worth of time that beginning a unit takes. With 0, 1, 2, 3, 4: 73.0, 71.4,
// 69.3, 69.0, 70.3 us (64 sequences of uneven lengths, 16 heads of one row, e4m3); 98.7 to
// 96.4 us from 2 on (4 sequences, 512 rows, e4m3).
constexpr int kTreeLead = 3;
// A CTA takes a unit alone, and nothing has to be joined, where it does not have to do
// more than this many 128 keys above an equal share for that. (Alone : shared, us: one
// sequence of 300 positions, 8 heads of 5 rows, d = 64: 5.9 : 8.1; 2 of 1000, e4m3: 11.9 :
// 9.8; 16 of 1500, 8 key heads of 128 rows, d = 128: 29.3 : 38.2; 8 of 2000, 4 key heads,
// e4m3: 31.2 : 23.1.) And in caches of at most so many 128 only, as the lengths may differ.
constexpr double kTreeShort = 7.5;
constexpr int kTreeAlone = 16, kTreeAloneMany = 8;  // (more units than places on the GPU)

template <int D, bool Q8>
struct Tree {
  static constexpr int ES = Q8 ? 1 : 2;                    // bytes of a cache element
  static constexpr int TK = (D == 128 && !Q8) ? 16 : 32;   // keys per tile of a warp
  static constexpr uint32_t KT = TK * D * ES;              // one K (or V) tile
  static constexpr uint32_t ROWB = D * ES <= 128 ? D * ES : 128;  // bytes of a row in a TMA box
  static constexpr uint32_t BOX = TK * ROWB;
  static constexpr int NBOX = D * ES / ROWB;
  static constexpr int BN = kTreeWarps * TK;               // keys of a CTA's tile
  static constexpr int STAGES = 2;
  static constexpr int CTAS = D == 128 ? 2 : 4;            // per SM
  static constexpr int NT = TK / 8;                        // n8 score tiles
  static constexpr int KS = D / 16;                        // k steps of the score product
  static constexpr uint32_t RING = kTreeWarps * STAGES * 2 * KT;
  static constexpr int OST = D + 4;                        // row pitch of the join area (fp32)
  static constexpr uint32_t JOIN = kTreeWarps * kTreeRows * OST * 4;
  static constexpr uint32_t SMEM = (RING > JOIN ? RING : JOIN) + 1024;  // + alignment slack
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

// e4m3 caches: which key of a group of eight stands in column g of a product.
// The order is chosen so that the threads that read shared memory together
// meet every bank once, for K (rows of neighbouring g) and V (rows of one t).
template <int D>
__device__ __forceinline__ int key_of(int g) {
  const int t = g >> 1;
  if (D == 128) return t + 4 * (g & 1);
  if (D == 64) return ((t & 1) + 4 * (t >> 1)) ^ ((g & 1) * 3);
  return (g & 1) ? (t ^ 2) + 4 : t;
}

// e4m3 caches, d = 128: the 16-byte column chunk of product column g (same reason).
template <int D>
__device__ __forceinline__ int col_of(int g) {
  return D == 128 ? (g >> 1) + 4 * (g & 1) : g;
}

// Byte offset of byte `at` of row r in a tile as TMA's swizzle lays it out.
template <int D, bool Q8>
__device__ __forceinline__ uint32_t tile_off(int r, int at) {
  using C = Tree<D, Q8>;
  const int box = at / static_cast<int>(C::ROWB), in = at % static_cast<int>(C::ROWB);
  const int chunk = in >> 4, low = in & 15;
  const int pc = C::ROWB == 128 ? (chunk ^ (r & 7)) : C::ROWB == 64 ? (chunk ^ ((r >> 1) & 3)) : chunk;
  return box * C::BOX + r * C::ROWB + (pc << 4) + low;
}

__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          const Watchdog& wd) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > wd.budget_ns) {
      *abort_flag = 1;
      atomicCAS(wd.status, 0u, kDevTimeout | kSiteTree);
      return false;
    }
  }
  return true;
}

// Copies in flight must land before the CTA's shared memory goes away.
__device__ __forceinline__ void tree_drain(uint64_t* bar, uint32_t parity, const Watchdog& wd) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > wd.budget_ns) {
      atomicCAS(wd.status, 0u, kDevTimeout | kSiteDrain);
      return;
    }
  }
}

// A value of the tile, for the rare rows that add one that is not finite themselves.
template <int D, bool Q8>
__device__ __forceinline__ float value_at(const uint8_t* tile, int r, int c) {
  if constexpr (Q8) {
    const uint32_t code = tile[tile_off<D, true>(r, c)];
    return (code & 0x7fu) == 0x7fu ? __uint_as_float(0x7fc00000u) : 0.f;  // only NaN matters here
  } else {
    const uint16_t h = *reinterpret_cast<const uint16_t*>(tile + tile_off<D, false>(r, 2 * c));
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
  }
}

// Zeroes the halves of a value pair that may not enter a product: keys at or
// past L (what the cache holds there is anyone's) and values that are not
// finite (a weight of 0 would make them NaN for rows that do not see them;
// `odd` reports them, and the rows that do see them add them afterwards).
__device__ __forceinline__ uint32_t clean_pair(uint32_t v, bool lo_real, bool hi_real, bool& odd) {
  if (!lo_real) v &= 0xffff0000u;
  if (!hi_real) v &= 0x0000ffffu;
  if ((v & 0x7f80u) == 0x7f80u) {
    odd = true;
    v &= 0xffff0000u;
  }
  if ((v & 0x7f800000u) == 0x7f800000u) {
    odd = true;
    v &= 0x0000ffffu;
  }
  return v;
}

// The k steps of the score product for a key's words (e4m3): word k holds the
// key's four codes that stand in columns 2t, 2t + 1, 2t + 8, 2t + 9 of step k.
template <int D>
__device__ __forceinline__ void key_words(const uint8_t* tile, int r, int t, uint32_t (&w)[D / 16]) {
  if constexpr (D == 128) {
    const uint4 u = *reinterpret_cast<const uint4*>(tile + tile_off<D, true>(r, 16 * t));
    const uint4 v = *reinterpret_cast<const uint4*>(tile + tile_off<D, true>(r, 16 * (t + 4)));
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
  } else if constexpr (D == 64) {
    const uint4 u = *reinterpret_cast<const uint4*>(tile + tile_off<D, true>(r, 16 * t));
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(tile + tile_off<D, true>(r, 8 * t));
    w[0] = u.x, w[1] = u.y;
  }
}

// The D / 8 codes of position r in product column g's output columns.
template <int D>
__device__ __forceinline__ void value_words(const uint8_t* tile, int r, int g, uint32_t (&w)[D / 32]) {
  const uint8_t* src = tile + tile_off<D, true>(r, col_of<D>(g) * (D / 8));
  if constexpr (D == 128) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (D == 64) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(src);
  }
}

// The four warps' results, `sall` [warp][row][D + 4], as a part's or the final result.
template <int D, int ROWS>
__device__ __forceinline__ void tree_join(const TreeParams& p, const TreePart& part, const float* sall,
                                          const float (&s_m)[kTreeWarps][ROWS], const float (&s_l)[kTreeWarps][ROWS],
                                          int row0) {
  constexpr int OST = D + 4, TPR = kTreeThreads / ROWS;  // pitch; threads of an output row
  const int tid = threadIdx.x, r = tid / TPR, row = row0 + r;
  if (row >= p.rows) return;
  float M = -INFINITY, sum = 0.f, f[kTreeWarps];
#pragma unroll
  for (int w = 0; w < kTreeWarps; ++w) M = fmaxf(M, s_m[w][r]);
#pragma unroll
  for (int w = 0; w < kTreeWarps; ++w) {
    f[w] = M == -INFINITY ? 0.f : ex2_approx(s_m[w][r] - M);
    sum = fmaf(f[w], s_l[w][r], sum);
  }
  auto joined = [&](int col) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kTreeWarps; ++w) o = fmaf(f[w], sall[(w * ROWS + r) * OST + col], o);
    return o;
  };
  if (part.whole) {
    const float inv = M == -INFINITY ? 0.f : 1.f / sum;  // a row that saw no key is the empty sum
    const size_t out = static_cast<size_t>(part.bh) * p.rows + row;
    for (int col = (tid % TPR) * 2; col < D; col += TPR * 2)
      *reinterpret_cast<uint32_t*>(p.o + out * D + col) = pack_bf16x2(joined(col) * inv, joined(col + 1) * inv);
    if (tid % TPR == 0 && p.lse != nullptr) p.lse[out] = M == -INFINITY ? -INFINITY : (M + log2f(sum)) * kTreeLn2;
  } else {
    const size_t at = static_cast<size_t>(part.slot) * p.block_rows + r;
    for (int col = (tid % TPR) * 2; col < D; col += TPR * 2)
      *reinterpret_cast<float2*>(p.part + at * D + col) = make_float2(joined(col), joined(col + 1));
    if (tid % TPR == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(M, sum);
  }
}

// One CTA per share of the line of tiles (attn_tree.cuh); a tile is the four
// warps' TK keys each.
template <int D, bool Q8>
__global__ void __launch_bounds__(kTreeThreads, Tree<D, Q8>::CTAS)
attn_tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const TreeParams p) {
  using C = Tree<D, Q8>;
  constexpr int H = 2;  // a thread's rows: g and g + 8
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kTreeWarps][C::STAGES];
  __shared__ int abort_word;
  __shared__ float s_m[kTreeWarps][kTreeRows], s_l[kTreeWarps][kTreeRows];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  volatile int* abort_flag = &abort_word;
  const Watchdog wd = p.wd;
  grid_follow();
  TreeWalk walk;
  if (!tree_start(p, C::BN, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), walk)) return;
  if (tid == 0) {
    for (int w = 0; w < kTreeWarps; ++w)
      for (int s = 0; s < C::STAGES; ++s) mbar_init(&full[w][s], 1);
    abort_word = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  __syncthreads();
  uint8_t* ring = smem + warp * (C::STAGES * 2 * C::KT);
  int turn = 0;  // tiles this warp has put through its ring
  TreePart part;
#pragma unroll 1
  while (tree_next(p, C::BN, walk, part)) {
    const int bh = part.bh, row0 = part.rb * kTreeRows, L = part.L;
    const int old = L - p.n;             // positions before the newest n (negative: fewer cached than n)
    const int mine = part.t1 - part.t0;  // of every tile this warp takes keys [warp TK, warp TK + TK)
    const int key0 = part.t0 * C::BN + warp * C::TK;
    auto load = [&](int x) {
      const int st = (turn + x) % C::STAGES;
      const int k0 = key0 + x * C::BN;
      uint8_t* dst = ring + st * 2 * C::KT;
      mbar_arrive_expect_tx(&full[warp][st], 2 * C::KT);
      for (int a = 0; a < C::NBOX; ++a) {
        tma_load_3d(dst + a * C::BOX, &tm_k, &full[warp][st], a * (C::ROWB / C::ES), k0, bh);
        tma_load_3d(dst + C::KT + a * C::BOX, &tm_v, &full[warp][st], a * (C::ROWB / C::ES), k0, bh);
      }
    };
    if (lane == 0)
      for (int x = 0; x < C::STAGES && x < mine; ++x) load(x);

    // The queries as the A operand (negated for a negative scale, so that the
    // factor below is positive). e4m3 caches multiply in f16, which holds every
    // code; the query row is brought to [2^14, 2^15) by a power of two first, so
    // that what f16 cannot hold of it lies 2^-39 below its largest element.
    uint32_t qa[C::KS][4];
    float c[H];  // per row: |scale| log2(e), and for e4m3 the inverse of the row's power of two
    unsigned long long word[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int row = min(row0 + g + 8 * h, p.rows - 1);
      const __nv_bfloat16* q = p.q + (static_cast<size_t>(bh) * p.rows + row) * D;
      const uint32_t sign = p.c < 0.f ? 0x80008000u : 0u;
      word[h] = tree_word(p, part.b, row);
      c[h] = fmaxf(fabsf(p.c), 1e-30f);  // (scale 0: 0 times the -inf of a masked score would be NaN)
      if constexpr (Q8) {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < C::KS; ++s) {
          const int at = D == 128 ? 16 * (t + 4 * (s >> 2)) + 4 * (s & 3) : D == 64 ? 16 * t + 4 * s : 8 * t + 4 * s;
          const uint2 u = *reinterpret_cast<const uint2*>(q + at);
          qa[s][h] = u.x ^ sign;
          qa[s][2 + h] = u.y ^ sign;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t w = qa[s][2 * e + h], lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
            top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
          }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t up = 268u - max(top >> 7, 15u);
        const float f = __uint_as_float(up << 23);
        c[h] = fmaxf(c[h] * __uint_as_float((254u - up) << 23), 1e-37f);
#pragma unroll
        for (int s = 0; s < C::KS; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 x = unpack_bf16x2(qa[s][2 * e + h]);
            qa[s][2 * e + h] = pack_f16x2(x.x * f, x.y * f);
          }
      } else {
#pragma unroll
        for (int s = 0; s < C::KS; ++s) {
          qa[s][h] = *reinterpret_cast<const uint32_t*>(q + 16 * s + 2 * t) ^ sign;
          qa[s][2 + h] = *reinterpret_cast<const uint32_t*>(q + 16 * s + 8 + 2 * t) ^ sign;
        }
      }
    }
    // keys of score columns 2t and 2t + 1 within a group of eight
    const int ka = Q8 ? key_of<D>(2 * t) : 2 * t, kb = Q8 ? key_of<D>(2 * t + 1) : 2 * t + 1;

    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float m[H], l[H];  // l: this thread's columns only
#pragma unroll
    for (int h = 0; h < H; ++h) m[h] = -INFINITY, l[h] = 0.f;

    // e4m3: lane j holds the scale bytes of key j of the tile, read one tile
    // ahead. V's scales go into the weights, relative to the largest met so far
    // (`top_v`), so that the weights fit f16: p 2^(e - top_v) 2^15.
    int ke = 0, ve = 0, top_v = 0;
    auto scales = [&](int x) {
      const int key = key0 + x * C::BN + lane;
      const bool in = x < mine && key < L;
      const size_t at = static_cast<size_t>(bh) * p.m + key;
      ke = in ? __ldg(p.k_exp + at) : 0;
      ve = in ? __ldg(p.v_exp + at) : 0;
    };
    if constexpr (Q8) scales(0);

    int x = 0;
    for (; x < mine; ++x) {
      const int st = (turn + x) % C::STAGES;
      const int k0 = key0 + x * C::BN;
      const uint8_t* sk = ring + st * 2 * C::KT;
      const uint8_t* sv = sk + C::KT;
      const uint32_t ak = smem_u32(sk), av = smem_u32(sv);
      float fk = 1.f, fv = 1.f, back = 1.f;
      if constexpr (Q8) {
        fk = pow2_of_byte(ke);
        const int top = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(ve)));
        if (top > top_v) {
          back = ex2_approx(static_cast<float>(top_v - top));  // (an empty product before the first: any factor)
          top_v = top;
        }
        const int e = ve - top_v + 127 + 15;
        fv = e > 0 ? __uint_as_float(static_cast<uint32_t>(e) << 23) : 0.f;
        scales(x + 1);
      }
      if (!__all_sync(0xffffffffu, tree_wait(&full[warp][st], ((turn + x) / C::STAGES) & 1, abort_flag, wd))) break;

      // scores of the tile's keys
      float s[C::NT][4];
#pragma unroll
      for (int i = 0; i < C::NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
      if constexpr (Q8) {
#pragma unroll
        for (int i = 0; i < C::NT; ++i) {
          uint32_t w[C::KS];
          key_words<D>(sk, i * 8 + key_of<D>(g), t, w);
#pragma unroll
          for (int k = 0; k < C::KS; ++k)
            mma_f16(s[i], qa[k], e4m3_to_f16x2(w[k] & 0xffffu), e4m3_to_f16x2(w[k] >> 16));
        }
      } else {
#pragma unroll
        for (int k = 0; k < C::KS; k += 2)
#pragma unroll
          for (int i = 0; i < C::NT; ++i) {
            uint32_t w[4];
            ldsm4(ak + tile_off<D, false>(i * 8 + (lane & 7), (2 * k + (lane >> 3)) * 16), w);
            mma_bf16(s[i], qa[k], w[0], w[1]);
            mma_bf16(s[i], qa[k + 1], w[2], w[3]);
          }
      }
      // the keys' scales, and the mask where the tile reaches past the positions that every row sees
      const bool tail = k0 + C::TK > old;
      float top[H];
#pragma unroll
      for (int h = 0; h < H; ++h) top[h] = -INFINITY;
#pragma unroll
      for (int i = 0; i < C::NT; ++i) {
        if constexpr (Q8) {
          const float fa = __shfl_sync(0xffffffffu, fk, i * 8 + ka), fb = __shfl_sync(0xffffffffu, fk, i * 8 + kb);
#pragma unroll
          for (int h = 0; h < H; ++h) s[i][2 * h] *= fa, s[i][2 * h + 1] *= fb;
        }
        if (tail) {
          const int ja = k0 + i * 8 + ka, jb = k0 + i * 8 + kb;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            if (!sees(word[h], ja, old, L)) s[i][2 * h] = -INFINITY;
            if (!sees(word[h], jb, old, L)) s[i][2 * h + 1] = -INFINITY;
          }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) top[h] = fmaxf(top[h], fmaxf(s[i][2 * h], s[i][2 * h + 1]));
      }
      bool grew = Q8 && back != 1.f;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2)) * c[h];  // in units of log2
        grew |= top[h] > m[h];
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float n = fmaxf(m[h], top[h]);
          const float f = ex2_approx(m[h] - (n == -INFINITY ? 0.f : n));
          m[h] = n;
          l[h] *= f;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            acc[i][2 * h] *= f * back;
            acc[i][2 * h + 1] *= f * back;
          }
        }
      }
      float ref[H];  // nothing seen yet: weights 0
#pragma unroll
      for (int h = 0; h < H; ++h) ref[h] = m[h] == -INFINITY ? 0.f : m[h];

      // weights and P V, 16 keys at a time. The weights are rounded to the
      // caches' product type: bf16 (2^-9 of a weight), f16 for e4m3 (2^-12).
      bool odd = false;
#pragma unroll
      for (int kk = 0; kk < C::TK / 16; ++kk) {
        uint32_t pa[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float* si = s[2 * kk + u];
          float fa = 1.f, fb = 1.f;
          if constexpr (Q8) {
            fa = __shfl_sync(0xffffffffu, fv, (2 * kk + u) * 8 + ka);
            fb = __shfl_sync(0xffffffffu, fv, (2 * kk + u) * 8 + kb);
          }
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const float w0 = ex2_approx(fmaf(si[2 * h], c[h], -ref[h]));
            const float w1 = ex2_approx(fmaf(si[2 * h + 1], c[h], -ref[h]));
            l[h] += w0 + w1;
            pa[2 * u + h] = Q8 ? pack_f16x2(w0 * fa, w1 * fb) : pack_bf16x2(w0, w1);
          }
        }
        if constexpr (Q8) {
          constexpr int W = D / 32;  // words of this thread's columns in a row
          uint32_t w[4][W];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            value_words<D>(sv, kk * 16 + (u >> 1) * 8 + ((u & 1) ? kb : ka), g, w[u]);
          if (tail) {
            // NaN codes may not enter a product here: a weight of 0 would make
            // them NaN for rows that do not see them
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int i = 0; i < W; ++i) {
                const uint32_t n = nan_codes(w[u][i]) & 0x80808080u;
                if (n != 0) {
                  odd = true;
                  w[u][i] &= ~((n >> 7) * 0xffu);
                }
              }
          }
#pragma unroll
          for (int i = 0; i < W; ++i) {
            // codes of the keys of columns 2t, 2t + 1 side by side, then of 2t + 8, 2t + 9
            const uint32_t a0 = __byte_perm(w[0][i], w[1][i], 0x5140), a1 = __byte_perm(w[0][i], w[1][i], 0x7362);
            const uint32_t b0 = __byte_perm(w[2][i], w[3][i], 0x5140), b1 = __byte_perm(w[2][i], w[3][i], 0x7362);
            mma_f16(acc[4 * i], pa, e4m3_to_f16x2(a0 & 0xffffu), e4m3_to_f16x2(b0 & 0xffffu));
            mma_f16(acc[4 * i + 1], pa, e4m3_to_f16x2(a0 >> 16), e4m3_to_f16x2(b0 >> 16));
            mma_f16(acc[4 * i + 2], pa, e4m3_to_f16x2(a1 & 0xffffu), e4m3_to_f16x2(b1 & 0xffffu));
            mma_f16(acc[4 * i + 3], pa, e4m3_to_f16x2(a1 >> 16), e4m3_to_f16x2(b1 >> 16));
          }
        } else {
          const int base = k0 + kk * 16;
          const bool ra = base + ka < L, rb = base + kb < L, rc = base + 8 + ka < L, rd = base + 8 + kb < L;
#pragma unroll
          for (int i = 0; i < D / 8; i += 2) {
            uint32_t v[4];
            ldsm4_t(av + tile_off<D, false>(kk * 16 + (lane & 15), (i + (lane >> 4)) * 16), v);
            if (tail) {
              v[0] = clean_pair(v[0], ra, rb, odd);
              v[1] = clean_pair(v[1], rc, rd, odd);
              v[2] = clean_pair(v[2], ra, rb, odd);
              v[3] = clean_pair(v[3], rc, rd, odd);
            }
            mma_bf16(acc[i], pa, v[0], v[1]);
            mma_bf16(acc[i + 1], pa, v[2], v[3]);
          }
        }
      }
      if (tail && __any_sync(0xffffffffu, odd)) {
        // values left out above that are not finite: only for the rows that see them
#pragma unroll 1
        for (int j = 0; j < C::TK; ++j)
#pragma unroll
          for (int h = 0; h < H; ++h)
            if (sees(word[h], k0 + j, old, L))
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float v = value_at<D, Q8>(sv, j, Q8 ? col_of<D>(2 * t + e) * (D / 8) + i : i * 8 + 2 * t + e);
                  if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u) acc[i][2 * h + e] += v;
                }
      }
      __syncwarp();
      if (lane == 0 && x + C::STAGES < mine) {
        fence_proxy_async_smem();  // the warp's reads of the stage come before the TMA write
        load(x + C::STAGES);
      }
    }
    if (x < mine && lane == 0)  // the watchdog fired: let the tiles in flight land
      for (int y = x; y < x + C::STAGES && y < mine; ++y)
        tree_drain(&full[warp][(turn + y) % C::STAGES], ((turn + y) / C::STAGES) & 1, wd);
    // join the four warps' results; every load has landed
    if (__syncthreads_or(x < mine)) return;
    float* so = reinterpret_cast<float*>(smem) + warp * (kTreeRows * C::OST);
    const float unit_v = Q8 ? pow2_of_byte(top_v) * 0x1p-15f : 1.f;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      // a row whose every score was NaN has no maximum: its sum is NaN, against the reference 0
      if (m[h] == -INFINITY && l[h] != 0.f) m[h] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          so[(g + 8 * h) * C::OST + (Q8 ? col_of<D>(2 * t + e) * (D / 8) + i : i * 8 + 2 * t + e)] =
              acc[i][2 * h + e] * unit_v;
      if (t == 0) {
        s_m[warp][g + 8 * h] = m[h];
        s_l[warp][g + 8 * h] = l[h];
      }
    }
    __syncthreads();
    tree_join<D, kTreeRows>(p, part, reinterpret_cast<const float*>(smem), s_m, s_l, row0);
    turn += mine;
    fence_proxy_async_smem();  // the results in the ring come before the next part's TMA writes
    __syncthreads();
  }
}

// At most 8 query rows a key head (decoding of one token, mostly): the products
// the other way round, 16 keys (or 16 output columns) against 8 query rows, so that
// no part of a product is idle. Half as many products as above and half the
// registers for O; the weights are turned from (key, row) to (row, key) by an
// 8 x 8 transposition in registers. Bound by reading the caches. (64 sequences of up
// to 4096 positions, 16 heads of one row, d = 64, e4m3: 64 us, 69 with the kernel
// above, reading alone 51; 32 such of bf16: 83, 90, 79. d = 32, e4m3: 57 us with 64 keys
// a warp's tile, 65 with 32; d = 64: 64 with either.)
template <int D, bool Q8>
struct Few : Tree<D, Q8> {
  using T = Tree<D, Q8>;
  static constexpr int CTAS = D == 128 ? 2 : Q8 ? 4 : 5;   // per SM
  static constexpr int TK = Q8 && D == 32 ? 64 : T::TK;    // keys per tile of a warp
  static constexpr uint32_t KT = TK * D * T::ES;           // one K (or V) tile
  static constexpr int BN = kTreeWarps * TK;               // keys of a CTA's tile
  static constexpr int NG = TK / 16;                       // groups of 16 keys in a warp's tile
  static constexpr int NB = Q8 ? TK / 32 : 1;              // scale bytes of a lane
  static constexpr int ND = D / 16;                        // groups of 16 output columns
  static constexpr uint32_t RING = kTreeWarps * T::STAGES * 2 * KT;
  static constexpr uint32_t JOIN = kTreeWarps * 8 * T::OST * 4;
  static constexpr uint32_t SMEM = (RING > JOIN ? RING : JOIN) + 1024;
};

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D, bool Q8>
__global__ void __launch_bounds__(kTreeThreads, Few<D, Q8>::CTAS)
attn_tree_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const TreeParams p) {
  using C = Few<D, Q8>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kTreeWarps][C::STAGES];
  __shared__ int abort_word;
  __shared__ float s_m[kTreeWarps][8], s_l[kTreeWarps][8];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  volatile int* abort_flag = &abort_word;
  const Watchdog wd = p.wd;
  grid_follow();
  TreeWalk walk;
  if (!tree_start(p, C::BN, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), walk)) return;
  if (tid == 0) {
    for (int w = 0; w < kTreeWarps; ++w)
      for (int s = 0; s < C::STAGES; ++s) mbar_init(&full[w][s], 1);
    abort_word = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  __syncthreads();
  uint8_t* ring = smem + warp * (C::STAGES * 2 * C::KT);
  int turn = 0;  // tiles this warp has put through its ring
  TreePart part;
#pragma unroll 1
  while (tree_next(p, C::BN, walk, part)) {
    const int bh = part.bh, L = part.L;
    const int old = L - p.n;             // positions before the newest n (negative: fewer cached than n)
    const int mine = part.t1 - part.t0;  // of every tile this warp takes keys [warp TK, warp TK + TK)
    const int key0 = part.t0 * C::BN + warp * C::TK;
    auto load = [&](int x) {
      const int st = (turn + x) % C::STAGES;
      const int k0 = key0 + x * C::BN;
      uint8_t* dst = ring + st * 2 * C::KT;
      mbar_arrive_expect_tx(&full[warp][st], 2 * C::KT);
      for (int a = 0; a < C::NBOX; ++a) {
        tma_load_3d(dst + a * C::BOX, &tm_k, &full[warp][st], a * (C::ROWB / C::ES), k0, bh);
        tma_load_3d(dst + C::KT + a * C::BOX, &tm_v, &full[warp][st], a * (C::ROWB / C::ES), k0, bh);
      }
    };
    if (lane == 0)
      for (int x = 0; x < C::STAGES && x < mine; ++x) load(x);

    // Row g of the queries as the B operand, in the types and scales of the kernel
    // above. What the softmax needs of a row, the threads of rows 2t, 2t + 1 have.
    uint32_t qb[C::KS][2];
    float c[2];
    unsigned long long word[2];
    {
      const __nv_bfloat16* q = p.q + (static_cast<size_t>(bh) * p.rows + min(g, p.rows - 1)) * D;
      const uint32_t sign = p.c < 0.f ? 0x80008000u : 0u;
      float mine_c = fmaxf(fabsf(p.c), 1e-30f);  // (scale 0: 0 times the -inf of a masked score would be NaN)
      if constexpr (Q8) {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < C::KS; ++s) {
          const int at = D == 128 ? 16 * (t + 4 * (s >> 2)) + 4 * (s & 3) : D == 64 ? 16 * t + 4 * s : 8 * t + 4 * s;
          const uint2 u = *reinterpret_cast<const uint2*>(q + at);
          qb[s][0] = u.x ^ sign;
          qb[s][1] = u.y ^ sign;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t lo = qb[s][e] & 0x7fffu, hi = (qb[s][e] >> 16) & 0x7fffu;
            top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
          }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t up = 268u - max(top >> 7, 15u);
        const float f = __uint_as_float(up << 23);
        mine_c = fmaxf(mine_c * __uint_as_float((254u - up) << 23), 1e-37f);
#pragma unroll
        for (int s = 0; s < C::KS; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 x = unpack_bf16x2(qb[s][e]);
            qb[s][e] = pack_f16x2(x.x * f, x.y * f);
          }
      } else {
#pragma unroll
        for (int s = 0; s < C::KS; ++s) {
          qb[s][0] = *reinterpret_cast<const uint32_t*>(q + 16 * s + 2 * t) ^ sign;
          qb[s][1] = *reinterpret_cast<const uint32_t*>(q + 16 * s + 8 + 2 * t) ^ sign;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        c[h] = __shfl_sync(0xffffffffu, mine_c, 4 * (2 * t + h));
        word[h] = tree_word(p, part.b, min(2 * t + h, p.rows - 1));
      }
    }
    // this thread's keys within a group of 16 scores: kg, kg + 8; within 16 of V: ka, kb, ka + 8, kb + 8
    const int kg = Q8 ? key_of<D>(g) : g;
    const int ka = Q8 ? key_of<D>(2 * t) : 2 * t, kb = Q8 ? key_of<D>(2 * t + 1) : 2 * t + 1;

    float acc[C::ND][4];  // columns (two), rows 2t and 2t + 1
#pragma unroll
    for (int i = 0; i < C::ND; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // l: this thread's keys only

    // e4m3: the scale bytes as above, of keys j, j + 32
    int ke[C::NB], ve[C::NB], top_v = 0;
    auto scales = [&](int x) {
#pragma unroll
      for (int u = 0; u < C::NB; ++u) {
        const int key = key0 + x * C::BN + u * 32 + lane;
        const bool in = x < mine && key < L;
        const size_t at = static_cast<size_t>(bh) * p.m + key;
        ke[u] = in ? __ldg(p.k_exp + at) : 0;
        ve[u] = in ? __ldg(p.v_exp + at) : 0;
      }
    };
    if constexpr (Q8) scales(0);

    int x = 0;
    for (; x < mine; ++x) {
      const int st = (turn + x) % C::STAGES;
      const int k0 = key0 + x * C::BN;
      const uint8_t* sk = ring + st * 2 * C::KT;
      const uint8_t* sv = sk + C::KT;
      const uint32_t ak = smem_u32(sk), av = smem_u32(sv);
      float fk[C::NB], fv[C::NB], back = 1.f;
      if constexpr (Q8) {
        int top = ve[0];
#pragma unroll
        for (int u = 1; u < C::NB; ++u) top = max(top, ve[u]);
        top = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(top)));
        if (top > top_v) {
          back = ex2_approx(static_cast<float>(top_v - top));  // (an empty product before the first: any factor)
          top_v = top;
        }
#pragma unroll
        for (int u = 0; u < C::NB; ++u) {
          fk[u] = pow2_of_byte(ke[u]);
          const int e = ve[u] - top_v + 127 + 15;
          fv[u] = e > 0 ? __uint_as_float(static_cast<uint32_t>(e) << 23) : 0.f;
        }
        scales(x + 1);
      }
      if (!__all_sync(0xffffffffu, tree_wait(&full[warp][st], ((turn + x) / C::STAGES) & 1, abort_flag, wd))) break;

      // scores of the tile's keys
      float s[C::NG][4];
#pragma unroll
      for (int i = 0; i < C::NG; ++i) {
        s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
        if constexpr (Q8) {
          uint32_t w0[C::KS], w1[C::KS];
          key_words<D>(sk, i * 16 + kg, t, w0);
          key_words<D>(sk, i * 16 + 8 + kg, t, w1);
#pragma unroll
          for (int k = 0; k < C::KS; ++k) {
            const uint32_t a[4] = {e4m3_to_f16x2(w0[k] & 0xffffu), e4m3_to_f16x2(w1[k] & 0xffffu),
                                   e4m3_to_f16x2(w0[k] >> 16), e4m3_to_f16x2(w1[k] >> 16)};
            mma_f16(s[i], a, qb[k][0], qb[k][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < C::KS; ++k) {
            uint32_t a[4];
            ldsm4(ak + tile_off<D, false>(i * 16 + (lane & 15), (2 * k + (lane >> 4)) * 16), a);
            mma_bf16(s[i], a, qb[k][0], qb[k][1]);
          }
        }
      }
      // the keys' scales, and the mask where the tile reaches past the positions that every row sees
      const bool tail = k0 + C::TK > old;
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < C::NG; ++i) {
        if constexpr (Q8) {
          const float f0 = __shfl_sync(0xffffffffu, fk[i / 2], (i & 1) * 16 + kg);
          const float f1 = __shfl_sync(0xffffffffu, fk[i / 2], (i & 1) * 16 + 8 + kg);
          s[i][0] *= f0, s[i][1] *= f0, s[i][2] *= f1, s[i][3] *= f1;
        }
        if (tail) {
          const int j = k0 + i * 16 + kg;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!sees(word[h], j, old, L)) s[i][h] = -INFINITY;
            if (!sees(word[h], j + 8, old, L)) s[i][2 + h] = -INFINITY;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) top[h] = fmaxf(top[h], fmaxf(s[i][h], s[i][2 + h]));
      }
      bool grew = Q8 && back != 1.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], o));
        top[h] *= c[h];  // in units of log2
        grew |= top[h] > m[h];
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float n = fmaxf(m[h], top[h]);
          const float f = ex2_approx(m[h] - (n == -INFINITY ? 0.f : n));
          m[h] = n;
          l[h] *= f;
#pragma unroll
          for (int i = 0; i < C::ND; ++i) {
            acc[i][h] *= f * back;
            acc[i][2 + h] *= f * back;
          }
        }
      }
      float ref[2];  // nothing seen yet: weights 0
#pragma unroll
      for (int h = 0; h < 2; ++h) ref[h] = m[h] == -INFINITY ? 0.f : m[h];

      // weights (rounded as above) and V^T P^T, 16 keys at a time
      bool odd = false;
#pragma unroll
      for (int i = 0; i < C::NG; ++i) {
        float f0 = 1.f, f1 = 1.f, w[4];
        if constexpr (Q8) {
          f0 = __shfl_sync(0xffffffffu, fv[i / 2], (i & 1) * 16 + kg);
          f1 = __shfl_sync(0xffffffffu, fv[i / 2], (i & 1) * 16 + 8 + kg);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[h] = ex2_approx(fmaf(s[i][h], c[h], -ref[h]));
          w[2 + h] = ex2_approx(fmaf(s[i][2 + h], c[h], -ref[h]));
          l[h] += w[h] + w[2 + h];
        }
        const uint32_t p0 = transposed(Q8 ? pack_f16x2(w[0] * f0, w[1] * f0) : pack_bf16x2(w[0], w[1]));
        const uint32_t p1 = transposed(Q8 ? pack_f16x2(w[2] * f1, w[3] * f1) : pack_bf16x2(w[2], w[3]));
        if constexpr (Q8) {
          constexpr int W = D / 32;  // words of this thread's columns in a row
          uint32_t v[4][W];
#pragma unroll
          for (int u = 0; u < 4; ++u) value_words<D>(sv, i * 16 + (u >> 1) * 8 + ((u & 1) ? kb : ka), g, v[u]);
          if (tail) {
            // NaN codes may not enter a product here: a weight of 0 would make
            // them NaN for rows that do not see them
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int j = 0; j < W; ++j) {
                const uint32_t n = nan_codes(v[u][j]) & 0x80808080u;
                if (n != 0) {
                  odd = true;
                  v[u][j] &= ~((n >> 7) * 0xffu);
                }
              }
          }
#pragma unroll
          for (int j = 0; j < W; ++j) {
            // codes of the keys of columns 2t, 2t + 1 side by side, then of 2t + 8, 2t + 9
            const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5140), a1 = __byte_perm(v[0][j], v[1][j], 0x7362);
            const uint32_t b0 = __byte_perm(v[2][j], v[3][j], 0x5140), b1 = __byte_perm(v[2][j], v[3][j], 0x7362);
            const uint32_t lo[4] = {e4m3_to_f16x2(a0 & 0xffffu), e4m3_to_f16x2(a0 >> 16), e4m3_to_f16x2(b0 & 0xffffu),
                                    e4m3_to_f16x2(b0 >> 16)};
            const uint32_t hi[4] = {e4m3_to_f16x2(a1 & 0xffffu), e4m3_to_f16x2(a1 >> 16), e4m3_to_f16x2(b1 & 0xffffu),
                                    e4m3_to_f16x2(b1 >> 16)};
            mma_f16(acc[2 * j], lo, p0, p1);
            mma_f16(acc[2 * j + 1], hi, p0, p1);
          }
        } else {
          const int base = k0 + i * 16;
          const bool ra = base + ka < L, rb = base + kb < L, rc = base + 8 + ka < L, rd = base + 8 + kb < L;
#pragma unroll
          for (int j = 0; j < C::ND; ++j) {
            uint32_t v[4];
            const int r = i * 16 + (lane & 7) + 8 * (lane >> 4);
            ldsm4_t(av + tile_off<D, false>(r, (2 * j + ((lane >> 3) & 1)) * 16), v);
            if (tail) {
              v[0] = clean_pair(v[0], ra, rb, odd);
              v[1] = clean_pair(v[1], ra, rb, odd);
              v[2] = clean_pair(v[2], rc, rd, odd);
              v[3] = clean_pair(v[3], rc, rd, odd);
            }
            mma_bf16(acc[j], v, p0, p1);
          }
        }
      }
      // column of acc[i][2 e + h]
      auto column = [&](int i, int e) { return Q8 ? col_of<D>(g) * (D / 8) + 2 * i + e : i * 16 + g + 8 * e; };
      if (tail && __any_sync(0xffffffffu, odd)) {
        // values left out above that are not finite: only for the rows that see them
#pragma unroll 1
        for (int j = 0; j < C::TK; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (sees(word[h], k0 + j, old, L))
#pragma unroll
              for (int i = 0; i < C::ND; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float v = value_at<D, Q8>(sv, j, column(i, e));
                  if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u) acc[i][2 * e + h] += v;
                }
      }
      __syncwarp();
      if (lane == 0 && x + C::STAGES < mine) {
        fence_proxy_async_smem();  // the warp's reads of the stage come before the TMA write
        load(x + C::STAGES);
      }
    }
    if (x < mine && lane == 0)  // the watchdog fired: let the tiles in flight land
      for (int y = x; y < x + C::STAGES && y < mine; ++y)
        tree_drain(&full[warp][(turn + y) % C::STAGES], ((turn + y) / C::STAGES) & 1, wd);
    // join the four warps' results; every load has landed
    if (__syncthreads_or(x < mine)) return;
    float* so = reinterpret_cast<float*>(smem) + warp * (8 * C::OST);
    const float unit_v = Q8 ? pow2_of_byte(top_v) * 0x1p-15f : 1.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
      // a row whose every score was NaN has no maximum: its sum is NaN, against the reference 0
      if (m[h] == -INFINITY && l[h] != 0.f) m[h] = 0.f;
#pragma unroll
      for (int i = 0; i < C::ND; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = Q8 ? col_of<D>(g) * (D / 8) + 2 * i + e : i * 16 + g + 8 * e;
          so[(2 * t + h) * C::OST + col] = acc[i][2 * e + h] * unit_v;
        }
      if (g == 0) {
        s_m[warp][2 * t + h] = m[h];
        s_l[warp][2 * t + h] = l[h];
      }
    }
    __syncthreads();
    tree_join<D, 8>(p, part, reinterpret_cast<const float*>(smem), s_m, s_l, 0);
    turn += mine;
    fence_proxy_async_smem();  // the results in the ring come before the next part's TMA writes
    __syncthreads();
  }
}

// Joins the parts of a unit's rows, rescaled to the common maximum and added in
// the line's order. Partial O lies as the step's threads write it without gaps:
//   mma.sync kernel   [slot][row][d]: a warp joins one row, lanes over the columns;
//   tcgen05 kernel    [slot][d / 4][row][4]: a lane joins one row, warps over the columns.
struct UnitParts {
  int first, parts;  // the first CTA that holds a part of the unit, and how many do
};

// Every lane of a warp calls this.
__device__ __forceinline__ UnitParts unit_parts(const TreeParams& p, const TreeLine& l, int unit, int bn) {
  const int lane = threadIdx.x & 31;
  const int b = unit / l.per_seq, idx = unit - b * l.per_seq;
  const int tiles = tiles_of(tree_len(p, b), bn);
  long long first = static_cast<long long>(b) * p.lead;  // where the unit's tiles begin on the line
  if (p.kv_len == nullptr) {
    first += static_cast<long long>(b) * tiles;
  } else {
    if (lane != 0) first = 0;
    for (int x = lane; x < b; x += 32) first += tiles_of(tree_len(p, x), bn);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) first += __shfl_xor_sync(0xffffffffu, first, o);
  }
  first = first * l.per_seq + static_cast<long long>(idx) * (tiles + p.lead) + p.lead;
  // the CTAs that hold its first and its last tile: the largest c with U c / ctas at or before them
  const int c0 = static_cast<int>(((first + 1) * l.ctas - 1) / l.U);
  const int c1 = static_cast<int>(((first + tiles) * l.ctas - 1) / l.U);
  return UnitParts{c0, c1 - c0 + 1};
}

// (The blocks wait beside the step's; they do not let the next kernel's in as early:
// a step right behind then took 83 us instead of 64, 64 sequences of 16 heads, e4m3.)
//
// A long cache of few heads has hundreds of parts a unit: so `group` warps share a
// row's (or 32 rows') parts, each joins every group-th of them, and the group's results
// are joined in shared memory. (One sequence of 40000 positions, one key head of 8 rows, d =
// 128, e4m3: 15 us; with one warp for all parts of a row 85.)
constexpr int kMergeWarps = 16;

// Grid: x = unit, y = kMergeWarps / group rows of its block (or fewer, where it has fewer).
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) attn_tree_merge_kernel(const TreeParams p, int bn, int grid,
                                                                           int group) {
  constexpr int PER = D / 32;
  extern __shared__ float4 merge_smem[];  // (none where a warp has all parts: the blocks wait beside the step's)
  float (*s_o)[D] = reinterpret_cast<float (*)[D]>(merge_smem);
  float2* s_ml = reinterpret_cast<float2*>(s_o[kMergeWarps]);
  const TreeLine l = tree_line(p, bn, grid);
  const int unit = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const UnitParts u = unit_parts(p, l, unit, bn);
  grid_wait();  // the parts are written
  if (u.parts == 1) return;  // one part: its CTA wrote the results
  const int rows = static_cast<int>(blockDim.x >> 5) / group, w = warp % group;
  const int r = blockIdx.y * rows + warp / group;
  const int row = (unit % p.row_blocks) * p.block_rows + r;
  const bool live = r < p.block_rows && row < p.rows;
  const size_t step = static_cast<size_t>(p.block_rows), at = (static_cast<size_t>(unit) + u.first) * step + r;
  float m = -INFINITY, sum = 0.f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.f;
  const int count = live ? (u.parts - w + group - 1) / group : 0;  // parts w, w + group, ...
  for (int base = 0; base < count; base += 32) {
    // a lane's part: its weight against the maximum so far (0 without a key that the row sees)
    float2 ml = make_float2(-INFINITY, 0.f);
    if (base + lane < count) {
      const size_t mine = at + static_cast<size_t>(w + (base + lane) * group) * step;
      ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * mine);
    }
    float top = ml.x;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    if (top > m) {
      const float f = ex2_approx(m - top);
      m = top;
      sum *= f;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] *= f;
    }
    const float weight = m == -INFINITY ? 0.f : ex2_approx(ml.x - m);
    float t = weight * ml.y;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
    sum += t;
    const int n = min(32, count - base);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float f = __shfl_sync(0xffffffffu, weight, k);
      const float* src = p.part + (at + static_cast<size_t>(w + (base + k) * group) * step) * D + lane;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] = fmaf(f, src[32 * i], o[i]);
    }
  }
  if (group > 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) s_o[warp][lane + 32 * i] = o[i];
    if (lane == 0) s_ml[warp] = make_float2(m, sum);
    __syncthreads();
    if (w != 0) return;
    for (int k = 1; k < group; ++k) m = fmaxf(m, s_ml[warp + k].x);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = 0.f;
    for (int k = 0; k < group; ++k) {
      const float f = m == -INFINITY ? 0.f : ex2_approx(s_ml[warp + k].x - m);
      sum = fmaf(f, s_ml[warp + k].y, sum);
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] = fmaf(f, s_o[warp + k][lane + 32 * i], o[i]);
    }
  }
  if (!live) return;
  const float inv = m == -INFINITY ? 0.f : 1.f / sum;
  const size_t out = static_cast<size_t>(unit / p.row_blocks) * p.rows + row;
#pragma unroll
  for (int i = 0; i < PER; ++i) p.o[out * D + lane + 32 * i] = __float2bfloat16_rn(o[i] * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[out] = m == -INFINITY ? -INFINITY : (m + log2f(sum)) * kTreeLn2;
}

// Grid: x = unit, y = 32 rows of its block (a lane a row), z = as many of the eight
// groups of D / 8 columns as the block has groups of warps.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) attn_tree_tc_merge_kernel(const TreeParams p, int bn, int grid,
                                                                              int group) {
  constexpr int C4 = D / 32;  // groups of four columns
  extern __shared__ float4 merge_smem[];
  float4 (*s_o)[C4][32] = reinterpret_cast<float4 (*)[C4][32]>(merge_smem);
  float2 (*s_ml)[32] = reinterpret_cast<float2 (*)[32]>(s_o[kMergeWarps]);
  const TreeLine l = tree_line(p, bn, grid);
  const int unit = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const UnitParts u = unit_parts(p, l, unit, bn);
  grid_wait();
  if (u.parts == 1) return;
  const int w = warp % group, cols = (blockIdx.z * static_cast<int>(blockDim.x >> 5) + warp) / group;
  const int r = blockIdx.y * 32 + lane;
  const int row = (unit % p.row_blocks) * p.block_rows + r;
  const size_t step = static_cast<size_t>(p.block_rows), slot = static_cast<size_t>(unit) + u.first;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + slot * step + r;
  float M = -INFINITY, sum = 0.f;
  float4 o[C4];
#pragma unroll
  for (int i = 0; i < C4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row < p.rows) {
#pragma unroll 4
    for (int s = w; s < u.parts; s += group) M = fmaxf(M, ml[s * step].x);
    if (M != -INFINITY) {
      const float4* part = reinterpret_cast<const float4*>(p.part) + (slot * (D / 4) + cols * C4) * step + r;
#pragma unroll 2
      for (int s = w; s < u.parts; s += group) {
        const float2 x = ml[s * step];
        const float f = ex2_approx(x.x - M);
        sum = fmaf(f, x.y, sum);
#pragma unroll
        for (int i = 0; i < C4; ++i) {
          const float4 v = part[(static_cast<size_t>(s) * (D / 4) + i) * step];
          o[i].x = fmaf(f, v.x, o[i].x);
          o[i].y = fmaf(f, v.y, o[i].y);
          o[i].z = fmaf(f, v.z, o[i].z);
          o[i].w = fmaf(f, v.w, o[i].w);
        }
      }
    }
  }
  const size_t out = static_cast<size_t>(unit / p.row_blocks) * p.rows + row;
  auto write = [&](int i, const float4& x, float inv) {
    *reinterpret_cast<uint2*>(p.o + out * D + cols * (D / 8) + i * 4) =
        make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
  };
  if (group == 1) {
    if (row >= p.rows) return;
    const float inv = M == -INFINITY ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < C4; ++i) write(i, o[i], inv);
  } else {
#pragma unroll
    for (int i = 0; i < C4; ++i) s_o[warp][i][lane] = o[i];
    s_ml[warp][lane] = make_float2(M, sum);
    __syncthreads();
    if (row >= p.rows) return;
    const int first = warp - w;
    for (int k = 0; k < group; ++k) M = fmaxf(M, s_ml[first + k][lane].x);
    auto factor = [&](int k) { return M == -INFINITY ? 0.f : ex2_approx(s_ml[first + k][lane].x - M); };
    sum = 0.f;
    for (int k = 0; k < group; ++k) sum = fmaf(factor(k), s_ml[first + k][lane].y, sum);
    const float inv = M == -INFINITY ? 0.f : 1.f / sum;
    for (int i = w; i < C4; i += group) {  // a warp of the group joins four columns
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < group; ++k) {
        const float f = factor(k);
        const float4 v = s_o[first + k][i][lane];
        x.x = fmaf(f, v.x, x.x);
        x.y = fmaf(f, v.y, x.y);
        x.z = fmaf(f, v.z, x.z);
        x.w = fmaf(f, v.w, x.w);
      }
      write(i, x, inv);
    }
  }
  if (cols == 0 && w == 0 && p.lse != nullptr)
    p.lse[out] = M == -INFINITY ? -INFINITY : (M + log2f(sum)) * kTreeLn2;
}

// Places of the mma.sync kernels on the GPU, and keys of a CTA's tile.
template <int D, bool Q8>
void small_shape_of(bool few, int* places, int* tile) {
  *places = kSms * (few ? Few<D, Q8>::CTAS : Tree<D, Q8>::CTAS);
  *tile = few ? Few<D, Q8>::BN : Tree<D, Q8>::BN;
}

template <int D>
void small_shape_d(bool quantised, bool few, int* places, int* tile) {
  quantised ? small_shape_of<D, true>(few, places, tile) : small_shape_of<D, false>(few, places, tile);
}

void small_shape(int d, bool quantised, bool few, int* places, int* tile) {
  switch (d) {
    case 32: return small_shape_d<32>(quantised, few, places, tile);
    case 64: return small_shape_d<64>(quantised, few, places, tile);
    default: return small_shape_d<128>(quantised, few, places, tile);
  }
}

// Which kernel: the mma.sync one multiplies with the keys of a tile once for every
// 16 rows, the tcgen05 one once for 128. Taking what the first needs for 16 rows and
// 128 keys as 1, the second was measured at `tile` for 128 keys, `start` for each
// unit it begins (e4m3: its scales are looked at first) and, where the whole step is
// so small that latency counts, `fill` more in all. (mma.sync : tcgen05 in us; 16
// sequences of 8192 positions, 8 key heads of d = 128, bf16: 16 rows 80 : 93, 32 rows
// 159 : 93; e4m3: 32 rows 91 : 94, 48 rows 133 : 95; 64 sequences of 1024, 64 rows,
// bf16 129 : 76, e4m3 112 : 107; 2 of 2000, 64 rows, bf16 19 : 21, 96 rows 23 : 22.)
bool tree_uses_tc(long long heads, int rows, int m, int d, bool quantised) {
  const double tile = d == 32 ? 2.4 : !quantised ? 1.0 : d == 64 ? 2.0 : 1.8;
  const double start = quantised ? 20.0 : 10.0, fill = d == 32 ? 3000.0 : d == 64 ? 600.0 : 1000.0;
  const double tiles = (m + 127) / 128, small = (rows + kTreeRows - 1) / kTreeRows, big = (rows + 127) / 128;
  return static_cast<double>(heads) * (small * tiles - big * (tile * tiles + start)) > fill;
}

template <int D, bool Q8, bool FEW>
cudaError_t launch_small(int grid, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                         cudaStream_t stream) {
  constexpr auto kernel = FEW ? attn_tree_few_kernel<D, Q8> : attn_tree_kernel<D, Q8>;
  constexpr uint32_t smem = FEW ? Few<D, Q8>::SMEM : Tree<D, Q8>::SMEM;
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!set[dev & 63].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    set[dev & 63].store(true, std::memory_order_relaxed);
  }
  prof_begin(kKindTree, stream);
  e = launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), dim3(kTreeThreads), smem, stream, tk, tv, p);
  prof_end(kKindTree, stream);
  return e;
}

template <int D, bool Q8>
cudaError_t launch_small_rows(int grid, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                              cudaStream_t stream) {
  return p.block_rows <= 8 ? launch_small<D, Q8, true>(grid, tk, tv, p, stream)
                           : launch_small<D, Q8, false>(grid, tk, tv, p, stream);
}

template <int D>
cudaError_t launch_tree_d(bool quantised, const TreePlan& plan, const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  cudaError_t e;
  if (plan.tc) e = launch_tree_tc(D, quantised, plan.grid, tq, tk, tv, p, stream);
  else if (quantised) e = launch_small_rows<D, true>(plan.grid, tk, tv, p, stream);
  else e = launch_small_rows<D, false>(plan.grid, tk, tv, p, stream);
  if (e != cudaSuccess || plan.by_unit) return e;
  const unsigned units = static_cast<unsigned>(p.B) * p.h_kv * p.row_blocks;
  // Warps for the parts of a unit: as many as it has on average, a power of two, from 2
  // on while the blocks do not fill the GPU. (4 sequences, 4 key heads of 512 rows: 1, 2, 8
  // warps 84, 81, 92 us; 8 sequences, 8 key heads, d = 64, where it has 1.2: 1, 2 217, 222.)
  int group = 1;
  auto blocks = [&](int g) {
    return static_cast<long long>(units) *
           (plan.tc ? p.block_rows / 32 * ((g + 1) / 2) : (p.block_rows * g + kMergeWarps - 1) / kMergeWarps);
  };
  while (group < kMergeWarps && 2ll * units * group <= plan.grid && (group == 1 || blocks(group) < kSms)) group *= 2;
  const int warps = group == 1 ? 8 : kMergeWarps;  // of a block
  const size_t smem = group == 1 ? 0 : plan.tc ? kMergeWarps * 32 * (D / 2 + 8) : kMergeWarps * (D * 4 + 8);
  prof_begin(kKindTreeMerge, stream);
  if (plan.tc) {
    const dim3 blocks_of(units, static_cast<unsigned>(p.block_rows / 32), static_cast<unsigned>(8 * group / warps));
    e = launch_dependent(attn_tree_tc_merge_kernel<D>, blocks_of, dim3(warps * 32), smem, stream, p, plan.tile,
                         plan.grid, group);
  } else {
    const int rows = std::min(p.block_rows, warps / group);  // of a block
    const dim3 blocks_of(units, static_cast<unsigned>((p.block_rows + rows - 1) / rows));
    e = launch_dependent(attn_tree_merge_kernel<D>, blocks_of, dim3(static_cast<unsigned>(rows * group * 32)), smem,
                         stream, p, plan.tile, plan.grid, group);
  }
  prof_end(kKindTreeMerge, stream);
  return e;
}

}  // namespace

TreePlan tree_plan(int B, int h_kv, int rows, int m, int d, bool quantised) {
  TreePlan l{};
  l.tc = tree_uses_tc(static_cast<long long>(B) * h_kv, rows, m, d, quantised);
  int room;
  if (l.tc) {
    l.pair = rows > 128 && d >= 64;
    l.block_rows = !l.pair ? 128 : rows > 256 ? 512 : 256;
    l.tile = 128;
    room = kSms / (l.pair ? 2 : 1);
  } else {
    l.block_rows = rows < kTreeRows ? rows : kTreeRows;
    small_shape(d, quantised, rows <= 8, &room, &l.tile);
  }
  l.row_blocks = (rows + l.block_rows - 1) / l.block_rows;
  const long long units = static_cast<long long>(B) * h_kv * l.row_blocks;
  const long long tiles = (m + l.tile - 1) / l.tile;
  // Short caches: a CTA for each unit. Else one CTA for each place (or pair of
  // places) on the GPU's SMs; fewer where the caches hold too few tiles.
  const long long blocks = (m + 127) / 128;
  l.by_unit = units <= room
                  ? blocks <= kTreeAlone && static_cast<double>(blocks) * (room - units) <= kTreeShort * room
                  : !l.tc && blocks <= kTreeAloneMany && units <= 0x7fffffffLL;
  if (l.by_unit) {
    l.grid = static_cast<int>(units);
  } else {
    l.lead = kTreeLead;
    const long long most = (units * (tiles + l.lead) + kTreeLeast - 1) / kTreeLeast;
    l.grid = static_cast<int>(most < room ? most : room);
  }
  l.slots = units + l.grid;
  return l;
}

cudaError_t launch_tree(int d, bool quantised, const TreePlan& plan, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  switch (d) {
    case 32: return launch_tree_d<32>(quantised, plan, tq, tk, tv, p, stream);
    case 64: return launch_tree_d<64>(quantised, plan, tq, tk, tv, p, stream);
    case 128: return launch_tree_d<128>(quantised, plan, tq, tk, tv, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
