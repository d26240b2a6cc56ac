// Decoding of drafted tokens with many query rows a key head (attn_tree.cu
// states the operator): tcgen05 tiles of 128 query rows against 128 keys.
//
// A CTA holds NQ tiles of 128 rows (one, or two where a key head has more than
// 128 rows, so that each K/V tile serves 256) and walks its share of the line of
// tiles (attn_tree.cuh). K and V tiles alternate through one ring of
// NB 128-key tiles in the tensor cores' layout:
//   producer    TMA loads. bf16 caches: straight into the ring. e4m3 caches:
//               the codes into a ring of their own, from which
//   converters  (4 warps, one key row a thread) write f16 values into the
//               ring, code 2^(e - top + 7) with `top` the largest scale of the
//               part's keys: so a code is converted once for all rows, one
//               conversion and one exact product for two codes, and the softmax
//               carries no scales. f16 holds them exactly down to 2^-22 of the
//               largest; below that they lose low bits, and 2^-33 becomes 0.
//               (Exact bf16 values took five operations for two codes: 64 tokens
//               with eight query heads a key head, d = 128: 119 us.)
//               The queries are brought to f16 as well, each row to [2^14, 2^15)
//               by a power of two, and the weights are f16 against a reference
//               2^7 below the maximum, so that they reach down to 2^-31 of it.
//   cleaner     (bf16) passes V tiles on; in tiles that reach the newest n
//               positions it zeroes the rows past the sequence and values that
//               are not finite (weight 0 times NaN is NaN). Rows that see such a
//               value get it added at the end. (The converters do this for e4m3.)
//   issuer g    S_g = Q_g K^T, O_g += P_g V_g, one thread a query tile.
//   softmax     one thread a row: x = S c, running maximum (O rescaled when it
//               grew by more than 2^8), p = 2^(x - m), bf16 P over S in TMEM.
// With NQ = 1 there are two S buffers, so that the next scores are computed
// during the softmax; with NQ = 2 the other tile's products fill that time.
#include "attn_tree.cuh"

#include <atomic>

namespace attn {
namespace {

using namespace sm103;

constexpr int kBN = 128;
constexpr float kGrow = 8.0f;  // log2 units a row maximum may run ahead of its reference

template <int D, int NQ, bool Q8>
struct Tc {
  static constexpr int ATOM = D >= 64 ? 64 : D;            // bf16 elements of a swizzle row
  static constexpr int NATOM = D / ATOM;
  static constexpr uint32_t SWZ = D >= 64 ? 2u : 4u;
  static constexpr uint32_t SBO = 8u * ATOM * 2u;
  static constexpr uint32_t TILE = kBN * D * 2u;           // a K, V or Q tile in bf16
  static constexpr uint32_t BOX = kBN * ATOM * 2u;
  static constexpr uint32_t RAW = Q8 ? kBN * D : 0;        // a tile of codes
  // Ring of bf16 tiles. For bf16 caches an even number, so that a place always
  // holds K or always V: the cleaner waits for V tiles only, and a place that K
  // passes through could complete two phases between its looks (a wait tells
  // phases apart by their parity alone).
  static constexpr int NB = Q8 ? (D == 128 ? 3 : 6) : (D == 128 && NQ == 2 ? 4 : 6);
  static_assert(Q8 || NB % 2 == 0, "the cleaner's waits");
  static constexpr int NR = Q8 ? (D == 128 ? (NQ == 2 ? 4 : 6) : 8) : 1;     // ring of code tiles
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_B = NQ * TILE;
  static constexpr uint32_t OFF_R = OFF_B + NB * TILE;
  static constexpr uint32_t SMEM = OFF_R + (Q8 ? NR * RAW : 0) + 1024;       // + alignment slack
  static_assert(SMEM <= 227u * 1024u, "shared memory");
  static constexpr int NS = NQ == 1 ? 2 : 1;               // S buffers of a query tile
  static constexpr int TM_O = NQ * NS * kBN;               // TMEM: S buffers, then O
  static constexpr int TMEM = TM_O + NQ * D <= 256 ? 256 : 512;
  static_assert(TM_O + NQ * D <= 512, "TMEM");
  static constexpr int SOFT = 4 * NQ;                      // softmax warps
  static constexpr int PRODUCER = SOFT, ISSUER = SOFT + 1, CLEANER = SOFT + 3;
  static constexpr int CONV = SOFT + 4;                    // converter warps (e4m3)
  static constexpr int THREADS = (SOFT + 4 + (Q8 ? 4 : 0)) * 32;
  // registers: the split must fit in what the CTA is launched with
  static constexpr bool SPLIT = THREADS > 256;
  static constexpr int R_LAUNCH = THREADS == 512 ? 128 : 168;
  static constexpr int R_SOFT = THREADS == 512 ? 184 : 208;
  static constexpr int R_CTRL = THREADS == 512 ? 48 : 72;
  static constexpr int R_CONV = !Q8 ? 0 : THREADS == 512 ? 96 : 136;
  static constexpr int R_SUM = SOFT * 32 * R_SOFT + 128 * R_CTRL + 128 * R_CONV;
  static_assert(!SPLIT || R_SUM <= R_LAUNCH * THREADS, "register split");
};

constexpr int kMaxRing = 8;

struct TcShared {
  uint64_t q_full, q_empty;
  uint64_t q_f16[2];                           // e4m3 caches: query tile g is in f16
  uint64_t scanned;                            // e4m3 caches: the part's scales were looked at
  uint64_t full[kMaxRing], empty[kMaxRing];    // bf16 tiles: filled (TMA or converters), released by the issuers
  uint64_t clean[kMaxRing];                    // bf16 caches: the V tile in this place is clean
  uint64_t raw_full[kMaxRing], raw_empty[kMaxRing];
  uint64_t s_full[2][2];                       // query tile, S buffer
  uint64_t p_full[2][2][2];                    // query tile, S buffer, half of the tile's keys
  uint64_t pv_done[2], o_full[2], o_free[2], drain[2];
  uint64_t turn[2];                            // two query tiles: their exponentials alternate
  uint32_t tmem_base;
  int abort_flag;
  int ref[4][2];                               // e4m3 caches: largest scale byte of K and V, by part
  int scan[4][4][2];                           // the converter warps' maxima, by part
  int odd[4];                                  // part + 1 whose newest positions hold values that are not finite
};

// One arrival for the warp, after everything its lanes did before.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Waits without looking at the abort flag: copies and products in flight must
// finish before the CTA's memory goes away.
__device__ __forceinline__ void tc_drain(uint64_t* bar, uint32_t parity, const Watchdog& wd) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > wd.budget_ns) {
      atomicCAS(wd.status, 0u, kDevTimeout | kSiteDrain);
      return;
    }
  }
}

// O = alpha O in TMEM after a row's reference moved; rare, so out of line.
template <int NCOL>
__device__ __noinline__ void tc_rescale(uint32_t t_o, float alpha) {
#pragma unroll
  for (int q = 0; q < NCOL / 16; ++q) {
    uint32_t o[16];
    tmem_ld16(t_o + q * 16, o);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    tmem_st16(t_o + q * 16, o);
  }
}

// Byte offset of 16-byte chunk cc of row r in a bf16 tile.
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int r, int cc) {
  constexpr int ATOM = D >= 64 ? 64 : D, CPA = ATOM / 8;
  const int a = cc / CPA, ca = cc % CPA;
  const int pc = ATOM == 64 ? (ca ^ (r & 7)) : (ca ^ ((r >> 1) & 3));
  return a * (kBN * ATOM * 2) + r * (ATOM * 2) + (pc << 4);
}

// Byte offset of 16-byte chunk cc of row r in a tile of codes.
template <int D>
__device__ __forceinline__ uint32_t raw_off(int r, int cc) {
  const int pc = D == 128 ? (cc ^ (r & 7)) : D == 64 ? (cc ^ ((r >> 1) & 3)) : cc;
  return r * D + (pc << 4);
}

// Two codes as f16 values times the pair of factors f.
__device__ __forceinline__ uint32_t codes_f16(uint32_t two, uint32_t f) {
  uint32_t h, r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(f));
  return r;
}

// The larger finite magnitude of a bf16 pair, as bf16 bits (0: none).
__device__ __forceinline__ uint32_t finite_top(uint32_t w) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  return max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u);
}

__device__ __forceinline__ uint32_t to_f16(uint32_t w, float f) {
  const float2 x = unpack_bf16x2(w);
  return pack_f16x2(x.x * f, x.y * f);
}

__device__ __forceinline__ uint32_t pack_f16x2_pair(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_f16x2(lo, hi);
}

// The value (bf16 bits) at column c of a position, for the rare rows that add it themselves.
template <int D, bool Q8>
__device__ __forceinline__ float value_of(const TreeParams& p, int bh, int key, int c) {
  const size_t row = static_cast<size_t>(bh) * p.m + key;
  if constexpr (Q8) {
    const uint32_t code = static_cast<const unsigned char*>(p.v)[row * D + c];
    return (code & 0x7fu) == 0x7fu ? __uint_as_float(0x7fc00000u) : 0.f;  // only NaN is not finite
  } else {
    const uint16_t h = static_cast<const uint16_t*>(p.v)[row * D + c];
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
  }
}

template <int D, int NQ, bool Q8>
__global__ void __launch_bounds__(Tc<D, NQ, Q8>::THREADS, 1)
attn_tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const TreeParams p, int least) {
  using C = Tc<D, NQ, Q8>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) TcShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sh.abort_flag;
  const Watchdog wd = p.wd;
  grid_launch_dependents();
  TreeWalk walk;
  if (!tree_start(p, kBN, least, walk)) return;
  if (tid == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, NQ);
    mbar_init(&sh.scanned, 4);
    for (int s = 0; s < C::NB; ++s) {
      mbar_init(&sh.full[s], Q8 ? 4 : 1);
      mbar_init(&sh.empty[s], NQ);
      mbar_init(&sh.clean[s], 1);
    }
    for (int s = 0; s < C::NR; ++s) {
      mbar_init(&sh.raw_full[s], 1);
      mbar_init(&sh.raw_empty[s], 4);
    }
    for (int g = 0; g < NQ; ++g) {
      mbar_init(&sh.q_f16[g], 4);
      for (int u = 0; u < 2; ++u) {
        mbar_init(&sh.s_full[g][u], 1);
        mbar_init(&sh.p_full[g][u][0], 4);
        mbar_init(&sh.p_full[g][u][1], 4);
      }
      mbar_init(&sh.pv_done[g], 1);
      mbar_init(&sh.o_full[g], 1);
      mbar_init(&sh.o_free[g], 4);
      mbar_init(&sh.drain[g], 1);
      mbar_init(&sh.turn[g], 4);
    }
    sh.abort_flag = 0;
    for (int i = 0; i < 4; ++i) sh.odd[i] = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == C::ISSUER) {
    tmem_alloc<C::TMEM>(&sh.tmem_base);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  TreePart part;
  int seg = 0;    // parts done
  int done = 0;   // tiles done: K tile j of the walk is ring tile 2 j, its V tile 2 j + 1
  bool ok = true;

  if (warp < C::SOFT) {
    // ------------------------------------------------------------ softmax, one thread a row
    if (C::SPLIT) reg_alloc<C::R_SOFT>();
    const int g = warp / 4;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_o = tmem + lane_base + C::TM_O + g * D;
    // e4m3: weights against a reference this far below the maximum (log2 units)
    constexpr float kLow = Q8 ? 7.f : 0.f;
#pragma unroll 1
    while (ok && tree_next(p, kBN, walk, part)) {
      const int old = part.L - p.n;
      const int row = part.rb * (NQ * 128) + g * 128 + r;
      const bool real = row < p.rows;
      const bool idle = __all_sync(0xffffffffu, !real);  // this warp's rows do not exist
      const unsigned long long word = real ? tree_word(p, part.b, row) : 0ull;
      const int T = part.t1 - part.t0;
      // scale 0: a tiny positive factor keeps -inf (masked) at weight 0
      float c = fmaxf(fabsf(p.c), 1e-30f);
      if constexpr (Q8) {
        ok = __all_sync(0xffffffffu, guarded_wait(&sh.q_full, seg & 1, abort_flag, wd, kSiteQFull));
        if (!ok) break;
        uint8_t* tile = smem + C::OFF_Q + g * C::TILE;
        uint4 w[D / 8];
        uint32_t top = 0;
#pragma unroll
        for (int cc = 0; cc < D / 8; ++cc) {
          w[cc] = *reinterpret_cast<const uint4*>(tile + chunk_off<D>(r, cc));
          top = max(top, max(max(finite_top(w[cc].x), finite_top(w[cc].y)), max(finite_top(w[cc].z), finite_top(w[cc].w))));
        }
        const uint32_t up = 268u - max(top >> 7, 15u);
        const float f = __uint_as_float(up << 23);
        c *= __uint_as_float((254u - up) << 23);
#pragma unroll
        for (int cc = 0; cc < D / 8; ++cc)
          *reinterpret_cast<uint4*>(tile + chunk_off<D>(r, cc)) =
              make_uint4(to_f16(w[cc].x, f), to_f16(w[cc].y, f), to_f16(w[cc].z, f), to_f16(w[cc].w, f));
        fence_proxy_async_smem();
        warp_arrive(&sh.q_f16[g]);
      }
      float m_used = -INFINITY, l = 0.f;
      uint64_t c2 = f2_pack(c, c);
#pragma unroll 1
      for (int j = 0; j < T; ++j) {
        const int gi = done + j;
        const int u = C::NS == 2 ? (gi & 1) : 0;
        const uint32_t ph = (C::NS == 2 ? gi >> 1 : gi) & 1;
        const uint32_t t_s = tmem + lane_base + (g * C::NS + u) * kBN;
        ok = __all_sync(0xffffffffu, guarded_wait(&sh.s_full[g][u], ph, abort_flag, wd, kSiteSFull));
        if (!ok) break;
        tc_fence_after();
        if (Q8 && j == 0) {  // the part's largest K scale is known by now
          c = fmaxf(c * pow2_of_byte(sh.ref[seg & 3][0]) * 0x1p-7f, 1e-37f);
          c2 = f2_pack(c, c);
        }
        if (idle) {
          if (NQ == 2) warp_arrive(&sh.turn[g ^ 1]);
          tc_fence_before();
          warp_arrive(&sh.p_full[g][u][0]);
          warp_arrive(&sh.p_full[g][u][1]);
          continue;
        }
        uint32_t s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(t_s + q * 32, s[q]);
        tmem_ld_wait();
        const int k0 = (part.t0 + j) * kBN;
        if (k0 + kBN > old) {
          // keys of this tile that the row sees
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t seen = sees32(word, k0 + q * 32, old, part.L);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((seen >> i) & 1u)) s[q][i] = __float_as_uint(-INFINITY);
          }
        }
        float mx[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) mx[v] = fmaxf(__uint_as_float(s[0][2 * v]), __uint_as_float(s[0][2 * v + 1]));
#pragma unroll
        for (int e = 8; e < kBN; e += 8)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            mx[v] = max3(mx[v], __uint_as_float(s[(e + 2 * v) >> 5][(e + 2 * v) & 31]),
                         __uint_as_float(s[(e + 2 * v + 1) >> 5][(e + 2 * v + 1) & 31]));
        const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        float alpha = 1.f;
        bool moved = false;
        if (j == 0) {
          m_used = m_new;
        } else if (m_new > m_used + kGrow) {
          alpha = ex2_approx(m_used - m_new);  // from -inf: 0
          m_used = m_new;
          moved = true;
        }
        const float m_ref = m_used == -INFINITY ? 0.f : m_used - kLow;  // nothing seen yet: weights 0
        const uint64_t nm2 = f2_pack(-m_ref, -m_ref);
        if (NQ == 2 && (g == 1 || gi > 0)) {
          // the exponentials of the two query tiles take turns (0, 1, 0, 1, ...), so
          // that one tile's overlap the other's products
          ok = __all_sync(0xffffffffu, guarded_wait(&sh.turn[g], (g == 1 ? gi : gi - 1) & 1, abort_flag, wd, kSiteExpTurn));
          if (!ok) break;
        }
        if (j > 0 && __any_sync(0xffffffffu, moved)) {
          // the products so far are in O (with two S buffers the scores do not show that)
          ok = __all_sync(0xffffffffu, guarded_wait(&sh.pv_done[g], (gi - 1) & 1, abort_flag, wd, kSitePFull));
          if (!ok) break;
          tc_fence_after();
          tc_rescale<D>(t_o, alpha);
          l *= alpha;
        }
        // weights of 64 keys, then of the other 64, whose products start meanwhile
        uint64_t acc0 = f2_pack(l, 0.f), acc1 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int q = 2 * half; q < 2 * half + 2; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t x2 =
                  fma2(f2_pack(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1])), c2, nm2);
              float x0, x1;
              f2_unpack(x2, x0, x1);
              const uint64_t p2 = f2_pack(ex2_approx(x0), ex2_approx(x1));
              pk[i] = Q8 ? pack_f16x2_pair(p2) : pack_bf16x2_pair(p2);
              if (i & 1) acc1 = add2(acc1, p2);
              else acc0 = add2(acc0, p2);
            }
            tmem_st16(t_s + q * 16, pk);
          }
          if (NQ == 2 && half == 1) warp_arrive(&sh.turn[g ^ 1]);
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(&sh.p_full[g][u][half]);
        }
        float a0, a1, a2, a3;
        f2_unpack(acc0, a0, a1);
        f2_unpack(acc1, a2, a3);
        l = (a0 + a1) + (a2 + a3);
      }
      if (ok)
        ok = __all_sync(0xffffffffu, guarded_wait(&sh.o_full[g], seg & 1, abort_flag, wd, kSiteOFull));
      if (!ok) break;
      tc_fence_after();
      if (!idle) {
        const bool odd = *static_cast<volatile int*>(&sh.odd[seg & 3]) == seg + 1;
        const float unit_v = Q8 ? pow2_of_byte(sh.ref[seg & 3][1]) * 0x1p-7f : 1.f;
        // the reference of l and O (only NaN scores: 0)
        m_used = m_used == -INFINITY ? (l != 0.f ? 0.f : -INFINITY) : m_used - kLow;
        const float inv = m_used == -INFINITY ? 0.f : unit_v / l;
        const size_t out = static_cast<size_t>(part.bh) * p.rows + row;
        const int at = g * 128 + r;  // row of the block
        // (not unrolled: each turn's loads and stores are independent of the others')
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          uint32_t o[16];
          tmem_ld16(t_o + q * 16, o);
          tmem_ld_wait();
          if (odd) {
            for (int key = max(part.t0 * kBN, old / kBN * kBN); key < min(part.L, part.t1 * kBN); ++key)
              if (real && sees(word, key, old, part.L))
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float v = value_of<D, Q8>(p, part.bh, key, q * 16 + i);
                  if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u)
                    o[i] = __float_as_uint(__uint_as_float(o[i]) + v);
                }
          }
          if (!real) continue;
          if (part.whole) {
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              pk[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
            uint4* dst = reinterpret_cast<uint4*>(p.o + out * D + q * 16);
            dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          } else {
            // Four columns of all rows side by side: a warp's rows are one run of
            // 512 bytes. (A row that saw nothing: its products are 0.)
            float4* dst = reinterpret_cast<float4*>(p.part) +
                          (static_cast<size_t>(part.slot) * (D / 4) + q * 4) * p.block_rows + at;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[static_cast<size_t>(i) * p.block_rows] =
                  make_float4(__uint_as_float(o[4 * i]) * unit_v, __uint_as_float(o[4 * i + 1]) * unit_v,
                              __uint_as_float(o[4 * i + 2]) * unit_v, __uint_as_float(o[4 * i + 3]) * unit_v);
          }
        }
        if (real) {
          if (!part.whole)
            *reinterpret_cast<float2*>(p.part_ml + 2 * (static_cast<size_t>(part.slot) * p.block_rows + at)) =
                make_float2(m_used, l);
          else if (p.lse != nullptr)
            p.lse[out] = m_used == -INFINITY ? -INFINITY : (m_used + log2f(l)) * kTreeLn2;
        }
      }
      tc_fence_before();
      warp_arrive(&sh.o_free[g]);
      done += T;
      ++seg;
    }
  } else if (Q8 && warp >= C::CONV) {
    // ------------------------------------------------------------ converters, one key row a thread
    if (C::SPLIT) reg_dealloc<C::R_CONV>();
    const int r = tid - C::CONV * 32;
#pragma unroll 1
    while (ok && tree_next(p, kBN, walk, part)) {
      const int old = part.L - p.n, T = part.t1 - part.t0;
      const size_t row0 = static_cast<size_t>(part.bh) * p.m;
      const int key_end = min(part.L, part.t1 * kBN);
      // the largest scales of the part's keys
      int top[2] = {0, 0};
#pragma unroll 4
      for (int key = part.t0 * kBN + r; key < key_end; key += kBN) {
        top[0] = max(top[0], static_cast<int>(__ldg(p.k_exp + row0 + key)));
        top[1] = max(top[1], static_cast<int>(__ldg(p.v_exp + row0 + key)));
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        top[u] = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(top[u])));
        if (lane == 0) sh.scan[seg & 3][warp - C::CONV][u] = top[u];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.scanned);
      ok = __all_sync(0xffffffffu, guarded_wait(&sh.scanned, seg & 1, abort_flag, wd, kSiteKFull));
      if (!ok) break;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int* of = &sh.scan[seg & 3][0][u];
        top[u] = max(max(of[0], of[2]), max(of[4], of[6]));
        if (r == 0) sh.ref[seg & 3][u] = top[u];
      }
      int bytes[2] = {0, 0};
      auto scales = [&](int j) {  // of the tile's K and V row, read a tile ahead
        const int key = (part.t0 + j) * kBN + r;
        if (key < key_end) {
          bytes[0] = __ldg(p.k_exp + row0 + key);
          bytes[1] = __ldg(p.v_exp + row0 + key);
        }
      };
      scales(0);
#pragma unroll 1
      for (int j = 0; ok && j < T; ++j) {
        // 2^(e - top + 7) in f16, below 2^-14 as the subnormal numbers it has
        uint32_t f2[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int e = bytes[u] - top[u] + 7;
          const uint32_t f = e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
          f2[u] = f | (f << 16);
        }
        scales(j + 1);
        const int key = (part.t0 + j) * kBN + r;
        const bool tail = (part.t0 + j + 1) * kBN > old;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const int h = 2 * (done + j) + kv;
          const int rs = h % C::NR, bs = h % C::NB;
          ok = guarded_wait(&sh.raw_full[rs], (h / C::NR) & 1, abort_flag, wd, kSiteKFull) &&
               (h < C::NB || guarded_wait(&sh.empty[bs], (h / C::NB - 1) & 1, abort_flag, wd, kSiteKEmpty));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* src = smem + C::OFF_R + rs * C::RAW;
          uint8_t* dst = smem + C::OFF_B + bs * C::TILE;
          const uint32_t f = f2[kv];
          if (kv == 1 && tail) {
            // Rows past the sequence are anyone's: zeros. NaN codes become zeros
            // too (a weight of 0 would make them NaN for rows that do not see
            // them); the rows that do see them add them at the end.
            const bool zero = key >= part.L;
            bool odd = false;
            for (int cc = 0; cc < D / 16; ++cc) {
              const uint4 w4 = *reinterpret_cast<const uint4*>(src + raw_off<D>(r, cc));
              uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
              uint32_t o[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t n = nan_codes(w[i]) & 0x80808080u;
                odd |= n != 0;
                w[i] = zero ? 0u : w[i] & ~((n >> 7) * 0xffu);
                o[2 * i] = codes_f16(w[i] & 0xffffu, f);
                o[2 * i + 1] = codes_f16(w[i] >> 16, f);
              }
              *reinterpret_cast<uint4*>(dst + chunk_off<D>(r, 2 * cc)) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4*>(dst + chunk_off<D>(r, 2 * cc + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            if (odd && !zero) sh.odd[seg & 3] = seg + 1;
          } else {
#pragma unroll
            for (int cc = 0; cc < D / 16; ++cc) {
              const uint4 w = *reinterpret_cast<const uint4*>(src + raw_off<D>(r, cc));
              *reinterpret_cast<uint4*>(dst + chunk_off<D>(r, 2 * cc)) =
                  make_uint4(codes_f16(w.x & 0xffffu, f), codes_f16(w.x >> 16, f), codes_f16(w.y & 0xffffu, f),
                             codes_f16(w.y >> 16, f));
              *reinterpret_cast<uint4*>(dst + chunk_off<D>(r, 2 * cc + 1)) =
                  make_uint4(codes_f16(w.z & 0xffffu, f), codes_f16(w.z >> 16, f), codes_f16(w.w & 0xffffu, f),
                             codes_f16(w.w >> 16, f));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.full[bs]);
            mbar_arrive(&sh.raw_empty[rs]);
          }
        }
      }
      done += T;
      ++seg;
    }
  } else {
    if (C::SPLIT) reg_dealloc<C::R_CTRL>();
    if (warp == C::PRODUCER) {
      // ---------------------------------------------------------- TMA producer
      if (lane == 0) {
        constexpr int N = Q8 ? C::NR : C::NB;
        uint64_t* fulls = Q8 ? sh.raw_full : sh.full;
        uint64_t* empties = Q8 ? sh.raw_empty : sh.empty;
        int loaded = 0;  // ring tiles put on their way
        int q_parts = 0;
#pragma unroll 1
        while (ok && tree_next(p, kBN, walk, part)) {
          const int T = part.t1 - part.t0;
          if (seg > 0) ok = guarded_wait(&sh.q_empty, (seg - 1) & 1, abort_flag, wd, kSiteQFull);
          if (!ok) break;
          const int q0 = part.rb * (NQ * 128);
          mbar_arrive_expect_tx(&sh.q_full, NQ * C::TILE);
          ++q_parts;
          for (int t = 0; t < NQ; ++t)  // (rows past the last load as zeros)
            for (int a = 0; a < C::NATOM; ++a)
              tma_load_3d(smem + C::OFF_Q + t * C::TILE + a * C::BOX, &tm_q, &sh.q_full, a * C::ATOM,
                          q0 + t * 128, part.bh);
          for (int x = 0; ok && x < 2 * T; ++x) {
            const int h = 2 * done + x, st = h % N;
            if (h >= N) ok = guarded_wait(&empties[st], (h / N - 1) & 1, abort_flag, wd, kSiteKEmpty);
            if (!ok) break;
            const CUtensorMap* map = (x & 1) ? &tm_v : &tm_k;
            const int k0 = (part.t0 + x / 2) * kBN;
            if (Q8) {
              mbar_arrive_expect_tx(&fulls[st], C::RAW);
              tma_load_3d(smem + C::OFF_R + st * C::RAW, map, &fulls[st], 0, k0, part.bh);
            } else {
              mbar_arrive_expect_tx(&fulls[st], C::TILE);
              for (int a = 0; a < C::NATOM; ++a)
                tma_load_3d(smem + C::OFF_B + st * C::TILE + a * C::BOX, map, &fulls[st], a * C::ATOM, k0, part.bh);
            }
            ++loaded;
          }
          done += T;
          ++seg;
        }
        // every copy lands before shared memory is released
        if (q_parts > 0) tc_drain(&sh.q_full, (q_parts - 1) & 1, wd);
        for (int x = max(0, loaded - N); x < loaded; ++x) tc_drain(&fulls[x % N], (x / N) & 1, wd);
      }
    } else if (warp < C::ISSUER + NQ) {
      // ---------------------------------------------------------- issuer of query tile g
      const int g = warp - C::ISSUER;
      if (lane == 0) {
        constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);  // operand formats of the descriptor; f16 is 0
        const uint32_t idesc_s =
            (idesc_bf16_f32(128, kBN, false, false) & ~(Q8 ? kBf16 : 0u)) | (p.c < 0.f ? (1u << 13) : 0u);
        const uint32_t idesc_o = idesc_bf16_f32(128, D, false, true) & ~(Q8 ? kBf16 : 0u);
        const uint32_t sq = smem_u32(smem + C::OFF_Q) + g * C::TILE;
        const uint32_t sb = smem_u32(smem + C::OFF_B);
        const uint32_t t_s = tmem + g * C::NS * kBN, t_o = tmem + C::TM_O + g * D;
        auto k_ready = [&](int gi) {
          const int h = 2 * gi;
          return guarded_wait(&sh.full[h % C::NB], (h / C::NB) & 1, abort_flag, wd, kSiteKFull);
        };
        auto scores = [&](int gi) {  // S of the walk's tile gi, whose K tile is there
          const int st = 2 * gi % C::NB, u = C::NS == 2 ? (gi & 1) : 0;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int a = k / (C::ATOM / 16), w = k % (C::ATOM / 16);
            mma_ss(t_s + u * kBN, smem_desc(sq + a * C::BOX + w * 32, 16, C::SBO, C::SWZ),
                   smem_desc(sb + st * C::TILE + a * C::BOX + w * 32, 16, C::SBO, C::SWZ), idesc_s, k > 0 ? 1u : 0u);
          }
          mma_commit(&sh.s_full[g][u]);
          mma_commit(&sh.empty[st]);
        };
#pragma unroll 1
        while (ok && tree_next(p, kBN, walk, part)) {
          const int T = part.t1 - part.t0;
          ok = guarded_wait(Q8 ? &sh.q_f16[g] : &sh.q_full, seg & 1, abort_flag, wd, kSiteQFull) && k_ready(done);
          if (ok) scores(done);
          for (int j = 0; ok && j < T; ++j) {
            const int gi = done + j, h = 2 * gi + 1, st = h % C::NB;
            const int u = C::NS == 2 ? (gi & 1) : 0;
            const uint32_t ph = (C::NS == 2 ? gi >> 1 : gi) & 1;
            if (C::NS == 2 && j + 1 < T) {
              if (!(ok = k_ready(gi + 1))) break;
              scores(gi + 1);
            }
            if (j + 1 == T) mma_commit(&sh.q_empty);  // this part's last scores are on their way
            // what is there long before the weights is waited for first
            ok = guarded_wait(Q8 ? &sh.full[st] : &sh.clean[st], (h / C::NB) & 1, abort_flag, wd, kSiteVFull);
            if (ok && C::NS == 1 && j + 1 < T) ok = k_ready(gi + 1);
            // the previous part's O has been read
            if (ok && j == 0 && seg > 0) ok = guarded_wait(&sh.o_free[g], (seg - 1) & 1, abort_flag, wd, kSiteOFull);
            for (int half = 0; ok && half < 2; ++half) {
              if (!(ok = guarded_wait(&sh.p_full[g][u][half], ph, abort_flag, wd, kSitePFull))) break;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < kBN / 32; ++k)
                mma_ts(t_o, t_s + u * kBN + half * 32 + k * 8,
                       smem_desc(sb + st * C::TILE + (half * 4 + k) * 16 * C::ATOM * 2, C::BOX, C::SBO, C::SWZ), idesc_o,
                       (j > 0 || half > 0 || k > 0) ? 1u : 0u);
            }
            if (!ok) break;
            mma_commit(&sh.empty[st]);
            mma_commit(&sh.pv_done[g]);
            if (j + 1 == T) mma_commit(&sh.o_full[g]);
            if (C::NS == 1 && j + 1 < T) scores(gi + 1);
          }
          done += T;
          ++seg;
        }
        // every product finishes before TMEM is released
        mma_commit(&sh.drain[g]);
        tc_drain(&sh.drain[g], 0, wd);
      }
      __syncwarp();
    } else if (!Q8 && warp == C::CLEANER) {
      // ---------------------------------------------------------- cleaner of V tiles
#pragma unroll 1
      while (ok && tree_next(p, kBN, walk, part)) {
        const int old = part.L - p.n, T = part.t1 - part.t0;
#pragma unroll 1
        for (int j = 0; ok && j < T; ++j) {
          const int h = 2 * (done + j) + 1, st = h % C::NB;
          ok = guarded_wait(&sh.full[st], (h / C::NB) & 1, abort_flag, wd, kSiteVFull);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const int k0 = (part.t0 + j) * kBN;
          if (k0 + kBN > old) {
            bool odd = false;
            uint8_t* tile = smem + C::OFF_B + st * C::TILE;
            for (int x = lane; x < kBN * (D / 8); x += 32) {
              const int r = x / (D / 8);
              uint4* at = reinterpret_cast<uint4*>(tile + chunk_off<D>(r, x % (D / 8)));
              uint4 v = *at;
              uint32_t* w = reinterpret_cast<uint32_t*>(&v);
              bool dirty = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t y = k0 + r < part.L ? w[i] : 0u;
                if ((y & 0x7f80u) == 0x7f80u) odd = true, y &= 0xffff0000u;
                if ((y & 0x7f800000u) == 0x7f800000u) odd = true, y &= 0x0000ffffu;
                dirty |= y != w[i];
                w[i] = y;
              }
              if (dirty) *at = v;
            }
            if (odd) sh.odd[seg & 3] = seg + 1;
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.clean[st]);
        }
        done += T;
        ++seg;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::ISSUER) {
    tc_fence_after();
    tmem_dealloc<C::TMEM>(tmem);
  }
}

template <int D, int NQ, bool Q8>
cudaError_t launch_tc(int grid, int least, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const TreeParams& p, cudaStream_t stream) {
  using C = Tc<D, NQ, Q8>;
  static std::atomic<int> ready[64];  // 1: usable, 2: the register split does not fit the compiled kernel
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int state = ready[dev & 63].load(std::memory_order_relaxed);
  if (state == 0) {
    e = cudaFuncSetAttribute(attn_tree_tc_kernel<D, NQ, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::SMEM));
    if (e != cudaSuccess) return e;
    state = 1;
    if (C::SPLIT) {
      // setmaxnreg.inc waits until registers are free: the shares must fit in
      // what the CTA is launched with, or the kernel would never proceed
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, attn_tree_tc_kernel<D, NQ, Q8>)) != cudaSuccess) return e;
      if (fa.numRegs * C::THREADS < C::R_SUM) state = 2;
    }
    ready[dev & 63].store(state, std::memory_order_relaxed);
  }
  if (state == 2) return cudaErrorInvalidConfiguration;
  prof_begin(kKindTree, stream);
  attn_tree_tc_kernel<D, NQ, Q8><<<static_cast<unsigned>(grid), C::THREADS, C::SMEM, stream>>>(tq, tk, tv, p, least);
  e = cudaGetLastError();
  prof_end(kKindTree, stream);
  return e;
}

template <int D>
cudaError_t launch_tc_d(bool quantised, int grid, int least, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  if (p.block_rows == 128)
    return quantised ? launch_tc<D, 1, true>(grid, least, tq, tk, tv, p, stream)
                     : launch_tc<D, 1, false>(grid, least, tq, tk, tv, p, stream);
  return quantised ? launch_tc<D, 2, true>(grid, least, tq, tk, tv, p, stream)
                   : launch_tc<D, 2, false>(grid, least, tq, tk, tv, p, stream);
}

}  // namespace

cudaError_t launch_tree_tc(int d, bool quantised, int grid, int least, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  switch (d) {
    case 32: return launch_tc_d<32>(quantised, grid, least, tq, tk, tv, p, stream);
    case 64: return launch_tc_d<64>(quantised, grid, least, tq, tk, tv, p, stream);
    case 128: return launch_tc_d<128>(quantised, grid, least, tq, tk, tv, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
