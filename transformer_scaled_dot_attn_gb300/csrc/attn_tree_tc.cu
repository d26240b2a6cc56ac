// Decoding of drafted tokens with many query rows a key head (attn_tree.cu
// states the operator): tcgen05 tiles of 128 query rows against 128 keys.
//
// A CTA walks its share of the line of tiles (attn_tree.cuh) with
//   128 rows: one query tile;
//   256 rows: two CTAs of a cluster as a pair (cta_group::2): each holds its 128
//     rows of Q, S, P and O but only half of every K tile (64 keys) and V tile (half
//     of the columns), so the pair reads, converts and keeps each K/V tile once.
//     The first CTA's issuers feed both SMs' tensor cores; what they wait for,
//     both CTAs report to them;
//   512 rows: a pair with two query tiles in each CTA, which take turns: while one
//     tile's scores are exponentiated, the tensor cores have the other's products.
// Bound by that exchange. 4 sequences of 20480 positions, 4 key heads of 512 rows,
// d = 128: 71 us over bf16 caches, 81 over e4m3 (the products alone need 44.5 at
// the rate of a large matrix product); a pair with one tile took 81 and 96. A turn
// of the two tiles takes some 2800 clocks, 2180 of them products, and a share of
// 34 turns starts with 10 us of first loads and set-up.
//   producer    TMA loads. bf16 caches: K and V into their rings in the tensor
//               cores' layout. e4m3 caches: the codes into rings of their own.
//   converters  (e4m3; 4 warps, for one query tile 4 for K and 4 for V) write f16
//               values into the K and V rings, code 2^(e - top + 7) with `top` the
//               largest scale of the part's keys: so a code is converted once for all
//               rows, one conversion and one exact product for two codes, and the
//               softmax carries no scales. f16 holds them exactly down to 2^-22 of
//               the largest; below that they lose low bits, and 2^-33 becomes 0.
//               The queries are brought to f16 as well, each row to [2^14, 2^15)
//               by a power of two, and the weights are f16 against a reference
//               2^7 below the maximum, so that they reach down to 2^-31 of it.
//   cleaner     (bf16) passes V tiles on; in tiles that reach the newest n
//               positions it zeroes the rows past the sequence and values that
//               are not finite (weight 0 times NaN is NaN). Rows that see such a
//               value get it added at the end. (The converters do this for e4m3.)
//               In a pair it reports Q and K tiles as well.
//   issuers     one query tile: a warp for S = Q K^T into one of two S buffers, one
//               for O += P V. Two: one warp, products of a tile's weights and then its
//               next scores into their place; with a warp for each tile both tiles
//               ran in step and the tensor cores stood still between (102 us for 75).
//               A warp's lanes look at the barriers it waits for at once: a wait for
//               one that is ready takes 150 clocks.
//   softmax     one thread a row: x = S c, p = 2^(x - m), P over S in TMEM, 64 keys
//               at a time so that their products start while the other 64 are
//               exponentiated. The reference m is the one so far; the tile's maximum is
//               sought meanwhile, and only if it is more than 2^8 above it the weights
//               are taken again and O is rescaled (maximum first: 87 us, this way 81).
// A waiter must not be overtaken: a wait tells a barrier's phases apart by their
// parity alone, so every phase that is waited for needs the waiter's own doing
// before the next one can complete. (So K and V have rings of their own: the
// cleaner waits for V tiles only.)
#include "attn_tree.cuh"

#include <atomic>

namespace attn {
namespace {

using namespace sm103;

constexpr int kBN = 128;
constexpr float kGrow = 8.0f;  // log2 units a row maximum may run ahead of its reference

template <int D, bool PAIR, int NQ, bool Q8>
struct Tc {
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr int KR = kBN / CTAS;                    // keys of a K tile in this CTA
  static constexpr int DV = D / CTAS;                      // columns of a V tile in this CTA
  static constexpr int ATOM = D >= 64 ? 64 : D;            // 16-bit elements of a swizzle row (Q, K)
  static constexpr int NATOM = D / ATOM;
  static constexpr uint32_t SWZ = D >= 64 ? 2u : 4u;
  static constexpr uint32_t SBO = 8u * ATOM * 2u;
  static constexpr int ATOMV = DV >= 64 ? 64 : DV;         // the same for V
  static constexpr int NATOMV = DV / ATOMV;
  static constexpr uint32_t SWZV = DV >= 64 ? 2u : 4u;
  static constexpr uint32_t SBOV = 8u * ATOMV * 2u;
  static constexpr uint32_t QTILE = 128u * D * 2u;
  static constexpr uint32_t TILE = static_cast<uint32_t>(KR) * D * 2u;   // a K or V tile (the same size)
  static constexpr uint32_t QBOX = 128u * ATOM * 2u, KBOX = KR * ATOM * 2u, VBOX = kBN * ATOMV * 2u;
  static constexpr uint32_t RAW = TILE / 2;                // a tile of codes
  // rings of K and of V, and of their codes: as many places as fit, six at most
  static constexpr uint32_t ROOM = 224u * 1024u - NQ * QTILE;
  static constexpr int at_most_six(uint32_t n) { return n < 6 ? static_cast<int>(n) : 6; }
  static constexpr int NT = !Q8 ? at_most_six(ROOM / (2 * TILE)) : D < 128 ? 4 : PAIR ? 3 : 2;
  static constexpr int NR = !Q8 ? 1 : at_most_six((ROOM - 2 * NT * TILE) / (2 * RAW));
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = NQ * QTILE;
  static constexpr uint32_t OFF_V = OFF_K + NT * TILE;
  static constexpr uint32_t OFF_RK = OFF_V + NT * TILE;
  static constexpr uint32_t OFF_RV = OFF_RK + (Q8 ? NR * RAW : 0);
  static constexpr uint32_t SMEM = OFF_RV + (Q8 ? NR * RAW : 0) + 1024;  // + alignment slack
  static_assert(NT >= 2 && NR >= 1 && SMEM <= 225u * 1024u, "shared memory");
  static_assert(DV >= 32, "V's swizzle");
  static constexpr int TM_O = 2 * kBN;                     // TMEM: two S buffers, then O of each query tile
  static constexpr int SOFT = 4 * NQ;                      // softmax warps: 0 to SOFT - 1
  static constexpr int PRODUCER = SOFT, ISSUE = SOFT + 1, CLEANER = SOFT + 3, CONV = SOFT + 4;  // issuers: ISSUE, + 1
  static constexpr int CONVERTERS = !Q8 ? 0 : NQ == 2 ? 4 : 8;  // one group of four warps for K and V, or one each
  static constexpr int THREADS = (CONV + CONVERTERS) * 32;
  static constexpr uint32_t FORMAT = Q8 ? (1u << 7) | (1u << 10) : 0u;  // cleared from bf16's descriptor: f16 operands
  // registers: the split must fit in what the CTA is launched with
  static constexpr bool SPLIT = Q8 || NQ == 2;
  static constexpr int R_SOFT = Q8 && NQ == 2 ? 176 : 208, R_CTRL = !Q8 ? 88 : NQ == 2 ? 72 : 64;
  static constexpr int R_CONV = NQ == 2 ? 88 : 112;
  static constexpr int R_SUM = 32 * (SOFT * R_SOFT + 4 * R_CTRL + CONVERTERS * R_CONV);
  static_assert(!SPLIT || R_SUM <= 65536 / THREADS / 8 * 8 * THREADS, "register split");
};

constexpr int kMaxRing = 6;

// Parts whose facts are kept: the loads of a part wait for the scores of the one
// before, which are at most two parts ahead of the weights, so whoever is ahead of
// the softmax has begun at most four parts more.
constexpr int kParts = 8;

struct TcShared {
  uint64_t q_full, q_empty;                    // TMA; released by the part's last scores
  uint64_t q_ready[2];                         // a query tile is there (e4m3: in f16) [issuer]
  uint64_t k_tma[kMaxRing], v_tma[kMaxRing];   // bf16: tile loaded
  uint64_t k_ready[kMaxRing], v_ready[kMaxRing];  // tile can be multiplied [issuer]
  uint64_t k_empty[kMaxRing], v_empty[kMaxRing];  // S, P V of the tile complete, of every query tile
  uint64_t raw_full[2][kMaxRing], raw_empty[2][kMaxRing];  // e4m3: codes of K, V
  uint64_t scanned[2];                         // e4m3: the part's scales of K, V were looked at
  uint64_t s_full[2];                          // by S buffer
  uint64_t p_full[2][2];                       // S buffer, half of the tile's keys [issuer]
  uint64_t o_full[2], o_free[2];               // by query tile: the part's O is complete; has been read
  uint64_t drain[2];                           // by issuer
  uint32_t tmem_base;
  int abort_flag;
  int ref[kParts][2];                          // e4m3: largest scale byte of K and V, by part
  int scan[kParts][2][4];                      // the converter warps' maxima, by part
  int odd[kParts];                             // part + 1 whose newest positions hold values that are not finite
};

// ---------------------------------------------------------------- the pair

template <bool PAIR>
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r = 0;
  if (PAIR) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One arrival for the warp on the issuer's barrier, after everything its lanes did before.
template <bool PAIR>
__device__ __forceinline__ void tell_issuer(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) != 0) return;
  // (Release at CTA scope: at cluster scope the arrival took 1200 to 2000 clocks.
  // What the other SM's thread starts on it, products of this SM's tensor cores,
  // reads this SM's shared memory and TMEM, whose writes have completed: the
  // proxy fence or the wait for the TMEM stores came before.)
  if (PAIR)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_cta(bar, 0)) : "memory");
  else
    mbar_arrive(bar);
}

template <bool PAIR>
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  if (!PAIR) return mbar_try_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait, at cluster scope in a pair; without guarded_wait's suspension for
// up to 20 us, from which warps came back late (16 sequences of 8192, 16 key heads of 40
// rows, d = 128, e4m3: 196 us with it, 166 without).
template <bool PAIR>
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const Watchdog& wd,
                                        uint32_t site) {
  if (try_wait<PAIR>(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!try_wait<PAIR>(bar, parity)) {
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > wd.budget_ns) {
      *abort_flag = 1;
      atomicCAS(wd.status, 0u, kDevTimeout | site);
      return false;
    }
  }
  return true;
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

template <bool PAIR>
__device__ __forceinline__ void tc_alloc(uint32_t* dst) {
  if (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc<512>(dst);
    tmem_relinquish();
  }
}

template <bool PAIR>
__device__ __forceinline__ void tc_dealloc(uint32_t taddr) {
  if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
  else tmem_dealloc<512>(taddr);
}

// A shared-memory descriptor whose start address is moved within its low word.
struct Desc {
  uint32_t lo, hi;
  __device__ __forceinline__ Desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
    const uint64_t d = smem_desc(addr, lbo, sbo, swizzle);
    lo = static_cast<uint32_t>(d);
    hi = static_cast<uint32_t>(d >> 32);
  }
  __device__ __forceinline__ uint64_t at(uint32_t bytes) const {
    return (static_cast<uint64_t>(hi) << 32) | (lo + (bytes >> 4));
  }
};

template <bool PAIR>
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_ss(d, a, b, idesc, acc);
}

template <bool PAIR>
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_ts(d, a, b, idesc, acc);
}

// Arrives on *bar (in both CTAs of a pair) when every product issued so far is complete.
template <bool PAIR>
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    mma_commit(bar);
}

// ---------------------------------------------------------------- layouts and conversions

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

// Byte offset of 16-byte chunk cc of row r in a 16-bit tile of COLS columns and ROWS rows.
template <int COLS, int ROWS>
__device__ __forceinline__ uint32_t chunk_off(int r, int cc) {
  constexpr int ATOM = COLS >= 64 ? 64 : COLS, CPA = ATOM / 8;
  const int a = cc / CPA, ca = cc % CPA;
  const int pc = ATOM == 64 ? (ca ^ (r & 7)) : (ca ^ ((r >> 1) & 3));
  return a * (ROWS * ATOM * 2) + r * (ATOM * 2) + (pc << 4);
}

// Byte offset of 16-byte chunk cc of row r in a tile of codes of COLS columns.
template <int COLS>
__device__ __forceinline__ uint32_t raw_off(int r, int cc) {
  const int pc = COLS == 128 ? (cc ^ (r & 7)) : COLS == 64 ? (cc ^ ((r >> 1) & 3)) : cc;
  return r * COLS + (pc << 4);
}

// Two codes as f16 values times the pair of factors f.
__device__ __forceinline__ uint32_t codes_f16(uint32_t two, uint32_t f) {
  uint32_t h, r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(f));
  return r;
}

// 2^e as a pair of f16, e <= 7; below 2^-14 the subnormal numbers that f16 has.
__device__ __forceinline__ uint32_t pow2_f16x2(int e) {
  const uint32_t f = e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
  return f | (f << 16);
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

// The largest of the bytes [b, e), this thread's share of 128. (Four loads at a
// time, whose latencies overlap.)
__device__ __forceinline__ uint32_t scan_bytes(const unsigned char* b, const unsigned char* e, int t) {
  const uintptr_t v0 = min((reinterpret_cast<uintptr_t>(b) + 15) & ~static_cast<uintptr_t>(15),
                           reinterpret_cast<uintptr_t>(e));
  const uintptr_t v1 = max(reinterpret_cast<uintptr_t>(e) & ~static_cast<uintptr_t>(15), v0);
  const uint4* v = reinterpret_cast<const uint4*>(v0);
  const long long count = static_cast<long long>(v1 - v0) / 16;
  uint32_t m = 0;
  if (b + t < reinterpret_cast<const unsigned char*>(v0)) m = __ldg(b + t);
  if (reinterpret_cast<const unsigned char*>(v1) + t < e)
    m = max(m, static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned char*>(v1) + t)));
#pragma unroll 1
  for (long long i = t; i < count; i += 512) {
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = i + u * 128 < count ? __ldg(v + i + u * 128) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < 4; ++u) m = __vmaxu4(m, __vmaxu4(__vmaxu4(x[u].x, x[u].y), __vmaxu4(x[u].z, x[u].w)));
  }
  return max(max(m & 0xffu, (m >> 8) & 0xffu), max((m >> 16) & 0xffu, m >> 24));
}

// The value at column c of a position, for the rare rows that add one that is not finite themselves.
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

// Reports (to both CTAs of a pair) that part `seg` holds values that are not finite among its newest positions.
template <bool PAIR>
__device__ __forceinline__ void mark_odd(TcShared& sh, int seg, uint32_t rank) {
  *static_cast<volatile int*>(&sh.odd[seg % kParts]) = seg + 1;
  if (PAIR)
    asm volatile("st.shared::cluster.u32 [%0], %1;\n\tfence.acq_rel.cluster;" ::"r"(
                     in_cta(&sh.odd[seg % kParts], rank ^ 1u)),
                 "r"(seg + 1)
                 : "memory");
}

template <int D, bool PAIR, int NQ, bool Q8>
__global__ void __launch_bounds__(Tc<D, PAIR, NQ, Q8>::THREADS, 1)
attn_tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
  using C = Tc<D, PAIR, NQ, Q8>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) TcShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cta_rank<PAIR>();
  volatile int* abort_flag = &sh.abort_flag;
  const Watchdog wd = p.wd;
  grid_follow();
  TreeWalk walk;
  if (!tree_start(p, kBN, static_cast<int>(blockIdx.x) / C::CTAS, static_cast<int>(gridDim.x) / C::CTAS, walk))
    return;  // (both CTAs of a pair, or neither)
  if (warp == C::PRODUCER) {
    // (a lane a place of the rings)
    if (lane < C::NT) {
      mbar_init(&sh.k_tma[lane], 1);
      mbar_init(&sh.v_tma[lane], 1);
      mbar_init(&sh.k_ready[lane], Q8 ? 4 * C::CTAS : C::CTAS);
      mbar_init(&sh.v_ready[lane], Q8 ? 4 * C::CTAS : C::CTAS);
      mbar_init(&sh.k_empty[lane], 1);
      mbar_init(&sh.v_empty[lane], 1);
    }
    if (lane < C::NR)
      for (int kind = 0; kind < 2; ++kind) {
        mbar_init(&sh.raw_full[kind][lane], 1);
        mbar_init(&sh.raw_empty[kind][lane], 4);
      }
    if (lane < 2) {
      mbar_init(&sh.q_ready[lane], Q8 ? 4 * C::CTAS : C::CTAS);
      mbar_init(&sh.scanned[lane], 4);
      mbar_init(&sh.s_full[lane], 1);
      mbar_init(&sh.p_full[lane][0], 4 * C::CTAS);
      mbar_init(&sh.p_full[lane][1], 4 * C::CTAS);
      mbar_init(&sh.o_full[lane], 1);
      mbar_init(&sh.o_free[lane], 4 * C::CTAS);
      mbar_init(&sh.drain[lane], 1);
    }
    if (lane < kParts) sh.odd[lane] = 0;
    if (lane == 0) {
      mbar_init(&sh.q_full, 1);
      mbar_init(&sh.q_empty, 1);
      sh.abort_flag = 0;
      prefetch_tensormap(&tm_q);
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
    fence_mbar_init();
  }
  if (warp == C::ISSUE) {
    tc_alloc<PAIR>(&sh.tmem_base);
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  TreePart part;
  int seg = 0;    // parts done
  int done = 0;   // tiles done
  bool ok = true;
  auto wait = [&](uint64_t* bar, int phase, uint32_t site) {
    return tc_wait<PAIR>(bar, static_cast<uint32_t>(phase) & 1u, abort_flag, wd, site);
  };

  if (warp < C::SOFT) {
    // ------------------------------------------------------------ softmax, one thread a row
    if (C::SPLIT) reg_alloc<C::R_SOFT>();
    const int tile = warp >> 2, r = tid & 127;  // query tile, its row
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_o = tmem + lane_base + C::TM_O + tile * D;
    // e4m3: weights against a reference this far below the maximum (log2 units)
    constexpr float kLow = Q8 ? 7.f : 0.f;
#pragma unroll 1
    while (ok && tree_next(p, kBN, walk, part)) {
      const int old = part.L - p.n;
      const int at = (tile * C::CTAS + static_cast<int>(rank)) * 128 + r;  // row of the block
      const int row = part.rb * (128 * C::CTAS * NQ) + at;
      const bool real = row < p.rows;
      const bool idle = __all_sync(0xffffffffu, !real);  // this warp's rows do not exist
      const unsigned long long word = real ? tree_word(p, part.b, row) : 0ull;
      const int T = part.t1 - part.t0;
      // scale 0: a tiny positive factor keeps -inf (masked) at weight 0
      float c = fmaxf(fabsf(p.c), 1e-30f);
      if constexpr (Q8) {
        ok = __all_sync(0xffffffffu, wait(&sh.q_full, seg, kSiteQFull));
        if (!ok) break;
        uint8_t* sq = smem + C::OFF_Q + tile * C::QTILE;
        uint4 w[D / 8];
        uint32_t top = 0;
#pragma unroll
        for (int cc = 0; cc < D / 8; ++cc) {
          w[cc] = *reinterpret_cast<const uint4*>(sq + chunk_off<D, 128>(r, cc));
          top = max(top, max(max(finite_top(w[cc].x), finite_top(w[cc].y)), max(finite_top(w[cc].z), finite_top(w[cc].w))));
        }
        const uint32_t up = 268u - max(top >> 7, 15u);
        const float f = __uint_as_float(up << 23);
        c *= __uint_as_float((254u - up) << 23);
#pragma unroll
        for (int cc = 0; cc < D / 8; ++cc)
          *reinterpret_cast<uint4*>(sq + chunk_off<D, 128>(r, cc)) =
              make_uint4(to_f16(w[cc].x, f), to_f16(w[cc].y, f), to_f16(w[cc].z, f), to_f16(w[cc].w, f));
        fence_proxy_async_smem();
        tell_issuer<PAIR>(&sh.q_ready[tile]);
      }
      float m_used = -INFINITY, l = 0.f;
      uint64_t c2 = f2_pack(c, c);
#pragma unroll 1
      for (int j = 0; j < T; ++j) {
        const int gi = done + j, u = NQ == 2 ? tile : gi & 1;
        const uint32_t t_s = tmem + lane_base + u * kBN;
        ok = __all_sync(0xffffffffu, wait(&sh.s_full[u], NQ == 2 ? gi : gi >> 1, kSiteSFull));
        if (!ok) break;
        tc_fence_after();
        if (Q8 && j == 0) {  // the part's largest K scale is known by now
          c = fmaxf(c * pow2_of_byte(sh.ref[seg % kParts][0]) * 0x1p-7f, 1e-37f);
          c2 = f2_pack(c, c);
        }
        if (idle) {
          tc_fence_before();
          tell_issuer<PAIR>(&sh.p_full[u][0]);
          tell_issuer<PAIR>(&sh.p_full[u][1]);
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
        // Weights of 64 keys, against the reference so far; if the tile's maximum,
        // found meanwhile, is too far above it, again against that one. Then the
        // other 64, while the products with the first are under way.
        uint64_t acc0, acc1, nm2;
        auto refer = [&]() {
          const float m_ref = m_used == -INFINITY ? 0.f : m_used - kLow;  // nothing seen yet: weights 0
          nm2 = f2_pack(-m_ref, -m_ref);
          acc0 = acc1 = f2_pack(0.f, 0.f);
        };
        auto weights = [&](int half) {
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
        };
        // (The second time in a loop over bf16 caches, so that the code of the first
        // tile, whose weights are always taken again, is there already: 71.9 us for
        // 74.0 of the case above. Over e4m3 caches, whose softmax warps share the
        // issue slots with the converters, as code of its own: 81.5 for 86.1.)
#pragma unroll 1
        while (true) {
          refer();
          weights(0);
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
          const bool moved = m_new > m_used + kGrow;
          tmem_st_wait();
          if (!__any_sync(0xffffffffu, moved)) break;
          const float alpha = moved ? ex2_approx(m_used - m_new) : 1.f;  // from -inf: 0
          if (moved) m_used = m_new;
          if (j > 0) {
            // the products so far are in O (two query tiles: the scores came after
            // them; the scores of one, a buffer ahead, do not show that)
            if (NQ == 1) {
              ok = __all_sync(0xffffffffu, wait(&sh.v_empty[(gi - 1) % C::NT], (gi - 1) / C::NT, kSitePFull));
              if (!ok) break;
              tc_fence_after();
            }
            tc_rescale<D>(t_o, alpha);
            l *= alpha;
          }
          if (Q8) {
            refer();
            weights(0);
            tmem_st_wait();
            break;
          }
        }
        if (!ok) break;
        tc_fence_before();
        tell_issuer<PAIR>(&sh.p_full[u][0]);
        weights(1);
        tmem_st_wait();
        tc_fence_before();
        tell_issuer<PAIR>(&sh.p_full[u][1]);
        float a0, a1, a2, a3;
        f2_unpack(acc0, a0, a1);
        f2_unpack(acc1, a2, a3);
        l += (a0 + a1) + (a2 + a3);
      }
      // the last tile's product
      done += T;
      if (ok) ok = __all_sync(0xffffffffu, wait(&sh.o_full[tile], seg, kSiteOFull));
      if (!ok) break;
      tc_fence_after();
      if (!idle) {
        const bool odd = *static_cast<volatile int*>(&sh.odd[seg % kParts]) == seg + 1;
        const float unit_v = Q8 ? pow2_of_byte(sh.ref[seg % kParts][1]) * 0x1p-7f : 1.f;
        // the reference of l and O (only NaN scores: 0)
        m_used = m_used == -INFINITY ? (l != 0.f ? 0.f : -INFINITY) : m_used - kLow;
        const float inv = m_used == -INFINITY ? 0.f : unit_v / l;
        const size_t out = static_cast<size_t>(part.bh) * p.rows + row;
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
      tell_issuer<PAIR>(&sh.o_free[tile]);
      ++seg;
    }
  } else if (Q8 && warp >= C::CONV) {
    // ------------------------------------------------------------ converters, one thread a row of K, V or both
    if (C::SPLIT) reg_dealloc<C::R_CONV>();
    const int t = tid & 127;
    const int first_kind = NQ == 2 ? 0 : (warp - C::CONV) >> 2, last_kind = NQ == 2 ? 1 : first_kind;  // 0: K, 1: V
    uint64_t* scanned = &sh.scanned[first_kind];
    // This thread's row of a tile and, as K tiles of a pair have 64 rows, its half
    // of the row; of the sequence's tile, whose other half the pair's other CTA has.
    const int row_of[2] = {t % C::KR, t}, c0[2] = {t / C::KR * (C::DV / 16), 0};
    const int first_row[2] = {static_cast<int>(rank) * C::KR + row_of[0], t};
#pragma unroll 1
    while (ok && tree_next(p, kBN, walk, part)) {
      const int old = part.L - p.n, T = part.t1 - part.t0;
      const size_t base = static_cast<size_t>(part.bh) * p.m;
      const int key_begin = part.t0 * kBN, key_end = min(part.L, part.t1 * kBN);
      int top[2] = {0, 0}, byte[2] = {0, 0};
      uint32_t most[2] = {0, 0};
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        if (kind < first_kind || kind > last_kind) continue;
        // the largest scale of the part's keys
        const unsigned char* row = (kind == 0 ? p.k_exp : p.v_exp) + base;
        const int key = key_begin + first_row[kind];
        if (key < key_end) byte[kind] = __ldg(row + key);  // read a tile ahead
        most[kind] = scan_bytes(row + min(key_begin, key_end), row + key_end, t);
      }
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        if (kind < first_kind || kind > last_kind) continue;
        const unsigned all = __reduce_max_sync(0xffffffffu, most[kind]);
        if (lane == 0) sh.scan[seg % kParts][kind][warp & 3] = static_cast<int>(all);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(scanned);
      ok = __all_sync(0xffffffffu, guarded_wait(scanned, seg & 1, abort_flag, wd, kSiteKFull));
      if (!ok) break;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        const int* of = sh.scan[seg % kParts][kind];
        if (kind < first_kind || kind > last_kind) continue;
        top[kind] = max(max(of[0], of[1]), max(of[2], of[3]));
        if (t == 0) sh.ref[seg % kParts][kind] = top[kind];
      }
#pragma unroll 1
      for (int x = 0; ok && x < T + last_kind; ++x) {
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          const int j = x - kind, gi = done + j, key = key_begin + j * kBN + first_row[kind];  // (V a tile behind)
          if (kind < first_kind || kind > last_kind || j < 0 || j >= T) continue;
          const int rs = gi % C::NR, bs = gi % C::NT, r = row_of[kind];
          const uint32_t f = pow2_f16x2(byte[kind] - top[kind] + 7);
          if (key + kBN < key_end) byte[kind] = __ldg((kind == 0 ? p.k_exp : p.v_exp) + base + key + kBN);
          ok = tc_wait<false>(&sh.raw_full[kind][rs], (gi / C::NR) & 1, abort_flag, wd, kSiteKFull) &&
               (gi < C::NT || wait(kind == 0 ? &sh.k_empty[bs] : &sh.v_empty[bs], gi / C::NT - 1, kSiteKEmpty));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* src = smem + (kind == 0 ? C::OFF_RK : C::OFF_RV) + rs * C::RAW;
          uint8_t* dst = smem + (kind == 0 ? C::OFF_K : C::OFF_V) + bs * C::TILE;
          // (an f16 tile's chunks: K has rows of D, V of DV)
          auto from = [&](int cc) {
            return *reinterpret_cast<const uint4*>(src + (kind == 0 ? raw_off<D>(r, c0[0] + cc) : raw_off<C::DV>(r, cc)));
          };
          auto to = [&](int cc) {
            return reinterpret_cast<uint4*>(
                dst + (kind == 0 ? chunk_off<D, C::KR>(r, 2 * c0[0] + cc) : chunk_off<C::DV, kBN>(r, cc)));
          };
          if (kind == 0 || (part.t0 + j + 1) * kBN <= old) {
#pragma unroll
            for (int cc = 0; cc < C::DV / 16; ++cc) {
              const uint4 w = from(cc);
              *to(2 * cc) = make_uint4(codes_f16(w.x & 0xffffu, f), codes_f16(w.x >> 16, f),
                                       codes_f16(w.y & 0xffffu, f), codes_f16(w.y >> 16, f));
              *to(2 * cc + 1) = make_uint4(codes_f16(w.z & 0xffffu, f), codes_f16(w.z >> 16, f),
                                           codes_f16(w.w & 0xffffu, f), codes_f16(w.w >> 16, f));
            }
          } else {
            // Rows past the sequence are anyone's: zeros. NaN codes become zeros
            // too (a weight of 0 would make them NaN for rows that do not see
            // them); the rows that do see them add them at the end.
            const bool zero = key >= part.L;
            bool odd = false;
            for (int cc = 0; cc < C::DV / 16; ++cc) {
              const uint4 w4 = from(cc);
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
              *to(2 * cc) = make_uint4(o[0], o[1], o[2], o[3]);
              *to(2 * cc + 1) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            if (odd && !zero) mark_odd<PAIR>(sh, seg, rank);
          }
          fence_proxy_async_smem();
          tell_issuer<PAIR>(kind == 0 ? &sh.k_ready[bs] : &sh.v_ready[bs]);
          if (lane == 0) mbar_arrive(&sh.raw_empty[kind][rs]);
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
        constexpr int N = Q8 ? C::NR : C::NT;
        constexpr uint32_t BYTES = Q8 ? C::RAW : C::TILE;
        const uint32_t off[2] = {Q8 ? C::OFF_RK : C::OFF_K, Q8 ? C::OFF_RV : C::OFF_V};
        uint64_t* full[2] = {Q8 ? sh.raw_full[0] : sh.k_tma, Q8 ? sh.raw_full[1] : sh.v_tma};
        uint64_t* empty[2] = {Q8 ? sh.raw_empty[0] : sh.k_empty, Q8 ? sh.raw_empty[1] : sh.v_empty};
        int loaded[2] = {0, 0}, q_loaded = 0;
#pragma unroll 1
        while (ok && tree_next(p, kBN, walk, part)) {
          const int T = part.t1 - part.t0;
          if (seg > 0) ok = wait(&sh.q_empty, seg - 1, kSiteQFull);
          if (!ok) break;
          mbar_arrive_expect_tx(&sh.q_full, NQ * C::QTILE);
          ++q_loaded;
          for (int x = 0; x < NQ * C::NATOM; ++x)  // (rows past the last load as zeros)
            tma_load_3d(smem + C::OFF_Q + x * C::QBOX, &tm_q, &sh.q_full, x % C::NATOM * C::ATOM,
                        ((part.rb * NQ + x / C::NATOM) * C::CTAS + static_cast<int>(rank)) * 128, part.bh);
#pragma unroll 1
          for (int j = 0; ok && j < T; ++j) {
            const int gi = done + j, k0 = (part.t0 + j) * kBN;
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
              const int st = gi % N;
              uint64_t* bar = &full[kind][st];
              uint8_t* dst = smem + off[kind] + st * BYTES;
              if (gi >= N) ok = wait(&empty[kind][st], gi / N - 1, kind == 0 ? kSiteKEmpty : kSiteVEmpty);
              if (!ok) break;
              mbar_arrive_expect_tx(bar, BYTES);
              const int kk = k0 + static_cast<int>(rank) * C::KR, vc = static_cast<int>(rank) * C::DV;
              if (kind == 0) {
                for (int a = 0; a < (Q8 ? 1 : C::NATOM); ++a)
                  tma_load_3d(dst + a * C::KBOX, &tm_k, bar, a * C::ATOM, kk, part.bh);
              } else {
                for (int a = 0; a < (Q8 ? 1 : C::NATOMV); ++a)
                  tma_load_3d(dst + a * C::VBOX, &tm_v, bar, vc + a * C::ATOMV, k0, part.bh);
              }
              ++loaded[kind];
            }
          }
          done += T;
          ++seg;
        }
        // every copy lands before shared memory is released
        if (q_loaded > 0) tc_drain(&sh.q_full, (q_loaded - 1) & 1, wd);
#pragma unroll
        for (int kind = 0; kind < 2; ++kind)
          for (int x = max(0, loaded[kind] - N); x < loaded[kind]; ++x)
            tc_drain(&full[kind][x % N], (x / N) & 1, wd);
      }
    } else if (warp == C::ISSUE || (NQ == 1 && warp == C::ISSUE + 1)) {
      // ---------------------------------------------------------- issuers (the pair's first CTA)
      // (The whole warp walks along, so that descriptors stay in uniform registers.)
      const int who = warp - C::ISSUE;
      const uint32_t idesc_s =
          (idesc_bf16_f32(128 * C::CTAS, kBN, false, false) & ~C::FORMAT) | (p.c < 0.f ? (1u << 13) : 0u);
      const uint32_t idesc_o = idesc_bf16_f32(128 * C::CTAS, D, false, true) & ~C::FORMAT;
      const Desc dq(smem_u32(smem + C::OFF_Q), 16, C::SBO, C::SWZ), dk(smem_u32(smem + C::OFF_K), 16, C::SBO, C::SWZ);
      const Desc dv(smem_u32(smem + C::OFF_V), C::VBOX, C::SBOV, C::SWZV);
      auto all_wait = [&](uint64_t* bar, int phase, uint32_t site) {
        return __all_sync(0xffffffffu, wait(bar, phase, site)) != 0;
      };
      // (several barriers at once: each lane looks at one of them)
      auto wait_both = [&](uint64_t* a, int phase_a, uint64_t* b, int phase_b, uint32_t site) {
        return all_wait(lane & 1 ? b : a, lane & 1 ? phase_b : phase_a, site);
      };
      auto q_there = [&](int tile) { return Q8 ? &sh.q_ready[tile] : PAIR ? &sh.q_ready[0] : &sh.q_full; };
      auto k_there = [&](int gi) { return Q8 || PAIR ? &sh.k_ready[gi % C::NT] : &sh.k_tma[gi % C::NT]; };
      auto v_there = [&](int gi) { return &sh.v_ready[gi % C::NT]; };
      // S of key tile gi and query tile `tile` into buffer u
      auto scores = [&](int gi, int tile, int u) {
        const int st = gi % C::NT;
        const uint32_t at = st * C::TILE, aq = tile * C::QTILE;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int a = k / (C::ATOM / 16), w = k % (C::ATOM / 16);
            tc_mma_ss<PAIR>(tmem + u * kBN, dq.at(aq + a * C::QBOX + w * 32), dk.at(at + a * C::KBOX + w * 32), idesc_s,
                            k > 0 ? 1u : 0u);
          }
          tc_commit<PAIR>(&sh.s_full[u]);
          if (tile == NQ - 1) tc_commit<PAIR>(&sh.k_empty[st]);
        }
        __syncwarp();
      };
      // O (+)= P V of 16-key steps [k0, k1) of the same, P in buffer u
      auto products = [&](int gi, int tile, int u, int k0, int k1, bool first) {
        const int st = gi % C::NT;
        const uint32_t at = st * C::TILE, t_o = tmem + C::TM_O + tile * D;
        if (elect_one()) {
#pragma unroll
          for (int k = k0; k < k1; ++k)
            tc_mma_ts<PAIR>(t_o, tmem + u * kBN + k * 8, dv.at(at + k * 16 * C::ATOMV * 2), idesc_o,
                            (!first || k > 0) ? 1u : 0u);
          if (k1 == kBN / 16 && tile == NQ - 1) tc_commit<PAIR>(&sh.v_empty[st]);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) tc_commit<PAIR>(bar);
        __syncwarp();
      };
      if (rank == 0) {
#pragma unroll 1
      while (ok && tree_next(p, kBN, walk, part)) {
        const int T = part.t1 - part.t0;
        if constexpr (NQ == 2) {
          // A query tile's products, then its next scores into the place of its
          // weights, while the other one's scores are exponentiated.
#pragma unroll
          for (int tile = 0; tile < 2; ++tile) {
            if (ok && (Q8 || tile == 0)) ok = all_wait(q_there(tile), seg, kSiteQFull);
            if (ok && tile == 0) ok = all_wait(k_there(done), done / C::NT, kSiteKFull);
            if (!ok) break;
            tc_fence_after();
            scores(done, tile, tile);
          }
          if (ok && T == 1) commit(&sh.q_empty);
#pragma unroll 1
          for (int j = 0; ok && j < T; ++j) {
            const int gi = done + j;
            const bool more = j + 1 < T;
#pragma unroll
            for (int tile = 0; tile < 2; ++tile) {
              // (the previous part's O has been read)
              if (j == 0 && seg > 0) ok = all_wait(&sh.o_free[tile], seg - 1, kSiteOFull);
              if (ok && tile == 0)
                ok = lane & 1      ? wait(v_there(gi), gi / C::NT, kSiteVFull)
                     : more && lane & 2 ? wait(k_there(gi + 1), (gi + 1) / C::NT, kSiteKFull)
                                   : wait(&sh.p_full[tile][0], gi, kSitePFull);
              else if (ok) ok = wait(&sh.p_full[tile][0], gi, kSitePFull);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_fence_after();
              products(gi, tile, tile, 0, kBN / 32, j == 0);
              ok = all_wait(&sh.p_full[tile][1], gi, kSitePFull);
              if (!ok) break;
              tc_fence_after();
              products(gi, tile, tile, kBN / 32, kBN / 16, j == 0);
              if (more) scores(gi + 1, tile, tile);
              else commit(&sh.o_full[tile]);
            }
            if (ok && j + 2 == T) commit(&sh.q_empty);  // the part's last scores
          }
        } else if (who == 0) {
          ok = all_wait(q_there(0), seg, kSiteQFull);
#pragma unroll 1
          for (int j = 0; ok && j < T; ++j) {
            const int gi = done + j;
            // (the buffer's weights have been multiplied)
            ok = gi >= 2 ? wait_both(k_there(gi), gi / C::NT, &sh.v_empty[(gi - 2) % C::NT], (gi - 2) / C::NT, kSiteKFull)
                         : all_wait(k_there(gi), gi / C::NT, kSiteKFull);
            if (!ok) break;
            tc_fence_after();
            scores(gi, 0, gi & 1);
          }
          if (ok) commit(&sh.q_empty);
        } else {
          if (seg > 0) ok = all_wait(&sh.o_free[0], seg - 1, kSiteOFull);
#pragma unroll 1
          for (int j = 0; ok && j < T; ++j) {
            const int gi = done + j, u = gi & 1;
            ok = wait_both(v_there(gi), gi / C::NT, &sh.p_full[u][0], gi >> 1, kSitePFull);
            if (!ok) break;
            tc_fence_after();
            products(gi, 0, u, 0, kBN / 32, j == 0);
            ok = all_wait(&sh.p_full[u][1], gi >> 1, kSitePFull);
            if (!ok) break;
            tc_fence_after();
            products(gi, 0, u, kBN / 32, kBN / 16, j == 0);
          }
          if (ok) commit(&sh.o_full[0]);
        }
        done += T;
        ++seg;
      }
      // every product finishes before TMEM is released
      commit(&sh.drain[who]);
      }
      // (the second CTA: the last of the arrivals that reach into it)
      tc_drain(&sh.drain[who], 0, wd);
      __syncwarp();
    } else if (!Q8 && warp == C::CLEANER) {
      // ---------------------------------------------------------- cleaner of V tiles
#pragma unroll 1
      while (ok && tree_next(p, kBN, walk, part)) {
        const int old = part.L - p.n, T = part.t1 - part.t0;
        if (PAIR) {
          ok = __all_sync(0xffffffffu, wait(&sh.q_full, seg, kSiteQFull));
          if (!ok) break;
          tell_issuer<PAIR>(&sh.q_ready[0]);
        }
#pragma unroll 1
        for (int j = 0; j < T; ++j) {
          const int gi = done + j, st = gi % C::NT;
          if (PAIR) {
            ok = __all_sync(0xffffffffu, wait(&sh.k_tma[st], gi / C::NT, kSiteKFull));
            if (!ok) break;
            tell_issuer<PAIR>(&sh.k_ready[st]);
          }
          ok = __all_sync(0xffffffffu, wait(&sh.v_tma[st], gi / C::NT, kSiteVFull));
          if (!ok) break;
          const int k0 = (part.t0 + j) * kBN;
          if (k0 + kBN > old) {
            bool odd = false;
            uint8_t* tile = smem + C::OFF_V + st * C::TILE;
            for (int x = lane; x < kBN * (C::DV / 8); x += 32) {
              const int r = x / (C::DV / 8);
              uint4* cell = reinterpret_cast<uint4*>(tile + chunk_off<C::DV, kBN>(r, x % (C::DV / 8)));
              uint4 v = *cell;
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
              if (dirty) *cell = v;
            }
            if (odd) mark_odd<PAIR>(sh, seg, rank);
            fence_proxy_async_smem();
          }
          tell_issuer<PAIR>(&sh.v_ready[st]);
        }
        done += T;
        ++seg;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // nothing reaches into the other CTA any more
  if (warp == C::ISSUE) {
    tc_fence_after();
    tc_dealloc<PAIR>(tmem);
  }
}

template <int D, bool PAIR, int NQ, bool Q8>
cudaError_t launch_tc(int grid, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const TreeParams& p, cudaStream_t stream) {
  using C = Tc<D, PAIR, NQ, Q8>;
  static std::atomic<int> ready[64];  // 1: usable, 2: the register split does not fit the compiled kernel
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int state = ready[dev & 63].load(std::memory_order_relaxed);
  if (state == 0) {
    e = cudaFuncSetAttribute(attn_tree_tc_kernel<D, PAIR, NQ, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::SMEM));
    if (e != cudaSuccess) return e;
    state = 1;
    if (C::SPLIT) {
      // setmaxnreg.inc waits until registers are free: the shares must fit in
      // what the CTA is launched with, or the kernel would never proceed
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, attn_tree_tc_kernel<D, PAIR, NQ, Q8>)) != cudaSuccess) return e;
      if (fa.numRegs * C::THREADS < C::R_SUM) state = 2;
    }
    ready[dev & 63].store(state, std::memory_order_relaxed);
  }
  if (state == 2) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C::CTAS;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid * C::CTAS));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  prof_begin(kKindTree, stream);
  e = cudaLaunchKernelEx(&cfg, attn_tree_tc_kernel<D, PAIR, NQ, Q8>, tq, tk, tv, p);
  prof_end(kKindTree, stream);
  return e;
}

template <int D, bool PAIR, int NQ>
cudaError_t launch_tc_of(bool quantised, int grid, const CUtensorMap& tq, const CUtensorMap& tk,
                         const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  return quantised ? launch_tc<D, PAIR, NQ, true>(grid, tq, tk, tv, p, stream)
                   : launch_tc<D, PAIR, NQ, false>(grid, tq, tk, tv, p, stream);
}

template <int D>
cudaError_t launch_tc_d(bool quantised, int grid, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  switch (p.block_rows) {
    case 128: return launch_tc_of<D, false, 1>(quantised, grid, tq, tk, tv, p, stream);
    case 256: return launch_tc_of<D, true, 1>(quantised, grid, tq, tk, tv, p, stream);
    case 512: return launch_tc_of<D, true, 2>(quantised, grid, tq, tk, tv, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_tree_tc(int d, bool quantised, int grid, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  switch (d) {
    case 32: return launch_tc_of<32, false, 1>(quantised, grid, tq, tk, tv, p, stream);
    case 64: return launch_tc_d<64>(quantised, grid, tq, tk, tv, p, stream);
    case 128: return launch_tc_d<128>(quantised, grid, tq, tk, tv, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
