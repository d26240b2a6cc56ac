// What the tree kernels share: how the key tiles of a batch are dealt out to
// CTAs, which keys a query sees, and the layout of partial results.
#pragma once

#include "attn_kernels.cuh"

namespace attn {

constexpr float kTreeLn2 = 0.69314718055994530942f;
// Tiles worth a CTA of their own. With 1, 2, 4, 8: 16.5, 12.0, 13.1, 14.6 us (one
// sequence of 1500 positions, 16 heads of one row, d = 128, e4m3); 23.1, 23.0, 23.1,
// 26.2 us (8 sequences of 2000, 4 key heads of 128 rows, e4m3).
constexpr int kTreeLeast = 2;

__device__ __forceinline__ float pow2_of_byte(int byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : static_cast<uint32_t>(byte) << 23);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Bit 7 of a byte of the result is set where that code is NaN (0x7f, 0xff).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }

// The newest positions a query row sees: bit t stands for position L - n + t.
__device__ __forceinline__ unsigned long long tree_word(const TreeParams& p, int b, int row) {
  const int i = row % p.n;
  if (p.tree != nullptr) return __ldg(p.tree + static_cast<size_t>(b) * p.n + i);
  return i >= 63 ? ~0ull : (1ull << (i + 1)) - 1ull;
}

// old = L - n: the positions before it are seen by every query.
__device__ __forceinline__ bool sees(unsigned long long word, int key, int old, int L) {
  return key < L && (key < old || ((word >> (key - old)) & 1ull));
}

// The same for the 32 keys from `key`: bit i for key + i.
__device__ __forceinline__ uint32_t sees32(unsigned long long word, int key, int old, int L) {
  const int s = key - old;
  uint32_t m;
  if (s >= 0) m = s < 64 ? static_cast<uint32_t>(word >> s) : 0u;
  else m = s <= -32 ? 0xffffffffu : (static_cast<uint32_t>(word) << -s) | ((1u << -s) - 1u);
  const int rem = L - key;
  return rem >= 32 ? m : rem <= 0 ? 0u : m & ((1u << rem) - 1u);
}

// Key tiles of a sequence; an empty one has a tile too (whose keys nobody
// sees), so that its rows are written like any other's.
__device__ __forceinline__ int tiles_of(int L, int bn) { return L > bn ? (L + bn - 1) / bn : 1; }

// The work is a line of tiles: the units (sequence, key head, block of query
// rows) one after the other, each with its sequence's tiles, after `lead` places
// that stand for the time that beginning a unit takes. CTA c of `ctas` takes the
// places [U c / ctas, U (c + 1) / ctas) of the U on the line: equal shares
// whatever the lengths, at the price of units that several CTAs hold a part
// of. The part of unit x that CTA c holds has its place x + c in the partial
// results (the sum grows from part to part along the line). A pair of CTAs that
// works as one counts as one here.
struct TreeLine {
  long long U;
  int ctas;
  int per_seq;  // units of a sequence
};

// Every lane of a warp calls this.
__device__ __forceinline__ TreeLine tree_line(const TreeParams& p, int bn, int grid) {
  TreeLine l;
  l.per_seq = p.h_kv * p.row_blocks;
  long long t = 0;
  if (p.kv_len == nullptr) {
    t = static_cast<long long>(p.B) * tiles_of(p.m, bn);
  } else {
    for (int b = static_cast<int>(threadIdx.x & 31); b < p.B; b += 32)
      t += tiles_of(min(max(__ldg(p.kv_len + b), 0), p.m), bn);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  l.U = (t + static_cast<long long>(p.B) * p.lead) * l.per_seq;
  const long long most = (l.U + kTreeLeast - 1) / kTreeLeast;
  l.ctas = static_cast<int>(most < grid ? most : grid);
  return l;
}

__device__ __forceinline__ int tree_len(const TreeParams& p, int b) {
  return p.kv_len == nullptr ? p.m : min(max(__ldg(p.kv_len + b), 0), p.m);
}

// A CTA's position on the line: the sequence and unit it is at.
struct TreeWalk {
  long long pos, end;   // places left: [pos, end)
  long long first;      // where the current unit's tiles begin
  int b, idx;           // sequence, unit within the sequence
  int L, tiles;         // the sequence's cached positions and tiles
  int cta;
};

struct TreePart {
  int b, bh, rb;        // sequence, (sequence, key head), block of query rows
  int t0, t1;           // the unit's tiles
  int L;
  bool whole;           // the unit has no other part
  long long unit, slot;
};

// Every lane of a warp calls this; false: the CTA has no share.
__device__ __forceinline__ bool tree_start(const TreeParams& p, int bn, int cta, int grid, TreeWalk& w) {
  if (p.by_unit) {  // short caches: CTA c takes unit c whole
    const int per_seq = p.h_kv * p.row_blocks;
    w.cta = 0;
    w.b = cta / per_seq;
    w.idx = cta - w.b * per_seq;
    w.L = tree_len(p, w.b);
    w.tiles = tiles_of(w.L, bn);
    w.first = w.pos = 0;
    w.end = w.tiles;
    return true;
  }
  const TreeLine l = tree_line(p, bn, grid);
  w.cta = cta;
  if (w.cta >= l.ctas) return false;
  w.pos = l.U * w.cta / l.ctas;
  w.end = l.U * (w.cta + 1) / l.ctas;
  const int lane = static_cast<int>(threadIdx.x & 31);
  if (p.kv_len == nullptr) {
    w.tiles = tiles_of(p.m, bn);
    w.L = p.m;
    const int span = w.tiles + p.lead;
    const long long unit = w.pos / span;
    w.b = static_cast<int>(unit / l.per_seq);
    w.idx = static_cast<int>(unit - static_cast<long long>(w.b) * l.per_seq);
    w.first = unit * span + p.lead;
    return true;
  }
  long long base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int L = b < p.B ? tree_len(p, b) : 0;
    const int tiles = b < p.B ? tiles_of(L, bn) : 0;
    long long incl = b < p.B ? static_cast<long long>(tiles + p.lead) * l.per_seq : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, base + incl > w.pos);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      w.b = b0 + src;
      w.L = __shfl_sync(0xffffffffu, L, src);
      w.tiles = __shfl_sync(0xffffffffu, tiles, src);
      const int span = w.tiles + p.lead;
      const long long at = base + __shfl_sync(0xffffffffu, incl, src) - static_cast<long long>(span) * l.per_seq;
      w.idx = static_cast<int>((w.pos - at) / span);
      w.first = at + static_cast<long long>(w.idx) * span + p.lead;
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;  // not reached: pos < U
}

// The walk's next part; false at its end.
__device__ __forceinline__ bool tree_next(const TreeParams& p, int bn, TreeWalk& w, TreePart& s) {
  if (w.pos < w.first) w.pos = w.first;
  if (w.pos >= w.end) return false;
  s.b = w.b;
  s.bh = w.b * p.h_kv + w.idx / p.row_blocks;
  s.rb = w.idx % p.row_blocks;
  s.L = w.L;
  s.t0 = static_cast<int>(w.pos - w.first);
  const long long left = w.end - w.pos;
  s.t1 = left < w.tiles - s.t0 ? s.t0 + static_cast<int>(left) : w.tiles;
  s.whole = s.t0 == 0 && s.t1 == w.tiles;
  s.unit = static_cast<long long>(w.b) * p.h_kv * p.row_blocks + w.idx;
  s.slot = s.unit + w.cta;
  w.pos += s.t1 - s.t0;
  if (s.t1 == w.tiles && w.pos < w.end) {
    w.first += w.tiles + p.lead;
    if (++w.idx == p.h_kv * p.row_blocks) {
      w.idx = 0;
      ++w.b;
      w.L = tree_len(p, w.b);
      w.tiles = tiles_of(w.L, bn);
    }
  }
  return true;
}

}  // namespace attn
