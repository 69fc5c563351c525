// attend_walk.cuh -- which part of a batch's attention each CTA takes. Plain arithmetic on the host and the device
// (tests compile it for the CPU).
//
// A unit is one sequence, one cache head and a block of its new tokens: the query heads of a cache head and consecutive tokens fill
// the 128 rows of one or two MMA tiles. A unit's items are the tiles of 128 keys that any of its rows sees (one, empty, where
// none sees any, so that its rows are written). All units' items, unit after unit, are dealt to the CTAs in equal consecutive
// runs: every CTA has the same work to within one tile whatever the lengths are, and a unit that a run's end cuts is put together from
// its parts. The lengths stay on the device; each CTA finds its run from them (paged_attention.cu).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define FP8GB_HD __host__ __device__ __forceinline__
#else
#define FP8GB_HD inline
#endif

namespace fp8gb {
namespace attend {

constexpr int kTile = 128;  // keys of an item, rows of an MMA tile

FP8GB_HD int least(int a, int b) { return a < b ? a : b; }
FP8GB_HD int most(int a, int b) { return a > b ? a : b; }

// A sequence: its first row, new tokens, cached tokens, and how many of those the page table reaches.
struct Seq {
  int first, n, len, seen;
};

FP8GB_HD Seq seq_of(int start, int end, int kv_len, int tokens, int capacity) {
  Seq s;
  s.first = least(most(start, 0), tokens);
  s.n = most(least(most(end, 0), tokens) - s.first, 0);
  s.len = most(kv_len, 0);
  s.seen = least(s.len, capacity);
  return s;
}

// Keys that new token i sees: lo .. hi - 1.
struct Keys {
  int lo, hi;
};
FP8GB_HD Keys keys_of(const Seq& s, int i, int window) {
  const int end = most(s.len - s.n + i, -1) + 1;  // position + 1
  Keys k;
  k.hi = least(end, s.seen);
  k.lo = window > 0 ? most(end - window, 0) : 0;
  return k;
}

// Tiles of keys that tokens i0 .. i1 - 1 see any of (some of the middle ones see none where lo > hi).
FP8GB_HD Keys tiles_of(const Seq& s, int i0, int i1, int window) {
  Keys t{0, 0};
  i1 = least(i1, s.n);
  if (i0 >= i1) return t;
  const int hi = keys_of(s, i1 - 1, window).hi;
  t.hi = (hi >> 7) + ((hi & 127) != 0);
  t.lo = least(keys_of(s, i0, window).lo >> 7, t.hi);
  return t;
}

// Whether a tile holds keys that some row of tokens i0 .. i1 - 1 does not see.
FP8GB_HD bool is_edge(const Seq& s, int i0, int i1, int window, int tile) {
  i1 = least(i1, s.n);
  return tile * kTile + kTile > keys_of(s, i0, window).hi || tile * kTile < keys_of(s, i1 - 1, window).lo;
}

FP8GB_HD int items_of(const Seq& s, int block, int per, int window) {
  const Keys t = tiles_of(s, block * per, block * per + per, window);
  return most(t.hi - t.lo, 1);
}

// CTA c of `ctas` takes items begin_of(c) .. begin_of(c + 1) - 1 of `total`; cta_of is the one that takes item x.
// (Small numbers in 32 bits: a division in 64 takes some hundred instructions. Both have to be: a long prompt's items pass 32 bits.)
FP8GB_HD int64_t quotient(int64_t a, int64_t b) {
  return (static_cast<uint64_t>(a) | static_cast<uint64_t>(b)) >> 32 == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}
FP8GB_HD int64_t begin_of(int64_t total, int c, int ctas) { return quotient(total * c, ctas); }
FP8GB_HD int cta_of(int64_t total, int64_t x, int ctas) { return static_cast<int>(quotient((x + 1) * ctas - 1, total)); }

// A CTA's run as segments, a unit or a part of one each. Source: seqs, and seq(int), a
// sequence.
struct Place {
  int seq, head, block, off;  // off: items of the unit before this CTA's
  int64_t item, end;          // the run's next item and its end
};

template <typename Source>
struct Walk {
  const Source& src;
  int heads, per, window;
  Place at;
  Seq s;
  Keys tiles;       // the unit's
  int items, take;  // the unit's, and this CTA's of them
  int a, b;         // this CTA's tiles: none in an empty unit
  int filled;       // segments with tiles before this one

  FP8GB_HD Walk(const Source& source, const Place& start, int n_heads, int tokens_per_block, int win) : src(source), heads(n_heads), per(tokens_per_block), window(win), at(start), filled(0) {
    take = 0;
    if (at.item < at.end) {
      s = src.seq(at.seq);
      set();
    }
  }
  FP8GB_HD bool live() const { return at.item < at.end; }
  FP8GB_HD bool first() const { return at.off == 0; }
  FP8GB_HD bool last() const { return at.off + take == items; }
  FP8GB_HD void set() {
    tiles = tiles_of(s, at.block * per, at.block * per + per, window);
    items = most(tiles.hi - tiles.lo, 1);
    const int64_t left = at.end - at.item;
    take = items - at.off;
    if (left < take) take = static_cast<int>(left);
    a = least(tiles.lo + at.off, tiles.hi);
    b = least(tiles.lo + at.off + take, tiles.hi);
  }
  FP8GB_HD void next() {
    filled += a < b;
    at.item += take;
    if (!live()) return;
    at.off = 0;
    ++at.block;
    if (at.block * per >= s.n) {
      at.block = 0;
      if (++at.head == heads) {
        at.head = 0;
        do {
          if (++at.seq >= src.seqs) {  // (lengths that changed under the call)
            at.item = at.end;
            return;
          }
          s = src.seq(at.seq);
        } while (s.n == 0);
      }
    }
    set();
  }
  FP8GB_HD bool edge(int tile) const { return is_edge(s, at.block * per, at.block * per + per, window, tile); }
  // tiles of this CTA's part that rows of tokens i0 .. i0 + n - 1 of the block need
  FP8GB_HD Keys part_of(int i0, int n) const {
    Keys t = tiles_of(s, at.block * per + i0, at.block * per + i0 + n, window);
    t.lo = most(t.lo, a);
    t.hi = least(t.hi, b);
    return t;
  }
};

}  // namespace attend
}  // namespace fp8gb
