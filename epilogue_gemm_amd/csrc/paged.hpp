// paged.hpp -- arithmetic of the paged key-value cache that the append and
// the decode attention share: lengths, pages and the split of a batch's keys
// into pieces.  Plain functions of integers, for device and host alike (the
// CPU tests compile them with a host compiler and check every bound).
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define GE_HD __host__ __device__ __forceinline__
#else
#define GE_HD inline
#endif

namespace ge {
namespace paged {

constexpr int kUnit = 128;  // keys are split in units of this many (4 waves x 32)

// Tokens of a sequence: its stored length clamped to what its row of the
// page table can hold (cap = width * page_size < 2^31).
GE_HD int seq_len(int stored, int cap) { return stored < 0 ? 0 : stored < cap ? stored : cap; }

// A page table entry that names a page of the cache, else -1.
GE_HD int page_or_none(int entry, int num_pages) { return entry >= 0 && entry < num_pages ? entry : -1; }

// n / d for n below 2^27 and d from 1 to 4096 (positions and page sizes in
// groups of 16), as a product and a shift: m = ceil(2^p / d) with 2^p >= 2^27 d,
// so that m d exceeds 2^p by less than d and n (m d - 2^p) stays below 2^p.
struct Divider {
  uint32_t m;
  int p;
};
GE_HD Divider make_divider(int d) {
  int p = 27;
  while (((int64_t)1 << (p - 27)) < d) ++p;
  return Divider{(uint32_t)((((uint64_t)1 << p) + d - 1) / d), p};
}
GE_HD int divide(int n, Divider d) { return (int)(((uint64_t)(uint32_t)n * d.m) >> d.p); }

// Row number of (page, head, slot) in a [num_pages, heads, page_size] array.
GE_HD int64_t row_of(int page, int heads, int head, int page_size, int slot) {
  return ((int64_t)page * heads + head) * page_size + slot;
}

// Where the new token `row` of a sequence whose rows end before `end` goes:
// its position, or -1 when that is outside the sequence or the table.
GE_HD int new_position(int stored_len, int end, int row, int cap) {
  const int64_t p = (int64_t)stored_len - ((int64_t)end - row);
  return p >= 0 && p < cap ? (int)p : -1;
}

// Units of a sequence (at most 2^24).
GE_HD int units_of(int len) { return len / kUnit + (len % kUnit != 0); }

// The keys of a batch are split evenly over its workgroups: with U the units
// of all sequences and `columns` the (key head, query tile) pairs, unit u of
// column c has number f = c U + u, of F = columns * U < 2^31 numbers, and each
// of n workgroups takes a share of consecutive ones, from floor(w F / n) on.  A
// sequence's units in one column are then cut into pieces where shares end.
// No share is empty: of more workgroups than units the first F take one each.
// The larger shares lie evenly among the others, so that any k consecutive ones
// hold more than k F / n - 1 numbers (all of them first would leave the last
// columns to the smaller ones, up to twice as many pieces: pieces_bound).
// Workgroups that share F units: all of `most`, but where that is two for
// each of 256 CUs, one each up to two units a workgroup (fewer pieces are
// joined sooner: 16 x 1000 E4M3 of mixed lengths, 8 heads of 64, some 560
// units, 12.7 us with 256, 15.6 with 512; 4 x 8192, 1400 units, 14.5 and
// 13.7).  Not numbers between, which leave some CUs two and others one (64 x
// 1000, D = 128, 40.7 us with 280 of them, 512 32.7).
GE_HD int workgroups_of(int F, int most) { return most > 256 && F <= 2 * most ? 256 : most; }
struct Shares {
  int n, base, more;  // shares, numbers in each, and how many have one more
  uint32_t inv;       // 2^32 / n, rounded up (n = 1: 0, as `more` then is)
  float ratio;        // n / F
};
GE_HD Shares make_shares(int F, int workgroups) {
  const int n = F < workgroups ? F : workgroups;
  if (n == 0) return Shares{0, 0, 0, 0, 0.0f};
  return Shares{n, (int)((uint32_t)F / (uint32_t)n), (int)((uint32_t)F % (uint32_t)n), 0xffffffffu / (uint32_t)n + 1,
                (float)n / (float)F};
}
// floor(w F / n), with F = n base + more: w more is below 2^18 (n is 512 at
// most), so that inv's error adds less than 2^-14, and so less than 1 / n.
GE_HD int share_begin(Shares s, int w) {
  return w * s.base + (int)(((uint64_t)(uint32_t)(w * s.more) * s.inv) >> 32);
}
// The share that has number f < F: f n / F in fp32 is within one of it, as
// every rounding is at most 2^-24 of a number of at most n.
GE_HD int share_of(Shares s, int f) {
  const int at = (int)((float)f * s.ratio), w = at < s.n ? at : s.n - 1;
  return w + (w + 1 < s.n && share_begin(s, w + 1) <= f) - (share_begin(s, w) > f);
}

// The share of a workgroup < n.  Workgroups go to the 8 XCDs in turn: consecutive
// shares go to one XCD, so that all have as many of the larger ones (share w to
// workgroup w, these can all fall on one: 48 x 700, 8 heads of 128, bf16, 24.2 and
// 22.1 us; 64 x 1000 E4M3 27.8 and 26.4).  Other n than multiples of 8 are those of
// few units, one a share.
GE_HD int share_at(Shares s, int workgroup) {
  return s.n % 8 != 0 ? workgroup : workgroup % 8 * (s.n / 8) + workgroup / 8;
}

// A wave's tiles of 32 keys are 128 keys apart, from key k1 on; tile `last` is its
// last one before kend.  The key whose page is looked up for one of the two
// groups of 16 of a tile: past the sequence's end the tile's first, past the last
// tile -1 (by the tile's number: near 2^31 the keys of tiles past it are no ints).
GE_HD int looked_up_key(int k1, int kend, int last, int tile, int group) {
  if (tile > last) return -1;
  const int k = k1 + 128 * tile;
  return kend - k > 16 * group ? k + 16 * group : k;
}

// The pieces of a cut sequence are joined by the last of its workgroups when
// that takes at most kRounds rounds of loads (a round: kBatch pieces for each
// group of threads, a group being rows * head_dim / 4 of the 256), else by
// the join kernel.
constexpr int kBatch = 16, kRounds = 5;
GE_HD bool joined_here(int pieces, int rows, int head_dim) {
  const int most = 1024 / head_dim;  // rows at a time
  const int passes = (rows + most - 1) / most, groups = rows < most ? most / rows : 1;
  return passes * ((pieces + kBatch * groups - 1) / (kBatch * groups)) <= kRounds;
}
// The most pieces a sequence of up to `cap` tokens can be cut into: one per
// unit, and one per share of a column and the two it ends in.  (The inner p - 2
// of its p shares are whole, and the outer two have a unit of it at least: of the
// U = F / columns units it can have, (p - 2) F / n - 1 < U - 2, and so p - 2 < n /
// columns, for every n up to `workgroups`.)
GE_HD int64_t pieces_bound(int64_t cap, int columns, int workgroups) {
  const int64_t units = (cap + kUnit - 1) / kUnit, shares = workgroups / columns + 2;
  return units < shares ? units : shares;
}

}  // namespace paged
}  // namespace ge
