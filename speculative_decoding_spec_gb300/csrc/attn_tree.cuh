// attn_tree.cuh -- how the attention of drafted trees is cut into pieces, shared
// by its kernels (attn_tree.cu, attn_tree_tc.cu) and the one that joins them.
//
// Sequence b has n rows, so n * G query rows on each KV head (G query heads a
// KV head; query row i*G + g), in tiles of `tile` rows; `tpu` tiles make a unit,
// which reads its KV head's blocks of `blk` keys once. The units of all
// sequences, in order (sequence, KV head, unit), lie on one axis on which a
// block of a unit has the length of the unit's tiles, and a unit's beginning that of
// `head` tiles (its queries' way in and its results' way out take as long). CTA c
// takes the c-th of `ctas` equal parts of that axis, so every CTA gets the same work
// whatever the lengths; a part may end inside a unit, and may hold several.
//
// A unit that lies in one part is finished there. Of a unit that is cut, each
// CTA leaves its rows' sums unnormalised, with their maxima and sums, in one of
// its two slots (slot 2c: a piece that does not start the unit; 2c + 1: one that
// does; a part can hold one of each), and tree_join_kernel adds them up.
#pragma once
#include "common.cuh"

namespace spec {
namespace tree {

constexpr int PAGE = 64;
constexpr float LOG2E = 1.4426950408889634f;

struct Plan {
  int blk, tile;             // keys a block, rows a tile: powers of two, as shifts
  int tpu, grid;             // tiles a unit (1 or 2), CTAs
  int min_cost, head;        // a part is not made shorter than this; length of a unit's beginning
  int units;                 // > 0: no cuts, a CTA a unit, so many a KV head
  int G;                     // query heads a KV head
  uint32_t inv_g;            // ceil(2^32 / G): rows below 2^16 are divided by G with a product
  SPEC_DEV int row_of(int q) const { return G == 1 ? q : (int)__umulhi((uint32_t)q, inv_g); }
};
inline void plan_heads(Plan& p, const TreeArgs& a) {
  p.G = a.nq / a.nkv;
  p.inv_g = (uint32_t)(((1ull << 32) + p.G - 1) / p.G);
}

// Sequence b of a call: slot, committed length, rows in use. A sequence whose
// numbers are out of range has no rows: its outputs stay as they are.
struct Seq {
  int slot, len, rows;
  bool ok;
};
SPEC_DEV Seq seq_of(const TreeArgs& a, int b) {
  Seq s;
  s.slot = a.seq_ids[b];
  s.ok = s.slot >= 0 && s.slot < a.n_slots;
  s.len = s.ok ? a.seq_len[s.slot] : 0;
  s.rows = a.n_rows ? a.n_rows[b] : a.R;
  s.ok = s.ok && s.len >= 0 && s.rows >= 0 && s.rows <= a.R &&
         (long long)s.len + s.rows <= min((long long)a.max_pages * PAGE, TREE_POSITIONS_MAX);
  if (!s.ok) s.rows = 0;
  return s;
}
SPEC_DEV int tiles_of(const Plan& p, int rows) { return (rows * p.G + (1 << p.tile) - 1) >> p.tile; }
SPEC_DEV int blocks_of(const Plan& p, const Seq& s) { return s.rows ? (s.len + s.rows + (1 << p.blk) - 1) >> p.blk : 0; }

// A KV head's part of the axis: T tiles of nb blocks.
SPEC_DEV int pair_length(const Plan& p, int T, int nb) { return nb * T + (T + p.tpu - 1) / p.tpu * p.head; }
SPEC_DEV int cost_of(const TreeArgs& a, const Plan& p, int b) {
  const Seq s = seq_of(a, b);
  return a.nkv * pair_length(p, tiles_of(p, s.rows), blocks_of(p, s));  // (the launcher keeps the axis below 2^31)
}
// This lane's sequence of 32: where it ends, from the start of the first.
SPEC_DEV int scan32(int c) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL, c, o);
    if (lane >= o) c += v;
  }
  return c;
}
// The sequences' places on the axis, by a whole warp: 32 of them in the lanes, the
// others looked at again when they are asked for.
struct Axis {
  int mine, end0, total;  // this lane's sequence's end, the 32 sequences', the axis's
  SPEC_DEV Axis(const TreeArgs& a, const Plan& p) {
    const int lane = threadIdx.x & 31;
    mine = scan32(lane < a.B ? cost_of(a, p, lane) : 0);
    end0 = total = __shfl_sync(FULL, mine, 31);
    for (int b0 = 32; b0 < a.B; b0 += 32) {
      int c = b0 + lane < a.B ? cost_of(a, p, b0 + lane) : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(FULL, c, o);
      total += c;
    }
  }
  // The sequence that holds x (< total), and where it starts.
  SPEC_DEV int at(const TreeArgs& a, const Plan& p, int x, int& start) const {
    const int lane = threadIdx.x & 31;
    int base = 0, end = mine, b0 = 0, last = end0;
    while (x >= last) {
      b0 += 32;
      base = last;
      end = base + scan32(b0 + lane < a.B ? cost_of(a, p, b0 + lane) : 0);
      last = __shfl_sync(FULL, end, 31);
    }
    const int i = __ffs(__ballot_sync(FULL, end > x)) - 1;
    const int before = __shfl_sync(FULL, end, (i + 31) & 31);
    start = i ? before : base;
    return b0 + i;
  }
};

// The axis cut into parts: the first `more` of them are one longer than the others.
struct Cut {
  int total, ctas, base, more;
  SPEC_DEV Cut(const Plan& p, int n) : total(n) {
    ctas = max(1, min((n + p.min_cost - 1) / p.min_cost, p.grid));
    base = n / ctas;
    more = n - base * ctas;
  }
  SPEC_DEV int start(int c) const { return base * c + min(c, more); }
  SPEC_DEV int part_of(int x) const {  // x < total
    const int edge = (base + 1) * more;
    return x < edge ? x / (base + 1) : more + (x - edge) / base;
  }
};

// A unit: its place on the axis and what it covers.
struct Unit {
  int b, kvh, u;       // sequence, KV head, unit of the pair
  int nb, w;           // blocks, tiles
  int start;
};
// The unit that holds position x (< total). By a whole warp.
SPEC_DEV Unit unit_at(const TreeArgs& a, const Plan& p, const Axis& axis, int x) {
  Unit n;
  int start;
  n.b = axis.at(a, p, x, start);
  const Seq s = seq_of(a, n.b);
  const int T = tiles_of(p, s.rows);
  n.nb = blocks_of(p, s);
  const int pair = pair_length(p, T, n.nb), unit = n.nb * p.tpu + p.head, off = x - start;
  n.kvh = off / pair;
  n.u = (off - n.kvh * pair) / unit;
  n.w = min(p.tpu, T - n.u * p.tpu);
  n.start = start + n.kvh * pair + n.u * unit;
  return n;
}
// The blocks of unit n in [x0, x1) of the axis.
SPEC_DEV int first_block(const Plan& p, const Unit& n, int x) {
  const int off = x - n.start - p.head;
  return off <= 0 ? 0 : min((off + n.w - 1) >> (n.w - 1), n.nb);
}

// The pieces of units in this CTA's part, one after the other.
// Without cuts (p.units) a CTA has one unit, on an axis of its own.
struct Walk {
  Unit n;
  Seq s;
  int k0, N;                            // first block, blocks
  int x, x1;
  // This CTA's part; false where there is none. By a whole warp.
  SPEC_DEV bool begin(const TreeArgs& a, const Plan& p) {
    if (p.units) {
      const int pair = blockIdx.x / p.units;
      n.u = blockIdx.x - pair * p.units;
      n.b = pair / a.nkv;
      n.kvh = pair - n.b * a.nkv;
      s = seq_of(a, n.b);
      n.w = min(p.tpu, tiles_of(p, s.rows) - n.u * p.tpu);
      n.nb = blocks_of(p, s);
      n.start = x = 0;
      x1 = n.nb * n.w + p.head;
      return n.w > 0;
    }
    const Axis axis(a, p);
    const Cut cut(p, axis.total);
    if ((int)blockIdx.x >= cut.ctas || cut.total == 0) return false;
    x = cut.start(blockIdx.x);
    x1 = cut.start(blockIdx.x + 1);
    n = unit_at(a, p, axis, x);
    s = seq_of(a, n.b);
    return true;
  }
  SPEC_DEV bool pieces(const TreeArgs& a, const Plan& p) {  // from unit n on: the next one with blocks here
    for (;;) {
      if (x >= x1) return false;
      k0 = first_block(p, n, x);
      N = first_block(p, n, x1) - k0;
      if (N > 0) return true;
      step(a, p);
    }
  }
  SPEC_DEV void step(const TreeArgs& a, const Plan& p) {
    x = n.start + p.head + n.nb * n.w;
    n.start = x;
    if (x >= x1) return;
    int T = tiles_of(p, s.rows);
    if ((n.u + 1) * p.tpu < T) {
      ++n.u;
    } else {
      n.u = 0;
      if (++n.kvh == a.nkv) {
        n.kvh = 0;
        do s = seq_of(a, ++n.b);        // (x < x1 <= the axis's end: there is one)
        while (s.rows == 0);
        T = tiles_of(p, s.rows);
        n.nb = blocks_of(p, s);
      }
    }
    n.w = min(p.tpu, T - n.u * p.tpu);
  }
};

// Bit j of path[r]: row j is row r or an ancestor of it (rows below 64). By
// threads 0 .. 63 of the CTA between barriers of all of them: `sync`. A parent
// that is not an earlier row counts as none.
template <class Sync>
SPEC_DEV void paths(const TreeArgs& a, int b, int rows, unsigned long long* path, int* up, int t, Sync sync) {
  if (t < 64) {
    int p = -1;
    if (t < rows) {
      p = a.parents ? a.parents[(size_t)b * a.R + t] : t - 1;
      if (p < 0 || p >= t) p = -1;
    }
    path[t] = 1ull << t;
    up[t] = p;
  }
  sync();
  for (int step = 1; step < rows; step <<= 1) {  // (pointer jumping: a path of 2^i rows after i steps)
    unsigned long long m = 0;
    int p = -1;
    if (t < 64 && up[t] >= 0) {
      m = path[up[t]];
      p = up[up[t]];
    }
    sync();
    if (t < 64) {
      path[t] |= m;
      up[t] = p;
    }
    sync();
  }
}
// Which of the 64 keys from `key0` on a row with this path sees.
SPEC_DEV unsigned long long visible(unsigned long long path, int len, int key0) {
  const long long off = (long long)len - key0;  // committed keys from key0 on
  if (off >= 64) return ~0ull;
  if (off >= 0) return ((1ull << off) - 1) | (path << off);
  return off > -64 ? path >> -off : 0ull;
}

// What a call finds wrong: sequences out of range, parents that are not earlier
// rows, pages that are not there. By threads 0 .. nthr - 1 (t) for the sequences
// first, first + step, ... With cuts a CTA looks at its share of them and leaves what
// it found, or a wait that ran out, in a word of its own, and the join gathers those;
// without, the first CTA looks at all.
SPEC_DEV bool bad_input(const TreeArgs& a, const Plan& p, int t, int nthr) {
  bool bad = false;
  if (p.units && blockIdx.x) return false;
  for (int b = p.units ? 0 : blockIdx.x; b < a.B; b += p.units ? 1 : gridDim.x) {
    const Seq s = seq_of(a, b);
    bad |= !s.ok;
    if (a.parents)
      for (int r = t; r < s.rows; r += nthr) {
        const int q = a.parents[(size_t)b * a.R + r];
        bad |= q < -1 || q >= r;
      }
    const int pages = s.rows ? (s.len + s.rows + PAGE - 1) / PAGE : 0;
#pragma unroll 4
    for (int i = t; i < pages; i += nthr) {
      const int g = a.block_table[(size_t)s.slot * a.max_pages + i];
      bad |= g < 0 || g >= a.n_pages;
    }
  }
  return bad;
}
// Where this CTA's findings go.
SPEC_DEV int* findings(const TreeArgs& a, const Plan& p) { return p.units ? a.err : a.flags + blockIdx.x; }
SPEC_DEV void found(const TreeArgs& a, const Plan& p, bool bad) {  // by one thread
  if (!p.units || blockIdx.x == 0) *findings(a, p) = bad ? SPEC_ERR_CAPACITY : 0;
}
// A page id that is out of range reads page 0 (the call records it).
SPEC_DEV int page_of(const TreeArgs& a, int slot, int i) {
  const int g = a.block_table[(size_t)slot * a.max_pages + i];
  return g < 0 || g >= a.n_pages ? 0 : g;
}

// The tcgen05 kernel (attn_tree_tc.cu).
bool tc_ok(const TreeArgs& a);
Plan tc_plan(const TreeArgs& a);
void tc_setup();
int tc_launch(const TreeArgs& a, const Plan& p, cudaStream_t st);

}  // namespace tree
}  // namespace spec
