// sample.cu -- one token per row of logits with temperature, top-k, top-p,
// min-p and a given uniform number, and the sampled accept of drafts.
//
// The pages speculate greedily; a served request brings sampling settings of
// its own. For a row of logits l with maximum m the weights are
// w_i = exp((l_i - m) / T); the filters keep a prefix of the order (logit
// descending, index ascending), so together they are ONE cut (key, index) of
// that order: top-k cuts at its k-th token, top-p at the first token whose
// preceding mass reaches p times the top-k mass, min-p at weight min_p. The token
// is the lowest index at which the kept mass, summed in index order, exceeds
// u times the kept mass.
//
// A draft is a single proposed token (the drafter's distribution is a point
// mass), so accepting it when the target's sample equals it IS rejection
// sampling: it is kept with probability p(d), and a rejected position emits a
// token distributed as p without d.
//
// Weights are integers: w_i in units of 2^-44 of the largest, rounded (a
// choice: tokens below 2^-45 of the most likely one count as zero). Their sums
// are exact, so the cut and the token do not depend on the order of the
// additions or the number of CTAs. The weight itself is evaluated to about 2^-37
// (the exponent as a float pair, a table of 4096 powers), because a token is
// decided by a sum of up to V weights next to a border: at the 2^-24 of plain
// floats about one token in 10^4 would differ from the 64-bit definition; here
// none of 27600 rows of 4096 to 262144 tokens did.
//
// Large calls without filters: a first kernel takes the rows in chunks of 4096
// tokens, in one pass that leaves each chunk's maximum and the sum of its weights,
// relative to that maximum; it loads the SMs evenly, with the next chunk's loads
// in flight under the exponentials of the last. A CTA a row then adds the sums
// up in the row's units, finds the drawn chunk and draws inside it.
//
// Otherwise a thread-block cluster takes a row; its CTAs push what the others
// need into their shared memory, so that a phase costs one cluster barrier. Scan
// 1 finds the maximum and the maxima of the row's segments (up to 1024). Without
// top-k and top-p, scan 2 sums the weights and the warp that holds the
// drawn mass finds the token. With top-k, scan 2 lists the tokens down to the
// k-th largest segment maximum -- at least k tokens, and rarely many more -- and
// the first CTA cuts and draws among those alone. With top-p alone, scan 2 adds
// up a histogram of 2048 bins, linear in the exponent, of exact masses (three
// 15-bit digits), and the tokens up to the bin in which the cut lies are listed
// and drawn from in the same way. Where the listed tokens are too many, those of
// that bin alone are listed and sorted for the cut (a radix search of their keys
// where even they are too many; top-k then has a histogram of counts), and a
// last scan sums the kept weights.
//
// What bounds it: one row, latency (13 us with top-k, about 20 dependent phases of
// 0.3 to 2 us); many rows, the weights: the table's random 8-byte reads of shared
// memory (about 6 wavefronts a warp, 0.2 cycles a token of an SM) and the
// histogram's atomics, not the 1 MB a row out of HBM. 262144 fp32 logits a row: 40
// rows at temperature 28.5 us (1.5 TB/s; the bytes alone 6.2 us), with top-k 50 36
// us; 64 rows with top-p of mixed breadth 104 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <utility>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace spec {

namespace {

typedef unsigned long long ull;

constexpr int NT = 512;             // threads of a CTA
constexpr int NW = NT / 32;
constexpr int BINS = 2048;
constexpr int BPT = BINS / NT;      // consecutive bins of a thread
constexpr int WBITS = 44;           // fraction bits of a weight
constexpr int DIGIT = 15;           // bits of a mass digit
constexpr int DIGIT_TOKENS = 120000;  // tokens of a CTA whose digits surely sum in 32 bits
constexpr int TAB_LOG = 12;
constexpr int TAB = 1 << TAB_LOG;   // 2^(-j/4096)
constexpr int MAX_C = 16;           // CTAs on one row (a thread-block cluster)
constexpr int LIST = 1024;          // tokens a CTA lists
constexpr int FEW = 2048;           // tokens the first CTA sorts
constexpr int COUNTED = NT / 2;     // at most so many are counted instead
constexpr int CHUNK_TOKENS = 4096;  // tokens of a chunk of the chunk kernel
constexpr int CNT = 256;            // its threads
constexpr int CNW = CNT / 32;
constexpr int SEG_MAX = 1024;       // segments of a row (the elements of 1, 2, 4 or 8 lanes)
constexpr int SEG_BINS = NT;        // bins of the segment maxima
constexpr float Z_END = 46.f;       // weights are zero beyond this exponent
constexpr int CHUNK = 8;            // vectors of a lane whose sum is kept apart, doubled until
constexpr int CHUNKS = 32;          // a warp's part has at most 32 chunks
constexpr int IDX_BITS = 19;        // V <= 2^19: an index and a 45-bit weight share a word

// 2^(44 - j/4096), from the exponential series at compile time.
struct Table {
  ull v[TAB];
};
constexpr double series_exp(double x) {
  double s = 1.0, t = 1.0;
  for (int i = 1; i < 24; ++i) {
    t *= x / i;
    s += t;
  }
  return s;
}
constexpr Table make_table() {
  Table t = {};
  for (int j = 0; j < TAB; ++j)
    t.v[j] = (ull)(series_exp(-0.69314718055994530942 * j / TAB) * (double)(1ull << WBITS) + 0.5);
  return t;
}
__device__ const Table g_table = make_table();

// A cut of the order: tokens with a smaller key, and those of this key up to
// this index, are kept.
struct Cut {
  uint32_t key;
  int idx;
};

struct Shared {
  ull tab[TAB];
  union {
    unsigned int hist[3][BINS];  // counts, or the masses' digits
    ull mass[BINS];              // radix search inside a bin
    ull sort[FEW];               // first CTA: the listed tokens
  };
  uint32_t list_key[LIST];
  int list_idx[LIST];
  int listed;                // tokens this CTA listed (more than LIST: they did not fit)
  // pushed by every CTA of the cluster
  ull x_best[MAX_C];         // packed maximum
  float x_low[MAX_C];        // minimum
  int x_nan[MAX_C];
  ull x_total[MAX_C];        // sum of the weights
  float seg[SEG_MAX];        // segment maxima
  int gathered;              // first CTA: tokens listed by all
  unsigned int seg_bins[SEG_BINS];
  Cut cut;                   // pushed by the first CTA: the cut of the row
  ull chunk[NW][CHUNKS];     // sums of the warps' chunks
  ull wsum[NW];
  ull total;                 // this CTA's sum, read by the cluster
  int bin;                   // crossing bin
  ull before, at;            // amount before it, and in it
  int found;                 // index found by find_in_order, written by its owner
  int base;
  int r;                     // tokens kept of the sorted ones
};

// Scale of a row: weights are 2^-z with z = (m - x) * (sh + sl); bins are
// linear in z.
struct Scale {
  float m, sh, sl, bins;
  // Monotone in x (each rounding is), so bins are ranges of the order.
  SPEC_DEV float place(float x) const { return (m - x) * sh * bins; }
  SPEC_DEV int bin(float x) const {
    if (m == INFINITY) return x == INFINITY ? 0 : BINS - 1;
    return (int)fminf(place(x), (float)(BINS - 1));
  }
};

// 2^(n-1), half a unit before the shift by n: a weight is rounded, not cut off.
// (The bias of V cut-off weights would move a border among the unlikely tokens
// by as much as their weights.) From n = 31 on a little less, within 32 bits.
SPEC_DEV float half_unit(int n) { return __int_as_float((min(n, 30) << 23) + 0x3f000000); }

// The weight of logit x in units of 2^-WBITS. z is formed as a float pair (an
// exact difference, an exact product), split into n + j/4096 + g, and
// 2^-z = 2^-n * tab[j] * e^(-g ln 2) with a quadratic (Tang's table-driven
// reduction, ACM TOMS 15(2), 1989). val: the weight as a float.
SPEC_DEV ull weight(const Scale& r, const ull* tab, float x, float* val = nullptr) {
  if (r.m == INFINITY) {
    if (val) *val = x == INFINITY ? 1.f : 0.f;
    return x == INFINITY ? 1ull << WBITS : 0ull;
  }
  const float d = __fsub_rn(r.m, x);
  const float bb = __fsub_rn(d, r.m);
  const float e = __fadd_rn(__fsub_rn(r.m, __fsub_rn(d, bb)), __fsub_rn(-x, bb));   // d + e == m - x
  float p = __fmul_rn(d, r.sh);
  const float pe = fmaf(e, r.sh, fmaf(d, r.sl, fmaf(d, r.sh, -p)));
  p = fminf(p, 63.f);
  // round(4096 p) in the low bits of p + 1.5 * 2^(23 - 12)
  const float t = __fadd_rn(p, 12582912.f / TAB);
  const float g = __fadd_rn(__fsub_rn(p, __fsub_rn(t, 12582912.f / TAB)), pe);      // |g| <= 2^-13
  const float q = __fmul_rn(fmaf(g, 0.240226507f, -0.693147181f), g);               // 2^-g - 1
  const uint32_t j = __float_as_uint(t);
  const ull T = tab[j & (TAB - 1)];
  const int n = (j >> TAB_LOG) & 63;
  // the table value as a float: its 24 leading bits (2^43 <= T <= 2^44)
  const float Tf = __uint_as_float((uint32_t)(T >> (WBITS - 24)) + 0x4a800000u) * (float)(1 << (WBITS - 24));
  const ull v = T + (long long)__float2int_rn(fmaf(Tf, q, half_unit(n)));
  if (val) *val = fmaf(Tf, q, Tf) * __int_as_float((127 - WBITS - n) << 23);
  return v >> n;
}

// The factor of logit x's weight as v * 2^-(WBITS + n), not yet cut to units.
SPEC_DEV ull weight_parts(const Scale& r, const ull* tab, float x, int& n) {
  n = 0;
  if (r.m == INFINITY) return x == INFINITY ? 1ull << WBITS : 0ull;
  const float d = __fsub_rn(r.m, x);
  const float bb = __fsub_rn(d, r.m);
  const float e = __fadd_rn(__fsub_rn(r.m, __fsub_rn(d, bb)), __fsub_rn(-x, bb));
  float p = __fmul_rn(d, r.sh);
  const float pe = fmaf(e, r.sh, fmaf(d, r.sl, fmaf(d, r.sh, -p)));
  if (!(p < 63.f)) return 0ull;
  const float t = __fadd_rn(p, 12582912.f / TAB);
  const float g = __fadd_rn(__fsub_rn(p, __fsub_rn(t, 12582912.f / TAB)), pe);
  const float q = __fmul_rn(fmaf(g, 0.240226507f, -0.693147181f), g);
  const uint32_t j = __float_as_uint(t);
  const ull T = tab[j & (TAB - 1)];
  n = (j >> TAB_LOG) & 63;
  const float Tf = __uint_as_float((uint32_t)(T >> (WBITS - 24)) + 0x4a800000u) * (float)(1 << (WBITS - 24));
  return T + (long long)__float2int_rn(__fmul_rn(Tf, q));
}
// A sum of weights relative to a chunk's maximum, in the row's units: times
// v * 2^-(WBITS + n), rounded down. Monotone in the sum.
SPEC_DEV ull in_row(ull sum, ull v, int n) {
  const ull lo = sum * v, hi = __umul64hi(sum, v);
  const int sh = WBITS + n;
  return sh < 64 ? (hi << (64 - sh)) | (lo >> sh) : hi >> (sh - 64);
}

// Two floats in one register pair, and Blackwell's packed operations on them.
SPEC_DEV ull pk(float a, float b) {
  ull r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
SPEC_DEV ull pk(float a) { return pk(a, a); }
SPEC_DEV void upk(ull p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
SPEC_DEV ull fma2(ull a, ull b, ull c) {
  ull r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
SPEC_DEV ull add2(ull a, ull b) {
  ull r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
SPEC_DEV ull mul2(ull a, ull b) {
  ull r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// weight() of two logits, operation for operation, in packed arithmetic (the
// scans that weigh a whole row are bound by their instructions).
SPEC_DEV void weight2(const Scale& r, const ull* tab, float x0, float x1, ull& w0, ull& w1) {
  if (r.m == INFINITY) {
    w0 = x0 == INFINITY ? 1ull << WBITS : 0ull;
    w1 = x1 == INFINITY ? 1ull << WBITS : 0ull;
    return;
  }
  constexpr float MAGIC = 12582912.f / TAB;
  const ull m = pk(r.m), x = pk(x0, x1), neg = pk(-1.f), sh = pk(r.sh);
  const ull d = fma2(x, neg, m), nb = fma2(d, neg, m);              // nb = -bb
  const ull e = add2(fma2(add2(d, nb), neg, m), fma2(x, neg, nb));
  ull np = mul2(d, pk(-r.sh));                                      // -p
  const ull pe = fma2(e, sh, fma2(d, pk(r.sl), fma2(d, sh, np)));
  float a, b;
  upk(np, a, b);
  np = pk(fmaxf(a, -63.f), fmaxf(b, -63.f));
  const ull t = fma2(np, neg, pk(MAGIC));
  const ull g = fma2(add2(np, add2(t, pk(-MAGIC))), neg, pe);
  // 2^-g - 1, in units that make its product with the table's 24 leading bits one with weight()'s
  constexpr float S = (float)(1 << (WBITS - 24));
  const ull q = mul2(fma2(g, pk(0.240226507f * S), pk(-0.693147181f * S)), g);
  upk(t, a, b);
  const uint32_t j0 = __float_as_uint(a), j1 = __float_as_uint(b);
  const ull T0 = tab[j0 & (TAB - 1)], T1 = tab[j1 & (TAB - 1)];
  const ull Tf = pk(__uint_as_float((uint32_t)(T0 >> (WBITS - 24)) + 0x4a800000u),
                    __uint_as_float((uint32_t)(T1 >> (WBITS - 24)) + 0x4a800000u));
  const int n0 = (j0 >> TAB_LOG) & 63, n1 = (j1 >> TAB_LOG) & 63;
  upk(fma2(Tf, q, pk(half_unit(n0), half_unit(n1))), a, b);
  w0 = (T0 + (long long)__float2int_rn(a)) >> n0;
  w1 = (T1 + (long long)__float2int_rn(b)) >> n1;
}

// The same out of line, where it is evaluated a few times.
__device__ __noinline__ ull weight_once(Scale r, const ull* tab, float x, float* val) { return weight(r, tab, x, val); }

// u * z for u in [0, 1), exactly, rounded down (up: rounded up).
SPEC_DEV ull scaled(float u, ull z, bool up) {
  const uint32_t b = __float_as_uint(u);
  const int e = max(1, (int)(b >> 23)), sh = 150 - e;           // u = m * 2^-sh, sh >= 24
  const ull m = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
  const ull lo = m * z, hi = __umul64hi(m, z);
  ull r, rest;
  if (sh < 64) {
    r = (hi << (64 - sh)) | (lo >> sh);
    rest = lo << (64 - sh);
  } else {
    r = sh < 128 ? hi >> (sh - 64) : 0ull;
    rest = lo | (sh < 128 ? hi << (128 - sh - 1) << 1 : hi);
  }
  return r + (up && rest ? 1 : 0);
}
// The mass at which top-p ends: at least 1, so that a token is kept.
SPEC_DEV ull top_p_mass(float p, ull z) { return p > 0.f ? max(1ull, scaled(p, z, true)) : 1ull; }
// The drawn mass, below z.
SPEC_DEV ull drawn_mass(float u, ull z) { return u > 0.f ? (u < 1.f ? scaled(u, z, false) : z - 1) : 0ull; }

// Order-preserving key, ascending from the best token: -0 counts as +0.
SPEC_DEV uint32_t rank_key(float x) { return ~ord_key(x + 0.f); }
SPEC_DEV float rank_val(uint32_t k) { return ord_val(~k); }

// The part of a row one warp owns, 16-byte vectors in index order; rows may
// start at any element, the first and last vectors are read element by element.
template <typename T>
struct Part {
  const T* p;
  int V, mis, v0, v1;   // vectors [v0, v1); vector v holds elements v * E - mis ...
  static constexpr int E = 16 / sizeof(T);
  static constexpr int U = 4;           // vectors a lane has in flight
  SPEC_DEV static float get(const uint4& q, int i) {
    const uint32_t w = sizeof(T) == 4 ? (i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w)
                                      : ((i >> 1) == 0 ? q.x : (i >> 1) == 1 ? q.y : (i >> 1) == 2 ? q.z : q.w);
    if (sizeof(T) == 4) return __uint_as_float(w);
    return (i & 1) ? bf16hi(w) : bf16lo(w);
  }
  SPEC_DEV static float one(const float* q) { return *q; }
  SPEC_DEV static float one(const __nv_bfloat16* q) { return __bfloat162float(*q); }
  SPEC_DEV void bind(const T* row, int V_, int cta, int C) {
    p = row;
    V = V_;
    mis = (int)(((uintptr_t)row & 15) / sizeof(T));
    const int nvec = (V + mis + E - 1) / E;
    const int per = (nvec + C * NW - 1) / (C * NW);
    const int w = cta * NW + (threadIdx.x >> 5);
    v0 = min(nvec, w * per);
    v1 = min(nvec, v0 + per);
  }
  // Vectors v, v + 32, ... of a lane, U in flight; q[j] is valid where the
  // returned bit j is set (the others lie outside the part or on its edges).
  SPEC_DEV unsigned int load(int v, uint4 (&q)[U]) const {
    unsigned int ok = 0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i0 = (v + 32 * j) * E - mis;
      if (v + 32 * j < v1 && i0 >= 0 && i0 + E <= V) {
        q[j] = *reinterpret_cast<const uint4*>(p + i0);
        ok |= 1u << j;
      }
    }
    return ok;
  }
  // f(index, value) of the vectors that hold a value of at least x0.
  template <typename F>
  SPEC_DEV void each_above(float x0, F f) const {
    if (v0 < v1) edge(v0, 0, f);
#pragma unroll 1
    for (int v = v0 + (int)(threadIdx.x & 31); v < v1; v += 32 * U) {
      uint4 q[U];
      const unsigned int ok = load(v, q);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float mx = get(q[j], 0);
#pragma unroll
        for (int i = 1; i < E; ++i) mx = fmaxf(mx, get(q[j], i));
        if ((ok & (1u << j)) && mx >= x0) {
#pragma unroll 1
          for (int i = 0; i < E; ++i) f((v + 32 * j) * E - mis + i, one(p + (v + 32 * j) * E - mis + i));
        }
      }
    }
    if (v0 < v1 - 1) edge(v1 - 1, 1, f);
  }
  template <typename F>
  SPEC_DEV void each(F f) const {
    if (v0 < v1) edge(v0, 0, f);
    for (int v = v0 + (int)(threadIdx.x & 31); v < v1; v += 32 * U) {
      uint4 q[U];
      const unsigned int ok = load(v, q);
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (ok & (1u << j)) {
#pragma unroll
          for (int i = 0; i < E; ++i) f((v + 32 * j) * E - mis + i, get(q[j], i));
        }
    }
    if (v0 < v1 - 1) edge(v1 - 1, 1, f);
  }
  // The same for a long f, in pairs: f.two(index, value, next value), or
  // f(index, value) on the row's edges. One copy of it for a vector's pairs
  // (the code of a scan that runs once comes from a cold instruction cache),
  // two vectors ahead; done(vectors of the lane so far) after each vector.
  template <typename F, typename D>
  SPEC_DEV void each_rolled(int from, int to, F& f, D done) const {
    const int lane = threadIdx.x & 31;
    uint4 q[3];
    bool ok[3];
    auto get_vec = [&](int v, uint4& x) {
      const int i0 = v * E - mis;
      const bool in = v < to && i0 >= 0 && i0 + E <= V;
      if (in) x = *reinterpret_cast<const uint4*>(p + i0);
      return in;
    };
    ok[0] = get_vec(from + lane, q[0]);
    ok[1] = get_vec(from + 32 + lane, q[1]);
    int n = 0;
#pragma unroll 1
    for (int v = from + lane; v - lane < to; v += 32) {
      ok[2] = get_vec(v + 64, q[2]);
      if (ok[0]) {
#pragma unroll
        for (int i = 0; i < E; i += 2) f.two(v * E - mis + i, get(q[0], i), get(q[0], i + 1));
      } else if (v < to) {
#pragma unroll 1
        for (int i = max(0, mis - v * E); i < E && v * E - mis + i < V; ++i) f(v * E - mis + i, one(p + v * E - mis + i));
      }
      q[0] = q[1];
      q[1] = q[2];
      ok[0] = ok[1];
      ok[1] = ok[2];
      done(++n);
    }
  }
  // The part's first or last vector, where the row does not fill it, in one
  // lane (the first before and the last behind the others, in index order).
  template <typename F>
  SPEC_DEV void edge(int v, int lane, F& f) const {
    const int i0 = v * E - mis;
    if ((int)(threadIdx.x & 31) != lane || (i0 >= 0 && i0 + E <= V)) return;
#pragma unroll 1
    for (int i = max(0, -i0); i < E && i0 + i < V; ++i) f(i0 + i, one(p + i0 + i));
  }
};

// Warp sum of values below 2^63, three hardware reductions of 21 bits each.
SPEC_DEV ull warp_sum_u64(ull v) {
  constexpr unsigned int M = (1u << 21) - 1;
  const ull a = __reduce_add_sync(FULL, (unsigned int)v & M);
  const ull b = __reduce_add_sync(FULL, (unsigned int)(v >> 21) & M);
  const ull c = __reduce_add_sync(FULL, (unsigned int)(v >> 42));
  return a + (b << 21) + (c << 42);
}
SPEC_DEV ull warp_scan_u64(ull v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const ull u = __shfl_up_sync(FULL, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

SPEC_DEV bool kept(const Cut& c, uint32_t key, int i) { return key < c.key || (key == c.key && i <= c.idx); }

// f(index, value) as a scan's functor.
template <typename F>
struct Single {
  F f;
  SPEC_DEV void operator()(int i, float x) { f(i, x); }
  SPEC_DEV void two(int i, float x0, float x1) {
    f(i, x0);
    f(i + 1, x1);
  }
};
// Amounts of tokens, summed by sum_part: one amount, or two together.
template <typename F>
struct Amount {
  F f;
  SPEC_DEV ull operator()(int i, float x) const { return f(i, x); }
  SPEC_DEV ull two(int i, float x0, float x1) const { return f(i, x0) + f(i + 1, x1); }
};
template <typename F>
struct Summing {
  const F& f;
  ull a;
  SPEC_DEV void operator()(int i, float x) { a += f(i, x); }
  SPEC_DEV void two(int i, float x0, float x1) { a += f.two(i, x0, x1); }
};
// The mass of the tokens inside a cut whose weight is at least qw.
struct Mass {
  Scale sc;
  const ull* tab;
  ull qw;
  Cut cut;
  bool cutting;
  SPEC_DEV ull keep(int i, float x, ull w) const {
    return w < qw || (cutting && !kept(cut, rank_key(x), i)) ? 0ull : w;
  }
  SPEC_DEV ull operator()(int i, float x) const { return keep(i, x, weight(sc, tab, x)); }
  SPEC_DEV ull two(int i, float x0, float x1) const {
    ull w0, w1;
    weight2(sc, tab, x0, x1, w0, w1);
    return keep(i, x0, w0) + keep(i + 1, x1, w1);
  }
};

// Counts or exact masses (in digits) of the kept tokens, by bin.
template <bool MASS, typename K>
struct Binned {
  Scale sc;
  const ull* tab;
  unsigned int* hist;
  K keep;
  SPEC_DEV void put(float x, ull w) const {
    unsigned int* h = hist + sc.bin(x);
    if (!MASS) {
      atomicAdd(h, 1u);
      return;
    }
    constexpr unsigned int M = (1u << DIGIT) - 1;
    if (w) atomicAdd(h, (unsigned int)w & M);
    if (w >> DIGIT) atomicAdd(h + BINS, (unsigned int)(w >> DIGIT) & M);
    if (w >> (2 * DIGIT)) atomicAdd(h + 2 * BINS, (unsigned int)(w >> (2 * DIGIT)));
  }
  SPEC_DEV void operator()(int i, float x) const {
    if (keep(i, x)) put(x, MASS ? weight(sc, tab, x) : 0ull);
  }
  SPEC_DEV void two(int i, float x0, float x1) const {
    const bool k0 = keep(i, x0), k1 = keep(i + 1, x1);
    if (!k0 && !k1) return;
    ull w0 = 0, w1 = 0;
    if (MASS) weight2(sc, tab, x0, x1, w0, w1);
    if (k0) put(x0, w0);
    if (k1) put(x1, w1);
  }
};

template <typename T>
struct Sampler {
  Shared& s;
  cg::cluster_group cl;
  int cta, C;
  Part<T> part;
  Scale sc;
  static constexpr int PT = FEW / NT;   // sorted tokens of a thread

  // f(index, value) of this CTA's tokens.
  template <typename F>
  SPEC_DEV void scan(const F& f) {
    Single<F> one{f};
    part.each_rolled(part.v0, part.v1, one, [](int) {});
  }

  // Exclusive sum of v over the CTA's threads, in thread order.
  SPEC_DEV ull block_scan(ull v) {
    const ull inc = warp_scan_u64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 31) s.wsum[threadIdx.x >> 5] = inc;
    __syncthreads();
    ull b = inc - v;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      if (i < (int)(threadIdx.x >> 5)) b += s.wsum[i];
    return b;
  }

  // This CTA's sum of f(index, value) in s.total, the warps' parts in wsum,
  // their chunks' in chunk; ends with a barrier.
  template <typename F>
  SPEC_DEV void sum_part(const F& f) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, per = chunk_vectors();
    ull all = 0;
    int c = 0;
    __syncthreads();
    Summing<F> add{f, 0};
    part.each_rolled(part.v0, part.v1, add, [&](int n) {
      if ((n & (per - 1)) == 0) {
        const ull a = warp_sum_u64(add.a);
        if (lane == 0) s.chunk[w][c] = a;
        ++c;
        all += a;
        add.a = 0;
      }
    });
    const ull a = warp_sum_u64(add.a);
    if (lane == 0) {
      if (c < CHUNKS) s.chunk[w][c] = a;
      s.wsum[w] = all + a;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      const ull t = warp_sum_u64(threadIdx.x < NW ? s.wsum[threadIdx.x] : 0ull);
      if (threadIdx.x == 0) s.total = t;
    }
    __syncthreads();
  }
  // A power of two.
  SPEC_DEV int chunk_vectors() const {
    int per = CHUNK;
    while (per * CHUNKS * 32 < part.v1 - part.v0) per *= 2;
    return per;
  }

  // Sum of f(index, value) over the row, and that of the cluster's earlier CTAs.
  template <typename F>
  SPEC_DEV ull sum(const F& f, ull* before) {
    sum_part(f);
    cl.sync();
    ull all = 0, b = 0;
    for (int c = 0; c < C; ++c) {
      const ull t = *cl.map_shared_rank(&s.total, c);
      if (c < cta) b += t;
      all += t;
    }
    cl.sync();
    *before = b;
    return all;
  }

  // Calls hit(index, value) in the lane that holds the lowest index at which
  // the sum of f in index order exceeds t (t below the row's sum; the CTA's
  // sums as sum_part left them, before: the sum of the earlier CTAs).
  template <typename F, typename H>
  SPEC_DEV void find_in_order(const F& f, ull t, ull before, H hit) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, per = chunk_vectors();
    ull b = before;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      if (i < w) b += s.wsum[i];
    if (t < b || t >= b + s.wsum[w]) return;
    // the chunk, then the vector, then the element
    const ull mine = lane * per * 32 < part.v1 - part.v0 ? s.chunk[w][lane] : 0ull;
    const ull upto = b + warp_scan_u64(mine);
    const int c = __ffs(__ballot_sync(FULL, t < upto)) - 1;
    b = __shfl_sync(FULL, upto - mine, c);
    const int from = part.v0 + c * per * 32;
    int v = from + lane;
    bool over = false;
    Summing<F> add{f, 0};
    part.each_rolled(from, min(part.v1, from + per * 32), add, [&](int) {
      const ull inc = warp_scan_u64(add.a);
      const ull tot = __shfl_sync(FULL, inc, 31);
      if (!over && t < b + tot) {
        over = true;
        const ull at = b + inc - add.a;
        if (t >= at && t < at + add.a) walk(f, max(0, v * Part<T>::E - part.mis), t, at, hit);
      }
      b += tot;
      add.a = 0;
      v += 32;
    });
  }
  // From index i on, in one lane: the element at which the sum b passes t.
  template <typename F, typename H>
  SPEC_DEV void walk(const F& f, int i, ull t, ull b, H hit) {
#pragma unroll 1
    for (; i < part.V; ++i) {
      const float x = Part<T>::one(part.p + i);
      b += f(i, x);
      if (t < b) {
        hit(i, x);
        return;
      }
    }
  }
  // The same index in every CTA.
  template <typename F>
  SPEC_DEV int find_all(const F& f, ull t, ull before) {
    find_in_order(f, t, before, [&](int i, float) {
      for (int r = 0; r < C; ++r) *cl.map_shared_rank(&s.found, r) = i;
    });
    cl.sync();
    const int found = s.found;
    cl.sync();
    return found;
  }

  // This CTA's sum of v over its threads in s.total (wsum: the warps' parts);
  // ends with a barrier.
  SPEC_DEV void block_total(ull v) {
    v = warp_sum_u64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.wsum[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
      const ull t = warp_sum_u64(threadIdx.x < NW ? s.wsum[threadIdx.x] : 0ull);
      if (threadIdx.x == 0) s.total = t;
    }
    __syncthreads();
  }

  // The bin in which the count or exact mass of the kept tokens, in order,
  // first reaches need(row's amount) >= 1: s.bin, with the amount before it and
  // in it in s.before and s.at, the same in every CTA. Each CTA counts its
  // tokens by bin, adds up the cluster's counts of a share of the bins, and the
  // owner of the bin tells the others. Returns the row's amount; *last: need.
  // Empties the lists.
  template <bool MASS, typename K, typename N>
  SPEC_DEV ull find_bin(K keep, N need, ull* last) {
    constexpr int D = MASS ? 3 : 1;
    if (threadIdx.x == 0) {
      s.listed = 0;
      s.gathered = 0;
    }
    for (int i = threadIdx.x; i < D * BINS; i += NT) s.hist[0][i] = 0u;
    __syncthreads();
    Binned<MASS, K> add{sc, s.tab, &s.hist[0][0], keep};
    part.each_rolled(part.v0, part.v1, add, [](int) {});
    cl.sync();
    const int share = (BINS + C - 1) / C, per = (share + NT - 1) / NT, b0 = cta * share + threadIdx.x * per;
    const int b1 = min(min(b0 + per, (cta + 1) * share), BINS);
    ull h[BPT], t = 0;
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
      h[j] = 0;
      if (b0 + j < b1) {
#pragma unroll 4
        for (int c = 0; c < C; ++c) {
          const unsigned int* o = cl.map_shared_rank(&s.hist[0][0], c) + b0 + j;
#pragma unroll
          for (int d = 0; d < D; ++d) h[j] += (ull)o[d * BINS] << (d * DIGIT);
        }
      }
      t += h[j];
    }
    ull b = block_scan(t);
    if (threadIdx.x == NT - 1) s.total = b + t;
    __syncthreads();
    if (threadIdx.x < C) *cl.map_shared_rank(&s.x_total[cta], threadIdx.x) = s.total;
    cl.sync();
    ull all = 0;
#pragma unroll
    for (int c = 0; c < MAX_C; ++c) {
      if (c == cta) b += all;
      if (c < C) all += s.x_total[c];
    }
    *last = need(all);
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
      if (b < *last && *last <= b + h[j])
        for (int c = 0; c < C; ++c) {
          Shared& o = *cl.map_shared_rank(&s, c);
          o.bin = b0 + j;
          o.before = b;
          o.at = h[j];
        }
      b += h[j];
    }
    cl.sync();
    return all;
  }

  // The bin in which the amount in order first reaches need >= 1 (s.bin), the
  // amount before it and in it (s.before, s.at).
  SPEC_DEV void cross(const ull (&h)[BPT], ull need, ull before) {
    ull n = 0;
#pragma unroll
    for (int j = 0; j < BPT; ++j) n += h[j];
    ull b = before + block_scan(n);
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
      if (b < need && need <= b + h[j]) {
        s.bin = threadIdx.x * BPT + j;
        s.before = b;
        s.at = h[j];
      }
      b += h[j];
    }
    __syncthreads();
  }

  // The key in bin `bin` at which the amount in order first reaches `need`
  // (`before` the bin): three levels of 11, 11 and 10 key bits. Returns the
  // key; s.before: amount strictly before it, s.at: amount of its tokens.
  template <bool MASS, typename K>
  SPEC_DEV uint32_t radix(int bin, ull need, ull before, K keep) {
    uint32_t pre = 0;
#pragma unroll 1
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
      const int bits = level == 2 ? 10 : 11;
      for (int i = threadIdx.x; i < BINS; i += NT) s.mass[i] = 0ull;
      __syncthreads();
      auto one = [&](int i, float x) {
        if (sc.bin(x) != bin) return;
        const uint32_t k = rank_key(x);
        if ((level > 0 && (k >> (shift + bits)) != pre) || !keep(i, x)) return;
        atomicAdd(&s.mass[(k >> shift) & ((1 << bits) - 1)], MASS ? weight(sc, s.tab, x) : 1ull);
      };
      scan(one);
      cl.sync();
      ull h[BPT] = {0, 0, 0, 0};
#pragma unroll 4
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < BPT; ++j) h[j] += cl.map_shared_rank(s.mass, c)[threadIdx.x * BPT + j];
      cross(h, need, before);
      cl.sync();
      pre = (pre << bits) | (uint32_t)s.bin;
      before = s.before;
    }
    return pre;
  }

  // The cut at which the amount in order (of the tokens kept so far) reaches
  // `need`, in bin s.bin with s.before ahead of it.
  template <bool MASS, typename K>
  SPEC_DEV void cut_in_bin(Cut& cut, ull need, K keep) {
    const int bin = s.bin;
    const ull before = s.before;
    if (threadIdx.x == 0) {
      s.listed = 0;
      s.gathered = 0;
    }
    __syncthreads();
    const float lo = (float)bin, hi = bin < BINS - 1 ? (float)(bin + 1) : INFINITY;
    auto one = [&](int i, float x) {
      if (keep(i, x)) list(i, x, lo, hi);
    };
    scan(one);
    cl.sync();
    push_list();
    cl.sync();
    const int n = *cl.map_shared_rank(&s.gathered, 0);
    if (n <= FEW) {
      if (cta == 0) {
        int n2 = 64;
        while (n2 < n) n2 <<= 1;
        for (int i = n + threadIdx.x; i < n2; i += NT) s.sort[i] = ~0ull;
        __syncthreads();
        sort(n2);
        ull w[PT], t = 0;
#pragma unroll
        for (int j = 0; j < PT; ++j) {
          const int i = threadIdx.x * PT + j;
          w[j] = i >= n ? 0ull : MASS ? weight_once(sc, s.tab, rank_val((uint32_t)(s.sort[i] >> 32)), nullptr) : 1ull;
          t += w[j];
        }
        ull b = before + block_scan(t);
#pragma unroll
        for (int j = 0; j < PT; ++j) {
          if (b < need && need <= b + w[j]) {
            const ull e = s.sort[threadIdx.x * PT + j];
            for (int c = 0; c < C; ++c) *cl.map_shared_rank(&s.cut, c) = Cut{(uint32_t)(e >> 32), (int)(uint32_t)e};
          }
          b += w[j];
        }
        // (tokens at -inf are not listed: a count that ends among them cuts nothing)
        if (threadIdx.x == NT - 1 && b < need)
          for (int c = 0; c < C; ++c) *cl.map_shared_rank(&s.cut, c) = Cut{0xffffffffu, 0x7fffffff};
      }
      cl.sync();
      cut = s.cut;
      return;
    }
    cl.sync();
    const uint32_t key = radix<MASS>(bin, need, before, keep);
    const ull w = MASS ? weight_once(sc, s.tab, rank_val(key), nullptr) : 1ull;
    cut_ties(cut, key, (need - s.before + w - 1) / w, s.at / w);
  }

  // Narrows the cut to the `r` lowest indices among the `n` kept tokens of key.
  SPEC_DEV void cut_ties(Cut& cut, uint32_t key, ull r, ull n) {
    if (r < n) {
      const Cut old = cut;
      auto same = [=](int i, float x) { return rank_key(x) == key && kept(old, key, i) ? 1ull : 0ull; };
      const Amount<decltype(same)> eq{same};
      ull before;
      sum(eq, &before);
      cut.idx = find_all(eq, r - 1, before);
    } else if (key < cut.key) {
      cut.idx = 0x7fffffff;
    }
    cut.key = key;
  }

  // The bin (of SEG_BINS) down to which at least `need` tokens lie: that of the
  // need-th largest of the row's n segment maxima. Every CTA finds the same.
  SPEC_DEV int threshold(int need, int n) {
    for (int i = threadIdx.x; i < n; i += NT) atomicAdd(&s.seg_bins[sc.bin(s.seg[i]) / (BINS / SEG_BINS)], 1u);
    __syncthreads();
    const unsigned int c = s.seg_bins[threadIdx.x];
    const ull b = block_scan(c);
    if (b < (ull)need && (ull)need <= b + c) s.bin = threadIdx.x;
    __syncthreads();
    return s.bin;
  }

  // Lists the tokens of exponents [lo, hi) in bin units.
  SPEC_DEV void list(int i, float x, float lo, float hi) {
    const float v = sc.m == INFINITY ? (x == INFINITY ? 0.f : INFINITY) : sc.place(x);
    if (v < hi && v >= lo && *(volatile int*)&s.listed <= LIST) {   // (full: no more of them)
      const int at = atomicAdd(&s.listed, 1);
      if (at < LIST) {
        s.list_key[at] = rank_key(x);
        s.list_idx[at] = i;
      }
    }
  }

  // Whether the tokens of the bins before `bins` are few enough to be listed and
  // sorted by one CTA: fewer than a quarter of the n segment maxima lie there, that
  // is about 0.3 tokens a segment. (64 rows with top-p: 104 us; trying wherever
  // they might fit, up to 7 of 8 of the segments, 114 us.)
  SPEC_DEV bool listable(int bins, int n) {
    int in = 0;
    for (int i0 = 0; i0 < n; i0 += NT)
      in += __syncthreads_count(i0 + (int)threadIdx.x < n && sc.bin(s.seg[min(i0 + (int)threadIdx.x, n - 1)]) < bins);
    return in < n / 4;
  }

  // Lists the tokens of the first bins in order, below `hi`, and hands them to
  // the first CTA. Returns their number; more than FEW: they did not fit.
  SPEC_DEV int list_below(float hi) {
    // a little below any value listed
    const float x0 = sc.m == INFINITY ? sc.m : hi == INFINITY || sc.bins == 0.f
                         ? -INFINITY : sc.m - hi / (sc.sh * sc.bins) * 1.0001f - fabsf(sc.m) * 1e-5f;
    part.each_above(x0, [&](int i, float x) { list(i, x, 0.f, hi); });
    __syncthreads();
    push_list();
    cl.sync();
    return *cl.map_shared_rank(&s.gathered, 0);
  }

  // Appends the listed tokens to the first CTA's; what does not fit is counted
  // as more than FEW.
  SPEC_DEV void push_list() {
    const int n = s.listed;
    int* gathered = cl.map_shared_rank(&s.gathered, 0);
    if (threadIdx.x == 0) s.base = atomicAdd(gathered, n <= LIST ? n : FEW + 1);
    __syncthreads();
    const int base = s.base;
    if (n > LIST || base + n > FEW) return;
    ull* sort0 = cl.map_shared_rank(s.sort, 0);
    for (int i = threadIdx.x; i < n; i += NT) sort0[base + i] = ((ull)s.list_key[i] << 32) | (unsigned int)s.list_idx[i];
  }

  // Ascending bitonic sort of s.sort[0, n2), n2 a power of two, at least 64.
  // A warp's pairs of a stride up to 32 stay inside 64 elements of its own.
  SPEC_DEV void sort(int n2) {
    for (int k = 2; k <= n2; k <<= 1)
      for (int j = k >> 1; j > 0; j >>= 1) {
        for (int t = threadIdx.x; t < n2 / 2; t += NT) {
          const int i = 2 * t - (t & (j - 1)), l = i + j;
          const ull a = s.sort[i], b = s.sort[l];
          if ((a > b) == ((i & k) == 0)) {
            s.sort[i] = b;
            s.sort[l] = a;
          }
        }
        if (j > 32 || (j == 1 && k >= 64)) __syncthreads();
        else __syncwarp();
      }
  }

  // draw_few for at most COUNTED tokens, which are not sorted: two threads a
  // token count the tokens (and their mass) ahead of it, in the order and then
  // in the vocabulary.
  SPEC_DEV int draw_counted(int n, int k, float p, ull qw, float u, ull mass, ull* kept_mass) {
    ull* w = s.sort + COUNTED;
    const int i = threadIdx.x >> 1, half = threadIdx.x & 1;
    const ull e = i < n ? s.sort[i] : ~0ull;
    const ull wi = i < n ? weight_once(sc, s.tab, rank_val((uint32_t)(e >> 32)), nullptr) : 0ull;
    if (half == 0) w[i] = wi;
    __syncthreads();
    ull ahead = 0;
    int rank = 0;
    if (i < n) {
#pragma unroll 4
      for (int j = half; j < n; j += 2)
        if (s.sort[j] < e) {
          ahead += w[j];
          ++rank;
        }
    }
    ahead += __shfl_xor_sync(FULL, ahead, 1);
    rank += __shfl_xor_sync(FULL, rank, 1);
    bool keep = i < n && (k <= 0 || rank < k);
    if (p < 1.f) {
      block_total(keep && half == 0 ? wi : 0ull);
      const ull need = top_p_mass(p, k > 0 ? s.total : mass);
      keep = keep && ahead < need;
    }
    keep = keep && wi >= qw;
    const ull ki = keep ? wi : 0ull;
    block_total(half == 0 ? ki : 0ull);
    const ull z = s.total, d = drawn_mass(u, z);
    if (half == 0) w[i] = ki;
    __syncthreads();
    if (ki) {
      ahead = 0;
#pragma unroll 4
      for (int j = half; j < n; j += 2)
        if ((uint32_t)s.sort[j] < (uint32_t)e) ahead += w[j];
    }
    ahead += __shfl_xor_sync(FULL, ahead, 1);
    if (half == 0 && d >= ahead && d < ahead + ki) s.found = (int)(uint32_t)e;
    __syncthreads();
    *kept_mass = z;
    return s.found;
  }

  // The first CTA's end of the usual case: the n listed tokens sorted by
  // (key, index), cut, and drawn from in index order. mass: the row's whole
  // mass (top-p without top-k). Returns the token, *kept_mass its kept mass.
  SPEC_DEV int draw_few(int n, int k, float p, ull qw, float u, ull mass, ull* kept_mass) {
    if (n <= COUNTED) return draw_counted(n, k, p, qw, u, mass, kept_mass);
    int n2 = 64;
    while (n2 < n) n2 <<= 1;
    for (int i = n + threadIdx.x; i < n2; i += NT) s.sort[i] = ~0ull;
    if (threadIdx.x == 0) s.r = k > 0 ? min(n, k) : n;
    __syncthreads();
    sort(n2);
    // weights of the first r tokens, PT consecutive ones a thread
    const int r1 = s.r;
    ull e[PT], w[PT], t = 0;
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      const int i = threadIdx.x * PT + j;
      e[j] = i < r1 ? s.sort[i] : 0ull;
      w[j] = i < r1 ? weight_once(sc, s.tab, rank_val((uint32_t)(e[j] >> 32)), nullptr) : 0ull;
      t += w[j];
    }
    const ull b0 = block_scan(t);
    if (threadIdx.x == NT - 1) s.total = b0 + t;
    __syncthreads();
    int r = r1;
    if (p < 1.f) {
      const ull need = top_p_mass(p, k > 0 ? s.total : mass);
      ull b = b0;
#pragma unroll
      for (int j = 0; j < PT; ++j) {  // the token at which the mass reaches need is the last kept
        if (b < need && need <= b + w[j]) s.r = threadIdx.x * PT + j + 1;
        b += w[j];
      }
      __syncthreads();
      r = s.r;
    }
    ull z = 0;
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      const int i = threadIdx.x * PT + j;
      if (i >= r || w[j] < qw) w[j] = 0ull;
      z += w[j];
      // index and weight in one word; tokens not kept go behind
      if (i < n2) s.sort[i] = w[j] ? ((e[j] & 0xffffffffull) << (64 - IDX_BITS)) | w[j] : ~0ull;
    }
    const ull zb = block_scan(z);
    if (threadIdx.x == NT - 1) s.total = zb + z;
    __syncthreads();
    *kept_mass = s.total;
    const ull d = drawn_mass(u, s.total);
    while (n2 > 64 && n2 / 2 >= r) n2 >>= 1;
    sort(n2);
    t = 0;
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      const int i = threadIdx.x * PT + j;
      e[j] = i < n2 ? s.sort[i] : ~0ull;
      w[j] = e[j] == ~0ull ? 0ull : e[j] & ((1ull << (64 - IDX_BITS)) - 1);
      t += w[j];
    }
    ull b = block_scan(t);
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      if (d >= b && d < b + w[j]) s.found = (int)(e[j] >> (64 - IDX_BITS));
      b += w[j];
    }
    __syncthreads();
    return s.found;
  }
};

// What the chunk kernel leaves of a chunk.
struct __align__(16) Record {
  ull sum;         // weights relative to the chunk's maximum
  ull best;        // packed maximum, 0: nothing above -inf
  int nan;
};

// log2(e) / T as a float pair.
SPEC_DEV void scale_of(float temp, float& sh, float& sl) {
  constexpr float L = 1.44269502f;                                   // log2(e) rounded
  constexpr float L_LO = (float)(1.4426950408889634 - (double)L);
  sh = L / temp;
  sl = (fmaf(-sh, temp, L) + L_LO) / temp;
}

// A vector of a row, -inf where the row does not fill it.
template <typename T>
SPEC_DEV uint4 row_vector(const T* p, int V, int mis, int v) {
  constexpr int E = 16 / sizeof(T);
  const int i0 = v * E - mis;
  if (i0 >= 0 && i0 + E <= V) return *reinterpret_cast<const uint4*>(p + i0);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i0 + i >= 0 && i0 + i < V) {
      if (sizeof(T) == 4) {
        w[i & 3] = *reinterpret_cast<const uint32_t*>(p + i0 + i);
      } else {
        const int sft = 16 * (i & 1);
        w[(i >> 1) & 3] = (w[(i >> 1) & 3] & (0xffff0000u >> sft)) |
                          ((uint32_t)*reinterpret_cast<const uint16_t*>(p + i0 + i) << sft);
      }
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Chunks per row: enough for any alignment of its first token.
__host__ __device__ inline int row_chunks(int V) { return (V + 7 + CHUNK_TOKENS - 1) / CHUNK_TOKENS; }

template <typename T>
__global__ void __launch_bounds__(CNT, 4) chunk_kernel(SampleArgs a, Record* records) {
  constexpr int E = 16 / sizeof(T), PER = CHUNK_TOKENS / E, NV = PER / CNT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ull* tab = reinterpret_cast<ull*>(smem_raw);
  __shared__ ull s_best[2][CNW], s_sum[2][CNW];
  for (int i = threadIdx.x; i < TAB / 2; i += CNT) {
    const unsigned int dst = (unsigned int)__cvta_generic_to_shared(tab + 2 * i);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(g_table.v + 2 * i) : "memory");
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = row_chunks(a.V), items = a.M * n;
  grid_dep_wait();
  uint4 q[NV], next[NV];
  float temp = 0.f, temp_next = 0.f;
  auto load = [&](int item, uint4 (&v)[NV], float& t) {
    if (item >= items) return;
    const int row = item / n, c = item - row * n;
    const T* p = (const T*)a.logits + (size_t)row * a.ld;
    const int mis = (int)(((uintptr_t)p & 15) / sizeof(T));
    const int i0 = c * CHUNK_TOKENS - mis;
    if (i0 >= 0 && i0 + CHUNK_TOKENS <= a.V) {   // for the whole CTA: plain loads, nothing to merge
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = reinterpret_cast<const uint4*>(p + i0)[j * CNT + threadIdx.x];
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = row_vector(p, a.V, mis, c * PER + j * CNT + threadIdx.x);
    }
    t = a.temperature ? a.temperature[row] : 1.f;
  };
  load(blockIdx.x, q, temp);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  int turn = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x, turn ^= 1) {
    load(item + gridDim.x, next, temp_next);
    const int row = item / n, c = item - row * n;
    const int mis = (int)(((uintptr_t)((const T*)a.logits + (size_t)row * a.ld) & 15) / sizeof(T));
    float bx = -INFINITY;
    int bi = -1, nan = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float x = Part<T>::get(q[j], i);
        nan |= x != x;
        if (x > bx) {
          bx = x;
          bi = (c * PER + j * CNT + threadIdx.x) * E - mis + i;
        }
      }
    ull best = bi >= 0 ? pack_best(bx + 0.f, (uint32_t)bi) : 0ull;
    const uint32_t key = __reduce_max_sync(FULL, (uint32_t)(best >> 32));
    const uint32_t idx = __reduce_max_sync(FULL, (uint32_t)(best >> 32) == key ? (uint32_t)best : 0u);
    best = ((ull)key << 32) | idx;
    if (lane == 0) s_best[turn][warp] = best;
    nan = __syncthreads_or(nan);
#pragma unroll
    for (int w = 0; w < CNW; ++w) best = s_best[turn][w] > best ? s_best[turn][w] : best;
    ull sum = 0;
    if (best && !nan && temp >= 1e-5f && temp < INFINITY) {
      Scale sc{best_value(best), 0.f, 0.f, 0.f};
      scale_of(temp, sc.sh, sc.sl);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          ull w0, w1;
          weight2(sc, tab, Part<T>::get(q[j], i), Part<T>::get(q[j], i + 1), w0, w1);
          sum += w0 + w1;
        }
      sum = warp_sum_u64(sum);
    }
    if (lane == 0) s_sum[turn][warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      sum = 0;
#pragma unroll
      for (int w = 0; w < CNW; ++w) sum += s_sum[turn][w];
      Record& r = records[item];
      r.sum = sum;
      r.best = best;
      r.nan = nan;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) q[j] = next[j];
    temp = temp_next;
  }
}

// A row of a call without filters, from its chunks' records: their sums in the
// row's units, the chunk in which the drawn mass lies, and the token in it.
template <typename T>
__global__ void __launch_bounds__(NT) draw_kernel(SampleArgs a, const Record* records) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ull* tab = reinterpret_cast<ull*>(smem_raw);
  __shared__ ull wsum[NW], before, factor, total;
  __shared__ int chunk, shift;
  for (int i = threadIdx.x; i < TAB / 2; i += NT) {
    const unsigned int dst = (unsigned int)__cvta_generic_to_shared(tab + 2 * i);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(g_table.v + 2 * i) : "memory");
  }
  const int row = blockIdx.x, chunks = row_chunks(a.V), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  const Record* rec = records + (size_t)row * chunks;
  const float temp = a.temperature ? a.temperature[row] : 1.f, u = a.uniform[row];
  auto scan = [&](ull v) {   // exclusive, in thread order
    const ull inc = warp_scan_u64(v);
    __syncthreads();
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    ull b = inc - v;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      if (i < warp) b += wsum[i];
    return b;
  };
  ull best = 0, mine = 0;
  int nan = 0;
  if (threadIdx.x < chunks) {
    mine = __ldcg(&rec[threadIdx.x].best);
    nan = __ldcg(&rec[threadIdx.x].nan);
  }
  {
    const uint32_t key = __reduce_max_sync(FULL, (uint32_t)(mine >> 32));
    const uint32_t idx = __reduce_max_sync(FULL, (uint32_t)(mine >> 32) == key ? (uint32_t)mine : 0u);
    if (lane == 0) wsum[warp] = ((ull)key << 32) | idx;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  nan = __syncthreads_or(nan);
#pragma unroll
  for (int i = 0; i < NW; ++i) best = wsum[i] > best ? wsum[i] : best;
  const bool greedy = temp < 1e-5f;
  if (best == 0ull || nan || !(temp >= 0.f && temp < INFINITY) || greedy) {
    const bool ok = best != 0ull && !nan && greedy && temp >= 0.f;   // else: no distribution
    if (threadIdx.x == 0) {
      a.tokens[row] = ok ? (int)best_index(best) : -1;
      if (a.probs) a.probs[row] = ok ? 1.f : 0.f;
    }
    return;
  }
  Scale sc{best_value(best), 0.f, 0.f, 0.f};
  scale_of(temp, sc.sh, sc.sl);
  ull v = 0, mass = 0;
  int n = 0;
  if (mine) {
    v = weight_parts(sc, tab, best_value(mine), n);
    mass = in_row(__ldcg(&rec[threadIdx.x].sum), v, n);
  }
  const ull from = scan(mass);
  if (threadIdx.x == NT - 1) total = from + mass;
  __syncthreads();
  const ull z = total, d = drawn_mass(u, z);
  if (d >= from && d < from + mass) {
    chunk = threadIdx.x;
    before = from;
    factor = v;
    shift = n;
  }
  __syncthreads();
  // the chunk again, NV consecutive vectors a thread
  constexpr int E = Part<T>::E, PER = CHUNK_TOKENS / E, NV = PER / NT;
  const int c = chunk;
  const ull t = d - before;
  v = factor;
  n = shift;
  const T* p = (const T*)a.logits + (size_t)row * a.ld;
  const int mis = (int)(((uintptr_t)p & 15) / sizeof(T));
  Scale in = sc;
  in.m = best_value(__ldcg(&rec[c].best));
  ull sum = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint4 q = row_vector(p, a.V, mis, c * PER + threadIdx.x * NV + j);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      ull w0, w1;
      weight2(in, tab, Part<T>::get(q, i), Part<T>::get(q, i + 1), w0, w1);
      sum += w0 + w1;
    }
  }
  ull b = scan(sum);
  if (in_row(b, v, n) <= t && t < in_row(b + sum, v, n)) {
#pragma unroll 1
    for (int i = 0; i < NV * E; ++i) {
      const int at = (c * PER + threadIdx.x * NV) * E + i - mis;
      if (at < 0 || at >= a.V) continue;
      const float x = Part<T>::one(p + at);
      b += weight(in, tab, x);
      if (t < in_row(b, v, n)) {
        float w;
        weight(sc, tab, x, &w);
        a.tokens[row] = at;
        if (a.probs) a.probs[row] = w / ((float)z * (1.f / (float)(1ull << WBITS)));
        break;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(NT, 2) sample_kernel(SampleArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Shared& s = *reinterpret_cast<Shared*>(smem_raw);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), cta = (int)cl.block_rank(), row = blockIdx.x / C;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < TAB / 2; i += NT) {
    const unsigned int dst = (unsigned int)__cvta_generic_to_shared(s.tab + 2 * i);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(g_table.v + 2 * i) : "memory");
  }
  s.seg_bins[threadIdx.x] = 0u;
  if (threadIdx.x == 0) {
    s.listed = 0;
    s.gathered = 0;
  }
  auto started = cl.barrier_arrive();   // every CTA runs before its shared memory is written
  Sampler<T> S{s, cl, cta, C};
  grid_dep_wait();
  const float temp = a.temperature ? a.temperature[row] : 1.f;
  int k = a.top_k ? a.top_k[row] : 0;
  if (k >= a.V) k = 0;
  const float p = a.top_p ? a.top_p[row] : 1.f;
  const float q = a.min_p ? fminf(a.min_p[row], 1.f) : 0.f;
  const float u = a.uniform[row];
  S.part.bind((const T*)a.logits + (size_t)row * a.ld, a.V, cta, C);
  const bool greedy = temp < 1e-5f, cuts = k > 0 || p < 1.f;
  int seg_lanes = 1;
  while (C * NT / seg_lanes > SEG_MAX) seg_lanes *= 2;

  // maximum with its lowest index, minimum, segment maxima; a NaN anywhere
  // leaves the row without a distribution
  float bx = -INFINITY, low = INFINITY;
  int bi = -1, nan = 0;
  S.part.each([&](int i, float x) {
    nan |= x != x;
    low = fminf(low, x);
    if (x > bx) {
      bx = x;
      bi = i;
    }
  });
  ull best = bi >= 0 ? pack_best(bx + 0.f, (uint32_t)bi) : 0ull;
  cl.barrier_wait(std::move(started));
  if (cuts && !greedy) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const float v = __shfl_xor_sync(FULL, bx, o);
      if (o < seg_lanes) bx = fmaxf(bx, v);
    }
    const int per = 32 / seg_lanes;   // segments of a warp, pushed to every CTA
    for (int j0 = 0; j0 < per * C; j0 += 32) {
      const int j = j0 + lane, g = j & (per - 1);
      const float v = __shfl_sync(FULL, bx, g * seg_lanes);
      if (j < per * C) cl.map_shared_rank(s.seg, j / per)[(cta * NW + warp) * per + g] = v;
    }
  }
  {
    // the largest key of the warp, and its lowest index
    const uint32_t key = __reduce_max_sync(FULL, (uint32_t)(best >> 32));
    const uint32_t idx = __reduce_max_sync(FULL, (uint32_t)(best >> 32) == key ? (uint32_t)best : 0u);
    best = ((ull)key << 32) | idx;
    low = ord_val(__reduce_min_sync(FULL, ord_key(low)));
  }
  if (lane == 0) {
    s.wsum[warp] = best;
    reinterpret_cast<float*>(s.list_idx)[warp] = low;
  }
  nan = __syncthreads_or(nan);
  if (threadIdx.x < C) {
    for (int i = 0; i < NW; ++i) {
      best = s.wsum[i] > best ? s.wsum[i] : best;
      low = fminf(low, reinterpret_cast<float*>(s.list_idx)[i]);
    }
    *cl.map_shared_rank(&s.x_best[cta], threadIdx.x) = best;
    *cl.map_shared_rank(&s.x_low[cta], threadIdx.x) = low;
    *cl.map_shared_rank(&s.x_nan[cta], threadIdx.x) = nan;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  cl.sync();
  best = 0;
  nan = 0;
#pragma unroll
  for (int c = 0; c < MAX_C; ++c)
    if (c < C) {
      best = s.x_best[c] > best ? s.x_best[c] : best;
      low = fminf(low, s.x_low[c]);
      nan |= s.x_nan[c];
    }

  auto write = [&](int token, float prob) {
    a.tokens[row] = token;
    if (a.probs) a.probs[row] = prob;
  };
  if (best == 0ull || nan || !(temp >= 0.f && temp < INFINITY) || greedy) {
    const bool ok = best != 0ull && !nan && greedy && temp >= 0.f;   // else: no distribution
    if (cta == 0 && threadIdx.x == 0) write(ok ? (int)best_index(best) : -1, ok ? 1.f : 0.f);
    return;
  }

  const float m = best_value(best);
  float sh, sl;
  scale_of(temp, sh, sl);
  // finer bins where the row's range of exponents is less than the weights'
  const float range = fminf((m - low) * sh, Z_END);
  S.sc = Scale{m, sh, sl, range > 1e-30f ? (float)(BINS - 1) / range : 0.f};
  // min-p's smallest weight
  const ull qw = q > 0.f ? (q < 1.f ? scaled(q, 1ull << WBITS, true) : 1ull << WBITS) : 0ull;
  auto result = [&](int token, float x, ull z) {
    float v;
    weight_once(S.sc, s.tab, x, &v);
    write(token, v / ((float)z * (1.f / (float)(1ull << WBITS))));
  };

  if (!cuts) {
    const Mass mass{S.sc, s.tab, qw, Cut{}, false};
    S.sum_part(mass);
    if (threadIdx.x < C) *cl.map_shared_rank(&s.x_total[cta], threadIdx.x) = s.total;
    cl.sync();
    ull z = 0, before = 0;
#pragma unroll
    for (int c = 0; c < MAX_C; ++c) {
      if (c == cta) before = z;
      if (c < C) z += s.x_total[c];
    }
    S.find_in_order(mass, drawn_mass(u, z), before, [&](int i, float x) { result(i, x, z); });
    return;
  }

  // the tokens that may be kept, listed for the first CTA
  // the last bin holds tokens without weight where the range was cut: not listed
  auto end_of = [&](int bins) { return bins < BINS ? (float)bins : range < Z_END ? INFINITY : (float)(BINS - 1); };
  // the first CTA draws among the n tokens handed to it, if they fit
  auto draw = [&](int n, ull all) {
    if (n <= FEW && cta == 0) {
      ull z;
      const int token = S.draw_few(n, k, p, qw, u, all, &z);
      if (threadIdx.x == 0) result(token, Part<T>::one((const T*)a.logits + (size_t)row * a.ld + token), z);
    }
    cl.sync();   // its count is read, and its tokens are, before either changes
    return n <= FEW;
  };
  auto every = [](int, float) { return true; };
  auto k_of = [&](ull) { return (ull)k; };
  auto p_of = [&](ull z) { return top_p_mass(p, z); };
  Cut cut{0xffffffffu, 0x7fffffff};
  ull need, before;
  const int segs = C * NT / seg_lanes;
  if (k > 0) {
    if (k <= segs && draw(S.list_below(end_of((S.threshold(k, segs) + 1) * (BINS / SEG_BINS))), 0ull)) return;
    S.template find_bin<false>(every, k_of, &need);
    S.template cut_in_bin<false>(cut, need, every);
  }
  if (p < 1.f) {
    if (k == 0) {
      const ull all = S.template find_bin<true>(every, p_of, &need);
      if (S.listable(s.bin + 1, segs) && draw(S.list_below(end_of(s.bin + 1)), all)) return;
      S.template cut_in_bin<true>(cut, need, every);
    } else {
      auto in = [&](int i, float x) { return kept(cut, rank_key(x), i); };
      S.template find_bin<true>(in, p_of, &need);
      S.template cut_in_bin<true>(cut, need, in);
    }
  }
  const Mass mass{S.sc, s.tab, qw, cut, true};
  const ull z = S.sum(mass, &before);
  S.find_in_order(mass, drawn_mass(u, z), before, [&](int i, float x) { result(i, x, z); });
}

// Sequences walk their sampled rows: drafts are kept while they equal the
// samples, then the target's own sample is emitted. A row without a
// distribution (-1) ends the emission before it; in a pass (state given) it is
// recorded and nothing of the pass is committed.
__global__ void __launch_bounds__(256) accept_sampled_kernel(AcceptSampledArgs a) {
  grid_dep_wait();
  const int R = a.k + 1;
  const int b0 = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
  if (a.seq_len)
    for (int b = b0; b < a.B; b += step) {
      const int32_t* t = a.out_tokens + (size_t)b * R;
      int A = 0;
      while (A < a.k && t[A] >= 0 && t[A] == a.drafts[(size_t)b * a.k + A]) ++A;
      if (t[A] < 0) set_error(a.err, SPEC_ERR_TOKEN);
    }
  __syncthreads();
  const int err = a.err ? *(volatile int*)a.err : 0;
  for (int b = b0; b < a.B; b += step) {
    int32_t* t = a.out_tokens + (size_t)b * R;
    int A = 0;
    while (A < a.k && t[A] >= 0 && t[A] == a.drafts[(size_t)b * a.k + A]) ++A;
    const int n = t[A] >= 0 ? A + 1 : A, last = t[A];
    for (int i = n; i < R; ++i) {
      t[i] = -1;
      if (a.probs) a.probs[(size_t)b * R + i] = 0.f;
    }
    a.n_emitted[b] = n;
    if (a.seq_len) {
      const int slot = a.seq_ids[b];
      if (!err) {
        a.seq_len[slot] += n;
        a.pending[slot] = last;
        a.stats[slot * 4 + 0] += 1;
        a.stats[slot * 4 + 1] += a.k;
        a.stats[slot * 4 + 2] += A;
        a.stats[slot * 4 + 3] += n;
      }
      a.sel_row[b] = b * R + A;
    }
  }
  if (a.best)
    for (int i = b0; i < a.B * R; i += step) a.best[i] = 0ull;
}

// Clusters of C CTAs of the kernel that device `dev`, the current one, holds at
// once (asked once).
template <typename T>
int max_clusters(int dev, int C) {
  static std::atomic<int> cache[MAX_DEVICES][MAX_C + 1];
  int n = cache[dev][C].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, sample_kernel<T>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = -1;  // not on this device
    }
    cache[dev][C].store(n, std::memory_order_relaxed);
  }
  return n;
}

// CTAs a row: the count with the least estimated time, waves of resident
// clusters at a fixed cost of about 8 us (0.1 more a CTA of the exchanges) and
// 0.17 ns a token of a CTA, twice that where two CTAs share an SM. 262144
// tokens, measured: 1 row with top-k and top-p 13 us with 16 CTAs, 15 with 8, 58
// with 1; 40 rows at temperature only 42 us with 6 (one wave), 51 with 8, 58 with
// 16. Rows with filters differ in length (a broad nucleus takes up to four
// scans), so they are spread over 8 CTAs at least where a CTA keeps 4096 tokens:
// 64 rows with top-p 128 us with 8, 143 with 6, 164 with 4.
template <typename T>
int cluster_size(int M, int V, bool filters) {
  int best = MAX_C, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) dev = 0;
  const int sms = num_sms();
  double least = 1e30;
  for (int C : {1, 2, 3, 4, 5, 6, 7, 8, 12, 16}) {
    if (V / C > DIGIT_TOKENS || (filters && C < std::min(8, V / 4096))) continue;
    const int fit = max_clusters<T>(dev, C);
    if (fit < 1) continue;
    double us = 0;
    for (int left = M; left > 0; left -= fit) {
      const int rows = std::min(left, fit);
      const int share = (rows * C + sms - 1) / sms;
      const double wave = 8.0 + 0.1 * C + 0.17e-3 * share * V / C;
      if (left > 8 * fit) {  // many waves: all but the last few at once
        const int n = left / fit - 4;
        us += n * wave;
        left -= n * fit;
      }
      us += wave;
    }
    if (us < least) {
      least = us;
      best = C;
    }
  }
  return best;
}

// Calls without filters of at least this many tokens take the chunk kernel: of
// 262144 tokens a row, 1 row 8.9 us (16.9 without), 40 rows 28.5 us (43).
constexpr long long CHUNKED_MIN = 1ll << 17;
bool chunked(int M, int V) { return (long long)M * V >= CHUNKED_MIN && V >= 2 * CHUNK_TOKENS; }

template <typename T>
int launch_chunked(const SampleArgs& a, int pdl, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(4 * num_sms(), (long long)a.M * row_chunks(a.V)));
  cfg.blockDim = dim3(CNT);
  cfg.dynamicSmemBytes = TAB * sizeof(ull);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, chunk_kernel<T>, a, (Record*)a.workspace) != cudaSuccess) return -1;
  cfg.gridDim = dim3(a.M);
  cfg.blockDim = dim3(NT);
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, draw_kernel<T>, a, (const Record*)a.workspace) == cudaSuccess ? 2 : -1;
}

template <typename T>
int launch_sample(const SampleArgs& a, int pdl, cudaStream_t st) {
  if (chunked(a.M, a.V) && !a.top_k && !a.top_p && !a.min_p) return launch_chunked<T>(a, pdl, st);
  const int C = cluster_size<T>(a.M, a.V, a.top_k || a.top_p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.M * C);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a) == cudaSuccess ? 1 : -1;
}

template <typename T>
void set_attributes() {
  cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
  cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  cudaFuncSetAttribute(chunk_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(TAB * sizeof(ull)));
  cudaFuncSetAttribute(draw_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(TAB * sizeof(ull)));
}

}  // namespace

void setup_sample_attributes() {
  set_attributes<float>();
  set_attributes<__nv_bfloat16>();
}

size_t sample_workspace_bytes(int M, int V) {
  return chunked(M, V) ? (size_t)M * row_chunks(V) * sizeof(Record) : 0;
}

int sample_rows(const SampleArgs& a, int pdl, cudaStream_t st) {
  return a.dtype == DT_F32 ? launch_sample<float>(a, pdl, st) : launch_sample<__nv_bfloat16>(a, pdl, st);
}

int accept_sampled(const AcceptSampledArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  // a pass commits in one CTA (its error check comes before every commit)
  cfg.gridDim = dim3(a.seq_len ? 1 : (unsigned)((a.B + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, accept_sampled_kernel, a) == cudaSuccess ? 1 : -1;
}

}  // namespace spec
