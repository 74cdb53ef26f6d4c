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
// choice; those below 2^13 units are cut off, and below one unit count as zero). In
// rows without filters they are in units of 2^-44 of the largest of their chunk, the
// 4096 tokens from a multiple of 4096 on, and the mass up to a token is rounded down
// to the row's units in its chunk: a chunk's sum needs no other chunk's maximum. The
// sums are exact, so the cut and the token do not depend on the order of the
// additions, the number of CTAs, the other rows or the row's address. The weight
// itself is evaluated to about 2^-37 (the exponent as a float pair, a table of 4096 powers), because a token is
// decided by a sum of up to V weights next to a border: at the 2^-24 of plain
// floats about one token in 10^4 would differ from the 64-bit definition; here
// none of 27600 rows of 4096 to 262144 tokens did.
//
// Large calls without filters: a first kernel takes the rows' chunks, in one pass
// that leaves each chunk's maximum and the sum of its weights,
// relative to that maximum; it loads the SMs evenly, with the next chunk's loads
// in flight under the exponentials of the last. A CTA a row then adds the sums
// up in the row's units, finds the drawn chunk and draws inside it.
//
// Otherwise a thread-block cluster takes a row; its CTAs push what the others
// need into their shared memory, so that a phase costs one cluster barrier. Scan
// 1 finds the maximum and the maxima of the row's segments (up to 1024). Without
// filters, the CTAs share the row's chunks and the first one draws, as above. With
// min-p alone, scan 2 sums the weights and the warp that holds the drawn mass
// finds the token. With top-k, scan 2 lists the tokens down to the k-th largest
// segment maximum -- at least k tokens, and rarely many more -- and the first CTA
// cuts and draws among those alone. With top-p alone, where the segment maxima
// promise a narrow nucleus, scan 2 lists the likeliest tokens and adds the others up
// in plain floats: bounds of the tail's mass that nearly always leave one cut. Else,
// or where they leave two, a scan counts the tokens in 2048 bins, linear in the
// exponent, which bound the mass up to each well enough to leave a few bins for the
// cut; the next adds all weights up exactly, lists those bins' tokens, and sums the
// tokens ahead of them in index order, so that the cut and the draw follow from the
// list and those sums. (A nucleus of few tokens is listed as a whole and drawn from
// as top-k's.) Where the listed tokens are too many, the cut comes from a radix
// search of their keys, or min-p's end lies ahead of it, and a last scan sums the
// kept weights.
//
// What bounds it: one row, latency (12 us with top-k, about 20 dependent phases of
// 0.3 to 2 us); many rows, the weights: about 42 instructions a token, among them
// random 8-byte reads of the table in shared memory, not the 1 MB a row out of
// HBM. 262144 fp32 logits a row: 40 rows at temperature 24.9 us (1.7 TB/s; the
// bytes alone 6.2 us), with top-k 50 26 us; 64 rows with top-p of mixed breadth 72
// to 97 us, 40 with few likely tokens 33 us.
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
constexpr int TAB_LOG = 12;
constexpr int TAB = 1 << TAB_LOG;   // 2^(-j/4096)
constexpr int MAX_C = 16;           // CTAs on one row (a thread-block cluster)
constexpr int FEW = 2048;           // tokens a CTA lists, and the first one cuts
constexpr int COUNTED = NT / 2;     // at most so many are counted instead
constexpr int HEAD = 128;           // segment maxima among which top-p looks first
constexpr int CHUNK_TOKENS = 4096;  // tokens of a chunk of a row without filters
constexpr int MAX_CHUNKS = (1 << 19) / CHUNK_TOKENS;
static_assert(MAX_CHUNKS <= NT, "a thread a chunk draws");
constexpr int CNT = 256;            // its threads
constexpr int CNW = CNT / 32;
constexpr int SEG_MAX = 1024;       // segments of a row (the elements of 1, 2, 4 or 8 lanes)
constexpr int SEG_BINS = NT;        // bins of the segment maxima
constexpr int FINE = NT;            // finer bins of listed tokens, one a thread
constexpr int TIED = 64;            // of one such bin, so many are counted
constexpr float Z_END = 46.f;       // weights are zero beyond this exponent
constexpr int CHUNK = 8;            // vectors of a lane whose sum is kept apart, doubled until
constexpr int CHUNKS = 32;          // a warp's part has at most 32 chunks

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

// What a CTA shares while it draws from a row's chunks.
struct Drawn {
  ull wsum[NW];
  ull before, factor, total;   // mass ahead of the drawn chunk, its units, the row's mass
  uint32_t top;                // key of the chunk's maximum
  int chunk, shift;
};

struct Shared {
  ull tab[TAB];
  union {
    unsigned int hist[BINS];     // counts
    ull mass[BINS];              // radix search inside some bins
    ull sort[FEW];               // first CTA: the tokens all listed
    struct {                     // first CTA of a row without filters
      ull sum[MAX_CHUNKS];       // pushed: its chunks' sums
      uint32_t top[MAX_CHUNKS];  // and keys of their maxima
      Drawn drawn;
    } chunks;
  };
  uint32_t list_key[FEW];
  int list_idx[FEW];
  int listed;                // tokens this CTA listed (more than FEW: they did not fit)
  // pushed by every CTA of the cluster
  uint32_t x_best[MAX_C];    // key of the maximum, 0: nothing above -inf
  float x_low[MAX_C];        // minimum
  ull x_total[MAX_C];        // sum of the weights
  union {
    float seg[SEG_MAX];      // segment maxima
    ull fine[FINE];          // first CTA: amounts of the listed tokens, by finer bins
  };
  ull tied[TIED][2];         // tokens of one of those, and their amounts
  ull word;                  // the selected one
  uint32_t key_lo, key_hi;
  int undecided;             // pushed by the first CTA
  float seen[2];             // weights of the listed segment maxima, and of all
  int n_tied;
  int gathered;              // first CTA: tokens listed by all
  unsigned int seg_bins[SEG_BINS];
  Cut cut;                   // pushed by the first CTA: the cut of the row
  ull chunk[NW][CHUNKS];     // sums of the warps' chunks
  ull wsum[NW];
  ull total;                 // this CTA's sum, read by the cluster
  int bin;                   // crossing bin
  ull before, at;            // amount before it, and in it
  ull x_bins[MAX_C][3];      // pushed: counts, least and largest mass of a share of the bins
  ull scan[NW][3];
  ull all;                   // this CTA's mass from bin lo on
  int lo, hi, n_lo, n_hi;    // pushed: bins in which a cut may lie, tokens before and through them
  int found;                 // index found by find_in_order, written by its owner
  int base;
};

// Scale of a row: weights are 2^-z with z = (m - x) * (sh + sl); bins are
// linear in z.
struct Scale {
  float m, sh, sl, bins;
  // Monotone in x (each rounding is), so bins are ranges of the order.
  SPEC_DEV float place(float x) const {
    return m == INFINITY ? (x == INFINITY ? 0.f : INFINITY) : (m - x) * sh * bins;
  }
  SPEC_DEV int bin(float x) const { return (int)fminf(place(x), (float)(BINS - 1)); }
};

// 2^(n-1), half a unit before the shift by n: a weight is rounded, not cut off.
// (The bias of V cut-off weights would move a border among the unlikely tokens
// by as much as their weights.) From n = 31 on, weights below 2^13 units, a fixed
// amount within 32 bits: next to nothing.
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
// v0, v1: their place().
SPEC_DEV void weight2(const Scale& r, const ull* tab, float x0, float x1, ull& w0, ull& w1, float& v0, float& v1) {
  if (r.m == INFINITY) {
    v0 = r.place(x0);
    v1 = r.place(x1);
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
  v0 = a * -r.bins;
  v1 = b * -r.bins;
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

SPEC_DEV void weight2(const Scale& r, const ull* tab, float x0, float x1, ull& w0, ull& w1) {
  float v0, v1;
  weight2(r, tab, x0, x1, w0, w1, v0, v1);
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

// The larger value, NaN if either is.
SPEC_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The part of a row one warp owns, 16-byte vectors in index order; rows may
// start at any element, the first and last vectors are read element by element.
template <typename T>
struct Part {
  const T* p;
  int V, mis, per, nvec, v0, v1;   // vectors [v0, v1); vector v holds elements v * E - mis ...
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
    nvec = (V + mis + E - 1) / E;
    per = (nvec + C * NW - 1) / (C * NW);
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
  // f(index, value) on the row's edges. W vectors of a lane a step, the next ones
  // in flight; one copy of f for them (the code of a scan that runs once comes
  // from a cold instruction cache). done(vectors of the lane so far) after each step.
  template <int W, typename F, typename D>
  SPEC_DEV void each_rolled(int from, int to, F& f, D done) const {
    constexpr int B = W == 1 ? 3 : 2 * W;   // buffers
    const int lane = threadIdx.x & 31;
    uint4 q[B];
    bool ok[B];
    auto get_vec = [&](int v, int j) {
      const int i0 = v * E - mis;
      ok[j] = v < to && i0 >= 0 && i0 + E <= V;
      if (ok[j]) q[j] = *reinterpret_cast<const uint4*>(p + i0);
    };
#pragma unroll
    for (int j = 0; j < B - W; ++j) get_vec(from + lane + 32 * j, j);
    int n = 0;
#pragma unroll 1
    for (int v = from + lane; v - lane < to; v += 32 * W) {
#pragma unroll
      for (int j = B - W; j < B; ++j) get_vec(v + 32 * j, j);
      bool all = true;
#pragma unroll
      for (int j = 0; j < W; ++j) all = all && ok[j];
      if (all) {
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
          for (int i = 0; i < E; i += 2) f.two((v + 32 * j) * E - mis + i, get(q[j], i), get(q[j], i + 1));
      } else {
#pragma unroll 1
        for (int j = 0; j < W; ++j) {
          const int i0 = (v + 32 * j) * E - mis;
#pragma unroll 1
          for (int i = max(0, -i0); i < E && i0 + i < V && v + 32 * j < to; ++i) f(i0 + i, one(p + i0 + i));
        }
      }
#pragma unroll
      for (int j = 0; j < B - W; ++j) {
        q[j] = q[j + W];
        ok[j] = ok[j + W];
      }
      done(n += W);
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

// What the chunk kernel leaves of a chunk.
struct __align__(16) Record {
  ull sum;         // weights relative to the chunk's maximum
  ull best;        // packed maximum, 0: nothing above -inf (its index in greedy rows only)
  int nan;
};

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

// The first n elements of b, then a's from n on.
template <typename T>
SPEC_DEV uint4 merge(const uint4& a, const uint4& b, int n) {
  auto word = [&](uint32_t x, uint32_t y, int j) {
    const int by = n * (int)sizeof(T) - 4 * j;   // bytes of b in this word
    return by <= 0 ? x : by >= 4 ? y : (y & 0xffffu) | (x & 0xffff0000u);
  };
  return make_uint4(word(a.x, b.x, 0), word(a.y, b.y, 1), word(a.z, b.z, 2), word(a.w, b.w, 3));
}

// Tokens v * E to (v + 1) * E - 1 of a row whose first one lies `mis` elements behind
// a 16-byte boundary, -inf past its end.
template <typename T>
SPEC_DEV uint4 token_vector(const T* p, int V, int mis, int v) {
  const uint4 a = row_vector(p, V, mis, v);
  if (mis == 0) return a;
  const uint4 b = row_vector(p, V, mis, v + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int by = mis * (int)sizeof(T), words = by >> 2;
  uint32_t x[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) x[i] = words == 0 ? w[i] : words == 1 ? w[i + 1] : words == 2 ? w[i + 2] : w[i + 3];
  const int bits = (by & 2) * 8;
  return make_uint4(__funnelshift_r(x[0], x[1], bits), __funnelshift_r(x[1], x[2], bits),
                    __funnelshift_r(x[2], x[3], bits), __funnelshift_r(x[3], x[4], bits));
}

// Chunks of a row: of the tokens, wherever the row starts.
__host__ __device__ inline int row_chunks(int V) { return (V + CHUNK_TOKENS - 1) / CHUNK_TOKENS; }


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
  F& f;
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

// One more of the tokens a CTA lists (when full, only their number is known).
SPEC_DEV void append(Shared& s, int i, float x) {
  if (*(volatile int*)&s.listed > FEW) return;
  const int at = atomicAdd(&s.listed, 1);
  if (at < FEW) {
    s.list_key[at] = rank_key(x);
    s.list_idx[at] = i;
  }
}

// Top-p's scan of the tokens inside a cut: returns the mass of those below lo, in
// bin units, adds the others' up, and lists those of them below hi.
struct Nucleus {
  Scale sc;
  Shared& s;
  Cut cut;
  bool cutting;
  float lo, hi;
  ull all;   // the others'
  SPEC_DEV ull take(int i, float x, float v, ull w) {
    if (cutting && !kept(cut, rank_key(x), i)) return 0ull;
    if (v < lo) return w;
    all += w;
    if (v < hi) append(s, i, x);
    return 0ull;
  }
  SPEC_DEV ull operator()(int i, float x) { return take(i, x, sc.place(x), weight(sc, s.tab, x)); }
  SPEC_DEV ull two(int i, float x0, float x1) {
    ull w0, w1;
    float v0, v1;
    weight2(sc, s.tab, x0, x1, w0, w1, v0, v1);
    return take(i, x0, v0, w0) + take(i + 1, x1, v1, w1);
  }
};

// The scan for a nucleus among the first few tokens: lists those below `end`, in
// bin units, and adds the weights of the others up in plain floats, a step's at a time.
struct Tail {
  Scale sc;
  Shared& s;
  float end, some;
  ull all;
  SPEC_DEV void operator()(int i, float x) {
    if (sc.place(x) < end) append(s, i, x);
    else some += exp2f((x - sc.m) * sc.sh);
  }
  SPEC_DEV void two(int i, float x0, float x1) {
    (*this)(i, x0);
    (*this)(i + 1, x1);
  }
  SPEC_DEV void step() {
    all += (ull)(some * (float)(1ull << WBITS));
    some = 0.f;
  }
};

// Counts of the tokens inside a cut, by bin.
struct Binned {
  Scale sc;
  unsigned int* hist;
  Cut cut;
  bool cutting;
  SPEC_DEV void operator()(int i, float x) const {
    if (!cutting || kept(cut, rank_key(x), i)) atomicAdd(hist + sc.bin(x), 1u);
  }
  SPEC_DEV void two(int i, float x0, float x1) const {
    (*this)(i, x0);
    (*this)(i + 1, x1);
  }
};

template <typename T>
struct Sampler {
  Shared& s;
  cg::cluster_group cl;
  int cta, C;
  Part<T> part;
  Scale sc;
  static constexpr int WIDE = 8 / Part<T>::E;   // vectors a step
  float range;      // of the row's exponents, up to Z_END
  static constexpr int PT = FEW / NT;   // sorted tokens of a thread

  // f(index, value) of this CTA's tokens.
  template <typename F>
  SPEC_DEV void scan(const F& f) {
    Single<F> one{f};
    part.template each_rolled<1>(part.v0, part.v1, one, [](int) {});
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
  SPEC_DEV void sum_part(F& f) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, per = chunk_vectors(part.v1 - part.v0);
    ull all = 0;
    int c = 0;
    __syncthreads();
    Summing<F> add{f, 0};
    part.template each_rolled<WIDE>(part.v0, part.v1, add, [&](int n) {
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
  // A lane's vectors in a chunk of a warp's n: a power of two.
  SPEC_DEV static int chunk_vectors(int n) {
    int per = CHUNK;
    while (per * CHUNKS * 32 < n) per *= 2;
    return per;
  }

  // The cluster's sum of the CTAs' v, and that of the earlier CTAs.
  SPEC_DEV ull cluster_sum(ull v, ull* before) {
    if (threadIdx.x < C) *cl.map_shared_rank(&s.x_total[cta], threadIdx.x) = v;
    cl.sync();
    ull all = 0;
#pragma unroll
    for (int c = 0; c < MAX_C; ++c) {
      if (c == cta) *before = all;
      if (c < C) all += s.x_total[c];
    }
    return all;
  }
  // Sum of f(index, value) over the row, and that of the cluster's earlier CTAs.
  template <typename F>
  SPEC_DEV ull sum(F& f, ull* before) {
    sum_part(f);
    return cluster_sum(s.total, before);
  }

  // Calls hit(index, value) in the lane that holds the lowest index at which
  // the sum of f in index order exceeds t (t below the row's sum; the CTA's
  // sums as sum_part left them, before: the sum of the earlier CTAs).
  template <typename F, typename H>
  SPEC_DEV void find_in_order(F& f, ull t, ull before, H hit) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, per = chunk_vectors(part.v1 - part.v0);
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
    part.template each_rolled<1>(from, min(part.v1, from + per * 32), add, [&](int) {
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
  SPEC_DEV void walk(F& f, int i, ull t, ull b, H hit) {
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
  SPEC_DEV int find_all(F& f, ull t, ull before) {
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

  // Where in the order of bins the tokens inside `cut` reach k tokens, or the
  // mass p of them (k = 0), the same in every CTA: in one of the bins s.lo to
  // s.hi, with s.n_lo tokens before those and s.n_hi through them. A bin's tokens
  // weigh the same to 1.6%, so their count bounds their mass; the cut may lie in a
  // bin unless the bounds of the mass up to it and of the mass behind it say
  // otherwise -- few bins, as the same error in both nearly cancels. Each CTA
  // counts its tokens by bin, adds up the cluster's counts of a share of the
  // bins, and the owners of the two bins tell the others. Empties the lists.
  // (Exact masses by bin, in three 15-bit digits, took three atomics and a weight
  // a token, and a further scan for the list: 64 rows of 262144 with a broad nucleus
  // took 154 us, 95 now.)
  SPEC_DEV void find_bins(const Cut& cut, bool cutting, int k, float p) {
    if (threadIdx.x == 0) {
      s.all = 0;
      s.listed = 0;
      s.gathered = 0;
    }
    for (int i = threadIdx.x; i < BINS; i += NT) s.hist[i] = 0u;
    __syncthreads();
    Binned add{sc, s.hist, cut, cutting};
    part.template each_rolled<WIDE>(part.v0, part.v1, add, [](int) {});
    cl.sync();
    // (rolled loops: what runs once comes from a cold instruction cache)
    const int share = (BINS + C - 1) / C, per = (share + NT - 1) / NT, b0 = cta * share + threadIdx.x * per;
    const int b1 = min(min(b0 + per, (cta + 1) * share), BINS);
    ull t[3] = {0, 0, 0};   // tokens, their least and largest mass
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      unsigned int n = 0;
#pragma unroll 4
      for (int c = 0; c < C; ++c) n += cl.map_shared_rank(s.hist, c)[b];
      s.list_key[b - cta * share] = n;
      add_bin(t, b, n);
    }
    ull at[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      at[i] = warp_scan_u64(t[i]);
      if ((threadIdx.x & 31) == 31) s.scan[threadIdx.x >> 5][i] = at[i];
      at[i] -= t[i];
    }
    __syncthreads();
    if (threadIdx.x < 3 * C) {   // a sum to each CTA
      const int i = threadIdx.x % 3;
      ull all = 0;
#pragma unroll 4
      for (int w = 0; w < NW; ++w) all += s.scan[w][i];
      cl.map_shared_rank(&s, threadIdx.x / 3)->x_bins[cta][i] = all;
    }
    for (int w = 0; w < (int)(threadIdx.x >> 5); ++w)
#pragma unroll
      for (int i = 0; i < 3; ++i) at[i] += s.scan[w][i];
    cl.sync();
    ull all[3] = {0, 0, 0};
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (c == cta) at[i] += all[i];
        all[i] += s.x_bins[c][i];
      }
    // Up to a bin: may the cut lie there or before (x), must it (y)?
    bool x0 = true, y0 = true;
#pragma unroll 1
    for (int b = b0 - 1; b < b1; ++b) {
      const int n0 = (int)at[0];
      if (b >= b0) add_bin(at, b, s.list_key[b - cta * share]);
      const bool x = k > 0 ? at[0] >= (ull)k : at[2] >= top_p_mass(p, at[2] + (all[1] - at[1]));
      const bool y = k > 0 ? x : at[1] >= top_p_mass(p, at[1] + (all[2] - at[2]));
      for (int c = 0; c < C; ++c) {
        Shared& o = *cl.map_shared_rank(&s, c);
        if (x && !x0) {
          o.lo = b;
          o.n_lo = n0;
        }
        if (y && !y0) {
          o.hi = b;
          o.n_hi = (int)at[0];
        }
      }
      x0 = x;
      y0 = y;
    }
    cl.sync();
  }
  // n tokens of bin b to a count and its bounds of mass.
  SPEC_DEV void add_bin(ull (&t)[3], int b, unsigned int n) const {
    ull least, most;
    bounds(b, least, most);
    t[0] += n;
    t[1] += n * least;
    t[2] += n * most;
  }

  // Bounds of the weight of a token in a bin.
  SPEC_DEV void bounds(int bin, ull& least, ull& most) const {
    if (sc.m == INFINITY) {
      least = most = bin == 0 ? 1ull << WBITS : 0ull;
      return;
    }
    // (place() is off by 4 roundings, 2e-5 in the exponent at most; the factors are 1 -+ 1e-4)
    const float step = sc.bins > 0.f ? 1.f / sc.bins : 0.f;
    most = (ull)(exp2f(WBITS - bin * step) * 1.0001f) + 1;
    least = (ull)(exp2f(WBITS - (bin + 1) * step) * 0.9999f);
    if (bin == BINS - 1) {   // ends with the least weight of all, or beyond all weights
      least = 0;
      if (range >= Z_END) most = 0;
    }
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

  // The key in bins lo to hi at which the amount in order first reaches `need`
  // (`before` those bins): three levels of 11, 11 and 10 key bits. Returns the
  // key; s.before: amount strictly before it, s.at: amount of its tokens.
  template <bool MASS, typename K>
  SPEC_DEV uint32_t radix(int lo, int hi, ull need, ull before, K keep) {
    uint32_t pre = 0;
#pragma unroll 1
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
      const int bits = level == 2 ? 10 : 11;
      for (int i = threadIdx.x; i < BINS; i += NT) s.mass[i] = 0ull;
      __syncthreads();
      auto one = [&](int i, float x) {
        const int b = sc.bin(x);
        if (b < lo || b > hi) return;
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

  // The n tokens handed to the first CTA, PT a thread: their order (key, index)
  // and weight (1 where they are counted); s.key_lo and s.key_hi: their keys' range.
  template <bool MASS>
  SPEC_DEV void take_listed(int n, ull (&e)[PT], ull (&w)[PT]) {
    if (threadIdx.x == 0) {
      s.key_lo = 0xffffffffu;
      s.key_hi = 0u;
    }
    __syncthreads();
    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      const int i = threadIdx.x + j * NT;
      e[j] = i < n ? s.sort[i] : ~0ull;
      const uint32_t key = (uint32_t)(e[j] >> 32);
      w[j] = i >= n ? 0ull : MASS ? weight_once(sc, s.tab, rank_val(key), nullptr) : 1ull;
      if (i < n) {
        lo = min(lo, key);
        hi = max(hi, key);
      }
    }
    lo = __reduce_min_sync(FULL, lo);
    hi = __reduce_max_sync(FULL, hi);
    if ((threadIdx.x & 31) == 0) {
      atomicMin(&s.key_lo, lo);
      atomicMax(&s.key_hi, hi);
    }
    __syncthreads();
  }

  // Of the first CTA's words in [lo, hi] with an amount, that at which the sum of
  // the amounts in the words' order, `before` ahead of all, reaches need >= 1 (~0:
  // nowhere); *ahead: the sum before it, *at: its amount. FINE bins of the range at
  // a time, until one holds few words, which are counted (sorting 700 tokens took
  // 10 us, one level of bins takes 1).
  SPEC_DEV ull select(const ull (&word)[PT], const ull (&amount)[PT], ull lo, ull hi, ull need, ull before,
                      ull* ahead, ull* at) {
#pragma unroll 1
    for (;;) {
      const int shift = max(0, 55 - __clzll((long long)((hi - lo) | 1)));
      s.fine[threadIdx.x] = 0ull;
      if (threadIdx.x == 0) {
        s.n_tied = 0;
        s.bin = -1;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < PT; ++j)
        if (amount[j] && word[j] >= lo && word[j] <= hi) atomicAdd(&s.fine[(word[j] - lo) >> shift], amount[j]);
      __syncthreads();
      const ull h = s.fine[threadIdx.x], b = before + block_scan(h);
      if (b < need && need <= b + h) {
        s.bin = threadIdx.x;
        s.before = b;
      }
      __syncthreads();
      const int bin = s.bin;
      if (bin < 0) return ~0ull;
      before = s.before;
      lo += (ull)bin << shift;
      hi = min(hi, lo + ((1ull << shift) - 1));
#pragma unroll
      for (int j = 0; j < PT; ++j)
        if (amount[j] && word[j] >= lo && word[j] <= hi) {
          const int i = atomicAdd(&s.n_tied, 1);
          if (i < TIED) {
            s.tied[i][0] = word[j];
            s.tied[i][1] = amount[j];
          }
        }
      __syncthreads();
      const int ties = s.n_tied;
      if (ties <= TIED) {
        if ((int)threadIdx.x < ties) {
          const ull mine = s.tied[threadIdx.x][0], own = s.tied[threadIdx.x][1];
          ull a = before;
          for (int j = 0; j < ties; ++j)
            if (s.tied[j][0] < mine) a += s.tied[j][1];
          if (a < need && need <= a + own) {
            s.word = mine;
            s.before = a;
            s.at = own;
          }
        }
        __syncthreads();
        *ahead = s.before;
        *at = s.at;
        const ull r = s.word;
        __syncthreads();
        return r;
      }
      __syncthreads();
    }
  }

  // The token of the n handed to the first CTA at which the amount in order,
  // `before` ahead of them, reaches `need`; the same cut in every CTA.
  template <bool MASS>
  SPEC_DEV void cut_listed(Cut& cut, int n, ull need, ull before) {
    if (cta == 0) {
      ull e[PT], w[PT], ahead, at;
      take_listed<MASS>(n, e, w);
      // (tokens without weight are not listed: a count that ends among them cuts nothing)
      const ull word = select(e, w, (ull)s.key_lo << 32, ((ull)s.key_hi << 32) | 0xffffffffu, need, before, &ahead, &at);
      const Cut found = word == ~0ull ? Cut{0xffffffffu, 0x7fffffff} : Cut{(uint32_t)(word >> 32), (int)(uint32_t)word};
      if (threadIdx.x < C) *cl.map_shared_rank(&s.cut, threadIdx.x) = found;
    }
    cl.sync();
    cut = s.cut;
  }

  // The cut behind k tokens, which lies in bin s.lo with s.n_lo ahead of it.
  SPEC_DEV void cut_count(Cut& cut, int k) {
    const int bin = s.lo;
    const ull before = s.n_lo;
    const float lo = (float)bin, hi = bin < BINS - 1 ? (float)(bin + 1) : INFINITY;
    scan([&](int i, float x) { list(i, x, lo, hi); });
    cl.sync();
    push_list();
    cl.sync();
    const int n = *cl.map_shared_rank(&s.gathered, 0);
    if (n <= FEW) {
      cut_listed<false>(cut, n, k, before);
      return;
    }
    cl.sync();
    const uint32_t key = radix<false>(bin, bin, k, before, [](int, float) { return true; });
    cut_ties(cut, key, k - s.before, s.at);
  }

  // Narrows the cut to the `r` lowest indices among the `n` kept tokens of key.
  SPEC_DEV void cut_ties(Cut& cut, uint32_t key, ull r, ull n) {
    if (r < n) {
      const Cut old = cut;
      auto same = [=](int i, float x) { return rank_key(x) == key && kept(old, key, i) ? 1ull : 0ull; };
      Amount<decltype(same)> eq{same};
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
    const float v = sc.place(x);
    if (v < hi && v >= lo) append(s, i, x);
  }

  // Whether top-p's nucleus probably lies among the tokens of the bins before `bins`,
  // as far as the row's n segment maxima tell: those behind hold at most a quarter of
  // the 1 - p that may be cut. (64 rows of 262144 of mixed breadth, mean of 12 draws of
  // the rows: 81 us, 82 with an eighth, 88 with a fiftieth, 90 without looking; one
  // draw: 85 with a quarter, 89 with a half, 94 with all of it. 40 rows with few likely
  // tokens 33 us, 64 without; 40 rows with a broad nucleus 82 us, 79 without.)
  SPEC_DEV bool promising(int bins, int n, float p) {
    if (threadIdx.x < 2) s.seen[threadIdx.x] = 0.f;
    __syncthreads();
    float in = 0.f, all = 0.f;
    for (int i = threadIdx.x; i < n; i += NT) {
      const float w = sc.m == INFINITY ? (s.seg[i] == INFINITY ? 1.f : 0.f) : exp2f((s.seg[i] - sc.m) * sc.sh);
      all += w;
      if (sc.bin(s.seg[i]) < bins) in += w;
    }
    in = warp_sum(in);
    all = warp_sum(all);
    if ((threadIdx.x & 31) == 0) {
      s.scan[threadIdx.x >> 5][0] = __float_as_uint(in);
      s.scan[threadIdx.x >> 5][1] = __float_as_uint(all);
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      float t = 0.f;
      for (int w = 0; w < NW; ++w) t += __uint_as_float((uint32_t)s.scan[w][threadIdx.x]);
      s.seen[threadIdx.x] = t;
    }
    __syncthreads();
    return s.seen[1] - s.seen[0] <= 0.25f * (1.f - p) * s.seen[1];
  }

  // Lists the tokens of the first bins in order, below `end`, for the first CTA,
  // with bounds of the mass of the tokens behind them. Returns their number.
  // (A weight of the tail is off by three roundings of its exponent, 4e-6 up to
  // 2^-32 of the largest weight, and by 1e-6 for the exponential and a step's sum:
  // below 2^-17 together. Smaller ones, their rounding to units and the steps' are
  // below a unit a token and 2^-30.)
  SPEC_DEV int list_head(float end, ull* tail_least, ull* tail_most) {
    if (threadIdx.x == 0) s.all = 0;
    __syncthreads();
    Tail f{sc, s, end, 0.f, 0ull};
    part.template each_rolled<WIDE>(part.v0, part.v1, f, [&](int) { f.step(); });
    const ull w = warp_sum_u64(f.all);
    if ((threadIdx.x & 31) == 0) atomicAdd(&s.all, w);
    __syncthreads();
    push_list();
    if (threadIdx.x < C) cl.map_shared_rank(&s, threadIdx.x)->x_bins[cta][0] = s.all;
    cl.sync();
    ull tail = 0;
    for (int c = 0; c < C; ++c) tail += s.x_bins[c][0];
    const ull off = (tail >> 17) + part.V + (1ull << (WBITS - 30));
    *tail_least = tail > off ? tail - off : 0ull;
    *tail_most = tail + off;
    return *cl.map_shared_rank(&s.gathered, 0);
  }

  // Top-p: the cut at which the tokens inside the present one reach the mass p, in
  // the bins of find_bins. SUMMED: *kept_mass and *before are sum()'s of the tokens
  // that the cut and min-p (weights from qw on) keep; DRAWN: a nucleus of few tokens
  // has been drawn from by draw(their number, false, the mass, the mass).
  enum Outcome { CUT, SUMMED, DRAWN };
  template <typename D>
  SPEC_DEV Outcome cut_mass(Cut& cut, bool cutting, float p, ull qw, D draw, ull* kept_mass, ull* before) {
    const int lo = s.lo, hi = s.hi;
    const bool few = s.n_hi <= COUNTED;
    ull least, most;
    bounds(lo, least, most);
    if (!few && qw > most) return CUT;   // min-p keeps fewer
    Nucleus f{sc, s, cut, cutting, few ? 0.f : (float)lo, end_of(hi + 1), 0ull};
    sum_part(f);
    const ull w = warp_sum_u64(f.all);
    if ((threadIdx.x & 31) == 0) atomicAdd(&s.all, w);
    push_list();
    if (threadIdx.x < C) {
      ull* o = *cl.map_shared_rank(&s.x_bins[cta], threadIdx.x);
      o[0] = s.total;
      o[1] = s.all;
    }
    cl.sync();
    ull ahead = 0, all = 0;
    for (int c = 0; c < C; ++c) {
      ahead += s.x_bins[c][0];
      all += s.x_bins[c][0] + s.x_bins[c][1];
    }
    const int n = *cl.map_shared_rank(&s.gathered, 0);
    if (few) {
      draw(n, false, all, all);
      return DRAWN;
    }
    const ull need = top_p_mass(p, all);
    if (n > FEW) {
      cl.sync();
      const Cut old = cut;
      const uint32_t key = radix<true>(lo, hi, need, ahead, [=](int i, float x) { return kept(old, rank_key(x), i); });
      const ull v = weight_once(sc, s.tab, rank_val(key), nullptr);
      cut_ties(cut, key, (need - s.before + v - 1) / v, s.at / v);
      return CUT;
    }
    cut_listed<true>(cut, n, need, ahead);
    if (lo > 0) {
      bounds(lo - 1, least, most);
      if (qw > least) return CUT;   // min-p's end may lie ahead of bin lo
    }
    // the sums ahead of bin lo, and the listed tokens that are kept
    for (int j = threadIdx.x; j < s.listed; j += NT) {
      const uint32_t key = s.list_key[j];
      const int i = s.list_idx[j];
      const ull v = kept(cut, key, i) ? weight_once(sc, s.tab, rank_val(key), nullptr) : 0ull;
      if (v == 0 || v < qw) continue;
      const int vec = (i + part.mis) / Part<T>::E, warp = vec / part.per;
      const int from = warp * part.per, len = min(part.nvec, from + part.per) - from;
      atomicAdd(&s.chunk[warp - cta * NW][(vec - from) / (32 * chunk_vectors(len))], v);
    }
    __syncthreads();
    const int len = part.v1 - part.v0, lane = threadIdx.x & 31;
    const ull sum = warp_sum_u64(lane * 32 * chunk_vectors(len) < len ? s.chunk[threadIdx.x >> 5][lane] : 0ull);
    if (lane == 0) s.wsum[threadIdx.x >> 5] = sum;
    __syncthreads();
    ull total = 0;
#pragma unroll 4
    for (int i = 0; i < NW; ++i) total += s.wsum[i];
    *kept_mass = cluster_sum(total, before);
    return SUMMED;
  }

  // Where the bins before `bins` end. The last bin holds tokens without weight
  // where the range was cut: not listed.
  SPEC_DEV float end_of(int bins) const {
    return bins < BINS ? (float)bins : range < Z_END ? INFINITY : (float)(BINS - 1);
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
    if (threadIdx.x == 0) s.base = atomicAdd(gathered, n <= FEW ? n : FEW + 1);
    __syncthreads();
    const int base = s.base;
    if (n > FEW || base + n > FEW) return;
    ull* sort0 = cl.map_shared_rank(s.sort, 0);
    for (int i = threadIdx.x; i < n; i += NT) sort0[base + i] = ((ull)s.list_key[i] << 32) | (unsigned int)s.list_idx[i];
  }

  // draw_few for at most COUNTED tokens, which are not sorted: two threads a
  // token count the tokens (and their mass) ahead of it, in the order and then
  // in the vocabulary.
  SPEC_DEV int draw_counted(int n, int k, float p, ull qw, float u, bool tail, ull least, ull most, ull* kept_mass) {
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
      const ull z = tail ? s.total : 0ull, need = top_p_mass(p, z + least), last = top_p_mass(p, z + most);
      if (__syncthreads_or(last > s.total || (keep && (ahead < need) != (ahead < last)))) return -1;
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

  // Of a row without filters: the sums of this CTA's chunks and the keys of their
  // maxima, pushed to the first CTA, as the chunk kernel leaves them.
  SPEC_DEV void chunk_sums() {
    constexpr int E = Part<T>::E, PER = CHUNK_TOKENS / E, NV = PER / NT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, chunks = row_chunks(part.V);
    auto& to = cl.map_shared_rank(&s, 0)->chunks;
    uint4 q[NV], next[NV];
    auto load = [&](int c, uint4 (&v)[NV]) {
      if (c >= chunks) return;
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = row_vector(part.p, part.V, part.mis, c * PER + j * NT + threadIdx.x);
      if (part.mis && threadIdx.x == 0)   // (as the chunk kernel)
        v[0] = merge<T>(v[0], row_vector(part.p, part.V, part.mis, (c + 1) * PER), part.mis);
    };
    load(cta, q);
#pragma unroll 1
    for (int c = cta; c < chunks; c += C) {
      load(c + C, next);
      float bx = -INFINITY;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) bx = fmaxf(bx, Part<T>::get(q[j], i));
      uint32_t key = __reduce_max_sync(FULL, bx > -INFINITY ? ord_key(bx + 0.f) : 0u);
      if (lane == 0) s.list_key[warp] = key;
      __syncthreads();
      key = __reduce_max_sync(FULL, s.list_key[lane & (NW - 1)]);
      ull sum = 0;
      if (key) {
        Scale in = sc;
        in.m = ord_val(key);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < E; i += 2) {
            ull w0, w1;
            weight2(in, s.tab, Part<T>::get(q[j], i), Part<T>::get(q[j], i + 1), w0, w1);
            sum += w0 + w1;
          }
        sum = warp_sum_u64(sum);
      }
      if (lane == 0) s.wsum[warp] = sum;
      __syncthreads();
      if (warp == 0) {
        sum = warp_sum_u64(lane < NW ? s.wsum[lane] : 0ull);
        if (lane == 0) {
          to.sum[c] = sum;
          to.top[c] = key;
        }
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) q[j] = next[j];
    }
  }

  // The first CTA's end of the usual case: the n listed tokens, the row's best, are
  // cut and drawn from in index order. Top-p takes the row's whole mass between
  // least and most, or with `tail` that of the tokens behind those (0: top-k); -1
  // where the cut depends on which, or lies behind them. Returns the token,
  // *kept_mass its kept mass.
  SPEC_DEV int draw_few(int n, int k, float p, ull qw, float u, bool tail, ull least, ull most,
                        ull* kept_mass) {
    if (n <= COUNTED) return draw_counted(n, k, p, qw, u, tail, least, most, kept_mass);
    ull e[PT], w[PT], t[PT], ahead, at, last = ~0ull;
    take_listed<true>(n, e, w);
    const ull lo = (ull)s.key_lo << 32, hi = ((ull)s.key_hi << 32) | 0xffffffffu;
    if (k > 0 && k < n) {
#pragma unroll
      for (int j = 0; j < PT; ++j) t[j] = e[j] != ~0ull;
      last = select(e, t, lo, hi, k, 0ull, &ahead, &at);
    }
    auto keep = [&](ull from) {   // in t, those of weight `from` on; returns their mass
      ull sum = 0;
#pragma unroll
      for (int j = 0; j < PT; ++j) {
        t[j] = e[j] <= last && w[j] >= from ? w[j] : 0ull;
        sum += t[j];
      }
      block_total(sum);
      return s.total;
    };
    if (p < 1.f) {
      const ull z = keep(0ull), need = top_p_mass(p, least + (tail ? z : 0ull)), far = top_p_mass(p, most + (tail ? z : 0ull));
      if (far > z) return -1;
      last = select(e, t, lo, hi, need, 0ull, &ahead, &at);
      if (far > ahead + at) return -1;
    }
    const ull z = keep(qw);
    *kept_mass = z;
#pragma unroll
    for (int j = 0; j < PT; ++j) e[j] = (uint32_t)e[j];
    return (int)select(e, t, 0ull, (ull)(part.V - 1), drawn_mass(u, z) + 1, 0ull, &ahead, &at);
  }
};

// log2(e) / T as a float pair.
SPEC_DEV void scale_of(float temp, float& sh, float& sl) {
  constexpr float L = 1.44269502f;                                   // log2(e) rounded
  constexpr float L_LO = (float)(1.4426950408889634 - (double)L);
  sh = L / temp;
  sl = (fmaf(-sh, temp, L) + L_LO) / temp;
}

// ALIGNED: every row starts on 16 bytes.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(CNT, 4) chunk_kernel(SampleArgs a, Record* records) {
  constexpr int E = 16 / sizeof(T), PER = CHUNK_TOKENS / E, NV = PER / CNT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ull* tab = reinterpret_cast<ull*>(smem_raw);
  __shared__ ull s_sum[2][CNW];
  __shared__ uint32_t s_key[2][CNW], s_at[2][CNW];
  for (int i = threadIdx.x; i < TAB / 2; i += CNT) {
    const unsigned int dst = (unsigned int)__cvta_generic_to_shared(tab + 2 * i);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(g_table.v + 2 * i) : "memory");
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = row_chunks(a.V), items = a.M * n;
  grid_dep_wait();
  // A chunk's vectors, as they lie in memory. Where its first token does not start one,
  // the first vector begins with tokens of the chunk before, and as many of this one's
  // are left in the vector behind the last (`tail`): they take those places.
  uint4 q[NV], next[NV], tail = {}, tail_next = {};
  float temp = 0.f, temp_next = 0.f;
  auto load = [&](int item, uint4 (&v)[NV], uint4& behind, float& t) {
    if (item >= items) return;
    const int row = item / n, c = item - row * n;
    const T* p = (const T*)a.logits + (size_t)row * a.ld;
    const int mis = ALIGNED ? 0 : (int)(((uintptr_t)p & 15) / sizeof(T));
    const int i0 = c * CHUNK_TOKENS - mis;
    if (i0 >= 0 && i0 + CHUNK_TOKENS <= a.V) {   // for the whole CTA: plain loads, nothing to merge
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = reinterpret_cast<const uint4*>(p + i0)[j * CNT + threadIdx.x];
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = row_vector(p, a.V, mis, c * PER + j * CNT + threadIdx.x);
    }
    if (mis && threadIdx.x == 0) behind = row_vector(p, a.V, mis, (c + 1) * PER);
    t = a.temperature ? a.temperature[row] : 1.f;
  };
  load(blockIdx.x, q, tail, temp);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  int turn = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x, turn ^= 1) {
    load(item + gridDim.x, next, tail_next, temp_next);
    const int row = item / n, c = item - row * n;
    const int mis = ALIGNED ? 0 : (int)(((uintptr_t)((const T*)a.logits + (size_t)row * a.ld) & 15) / sizeof(T));
    if (mis && threadIdx.x == 0) q[0] = merge<T>(q[0], tail, mis);
    float bx = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) bx = max_nan(bx, Part<T>::get(q[j], i));
    uint32_t key = bx > -INFINITY ? ord_key(bx + 0.f) : 0u;
    key = __reduce_max_sync(FULL, key);
    if (lane == 0) s_key[turn][warp] = key;
    const int nan = __syncthreads_or(bx != bx);
#pragma unroll
    for (int w = 0; w < CNW; ++w) key = max(key, s_key[turn][w]);
    ull best = key ? pack_best(ord_val(key), 0u) : 0ull;
    if (key && temp < 1e-5f) {   // (greedy: the whole CTA) the lowest index of the maximum
      uint32_t at = 0xffffffffu;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (Part<T>::get(q[j], i) == ord_val(key)) {
            const int place = (j * CNT + threadIdx.x) * E - mis + i;
            at = min(at, (uint32_t)(c * CHUNK_TOKENS + (place < 0 ? place + CHUNK_TOKENS : place)));
          }
      at = __reduce_min_sync(FULL, at);
      if (lane == 0) s_at[turn][warp] = at;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < CNW; ++w) at = min(at, s_at[turn][w]);
      best = pack_best(ord_val(key), at);
    }
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
    tail = tail_next;
    temp = temp_next;
  }
}

// Draws from a row without filters: its chunks' sums in the row's units, the chunk in
// which the drawn mass lies, and the token in it. Thread c brings chunk c's sum and the
// key of its maximum (0: nothing above -inf, or no such chunk).
template <typename T>
SPEC_DEV void draw_row(const SampleArgs& a, int row, const ull* tab, const Scale& sc, float u, ull sum, uint32_t key,
                       Drawn& d) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](ull v) {   // exclusive, in thread order
    const ull inc = warp_scan_u64(v);
    __syncthreads();
    if (lane == 31) d.wsum[warp] = inc;
    __syncthreads();
    ull b = inc - v;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      if (i < warp) b += d.wsum[i];
    return b;
  };
  ull v = 0, mass = 0;
  int n = 0;
  if (key) {
    v = weight_parts(sc, tab, ord_val(key), n);
    mass = in_row(sum, v, n);
  }
  const ull from = scan(mass);
  if (threadIdx.x == NT - 1) d.total = from + mass;
  __syncthreads();
  const ull z = d.total, drawn = drawn_mass(u, z);
  if (drawn >= from && drawn < from + mass) {
    d.chunk = threadIdx.x;
    d.top = key;
    d.before = from;
    d.factor = v;
    d.shift = n;
  }
  __syncthreads();
  // the chunk again, NV consecutive vectors a thread
  constexpr int E = Part<T>::E, PER = CHUNK_TOKENS / E, NV = PER / NT;
  const int c = d.chunk;
  const ull t = drawn - d.before;
  v = d.factor;
  n = d.shift;
  const T* p = (const T*)a.logits + (size_t)row * a.ld;
  const int mis = (int)(((uintptr_t)p & 15) / sizeof(T));
  Scale in = sc;
  in.m = ord_val(d.top);
  sum = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint4 q = token_vector(p, a.V, mis, c * PER + threadIdx.x * NV + j);
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
    for (int i = (c * PER + threadIdx.x * NV) * E; i < a.V; ++i) {
      const float x = Part<T>::one(p + i);
      b += weight(in, tab, x);
      if (t < in_row(b, v, n)) {
        float w;
        weight(sc, tab, x, &w);
        a.tokens[row] = i;
        if (a.probs) a.probs[row] = w / ((float)z * (1.f / (float)(1ull << WBITS)));
        break;
      }
    }
  }
}

// A row of a call without filters, from its chunks' records.
template <typename T>
__global__ void __launch_bounds__(NT) draw_kernel(SampleArgs a, const Record* records) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ull* tab = reinterpret_cast<ull*>(smem_raw);
  __shared__ Drawn d;
  for (int i = threadIdx.x; i < TAB / 2; i += NT) {
    const unsigned int dst = (unsigned int)__cvta_generic_to_shared(tab + 2 * i);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(g_table.v + 2 * i) : "memory");
  }
  const int row = blockIdx.x, chunks = row_chunks(a.V), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  const Record* rec = records + (size_t)row * chunks;
  const float temp = a.temperature ? a.temperature[row] : 1.f, u = a.uniform[row];
  ull best = 0, mine = 0, sum = 0;
  int nan = 0;
  if (threadIdx.x < chunks) {
    mine = __ldcg(&rec[threadIdx.x].best);
    sum = __ldcg(&rec[threadIdx.x].sum);
    nan = __ldcg(&rec[threadIdx.x].nan);
  }
  {
    const uint32_t key = __reduce_max_sync(FULL, (uint32_t)(mine >> 32));
    const uint32_t idx = __reduce_max_sync(FULL, (uint32_t)(mine >> 32) == key ? (uint32_t)mine : 0u);
    if (lane == 0) d.wsum[warp] = ((ull)key << 32) | idx;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  nan = __syncthreads_or(nan);
#pragma unroll
  for (int i = 0; i < NW; ++i) best = d.wsum[i] > best ? d.wsum[i] : best;
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
  draw_row<T>(a, row, tab, sc, u, sum, (uint32_t)(mine >> 32), d);
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
  const float q = a.min_p ? a.min_p[row] : 0.f;
  const float u = a.uniform[row];
  S.part.bind((const T*)a.logits + (size_t)row * a.ld, a.V, cta, C);
  const bool greedy = temp < 1e-5f, cuts = k > 0 || p < 1.f;
  int seg_lanes = 1;
  while (C * NT / seg_lanes > SEG_MAX) seg_lanes *= 2;

  // maximum, minimum, segment maxima; a NaN anywhere leaves the row without a
  // distribution
  float bx = -INFINITY, low = INFINITY;
  S.part.each([&](int, float x) {
    low = fminf(low, x);
    bx = max_nan(bx, x);
  });
  int nan = bx != bx;
  uint32_t key = bx > -INFINITY ? ord_key(bx + 0.f) : 0u;
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
  key = __reduce_max_sync(FULL, key);
  low = ord_val(__reduce_min_sync(FULL, ord_key(low)));
  if (lane == 0) {
    s.list_key[warp] = key;
    reinterpret_cast<float*>(s.list_idx)[warp] = low;
  }
  nan = __syncthreads_or(nan);
  if (threadIdx.x < C) {
    for (int i = 0; i < NW; ++i) {
      key = max(key, s.list_key[i]);
      low = fminf(low, reinterpret_cast<float*>(s.list_idx)[i]);
    }
    *cl.map_shared_rank(&s.x_best[cta], threadIdx.x) = nan ? 0xffffffffu : key;   // (no value's key)
    *cl.map_shared_rank(&s.x_low[cta], threadIdx.x) = low;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  cl.sync();
  key = 0;
#pragma unroll
  for (int c = 0; c < MAX_C; ++c)
    if (c < C) {
      key = max(key, s.x_best[c]);
      low = fminf(low, s.x_low[c]);
    }

  auto write = [&](int token, float prob) {
    a.tokens[row] = token;
    if (a.probs) a.probs[row] = prob;
  };
  const float m = ord_val(key);
  if (key == 0u || key == 0xffffffffu || !(temp >= 0.f && temp < INFINITY)) {   // no distribution
    if (cta == 0 && threadIdx.x == 0) write(-1, 0.f);
    return;
  }
  if (greedy) {   // the lowest index of the maximum
    uint32_t at = 0xffffffffu;
    S.part.each([&](int i, float x) {
      if (x == m) at = min(at, (uint32_t)i);
    });
    at = __reduce_min_sync(FULL, at);
    if (lane == 0) s.list_key[warp] = at;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 0; i < NW; ++i) at = min(at, s.list_key[i]);
      *cl.map_shared_rank(&s.x_total[cta], 0) = at;
    }
    cl.sync();
    if (cta == 0 && threadIdx.x == 0) {
      ull first = s.x_total[0];
      for (int c = 1; c < C; ++c) first = min(first, s.x_total[c]);
      write((int)first, 1.f);
    }
    return;
  }

  float sh, sl;
  scale_of(temp, sh, sl);
  // finer bins where the row's range of exponents is less than the weights'
  const float range = fminf((m - low) * sh, Z_END);
  S.range = range;
  S.sc = Scale{m, sh, sl, range > 1e-30f ? (float)(BINS - 1) / range : 0.f};
  // min-p's smallest weight
  const ull qw = q > 0.f ? (q < 1.f ? scaled(q, 1ull << WBITS, true) : 1ull << WBITS) : 0ull;
  auto result = [&](int token, float x, ull z) {
    float v;
    weight_once(S.sc, s.tab, x, &v);
    write(token, v / ((float)z * (1.f / (float)(1ull << WBITS))));
  };

  // no filter: as a call without any gives it (of a row of one chunk the sum below is
  // the same, by all CTAs: 1 x 4096 8.1 us, 9.1 by the first one alone)
  if (!cuts && qw == 0 && a.V > CHUNK_TOKENS) {
    S.chunk_sums();
    cl.sync();
    if (cta == 0) {
      const bool mine = threadIdx.x < row_chunks(a.V);
      draw_row<T>(a, row, s.tab, S.sc, u, mine ? s.chunks.sum[threadIdx.x] : 0ull, mine ? s.chunks.top[threadIdx.x] : 0u,
                  s.chunks.drawn);
    }
    return;
  }
  if (!cuts) {
    Mass mass{S.sc, s.tab, qw, Cut{}, false};
    ull before;
    const ull z = S.sum(mass, &before);
    S.find_in_order(mass, drawn_mass(u, z), before, [&](int i, float x) { result(i, x, z); });
    return;
  }

  // the first CTA draws among the n tokens handed to it, if they fit and decide it
  auto draw = [&](int n, bool tail, ull least, ull most) {
    if (n <= FEW && cta == 0) {
      ull z;
      const int token = S.draw_few(n, k, p, qw, u, tail, least, most, &z);
      if (threadIdx.x == 0 && token >= 0) result(token, Part<T>::one((const T*)a.logits + (size_t)row * a.ld + token), z);
      if (threadIdx.x < C) *cl.map_shared_rank(&s.undecided, threadIdx.x) = token < 0;
    }
    cl.sync();   // its count is read, and its tokens are, before either changes
    return n <= FEW && !s.undecided;
  };
  Cut cut{0xffffffffu, 0x7fffffff};
  ull z = 0, before = 0;
  bool summed = false;
  const int segs = C * NT / seg_lanes;
  if (k > 0) {
    if (k <= segs && draw(S.list_below(S.end_of((S.threshold(k, segs) + 1) * (BINS / SEG_BINS))), true, 0ull, 0ull)) return;
    S.find_bins(cut, false, k, 1.f);
    S.cut_count(cut, k);
    k = 0;   // (the cut holds it)
  } else {
    const int bins = (S.threshold(HEAD, segs) + 1) * (BINS / SEG_BINS);
    if (S.promising(bins, segs, p)) {
      ull least, most;
      const int n = S.list_head(S.end_of(bins), &least, &most);
      if (draw(n, true, least, most)) return;
    }
  }
  if (p < 1.f) {
    const bool cutting = cut.idx != 0x7fffffff || cut.key != 0xffffffffu;
    S.find_bins(cut, cutting, 0, p);
    const auto outcome = S.cut_mass(cut, cutting, p, qw, draw, &z, &before);
    if (outcome == Sampler<T>::DRAWN) return;
    summed = outcome == Sampler<T>::SUMMED;
  }
  Mass mass{S.sc, s.tab, qw, cut, true};
  if (!summed) z = S.sum(mass, &before);
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
// clusters at a fixed cost of about 9 us (0.2 more a CTA of the exchanges) and
// 0.25 ns a token of a CTA, up to 0.5 ns as the SMs hold two CTAs each. Measured,
// 262144 tokens a row: 1 row with top-k 50 13 us with 16 CTAs, 15 with 8, 60 with
// 1; 64 rows with top-k 50 32 us with 4 CTAs, 46 with 2, 39 with 8.
template <typename T>
int cluster_size(int M, int V) {
  int best = MAX_C, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) dev = 0;
  const int sms = num_sms();
  double least = 1e30;
  for (int C : {1, 2, 3, 4, 6, 8, 16}) {
    const int fit = max_clusters<T>(dev, C);
    if (fit < 1) continue;
    double us = 0;
    for (int left = M; left > 0; left -= fit) {
      const double held = (double)std::min(left, fit) * C / sms;
      const double wave = 9.0 + 0.2 * C + (0.25 + 0.12 * held) * 1e-3 * V / C;
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
// 262144 tokens a row, 1 row 8.3 us (14.0 without), 40 rows 23.1 us (33.6).
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
  const bool aligned = (uintptr_t)a.logits % 16 == 0 && (a.M == 1 || a.ld * sizeof(T) % 16 == 0);
  if (cudaLaunchKernelEx(&cfg, aligned ? chunk_kernel<T, true> : chunk_kernel<T, false>, a, (Record*)a.workspace) !=
      cudaSuccess)
    return -1;
  cfg.gridDim = dim3(a.M);
  cfg.blockDim = dim3(NT);
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, draw_kernel<T>, a, (const Record*)a.workspace) == cudaSuccess ? 2 : -1;
}

template <typename T>
int launch_sample(const SampleArgs& a, int pdl, cudaStream_t st) {
  if (chunked(a.M, a.V) && !a.top_k && !a.top_p && !a.min_p) return launch_chunked<T>(a, pdl, st);
  const int C = cluster_size<T>(a.M, a.V);
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
  cudaFuncSetAttribute(chunk_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(TAB * sizeof(ull)));
  cudaFuncSetAttribute(chunk_kernel<T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(TAB * sizeof(ull)));
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
