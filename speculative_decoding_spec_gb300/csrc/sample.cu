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
// Weights are integers: w_i in units of 2^-44 of the largest, rounded down (a
// choice: tokens below 2^-44 of the most likely one count as zero). Their sums
// are exact, so the cut and the token do not depend on the order of the
// additions, the number of CTAs or the other rows of the batch. The weight
// itself is evaluated to about 2^-37 (the exponent as a float pair, a table of
// 4096 powers), because a token is decided by a sum of up to V weights next to
// a border: at the 2^-24 of plain floats about one token in 10^4 would differ
// from the 64-bit definition.
//
// A thread-block cluster takes a row; its CTAs push what the others need into
// their shared memory, so that a phase costs one cluster barrier. Scan 1 finds
// the maximum and the maxima of the row's segments (up to 1024).
// Without top-k and top-p, scan 2 sums the weights and the warp that holds the
// drawn mass finds the token. With them, scan 2 lists the tokens down to the
// k-th largest segment maximum -- at least k tokens, and rarely many more -- (top-p
// alone: down to the median one, and sums the weights too), and the first CTA
// sorts, cuts and draws among those alone. Where they are too many, or hold too
// little mass for top-p, the cut is found in the whole row: a histogram of 2048
// bins, linear in the exponent, of counts or of exact masses (three 15-bit
// digits), then a radix search of the keys inside one bin.
#include <cooperative_groups.h>

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
constexpr int DIGIT = 15;           // bits of a mass digit: 2^17 tokens of a CTA sum in 32 bits
constexpr int TAB_LOG = 12;
constexpr int TAB = 1 << TAB_LOG;   // 2^(-j/4096)
constexpr int MAX_C = 16;           // CTAs on one row (a thread-block cluster)
constexpr int LIST = 1024;          // tokens a CTA lists
constexpr int FEW = 2048;           // tokens the first CTA sorts
constexpr int SEG_MAX = 1024;       // segments of a row (the elements of 1, 2, 4 or 8 lanes)
constexpr int SEG_BINS = NT;        // bins of the segment maxima
constexpr float Z_END = 46.f;       // weights are zero beyond this exponent
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
  int few;                   // the first CTA's verdict: the listed tokens suffice
  unsigned int seg_bins[SEG_BINS];
  uint32_t threshold;        // largest rank key listed
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
  SPEC_DEV int bin(float x) const {
    if (m == INFINITY) return x == INFINITY ? 0 : BINS - 1;
    return (int)fminf((m - x) * sh * bins, (float)(BINS - 1));
  }
};

// The weight of logit x in units of 2^-WBITS. z is formed as a float pair (an
// exact difference, an exact product), split into n + j/4096 + g, and
// 2^-z = 2^-n * tab[j] * e^(-g ln 2) with a quadratic (Tang's table-driven
// reduction, ACM TOMS 15(2), 1989). val: the weight as a float.
SPEC_DEV ull weight(const Scale& r, const ull* tab, float x, float* val = nullptr) {
  if (r.m == INFINITY) {
    if (val) *val = x == INFINITY ? 1.f : 0.f;
    return x == INFINITY ? 1ull << WBITS : 0ull;
  }
  const float d = r.m - x;
  const float bb = d - r.m;
  const float e = (r.m - (d - bb)) + (-x - bb);       // d + e == m - x
  float p = d * r.sh;
  const float pe = fmaf(e, r.sh, fmaf(d, r.sl, fmaf(d, r.sh, -p)));
  p = fminf(p, 63.f);
  // round(4096 p) in the low bits of p + 1.5 * 2^(23 - 12)
  const float t = p + 12582912.f / TAB;
  const int j = __float_as_int(t) & 0x3fffff;
  const float g = (p - (t - 12582912.f / TAB)) + pe;  // |g| <= 2^-13
  const float q = fmaf(g, 0.240226507f, -0.693147181f) * g;   // 2^-g - 1
  const ull T = tab[j & (TAB - 1)];
  const int n = j >> TAB_LOG;
  // the table value as a float: its 24 leading bits (2^43 <= T <= 2^44)
  const float Tf = __uint_as_float((uint32_t)(T >> (WBITS - 24)) + 0x4a800000u) * (float)(1 << (WBITS - 24));
  const ull v = T + (long long)__float2int_rn(Tf * q);
  if (val) *val = fmaf(Tf, q, Tf) * __int_as_float((127 - WBITS - n) << 23);
  return v >> n;
}

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
  // f(index, value) for the elements of vector v
  template <typename F>
  SPEC_DEV void vec(int v, F& f) const {
    const int i0 = v * E - mis;
    if (i0 >= 0 && i0 + E <= V) {
      const uint4 q = *reinterpret_cast<const uint4*>(p + i0);
#pragma unroll
      for (int i = 0; i < E; ++i) f(i0 + i, get(q, i));
    } else {
      for (int i = max(0, -i0); i < E && i0 + i < V; ++i) f(i0 + i, one(p + i0 + i));
    }
  }
  template <typename F>
  SPEC_DEV void each(F f) const {
    int v = v0 + (int)(threadIdx.x & 31);
    for (; v + 32 * (U - 1) < v1 && v * E >= mis && (v + 32 * (U - 1)) * E - mis + E <= V; v += 32 * U) {
      uint4 q[U];
#pragma unroll
      for (int j = 0; j < U; ++j) q[j] = *reinterpret_cast<const uint4*>(p + (v + 32 * j) * E - mis);
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) f((v + 32 * j) * E - mis + i, get(q[j], i));
    }
#pragma unroll 1
    for (; v < v1; v += 32) vec(v, f);
  }
};

SPEC_DEV ull warp_sum_u64(ull v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
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

// A cut of the order: tokens with a smaller key, and those of this key up to
// this index, are kept.
struct Cut {
  uint32_t key;
  int idx;
};
SPEC_DEV bool kept(const Cut& c, uint32_t key, int i) { return key < c.key || (key == c.key && i <= c.idx); }

template <typename T>
struct Sampler {
  Shared& s;
  cg::cluster_group cl;
  int cta, C;
  Part<T> part;
  Scale sc;

  // Exclusive sum of v over the CTA's threads, in thread order.
  SPEC_DEV ull block_scan(ull v) {
    const ull inc = warp_scan_u64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 31) s.wsum[threadIdx.x >> 5] = inc;
    __syncthreads();
    ull b = inc - v;
    for (int i = 0; i < (int)(threadIdx.x >> 5); ++i) b += s.wsum[i];
    return b;
  }

  // Sum of f(index, value) over the row; wsum holds the warps' parts, and
  // `before` gets the sum of the cluster's earlier CTAs.
  template <typename F>
  SPEC_DEV ull sum(F f, ull* before) {
    ull a = 0;
    part.each([&](int i, float x) { a += f(i, x); });
    block_total(a);
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
  // the sum of f in index order exceeds t (t below the row's sum; wsum: the
  // warps' parts, before: the sum of the earlier CTAs).
  template <typename F, typename H>
  SPEC_DEV void find_in_order(F f, ull t, ull before, H hit) {
    constexpr int U = 4;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    ull b = before;
    for (int i = 0; i < w; ++i) b += s.wsum[i];
    if (t < b || t >= b + s.wsum[w]) return;
    for (int v0 = part.v0 + lane; v0 - lane < part.v1; v0 += 32 * U) {
      ull a[U], inc[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        a[j] = 0;
        auto add = [&](int i, float x) { a[j] += f(i, x); };
        if (v0 + 32 * j < part.v1) part.vec(v0 + 32 * j, add);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) inc[j] = warp_scan_u64(a[j]);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const ull tot = __shfl_sync(FULL, inc[j], 31);
        ull c = b + inc[j] - a[j];
        if (t >= c && t < c + a[j]) {
          bool done = false;
          auto walk = [&](int i, float x) {
            c += f(i, x);
            if (!done && t < c) {
              done = true;
              hit(i, x);
            }
          };
          part.vec(v0 + 32 * j, walk);
        }
        b += tot;
      }
      if (t < b) return;
    }
  }
  // The same index in every CTA.
  template <typename F>
  SPEC_DEV int find_all(F f, ull t, ull before) {
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

  // Histogram of the kept tokens' counts or exact masses by bin, in every
  // CTA: h[j] is the row's amount in bin threadIdx.x * BPT + j.
  template <bool MASS, typename K>
  SPEC_DEV void histogram(K keep, ull (&h)[BPT]) {
    constexpr int D = MASS ? 3 : 1;
    for (int i = threadIdx.x; i < D * BINS; i += NT) s.hist[0][i] = 0u;
    __syncthreads();
    part.each([&](int i, float x) {
      if (!keep(i, x)) return;
      const int b = sc.bin(x);
      if (MASS) {
        const ull w = weight(sc, s.tab, x);
        const unsigned int d0 = (unsigned int)w & ((1u << DIGIT) - 1),
                           d1 = (unsigned int)(w >> DIGIT) & ((1u << DIGIT) - 1),
                           d2 = (unsigned int)(w >> (2 * DIGIT));
        if (w) atomicAdd(&s.hist[0][b], d0);
        if (w >> DIGIT) atomicAdd(&s.hist[1][b], d1);
        if (d2) atomicAdd(&s.hist[2][b], d2);
      } else {
        atomicAdd(&s.hist[0][b], 1u);
      }
    });
    cl.sync();
#pragma unroll
    for (int j = 0; j < BPT; ++j) h[j] = 0;
#pragma unroll 4
    for (int c = 0; c < C; ++c) {
      const unsigned int* o = cl.map_shared_rank(&s.hist[0][0], c);
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const uint4 q = *reinterpret_cast<const uint4*>(o + d * BINS + threadIdx.x * BPT);
        h[0] += (ull)q.x << (d * DIGIT);
        h[1] += (ull)q.y << (d * DIGIT);
        h[2] += (ull)q.z << (d * DIGIT);
        h[3] += (ull)q.w << (d * DIGIT);
      }
    }
    cl.sync();  // read everywhere before it is written again
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
      part.each([&](int i, float x) {
        if (sc.bin(x) != bin) return;
        const uint32_t k = rank_key(x);
        if ((level > 0 && (k >> (shift + bits)) != pre) || !keep(i, x)) return;
        atomicAdd(&s.mass[(k >> shift) & ((1 << bits) - 1)], MASS ? weight(sc, s.tab, x) : 1ull);
      });
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

  // Narrows the cut to the `r` lowest indices among the `n` kept tokens of key.
  SPEC_DEV void cut_ties(Cut& cut, uint32_t key, ull r, ull n) {
    if (r < n) {
      const Cut old = cut;
      auto eq = [&](int i, float x) { return rank_key(x) == key && kept(old, key, i) ? 1ull : 0ull; };
      ull before;
      sum(eq, &before);
      cut.idx = find_all(eq, r - 1, before);
    } else if (key < cut.key) {
      cut.idx = 0x7fffffff;
    }
    cut.key = key;
  }

  // The rank key down to which at least `need` tokens of weight lie: that of the
  // need-th largest segment maximum, found to a bin of them (and tokens
  // without weight are never listed). Every CTA finds the same.
  SPEC_DEV uint32_t threshold(int need, int n) {
    if (threadIdx.x == 0) s.threshold = 0u;
    const float end = sc.m == INFINITY ? sc.m : sc.m - Z_END / sc.sh;
    for (int i = threadIdx.x; i < n; i += NT) atomicAdd(&s.seg_bins[sc.bin(s.seg[i]) / (BINS / SEG_BINS)], 1u);
    __syncthreads();
    const unsigned int c = s.seg_bins[threadIdx.x];
    const ull b = block_scan(c);
    if (b < (ull)need && (ull)need <= b + c) s.bin = threadIdx.x;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT)
      if (sc.bin(s.seg[i]) / (BINS / SEG_BINS) <= s.bin) atomicMax(&s.threshold, rank_key(s.seg[i]));
    __syncthreads();
    return min(s.threshold, rank_key(end));
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

  // Ascending bitonic sort of s.sort[0, n2), n2 a power of two.
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
        __syncthreads();
      }
  }

  // The first CTA's end of the usual case: the n listed tokens sorted by
  // (key, index), cut, and drawn from in index order. mass: the row's whole
  // mass (top-p without top-k). Returns the token, *kept_mass its kept mass; -1
  // if the listed tokens hold less than top-p's mass.
  SPEC_DEV int draw_few(int n, int k, float p, ull qw, float u, ull mass, ull* kept_mass) {
    int n2 = 64;
    while (n2 < n) n2 <<= 1;
    for (int i = n + threadIdx.x; i < n2; i += NT) s.sort[i] = ~0ull;
    if (threadIdx.x == 0) s.r = k > 0 ? min(n, k) : n;
    __syncthreads();
    sort(n2);
    constexpr int PT = FEW / NT;
    // weights of the first r tokens, PT consecutive ones a thread
    const int r1 = s.r;
    ull e[PT], w[PT], t = 0;
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      const int i = threadIdx.x * PT + j;
      e[j] = i < r1 ? s.sort[i] : 0ull;
      w[j] = i < r1 ? weight(sc, s.tab, rank_val((uint32_t)(e[j] >> 32))) : 0ull;
      t += w[j];
    }
    const ull b0 = block_scan(t);
    if (threadIdx.x == NT - 1) s.total = b0 + t;
    __syncthreads();
    int r = r1;
    if (p < 1.f) {
      const ull need = top_p_mass(p, k > 0 ? s.total : mass);
      if (need > s.total) return -1;
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
  const int seg_lanes = max(1, C * NT / SEG_MAX);

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
    for (int j = lane; j < per * C; j += 32) {
      const float v = __shfl_sync(FULL, bx, (j & (per - 1)) * seg_lanes);
      cl.map_shared_rank(s.seg, j / per)[(cta * NW + warp) * per + (j & (per - 1))] = v;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const ull other = __shfl_xor_sync(FULL, best, o);
    best = other > best ? other : best;
    low = fminf(low, __shfl_xor_sync(FULL, low, o));
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
  for (int c = 0; c < C; ++c) {
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
  // log2(e) / T as a float pair
  constexpr float L = 1.44269502f;                                   // log2(e) rounded
  constexpr float L_LO = (float)(1.4426950408889634 - (double)L);
  const float sh = L / temp, sl = (fmaf(-sh, temp, L) + L_LO) / temp;
  // finer bins where the row's range of exponents is less than the weights'
  const float range = fminf((m - low) * sh, Z_END);
  S.sc = Scale{m, sh, sl, range > 1e-30f ? (float)(BINS - 1) / range : 0.f};
  // min-p's smallest weight
  const ull qw = q > 0.f ? (q < 1.f ? scaled(q, 1ull << WBITS, true) : 1ull << WBITS) : 0ull;
  auto result = [&](int token, float x, ull z) {
    float v;
    weight(S.sc, s.tab, x, &v);
    write(token, v / ((float)z * (1.f / (float)(1ull << WBITS))));
  };

  if (!cuts) {
    auto mass = [&](int, float x) {
      const ull w = weight(S.sc, s.tab, x);
      return w < qw ? 0ull : w;
    };
    ull t = 0;
    S.part.each([&](int i, float x) { t += mass(i, x); });
    S.block_total(t);
    if (threadIdx.x < C) *cl.map_shared_rank(&s.x_total[cta], threadIdx.x) = s.total;
    cl.sync();
    ull z = 0, before = 0;
    for (int c = 0; c < C; ++c) {
      if (c == cta) before = z;
      z += s.x_total[c];
    }
    S.find_in_order(mass, drawn_mass(u, z), before, [&](int i, float x) { result(i, x, z); });
    return;
  }

  // the tokens that may be kept, listed for the first CTA
  const bool by_mass = k == 0;
  const int segs = C * NT / seg_lanes, need_k = by_mass ? segs / 2 : k;
  if (need_k <= segs) {
    const uint32_t thr = S.threshold(need_k, segs);
    const float xthr = rank_val(thr);
    auto add = [&](int i, float x) {
      if (x >= xthr) {
        const int at = atomicAdd(&s.listed, 1);
        if (at < LIST) {
          s.list_key[at] = rank_key(x);
          s.list_idx[at] = i;
        }
      }
    };
    if (by_mass) {
      ull t = 0;
      S.part.each([&](int i, float x) {
        t += weight(S.sc, s.tab, x);
        add(i, x);
      });
      S.block_total(t);
      if (threadIdx.x == 0) *cl.map_shared_rank(&s.x_total[cta], 0) = s.total;
    } else {
      S.part.each(add);
      __syncthreads();
    }
    S.push_list();
    cl.sync();
    const int n = *cl.map_shared_rank(&s.gathered, 0);
    int token = -1;
    if (n <= FEW && cta == 0) {
      ull mass = 0, z = 0;
      if (by_mass)
        for (int c = 0; c < C; ++c) mass += s.x_total[c];
      token = S.draw_few(n, k, p, qw, u, mass, &z);
      if (token >= 0 && threadIdx.x == 0)
        result(token, Part<T>::one((const T*)a.logits + (size_t)row * a.ld + token), z);
    }
    cl.sync();   // the first CTA's count is read, and its tokens are, before either changes
    if (!by_mass && n <= FEW) return;
    if (by_mass) {
      if (cta == 0 && threadIdx.x < C) *cl.map_shared_rank(&s.few, threadIdx.x) = token >= 0;
      cl.sync();
      if (s.few) return;
    }
  }

  // the cut in the whole row
  auto all = [](int, float) { return true; };
  Cut cut{0xffffffffu, 0x7fffffff};
  ull h[BPT], before;
  if (k > 0) {
    S.template histogram<false>(all, h);
    S.cross(h, (ull)k, 0ull);
    const uint32_t key = S.template radix<false>(s.bin, (ull)k, s.before, all);
    S.cut_ties(cut, key, (ull)k - s.before, s.at);
  }
  if (p < 1.f) {
    auto in = [&](int i, float x) { return kept(cut, rank_key(x), i); };
    S.template histogram<true>(in, h);
    ull t = 0;
#pragma unroll
    for (int j = 0; j < BPT; ++j) t += h[j];
    S.block_total(t);
    const ull need = top_p_mass(p, s.total);
    S.cross(h, need, 0ull);
    const uint32_t key = S.template radix<true>(s.bin, need, s.before, in);
    const ull w = weight(S.sc, s.tab, rank_val(key));
    S.cut_ties(cut, key, (need - s.before + w - 1) / w, s.at / w);
  }
  auto mass = [&](int i, float x) {
    if (!kept(cut, rank_key(x), i)) return 0ull;
    const ull w = weight(S.sc, s.tab, x);
    return w < qw ? 0ull : w;
  };
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

template <typename T>
int launch_sample(const SampleArgs& a, int pdl, cudaStream_t st) {
  int C = 1;
  while (C < MAX_C && (long long)C * 8192 < a.V) C *= 2;
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
}

}  // namespace

void setup_sample_attributes() {
  set_attributes<float>();
  set_attributes<__nv_bfloat16>();
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
