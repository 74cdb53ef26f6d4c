// sample.cu -- one token per row of logits with temperature, top-k, top-p,
// min-p and a given uniform number, and the sampled accept of drafts.
//
// The pages speculate greedily; a served request brings sampling settings of
// its own. For a row of logits l with maximum m the weights are
// w_i = exp((l_i - m) / T); the filters keep a prefix of the order (logit
// descending, index ascending), so together they are ONE cut (key, index) of
// that order: top-k cuts at its k-th token, top-p at the first token whose
// preceding mass reaches p times the top-k mass, min-p at w = min_p. The token
// is the lowest index at which the kept mass, summed in index order, exceeds
// u times the kept mass.
//
// A draft is a single proposed token (the drafter's distribution is a point
// mass), so accepting it when the target's sample equals it IS rejection
// sampling: it is kept with probability p(d), and a rejected position emits a
// token distributed as p without d.
//
// Weights are integers: w_i in units of 2^-40 of the largest (a rounding:
// tokens below 2^-41 of the most likely one count as zero). Their sums are
// exact, so the cut and the token do not depend on the order of the additions,
// the number of CTAs or the other rows of the batch. The weight itself is
// evaluated to about 2^-33 (the exponent as a float pair), because a token is
// decided by a sum of up to V weights next to a border: at the 2^-24 of plain
// floats about one token in 10^4 would differ from the 64-bit definition.
#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace spec {

namespace {

typedef unsigned long long ull;

constexpr int NT = 1024;            // threads of a CTA
constexpr int NW = NT / 32;
constexpr int BINS = 2048;          // bins of a selection level (11 bits of the key)
constexpr int WBITS = 40;           // fraction bits of a weight
constexpr int TAB = 256;            // 2^(-j/256)
constexpr int MAX_C = 8;            // CTAs on one row (a thread-block cluster)

// 2^(40 - j/256), from the exponential series at compile time.
struct Table {
  ull v[TAB];
};
constexpr double series_exp(double x) {
  double s = 1.0, t = 1.0;
  for (int i = 1; i < 30; ++i) {
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
  ull mass[BINS];
  unsigned int count[BINS];
  ull wsum[NW];
  ull total;                 // this CTA's sum, read by the cluster
  ull best;                  // this CTA's packed maximum, read by the cluster
  int nan;
  int bin;                   // crossing bin of a selection level
  ull before, at;            // amount before it, and in it
  int found;                 // index found by find_in_order, written by its owner
  float sh, sl, lq;          // log2(e) / T as a float pair, T * ln(min_p)
  double lqd;
};

// Scale of a row: weights are 2^-((m - x) * (sh + sl)).
struct Scale {
  float m, sh, sl;
};

// The weight of logit x as a float pair (value hi + lo in units of 2^(40-n)).
// z = (m - x) * s is formed as a float pair (an exact difference, an exact
// product), split into n + j/256 + g, and 2^-z = 2^-n * tab[j] * e^(-g ln 2)
// with a cubic (Tang's table-driven reduction, ACM TOMS 15(2), 1989).
SPEC_DEV ull weight(const Scale& r, const ull* tab, float x, float* val = nullptr) {
  if (r.m == INFINITY) {
    if (val) *val = x == INFINITY ? 1.f : 0.f;
    return x == INFINITY ? 1ull << WBITS : 0ull;
  }
  const float d = r.m - x;
  const float bb = d - r.m;
  const float e = (r.m - (d - bb)) + (-x - bb);   // d + e == m - x
  float p = d * r.sh;
  const float pe = fmaf(e, r.sh, fmaf(d, r.sl, fmaf(d, r.sh, -p)));
  p = fminf(p, 63.f);
  const float t = fmaf(p, (float)TAB, 12582912.f);  // round(256 p) in the low bits
  const int j = __float_as_int(t) & 0x3fffff;
  const float g = fmaf(t - 12582912.f, -1.f / TAB, p) + pe;
  const float h = g * -0.693147181f;
  const float q = fmaf(fmaf(h, 0.16666667f, 0.5f) * h, h, h);  // e^h - 1, |h| < 0.0014
  const ull T = tab[j & (TAB - 1)];
  const int n = j >> 8;
  const float Tf = (float)T;
  if (val) *val = n > 125 ? 0.f : (Tf + Tf * q) * __int_as_float((127 - WBITS - n) << 23);
  const ull v = T + (long long)__float2int_rn(Tf * q);
  return (v + ((1ull << n) >> 1)) >> n;
}

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
  SPEC_DEV void vec(int v, F f) const {
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
    for (int v = v0 + (int)(threadIdx.x & 31); v < v1; v += 32) vec(v, f);
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

  // Sum of f(index, value) over the row; wsum holds the warps' parts, and
  // `before` gets the sum of the cluster's earlier CTAs.
  template <typename F>
  SPEC_DEV ull sum(F f, ull* before) {
    ull a = 0;
    part.each([&](int i, float x) { a += f(i, x); });
    a = warp_sum_u64(a);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.wsum[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x < 32) {
      const ull t = warp_sum_u64(s.wsum[threadIdx.x]);
      if (threadIdx.x == 0) s.total = t;
    }
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

  // The lowest index at which the sum of f in index order exceeds t (t below
  // the row's sum, wsum and before as left by sum()). Every CTA gets it.
  template <typename F>
  SPEC_DEV int find_in_order(F f, ull t, ull before) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    ull b = before;
    for (int i = 0; i < w; ++i) b += s.wsum[i];
    if (t >= b && t < b + s.wsum[w]) {
      for (int v = part.v0 + lane; v - lane < part.v1; v += 32) {
        ull a = 0;
        if (v < part.v1) part.vec(v, [&](int i, float x) { a += f(i, x); });
        const ull inc = warp_scan_u64(a);
        const ull tot = __shfl_sync(FULL, inc, 31);
        if (t < b + tot) {
          ull c = b + inc - a;
          if (t >= c && t < c + a) {
            int hit = -1;
            part.vec(v, [&](int i, float x) {
              c += f(i, x);
              if (hit < 0 && t < c) hit = i;
            });
            for (int r = 0; r < C; ++r) *cl.map_shared_rank(&s.found, r) = hit;
          }
          break;
        }
        b += tot;
      }
    }
    cl.sync();
    const int found = s.found;
    cl.sync();
    return found;
  }

  // The key at which the amount (count or mass) in order first reaches
  // `need` >= 1: three levels of 11, 11 and 10 bits, each a histogram of the
  // keys that share the prefix found so far. Returns the key; s.before: amount
  // strictly before it, s.at: amount of the tokens with it.
  template <bool MASS, typename F>
  SPEC_DEV uint32_t select(ull need, F amount) {
    uint32_t pre = 0;
    ull before = 0;
#pragma unroll
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
      const int bits = level == 2 ? 10 : 11;
      for (int i = threadIdx.x; i < BINS; i += NT) {
        if (MASS) s.mass[i] = 0ull;
        else s.count[i] = 0u;
      }
      __syncthreads();
      part.each([&](int i, float x) {
        const uint32_t k = rank_key(x);
        if (level > 0 && (k >> (shift + bits)) != pre) return;
        const ull a = amount(i, x, k);
        if (!a) return;
        const int b = (k >> shift) & ((1 << bits) - 1);
        if (MASS) atomicAdd(&s.mass[b], a);
        else atomicAdd(&s.count[b], 1u);
      });
      cl.sync();
      ull h[2] = {0, 0};
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          h[j] += MASS ? cl.map_shared_rank(s.mass, c)[threadIdx.x * 2 + j]
                       : (ull)cl.map_shared_rank(s.count, c)[threadIdx.x * 2 + j];
      const ull inc = warp_scan_u64(h[0] + h[1]);
      if ((threadIdx.x & 31) == 31) s.wsum[threadIdx.x >> 5] = inc;
      __syncthreads();
      ull b = before + inc - h[0] - h[1];
      for (int i = 0; i < (int)(threadIdx.x >> 5); ++i) b += s.wsum[i];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (b < need && need <= b + h[j]) {
          s.bin = threadIdx.x * 2 + j;
          s.before = b;
          s.at = h[j];
        }
        b += h[j];
      }
      cl.sync();  // the histogram is read everywhere before it is cleared again
      pre = (pre << bits) | (uint32_t)s.bin;
      before = s.before;
    }
    return pre;
  }
};

template <typename T>
__global__ void __launch_bounds__(NT, 1) sample_kernel(SampleArgs a) {
  __shared__ Shared s;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), cta = (int)cl.block_rank(), row = blockIdx.x / C;
  for (int i = threadIdx.x; i < TAB; i += NT) s.tab[i] = g_table.v[i];
  Sampler<T> S{s, cl, cta, C};
  grid_dep_wait();
  const float temp = a.temperature ? a.temperature[row] : 1.f;
  const int k = a.top_k ? a.top_k[row] : 0;
  const float p = a.top_p ? a.top_p[row] : 1.f;
  const float q = a.min_p ? fminf(a.min_p[row], 1.f) : 0.f;
  const float u = a.uniform[row];
  S.part.bind((const T*)a.logits + (size_t)row * a.ld, a.V, cta, C);
  const bool greedy = temp < 1e-5f;
  if (threadIdx.x == 0 && !greedy) {
    const double r = 1.4426950408889634 / (double)temp;
    s.sh = (float)r;
    s.sl = (float)(r - (double)s.sh);
    s.lqd = q > 0.f ? (double)temp * log((double)q) : 0.0;
  }

  // maximum and its lowest index; a NaN anywhere leaves the row without a distribution
  ull best = 0;
  int nan = 0;
  {
    float bx = -INFINITY;
    int bi = -1;
    S.part.each([&](int i, float x) {
      nan |= x != x;
      if (x > bx) {
        bx = x;
        bi = i;
      }
    });
    if (bi >= 0) best = pack_best(bx + 0.f, (uint32_t)bi);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const ull other = __shfl_xor_sync(FULL, best, o);
    best = other > best ? other : best;
  }
  if ((threadIdx.x & 31) == 0) s.wsum[threadIdx.x >> 5] = best;
  nan = __syncthreads_or(nan);
  if (threadIdx.x == 0) {
    for (int i = 0; i < NW; ++i) best = s.wsum[i] > best ? s.wsum[i] : best;
    s.best = best;
    s.nan = nan;
  }
  cl.sync();
  best = 0;
  nan = 0;
  for (int c = 0; c < C; ++c) {
    const ull o = *cl.map_shared_rank(&s.best, c);
    best = o > best ? o : best;
    nan |= *cl.map_shared_rank(&s.nan, c);
  }
  cl.sync();

  int token = -1;
  float prob = 0.f;
  const bool ok = best != 0ull && !nan && temp >= 0.f && temp < INFINITY;  // else: no distribution
  if (ok && greedy) {
    token = (int)best_index(best);
    prob = 1.f;
  } else if (ok) {
    const float m = best_value(best);
    const Scale sc{m, s.sh, s.sl};
    const ull* tab = s.tab;
    Cut cut{0xffffffffu, 0x7fffffff};
    ull before;
    if (k > 0 && k < a.V) {
      const uint32_t key = S.template select<false>((ull)k, [](int, float, uint32_t) { return 1ull; });
      const ull r = (ull)k - s.before;   // tokens of this key that stay
      cut.key = key;
      if (r < s.at) {
        auto eq = [&](int, float x) { return rank_key(x) == key ? 1ull : 0ull; };
        __syncthreads();
        S.sum(eq, &before);
        cut.idx = S.find_in_order(eq, r - 1, before);
      }
    }
    if (p < 1.f) {
      auto mass = [&](int i, float x) { return kept(cut, rank_key(x), i) ? weight(sc, tab, x) : 0ull; };
      const ull z1 = S.sum(mass, &before);
      ull need = (ull)ceil((double)fmaxf(p, 0.f) * (double)z1);
      need = need < 1 ? 1 : need > z1 ? z1 : need;
      const uint32_t key = S.template select<true>(
          need, [&](int i, float x, uint32_t kx) { return kept(cut, kx, i) ? weight(sc, tab, x) : 0ull; });
      const ull w = weight(sc, tab, rank_val(key));
      const ull r = (need - s.before + w - 1) / w;   // tokens of this key that stay
      auto eq = [&](int i, float x) { return rank_key(x) == key && kept(cut, key, i) ? 1ull : 0ull; };
      if (r * w < s.at) {
        __syncthreads();
        S.sum(eq, &before);
        cut.idx = S.find_in_order(eq, r - 1, before);
      } else if (key < cut.key) {
        cut.idx = 0x7fffffff;
      }
      cut.key = key;
    }
    if (q > 0.f) {
      const uint32_t key = rank_key(__double2float_ru((double)m + s.lqd));
      if (key < cut.key) cut = Cut{key, 0x7fffffff};
    }
    auto mass = [&](int i, float x) { return kept(cut, rank_key(x), i) ? weight(sc, tab, x) : 0ull; };
    const ull z = S.sum(mass, &before);
    ull t = u > 0.f ? (ull)((double)u * (double)z) : 0ull;
    t = t < z ? t : z - 1;
    token = S.find_in_order(mass, t, before);
    if (cta == 0 && threadIdx.x == 0) {
      const T* lr = (const T*)a.logits + (size_t)row * a.ld;
      float v;
      weight(sc, tab, Part<T>::one(lr + token), &v);
      prob = v / ((float)z * (1.f / (float)(1ull << WBITS)));
    }
  }
  if (cta == 0 && threadIdx.x == 0) {
    a.tokens[row] = token;
    if (a.probs) a.probs[row] = prob;
  }
  cl.sync();  // no CTA leaves while another may still read its shared memory
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

}  // namespace

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
