// adjust.cu -- penalties for repeated tokens, biases and grammar masks on the
// logits of a pass, before they are sampled.
//
// Row r of sequence b follows the sequence's history and the tokens of the
// rows on r's path. For a token that occurs there c times as output, with the
// sequence's settings: x > 0 becomes x / repetition, other x x * repetition, if
// the token occurs at all (in the prompt too); then x - c * frequency
// - (c > 0) * presence + bias. Forbidden tokens get -inf. All in fp32, rounded
// once.
//
// Bound by HBM: every logit is read and written once. A CTA takes a chunk of
// the vocabulary for some rows of a sequence (all of them where that makes enough
// CTAs) and keeps one word a token of it in shared memory, counted once from the
// history, so a row costs its tokens' words (few are not zero: the other logits pass through)
// and a step costs no table of [rows][V] in memory. Rows differ by a few tokens of
// their paths; they are counted in and out between rows. The logits are on their
// way while the words are counted.
#include <algorithm>

#include "common.cuh"

namespace spec {
namespace {

constexpr int NTHR = 256;
constexpr int K = 4;            // vectors of a row in a thread's hands at a time
// A token's word: times it occurs as output (19 bits), occurs at all, place of its bias in the list + 1 (12 bits).
constexpr uint32_t COUNT = (1u << 19) - 1, SEEN = 1u << 19;
constexpr int BIAS_AT = 20;

struct Rules {
  float rep, freq, pres;
  const float* bias;
};

SPEC_DEV float adjusted(float x, uint32_t w, const Rules& k) {
  if (x == -INFINITY) return x;  // (also where a reward is infinite)
  if (w & (COUNT | SEEN)) {
    x = x > 0.f ? __fdiv_rn(x, k.rep) : x * k.rep;
    const uint32_t c = w & COUNT;
    if (c) x = x - (float)c * k.freq - k.pres;
  }
  if (w >> BIAS_AT) {
    const float b = k.bias[(w >> BIAS_AT) - 1];
    x = b == -INFINITY || x == -INFINITY ? -INFINITY : isnan(b) ? x : x + b;
  }
  return x;
}

template <typename T>
struct Vec;  // a 16-byte vector of logits
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static SPEC_DEV float get(const uint4& v, int i) { return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w); }
  static SPEC_DEV void pack(uint4& v, const float* f) {
    v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
SPEC_DEV uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static SPEC_DEV float get(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return i & 1 ? bf16hi(w) : bf16lo(w);
  }
  static SPEC_DEV void pack(uint4& v, const float* f) {
    v = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
};
SPEC_DEV float value(float x) { return x; }
SPEC_DEV float value(__nv_bfloat16 x) { return __bfloat162float(x); }
SPEC_DEV void put(float* p, float v) { *p = v; }
SPEC_DEV void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

SPEC_DEV float setting(const float* p, int b, float off, bool positive) {
  const float v = p ? p[b] : off;
  return isfinite(v) && (!positive || v > 0.f) ? v : off;
}

// The 16 bytes at byte offset `at` of a row whose start lies `mis` bytes behind
// a 16-byte boundary: two aligned loads joined (the second only where the row
// has bytes in it).
SPEC_DEV uint4 load_shifted(const char* row, long long at, int mis, long long bytes) {
  const char* p = row + at - mis;
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  if (mis == 0) return a;
  uint4 b = make_uint4(0, 0, 0, 0);
  if (at - mis + 16 < bytes) b = *reinterpret_cast<const uint4*>(p + 16);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t r[4];
  const int word = mis >> 2, bits = (mis & 3) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // (word is the same for all threads)
      if (word == j) {
        lo = w[i + j];
        hi = i + j + 1 < 8 ? w[i + j + 1] : 0;
      }
    }
    r[i] = __funnelshift_r(lo, hi, bits);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// What a CTA's rows share: the sequence's settings, and the words of the chunk.
struct Words {
  const AdjustArgs& a;
  uint32_t *tab, *mark;          // [chunk]; a bit for each word that is, or was, not zero
  unsigned long long* path;      // [64]
  int b, c0, nc, r0, r1;
  size_t m0;
  Rules k;
  bool count, use, bad;          // penalties, any words at all; something out of range

  int n_hist, n_prompt;          // tokens of the history, of its prompt

  SPEC_DEV Words(const AdjustArgs& a, uint32_t* tab, unsigned long long* path)
      : a(a), tab(tab), mark(tab + a.chunk), path(path), b(blockIdx.y), bad(false) {
    c0 = blockIdx.x * a.chunk;
    nc = min(a.chunk, a.V - c0);
    r0 = blockIdx.z * a.rows;
    r1 = min(r0 + a.rows, a.R);
    m0 = (size_t)b * a.R;
    k.rep = setting(a.repetition, b, 1.f, true);
    k.freq = setting(a.frequency, b, 0.f, false);
    k.pres = setting(a.presence, b, 0.f, false);
    k.bias = a.bias_values + (size_t)b * a.n_bias;
    count = k.rep != 1.f || k.freq != 0.f || k.pres != 0.f;
    use = count || a.n_bias > 0;
    n_hist = a.hist_len ? a.hist_len[b] : a.n_history;
    n_prompt = a.prompt_len ? a.prompt_len[b] : 0;
    bad = a.history && count && (n_hist < 0 || n_hist > a.n_history || n_prompt < 0 || n_prompt > n_hist);
    n_hist = min(max(n_hist, 0), a.n_history);
  }
  SPEC_DEV void check() {
    if (!a.status || blockIdx.x || blockIdx.z) return;
    if (a.parents && a.tokens && count)
      for (int r = threadIdx.x; r < a.R; r += NTHR) {
        const int p = a.parents[m0 + r];
        bad |= p < -1 || p >= r;
      }
  }
  SPEC_DEV void note(unsigned at, uint32_t old) const {
    if (!old) atomicOr(&mark[at >> 5], 1u << (at & 31));
  }
  SPEC_DEV void add(int token, uint32_t by) const {
    const unsigned at = (unsigned)(token - c0);
    if (token >= 0 && at < (unsigned)nc) note(at, atomicAdd(&tab[at], by));
  }
  SPEC_DEV void build() {
    const int t = threadIdx.x;
    if (!use) return;
    // (the marks lie behind the words)
    for (int i = t; i < (a.chunk + a.chunk / 32) / 4; i += NTHR) reinterpret_cast<uint4*>(tab)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (a.n_bias > 0) {
      const int32_t* list = a.bias_tokens + (size_t)b * a.n_bias;
      for (int i = t; i < a.n_bias; i += NTHR) {
        const unsigned at = (unsigned)(list[i] - c0);
        // the last of several entries for a token counts
        if (at < (unsigned)nc) note(at, atomicMax(&tab[at], (uint32_t)(i + 1) << BIAS_AT));
      }
      __syncthreads();
    }
    if (!count) return;
    if (a.history) {
      const int32_t* h = a.history + (size_t)b * a.ld_history;
      constexpr int U = 8;
      for (int i = t; i < n_hist; i += U * NTHR) {
        int tok[U];
#pragma unroll
        for (int j = 0; j < U; ++j) tok[j] = i + j * NTHR < n_hist ? h[i + j * NTHR] : -1;
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const unsigned at = (unsigned)(tok[j] - c0);
          if (tok[j] >= 0 && at < (unsigned)nc) {
            note(at, i + j * NTHR < n_prompt ? atomicOr(&tab[at], SEEN) : atomicAdd(&tab[at], 1u));
          }
        }
      }
    }
    if (a.tokens && a.parents) {
      // a row's path as bits (a parent that is not an earlier row counts as none)
      if (t < TREE_ROWS_MAX) {
        unsigned long long m = 0;
        if (t < r1)
          for (int r = t; r >= 0;) {
            m |= 1ull << r;
            const int p = a.parents[m0 + r];
            r = p < r ? p : -1;
          }
        path[t] = m;
      }
    } else if (a.tokens) {
      for (int r = t; r < r0; r += NTHR) add(a.tokens[m0 + r], 1u);  // (a chain's rows before this CTA's first)
    }
    __syncthreads();
  }
  // From row r - 1's words (or those of no row) to row r's. Between barriers: the
  // words of the row before are done with, those of this one are ready.
  SPEC_DEV void to_row(int r) const {
    if (!count || !a.tokens) return;
    if (r > r0) __syncthreads();
    if (a.parents) {
      const unsigned long long now = path[r], was = r > r0 ? path[r - 1] : 0ull;
      const int t = threadIdx.x;
      if (t < a.R && ((now ^ was) >> t) & 1) add(a.tokens[m0 + t], (now >> t) & 1 ? 1u : ~0u);
    } else if (threadIdx.x == 0) {
      add(a.tokens[m0 + r], 1u);
    }
    __syncthreads();
  }
  // Row r's bits of this chunk (chunks start on words), or null.
  SPEC_DEV const uint32_t* mask_of(int r) {
    if (!a.mask) return nullptr;
    const int id = a.mask_ids ? a.mask_ids[m0 + r] : (int)(m0 + r);
    const bool ok = id >= -1 && id < a.n_masks;
    bad |= !ok;
    return ok && id >= 0 ? a.mask + (size_t)id * a.ld_mask + (c0 >> 5) : nullptr;
  }
  // What is forbidden of N logits from i on, as bits.
  template <int N>
  static SPEC_DEV uint32_t banned(const uint32_t* bits, int i) {
    return ~bits[i >> 5] >> (i & 31) & ((1u << N) - 1);
  }
  template <typename T>
  static SPEC_DEV void ban(uint4& v, uint32_t which) {
    using V = Vec<T>;
    float f[V::N];
#pragma unroll
    for (int e = 0; e < V::N; ++e) f[e] = (which >> e) & 1 ? -INFINITY : V::get(v, e);
    V::pack(v, f);
  }
  // In place: the forbidden of a row's n logits set, so that the others are neither read
  // nor written. A warp takes g <= 32 words of the mask at a time, those w, w + 1, ...,
  // then `step` further on; a word's tokens are a lane each.
  template <typename T>
  static SPEC_DEV void forbid(T* row, const uint32_t* bits, int n, int w, int step, int g) {
    const int lane = threadIdx.x & 31, words = (n + 31) / 32;
    for (; w < words; w += step) {
      const uint32_t mine = lane < g && w + lane < words ? ~bits[w + lane] : 0u;
      for (uint32_t some = __ballot_sync(FULL, mine != 0); some; some &= some - 1) {
        const int j = __ffs(some) - 1, i = 32 * (w + j) + lane;
        if ((__shfl_sync(FULL, mine, j) >> lane) & 1 && i < n) put(row + i, -INFINITY);
      }
    }
  }
  // f(i, word) for the words of [i0, i1) that are not zero (i0 a multiple of 16): 16
  // marks a thread. Few tokens of a vocabulary occur in a text, so a pass over the
  // marks costs less than a look at every word beside its logit, where one in 32
  // sends the whole warp through the arithmetic.
  template <class F>
  SPEC_DEV void each_word(int i0, int i1, F f) const {
    if (!use) return;
    for (int h = i0 / 16 + threadIdx.x; 16 * h < i1; h += NTHR)
      for (uint32_t m = mark[h >> 1] >> (16 * (h & 1)) & 0xffffu; m; m &= m - 1) {
        const int i = 16 * h + __ffs(m) - 1;
        const uint32_t w = tab[i];
        if (w && i < i1) f(i, w);
      }
  }
  // Logits [i0, nc) of row r, one a thread and turn.
  template <typename T>
  SPEC_DEV void singles(int r, int i0, const uint32_t* bits) const {
    const T* src = (const T*)a.logits + (m0 + r) * a.ld + c0;
    T* dst = (T*)a.out + (m0 + r) * a.ld_out + c0;
    for (int i = i0 + threadIdx.x; i < nc; i += NTHR) {
      const uint32_t w = use ? tab[i] : 0u;
      const bool ban = bits && !((bits[i >> 5] >> (i & 31)) & 1);
      float x = value(src[i]);
      if (w) x = adjusted(x, w, k);
      put(dst + i, ban ? -INFINITY : x);
    }
  }
  SPEC_DEV void done() const {
    if (a.status && bad) atomicCAS(a.status, 0, (int)SPEC_ERR_CAPACITY);
  }
};

// Small calls, long histories and many rows: all in one kernel. VEC: the output's
// rows start on 16-byte boundaries. SAME: in place, so what stays as it is is
// neither read nor written. The logits are copied first, what is forbidden set, four
// vectors in a thread's hands and the next four on the way (the first while the words
// are counted); then the tokens with words.
template <typename T, bool VEC, bool SAME>
__global__ void __launch_bounds__(NTHR, 4) adjust_kernel(const __grid_constant__ AdjustArgs a) {
  using V = Vec<T>;
  extern __shared__ __align__(16) uint32_t tab[];  // [chunk + chunk / 32]
  __shared__ unsigned long long path[TREE_ROWS_MAX];
  const int t = threadIdx.x;
  Words w(a, tab, path);
  // the rows' vectors, K a thread and turn: `turns` turns a row
  const int nv = VEC ? w.nc / V::N : 0, turns = (nv + K * NTHR - 1) / (K * NTHR);
  uint4 next[K];
  auto fetch = [&](int r, int turn) {
    const char* src = (const char*)((const T*)a.logits + (w.m0 + r) * a.ld + w.c0);
    const int mis = (int)((uintptr_t)src & 15);
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const int i = (turn * K + u) * NTHR + t;
      if (i < nv) next[u] = load_shifted(src, (long long)i * 16, mis, (long long)w.nc * sizeof(T));
    }
  };
  if (VEC && !SAME) fetch(w.r0, 0);
  w.check();
  w.build();
  for (int r = w.r0; r < w.r1; ++r) {
    w.to_row(r);
    const uint32_t* bits = w.mask_of(r);
    const T* src = (const T*)a.logits + (w.m0 + r) * a.ld + w.c0;
    T* dst = (T*)a.out + (w.m0 + r) * a.ld_out + w.c0;
    auto change = [&](int i, uint32_t word) {
      if (!bits || (bits[i >> 5] >> (i & 31)) & 1) put(dst + i, adjusted(value(src[i]), word, w.k));
    };
    if constexpr (SAME) {
      if (bits) {  // (chunks have 32 words and more: all warps have some)
        const int g = min(32, a.chunk / NTHR);
        Words::forbid(dst, bits, w.nc, (t >> 5) * g, NTHR / 32 * g, g);
      }
      w.each_word(0, w.nc, change);
      continue;
    }
    for (int turn = 0; turn < turns; ++turn) {
      uint4 v[K];
      uint32_t which[K];
#pragma unroll
      for (int u = 0; u < K; ++u) {
        const int i = (turn * K + u) * NTHR + t;
        which[u] = bits && i < nv ? w.template banned<V::N>(bits, i * V::N) : 0u;
        v[u] = next[u];
      }
      if (turn + 1 < turns) fetch(r, turn + 1);
      else if (r + 1 < w.r1) fetch(r + 1, 0);
#pragma unroll
      for (int u = 0; u < K; ++u) {
        const int i = (turn * K + u) * NTHR + t;
        if (which[u]) w.template ban<T>(v[u], which[u]);
        if (i < nv) __stcs(reinterpret_cast<uint4*>(dst) + i, v[u]);
      }
    }
    w.template singles<T>(r, nv * V::N, bits);
    if (nv && w.use) {
      __syncthreads();  // (their copies are stored)
      w.each_word(0, nv * V::N, change);
    }
  }
  w.done();
}

// Large calls take two kernels. The first copies the logits and sets what is
// forbidden: lines of 256 vectors, four of them on the way in each of five CTAs an
// SM, every CTA the same number.
constexpr int COPY_CTAS = 5;
template <typename T, bool VEC>
__global__ void __launch_bounds__(NTHR, 8) adjust_copy_kernel(const __grid_constant__ AdjustArgs a) {
  using V = Vec<T>;
  constexpr int N = VEC ? V::N : 1;
  grid_dep_launch();
  const int t = threadIdx.x, nv = a.V / N, per = (nv + NTHR - 1) / NTHR;  // vectors and lines of a row
  const int lines = per * a.B * a.R;
  bool bad = false;
  for (int l0 = blockIdx.x; l0 < lines; l0 += K * gridDim.x) {
    uint4 v[K];
    uint32_t ban[K];
    int at[K], row[K];
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const int l = l0 + u * gridDim.x;
      row[u] = l / per;
      at[u] = (l - row[u] * per) * NTHR + t;
      if (l >= lines) at[u] = nv;
      ban[u] = 0;
      if (at[u] >= nv) continue;
      if (a.mask) {
        const int id = a.mask_ids ? a.mask_ids[row[u]] : row[u];
        bad |= id < -1 || id >= a.n_masks;
        if (id >= 0 && id < a.n_masks)
          ban[u] = ~a.mask[(size_t)id * a.ld_mask + ((at[u] * N) >> 5)] >> ((at[u] * N) & 31) & ((1u << N) - 1);
      }
      const char* src = (const char*)((const T*)a.logits + (size_t)row[u] * a.ld);
      if constexpr (VEC) v[u] = load_shifted(src, (long long)at[u] * 16, (int)((uintptr_t)src & 15), (long long)a.V * sizeof(T));
      else v[u].x = sizeof(T) == 4 ? reinterpret_cast<const uint32_t*>(src)[at[u]] : reinterpret_cast<const uint16_t*>(src)[at[u]];
    }
#pragma unroll
    for (int u = 0; u < K; ++u) {
      if (at[u] >= nv) continue;
      T* dst = (T*)a.out + (size_t)row[u] * a.ld_out;
      if constexpr (VEC) {
        if (ban[u]) Words::ban<T>(v[u], ban[u]);
        __stcs(reinterpret_cast<uint4*>(dst) + at[u], v[u]);
      } else if (ban[u]) {
        put(dst + at[u], -INFINITY);
      } else if (sizeof(T) == 4) {
        reinterpret_cast<uint32_t*>(dst)[at[u]] = v[u].x;
      } else {
        reinterpret_cast<uint16_t*>(dst)[at[u]] = (uint16_t)v[u].x;
      }
    }
  }
  if constexpr (VEC) {  // the rows' ends, less than a vector each
    const int rest = a.V - nv * N;
    for (int i = blockIdx.x * NTHR + t; i < rest * a.B * a.R; i += gridDim.x * NTHR) {
      const int r = i / rest, c = nv * N + i - r * rest;
      bool ban = false;
      if (a.mask) {
        const int id = a.mask_ids ? a.mask_ids[r] : r;
        bad |= id < -1 || id >= a.n_masks;
        ban = id >= 0 && id < a.n_masks && !((a.mask[(size_t)id * a.ld_mask + (c >> 5)] >> (c & 31)) & 1);
      }
      put((T*)a.out + (size_t)r * a.ld_out + c, ban ? -INFINITY : value(((const T*)a.logits)[(size_t)r * a.ld + c]));
    }
  }
  if (a.status && bad) atomicCAS(a.status, 0, (int)SPEC_ERR_CAPACITY);
}

// In place, the first kernel sets what is forbidden and does no more: FW words of a
// row's mask a CTA and turn. Bound by the stores, 2 or 4 bytes a lane in whole lines:
// 40 fp32 rows of 262144 with three quarters of the tokens forbidden take 10.5 us, with two
// in a thousand 3.9; 64 bf16 rows 15.7 and 5.1 (whole vectors read, changed and written
// back took 13.7, 9.6, 11.8 and 8.7, but touched what stays as it is).
constexpr int FW = 16 * NTHR / 32;
template <typename T>
__global__ void __launch_bounds__(NTHR, 8) adjust_forbid_kernel(const __grid_constant__ AdjustArgs a) {
  grid_dep_launch();
  const int words = (a.V + 31) / 32, per = (words + FW - 1) / FW;
  bool bad = false;
  for (int l = blockIdx.x; l < per * a.B * a.R; l += gridDim.x) {
    const int r = l / per, w0 = (l - r * per) * FW, id = a.mask_ids ? a.mask_ids[r] : r;
    bad |= id < -1 || id >= a.n_masks;
    if (id >= 0 && id < a.n_masks)
      Words::forbid((T*)a.out + (size_t)r * a.ld_out + 32 * w0, a.mask + (size_t)id * a.ld_mask + w0, min(32 * FW, a.V - 32 * w0),
                    16 * (threadIdx.x >> 5), FW, 16);
  }
  if (a.status && bad) atomicCAS(a.status, 0, (int)SPEC_ERR_CAPACITY);
}

// The second one, started beside it, counts a sequence's tokens in a hash table in
// shared memory (a.parts CTAs a sequence, each for a share of the tokens), works out
// what their logits become, and writes that over the copies when those are stored.
// The table has room for every token of the history, pass and list. The loops are
// rolled and the tokens of a CTA's share are queued before they are counted: what
// runs once pays for its instructions (20 to 40 cycles each out of cold caches: with
// eight tokens unrolled the kernel took 17 us for 8 x 5 rows, 15 now), and a warp that
// counts for one lane waits as long as for all.
constexpr int HASH_MAX = 16384;  // slots; three quarters of them at most are used
constexpr int WTHR = 512;        // (beside the copy's registers an SM has room for one such CTA of 48 a thread)
constexpr int SCAN = 4;          // tokens a thread and round
constexpr int HELD = 2048;       // results held while the copy runs
constexpr uint32_t NONE = 0xffffdeadu;  // (a result that is NaN is another)
struct Hash {
  uint32_t *key, *word;          // [slots]: token (bit 31: fed in this pass), its word; EMPTY
  uint16_t* list;                // [slots * 3 / 4] slots in use
  int* n;
  uint32_t mask;
  static constexpr uint32_t EMPTY = 0x7fffffffu, FED = 0x80000000u;
  SPEC_DEV uint32_t slot(uint32_t token) const {
    uint32_t s = token * 0x9E3779B1u >> 15 & mask;
    for (;;) {
      const uint32_t k = atomicCAS(&key[s], EMPTY, token);
      if (k == EMPTY) list[atomicAdd(n, 1)] = (uint16_t)s;
      if (k == EMPTY || (k & ~FED) == token) return s;
      s = (s + 1) & mask;
    }
  }
};

template <typename T>
__global__ void __maxnreg__(48) adjust_words_kernel(const __grid_constant__ AdjustArgs a) {
  extern __shared__ __align__(16) uint32_t sm[];  // keys, words, list
  __shared__ unsigned long long path[TREE_ROWS_MAX];
  __shared__ int fed[TREE_ROWS_MAX], ids[TREE_ROWS_MAX], used, queued;
  __shared__ uint32_t held[HELD];                 // (first the queue: a token, bit 31: of the prompt)
  const int t = threadIdx.x, b = blockIdx.y, part = blockIdx.x, slots = a.slots;
  const size_t m0 = (size_t)b * a.R;
  Hash h{sm, sm + slots, reinterpret_cast<uint16_t*>(sm + 2 * slots), &used, (uint32_t)slots - 1};
  Rules k;
  k.rep = setting(a.repetition, b, 1.f, true);
  k.freq = setting(a.frequency, b, 0.f, false);
  k.pres = setting(a.presence, b, 0.f, false);
  k.bias = a.bias_values + (size_t)b * a.n_bias;
  const bool count = k.rep != 1.f || k.freq != 0.f || k.pres != 0.f;
  int n = a.hist_len ? a.hist_len[b] : a.n_history;
  const int np = a.prompt_len ? a.prompt_len[b] : 0;
  bool bad = a.history && count && (n < 0 || n > a.n_history || np < 0 || np > n);
  n = a.history && count ? min(max(n, 0), a.n_history) : 0;
  const int R = a.tokens && count ? a.R : 0;
  for (int i = t; i < slots / 4; i += WTHR) {
    reinterpret_cast<uint4*>(h.key)[i] = make_uint4(Hash::EMPTY, Hash::EMPTY, Hash::EMPTY, Hash::EMPTY);
    reinterpret_cast<uint4*>(h.word)[i] = make_uint4(0, 0, 0, 0);
  }
  if (t == 0) used = queued = 0;
  if (t < a.R) {
    unsigned long long m = 0;
    for (int r = t; r >= 0;) {  // (a parent that is not an earlier row counts as none)
      m |= 1ull << r;
      const int p = a.parents ? a.parents[m0 + r] : r - 1;
      bad |= R > 0 && (p < -1 || p >= r);
      r = p < r ? p : -1;
    }
    path[t] = m;
    fed[t] = -1;
    // (forbidden stays forbidden; ids out of range are recorded by the copy)
    const int id = a.mask ? (a.mask_ids ? a.mask_ids[m0 + t] : (int)(m0 + t)) : -1;
    ids[t] = id < a.n_masks ? id : -1;
  }
  __syncthreads();
  auto mine = [&](int token) {
    return (unsigned)token < (unsigned)a.V && (int)__umulhi((uint32_t)token * 0x85EBCA6Bu, (uint32_t)a.parts) == part;
  };
  if (a.n_bias > 0) {
    const int32_t* list = a.bias_tokens + (size_t)b * a.n_bias;
    for (int i = t; i < a.n_bias; i += WTHR)  // (the last of several entries for a token counts)
      if (mine(list[i])) atomicMax(&h.word[h.slot(list[i])], (uint32_t)(i + 1) << BIAS_AT);
    __syncthreads();
  }
  const int32_t* hist = a.history + (size_t)b * a.ld_history;
  int tok[SCAN];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int j = 0; j < SCAN; ++j) {
      const int i = i0 + j * WTHR + t;
      tok[j] = i < n ? hist[i] : -1;
    }
  };
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += SCAN * WTHR) {
    static_assert(SCAN * WTHR <= HELD, "");
    if (i0 == 0) fetch(0);
    int c = 0;
#pragma unroll
    for (int j = 0; j < SCAN; ++j) {
      if (!mine(tok[j])) tok[j] = -1;
      c += tok[j] >= 0;
    }
    int at = c ? atomicAdd(&queued, c) : 0;
#pragma unroll
    for (int j = 0; j < SCAN; ++j)
      if (tok[j] >= 0) held[at++] = (uint32_t)tok[j] | (i0 + j * WTHR + t < np ? 0x80000000u : 0u);
    fetch(i0 + SCAN * WTHR);  // (the next round's, while this one's are counted)
    __syncthreads();
    const int q = queued;
    for (int e = t; e < q; e += WTHR) {
      uint32_t* w = &h.word[h.slot(held[e] & 0x7fffffffu)];
      if (held[e] >> 31) atomicOr(w, SEEN);
      else atomicAdd(w, 1u);
    }
    __syncthreads();
    if (t == 0) queued = 0;
    __syncthreads();
  }
  if (t < R) {
    const int token = a.tokens[m0 + t];
    if (mine(token)) {
      fed[t] = h.slot(token);
      atomicOr(&h.key[fed[t]], Hash::FED);
    }
  }
  __syncthreads();
  const int L = used, items = L * a.R;
  const T* in = (const T*)a.logits + m0 * a.ld;
  T* out = (T*)a.out + m0 * a.ld_out;
  for (int base = 0; base == 0 || base < items; base += HELD) {
    const int end = min(base + HELD, items);
    // their logits, four on the way; NONE where the mask forbids the token
#pragma unroll 4
    for (int e = base + t; e < end; e += WTHR) {
      const int r = e / L, token = (int)(h.key[h.list[e - r * L]] & ~Hash::FED), id = ids[r];
      const uint32_t bits = id >= 0 ? a.mask[(size_t)id * a.ld_mask + (token >> 5)] >> (token & 31) : 1u;
      const float f = value(in[(size_t)r * a.ld + token]);
      held[e - base] = bits & 1 ? (isnan(f) ? 0x7fffffffu : __float_as_uint(f)) : NONE;
    }
#pragma unroll 1
    for (int e = base + t; e < end; e += WTHR) {
      const uint32_t x = held[e - base];
      if (x == NONE) continue;
      const int r = e / L, s = h.list[e - r * L];
      uint32_t w = h.word[s];
      if (h.key[s] & Hash::FED)
        for (unsigned long long m = path[r]; m; m &= m - 1) w += fed[__ffsll((long long)m) - 1] == s;
      const float f = adjusted(__uint_as_float(x), w, k);
      held[e - base] = w ? (isnan(f) ? 0x7fffffffu : __float_as_uint(f)) : NONE;
    }
    if (base == 0) grid_dep_wait();
#pragma unroll 1
    for (int e = base + t; e < end; e += WTHR) {  // (a thread stores what it worked out)
      const int r = e / L, token = (int)(h.key[h.list[e - r * L]] & ~Hash::FED);
      const uint32_t y = held[e - base];
      if (y != NONE) put(out + (size_t)r * a.ld_out + token, __uint_as_float(y));
    }
  }
  if (a.status && bad) atomicCAS(a.status, 0, (int)SPEC_ERR_CAPACITY);
}

template <typename T>
const void* pick(bool vec, bool same) {
  return same ? (const void*)adjust_kernel<T, false, true>
              : vec ? (const void*)adjust_kernel<T, true, false> : (const void*)adjust_kernel<T, false, false>;
}

template <typename T>
const void* pick_copy(bool vec, bool same) {
  return same ? (const void*)adjust_forbid_kernel<T>
              : vec ? (const void*)adjust_copy_kernel<T, true> : (const void*)adjust_copy_kernel<T, false>;
}
template <typename T>
void set_up() {
  for (bool v : {false, true})
    for (bool s : {false, true}) {
      cudaFuncSetAttribute(pick<T>(v, s), cudaFuncAttributeMaxDynamicSharedMemorySize, 16384 * 4 + 16384 / 8);
      // (so that the other kernel's tables find their shared memory while this one runs)
      cudaFuncSetAttribute(pick_copy<T>(v, s), cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    }
  cudaFuncSetAttribute(adjust_words_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, HASH_MAX * 8 + HASH_MAX * 3 / 2);
}

}  // namespace

void setup_adjust_attributes() {
  set_up<float>();
  set_up<__nv_bfloat16>();
}

int adjust_logits(AdjustArgs a, cudaStream_t st) {
  const int es = a.dtype == DT_F32 ? 4 : 2;
  const bool f32 = a.dtype == DT_F32, same = a.out == a.logits;
  const bool vec = ((uintptr_t)a.out & 15) == 0 && (a.B * a.R == 1 || ((a.ld_out * es) & 15) == 0);
  const bool counts = (a.history || a.tokens) && (a.repetition || a.presence || a.frequency);
  const bool words = counts || a.n_bias > 0;
  const long long tokens = (long long)a.n_history + a.R + a.n_bias;
  const long long bytes = (long long)a.B * a.R * a.V * es;
  void* args[] = {(void*)&a};
  // From 1 MB on two kernels: 8 x 5 rows of 262144 19.5 us (one 31.5), 64 rows 27 (38), 4 x 5 rows of 32003
  // 7.2 (11.7), one row of 262144 5.7 (6.2). Below, the launch saved is more: a call 16 us with the host, 18.5 with two.
  if (!words || (bytes >= (1 << 20) && tokens <= HASH_MAX * 3 / 4 && a.R <= TREE_ROWS_MAX && bytes < (1ll << 40))) {
    int launched = 0;
    if (!same || a.mask) {
      const long long lines = (same ? (a.V + 32 * FW - 1ll) / (32 * FW) : ((long long)a.V / (vec ? 16 / es : 1) + NTHR - 1) / NTHR) * a.B * a.R;
      const unsigned grid = (unsigned)std::max(1ll, std::min<long long>(lines, (same ? 8 : COPY_CTAS) * num_sms()));
      if (cudaLaunchKernel(f32 ? pick_copy<float>(vec, same) : pick_copy<__nv_bfloat16>(vec, same), dim3(grid), dim3(NTHR), args, 0,
                           st) != cudaSuccess)
        return -1;
      launched = 1;
    }
    if (!words) return launched;
    a.slots = 256;
    while (a.slots * 3 / 4 < tokens) a.slots *= 2;
    a.parts = std::max(1, std::min(64, num_sms() / a.B));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.parts, a.B);
    cfg.blockDim = dim3(WTHR);
    cfg.dynamicSmemBytes = (size_t)a.slots * 8 + (size_t)a.slots * 3 / 2;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = launched;  // (alone it waits for what is before it)
    const void* f = f32 ? (const void*)adjust_words_kernel<float> : (const void*)adjust_words_kernel<__nv_bfloat16>;
    return cudaLaunchKernelExC(&cfg, f, args) == cudaSuccess ? launched + 1 : -1;
  }
  // Four CTAs an SM: long chunks (a history is counted once for each), all of a
  // sequence's rows in a CTA; shorter chunks, then fewer rows, where that is too few.
  const long long enough = 4ll * num_sms();
  auto ctas = [&] { return (long long)a.B * ((a.V + a.chunk - 1) / a.chunk) * ((a.R + a.rows - 1) / a.rows); };
  a.chunk = 16384;
  a.rows = a.R;
  while (a.chunk > 4096 && ctas() < enough) a.chunk /= 2;
  while (a.rows > 1 && ctas() < enough) a.rows = (a.rows + 1) / 2;
  while (a.chunk > 1024 && ctas() < enough) a.chunk /= 2;
  const dim3 grid((a.V + a.chunk - 1) / a.chunk, a.B, (a.R + a.rows - 1) / a.rows);
  return cudaLaunchKernel(f32 ? pick<float>(vec, same) : pick<__nv_bfloat16>(vec, same), grid, dim3(NTHR), args,
                          (size_t)a.chunk * 4 + a.chunk / 8, st) == cudaSuccess
             ? 1
             : -1;
}

}  // namespace spec
