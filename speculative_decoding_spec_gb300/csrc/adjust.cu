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
// the vocabulary for all rows of a sequence and keeps one word a token of it in
// shared memory, counted once from the history, so a row costs its tokens'
// words (mostly zero: the logit passes through) and a step costs no table of
// [rows][V] in memory. The rows of a path differ by a few tokens; they are
// counted in and out between rows.
#include <algorithm>

#include "common.cuh"

namespace spec {
namespace {

constexpr int NTHR = 512;
// A token's word: times said (19 bits), occurs at all, place of its bias in the list + 1 (12 bits).
constexpr uint32_t COUNT = (1u << 19) - 1, SEEN = 1u << 19;
constexpr int BIAS_AT = 20;

struct Rules {
  float rep, freq, pres;
  const float* bias;
};

SPEC_DEV float adjusted(float x, uint32_t w, const Rules& k) {
  if (w & (COUNT | SEEN)) {
    x = x > 0.f ? __fdiv_rn(x, k.rep) : x * k.rep;
    const uint32_t c = w & COUNT;
    if (c) x = x - (float)c * k.freq - k.pres;
  }
  if (w >> BIAS_AT) {
    const float b = k.bias[(w >> BIAS_AT) - 1];
    x = b == -INFINITY || x == -INFINITY ? -INFINITY : x + b;
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

// VEC: rows of the output start on 16-byte boundaries. SAME: in place, so what
// stays as it is is neither read nor written.
template <typename T, bool VEC, bool SAME>
__global__ void __launch_bounds__(NTHR) adjust_kernel(const __grid_constant__ AdjustArgs a) {
  using V = Vec<T>;
  extern __shared__ __align__(16) uint32_t tab[];  // [chunk]
  __shared__ unsigned long long path[TREE_ROWS_MAX];
  const int t = threadIdx.x, b = blockIdx.y;
  const int c0 = blockIdx.x * a.chunk, nc = min(a.chunk, a.V - c0);
  Rules k;
  k.rep = setting(a.repetition, b, 1.f, true);
  k.freq = setting(a.frequency, b, 0.f, false);
  k.pres = setting(a.presence, b, 0.f, false);
  const bool count = k.rep != 1.f || k.freq != 0.f || k.pres != 0.f;
  const bool use = count || a.n_bias > 0;
  bool bad = false;
  if (a.status && blockIdx.x == 0 && a.parents)
    for (int r = t; r < a.R; r += NTHR) {
      const int p = a.parents[(size_t)b * a.R + r];
      bad |= p < -1 || p >= r;
    }
  if (use) {
    for (int i = t; i < (nc + 3) / 4; i += NTHR) reinterpret_cast<uint4*>(tab)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (a.n_bias > 0) {
      k.bias = a.bias_values + (size_t)b * a.n_bias;
      for (int i = t; i < a.n_bias; i += NTHR) {
        const unsigned at = (unsigned)(a.bias_tokens[(size_t)b * a.n_bias + i] - c0);
        // the last of several entries for a token counts
        if (at < (unsigned)nc) atomicMax(&tab[at], (uint32_t)(i + 1) << BIAS_AT);
      }
      __syncthreads();
      // (a bias of NaN is none)
      for (int i = t; i < a.n_bias; i += NTHR) {
        const unsigned at = (unsigned)(a.bias_tokens[(size_t)b * a.n_bias + i] - c0);
        if (at < (unsigned)nc && isnan(k.bias[i]) && tab[at] == (uint32_t)(i + 1) << BIAS_AT) tab[at] = 0;
      }
      __syncthreads();
    }
    if (count) {
      if (a.history) {
        int n = a.hist_len ? a.hist_len[b] : a.n_history, np = a.prompt_len ? a.prompt_len[b] : 0;
        bad |= n < 0 || n > a.n_history || np < 0 || np > n;
        n = min(max(n, 0), a.n_history);
        const int32_t* h = a.history + (size_t)b * a.ld_history;
        int i = t;
        for (; i + 3 * NTHR < n; i += 4 * NTHR) {
          int tok[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) tok[j] = h[i + j * NTHR];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const unsigned at = (unsigned)(tok[j] - c0);
            if (at < (unsigned)nc) {
              if (i + j * NTHR < np) atomicOr(&tab[at], SEEN);
              else atomicAdd(&tab[at], 1u);
            }
          }
        }
        for (; i < n; i += NTHR) {
          const unsigned at = (unsigned)(h[i] - c0);
          if (at < (unsigned)nc) {
            if (i < np) atomicOr(&tab[at], SEEN);
            else atomicAdd(&tab[at], 1u);
          }
        }
      }
      if (a.tokens && a.parents) {
        // a row's path as bits (a parent that is not an earlier row counts as none)
        if (t < TREE_ROWS_MAX) {
          unsigned long long m = 0;
          if (t < a.R)
            for (int r = t; r >= 0;) {
              m |= 1ull << r;
              const int p = a.parents[(size_t)b * a.R + r];
              r = p < r ? p : -1;
            }
          path[t] = m;
        }
      }
      __syncthreads();
    }
  }
  for (int r = 0; r < a.R; ++r) {
    const size_t m = (size_t)b * a.R + r;
    if (count && a.tokens) {
      if (a.parents) {
        const unsigned long long now = path[r], was = r ? path[r - 1] : 0ull;
        if (t < a.R && ((now ^ was) >> t) & 1) {
          const unsigned at = (unsigned)(a.tokens[(size_t)b * a.R + t] - c0);
          if (at < (unsigned)nc) {
            if ((now >> t) & 1) atomicAdd(&tab[at], 1u);
            else atomicSub(&tab[at], 1u);
          }
        }
      } else if (t == 0) {
        const unsigned at = (unsigned)(a.tokens[m] - c0);
        if (at < (unsigned)nc) tab[at] += 1u;
      }
      __syncthreads();
    }
    int id = a.mask_ids ? a.mask_ids[m] : (int)m;
    if (a.mask && (id < -1 || id >= a.n_masks)) {
      bad = true;
      id = -1;
    }
    const uint32_t* bits = a.mask && id >= 0 ? a.mask + (size_t)id * a.ld_mask + (c0 >> 5) : nullptr;  // (chunks start on words)
    const char* src = (const char*)((const T*)a.logits + (size_t)m * a.ld + c0);
    T* dst = (T*)a.out + (size_t)m * a.ld_out + c0;
    if constexpr (VEC) {
      const int mis = (int)((uintptr_t)src & 15);
      const long long bytes = (long long)nc * sizeof(T);
      const int nv = nc / V::N;
      constexpr int U = 4;
      for (int i0 = t; i0 < nv; i0 += U * NTHR) {
        uint4 v[U];
        uint32_t ban[U];
        bool touch[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * NTHR;
          if (i >= nv) break;
          ban[u] = bits ? ~bits[(i * V::N) >> 5] >> ((i * V::N) & 31) & ((1u << V::N) - 1) : 0u;
          touch[u] = ban[u] != 0;
          if (use) {
#pragma unroll
            for (int e = 0; e < V::N; e += 4) {
              const uint4 w = *reinterpret_cast<const uint4*>(tab + i * V::N + e);
              touch[u] |= (w.x | w.y | w.z | w.w) != 0;
            }
          }
          if (!SAME || touch[u]) v[u] = load_shifted(src, (long long)i * 16, mis, bytes);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * NTHR;
          if (i >= nv) break;
          if (touch[u]) {
            float f[V::N];
#pragma unroll
            for (int e = 0; e < V::N; ++e) {
              f[e] = V::get(v[u], e);
              const uint32_t w = use ? tab[i * V::N + e] : 0u;
              if (w) f[e] = adjusted(f[e], w, k);
              if ((ban[u] >> e) & 1) f[e] = -INFINITY;
            }
            V::pack(v[u], f);
          }
          if (!SAME || touch[u]) __stcs(reinterpret_cast<uint4*>(dst) + i, v[u]);
        }
      }
    }
    for (int i = (VEC ? nc / V::N * V::N : 0) + t; i < nc; i += NTHR) {
      const uint32_t w = use ? tab[i] : 0u;
      const bool ban = bits && !((bits[i >> 5] >> (i & 31)) & 1);
      if (SAME && !w && !ban) continue;
      float x = value(reinterpret_cast<const T*>(src)[i]);
      if (w) x = adjusted(x, w, k);
      put(dst + i, ban ? -INFINITY : x);
    }
    if (count && a.tokens) __syncthreads();
  }
  if (a.status && bad) atomicCAS(a.status, 0, (int)SPEC_ERR_CAPACITY);
}

template <typename T>
const void* pick(bool vec, bool same) {
  return vec ? (same ? (const void*)adjust_kernel<T, true, true> : (const void*)adjust_kernel<T, true, false>)
             : (same ? (const void*)adjust_kernel<T, false, true> : (const void*)adjust_kernel<T, false, false>);
}

constexpr int CHUNK_MAX = 16384;

}  // namespace

void setup_adjust_attributes() {
  for (bool v : {false, true})
    for (bool s : {false, true}) {
      cudaFuncSetAttribute(pick<float>(v, s), cudaFuncAttributeMaxDynamicSharedMemorySize, CHUNK_MAX * 4);
      cudaFuncSetAttribute(pick<__nv_bfloat16>(v, s), cudaFuncAttributeMaxDynamicSharedMemorySize, CHUNK_MAX * 4);
    }
}

int adjust_logits(AdjustArgs a, cudaStream_t st) {
  const int es = a.dtype == DT_F32 ? 4 : 2;
  const bool same = a.out == a.logits;
  const bool vec = ((uintptr_t)a.out & 15) == 0 && (a.B * a.R == 1 || ((a.ld_out * es) & 15) == 0);
  // the longest chunk that still gives every SM two CTAs
  a.chunk = CHUNK_MAX;
  while (a.chunk > 1024 && (long long)a.B * ((a.V + a.chunk - 1) / a.chunk) < 2ll * num_sms()) a.chunk /= 2;
  const void* f = a.dtype == DT_F32 ? pick<float>(vec, same) : pick<__nv_bfloat16>(vec, same);
  void* args[] = {(void*)&a};
  const dim3 grid((a.V + a.chunk - 1) / a.chunk, a.B);
  return cudaLaunchKernel(f, grid, dim3(NTHR), args, (size_t)a.chunk * 4, st) == cudaSuccess ? 1 : -1;
}

}  // namespace spec
