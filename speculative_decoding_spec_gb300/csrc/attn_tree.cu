// attn_tree.cu -- attention of the rows of drafted trees over the paged cache:
// the CUDA-core kernel (fp32 caches, head dims other than 64 and 128), and the
// kernel that joins units cut between CTAs (attn_tree.cuh says how).
//
// Row r of sequence b, its own key and value already at position n + r of the
// cache, attends the n committed keys and those of the rows on its path:
//   o_r = sum_j p_j v_j / sum_j p_j,  p_j = exp(q_r . k_j / sqrt(hd) - m_r),
// one pass over the keys with the running maximum m_r, sum and row of o, in fp32.
//
// A CTA of 256 threads holds 16 * TR query rows and walks its pages: the scores
// of a page are a TR x 4 tile a thread (K transposed in shared memory, so a
// step of the head dim is two vector loads for 4 * TR products), the
// probabilities go through shared memory, the output is TR rows x 4 dims x NJ
// a thread. 16 rows a tile where a KV head has no more.
#include <algorithm>

#include "attn_tree.cuh"

namespace spec {
namespace tree {
namespace {

constexpr int NTHR = 256;

SPEC_DEV float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
SPEC_DEV float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}
SPEC_DEV void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
SPEC_DEV void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&x), *reinterpret_cast<uint32_t*>(&y));
}
SPEC_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr int KLD = PAGE + 4;  // row of the transposed keys, a multiple of 16 bytes
size_t cc_smem(int hd, int TR) {
  const int rows = 16 * TR;
  return ((size_t)hd * rows + (size_t)hd * KLD + (size_t)PAGE * hd + (size_t)PAGE * (rows + 4)) * 4;
}

template <typename QT, typename KT, int TR, int NJ>
__global__ void __launch_bounds__(NTHR) tree_cc_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ Plan p) {
  constexpr int ROWS = 16 * TR, PLD = ROWS + 4;
  extern __shared__ __align__(16) float sm[];
  __shared__ unsigned long long path[64];
  __shared__ int up[64];
  grid_dep_launch();
  const int t = threadIdx.x, tx = t & 15, ty = t >> 4, hd = a.hd, G = p.G;
  float* qs = sm;                 // [hd][ROWS]
  float* ks = qs + hd * ROWS;     // [hd][KLD]
  float* vs = ks + hd * KLD;      // [PAGE][hd]
  float* ps = vs + PAGE * hd;     // [PAGE][PLD]
  const int bad = __syncthreads_or(bad_input(a, p, t, NTHR));
  if (t == 0) found(a, p, bad);
  Walk part;
  if (!part.begin(a, p)) return;
  const float scale2 = LOG2E / sqrtf((float)hd);

  for (; part.pieces(a, p); part.step(a, p)) {
    const Unit n = part.n;
    const Seq s = part.s;
    const int k0 = part.k0, k1 = k0 + part.N;
    const int row0 = n.u * ROWS, nrow = min(ROWS, s.rows * G - row0);
    __syncthreads();
    paths(a, n.b, s.rows, path, up, t, [] { __syncthreads(); });
    for (int i = t; i < ROWS * (hd / 4); i += NTHR) {
      const int r = i / (hd / 4), c = (i % (hd / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrow) {
        const int qr = p.row_of(row0 + r), g = row0 + r - qr * G;
        v = load4((const QT*)a.q + ((size_t)n.b * a.R + qr) * a.ldq + (size_t)(n.kvh * G + g) * hd + c);
      }
      qs[(c + 0) * ROWS + r] = v.x * scale2;
      qs[(c + 1) * ROWS + r] = v.y * scale2;
      qs[(c + 2) * ROWS + r] = v.z * scale2;
      qs[(c + 3) * ROWS + r] = v.w * scale2;
    }
    float m[TR], l[TR], o[TR][NJ][4];
#pragma unroll
    for (int i = 0; i < TR; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
    }
    for (int k = k0; k < k1; ++k) {
      const size_t base = ((size_t)page_of(a, s.slot, k) * 2 * a.nkv + n.kvh) * PAGE * hd;
      const KT* kp = (const KT*)a.pool + base;
      const KT* vp = kp + (size_t)a.nkv * PAGE * hd;
      const int valid = min(PAGE, s.len + s.rows - k * PAGE);  // keys that are there; behind them the page holds anything
      __syncthreads();
      for (int i = t; i < PAGE * (hd / 4); i += NTHR) {
        const int key = i / (hd / 4), c = (i % (hd / 4)) * 4;
        float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
        if (key < valid) {
          kv = load4(kp + (size_t)key * hd + c);
          vv = load4(vp + (size_t)key * hd + c);
        }
        ks[(c + 0) * KLD + key] = kv.x;
        ks[(c + 1) * KLD + key] = kv.y;
        ks[(c + 2) * KLD + key] = kv.z;
        ks[(c + 3) * KLD + key] = kv.w;
        *reinterpret_cast<float4*>(vs + key * hd + c) = vv;
      }
      __syncthreads();
      float acc[TR][4];
#pragma unroll
      for (int i = 0; i < TR; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll 4
      for (int d = 0; d < hd; ++d) {
        const float4 kk = *reinterpret_cast<const float4*>(ks + d * KLD + 4 * tx);
        float qq[TR];
        if constexpr (TR == 4) {
          const float4 v = *reinterpret_cast<const float4*>(qs + d * ROWS + 4 * ty);
          qq[0] = v.x; qq[1] = v.y; qq[2] = v.z; qq[3] = v.w;
        } else {
          qq[0] = qs[d * ROWS + ty];
        }
#pragma unroll
        for (int i = 0; i < TR; ++i) {
          acc[i][0] = fmaf(qq[i], kk.x, acc[i][0]);
          acc[i][1] = fmaf(qq[i], kk.y, acc[i][1]);
          acc[i][2] = fmaf(qq[i], kk.z, acc[i][2]);
          acc[i][3] = fmaf(qq[i], kk.w, acc[i][3]);
        }
      }
      const bool all = (k + 1) * PAGE <= s.len;  // no key of this page is a row of the tree
#pragma unroll
      for (int i = 0; i < TR; ++i) {
        const int r = ty * TR + i;
        const unsigned long long vis =
            r < nrow ? (all ? ~0ull : visible(path[p.row_of(row0 + r)], s.len, k * PAGE)) : 0ull;
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!((vis >> (4 * tx + e)) & 1)) acc[i][e] = -INFINITY;
          mx = fmaxf(mx, acc[i][e]);
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, w));
        const float mn = fmaxf(m[i], mx);
        // (nothing above -inf so far: no weights yet; a row that ends so has 0 / 0, as in the formula)
        const float f = m[i] == -INFINITY ? 0.f : ex2(m[i] - mn), mb = mn == -INFINITY ? 0.f : mn;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float pr = ex2(acc[i][e] - mb);
          sum += pr;
          ps[(4 * tx + e) * PLD + r] = pr;
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(FULL, sum, w);
        l[i] = l[i] * f + sum;
        m[i] = mn;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][j][e] *= f;
      }
      __syncthreads();
      auto values = [&](bool some) {  // some: a row may not see a key, whose value is then left out (it may be infinite)
        unsigned long long vis[TR];
#pragma unroll
        for (int i = 0; i < TR; ++i) {
          const int r = ty * TR + i;
          vis[i] = some && r < nrow ? visible(path[p.row_of(row0 + r)], s.len, k * PAGE) : ~0ull;
        }
#pragma unroll 2
        for (int key = 0; key < valid; ++key) {
          float pp[TR];
          if constexpr (TR == 4) {
            const float4 v = *reinterpret_cast<const float4*>(ps + key * PLD + 4 * ty);
            pp[0] = v.x; pp[1] = v.y; pp[2] = v.z; pp[3] = v.w;
          } else {
            pp[0] = ps[key * PLD + ty];
          }
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int d = 4 * tx + 64 * j;
            if (NJ * 64 != hd && d >= hd) break;
            const float4 v = *reinterpret_cast<const float4*>(vs + key * hd + d);
#pragma unroll
            for (int i = 0; i < TR; ++i) {
              if (some && !((vis[i] >> key) & 1)) continue;
              o[i][j][0] = fmaf(pp[i], v.x, o[i][j][0]);
              o[i][j][1] = fmaf(pp[i], v.y, o[i][j][1]);
              o[i][j][2] = fmaf(pp[i], v.z, o[i][j][2]);
              o[i][j][3] = fmaf(pp[i], v.w, o[i][j][3]);
            }
          }
        }
      };
      if (all) values(false);
      else values(true);
    }
    const bool whole = k0 == 0 && k1 == n.nb;
    const size_t slot = (size_t)(2 * blockIdx.x + (k0 == 0)) * ROWS;
#pragma unroll
    for (int i = 0; i < TR; ++i) {
      const int r = ty * TR + i;
      if (r >= nrow) continue;
      const int qr = p.row_of(row0 + r), g = row0 + r - qr * G;
      const float inv = whole ? 1.f / l[i] : 1.f;
      if (!whole && tx == 0) a.part_ml[slot + r] = make_float2(m[i], l[i]);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int d = 4 * tx + 64 * j;
        if (d >= hd) break;
        const float4 v = make_float4(o[i][j][0] * inv, o[i][j][1] * inv, o[i][j][2] * inv, o[i][j][3] * inv);
        if (whole) store4((QT*)a.out + ((size_t)n.b * a.R + qr) * a.ldo + (size_t)(n.kvh * G + g) * hd + d, v);
        else store4(a.part_o + (slot + r) * hd + d, v);
      }
    }
  }
}

// pre[b] = where sequence b starts on the axis, pre[B] its end. By one warp.
SPEC_DEV void starts(const TreeArgs& a, const Plan& p, int* pre) {
  const int lane = threadIdx.x & 31;
  int run = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int c = b0 + lane < a.B ? cost_of(a, p, b0 + lane) : 0, end = run + scan32(c);
    if (b0 + lane < a.B) pre[b0 + lane] = end - c;
    run = __shfl_sync(FULL, end, 31);
  }
  if (lane == 0) pre[a.B] = run;
}

// What a lane knows of the pieces of a unit: lane i has CTA c + i's (c + 8 i's).
SPEC_DEV int piece_slot(const Plan& p, const Unit& n, const Cut& cut, int c, int c1) {
  if (c > c1) return -1;
  const int k0 = first_block(p, n, cut.start(c)), k1 = first_block(p, n, cut.start(c + 1));
  return k0 < k1 && k1 - k0 < n.nb ? 2 * c + (k0 == 0) : -1;
}

// Units that one CTA finished are left alone; of the others a warp joins four
// query rows (ALL: the CTA's eight warps one row, each an eighth of its pieces). LN
// lanes hold a row, 32 / LN pieces go side by side, ROUND of them in flight.
template <typename QT, int LN, int NJ, bool ALL>
__global__ void __launch_bounds__(NTHR) tree_join_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ Plan p) {
  constexpr int SIDE = 32 / LN, RW = ALL ? 1 : 4, ROUND = ALL ? 8 : 2;
  __shared__ int pre[TREE_B_MAX + 1];
  __shared__ float2 wml[8];
  __shared__ float4 wacc[ALL ? 8 : 1][32][NJ];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.G, hd = a.hd;
  if (w == 0) starts(a, p, pre);  // (the call's inputs are not written by the kernel before this one)
  __syncthreads();
  const Cut cut(p, pre[a.B]);
  grid_dep_wait();
  if (blockIdx.x == 0 && w == 0) {  // the call's outcome: the worst of the CTAs'
    int worst = 0;
    for (int c = lane; c < p.grid; c += 32) worst = max(worst, a.flags[c]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) worst = max(worst, __shfl_xor_sync(FULL, worst, o));
    if (lane == 0) *a.err = worst;
  }
  if (cut.ctas == 1) return;
  const int urows = p.tpu << p.tile, sub = lane / LN, ln = lane % LN;
  const int groups = (a.R * G + RW - 1) / RW;  // of a (sequence, KV head) pair's rows (a group lies in one unit)
  for (int i = ALL ? blockIdx.x : blockIdx.x * 8 + w; i < a.B * a.nkv * groups; i += gridDim.x * (ALL ? 1 : 8)) {
    const int pair = i / groups, q0 = (i - pair * groups) * RW, b = pair / a.nkv, kvh = pair - b * a.nkv;
    const Seq s = seq_of(a, b);
    const int nrow = min(RW, s.rows * G - q0);
    if (nrow <= 0) continue;
    const int T = tiles_of(p, s.rows), nb = blocks_of(p, s);
    Unit n;
    n.u = q0 / urows;
    n.nb = nb;
    n.w = min(p.tpu, T - n.u * p.tpu);
    n.start = pre[b] + kvh * pair_length(p, T, nb) + n.u * (nb * p.tpu + p.head);
    // the first and last CTA whose parts meet the unit
    const int c0 = cut.part_of(n.start), c1 = cut.part_of(n.start + p.head + nb * n.w - 1), at = q0 - n.u * urows;
    if (c0 == c1) continue;
    float M[RW], L[RW];
    float4 acc[RW][NJ];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      M[r] = -INFINITY;
      L[r] = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[r][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    bool cutup = false;
    for (int c = c0 + (ALL ? w : 0); c <= c1; c += ALL ? 256 : 32) {
      const int slot = piece_slot(p, n, cut, c + lane * (ALL ? 8 : 1), c1);
      if (!__any_sync(FULL, slot >= 0)) continue;
      cutup = true;
      float f[RW];
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const float2 ml = slot >= 0 && r < nrow ? a.part_ml[(size_t)slot * urows + at + r] : make_float2(-INFINITY, 0.f);
        const float mn = fmaxf(M[r], warp_max(ml.x));
        f[r] = ml.x == -INFINITY ? 0.f : ex2(ml.x - mn);
        const float old = M[r] == -INFINITY ? 0.f : ex2(M[r] - mn);
        M[r] = mn;
        L[r] = L[r] * old + warp_sum(f[r] * ml.y);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          acc[r][j].x *= old; acc[r][j].y *= old; acc[r][j].z *= old; acc[r][j].w *= old;
        }
      }
      const int last = min(32, (ALL ? (c1 - c) >> 3 : c1 - c) + 1);
      for (int i0 = 0; i0 < last; i0 += ROUND * SIDE) {
        float4 v[ROUND][RW][NJ];
#pragma unroll
        for (int e = 0; e < ROUND; ++e) {
          const int k = i0 + e * SIDE + sub, si = __shfl_sync(FULL, slot, k & 31);
          const float* src = a.part_o + ((size_t)si * urows + at) * hd;
#pragma unroll
          for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const int d = 4 * ln + 4 * LN * j;
              v[e][r][j] = k < last && si >= 0 && r < nrow && d < hd ? *reinterpret_cast<const float4*>(src + r * hd + d)
                                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
#pragma unroll
        for (int e = 0; e < ROUND; ++e) {
          const int k = i0 + e * SIDE + sub;
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float fk = __shfl_sync(FULL, f[r], k & 31), x = k < last ? fk : 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              acc[r][j].x = fmaf(x, v[e][r][j].x, acc[r][j].x);
              acc[r][j].y = fmaf(x, v[e][r][j].y, acc[r][j].y);
              acc[r][j].z = fmaf(x, v[e][r][j].z, acc[r][j].z);
              acc[r][j].w = fmaf(x, v[e][r][j].w, acc[r][j].w);
            }
          }
        }
      }
    }
    if (ALL ? !__syncthreads_or(cutup) : !cutup) continue;  // one CTA had all of its blocks
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int o = LN; o < 32; o <<= 1) {
          acc[r][j].x += __shfl_xor_sync(FULL, acc[r][j].x, o);
          acc[r][j].y += __shfl_xor_sync(FULL, acc[r][j].y, o);
          acc[r][j].z += __shfl_xor_sync(FULL, acc[r][j].z, o);
          acc[r][j].w += __shfl_xor_sync(FULL, acc[r][j].w, o);
        }
    if (ALL) {
      if (lane == 0) wml[w] = make_float2(M[0], L[0]);
#pragma unroll
      for (int j = 0; j < NJ; ++j) wacc[w][lane][j] = acc[0][j];
      __syncthreads();
      if (w == 0) {
        for (int k = 0; k < 8; ++k) M[0] = fmaxf(M[0], wml[k].x);
        L[0] = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[0][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < 8; ++k) {
          const float f = wml[k].x == -INFINITY ? 0.f : ex2(wml[k].x - M[0]);
          L[0] = fmaf(f, wml[k].y, L[0]);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const float4 v = wacc[k][lane][j];
            acc[0][j].x = fmaf(f, v.x, acc[0][j].x);
            acc[0][j].y = fmaf(f, v.y, acc[0][j].y);
            acc[0][j].z = fmaf(f, v.z, acc[0][j].z);
            acc[0][j].w = fmaf(f, v.w, acc[0][j].w);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      if (r >= nrow || (ALL && w)) break;
      const float inv = 1.f / L[r];
      const int qr = p.row_of(q0 + r), g = q0 + r - qr * G;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int d = 4 * ln + 4 * LN * j;
        if (sub == 0 && d < hd)
          store4((QT*)a.out + ((size_t)b * a.R + qr) * a.ldo + (size_t)(kvh * G + g) * hd + d,
                 make_float4(acc[r][j].x * inv, acc[r][j].y * inv, acc[r][j].z * inv, acc[r][j].w * inv));
      }
    }
    if (ALL) __syncthreads();
  }
}

template <typename QT, bool ALL>
const void* join_kernel(int hd) {
  return hd <= 64 ? (const void*)tree_join_kernel<QT, 16, 1, ALL>
                  : hd <= 128 ? (const void*)tree_join_kernel<QT, 32, 1, ALL> : (const void*)tree_join_kernel<QT, 32, 2, ALL>;
}

template <typename QT, typename KT, int TR>
const void* cc_kernel(int hd) {
  return hd <= 64 ? (const void*)tree_cc_kernel<QT, KT, TR, 1>
                  : hd <= 128 ? (const void*)tree_cc_kernel<QT, KT, TR, 2> : (const void*)tree_cc_kernel<QT, KT, TR, 4>;
}
const void* cc_pick(int q_dtype, int kv_dtype, int TR, int hd) {
  if (q_dtype == DT_F32 && kv_dtype == DT_F32)
    return TR == 1 ? cc_kernel<float, float, 1>(hd) : cc_kernel<float, float, 4>(hd);
  if (q_dtype == DT_F32)
    return TR == 1 ? cc_kernel<float, __nv_bfloat16, 1>(hd) : cc_kernel<float, __nv_bfloat16, 4>(hd);
  if (kv_dtype == DT_F32)
    return TR == 1 ? cc_kernel<__nv_bfloat16, float, 1>(hd) : cc_kernel<__nv_bfloat16, float, 4>(hd);
  return TR == 1 ? cc_kernel<__nv_bfloat16, __nv_bfloat16, 1>(hd) : cc_kernel<__nv_bfloat16, __nv_bfloat16, 4>(hd);
}
int cc_rows(const TreeArgs& a) { return a.R * (a.nq / a.nkv) <= 16 ? 1 : 4; }

Plan cc_plan(const TreeArgs& a) {
  Plan p;
  const int TR = cc_rows(a);
  p.blk = 6;
  p.tile = TR == 1 ? 4 : 6;
  p.tpu = 1;
  const int per_sm = std::max(1, std::min(4, (int)(220 * 1024 / cc_smem(a.hd, TR))));
  p.grid = std::min(1024, num_sms() * per_sm);
  p.min_cost = 2;
  p.head = 1;
  p.units = 0;
  plan_heads(p, a);
  return p;
}

// The longest axis a call of this shape can have.
long long axis_of(const TreeArgs& a, const Plan& p) {
  const long long T = (a.R * p.G + (1 << p.tile) - 1) >> p.tile;
  return (long long)a.B * a.nkv * T * ((((long long)a.max_pages * PAGE + (1 << p.blk) - 1) >> p.blk) + p.head);
}

Plan plan_of(const TreeArgs& a) {
  Plan p = tc_ok(a) ? tc_plan(a) : cc_plan(a);
  // no more CTAs than the axis can have blocks
  const long long most = axis_of(a, p);
  const long long T = (a.R * p.G + (1 << p.tile) - 1) >> p.tile;
  // no cuts up to 256 keys: they cost a second kernel (4 x 68 keys, fp32: 12.9 us, 16.5 with)
  if ((long long)a.max_pages * PAGE <= 256) {
    p.units = (int)((T + p.tpu - 1) / p.tpu);
    p.grid = a.B * a.nkv * p.units;
    return p;
  }
  p.grid = (int)std::max<long long>(1, std::min<long long>(p.grid, (most + p.min_cost - 1) / p.min_cost));
  return p;
}

}  // namespace
}  // namespace tree

using namespace tree;

static TreeArgs shape_args(int B, int R, int nq, int nkv, int hd, int max_pages, int q_dtype, int kv_dtype) {
  TreeArgs a = {};
  a.B = B; a.R = R; a.nq = nq; a.nkv = nkv; a.hd = hd; a.max_pages = max_pages;
  a.q_dtype = q_dtype; a.kv_dtype = kv_dtype;
  return a;
}
constexpr size_t HEAD_BYTES = 256 + 4 * 1024;  // (no kernel has more than 1024 CTAs where it cuts)
static size_t part_rows(const Plan& p) { return p.units ? 0 : (size_t)2 * p.grid * p.tpu << p.tile; }

// error word (256 bytes), the CTAs' words, maxima and sums, rows; 0 where a kernel's axis (whose
// numbers have 32 bits, slots of rows among them) may not hold the call, or a KV head has too many rows
size_t attn_tree_bytes(int B, int R, int nq, int nkv, int hd, int max_pages) {
  if ((long long)R * (nq / nkv) > TREE_HEAD_ROWS_MAX) return 0;
  size_t most = 0;
  for (int q : {DT_F32, DT_BF16})
    for (int kv : {DT_F32, DT_BF16}) {
      const TreeArgs a = shape_args(B, R, nq, nkv, hd, max_pages, q, kv);
      const Plan p = plan_of(a);
      if (axis_of(a, p) + 512 > 0x7fffffffll || (long long)B * R * nq > (1ll << 30)) return 0;
      const size_t rows = part_rows(p);
      most = std::max(most, HEAD_BYTES + rows * (sizeof(float2) + (size_t)hd * sizeof(float)));
    }
  return most;
}

void setup_attn_tree_attributes() {
  for (int q : {DT_F32, DT_BF16})
    for (int kv : {DT_F32, DT_BF16})
      for (int TR : {1, 4})
        for (int hd : {64, 128, 256})
          cudaFuncSetAttribute(cc_pick(q, kv, TR, hd), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cc_smem(hd, TR));
  tc_setup();
}

int attn_tree(TreeArgs a, void* ws, cudaStream_t st) {
  const Plan p = plan_of(a);
  a.err = (int*)ws;
  a.flags = (int*)((char*)ws + 256);
  a.part_ml = (float2*)((char*)ws + HEAD_BYTES);
  a.part_o = (float*)(a.part_ml + part_rows(p));
  int r = 1;
  if (tc_ok(a)) {
    r = tc_launch(a, p, st);
  } else {
    const int TR = cc_rows(a);
    void* cargs[] = {(void*)&a, (void*)&p};
    if (cudaLaunchKernel(cc_pick(a.q_dtype, a.kv_dtype, TR, a.hd), dim3(p.grid), dim3(NTHR), cargs, cc_smem(a.hd, TR), st) !=
        cudaSuccess)
      r = -1;
  }
  if (r < 0) return r;
  if (p.units) return r;  // nothing is cut
  cudaLaunchConfig_t cfg = {};
  const long long rows = (long long)a.B * a.R * a.nq;
  // few rows are cut into many pieces: a CTA a row then (84 rows of 38 pieces, both kernels: 53 us, 72 with a warp a row)
  const bool all = rows <= 4 * num_sms();
  // else as many CTAs as fit at once, which begin once (24576 rows: 112.7 us, 114.1 with a CTA for each 32 rows)
  cfg.gridDim = dim3((unsigned)std::min<long long>(all ? rows : (rows + 31) / 32, (all ? 8ll : 2ll) * num_sms()));
  cfg.blockDim = dim3(NTHR);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {(void*)&a, (void*)&p};
  const void* f = a.q_dtype == DT_F32 ? (all ? join_kernel<float, true>(a.hd) : join_kernel<float, false>(a.hd))
                                      : (all ? join_kernel<__nv_bfloat16, true>(a.hd) : join_kernel<__nv_bfloat16, false>(a.hd));
  return cudaLaunchKernelExC(&cfg, f, args) == cudaSuccess ? r + 1 : -1;
}

}  // namespace spec
