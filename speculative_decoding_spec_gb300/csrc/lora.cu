// lora.cu -- low-rank adapters of many requests beside one shared projection:
// y[m] = W xn[m] + s_a B_a (A_a xn[m]) with a = ids[m], the adapter row m's
// request brings (-1: none), and xn = x or RMSNorm(x) * gain; for the weight and
// adapter types that the one-stream kernel (lora_gemm.cu) does not cover.
//
// Two small kernels in front of the shared weight stream (gemv): the shrink
// t[m] = s_a A_a xn[m] (rank numbers a row) and the expand B_a t[m]. The expand
// writes y and the projection adds to it in its residual-add epilogue, so y
// makes one trip less than with the adapters added behind the projection, and
// each kernel of the chain starts while the one before it runs. (Rows of y that
// do not start on 16 bytes, N % 4 != 0, take the other order: the residual-add
// epilogue prefetches y in 16-byte pieces.) Bound by the Q4_0 projection: 12288 x
// 1536, 20 rows, 4 adapters of rank 32 30 us, 25 of them the projection's kernel.
#include <algorithm>

#include "common.cuh"

namespace spec {

namespace {

constexpr int SHRINK_THR = 256, EXPAND_THR = 128;
constexpr int RANKS = 8;       // ranks of a shrink block
constexpr int HELD = 32;       // ranks of B a thread of the expand holds

template <typename T>
SPEC_DEV void load8(const T* p, float (&v)[8]);
template <>
SPEC_DEV void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
SPEC_DEV void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  v[0] = bf16lo(q.x); v[1] = bf16hi(q.x); v[2] = bf16lo(q.y); v[3] = bf16hi(q.y);
  v[4] = bf16lo(q.z); v[5] = bf16hi(q.z); v[6] = bf16lo(q.w); v[7] = bf16hi(q.w);
}

// t[m][r] for one row m and 8 of its ranks, all warps together along K; CTA
// (0, 0) also clears the projection's arrival counters and records an id out of
// range.
template <typename T>
__global__ void __launch_bounds__(SHRINK_THR) shrink_kernel(LoraArgs a) {
  __shared__ float sums[SHRINK_THR / 32][RANKS + 1];
  grid_dep_launch();
  const int m = blockIdx.x, r0 = blockIdx.y * RANKS, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int i = threadIdx.x; i < a.n_cnt; i += blockDim.x) a.cnt[i] = 0u;
    int bad = 0;
    for (int i = threadIdx.x; i < a.M; i += blockDim.x) bad |= a.ids[i] < -1 || a.ids[i] >= a.n_adapters;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.err = bad ? SPEC_ERR_CAPACITY : SPEC_ERR_NONE;
  }
  const int id = a.ids[m];
  if (id < 0 || id >= a.n_adapters) return;
  const float* x = a.x + (size_t)m * a.K;
  const T* A = (const T*)a.a + ((size_t)id * a.rank + r0) * a.K;
  float acc[RANKS], ss = 0.f;
#pragma unroll
  for (int r = 0; r < RANKS; ++r) acc[r] = 0.f;
  for (int c = threadIdx.x * 8; c < a.K; c += SHRINK_THR * 8) {
    float v[8];
    load8(x + c, v);
    if (a.gain) {
      float g[8];
      load8(a.gain + c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(v[i], v[i], ss);
        v[i] *= g[i];
      }
    }
#pragma unroll
    for (int r = 0; r < RANKS; ++r) {
      float w[8];
      load8(A + (size_t)r * a.K + c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[r] = fmaf(w[i], v[i], acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < RANKS; ++r) acc[r] = warp_sum(acc[r]);
  ss = warp_sum(ss);
  if (lane == 0) {
#pragma unroll
    for (int r = 0; r < RANKS; ++r) sums[warp][r] = acc[r];
    sums[warp][RANKS] = ss;
  }
  __syncthreads();
  if (threadIdx.x < RANKS) {
    float t = 0.f, s = 0.f;
    for (int w = 0; w < SHRINK_THR / 32; ++w) {
      t += sums[w][threadIdx.x];
      s += sums[w][RANKS];
    }
    if (a.gain) t *= rsqrtf(s / (float)a.K + a.eps);
    a.t[(size_t)m * a.rank + r0 + threadIdx.x] = t * (a.scale ? a.scale[id] : 1.f);
  }
}

// y[m][n] (= or +=) B_a[n] . t[m]: a thread a column, `rows` rows of t in shared
// memory. Up to HELD ranks of B stay in registers over the rows of a request.
template <typename T>
__global__ void __launch_bounds__(EXPAND_THR) expand_kernel(LoraArgs a, int rows) {
  extern __shared__ __align__(16) float ts[];
  __shared__ int ids[64];
  grid_dep_launch();
  const int m0 = blockIdx.y * rows, nr = min(rows, a.M - m0);
  if (threadIdx.x < nr) {   // (the call's input: complete before the shrink)
    const int id = a.ids[m0 + threadIdx.x];
    ids[threadIdx.x] = id < 0 || id >= a.n_adapters ? -1 : id;
  }
  grid_dep_wait();
  for (int i = threadIdx.x * 4; i < nr * a.rank; i += blockDim.x * 4)
    *reinterpret_cast<float4*>(ts + i) = __ldcg(reinterpret_cast<const float4*>(a.t + (size_t)m0 * a.rank + i));
  __syncthreads();
  const int n = blockIdx.x * blockDim.x + threadIdx.x;
  if (n >= a.N) return;
  float w[HELD / 8][8];
  int held = -1;
  for (int m = 0; m < nr; ++m) {
    const int id = ids[m];
    if (id < 0 && a.add) continue;
    float acc = 0.f;
    if (id >= 0) {
      const T* B = (const T*)a.b + ((size_t)id * a.N + n) * a.rank;
      const float* t = ts + m * a.rank;
      if (a.rank <= HELD) {
        if (id != held) {
#pragma unroll
          for (int r = 0; r < HELD / 8; ++r)
            if (r * 8 < a.rank) load8(B + r * 8, w[r]);
          held = id;
        }
#pragma unroll
        for (int r = 0; r < HELD / 8; ++r)
          if (r * 8 < a.rank)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc = fmaf(w[r][i], t[r * 8 + i], acc);
      } else {
        for (int r = 0; r < a.rank; r += 8) {
          float v[8];
          load8(B + r, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc = fmaf(v[i], t[r + i], acc);
        }
      }
    }
    float* y = a.y + (size_t)(m0 + m) * a.N + n;
    *y = a.add ? *y + acc : acc;
  }
}

template <typename T>
int shrink(const LoraArgs& a, cudaStream_t st) {
  shrink_kernel<T><<<dim3(a.M, a.rank / RANKS), SHRINK_THR, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? 1 : -1;
}

template <typename T>
int expand(const LoraArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  // rows of a block: all, where the columns alone give every SM four blocks, else
  // fewer (12288 columns, 20 rows of 4 adapters: 4.0 us, 7 with all rows a block)
  const int cols = (a.N + EXPAND_THR - 1) / EXPAND_THR;
  const int rows = std::min(a.M, std::max(1, (int)((long long)a.M * cols / (4 * num_sms()))));
  cfg.gridDim = dim3(cols, (a.M + rows - 1) / rows);
  cfg.blockDim = dim3(EXPAND_THR);
  cfg.dynamicSmemBytes = (size_t)rows * a.rank * sizeof(float);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.add ? 0 : 1;   // behind the projection: an ordinary launch
  return cudaLaunchKernelEx(&cfg, expand_kernel<T>, a, rows) == cudaSuccess ? 1 : -1;
}

}  // namespace

int lora_shrink(const LoraArgs& a, cudaStream_t st) {
  return a.dtype == DT_F32 ? shrink<float>(a, st) : shrink<__nv_bfloat16>(a, st);
}

int lora_expand(const LoraArgs& a, cudaStream_t st) {
  return a.dtype == DT_F32 ? expand<float>(a, st) : expand<__nv_bfloat16>(a, st);
}

}  // namespace spec
