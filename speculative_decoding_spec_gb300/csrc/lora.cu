// lora.cu -- low-rank adapters of many requests beside one shared projection:
// y[m] = W xn[m] + s_a B_a (A_a xn[m]) with a = ids[m], the adapter row m's
// request brings (-1: none), and xn = x or RMSNorm(x) * gain.
//
// Two small kernels around the shared weight stream (gemv): the shrink
// t[m] = s_a A_a xn[m] (rank numbers a row) and the expand B_a t[m]. The expand
// writes y and the projection adds to it in its residual-add epilogue, so y
// makes one trip less than with the adapters added behind the projection, and
// the projection's weight stream can start while they run. (Rows of y that do
// not start on 16 bytes, N % 4 != 0, take the other order: the residual-add
// epilogue prefetches y in 16-byte pieces.)
#include "common.cuh"

namespace spec {

namespace {

constexpr int SHRINK_RANKS = 8;   // rank rows of a CTA, one a warp

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

// t[m][r] for one row m and 8 of its rank rows; CTA (0, 0) also clears the
// projection's arrival counters and records an id out of range.
template <typename T>
__global__ void __launch_bounds__(256) shrink_kernel(LoraArgs a) {
  __shared__ float red[32];
  const int m = blockIdx.x, r = blockIdx.y * SHRINK_RANKS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
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
  float inv = 1.f;
  if (a.gain) {
    float ss = 0.f;
    for (int c = threadIdx.x * 4; c < a.K; c += blockDim.x * 4) {
      const float4 v = *reinterpret_cast<const float4*>(x + c);
      ss += v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
    }
    inv = rsqrtf(block_sum(ss, red) / (float)a.K + a.eps);
  }
  const T* A = (const T*)a.a + ((size_t)id * a.rank + r) * a.K;
  float acc = 0.f;
  for (int c = lane * 8; c < a.K; c += 256) {
    float w[8], v[8];
    load8(A + c, w);
    load8(x + c, v);
    if (a.gain) {
      float g[8];
      load8(a.gain + c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= g[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = fmaf(w[i], v[i], acc);
  }
  acc = warp_sum(acc) * inv * (a.scale ? a.scale[id] : 1.f);
  if (lane == 0) a.t[(size_t)m * a.rank + r] = acc;
}

// y[m][n] (= or +=) B_a[n] . t[m]: a thread a column, the rows of t in shared memory.
template <typename T>
__global__ void __launch_bounds__(128) expand_kernel(LoraArgs a) {
  extern __shared__ __align__(16) float ts[];
  for (int i = threadIdx.x; i < a.M * a.rank; i += blockDim.x) ts[i] = a.t[i];
  __syncthreads();
  const int n = blockIdx.x * blockDim.x + threadIdx.x;
  if (n >= a.N) return;
  for (int m = 0; m < a.M; ++m) {
    const int id = a.ids[m];
    float acc = 0.f;
    if (id >= 0 && id < a.n_adapters) {
      const T* B = (const T*)a.b + ((size_t)id * a.N + n) * a.rank;
      const float* t = ts + m * a.rank;
      for (int r = 0; r < a.rank; r += 8) {
        float w[8];
        load8(B + r, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = fmaf(w[i], t[r + i], acc);
      }
    } else if (a.add) {
      continue;
    }
    float* y = a.y + (size_t)m * a.N + n;
    *y = a.add ? *y + acc : acc;
  }
}

template <typename T>
int launch(const LoraArgs& a, bool shrink, cudaStream_t st) {
  if (shrink)
    shrink_kernel<T><<<dim3(a.M, a.rank / SHRINK_RANKS), 256, 0, st>>>(a);
  else
    expand_kernel<T><<<(a.N + 127) / 128, 128, (size_t)a.M * a.rank * sizeof(float), st>>>(a);
  return cudaGetLastError() == cudaSuccess ? 1 : -1;
}

}  // namespace

int lora_shrink(const LoraArgs& a, cudaStream_t st) {
  return a.dtype == DT_F32 ? launch<float>(a, true, st) : launch<__nv_bfloat16>(a, true, st);
}

int lora_expand(const LoraArgs& a, cudaStream_t st) {
  return a.dtype == DT_F32 ? launch<float>(a, false, st) : launch<__nv_bfloat16>(a, false, st);
}

}  // namespace spec
