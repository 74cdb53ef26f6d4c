// lora_gemm.cu -- a bf16 projection and its rows' low-rank adapters in one
// weight stream on the fifth-generation tensor cores.
//
// y[m] = r_m (W (x_m * gain) + s_a B_a (A_a (x_m * gain))) with a = ids[m] and r_m
// RMSNorm's 1/rms (1 without a gain). A preparation kernel writes the
// activations and the shrunken rows t_m = s_a A_a (x_m * gain); the projection
// then treats the adapters in use as more columns of W: a tile of 128 output
// rows reduces over K / 64 chunks of W and, for every adapter in use, over the
// chunks of B_a's 128 rows, against activation columns that hold t_m in the
// rows of that adapter and zero elsewhere. y is written once, and W and each
// B_a in use are read once: the operator's floor is those bytes.
//
// Precision. The activations enter as three bf16 planes (hi, mid, lo: 24 bits,
// x to 2^-25) against exact bf16 weights, and the tensor cores' sums, which
// round towards zero, leave tensor memory every FLUSH chunks and are added up in
// registers: the result is a binary32 projection's. (Measured at 40 x 49152 x
// 6144 against 64 bits: 6.0e-6 with one sum over all of K. The projection
// kernels of a pass use two planes, 2^-17.) The planes are consecutive rows of
// the MMA's B operand, so each 16-column k-step is one MMA with N = 3 x rows.
//
// Work split: units are (tile, chunk of W) pairs in tile-major order, and CTA b
// of G owns [U b / G, U (b + 1) / G), of small matrices whole shares of a tile; the CTA with a tile's last chunk also takes
// the adapters' (counted on the device from the ids, by every CTA alike). A tile
// cut between CTAs is summed by the last CTA to arrive, in CTA order. So a row's
// result depends on neither timing, nor the other rows, nor their adapters, whose
// chunks add exact zeros to it. Infinities and NaN among the activations, the weights
// or an adapter come out of the planes as NaN, an adapter's in every row: a tile with
// a sum that is not finite is taken again, by its CTA and behind its others, where the
// leading plane's infinities and NaN count alone and each adapter has a sum of its own
// that only the rows that bring it take. (All of that from the start: 49152 x 6144, 64
// rows of 64 adapters 311 us instead of 191.)
//
// What bounds it: HBM from about 80 MB of weights on (49152 x 6144, 40 rows, 8
// adapters of rank 16: 109 to 112 us, 5.7 TB/s; 262144 x 2560, rank 64: 255 to 260 us,
// 6.2 TB/s, measured copy 6.8); below that the chain of preparation, stream, split tiles'
// sums (2560 x 1536, 4 rows: 12.7 us, 0.6 TB/s).
//
// Roles of a CTA's 6 warps, one CTA an SM: TMA producer (warp 0, one thread; a
// ring of stages of a weight tile's 64 columns and the activations', both in the
// 128-byte-swizzled K-major layout; an adapter's columns past its rank read as
// zero), MMA issue (warp 1, one thread; two accumulators alternate where they
// fit), epilogue (warps 2-5: lane = output row,
// so stores of an activation row are consecutive). A tile of 256 rows is two MMAs
// a k-step on one load of the activations: half their traffic out of L2, and half
// the barrier work of the two single threads, which bound 128-row tiles. Every wait is bounded; on a
// timeout the CTA records it, drains its copies and MMAs and returns.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "mbar.cuh"

namespace spec {

namespace {

constexpr int TM = 128;               // weight rows of an MMA; a tile is one or two of them
constexpr int KC = 64;                // columns of a chunk (one 128-byte swizzle row of bf16)
constexpr int SUB_BYTES = TM * KC * 2;
constexpr int ROWS = 64;              // activation rows of a call
constexpr int PREP_COLS = 1024;       // columns of a preparation block
constexpr int RMS_PARTS = 32;         // blocks of a row that leave a sum of squares (K <= 32768)
constexpr int MAX_STAGES = 10;
constexpr int SMEM_LIMIT = 227 * 1024;
constexpr int NTHR = 192;
constexpr int EPI0 = 64;              // first epilogue thread
constexpr int TMEM_COLS = 512;
constexpr int FLUSH = 8;              // chunks summed in tensor memory (a multiple of an adapter's chunks)
constexpr unsigned SPIN_LIMIT = 1u << 26;

// The adapters in use, in order of first appearance, and each row's place
// among them (-1: none). Called by every thread; ends with a barrier.
struct Slots {
  int4 id[ROWS / 4];
  int slot[ROWS], used[ROWS], lead[2];
  uint2 rows[ROWS];   // of each adapter in use: a bit a row
  int n;
};
SPEC_DEV void find_slots(Slots& s, const int32_t* ids, int M, int n_adapters) {
  const int t = threadIdx.x;
  int id = -1;
  if (t < M) id = ids[t];
  if (id < 0 || id >= n_adapters) id = -1;
  if (t < ROWS) reinterpret_cast<int*>(s.id)[t] = id;
  __syncthreads();
  int lead = 0;   // the first row of this row's adapter
  unsigned int lo = 0, hi = 0;   // the rows of this adapter
  if (t < ROWS) {
#pragma unroll
    for (int j = 0; j < ROWS / 4; ++j) {
      const int4 o = s.id[j];
      const unsigned int bits = (o.x == id ? 1u : 0u) | (o.y == id ? 2u : 0u) | (o.z == id ? 4u : 0u) | (o.w == id ? 8u : 0u);
      if (j < 8) lo |= bits << (4 * j);
      else hi |= bits << (4 * (j - 8));
    }
    lead = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
    const unsigned int first = __ballot_sync(FULL, id >= 0 && lead == t);
    if ((t & 31) == 0) s.lead[t >> 5] = (int)first;
  }
  __syncthreads();
  if (t < ROWS) {
    const unsigned int l0 = (unsigned int)s.lead[0], l1 = (unsigned int)s.lead[1];
    const int n = lead < 32 ? __popc(l0 & ((1u << lead) - 1)) : __popc(l0) + __popc(l1 & ((1u << (lead - 32)) - 1));
    s.slot[t] = id < 0 ? -1 : n;
    if (id >= 0 && lead == t) {
      s.used[n] = id;
      s.rows[n] = make_uint2(lo, hi);
    }
    if (t == 0) s.n = __popc(l0) + __popc(l1);
  }
  __syncthreads();
}

// v as three bf16 numbers, hi + mid + lo = v to 2^-25 (hi rounds to an infinity for
// an infinity alone).
SPEC_DEV void split3(float v, uint16_t (&o)[3]) {
  const float most = 3.38953139e38f;   // bf16's largest number
  const __nv_bfloat16 h = __float2bfloat16_rn(fabsf(v) < INFINITY ? fmaxf(-most, fminf(v, most)) : v);
  const float r = v - __bfloat162float(h);
  const __nv_bfloat16 m = __float2bfloat16_rn(r);
  o[0] = __bfloat16_as_ushort(h);
  o[1] = __bfloat16_as_ushort(m);
  o[2] = __bfloat16_as_ushort(__float2bfloat16_rn(r - __bfloat162float(m)));
}

// Blocks (m, y): y below the row's column blocks writes the planes of 1024
// columns of row m and their sum of squares; the others take RB ranks each of
// row m's shrink, all warps together along K, two steps of loads in flight, and
// write its planes' adapter columns. Rows that share an adapter read it from L2.
// (A latency chain beside the weight stream's start: 40 rows, K = 6144, rank 16
// 5.7 us; 8 ranks a block and one step in flight 8.1 us.)
constexpr int PREP_THR = 256;
constexpr int RB = 4;
__global__ void __launch_bounds__(PREP_THR) lora_prep_kernel(LoraArgs a, int col_blocks, int MP, int Kp, int KT,
                                                             uint16_t* planes, float* rms) {
  __shared__ Slots sl;
  __shared__ float red[32];
  __shared__ float sums[PREP_THR / 32][RB];
  grid_dep_launch();   // the projection starts on its weights
  const int m = blockIdx.x, y = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t plane = (size_t)MP * KT;
  uint16_t* out = planes + (size_t)m * KT;
  const float* x = a.x + (size_t)m * a.K;
  if (y < col_blocks) {
    if (m == 0 && y == 0) {
      int bad = 0;
      for (int i = threadIdx.x; i < a.M; i += blockDim.x) bad |= a.ids[i] < -1 || a.ids[i] >= a.n_adapters;
      bad = __syncthreads_or(bad);
      if (threadIdx.x == 0) *a.err = bad ? SPEC_ERR_CAPACITY : SPEC_ERR_NONE;
      for (int i = threadIdx.x; i < a.n_cnt; i += blockDim.x) a.cnt[i] = 0u;
    }
    float ss = 0.f;
    const int c = y * PREP_COLS + threadIdx.x * 4;
    if (c < Kp) {   // (the columns up to a whole chunk are zero, as the weights' read)
      const float4 u = c < a.K ? *reinterpret_cast<const float4*>(x + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      float v[4] = {u.x, u.y, u.z, u.w};
      if (a.gain && c < a.K) {
        const float4 g = *reinterpret_cast<const float4*>(a.gain + c);
        ss = fmaf(v[0], v[0], fmaf(v[1], v[1], fmaf(v[2], v[2], v[3] * v[3])));
        v[0] *= g.x; v[1] *= g.y; v[2] *= g.z; v[3] *= g.w;
      }
      uint16_t o[4][3];
#pragma unroll
      for (int i = 0; i < 4; ++i) split3(v[i], o[i]);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        *reinterpret_cast<uint2*>(out + p * plane + c) =
            make_uint2(o[0][p] | ((uint32_t)o[1][p] << 16), o[2][p] | ((uint32_t)o[3][p] << 16));
    }
    if (a.gain) {
      const float tot = block_sum(ss, red);
      if (threadIdx.x == 0) rms[m * RMS_PARTS + y] = tot;
    }
    return;
  }
  const int r0 = (y - col_blocks) * RB, rc = (a.rank + KC - 1) / KC, id = a.ids[m];
  const bool has = id >= 0 && id < a.n_adapters;
  if (has) {
    const __nv_bfloat16* A = (const __nv_bfloat16*)a.a + ((size_t)id * a.rank + r0) * a.K;
    float acc[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) acc[r] = 0.f;
    constexpr int STEP = PREP_THR * 8;
    for (int c0 = threadIdx.x * 8; c0 < a.K; c0 += 2 * STEP) {
      uint4 w[2][RB];
      float4 u[2][2], g[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = c0 + i * STEP;
        if (c >= a.K) break;
#pragma unroll
        for (int r = 0; r < RB; ++r) w[i][r] = *reinterpret_cast<const uint4*>(A + (size_t)r * a.K + c);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          u[i][j] = *reinterpret_cast<const float4*>(x + c + 4 * j);
          if (a.gain) g[i][j] = *reinterpret_cast<const float4*>(a.gain + c + 4 * j);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (c0 + i * STEP >= a.K) break;
        float v[8] = {u[i][0].x, u[i][0].y, u[i][0].z, u[i][0].w, u[i][1].x, u[i][1].y, u[i][1].z, u[i][1].w};
        if (a.gain) {
          v[0] *= g[i][0].x; v[1] *= g[i][0].y; v[2] *= g[i][0].z; v[3] *= g[i][0].w;
          v[4] *= g[i][1].x; v[5] *= g[i][1].y; v[6] *= g[i][1].z; v[7] *= g[i][1].w;
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const uint32_t b[4] = {w[i][r].x, w[i][r].y, w[i][r].z, w[i][r].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[r] = fmaf(bf16lo(b[j]), v[2 * j], fmaf(bf16hi(b[j]), v[2 * j + 1], acc[r]));
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) acc[r] = warp_sum(acc[r]);
    if (lane == 0)
#pragma unroll
      for (int r = 0; r < RB; ++r) sums[warp][r] = acc[r];
    __syncthreads();
    if (threadIdx.x < RB) {
      float t = 0.f;
      for (int w = 0; w < PREP_THR / 32; ++w) t += sums[w][threadIdx.x];
      red[threadIdx.x] = t * (a.scale ? a.scale[id] : 1.f);
    }
  }
  find_slots(sl, a.ids, a.M, a.n_adapters);
  const int mine = sl.slot[m];
  // RB columns of every adapter in use: t in this row's, zero in the others; the
  // last block also clears the columns up to a whole k-step
  const int width = r0 + RB >= a.rank && (a.rank & 15) ? 1 + 8 / RB : 1;
  for (int i = threadIdx.x; i < sl.n * 3 * width; i += blockDim.x) {
    const int part = i % width, p = i / width % 3, s = i / width / 3;
    uint32_t q[RB / 2] = {};
    if (s == mine && part == 0)
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        uint16_t o[3];
        split3(red[j], o);
        q[j >> 1] |= (uint32_t)(p == 0 ? o[0] : p == 1 ? o[1] : o[2]) << (16 * (j & 1));
      }
    *reinterpret_cast<uint2*>(out + p * plane + Kp + s * rc * KC + r0 + part * RB) = make_uint2(q[0], q[1]);
  }
}

// ---- the projection ----------------------------------------------------------

SPEC_DEV void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
SPEC_DEV void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// K-major operand in the 128-byte swizzle layout (8-row groups of 1024 bytes).
SPEC_DEV uint64_t sw128_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16: fp32 accumulate, bf16 A and B, both K-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
SPEC_DEV void mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
SPEC_DEV void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sa(bar))
               : "memory");
}
SPEC_DEV void tma_load(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          sa(dst)),
      "l"(map), "r"(x), "r"(y), "r"(sa(bar))
      : "memory");
}
// The same for weights, read once: first to leave L2.
SPEC_DEV void tma_load_once(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
      "%3}], [%4], %5;" ::"r"(sa(dst)),
      "l"(map), "r"(x), "r"(y), "r"(sa(bar)), "l"(policy)
      : "memory");
}
SPEC_DEV uint64_t l2_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// 8 consecutive accumulator columns of this warp's 32 lanes.
SPEC_DEV void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
SPEC_DEV void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
SPEC_DEV void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
SPEC_DEV bool epi_any(bool v) {
  unsigned int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(v ? 1u : 0u)
      : "memory");
  return any != 0;
}

SPEC_DEV bool wait_phase(uint64_t* b, unsigned parity, volatile int* abort_s, int* err) {
  for (unsigned it = 0; it < SPIN_LIMIT; ++it) {
    if (mbar_test(b, parity)) return true;
    if (*abort_s) return false;
  }
  *abort_s = 1;
  set_error(err, SPEC_ERR_TIMEOUT);
  return false;
}
SPEC_DEV void drain_phase(uint64_t* b, unsigned parity) {
  for (unsigned it = 0; it < SPIN_LIMIT; ++it)
    if (mbar_test(b, parity)) return;
}

struct GemmArgs {
  int M, N, K, rank, n_adapters, T, grid, stages;
  const int32_t* ids;
  bool norm;
  float eps;
  const float* rms;       // [M][RMS_PARTS]
  float* y;               // [M][N]
  float* fix;             // [grid][2][tile rows / TM][MP][TM]
  unsigned int* cnt;      // [T] arrivals, [T] tiles to be taken again
  int* err;
};

// The larger magnitude, NaN if either is.
SPEC_DEV float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// A sum from its planes' sums. Where that of the leading plane is not finite it is the
// result: an infinity among the activations or the weights has NaN in the other
// planes (their zeros meet it, and the infinity's remainder is one).
template <bool ODD>
SPEC_DEV float join(uint32_t hi, uint32_t mid, uint32_t lo) {
  const float h = __uint_as_float(hi), s = h + (__uint_as_float(mid) + __uint_as_float(lo));
  return !ODD || fabsf(h) < INFINITY ? s : h;
}

// MMA N: the three planes of MP rows.
constexpr int mma_n(int MP) { return (3 * MP + 15) / 16 * 16; }

// NS: MMAs a k-step (128-row parts of a tile).
template <int MP, int NS>
struct Gemm {
  static constexpr int NB = mma_n(MP);
  static constexpr int ACC_COLS = NB <= 128 ? 128 : 256;
  static constexpr int SETS = NS * ACC_COLS <= TMEM_COLS / 2 ? 2 : 1;
  static constexpr int ROWS_T = NS * TM;
  static constexpr int W_BYTES = NS * SUB_BYTES;
  static constexpr int X_BYTES = NB * KC * 2;
  static constexpr int STAGE = W_BYTES + X_BYTES;
  const GemmArgs& a;
  const CUtensorMap *tmw, *tmb, *tmx;
  const Slots& sl;
  unsigned char* ring;
  uint64_t *full, *empty, *accf, *acce, *drain;
  float* rms_s;
  volatile int *abort_s, *redo;
  int* bc;
  uint32_t tmem;
  int CW, RC, E, U, u0, u1;   // chunks of a tile: CW of W, then RC of every adapter in use, E in all

  // The (tile, chunk) pairs of the CTA, in the order they are streamed. Counted
  // up without a division: one thread issues a chunk every 700 cycles or so, and
  // with divisions here and for the ring's slots (1200 cycles a chunk) the
  // stream ran at half its rate.
  struct Items {
    const Gemm& k;
    const bool again;   // tiles to be taken again only
    int t, c, last;     // the pair, and the CTA's last chunk of its tile
    SPEC_DEV Items(const Gemm& k_, bool again_) : k(k_), again(again_), t(k_.u0 / k_.CW - 1), c(0), last(0) {}
    SPEC_DEV bool next() {
      if (c != last) {
        ++c;
        return true;
      }
      for (;;) {
        const int at = ++t * k.CW;
        if (at >= k.u1) return false;
        c = max(0, k.u0 - at);
        last = at + k.CW <= k.u1 ? k.CW + k.E - 1 : k.u1 - at - 1;
        if (!again || k.marked(t, last)) return true;
      }
    }
    SPEC_DEV bool ends() const { return c == last; }
    // the last of a sum in tensor memory: the same chunks of W, and of a row's adapter,
    // meet there whatever else the call holds
    SPEC_DEV bool flushes() const {
      if (c == last || c == k.CW - 1) return true;
      if (c < k.CW) return (c + 1) % FLUSH == 0;
      return again ? k.part_of(c) == k.RC - 1 : (c - k.CW + 1) % FLUSH == 0;
    }
  };
  // Tiles to be taken again: a word each behind the arrival counters, written and read
  // by the CTA with the tile's last chunk of W; of a CTA that ends inside a tile, its
  // part of that one (redo[1]).
  SPEC_DEV bool marked(int t, int last) const {
    return last < CW - 1 ? redo[1] != 0 : *(volatile unsigned int*)(a.cnt + a.T + t) != 0u;
  }
  SPEC_DEV void mark(int t, int last) const {
    redo[0] = 1;
    if (last < CW - 1) redo[1] = 1;
    else *(volatile unsigned int*)(a.cnt + a.T + t) = 1u;
  }
  // A place in the ring, and the parity of its turn.
  struct Slot {
    int s = 0;
    unsigned turn = 0;
    SPEC_DEV void next(int stages) {
      if (++s == stages) {
        s = 0;
        turn ^= 1;
      }
    }
  };

  SPEC_DEV int unit_begin(int b) const { return (int)(((long long)b * U) / a.grid); }
  SPEC_DEV int cta_of(int u) const {
    int b = (int)((((long long)u + 1) * a.grid - 1) / U);
    b = min(b, a.grid - 1);
    while (b > 0 && unit_begin(b) > u) --b;
    while (b + 1 < a.grid && unit_begin(b + 1) <= u) ++b;
    return b;
  }
  // 16-column k-steps of chunk c
  SPEC_DEV int steps(int c) const {
    return c < CW ? KC / 16 : min(KC / 16, (a.rank - part_of(c) * KC + 15) / 16);
  }
  // chunk c's adapter among those in use, and its place in it (RC is 1 or 2: ranks to 128)
  SPEC_DEV int slot_of(int c) const { return (c - CW) >> (RC - 1); }
  SPEC_DEV int part_of(int c) const { return (c - CW) & (RC - 1); }
  SPEC_DEV unsigned char* stage(int s) const { return ring + (size_t)s * STAGE; }

  SPEC_DEV void load_w(int s, const Items& it, uint64_t pol) const {
    if (it.c < CW) {
      tma_load_once(stage(s), tmw, it.c * KC, it.t * ROWS_T, &full[s], pol);
    } else {
      tma_load_once(stage(s), tmb, part_of(it.c) * KC, sl.used[slot_of(it.c)] * a.N + it.t * ROWS_T, &full[s], pol);
    }
  }
  SPEC_DEV void load_x(int s, const Items& it) const { tma_load(stage(s) + W_BYTES, tmx, it.c * KC, 0, &full[s]); }

  // Where a role stands: chunks, or sums, so far, and the next place in the ring (for
  // the producer, the next one to be emptied).
  struct Role {
    int n = 0;
    Slot at;
  };

  SPEC_DEV void producer(Role& p, bool again) {
    const uint64_t pol = l2_evict_first();
    Items it(*this, again);
    bool more = it.next();
    if (!again) {   // the ring filled: the weights, and behind the wait the activations
      Items ix(*this, false);
      while (more && p.n < a.stages) {
        mbar_expect_tx(&full[p.n], (unsigned)STAGE);
        load_w(p.n++, it, pol);
        more = it.next();
      }
      grid_dep_wait();  // the activation planes come from the preparation
      for (int n = 0; n < p.n; ++n) {
        ix.next();
        load_x(n, ix);
      }
    }
    while (more) {
      int s = p.n;
      if (s >= a.stages) {
        s = p.at.s;
        if (!wait_phase(&empty[s], p.at.turn, abort_s, a.err)) break;
        p.at.next(a.stages);
      }
      mbar_expect_tx(&full[s], (unsigned)STAGE);
      load_w(s, it, pol);
      load_x(s, it);
      ++p.n;
      more = it.next();
    }
    if (*abort_s)  // this CTA's copies land before its shared memory is released
      for (int n = max(0, p.n - a.stages); n < p.n; ++n) drain_phase(&full[n % a.stages], (n / a.stages) & 1);
  }

  SPEC_DEV void mma_loop(Role& p, bool again) {
    constexpr uint32_t idesc = idesc_bf16(TM, NB);
    Items it(*this, again);
    int& i = p.n;      // sums so far
    int ks = 0;        // k-steps of the current one
    uint32_t d = tmem;
    for (; it.next(); p.at.next(a.stages)) {
      if (ks == 0) {
        const int set = i % SETS;
        if (i >= SETS && !wait_phase(&acce[set], (i / SETS - 1) & 1, abort_s, a.err)) break;
        fence_after();
        d = tmem + (uint32_t)(set * NS * ACC_COLS);
      }
      if (!wait_phase(&full[p.at.s], p.at.turn, abort_s, a.err)) break;
      fence_after();
      const uint32_t w = sa(stage(p.at.s)), x = w + (uint32_t)W_BYTES;
      const int ns = steps(it.c);
      const uint64_t wd = sw128_desc(w), xd = sw128_desc(x);
      auto step = [&](int j) {   // 32 bytes a k-step: 2 in the descriptors' units
#pragma unroll
        for (int h = 0; h < NS; ++h)
          mma_bf16(d + (uint32_t)(h * ACC_COLS), wd + h * (SUB_BYTES >> 4) + 2 * j, xd + 2 * j, idesc,
                   ks + j > 0 ? 1u : 0u);
      };
      if (ns == KC / 16) {
#pragma unroll
        for (int j = 0; j < KC / 16; ++j) step(j);
      } else {
        for (int j = 0; j < ns; ++j) step(j);
      }
      ks += ns;
      mma_commit(&empty[p.at.s]);
      if (it.flushes()) {
        mma_commit(&accf[i % SETS]);
        ++i;
        ks = 0;
      }
    }
  }
  // Every MMA of this CTA is complete before its tensor memory is freed.
  SPEC_DEV void mma_drain() const {
    mma_commit(drain);
    drain_phase(drain, 0);
  }

  // thread = output row n of the tile's parts, lane by lane: a warp's stores of
  // an activation row are consecutive
  SPEC_DEV void finish(int t, int r, const float (&v)[NS][MP]) const {
#pragma unroll
    for (int h = 0; h < NS; ++h) {
      const int n = t * ROWS_T + h * TM + r;
      if (n >= a.N) break;
#pragma unroll
      for (int m = 0; m < MP; ++m)
        if (m < a.M) a.y[(size_t)m * a.N + n] = v[h][m] * rms_s[m];
    }
  }

  SPEC_DEV float* slot(int b, int t) const {
    return a.fix + (size_t)(b * 2 + (t == unit_begin(b) / CW ? 0 : 1)) * NS * MP * TM;
  }
  // A tile shared with other CTAs: publish this CTA's sums; the last to arrive
  // adds all of them in CTA order and finishes the tile. i: the CTA's tiles so far.
  SPEC_DEV void partial(int t, int i, int r, int e, float (&v)[NS][MP]) const {
    float* f = slot(blockIdx.x, t);
#pragma unroll
    for (int h = 0; h < NS; ++h)
#pragma unroll
      for (int m = 0; m < MP; ++m) __stcg(f + (h * MP + m) * TM + r, v[h][m]);
    epi_sync();
    if (e == 0) bc[2 + (i & 1)] = (int)atomic_add_acq_rel(a.cnt + t, 1u);
    epi_sync();
    const int bf = cta_of(t * CW), bl = cta_of(t * CW + CW - 1);
    if (bc[2 + (i & 1)] != bl - bf) return;
    __threadfence();
#pragma unroll
    for (int h = 0; h < NS; ++h)
#pragma unroll
      for (int m = 0; m < MP; ++m) v[h][m] = 0.f;
#pragma unroll NS == 1 ? 2 : 1
    for (int bb = bf; bb <= bl; ++bb) {
      const float* g = slot(bb, t);
#pragma unroll
      for (int h = 0; h < NS; ++h) {
        float o[MP];
#pragma unroll
        for (int m = 0; m < MP; ++m) o[m] = __ldcg(g + (h * MP + m) * TM + r);
#pragma unroll
        for (int m = 0; m < MP; ++m) v[h][m] += o[m];
      }
    }
    if (e == 0) a.cnt[t] = 0u;
    finish(t, r, v);
  }

  SPEC_DEV void row_scales() const {
    const int e = threadIdx.x - EPI0;
    grid_dep_wait();
    if (e < ROWS) {
      float f = 1.f;
      if (a.norm && e < a.M) {
        float tot = 0.f;
        for (int y = 0; y < (a.K + PREP_COLS - 1) / PREP_COLS; ++y) tot += __ldcg(a.rms + e * RMS_PARTS + y);
        f = rsqrtf(tot / (float)a.K + a.eps);
      }
      rms_s[e] = f;
    }
    epi_sync();
  }

  // The rows that take the sum over adapters that ends with chunk c: those that bring
  // one of them.
  SPEC_DEV uint2 takers(int c, bool again) const {
    const int s1 = slot_of(c);
    uint2 r = make_uint2(0u, 0u);
    for (int i = again ? s1 : slot_of(CW + (c - CW) / FLUSH * FLUSH); i <= s1; ++i) {
      r.x |= sl.rows[i].x;
      r.y |= sl.rows[i].y;
    }
    return r;
  }
  // This thread's sums of a tile's rows, from tensor memory, added to v; of those
  // with a bit in `take` (ALL: every row).
  template <bool ODD, bool ALL>
  SPEC_DEV void add_sums(uint32_t acc, uint2 rows, float (&v)[NS][MP]) const {
#pragma unroll
    for (int h = 0; h < NS; ++h)
#pragma unroll
      for (int j = 0; j < MP / 8; ++j) {
        const unsigned int take = ALL ? 0xffu : (j < 4 ? rows.x : rows.y) >> (8 * (j & 3)) & 0xffu;
        if (!ALL && take == 0) continue;
        uint32_t q[3][8];   // hi, mid, lo
#pragma unroll
        for (int p = 0; p < 3; ++p) tmem_ld8(acc + h * ACC_COLS + p * MP + 8 * j, q[p]);
        tmem_wait_ld();
#pragma unroll
        for (int l = 0; l < 8; ++l)
          if (ALL || take >> l & 1) v[h][8 * j + l] += join<ODD>(q[0][l], q[1][l], q[2][l]);
      }
  }

  SPEC_DEV bool finite(const float (&v)[NS][MP]) const {
    float top = 0.f;
#pragma unroll
    for (int m = 0; m < MP; ++m)
      if (m < a.M)
#pragma unroll
        for (int h = 0; h < NS; ++h) top = max_abs(top, v[h][m]);
    return top < INFINITY;
  }

  // p.n: sums so far, p.at.s: tiles so far
  SPEC_DEV void epilogue(Role& p, bool again) const {
    const int e = threadIdx.x - EPI0, r = ((threadIdx.x >> 5) & 3) * 32 + (threadIdx.x & 31);
    const uint32_t lanes = tmem + ((uint32_t)(((threadIdx.x >> 5) & 3) * 32) << 16);
    Items it(*this, again);
    int& i = p.n;
    int& tile = p.at.s;
    int c0 = -1;
    float v[NS][MP];
    while (it.next()) {
      if (c0 < 0) {
        c0 = it.c;
#pragma unroll
        for (int h = 0; h < NS; ++h)
#pragma unroll
          for (int m = 0; m < MP; ++m) v[h][m] = 0.f;
      }
      if (!it.flushes()) continue;
      const int set = i % SETS;
      if (e == 0) bc[i & 1] = wait_phase(&accf[set], (i / SETS) & 1, abort_s, a.err) ? 1 : 0;
      epi_sync();
      if (!bc[i & 1]) break;
      fence_after();
      const uint32_t acc = lanes + (uint32_t)(set * NS * ACC_COLS);
      if (it.c < CW) {
        if (again) add_sums<true, true>(acc, make_uint2(0u, 0u), v);
        else add_sums<false, true>(acc, make_uint2(0u, 0u), v);
      } else {
        if (again) add_sums<true, false>(acc, takers(it.c, true), v);
        else add_sums<false, false>(acc, takers(it.c, false), v);
      }
      fence_before();
      mbar_arrive(&acce[set]);
      ++i;
      if (!it.ends()) continue;
      if (!again && epi_any(!finite(v))) {
        if (e == 0) mark(it.t, it.c);
      } else {
        if (c0 == 0 && it.c >= CW - 1) finish(it.t, r, v);
        else partial(it.t, tile, r, e, v);
        ++tile;
      }
      c0 = -1;
    }
  }
};

template <int MP, int NS>
__global__ void __launch_bounds__(NTHR, 1)
    lora_gemm_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ CUtensorMap tmw,
                     const __grid_constant__ CUtensorMap tmb, const __grid_constant__ CUtensorMap tmx) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ Slots sl;
  __shared__ __align__(8) uint64_t bars[2 * MAX_STAGES + 5];
  __shared__ float rms_s[ROWS];
  __shared__ uint32_t tmem_slot;
  __shared__ int flags[7];
  const uint32_t mis = sa(smem_raw) & 1023u;
  Gemm<MP, NS> k{a, &tmw, &tmb, &tmx, sl, smem_raw + (mis ? 1024 - mis : 0)};
  k.full = bars;
  k.empty = bars + MAX_STAGES;
  k.accf = bars + 2 * MAX_STAGES;
  k.acce = k.accf + 2;
  k.drain = k.acce + 2;
  k.rms_s = rms_s;
  k.abort_s = flags;
  k.redo = flags + 1;
  k.bc = flags + 3;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&k.full[s], 1);
      mbar_init(&k.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k.accf[i], 1);
      mbar_init(&k.acce[i], 128);
    }
    mbar_init(k.drain, 1);
    flags[0] = flags[1] = flags[2] = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // (the ids are the call's input, complete before the preparation started)
  find_slots(sl, a.ids, a.M, a.n_adapters);
  fence_before();
  __syncthreads();
  fence_after();
  k.tmem = tmem_slot;
  k.CW = (a.K + KC - 1) / KC;
  k.RC = (a.rank + KC - 1) / KC;
  k.E = sl.n * k.RC;
  k.U = a.T * k.CW;
  k.u0 = k.unit_begin(blockIdx.x);
  k.u1 = k.unit_begin(blockIdx.x + 1);
  typename Gemm<MP, NS>::Role role;
  if (warp >= 2) k.row_scales();
#pragma unroll 1
  for (int again = 0; again < 2; ++again) {
    if (warp == 0) {
      if (lane == 0) k.producer(role, again);
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) k.mma_loop(role, again);
      __syncwarp();
    } else {
      k.epilogue(role, again);
    }
    __syncthreads();
    if (!k.redo[0] || *k.abort_s) break;
  }
  if (threadIdx.x == 32) k.mma_drain();
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(k.tmem), "r"(TMEM_COLS) : "memory");
  }
}

// ---- host ----------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_once;

void init_encode() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    g_encode = (PFN_cuTensorMapEncodeTiled_v12000)fn;
}

// Row-major bf16 [rows][inner]; boxes of box_rows x 64 columns in the 128-byte
// swizzle layout, zero past the ends.
bool encode(CUtensorMap* m, const void* base, long long inner, long long rows, int box_rows) {
  if (!g_encode || ((uintptr_t)base & 15) || (inner * 2) % 16) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)inner * 2};
  const cuuint32_t box[2] = {(cuuint32_t)KC, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int rows_padded(int M) {
  for (int mp : {8, 16, 32, 40, 48})
    if (M <= mp) return mp;
  return 64;
}

// Tiles of 256 rows where every SM has 16 of their chunks or more (80 MB of
// weights), else of 128. 49152 x 6144, 40 rows, 8 adapters of rank 16: 111 us with
// 256 (5.6 TB/s), 163 us with 128.
int parts(int N, int K) { return (long long)N * K >= 16ll * num_sms() * 2 * TM * KC ? 2 : 1; }

// CTAs of T tiles of CW chunks: whole shares of a tile each, as many as the SMs hold
// and no more than pay for their part of the tile's sum (a chunk takes a CTA about
// 0.4 us, a share 0.3 to 0.8 us of the last one); every SM where that would leave
// more than 40% of them idle. In us, with every SM: 333 x 7392, 60 rows 43 (107);
// 2560 x 1536, 4 rows 13.4 (15.5); 4096 x 4096, 40 rows 24.6 (29.9); 12288 x 1536,
// 20 rows 23.2 (25.4); but 10240 x 2560, 4 rows 26.6 (23.6), 53% of the SMs.
int ctas(int T, int CW) {
  const int sms = num_sms(), fit = sms / T, pays = std::max(1, (int)(0.75 * std::sqrt((double)CW) + 0.5));
  if (fit >= 1 && (pays < fit || 10 * fit * T >= 6 * sms)) return T * std::min(fit, pays);
  return (int)std::min<long long>((long long)T * CW, sms);
}

// Scratch of the fused path: sums of squares, counters, split-tile sums, planes.
struct Scratch {
  size_t rms, cnt, fix, planes, bytes;
};
Scratch scratch(int N, int K, int M, int rank) {
  const int MP = rows_padded(M), rc = (rank + KC - 1) / KC;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  Scratch s;
  s.rms = 0;
  s.cnt = s.rms + up((size_t)ROWS * RMS_PARTS * sizeof(float));
  s.fix = s.cnt + up((size_t)((N + TM - 1) / TM) * 2 * sizeof(unsigned int));
  s.planes = s.fix + up((size_t)num_sms() * 2 * 2 * MP * TM * sizeof(float));
  s.bytes = s.planes + up((size_t)mma_n(MP) * ((K + KC - 1) / KC * KC + (size_t)M * rc * KC) * 2);
  return s;
}

template <int MP, int NS>
cudaError_t launch_gemm(GemmArgs& g, const CUtensorMap& tmw, const CUtensorMap& tmb, const CUtensorMap& tmx,
                        cudaStream_t st) {
  g.stages = std::min(MAX_STAGES, (SMEM_LIMIT - 4096) / Gemm<MP, NS>::STAGE);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.grid);
  cfg.blockDim = dim3(NTHR);
  cfg.dynamicSmemBytes = (size_t)g.stages * Gemm<MP, NS>::STAGE + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_gemm_kernel<MP, NS>, g, tmw, tmb, tmx);
}

template <int MP>
void set_attributes() {
  const int n = SMEM_LIMIT - 3 * 1024;
  cudaFuncSetAttribute(lora_gemm_kernel<MP, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
  cudaFuncSetAttribute(lora_gemm_kernel<MP, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
}

}  // namespace

void setup_lora_attributes() {
  set_attributes<8>();
  set_attributes<16>();
  set_attributes<32>();
  set_attributes<40>();
  set_attributes<48>();
  set_attributes<64>();
}

size_t lora_gemm_bytes(int N, int K, int M, int rank) { return scratch(N, K, M, rank).bytes; }

bool lora_gemm_ok(const LoraArgs& a, int w_dtype) {
  return w_dtype == DT_BF16 && a.dtype == DT_BF16 && a.K % 8 == 0 && a.K <= PREP_COLS * RMS_PARTS &&
         (long long)a.n_adapters * a.N + 2 * TM < (1ll << 31);
}

int lora_gemm(LoraArgs a, const void* w, void* ws, cudaStream_t st) {
  std::call_once(g_once, init_encode);
  const int MP = rows_padded(a.M), rc = (a.rank + KC - 1) / KC, Kp = (a.K + KC - 1) / KC * KC;
  const int KT = Kp + std::min(a.M, a.n_adapters) * rc * KC;
  const Scratch s = scratch(a.N, a.K, a.M, a.rank);
  char* base = (char*)ws;
  uint16_t* planes = (uint16_t*)(base + s.planes);
  GemmArgs g = {};
  g.M = a.M; g.N = a.N; g.K = a.K; g.rank = a.rank; g.n_adapters = a.n_adapters;
  const int ns = parts(a.N, a.K), rows_t = ns * TM;
  g.T = (a.N + rows_t - 1) / rows_t;
  g.grid = ctas(g.T, Kp / KC);
  g.ids = a.ids; g.norm = a.gain != nullptr; g.eps = a.eps;
  g.rms = (const float*)(base + s.rms); g.y = a.y; g.fix = (float*)(base + s.fix);
  g.cnt = (unsigned int*)(base + s.cnt); g.err = a.err;
  a.cnt = g.cnt;
  a.n_cnt = 2 * g.T;
  CUtensorMap tmw, tmb, tmx;
  if (!encode(&tmw, w, a.K, a.N, rows_t) ||
      !encode(&tmb, a.b, a.rank, (long long)a.n_adapters * a.N, rows_t) ||
      !encode(&tmx, planes, KT, mma_n(MP), mma_n(MP)))
    return -1;
  const int col_blocks = (a.K + PREP_COLS - 1) / PREP_COLS;
  lora_prep_kernel<<<dim3(a.M, col_blocks + a.rank / RB), PREP_THR, 0, st>>>(a, col_blocks, MP, Kp, KT, planes, (float*)(base + s.rms));
  if (cudaGetLastError() != cudaSuccess) return -1;
  cudaError_t e;
  switch (MP) {
    case 8: e = ns == 2 ? launch_gemm<8, 2>(g, tmw, tmb, tmx, st) : launch_gemm<8, 1>(g, tmw, tmb, tmx, st); break;
    case 16: e = ns == 2 ? launch_gemm<16, 2>(g, tmw, tmb, tmx, st) : launch_gemm<16, 1>(g, tmw, tmb, tmx, st); break;
    case 32: e = ns == 2 ? launch_gemm<32, 2>(g, tmw, tmb, tmx, st) : launch_gemm<32, 1>(g, tmw, tmb, tmx, st); break;
    case 40: e = ns == 2 ? launch_gemm<40, 2>(g, tmw, tmb, tmx, st) : launch_gemm<40, 1>(g, tmw, tmb, tmx, st); break;
    case 48: e = ns == 2 ? launch_gemm<48, 2>(g, tmw, tmb, tmx, st) : launch_gemm<48, 1>(g, tmw, tmb, tmx, st); break;
    default: e = ns == 2 ? launch_gemm<64, 2>(g, tmw, tmb, tmx, st) : launch_gemm<64, 1>(g, tmw, tmb, tmx, st); break;
  }
  return e == cudaSuccess ? 2 : -1;
}

}  // namespace spec
