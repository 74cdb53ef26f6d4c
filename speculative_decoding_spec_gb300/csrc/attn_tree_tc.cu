// attn_tree_tc.cu -- attention of the rows of drafted trees on the fifth-
// generation tensor cores: bf16 caches, head dims 64 and 128.
//
//   S = Q K^T       (M = 128 query rows, N = 128 keys, 64 with float rows, K = head dim)
//   O += P V        (M = 128 query rows, N = head dim, K = those keys)
//
// with P = exp(S - m) written back over S in tensor memory, where the second
// product takes it from. A thread owns a query row (a lane of tensor memory),
// so maxima and sums need no exchange between threads. Q and P are bf16, or three
// bf16 planes each of float rows and their weights (all 24 bits), K and V as they lie
// in the cache: pages arrive by TMA in the 128-byte swizzle layout, K a K-major
// operand, V (stored [key][dim]) an MN-major one.
//
// A product cuts its sum to 24 bits, so float rows take care: their smallest parts
// first for S, and O out of tensor memory after every 8 blocks. 8 x 24 rows (contexts
// of 1024 to 8192) are off by 1.1e-6 relative to all outputs, 3.3e-6 without either;
// two planes of P, in blocks of 128 keys, 3.6e-6 (32 us instead of 47; a binary32
// library product 1.4e-6).
//
// Few rows leave most of the 128 lanes idle, and may: 128 keys are 64 KB at head
// dim 128, about 2800 cycles at an SM's share of the HBM rate, while their products
// take 1024 cycles and their softmax 1900 in either stream (500 for the maximum, 1400
// for the weights). 8 x 64 rows take 1.02 us (1960 cycles) a block and tile, from the
// slope over contexts of 4096 to 16384: a product of S takes 80 cycles there, 64 alone, as
// its operands fill shared memory's bandwidth and copies arrive beside them, and a
// stream's chain (weights, P V, S, maximum) has a wait at each step. Neither a softmax in
// one pass nor fewer tries changes the total. The other 38 of their 121 us are the launch,
// the beginnings and ends of two or three units a CTA, and the join. Float rows take 1.8 us
// (3400 cycles) for 64 keys and a tile, of which three planes' products are 1920 (those of S 48
// cycles for 64 keys, 64 for 128: the queries are read again), and 19 of the 47 us of 8 x 24
// rows are the call's beginning, end and join; the tensor pipe is active for a third of the
// time. Warps whose lanes hold no row skip the softmax.
//
// Two streams hide the softmax behind the products: while one stream's softmax
// runs, the tensor cores work on the other's. With one tile of query rows the
// streams take alternate blocks of keys and keep a maximum, a sum and an O each,
// added up at the end; with two tiles a unit (bf16 rows, more than 128 on a KV
// head) each stream is a tile and a block is read once for both.
//
// Roles (384 threads, one CTA an SM): warp 0 loads (a ring of tiles, K and V in
// the order in which they are used), warp 1 issues the products, warp 2 checks the CTA's
// share of the arguments (without cuts CTA 0's all of them), warps 4-7 and 8-11 are the streams' softmax. Waits are
// bounded; one that runs out sets SPEC_ERR_TIMEOUT and an abort flag that lets
// every other wait pass, so that the CTA drains its copies and ends.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "attn_tree.cuh"
#include "mbar.cuh"

namespace spec {
namespace tree {
namespace {

constexpr int ROWS = 128;               // query rows a tile
constexpr int NTHR = 384, NSM = 256;    // threads; softmax threads
constexpr int BOX = PAGE * 128;         // 64 dims of a page: 64 rows of 128 bytes
constexpr int ST_MAX = 16;
constexpr int keys_of(bool f32) { return f32 ? 64 : 128; }  // keys a block: a page or two
constexpr float TAU = 8.f;              // the running maximum is raised past a growth of 2^8
constexpr long long WAIT_CYCLES = 2000000000ll;  // a wait's limit: a second or so

// Shared memory: small items in the first 3 KB, then the query tiles and the ring.
struct Small {
  uint64_t full[ST_MAX], empty[ST_MAX], sfull[2], pfull[2][2], odone[2], qfull, drain;
  uint32_t tmem;
  int abort;
  unsigned long long bad;               // rows of the tree whose values are not finite
  float2 ml[2][ROWS];                   // the streams' maxima and sums
  int up[64];                           // parents
};
constexpr size_t SMALL = 3 * 1024, SMEM_MAX = 227 * 1024;
static_assert(sizeof(Small) <= SMALL, "");

struct Shape {
  int stages, q_bytes;                  // of the ring; of the query tiles
  float scale2;
  int wait_extra;                       // arrivals that the first weights' barrier waits for and that never come (tests)
};

SPEC_DEV void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
SPEC_DEV void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
SPEC_DEV void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
SPEC_DEV void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
SPEC_DEV void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
SPEC_DEV void sm_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// Warps 0-3 set up and go on; warps 4-11 wait for that when they first need it.
SPEC_DEV void set_up() {
  asm volatile("bar.sync 2, 128;" ::: "memory");
  asm volatile("bar.arrive 3, 384;" ::: "memory");
}
SPEC_DEV void all_ready() { asm volatile("bar.sync 3, 384;" ::: "memory"); }

// Operands in the 128-byte swizzle layout (bits 61-63 = 2, 46-48 = 0b001), groups
// of 8 rows 1024 bytes apart; MN-major: halves of 64 elements `lbo` bytes apart.
SPEC_DEV uint64_t desc_k(uint32_t at) {
  return (uint64_t)((at & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
SPEC_DEV uint64_t desc_mn(uint32_t at, uint32_t lbo) {
  return (uint64_t)((at & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// fp32 accumulators, bf16 operands; bit 16: B is MN-major.
constexpr uint32_t idesc(int M, int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? (1u << 16) : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// The whole warp comes here with the same operands, which stay in uniform
// registers that way; the lane with `go` issues (a product takes 35 cycles to issue
// so, 55 where one thread alone runs the loop; a commit 4, else 50).
SPEC_DEV void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc, uint32_t go) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc), "r"(go)
      : "memory");
}
// A in tensor memory: a lane's 32-bit column holds two consecutive elements of its row.
SPEC_DEV void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc, uint32_t go) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc), "r"(go)
      : "memory");
}
SPEC_DEV void commit(uint64_t* bar, uint32_t go) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(sa(bar)),
      "r"(go)
      : "memory");
}
SPEC_DEV uint32_t elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(e));
  return e;
}
SPEC_DEV void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          sa(dst)),
      "l"(map), "r"(x), "r"(y), "r"(sa(bar))
      : "memory");
}
SPEC_DEV void ld32(uint32_t at, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// The largest of 32 columns of this thread's lane (the load reduces them on its
// way; what it loads is not looked at, and waited for in the same breath).
SPEC_DEV float ldmax32(uint32_t at) {
  uint32_t r[32];
  float m;
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%2"
      "7,%28,%29,%30,%31}, %32, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=f"(m)
      : "r"(at)
      : "memory");
  (void)r[0];
  return m;
}
SPEC_DEV void st16(uint32_t at, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
SPEC_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two products and sums at once.
SPEC_DEV float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
SPEC_DEV float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\t"
      "mov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
SPEC_DEV uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Byte offset of (row, byte) in 128-byte rows: 16-byte chunk c of row r lies at c ^ (r % 8).
SPEC_DEV uint32_t swz(int row, int byte) { return (uint32_t)(row * 128 + ((((byte >> 4) ^ (row & 7)) << 4) | (byte & 15))); }

// (a try suspends the thread for a while, so that waiting warps leave the issue slots to others)
SPEC_DEV bool mbar_try(uint64_t* b, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(sa(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
SPEC_DEV bool wait_phase(uint64_t* b, unsigned parity, volatile int* abort, int* err) {
  if (mbar_try(b, parity)) return true;
  const long long t0 = clock64();
  do {
    if (mbar_try(b, parity)) return true;
    if (*abort) return false;
  } while (clock64() - t0 < WAIT_CYCLES);
  *abort = 1;
  set_error(err, SPEC_ERR_TIMEOUT);
  return false;
}
SPEC_DEV void drain_phase(uint64_t* b, unsigned parity) {
  const long long t0 = clock64();
  while (!mbar_try(b, parity) && clock64() - t0 < WAIT_CYCLES) {
  }
}

// Places in the ring of a piece's tiles. One tile of rows: K0 K1 V0 K2 V1 ..; two: K0 V0 K1 V1 ..
SPEC_DEV int place_k(int n, bool pair) { return pair ? 2 * n : n < 2 ? n : 2 * n - 1; }
SPEC_DEV int place_v(int n, int N, bool pair) { return pair ? 2 * n + 1 : min(N, n + 2) + n; }

template <int HD, bool F32>
struct Cta {
  static constexpr int BK = keys_of(F32), PPB = BK / PAGE;
  static constexpr int NH = HD / 64, HALF = BK * 128, TILE = NH * HALF;      // of a block's keys or values
  static constexpr int QPL = F32 ? 3 : 1, QHALF = ROWS * 128, QTILE = NH * QHALF;  // of a tile of query rows
  // Float rows: blocks after which O leaves tensor memory and is added up in binary32 (three
  // products cut it for 16 keys; 8 x 24 rows took 45 us, 43 with 16 blocks, 40 with 32).
  static constexpr int RUN = 8;
  static constexpr uint32_t O_COL = 256;
  const TreeArgs& a;
  const Plan& p;
  const Shape& sh;
  const CUtensorMap* tm;
  Small* sm;
  unsigned char *qt, *ring;
  uint32_t tmem;
  Walk w;

  SPEC_DEV bool wait(uint64_t* b, unsigned parity) { return wait_phase(b, parity, (volatile int*)&sm->abort, findings(a, p)); }
  SPEC_DEV unsigned char* stage(unsigned i) { return ring + (size_t)(i % sh.stages) * TILE; }
  SPEC_DEV unsigned parity(unsigned i) { return (i / sh.stages) & 1; }

  // ---- warp 0 ----
  SPEC_DEV void load(unsigned i, int page0, int page1, int plane) {
    const int s = i % sh.stages;
    unsigned char* dst = stage(i);
    const int r0 = ((page0 * 2 + plane) * a.nkv + w.n.kvh) * PAGE, r1 = ((page1 * 2 + plane) * a.nkv + w.n.kvh) * PAGE;
    // (a second page that is not there is left out: nothing in it is seen, and its values are cleared)
    const bool two = PPB == 2 && page1 >= 0;
    mbar_expect_tx(&sm->full[s], (two ? 2 : 1) * NH * BOX);
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      tma_2d(dst + h * HALF, tm, 64 * h, r0, &sm->full[s]);
      if (two) tma_2d(dst + h * HALF + BOX, tm, 64 * h, r1, &sm->full[s]);
    }
  }
  SPEC_DEV void producer() {
    const int lane = threadIdx.x & 31;
    unsigned t0 = 0, issued = 0;
    bool ok = true;
    while (ok && w.pieces(a, p)) {
      const bool pair = w.n.w == 2;
      const int pages = (w.s.len + w.s.rows + PAGE - 1) / PAGE;
      // page ids: a window of 32 pages in the lanes of `cur`, the next one in `nxt`
      constexpr int WIN = 32 / PPB;  // in blocks
      auto window = [&](int i) {
        const int pg = PPB * (w.k0 + WIN * i) + lane;
        return pg < pages ? page_of(a, w.s.slot, pg) : -1;
      };
      int win = 0, cur = window(0), nxt = window(1);
      auto tile = [&](int n, int plane, int place) {
        const int from = n / WIN == win ? cur : nxt;
        const int p0 = __shfl_sync(FULL, from, PPB * (n % WIN)), p1 = __shfl_sync(FULL, from, PPB * (n % WIN) + PPB - 1);
        const unsigned i = t0 + place;
        if (lane == 0) {
          ok = i < (unsigned)sh.stages || wait(&sm->empty[i % sh.stages], parity(i) ^ 1);
          if (ok) load(i, p0, p1, plane);
        }
        ok = __shfl_sync(FULL, ok, 0);
        if (ok) issued = i + 1;
      };
      tile(0, 0, 0);
      if (ok && !pair && w.N > 1) tile(1, 0, 1);
      for (int n = 0; ok && n < w.N; ++n) {
        if (n / WIN != win) {
          ++win;
          cur = nxt;
          nxt = window(win + 1);
        }
        tile(n, 1, place_v(n, w.N, pair));
        const int k = n + (pair ? 1 : 2);
        if (ok && k < w.N) tile(k, 0, place_k(k, pair));
      }
      t0 += 2 * w.N;
      w.step(a, p);
    }
    // what was issued lands before the shared memory goes (normally it was all consumed)
    if (lane == 0)
      for (unsigned i = issued > (unsigned)sh.stages ? issued - sh.stages : 0; i < issued; ++i)
        drain_phase(&sm->full[i % sh.stages], parity(i));
  }

  // ---- warp 1 ----
  // A place in the ring, and the parity of its tile.
  struct Place {
    int s = 0;
    unsigned ph = 0;
  };
  SPEC_DEV Place next(Place c) const {
    const bool wrap = c.s + 1 == sh.stages;
    c.s = wrap ? 0 : c.s + 1;
    c.ph ^= wrap;
    return c;
  }
  SPEC_DEV void issue_s(int s, int t, Place k, bool last, uint32_t go) {
    // (the last parts of float rows first: what is cut is small until the first parts come)
    uint64_t q = desc_k(sa(qt) + (uint32_t)((t * QPL + QPL - 1) * QTILE));
    const uint64_t kd = desc_k(sa(ring) + (uint32_t)(k.s * TILE));
    const uint32_t d = tmem + s * 128;
#pragma unroll 1
    for (int pl = 0; pl < QPL; ++pl) {
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        const uint32_t h = i >> 2, off = 2 * (i & 3);
        mma_ss(d, q + h * (QHALF >> 4) + off, kd + h * (HALF >> 4) + off, idesc(ROWS, BK, false), i > 0 || pl > 0, go);
      }
      q -= QTILE >> 4;
    }
    commit(&sm->sfull[s], go);
    commit(&sm->empty[k.s], go && last);
  }
  SPEC_DEV void issue_pv(int s, int h, Place v, bool first, bool last, uint32_t go) {  // half h of a block's keys
    const uint64_t vd = desc_mn(sa(ring) + (uint32_t)(v.s * TILE + h * (BK / 2) * 128), HALF);
    const uint32_t pb = tmem + s * 128 + weights_at(h * (BK / 64)), ob = tmem + O_COL + s * HD;
#pragma unroll
    for (int i = 0; i < BK / 32; ++i)  // 16 keys: two groups of 8 rows of V, 8 columns of P
#pragma unroll
      for (int pl = 0; pl < QPL; ++pl)
        mma_ts(ob, pb + 16 * pl + 8 * i, vd + i * (2048 >> 4), idesc(ROWS, HD, true), i > 0 || pl > 0 || !first, go);
    if (h) {
      commit(&sm->odone[s], go);
      commit(&sm->empty[v.s], go && last);
    }
  }
  SPEC_DEV void products() {
    const uint32_t go = elect();
    unsigned piece = 0, round = 0;       // bit s of round: parity of stream s's next output
    Place at, kt, vt;                    // the next tile, the ones in use
    bool ok = true;
    while (ok && w.pieces(a, p)) {
      const bool pair = w.n.w == 2;
      const int steps = pair ? 2 * w.N : w.N;
      ok = wait(&sm->qfull, piece & 1);
      fence_after();
      // the first scores of both streams, then in turn a stream's output and its next scores
#pragma unroll 1
      for (int n = -2, s = 0; ok && n < steps; ++n, s ^= 1) {
        // (two tiles: step n is block n / 2 of stream n & 1, and a tile of the ring serves two steps)
        const bool shared = pair && s == 1, last = !pair || shared;
        // (the tiles' arrivals first: with the weights there, 16 products go out without a wait)
        const bool v = n >= 0, k = n + 2 < steps;
        if (v && !shared) {
          vt = at;
          at = next(at);
          ok = wait(&sm->full[vt.s], vt.ph);
        }
        if (k && !shared) {
          kt = at;
          at = next(at);
          ok = ok && wait(&sm->full[kt.s], kt.ph);
        }
        if (v) {
          ok = ok && wait(&sm->pfull[s][0], (round >> s) & 1);
        }
        if (!ok) break;
        fence_after();
        if (v) {
          issue_pv(s, 0, vt, (F32 ? n % RUN : n) < 2, last, go);
          ok = wait(&sm->pfull[s][1], (round >> s) & 1);
          round ^= 1u << s;
          if (!ok) break;
          fence_after();
          issue_pv(s, 1, vt, false, last, go);
          // the next scores overwrite the weights that these products read, in other columns than
          // they write: only products of one accumulator and shape are ordered by themselves
          // (8 x 64 rows 121 us, 114 without; with the upper half of the scores, which the weights
          // do not reach, made before the wait 119)
          if (k) {
            ok = wait(&sm->odone[s], ((round >> s) & 1) ^ 1);
            if (!ok) break;
            fence_after();
          }
        }
        if (k) issue_s(s, pair ? s : 0, kt, last, go);
      }
      ++piece;
      w.step(a, p);
    }
    commit(&sm->drain, go);  // every product done before tensor memory is freed
    drain_phase(&sm->drain, 0);
  }

  // ---- warps 4-11: thread = row of a tile ----
  SPEC_DEV void load_q(int row0, int nrow) {
    const int t = threadIdx.x - 128, G = p.G, c = t % (HD / 8);
    constexpr int STEP = NSM / (HD / 8), U = F32 ? 2 : 4;  // rows a round, rounds in flight
    #pragma unroll 1
    for (int r0 = t / (HD / 8); r0 < nrow; r0 += U * STEP) {  // (other rows stay what they are: a row's results are its own)
      uint4 v[U][F32 ? 2 : 1];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * STEP, gr = row0 + r, qi = p.row_of(gr), g = gr - qi * G;
        const size_t at = ((size_t)w.n.b * a.R + qi) * a.ldq + (size_t)(w.n.kvh * G + g) * HD + 8 * c;
#pragma unroll
        for (int e = 0; e < (F32 ? 2 : 1); ++e)
          v[u][e] = r < nrow ? *reinterpret_cast<const uint4*>((const char*)a.q + at * (F32 ? 4 : 2) + 16 * e)
                             : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * STEP;
        if (r >= nrow) break;
        unsigned char* dst = qt + (size_t)(r / ROWS) * QPL * QTILE + (c >> 3) * QHALF + swz(r % ROWS, (c & 7) * 16);
        if (!F32) {
          *reinterpret_cast<uint4*>(dst) = v[u][0];
        } else {
          const uint4 x = v[u][0], y = v[u][F32 ? 1 : 0];
          float f[8] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w),
                        __uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w)};
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) {  // x = hi + mid + lo: 24 bits in three times 8
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[e] = pack2(f[2 * e], f[2 * e + 1]);
              f[2 * e] -= bf16lo(o[e]);
              f[2 * e + 1] -= bf16hi(o[e]);
            }
            *reinterpret_cast<uint4*>(dst + pl * QTILE) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
    }
  }

  // What lies behind the sequence's last key is anything, and a row of the tree
  // that some rows do not see may be anything: their probabilities are zero, and
  // so that zero times infinity stays out, their values are cleared; rows of the
  // tree with values that are not finite are noted and added to the rows that see
  // them at the end.
  SPEC_DEV void clean_values(unsigned i, int key0) {
    wait(&sm->full[i % sh.stages], parity(i));
    const int r = (threadIdx.x - 128) & 127, key = key0 + r, j = key - w.s.len;
    if (j < 0 || r >= BK) return;
    uint4* row = reinterpret_cast<uint4*>(stage(i) + (size_t)r * 128);
    bool clear = j >= w.s.rows;
    if (!clear) {
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v = row[h * (HALF / 16) + c];
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) clear |= (e[k] & 0x7f80u) == 0x7f80u || (e[k] & 0x7f800000u) == 0x7f800000u;
        }
      if (clear) atomicOr(&sm->bad, 1ull << j);
    }
    if (clear)
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int c = 0; c < 8; ++c) row[h * (HALF / 16) + c] = make_uint4(0, 0, 0, 0);
  }

  // A key that was noted: its probability for this row, from the definition.
  SPEC_DEV float noted(size_t qat, int j, float M, const __nv_bfloat16** v) {
    const int pos = w.s.len + j;
    const __nv_bfloat16* k = (const __nv_bfloat16*)a.pool +
                             (((size_t)page_of(a, w.s.slot, pos / PAGE) * 2 * a.nkv + w.n.kvh) * PAGE + pos % PAGE) * HD;
    *v = k + (size_t)a.nkv * PAGE * HD;
    float s = 0.f;
    for (int d = 0; d < HD; ++d)
      s = fmaf(F32 ? ((const float*)a.q)[qat + d] : __bfloat162float(((const __nv_bfloat16*)a.q)[qat + d]),
               __bfloat162float(k[d]), s);
    return ex2(fmaf(s, sh.scale2, -M));
  }

  // The loops over a block's scores of this thread's row take 32 a turn and
  // stay rolled: an instruction that runs once costs 20 to 40 cycles, as the caches
  // are cold at a launch.
  // Scores that the row does not see: -inf.
  SPEC_DEV void hide(uint32_t sb, unsigned long long lo, unsigned long long hi) const {
#pragma unroll 1
    for (int c = 0; c < BK / 32; ++c) {
      const uint32_t b = (uint32_t)((c < 2 ? lo : hi) >> (32 * (c & 1)));
      if (__all_sync(FULL, b == ~0u)) continue;
      float v[32];
      ld32(sb + 32 * c, v);
      wait_ld();
      uint32_t u[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) u[e] = (b >> e) & 1 ? __float_as_uint(v[e]) : 0xff800000u;
      st16(sb + 32 * c, u);
      st16(sb + 32 * c + 16, u + 16);
    }
    wait_st();
  }
  // Where the weights of 32 keys lie in a stream's columns: 16 columns of two each,
  // over scores that have been read; with float rows three times 16 (leading parts,
  // middle ones, last ones), the first 32 keys' behind the 64 scores.
  static SPEC_DEV uint32_t weights_at(int c) { return F32 ? (c ? 0u : 64u) : 16u * c; }
  // The weights of the scores, and their sum. A bf16 row's are rounded to bf16, and
  // the sum is that of the rounded ones: a rounding then moves a value's share, not
  // the row's scale. A float row's go out as three bf16 parts each, which hold all
  // 24 bits. The products of the first half start while the others are made.
  SPEC_DEV float weights(uint32_t sb, float m, int s) const {
    const float2 sc = make_float2(sh.scale2, sh.scale2), mm = make_float2(-m, -m);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
    for (int c = 0; c < BK / 32; ++c) {
      float v[32];
      ld32(sb + 32 * c, v);
      wait_ld();
      uint32_t part[QPL][16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float2 x = fma2(make_float2(v[2 * e], v[2 * e + 1]), sc, mm);
        x.x = ex2(x.x);
        x.y = ex2(x.y);
        if (F32) sum[e & 1] = add2(sum[e & 1], x);
#pragma unroll
        for (int pl = 0; pl < QPL; ++pl) {
          part[pl][e] = pack2(x.x, x.y);
          const float2 r = make_float2(bf16lo(part[pl][e]), bf16hi(part[pl][e]));
          if (!F32) sum[e & 1] = add2(sum[e & 1], r);
          x.x -= r.x;
          x.y -= r.y;
        }
      }
#pragma unroll
      for (int pl = 0; pl < QPL; ++pl) st16(sb + weights_at(c) + 16 * pl, part[pl]);
      if ((c + 1) % (BK / 64) == 0) hand_over(s, c / (BK / 64));
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
  }

  // Half h of this warp's weights is in tensor memory.
  SPEC_DEV void hand_over(int s, int h) const {
    wait_st();
    fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm->pfull[s][h]);
  }

  SPEC_DEV void softmax() {
    const int t = threadIdx.x - 128, s = t >> 7, r = t & 127, lane = t & 31, G = p.G;
    const uint32_t lanes = (uint32_t)(r & ~31) << 16;
    unsigned t0 = 0, round = 0, other = 0;  // this stream's blocks so far, the other's
    bool begun = false;
    while (w.pieces(a, p)) {
      const bool pair = w.n.w == 2;
      const int N = w.N;
      const int row0 = w.n.u * p.tpu * ROWS, nrow = min(w.n.w * ROWS, w.s.rows * G - row0);
      sm_sync();                         // the piece before is read out
      if (t < 64) {
        int q = -1;
        if (t < w.s.rows) q = a.parents ? a.parents[(size_t)w.n.b * a.R + t] : t - 1;
        sm->up[t] = q < t ? q : -1;
      }
      if (t == 0) sm->bad = 0;
      load_q(row0, nrow);
      fence_async();
      if (!begun) {                      // the barriers are set up, and tensor memory is there
        all_ready();
        tmem = sm->tmem;
        begun = true;
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->qfull);
      sm_sync();
      const uint32_t sb = tmem + lanes + s * 128, ob = tmem + lanes + O_COL + s * HD;
      const int mine = pair ? s * ROWS + r : r;                       // row of the unit
      const bool work = (mine & ~31) < nrow;                          // this warp holds a row
      const int gr = row0 + mine, qi = mine < nrow ? p.row_of(gr) : 0, g = gr - qi * G;
      unsigned long long path = 0;
      for (int q = qi; q >= 0; q = sm->up[q]) path |= 1ull << q;
      float m = -INFINITY, l = 0.f, Ma = -INFINITY, La = 0.f;  // (this stream's; both, of the runs before)
      float acc[F32 ? 2 : 1][32];  // the runs before: this thread's share of its row (in local memory: a rolled loop indexes it)
      for (int e0 = 0, e1; e0 < N; e0 = e1) {
        e1 = F32 ? min(N, e0 + RUN) : N;
        const int n0 = pair ? e0 : e0 + s, dn = pair ? 1 : 2;
        l = 0.f;
        for (int n = n0; n < e1; n += dn) {
          wait(&sm->sfull[s], round & 1);
          fence_after();
          const int key0 = (w.k0 + n) * BK;
          const bool edge = key0 + BK > w.s.len;                        // rows of the tree, or the end, in this block
          if (edge && (!pair || s == 0)) {
            clean_values(t0 + place_v(n, N, pair), key0);
            fence_async();
          }
          if (work) {
            if (edge) hide(sb, visible(path, w.s.len, key0), visible(path, w.s.len, key0 + 64));
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < BK / 32; ++c) mx = fmaxf(mx, ldmax32(sb + 32 * c));
            mx *= sh.scale2;
            const bool raise = mx > m + TAU || (m == -INFINITY && mx > -INFINITY);
            if (__any_sync(FULL, raise)) {
              const float f = !raise ? 1.f : m == -INFINITY ? 0.f : ex2(m - mx);
              if (raise) m = mx;
              l *= f;
              if (n != n0) {
                wait(&sm->odone[s], (round & 1) ^ 1);
                fence_after();
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                  float v[32];
                  ld32(ob + 32 * c, v);
                  wait_ld();
                  uint32_t u[32];
#pragma unroll
                  for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(v[e] * f);
                  st16(ob + 32 * c, u);
                  st16(ob + 32 * c + 16, u + 16);
                }
              }
            }
            const float mb = m == -INFINITY ? 0.f : m;
            l += weights(sb, mb, s);
          } else {
            hand_over(s, 0);
            hand_over(s, 1);
          }
          ++round;
        }
        // (the other stream's rounds are known too: both streams' O are read below)
        other += pair ? N : (e1 - e0 + s) / 2;
        sm->ml[s][r] = make_float2(m, l);
        const bool both = pair || e1 - e0 > 1, end = e1 == N;
        wait(&sm->odone[s], (round & 1) ^ 1);
        if (!pair && both) wait(&sm->odone[s ^ 1], (other & 1) ^ 1);
        sm_sync();
        fence_after();
        if (work) {
          const bool whole = w.k0 == 0 && N == w.n.nb;
          float f[2] = {1.f, 1.f}, M = m, L = l;
          if (!pair) {
            const float2 u = sm->ml[0][r], v = sm->ml[1][r];
            M = fmaxf(u.x, v.x);
            f[0] = u.x == -INFINITY ? 0.f : ex2(u.x - M);
            f[1] = v.x == -INFINITY ? 0.f : ex2(v.x - M);
            L = f[0] * u.y + f[1] * v.y;
          }
          float fa = 0.f;
          if (F32) {
            const float top = fmaxf(Ma, M), fn = M == -INFINITY ? 0.f : ex2(M - top);
            fa = Ma == -INFINITY ? 0.f : ex2(Ma - top);
            f[0] *= fn;
            f[1] *= fn;
            La = L = fa * La + fn * L;
            Ma = M = top;
          }
          const unsigned long long bad = sm->bad & path;
          const float inv = whole && end ? 1.f / L : 1.f;
          const int c0 = pair ? 0 : s * (HD / 64), c1 = pair ? HD / 32 : c0 + HD / 64;
          const size_t qat = ((size_t)w.n.b * a.R + qi) * a.ldq + (size_t)(w.n.kvh * G + g) * HD;
          const size_t oat = ((size_t)w.n.b * a.R + qi) * a.ldo + (size_t)(w.n.kvh * G + g) * HD;
          const size_t slot = (size_t)(2 * blockIdx.x + (w.k0 == 0)) * (p.tpu << p.tile) + mine;
          float4* stg = reinterpret_cast<float4*>(qt) + (t >> 5) * 256;
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            float v[32];
            if (pair) {
              ld32(ob + 32 * c, v);
              wait_ld();
            } else {
              const uint32_t o0 = tmem + lanes + O_COL + 32 * c;
              ld32(o0, v);
              wait_ld();
              if (both) {
                float u[32];
                ld32(o0 + HD, u);
                wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = f[0] * v[e] + f[1] * u[e];
              } else if (F32) {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= f[0];
              }
            }
            if (F32) {
              float* sum = acc[c - c0];
              if (e0 > 0)
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] += fa * sum[e];
              if (!end) {
#pragma unroll
                for (int e = 0; e < 32; ++e) sum[e] = v[e];
                continue;
              }
            }
            if (bad && mine < nrow && key_here(bad)) {
              for (unsigned long long b = bad; b; b &= b - 1) {
                const int j = __ffsll((long long)b) - 1;
                if (!in_piece(j)) continue;
                const __nv_bfloat16* val;
                const float pr = noted(qat, j, M == -INFINITY ? 0.f : M, &val);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = fmaf(pr, __bfloat162float(val[32 * c + e]), v[e]);
              }
            }
            // through shared memory (the query tiles are done with), so that stores are whole 128-byte (64: bf16) pieces of rows
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              stg[lane * 8 + (e ^ (lane & 7))] = make_float4(v[4 * e] * inv, v[4 * e + 1] * inv, v[4 * e + 2] * inv, v[4 * e + 3] * inv);
            __syncwarp();
            const int w0 = mine & ~31;                                  // the warp's first row
            if (F32 || !whole) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int rr = 4 * i + (lane >> 3), e = lane & 7;
                const float4 x = stg[rr * 8 + (e ^ (rr & 7))];
                const size_t to = __shfl_sync(FULL, (unsigned long long)oat, rr);
                float* dst = whole ? (float*)a.out + to : a.part_o + (slot - lane + rr) * HD;
                if (w0 + rr < nrow) *reinterpret_cast<float4*>(dst + 32 * c + 4 * e) = x;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int rr = 8 * i + (lane >> 2), e = 2 * (lane & 3);
                const float4 x = stg[rr * 8 + (e ^ (rr & 7))], y = stg[rr * 8 + ((e + 1) ^ (rr & 7))];
                const size_t to = __shfl_sync(FULL, (unsigned long long)oat, rr);
                if (w0 + rr < nrow)
                  *reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + to + 32 * c + 4 * e) =
                      make_uint4(pack2(x.x, x.y), pack2(x.z, x.w), pack2(y.x, y.y), pack2(y.z, y.w));
              }
            }
          }
          if (!whole && end && mine < nrow && (pair || s == 0)) a.part_ml[slot] = make_float2(M, L);
        }
        fence_before();
        if (!end) sm_sync();               // (O is read: its next products may come)
      }
      t0 += 2 * N;
      w.step(a, p);
    }
  }
  // Whether key len + j lies in this piece's blocks.
  SPEC_DEV bool in_piece(int j) const {
    const int k = (w.s.len + j) / BK - w.k0;
    return k >= 0 && k < w.N;
  }
  SPEC_DEV bool key_here(unsigned long long b) const {
    for (; b; b &= b - 1)
      if (in_piece(__ffsll((long long)b) - 1)) return true;
    return false;
  }
};

template <int HD, bool F32>
__global__ void __launch_bounds__(NTHR, 1)
    tree_tc_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ Plan p, const __grid_constant__ Shape sh,
                   const __grid_constant__ CUtensorMap tm) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Small* sm = reinterpret_cast<Small*>(smem);
  Cta<HD, F32> k{a, p, sh, &tm, sm};
  k.qt = smem + SMALL;
  k.ring = k.qt + sh.q_bytes;
  grid_dep_launch();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sa(&sm->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (threadIdx.x == 64) {
    for (int i = 0; i < sh.stages; ++i) {
      mbar_init(&sm->full[i], 1);
      mbar_init(&sm->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->sfull[i], 1);
      mbar_init(&sm->pfull[i][0], 4 + (i == 0 ? sh.wait_extra : 0));
      mbar_init(&sm->pfull[i][1], 4);
      mbar_init(&sm->odone[i], 1);
    }
    mbar_init(&sm->qfull, NSM / 32);
    mbar_init(&sm->drain, 1);
    sm->abort = 0;
    mbar_init_fence();
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm) : "memory");
  }
  const bool work = k.w.begin(a, p);                        // (every warp for itself)
  if (work && warp < 4) {
    fence_before();
    set_up();
    fence_after();
    k.tmem = sm->tmem;
  }
  if (warp == 2) {
    const bool bad = __any_sync(FULL, bad_input(a, p, lane, 32));
    if (lane == 0) found(a, p, bad);
  } else if (work && warp == 0) {
    k.producer();
    __syncwarp();
  } else if (work && warp == 1) {
    k.products();
    __syncwarp();
  } else if (work && warp >= 4) {
    k.softmax();
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sm->tmem) : "memory");
  }
}

std::atomic<int> g_wait_extra{0};
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_once;
void init_encode() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    g_encode = (PFN_cuTensorMapEncodeTiled_v12000)fn;
}
// A layer of the pool as rows of head-dim elements, boxes of a page's 64 rows x 64 dims.
bool encode(CUtensorMap* m, const TreeArgs& a) {
  if (!g_encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)a.hd, (cuuint64_t)a.n_pages * 2 * a.nkv * PAGE};
  const cuuint64_t strides[1] = {(cuuint64_t)a.hd * 2};
  const cuuint32_t box[2] = {64, PAGE}, es[2] = {1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(a.pool), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

const void* kernel_of(int hd, bool f32) {
  return hd == 64 ? (f32 ? (const void*)tree_tc_kernel<64, true> : (const void*)tree_tc_kernel<64, false>)
                  : (f32 ? (const void*)tree_tc_kernel<128, true> : (const void*)tree_tc_kernel<128, false>);
}

}  // namespace

bool tc_ok(const TreeArgs& a) {
  return a.kv_dtype == DT_BF16 && (a.hd == 64 || a.hd == 128) &&
         (long long)a.n_pages * 2 * a.nkv * PAGE <= 0x7fffffffll;
}

Plan tc_plan(const TreeArgs& a) {
  Plan p;
  p.blk = a.q_dtype == DT_BF16 ? 7 : 6;
  p.tile = 7;
  // what a unit's beginning and end cost, in tiles (8 x 64 rows, 30B-class: 121 us at 12, 124 at 5 and at 16; fp32 rows,
  // 8 x 24: within 3% at 3, 5 and 8, 2% more at 11)
  p.head = a.q_dtype == DT_BF16 ? 12 : 5;
  p.units = 0;
  plan_heads(p, a);
  // two tiles share a block's reads; three planes of each do not fit beside a ring
  p.tpu = a.q_dtype == DT_BF16 && a.R * (a.nq / a.nkv) > ROWS ? 2 : 1;
  p.grid = num_sms();
  p.min_cost = 1;
  return p;
}

void tc_setup() {
  std::call_once(g_once, init_encode);
  for (int hd : {64, 128})
    for (bool f : {false, true}) cudaFuncSetAttribute(kernel_of(hd, f), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_MAX);
}

int tc_launch(const TreeArgs& a, const Plan& p, cudaStream_t st) {
  const bool f32 = a.q_dtype == DT_F32;
  const int tile = a.hd * keys_of(f32) * 2;
  Shape sh;
  const size_t q = std::max((size_t)p.tpu * (f32 ? 3 : 1) * ROWS * a.hd * 2, (size_t)NSM * 128);  // (and a row of results a softmax thread)
  sh.q_bytes = (int)q;
  sh.stages = std::min(ST_MAX, (int)((SMEM_MAX - SMALL - q) / tile));
  sh.scale2 = LOG2E / sqrtf((float)a.hd);
  sh.wait_extra = g_wait_extra;
  CUtensorMap tm;
  if (!encode(&tm, a)) return -1;
  void* args[] = {(void*)&a, (void*)&p, (void*)&sh, (void*)&tm};
  return cudaLaunchKernel(kernel_of(a.hd, f32), dim3(p.grid), dim3(NTHR), args, SMALL + q + (size_t)sh.stages * tile, st) ==
                 cudaSuccess
             ? 1
             : -1;
}

}  // namespace tree
}  // namespace spec

// For failure-detection tests only, and in no header: with 1, a wait of the next
// launches runs out after about a second.
extern "C" void spec_test_attention_tree_wait(int32_t extra) { spec::tree::g_wait_extra = extra > 0 ? 1 : 0; }
