// pages.cu -- pages of the cache handed out, shared, given back and moved: a
// slot's table names its pages in order (-1 behind the last), and refs counts
// for each page how often tables name it. Free pages are those that nothing
// names; they are handed out lowest number first, so what a call does follows
// from its arguments alone.
//
// The tables are small (a count a page, a row a slot): one CTA plans a call,
// checks it against the free pages before it changes anything, and leaves a list
// of copies in the workspace; a second kernel, launched while the first runs,
// moves the bytes with the whole GPU. Bound by HBM: rows read and written once.
#include <algorithm>

#include "common.cuh"

namespace spec {
namespace {

constexpr int PAGE = 64;
constexpr int PT = 1024;      // threads of a planning CTA
constexpr int N_MAX = 1024;   // slots of a call

// Workspace: [0] error word, [1] copies (-1: the call changes nothing), [2] runs, from [64]
// on the copies (fork: source page, page, rows; compact: from, to) and, behind a
// fork's, the pages handed out (reserve: those alone) and where runs of copies of
// the same rows begin.
struct Ws {
  int *err, *jobs;
};
SPEC_DEV Ws ws_of(int* w) { return Ws{w, w + 64}; }

// Exclusive prefix sum over a CTA of PT threads; the total to *sum.
SPEC_DEV int scan(int v, int* red, int* sum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();
  if (lane == 31) red[w] = incl;
  __syncthreads();
  if (w == 0) {
    int x = red[lane], s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(FULL, s, o);
      if (lane >= o) s += u;
    }
    red[lane] = s - x;
    if (lane == 31) red[32] = s;
  }
  __syncthreads();
  *sum = red[32];
  return red[w] + incl - v;
}

// The `need` lowest free pages, ascending, to list; false when there are fewer.
SPEC_DEV bool lowest_free(const int32_t* refs, int n_pages, int need, int* list, int* red) {
  int got = 0;
  for (int p0 = 0; p0 < n_pages && got < need; p0 += 4 * PT) {
    int f[4], c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = p0 + 4 * threadIdx.x + j;
      f[j] = p < n_pages && refs[p] == 0;
      c += f[j];
    }
    int sum, at = got + scan(c, red, &sum);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (f[j]) {
        if (at < need) list[at] = p0 + 4 * threadIdx.x + j;
        ++at;
      }
    got += sum;
    __syncthreads();
  }
  return got >= need;
}

SPEC_DEV bool page_ok(const PagesArgs& a, int p) { return p >= 0 && p < a.n_pages; }

// How many pages a slot's table names (to the first entry that names none); -1
// where one of them is out of range. By one warp.
SPEC_DEV int held(const PagesArgs& a, int slot) {
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < a.max_pages; i0 += 32) {
    const int i = i0 + lane;
    const int p = i < a.max_pages ? a.table[(size_t)slot * a.max_pages + i] : -1;
    const unsigned end = __ballot_sync(FULL, p < 0), out = __ballot_sync(FULL, p >= a.n_pages);
    if (out & (end ? (end & -end) - 1 : ~0u)) return -1;  // (ahead of the end)
    if (end) return i0 + __ffs(end) - 1;
  }
  return a.max_pages;
}

// A slot that is out of range, or named twice.
SPEC_DEV bool ids_bad(const PagesArgs& a) {
  bool bad = false;
  for (int i = threadIdx.x; i < a.n; i += PT) {
    const int s = a.ids[i];
    bad |= s < 0 || s >= a.n_slots;
    for (int j = 0; j < i; ++j) bad |= a.ids[j] == s;
  }
  return __syncthreads_or(bad);
}

// f(i, k) for the entries k >= keep(i) of every named slot's row: a warp a slot,
// so that a call's slots wait for memory together.
template <class Keep, class F>
SPEC_DEV void each_entry(const PagesArgs& a, Keep keep, F f) {
  for (int i = threadIdx.x >> 5; i < a.n; i += PT / 32)
    for (int k = keep(i) + (threadIdx.x & 31); k < a.max_pages; k += 32) f(i, k);
}
// Entries of the named slots from keep(i) on: `by` added to their pages' counts
// (0: whether one is out of range, or a page that nothing names).
template <class Keep>
SPEC_DEV bool count_entries(const PagesArgs& a, int by, Keep keep) {
  bool bad = false;
  each_entry(a, keep, [&](int i, int k) {
    const int p = a.table[(size_t)a.ids[i] * a.max_pages + k];
    if (p < 0) return;
    if (!page_ok(a, p)) bad = true;
    else if (by) atomicAdd(&a.refs[p], by);
    else bad |= a.refs[p] <= 0;
  });
  return __syncthreads_or(bad);
}

SPEC_DEV int pages_for(int len) { return len / PAGE + (len % PAGE != 0); }

__global__ void __launch_bounds__(PT) reserve_kernel(const __grid_constant__ PagesArgs a) {
  __shared__ int red[33], want[N_MAX], have[N_MAX];
  int* list = ws_of(a.ws).jobs;
  bool bad = ids_bad(a);
  if (!bad) {
    for (int i = threadIdx.x >> 5; i < a.n; i += PT / 32) {
      const int h = held(a, a.ids[i]), len = a.lens[i];
      if ((threadIdx.x & 31) == 0) {
        have[i] = h;
        // (one page more than there are is enough to be refused: N_MAX slots' sum stays below 2^31)
        want[i] = h < 0 || len < 0 || pages_for(len) > a.max_pages ? -1 : min(max(pages_for(len) - h, 0), a.n_pages + 1);
      }
    }
    __syncthreads();
    const int mine = threadIdx.x < a.n ? want[threadIdx.x] : 0;
    bad = __syncthreads_or(mine < 0);
    if (!bad) {
      int need;
      const int at = scan(mine, red, &need);
      bad = !lowest_free(a.refs, a.n_pages, need, list, red);
      if (!bad) {
        __syncthreads();
        if (threadIdx.x < a.n) want[threadIdx.x] = at;
        __syncthreads();
        for (int i = threadIdx.x >> 5; i < a.n; i += PT / 32) {
          const int first = want[i], last = i + 1 < a.n ? want[i + 1] : need;
          for (int k = first + (threadIdx.x & 31); k < last; k += 32) {
            a.table[(size_t)a.ids[i] * a.max_pages + have[i] + k - first] = list[k];
            a.refs[list[k]] = 1;
          }
        }
      }
    }
  }
  if (threadIdx.x == 0) *a.ws = bad ? SPEC_ERR_CAPACITY : 0;
}

__global__ void __launch_bounds__(PT) release_kernel(const __grid_constant__ PagesArgs a) {
  bool bad = ids_bad(a);
  if (!bad && a.lens) {
    bool neg = false;
    for (int i = threadIdx.x; i < a.n; i += PT) neg |= a.lens[i] < 0;
    bad = __syncthreads_or(neg);
  }
  auto keep = [&](int i) { return a.lens ? min(pages_for(a.lens[i]), a.max_pages) : 0; };
  if (!bad) bad = count_entries(a, 0, keep);
  if (!bad) {
    count_entries(a, -1, keep);
    each_entry(a, keep, [&](int i, int k) { a.table[(size_t)a.ids[i] * a.max_pages + k] = -1; });
  }
  if (threadIdx.x == 0) *a.ws = bad ? SPEC_ERR_CAPACITY : 0;
}

// One step a call: the slots forked to give their pages back, take their
// sources' full pages and a free one each for the rows of a last page that is not
// full. Nothing changes where an argument is out of range or the pages do not
// suffice (the counts that were taken back to see it are restored).
__global__ void __launch_bounds__(PT) fork_kernel(const __grid_constant__ PagesArgs a) {
  __shared__ int red[33], len[N_MAX], at[N_MAX];
  grid_dep_launch();
  const Ws w = ws_of(a.ws);
  int* list = w.jobs + 3 * N_MAX;
  bool bad = ids_bad(a);
  if (!bad) {
    bool b = false;
    for (int i = threadIdx.x; i < a.n; i += PT) {
      const int s = a.src[i];
      bool x = s < 0 || s >= a.n_slots;
      for (int j = 0; j < a.n; ++j) x |= a.ids[j] == s;  // a source is no slot forked to
      len[i] = x ? -1 : a.seq_len[s];
      b |= len[i] < 0 || pages_for(len[i]) > a.max_pages;
    }
    bad = __syncthreads_or(b);
  }
  auto all = [](int) { return 0; };
  if (!bad) {
    bool b = false;
    each_entry(a, all, [&](int i, int k) {
      const int p = k < pages_for(len[i]) ? a.table[(size_t)a.src[i] * a.max_pages + k] : 0;
      const int q = a.table[(size_t)a.ids[i] * a.max_pages + k];
      b |= k < pages_for(len[i]) && (!page_ok(a, p) || a.refs[p] <= 0);
      b |= q >= 0 && (!page_ok(a, q) || a.refs[q] <= 0);
    });
    bad = __syncthreads_or(b);
  }
  int need = 0;
  if (!bad) {
    count_entries(a, -1, all);
    const int mine = threadIdx.x < a.n && len[threadIdx.x] % PAGE != 0;
    const int rank = scan(mine, red, &need);
    if (threadIdx.x < a.n) at[threadIdx.x] = mine ? rank : -1;
    __syncthreads();
    bad = !lowest_free(a.refs, a.n_pages, need, list, red);
    if (bad) {
      __syncthreads();
      count_entries(a, 1, all);
    }
  }
  __syncthreads();
  if (!bad) {
    each_entry(a, all, [&](int i, int k) {
      const int full = len[i] / PAGE;
      int p = -1;
      if (k <= full) {
        const int from = k < full || at[i] >= 0 ? a.table[(size_t)a.src[i] * a.max_pages + k] : -1;
        if (k < full) {
          p = from;
          atomicAdd(&a.refs[p], 1);
        } else if (at[i] >= 0) {
          p = list[at[i]];
          a.refs[p] = 1;
          w.jobs[3 * at[i]] = from;
          w.jobs[3 * at[i] + 1] = p;
          w.jobs[3 * at[i] + 2] = len[i] % PAGE;
        }
      }
      a.table[(size_t)a.ids[i] * a.max_pages + k] = p;
    });
    for (int i = threadIdx.x; i < a.n; i += PT) {
      a.seq_len[a.ids[i]] = len[i];
      if (a.pending) a.pending[a.ids[i]] = a.pending[a.src[i]];
    }
  }
  // copies of the same rows follow each other in the list (slots forked from one
  // source): where each such run begins. Sources that were cut back into a page that
  // they share may hold different numbers of its rows.
  __syncthreads();
  const int j = 3 * threadIdx.x;
  const bool first = !bad && threadIdx.x < need &&
                     (j == 0 || w.jobs[j] != w.jobs[j - 3] || w.jobs[j + 2] != w.jobs[j - 1]);
  int runs;
  const int run = scan(first, red, &runs);
  if (first) list[N_MAX + run] = threadIdx.x;
  if (threadIdx.x == 0) {
    *w.err = bad ? SPEC_ERR_CAPACITY : 0;
    w.err[1] = bad ? -1 : need;
    w.err[2] = runs;
  }
}

// The list's copies: the first rows of a page, in all layers, planes and heads. The
// rows of a plane are one piece of up to 64 rows; half of it is a CTA's unit (128
// threads, four 16-byte reads in flight, no division in the loop), read once for all
// slots forked from one source. Behind those units the hidden states'.
constexpr int HID = 4 * 128 * 4;  // floats a unit
__global__ void __launch_bounds__(128) fork_copy_kernel(const __grid_constant__ PagesArgs a) {
  grid_dep_wait();
  const Ws w = ws_of(a.ws);
  const int n = w.err[1], runs = w.err[2], t = threadIdx.x;
  if (n < 0) return;
  const size_t plane = (size_t)PAGE * a.row_bytes;
  const int pieces = 2 * a.L * a.planes, hids = a.hid ? (a.d + HID - 1) / HID : 0;
  const long long copies = (long long)runs * pieces, units = copies + (long long)a.n * hids;
  auto move = [&](const uint4* src, int v0, int v1, auto each) {  // [v0, v1) of src to each() of them
    for (int v = v0 + t; v < v1; v += 4 * 128) {
      uint4 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v + e * 128 < v1) x[e] = src[v + e * 128];
      each([&](uint4* dst) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (v + e * 128 < v1) dst[v + e * 128] = x[e];
      });
    }
  };
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    if (u < copies) {
      const int r = (int)(u / pieces), k = (int)(u - (long long)r * pieces), pl = k >> 1;
      const int j = w.jobs[4 * N_MAX + r], last = r + 1 < runs ? w.jobs[4 * N_MAX + r + 1] : n;
      const int vecs = w.jobs[3 * j + 2] * (a.row_bytes / 16), mid = vecs / 2;
      char* base = a.pool + (size_t)(pl / a.planes) * a.layer_bytes + (size_t)(pl % a.planes) * plane;
      move(reinterpret_cast<const uint4*>(base + (size_t)w.jobs[3 * j] * a.page_bytes), k & 1 ? mid : 0, k & 1 ? vecs : mid,
           [&](auto put) {
             for (int i = j; i < last; ++i) put(reinterpret_cast<uint4*>(base + (size_t)w.jobs[3 * i + 1] * a.page_bytes));
           });
    } else {
      const int i = (int)((u - copies) / hids), c = (int)((u - copies) % hids);
      move(reinterpret_cast<const uint4*>(a.hid + (size_t)a.src[i] * a.d), c * HID / 4, min((c + 1) * HID, a.d) / 4,
           [&](auto put) { put(reinterpret_cast<uint4*>(a.hid + (size_t)a.ids[i] * a.d)); });
    }
  }
}

// With n pages in use, those numbered n or higher go to the free ones below, both
// in ascending order. A page that only the caller holds moves too.
__global__ void __launch_bounds__(PT) compact_kernel(const __grid_constant__ PagesArgs a) {
  __shared__ int red[33];
  grid_dep_launch();
  const Ws w = ws_of(a.ws);
  int live = 0;
  for (int p0 = 0; p0 < a.n_pages; p0 += PT) {
    const int p = p0 + threadIdx.x;
    live += __syncthreads_count(p < a.n_pages && a.refs[p] > 0);
  }
  // the holes below, then the pages above, each into its list
  int holes = 0, moves = 0;
  for (int p0 = 0; p0 < a.n_pages; p0 += PT) {
    const int p = p0 + threadIdx.x;
    const bool in = p < a.n_pages, used = in && a.refs[p] > 0;
    const bool hole = in && p < live && !used, move = used && p >= live;
    int n;
    const int at = scan(hole || move, red, &n), h = __syncthreads_count(hole);
    if (hole) w.jobs[2 * (holes + at) + 1] = p;
    if (move) w.jobs[2 * (moves + at - h)] = p;  // (every hole lies below every page that moves)
    holes += h;
    moves += n - h;
  }
  for (int p = threadIdx.x; p < a.n_pages; p += PT) {
    const int r = a.refs[p];
    a.moved[p] = r > 0 && p < live ? p : -1;
    if (a.refs_out != a.refs) a.refs_out[p] = p < live ? r : 0;
  }
  __syncthreads();
  for (int j = threadIdx.x; j < moves; j += PT) {
    const int from = w.jobs[2 * j], to = w.jobs[2 * j + 1];
    a.moved[from] = to;
    a.refs_out[to] = a.refs[from];
    if (a.refs_out == a.refs) a.refs[from] = 0;
  }
  if (threadIdx.x == 0) {
    *w.err = 0;
    w.err[1] = moves;
    *a.n_live = live;
  }
}

__global__ void __launch_bounds__(256) compact_copy_kernel(const __grid_constant__ PagesArgs a) {
  grid_dep_wait();
  const Ws w = ws_of(a.ws);
  const int n = w.err[1];
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x, nt = (long long)gridDim.x * 256;
  for (long long i = t; i < (long long)a.n_slots * a.max_pages; i += nt) {
    const int p = a.table[i];
    a.table_out[i] = page_ok(a, p) ? a.moved[p] : -1;
  }
  // a page of a layer is one piece; the pieces of all moves in one range
  const int vec = a.page_bytes / 16;
  const long long per = (long long)a.L * vec, all = per * n;
  auto off = [&](long long i, int side) {
    const long long j = i / per, in = i % per;
    return (size_t)(in / vec) * a.layer_bytes + (size_t)w.jobs[2 * j + side] * a.page_bytes + (size_t)(in % vec) * 16;
  };
  long long i = t;
  for (; i + 3 * nt < all; i += 4 * nt) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint4*>(a.pool + off(i + j * nt, 0));
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(a.pool + off(i + j * nt, 1)) = v[j];
  }
  for (; i < all; i += nt) *reinterpret_cast<uint4*>(a.pool + off(i, 1)) = *reinterpret_cast<const uint4*>(a.pool + off(i, 0));
}

// Sequence b's row rows[i] to row i, for i in order: with rows ascending, a row
// is never behind its place, so a thread that walks them in order (four reads
// ahead of their writes) reads nothing that it has overwritten; threads share
// no bytes.
SPEC_DEV bool keep_ok(const KeepArgs& a, int b, int t, int nthr) {
  const int slot = a.seq_ids[b], n = a.n_keep[b];
  if (slot < 0 || slot >= a.n_slots || n < 0 || n > a.n) return false;
  const int len = a.seq_len[slot];
  const int32_t* r = a.rows + (size_t)b * a.n;
  if (len < 0) return false;
  bool ok = true;
  for (int i = t; i < n; i += nthr) {
    ok &= r[i] >= i && (i == 0 || r[i] > r[i - 1]);
    const long long p[2] = {(long long)len + r[i], (long long)len + i};
    for (int e = 0; e < 2 && ok; ++e) {
      ok &= p[e] < min((long long)a.max_pages * PAGE, TREE_POSITIONS_MAX);
      if (ok) {
        const int g = a.table[(size_t)slot * a.max_pages + p[e] / PAGE];
        ok &= g >= 0 && g < a.n_pages;
      }
    }
  }
  return ok;
}

__global__ void __launch_bounds__(256) rows_keep_kernel(const __grid_constant__ KeepArgs a) {
  const int b = blockIdx.y;
  const bool ok = !__syncthreads_or(!keep_ok(a, b, threadIdx.x, 256));
  if (blockIdx.x == 0 && b == 0) {
    bool bad = false;
    for (int s = 0; s < a.B; ++s) bad |= !keep_ok(a, s, threadIdx.x, 256);
    // (two sequences of one slot would move the same rows twice)
    for (int s = threadIdx.x; s < a.B; s += 256)
      for (int j = 0; j < s; ++j) bad |= a.seq_ids[j] == a.seq_ids[s];
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.err = bad ? SPEC_ERR_CAPACITY : 0;
  }
  bool twice = false;
  for (int j = threadIdx.x; j < a.B; j += 256) twice |= j != b && a.seq_ids[j] == a.seq_ids[b];
  if (__syncthreads_or(twice) || !ok) return;
  const int slot = a.seq_ids[b], n = a.n_keep[b], len = a.seq_len[slot];
  const int32_t* r = a.rows + (size_t)b * a.n;
  const int32_t* tab = a.table + (size_t)slot * a.max_pages;
  const int vec = a.row_bytes / 16;
  const size_t plane = (size_t)PAGE * a.row_bytes, page = plane * a.planes;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < (long long)a.L * a.planes * vec; i += (long long)gridDim.x * 256) {
    const long long pl = i / vec;
    char* base = a.pool + (size_t)(pl / a.planes) * a.layer_bytes + (size_t)(pl % a.planes) * plane + (size_t)(i % vec) * 16;
    auto at = [&](int pos) { return reinterpret_cast<uint4*>(base + (size_t)tab[pos / PAGE] * page + (size_t)(pos % PAGE) * a.row_bytes); };
    for (int k = 0; k < n; k += 4) {
      uint4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (k + e < n) v[e] = *at(len + r[k + e]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (k + e < n && r[k + e] != k + e) *at(len + k + e) = v[e];
    }
  }
}

cudaError_t launch_after(const void* f, int grid, int threads, const PagesArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {(void*)&a};
  return cudaLaunchKernelExC(&cfg, f, args);
}

}  // namespace

size_t pages_bytes(int n_pages, int n) {
  // the head; three words a copy, one a page handed out and one a run (fork), one a page (reserve), two a page (compact)
  return (size_t)4 * (64 + std::max(5 * N_MAX, 2 * n_pages));
}

int pages_reserve(const PagesArgs& a, cudaStream_t st) {
  reserve_kernel<<<1, PT, 0, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? 1 : -1;
}
int pages_release(const PagesArgs& a, cudaStream_t st) {
  release_kernel<<<1, PT, 0, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? 1 : -1;
}
int pages_fork(const PagesArgs& a, cudaStream_t st) {
  fork_kernel<<<1, PT, 0, st>>>(a);
  if (cudaPeekAtLastError() != cudaSuccess) return -1;
  return launch_after((const void*)fork_copy_kernel, (int)std::min<long long>(16ll * num_sms(), (2ll * a.L * a.planes + a.d / HID + 1) * a.n), 128, a, st) == cudaSuccess ? 2 : -1;
}
int pages_compact(const PagesArgs& a, cudaStream_t st) {
  compact_kernel<<<1, PT, 0, st>>>(a);
  if (cudaPeekAtLastError() != cudaSuccess) return -1;
  return launch_after((const void*)compact_copy_kernel, 8 * num_sms(), 256, a, st) == cudaSuccess ? 2 : -1;
}
int rows_keep(const KeepArgs& a, cudaStream_t st) {
  const long long vecs = (long long)a.L * a.planes * (a.row_bytes / 16);
  rows_keep_kernel<<<dim3((unsigned)std::min<long long>((vecs + 255) / 256, 65535), a.B), 256, 0, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? 1 : -1;
}

}  // namespace spec
