// Page tables and slot maps of a paged cache, built on the GPU from request lengths.
//
// Request b holds have[b] entries in pages(have) = ceil(have / P) pages and gets new[b] more
// (negative: drops its last -new).  With three exclusive sums over the requests
//   rows  R_b = sum max(new, 0)              one map row per new entry,
//   need  N_b = sum pages(have + new) - pages(have)  (new >= 0)   pages taken,
//   gone  G_b = sum pages(have) - max(pages(have + new), kept)  (new < 0)   pages given back,
// every output is a closed form: given back page i goes to free[n_free + i], taken page a is the
// stack's element n_free + G - 1 - a (an element at or above n_free is the given back page itself,
// so nothing waits for the pushes), and row r finds its request by a search in R.
//
// The work is a few kilobytes: launches and dependent loads bound it, not bandwidth.
#include "common.cuh"
#include "ptx.cuh"
#include "timing.cuh"

namespace csa2 {
namespace {

constexpr int kPlanThreads = 1024;  // at most

struct PageArgs {
  int32_t B;
  const int32_t* have;
  const int32_t* add;
  const int32_t* kept;  // or null: 0
  int32_t P, m;
  int32_t* table;
  int32_t max_pages, n_pages;
  int32_t* free_pages;
  const int32_t* n_free;
  int32_t* n_free_out;
  int32_t* n_entries;
  int32_t n_rows;
  int32_t* query;  // the maps, each or null
  int32_t* slot;
  int64_t* entry;
  int64_t* pos;
  int32_t* row_start;
  void* ws;
};

// What the plan leaves for the fill: the sums, the lengths read before n_entries overwrites them,
// the totals (total rows 0 and ok 0 after an error).
struct PlanState {
  int32_t ok, n_free, total_rows, total_gone;
};
struct PlanView {
  int32_t* have;  // [B]
  int32_t* rows;  // [B + 1] exclusive sums
  int32_t* need;  // [B + 1]
  int32_t* gone;  // [B + 1]
  PlanState* st;
  int32_t* ids;   // the first id_cap ids that move, given back ones first, as the checks have read them
  int id_cap;     // 0: they are read again
};

__device__ __forceinline__ int pages_of(int n, int P) {  // n >= 0
  return n > 0 ? (int)((uint32_t)(n - 1) / (uint32_t)P) + 1 : 0;
}

// largest i in [lo, hi) with sum[i] <= x (sum ascending, sum[lo] <= x)
__device__ __forceinline__ int find_le(const int32_t* sum, int lo, int hi, int x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// given back page i
__device__ __forceinline__ int find_gone(const PageArgs& a, const PlanView& v, int i) {
  const int b = find_le(v.gone, 0, a.B, i);
  const int first = pages_of(v.have[b], a.P) - (v.gone[b + 1] - v.gone[b]);
  return a.table[(int64_t)b * a.max_pages + first + i - v.gone[b]];
}
__device__ __forceinline__ int gone_page(const PageArgs& a, const PlanView& v, int i) {
  return i < v.id_cap ? v.ids[i] : find_gone(a, v, i);
}
// taken page i: from the top of the stack, on which the pages given back by this call lie
__device__ __forceinline__ int taken_page(const PageArgs& a, const PlanView& v, int i) {
  const int gone = v.st->total_gone;
  if (i < gone) return gone_page(a, v, gone - 1 - i);
  return i < v.id_cap ? v.ids[i] : a.free_pages[v.st->n_free + gone - 1 - i];
}

// Exclusive sums over the block of three values a thread, and their totals.  32-bit steps where no value
// reaches 2^20 (1,024 of them stay below 2^30), else 64-bit ones.
template <typename T>
__device__ __forceinline__ void block_scan3(const T (&x)[3], T (*s_warp)[kPlanThreads / 32], long long (&before)[3],
                                            long long (&total)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T inc[3] = {x[0], x[1], x[2]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const T y = __shfl_up_sync(0xffffffffu, inc[q], o);
      if (lane >= o) inc[q] += y;
    }
  if (lane == 31)
#pragma unroll
    for (int q = 0; q < 3; ++q) s_warp[q][warp] = inc[q];
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    T w = lane < warps ? s_warp[q][lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    const T b = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    total[q] = __shfl_sync(0xffffffffu, w, 31);
    before[q] = (long long)(inc[q] - x[q]) + (warp > 0 ? (long long)b : 0);
  }
  __syncthreads();  // s_warp is written again by the next strip
}

// The plan, by one CTA: sums, checks, n_entries, n_free_out, row_start.  It also clears the error word,
// which no other CTA of the call writes.
__device__ void plan_block(const PageArgs& a, const PlanView& v) {
  __shared__ union {
    long long l[3][kPlanThreads / 32];
    int i[3][kPlanThreads / 32];
  } s_warp;
  __shared__ int s_bad;
  const int tid = threadIdx.x, step = blockDim.x;
  const int n_free = *a.n_free;
  if (tid == 0) {
    s_bad = 0;
    *reinterpret_cast<ErrWord*>(a.ws) = ErrWord{0, 0, 0};
    v.rows[0] = v.need[0] = v.gone[0] = 0;
  }
  __syncthreads();
  const long long cap = min((long long)a.max_pages * a.P, (long long)INT32_MAX);
  long long base[3] = {0, 0, 0};
  for (int b0 = 0; b0 < a.B; b0 += step) {
    const int b = b0 + tid;
    int x[3] = {0, 0, 0};
    if (b < a.B) {
      const int have = a.have[b], add = a.add[b], kept = a.kept ? a.kept[b] : 0;
      const long long total = (long long)have + add;
      v.have[b] = have;
      if (have < 0 || total < 0 || have > cap || total > cap || kept < 0) {
        s_bad = 1;
        report_error(a.ws, CSA2_ERR_INDEX_RANGE, b);
      } else {
        const int pc = pages_of(have, a.P), pa = pages_of((int)total, a.P);
        if (add >= 0) {
          x[0] = add;
          x[1] = pa - pc;
        } else {
          x[2] = pc - max(pa, min(kept, pc));
        }
      }
    }
    long long before[3], total[3];
    if (__syncthreads_or(max(max(x[0], x[1]), x[2]) >= 1 << 20)) {
      const long long y[3] = {x[0], x[1], x[2]};
      block_scan3<long long>(y, s_warp.l, before, total);
    } else {
      block_scan3<int>(x, s_warp.i, before, total);
    }
    if (b < a.B) {  // sums past 32 bits are refused below; what they leave here is not used
      v.rows[b + 1] = (int)(base[0] + before[0] + x[0]);
      v.need[b + 1] = (int)(base[1] + before[1] + x[1]);
      v.gone[b + 1] = (int)(base[2] + before[2] + x[2]);
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) base[q] += total[q];
  }
  if (tid == 0) {
    const bool maps = a.query || a.slot || a.entry || a.pos;
    if (base[0] > INT32_MAX || (maps && base[0] > a.n_rows)) {
      s_bad = 1;
      report_error(a.ws, CSA2_ERR_INDEX_RANGE, base[0]);
    }
    if (n_free < 0 || n_free > a.n_pages || base[2] > a.n_pages - n_free) {
      s_bad = 1;
      report_error(a.ws, CSA2_ERR_INDEX_RANGE, n_free);
    } else if (base[1] > n_free + base[2]) {
      s_bad = 1;
      report_error(a.ws, CSA2_ERR_NO_PAGES, base[1] - n_free - base[2]);
    }
    *v.st = PlanState{1, n_free, (int)base[0], (int)base[2]};
  }
  __syncthreads();
  if (!s_bad) {  // the ids that would move: a bad one refuses the call
    bool bad = false;
    int id = 0;
    const int from_stack = (int)min(max(base[1] - base[2], 0LL), (long long)n_free);
    const int gone = (int)base[2], moved = gone + from_stack;  // ids, at most n_pages
    for (int i = tid; i < moved && !bad; i += step) {
      id = i < gone ? find_gone(a, v, i) : a.free_pages[n_free - 1 - (i - gone)];
      bad = id < 0 || id >= a.n_pages;
      if (i < v.id_cap) v.ids[i] = id;
    }
    if (bad) report_error(a.ws, CSA2_ERR_INDEX_RANGE, id);
    if (__syncthreads_or(bad) && tid == 0) s_bad = 1;
  }
  __syncthreads();
  const bool ok = !s_bad;
  if (tid == 0) {
    if (!ok) *v.st = PlanState{0, n_free, 0, 0};
    *a.n_free_out = ok ? (int)(n_free + base[2] - base[1]) : n_free;
    if (a.row_start) a.row_start[0] = 0;
  }
  for (int b = tid; b < a.B; b += step) {
    a.n_entries[b] = ok ? v.have[b] + a.add[b] : v.have[b];
    if (a.row_start) a.row_start[b + 1] = ok ? v.rows[b + 1] : 0;
  }
  __syncthreads();
}

// The map's rows, by the calling threads (row r, r + step, ..).
__device__ void fill_rows(const PageArgs& a, const PlanView& v, int64_t r, int64_t step) {
  const int total = v.st->total_rows;
  for (; r < a.n_rows; r += step) {
    int b = -1, slot = -1;
    int64_t off = -1, pos = -1;
    if (r < total) {
      b = find_le(v.rows, 0, a.B, (int)r);
      const int have = v.have[b];
      const int e = have + (int)r - v.rows[b];
      const int p = (int)((uint32_t)e / (uint32_t)a.P), pc = pages_of(have, a.P);
      slot = p < pc ? a.table[(int64_t)b * a.max_pages + p] : taken_page(a, v, v.need[b] + p - pc);
      off = e - p * a.P;
      pos = (int64_t)e * a.m;
    }
    if (a.query) a.query[r] = b;
    if (a.slot) a.slot[r] = slot;
    if (a.entry) a.entry[r] = off;
    if (a.pos) a.pos[r] = pos;
  }
}
// The pages that move, by the calling threads (tid i of step): taken ones into their rows, given back
// ones onto the stack.
__device__ void fill_pages(const PageArgs& a, const PlanView& v, int64_t first, int64_t step) {
  if (!v.st->ok) return;
  const int taken = v.need[a.B], gone = v.gone[a.B];
  for (int64_t i = first; i < taken; i += step) {
    const int b = find_le(v.need, 0, a.B, (int)i);
    a.table[(int64_t)b * a.max_pages + pages_of(v.have[b], a.P) + i - v.need[b]] = taken_page(a, v, (int)i);
  }
  for (int64_t i = first; i < gone; i += step) a.free_pages[v.st->n_free + i] = gone_page(a, v, (int)i);
}

// Everything in one CTA, the plan and the first kIds ids in shared memory.
constexpr int kIds = 2048;
__global__ void __launch_bounds__(kPlanThreads) k_page_tables(PageArgs a) {
  extern __shared__ int32_t smem[];
  __shared__ PlanState st;
  __shared__ int32_t ids[kIds];
  const PlanView v{smem, smem + a.B, smem + 2 * a.B + 1, smem + 3 * a.B + 2, &st, ids, kIds};
  ptx::griddep_wait();
  plan_block(a, v);
  fill_pages(a, v, threadIdx.x, blockDim.x);
  fill_rows(a, v, threadIdx.x, blockDim.x);
}

// The plan by one CTA into the workspace, then the fill by many.
__global__ void __launch_bounds__(kPlanThreads) k_page_plan(PageArgs a, PlanView v) {
  ptx::griddep_launch();
  ptx::griddep_wait();
  plan_block(a, v);
}
constexpr int kFillThreads = 256;
__global__ void __launch_bounds__(kFillThreads) k_page_fill(PageArgs a, PlanView v) {
  ptx::griddep_wait();
  const int64_t t = (int64_t)blockIdx.x * kFillThreads + threadIdx.x, n = (int64_t)gridDim.x * kFillThreads;
  fill_pages(a, v, t, n);
  fill_rows(a, v, t, n);
}

// One CTA up to this many map rows and requests (whose plan its shared memory holds).  From a graph, one CTA /
// plan and fill, us: 64 requests with 1,000 new entries 4.8 / 7.0, 256 with 1,000 5.8 / 7.0, 2,000 with 1,000
// 8.7 / 11.5; 64 with 4,000 7.5 / 6.9, 256 with 4,000 8.0 / 7.6, 64 with 8,000 10.7 / 6.8.
constexpr int kOneCtaRows = 2048, kOneCtaRequests = 2048;

PlanView plan_view(void* ws, int32_t B, size_t* bytes) {
  size_t off = kWsHeader;
  char* base = (char*)ws;
  auto take = [&](size_t n) {
    char* p = base ? base + off : nullptr;
    off += align_up(n, 256);
    return (int32_t*)p;
  };
  PlanView v;
  v.st = (PlanState*)take(sizeof(PlanState));
  v.have = take((size_t)B * 4);
  v.rows = take(((size_t)B + 1) * 4);
  v.need = take(((size_t)B + 1) * 4);
  v.gone = take(((size_t)B + 1) * 4);
  v.ids = nullptr;
  v.id_cap = 0;
  if (bytes) *bytes = off;
  return v;
}

}  // namespace
}  // namespace csa2

extern "C" size_t csa2_page_tables_workspace_size(int32_t B) {
  if (B <= 0 || B > 65535) return 0;
  size_t n;
  csa2::plan_view(nullptr, B, &n);
  return n;
}

extern "C" csa2_status csa2_page_tables(int32_t B, const int32_t* n_have, const int32_t* n_new, int32_t page_entries,
                                        int32_t m, const int32_t* n_kept, int32_t* page_table, int32_t max_pages,
                                        int32_t n_pages, int32_t* free_pages, const int32_t* n_free,
                                        int32_t* n_free_out, int32_t* n_entries, int32_t n_rows, int32_t* row_query,
                                        int32_t* row_slot, int64_t* row_entry, int64_t* row_pos, int32_t* row_start,
                                        void* ws, size_t ws_bytes, csa2_stream stream) {
  using namespace csa2;
  if (B <= 0 || B > 65535 || page_entries <= 0 || m <= 0 || max_pages < 0 || n_pages <= 0 || n_rows < 0)
    return CSA2_ERR_INVALID_ARG;
  if (!n_have || !n_new || (max_pages > 0 && !page_table) || !free_pages || !n_free || !n_free_out || !n_entries)
    return CSA2_ERR_INVALID_ARG;
  const void* p4[] = {n_have, n_new, n_kept, page_table, free_pages, n_free, n_free_out, n_entries, row_query,
                      row_slot, row_start};
  for (const void* p : p4)
    if (!aligned(p, 4)) return CSA2_ERR_INVALID_ARG;
  if (!aligned(row_entry, 8) || !aligned(row_pos, 8)) return CSA2_ERR_INVALID_ARG;
  if (n_rows > 0 && !row_query && !row_slot && !row_entry && !row_pos) return CSA2_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256)) return CSA2_ERR_WORKSPACE;
  size_t need;
  const PlanView v = plan_view(ws, B, &need);
  if (ws_bytes < need) return CSA2_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  const PageArgs a{B, n_have, n_new, n_kept, page_entries, m, page_table, max_pages, n_pages, free_pages, n_free,
                   n_free_out, n_entries, n_rows, row_query, row_slot, row_entry, row_pos, row_start, ws};
  if (n_rows <= kOneCtaRows && B <= kOneCtaRequests) {
    KernelTimer timer("k_page_tables", st);
    // a thread for each request and each row: fewer warps wait less for one another
    const int want = B > n_rows ? B : n_rows;
    const int threads = want > kPlanThreads ? kPlanThreads : want < 128 ? 128 : (want + 31) / 32 * 32;
    launch_pdl(k_page_tables, dim3(1), dim3(threads), (4 * (size_t)B + 3) * 4, st, a);
  } else {
    {
      KernelTimer timer("k_page_plan", st);
      if (launch_pdl(k_page_plan, dim3(1), dim3(kPlanThreads), 0, st, a, v) != cudaSuccess)
        return launch_status();  // the fill would follow whatever plan the workspace held
    }
    const int64_t threads = n_rows > 4096 ? n_rows : 4096;
    const int blocks = (int)(cdiv(threads, kFillThreads) < 1216 ? cdiv(threads, kFillThreads) : 1216);
    KernelTimer timer("k_page_fill", st);
    launch_pdl(k_page_fill, dim3(blocks), dim3(kFillThreads), 0, st, a, v);
  }
  return launch_status();
}
