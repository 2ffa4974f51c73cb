// Commit of the accepted tokens of draft trees (csa2_tree_commit): their entries move up behind the context, their
// window rows enter the ring.
//
// A CTA has a request: all its entries are read before one is written, so the path's order does not matter.  The
// work is a few kilobytes a request: launches and dependent loads (lengths and path, pages, entries) bound it.  From a
// graph 16 trees of 16 tokens 2.8 us, 256 of up to 64 7.4 (6.7 MB; 6.4 without the CTAs that report).
#include "ptx.cuh"
#include "timing.cuh"
#include "common.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 256;
// CTAs that look at what is asked for: a cluster, so that none reports before the word is cleared; one for few paths
constexpr int kReporters = 8, kManyPlaces = 512;
constexpr int kPieces = 23;  // of an entry: 16 x 16 bytes of main codes, 2 of scales, 4 of key codes, 4 bytes of scales
constexpr int kHold = (CSA2_MAX_TREE * kPieces + kThreads - 1) / kThreads;

struct CommitArgs {
  csa2_kv_planes kv;
  const int32_t* table;
  int32_t max_pages, n_pages;
  csa2_trees trees;
  const int32_t *n_entries, *n_accept, *path;
  int32_t n_path;
  int32_t* n_new;
  const uint8_t* draft;
  const int64_t* pos;
  uint8_t* ring;
  int64_t* ring_pos;
  int32_t n_win, reporters;
  void* ws;
};

// what request g asks for; false where its numbers are out of range
struct Commit {
  int first, tokens, keep, have;
  int64_t pos;
};
__device__ __forceinline__ bool commit_of(const CommitArgs& a, int g, Commit& c) {
  const int lo = a.trees.start[g], hi = a.trees.start[g + 1];
  c.first = lo;
  c.tokens = hi - lo;
  c.keep = a.n_accept[g];
  c.have = a.trees.entries ? a.n_entries[g] : 0;
  c.pos = a.n_win > 0 ? a.pos[g] : 0;
  if (lo < 0 || hi < lo || hi > a.trees.B || c.tokens > a.trees.max_tokens) return false;
  if (c.keep < 0 || c.keep > min(c.tokens, a.n_path) || c.have < 0) return false;
  if (c.pos < 0 || c.pos > INT64_MAX - CSA2_MAX_TREE) return false;  // the last token's position is one too
  return !a.trees.entries || (int64_t)c.have + c.tokens <= (int64_t)a.max_pages * a.kv.seq_stride;
}
// plane row of entry e of request g, or -1
__device__ __forceinline__ int64_t row_of(const CommitArgs& a, int g, int64_t e) {
  const int64_t pi = e / a.kv.seq_stride;
  const int page = a.table[(int64_t)g * a.max_pages + pi];
  return page < 0 || page >= a.n_pages ? -1 : page * a.kv.seq_stride + (e - pi * a.kv.seq_stride);
}
// place i of request g's path, whether it counts or not: asked for with the lengths that say so
__device__ __forceinline__ int path_at(const CommitArgs& a, int g, int i) {
  return i < a.n_path ? a.path[(int64_t)g * a.n_path + i] : -1;
}
// the rows of token t's entry, place i of the path, by one thread; false where they are none
__device__ __forceinline__ bool kept_token(const CommitArgs& a, int g, const Commit& c, int i, int t, int64_t& from,
                                           int64_t& to) {
  from = to = 0;
  if (t < 0 || t >= c.tokens) return false;
  if (!a.trees.entries) return true;
  from = row_of(a, g, (int64_t)c.have + t);
  to = row_of(a, g, (int64_t)c.have + i);
  return from >= 0 && to >= 0;
}

__device__ __forceinline__ const uint8_t* piece_at(const csa2_kv_planes& p, int64_t row, int i) {
  return i < 16 ? p.kv_codes + row * 256 + 16 * i
         : i < 18 ? p.kv_scales + row * 32 + 16 * (i - 16)
         : i < 22 ? p.ix_codes + row * 64 + 16 * (i - 18) : p.ix_scales + row * 4;
}

__global__ void __launch_bounds__(kThreads) k_tree_commit(CommitArgs a) {
  __shared__ int s_token[CSA2_MAX_TREE];
  __shared__ int64_t s_from[CSA2_MAX_TREE], s_to[CSA2_MAX_TREE];
  ptx::griddep_launch();
  ptx::griddep_wait();
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < a.reporters) {  // these report: the error word is theirs alone
    if (blockIdx.x == 0 && tid == 0) *reinterpret_cast<ErrWord*>(a.ws) = ErrWord{0, 0, 0};
    if (a.reporters > 1) ptx::cluster_sync();
    else __syncthreads();
    const int per = max(min(a.n_path, CSA2_MAX_TREE), 1), all = a.trees.R * per;  // a thread for each place of each path
#pragma unroll 4
    for (int i = blockIdx.x * kThreads + tid; i < all; i += a.reporters * kThreads) {
      const int g = i / per, k = i - g * per;
      Commit c;
      int64_t from, to;
      const int t = path_at(a, g, k);
      if (!commit_of(a, g, c) || (k < c.keep && !kept_token(a, g, c, k, t, from, to)))
        report_error(a.ws, CSA2_ERR_INDEX_RANGE, g);
    }
    return;
  }
  const int g = (int)blockIdx.x - a.reporters;
  if (g >= a.trees.R) return;
  Commit c;
  const int t = tid < CSA2_MAX_TREE ? path_at(a, g, tid) : -1;
  bool ok = commit_of(a, g, c);
  if (ok && tid < c.keep) {
    s_token[tid] = t;
    ok = kept_token(a, g, c, tid, t, s_from[tid], s_to[tid]);
  }
  ok = __syncthreads_and(ok);
  if (a.n_new && tid == 0) a.n_new[g] = ok && a.trees.entries ? c.keep - c.tokens : 0;
  if (!ok) return;
  const int skip = max(c.keep - a.n_win, 0);  // of more tokens than the ring has places the last are kept
  for (int i = tid; a.n_win > 0 && i < (c.keep - skip) * 32; i += kThreads) {
    const int k = skip + i / 32;
    const int64_t p = c.pos + k, place = (int64_t)g * a.n_win + p % a.n_win;
    reinterpret_cast<uint4*>(a.ring + place * kDMain)[i % 32] =
        reinterpret_cast<const uint4*>(a.draft + (int64_t)(c.first + s_token[k]) * kDMain)[i % 32];
    if (i % 32 == 0) a.ring_pos[place] = p;
  }
  if (!a.trees.entries) return;
  uint4 held[kHold];
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    const int i = tid + j * kThreads, k = i / kPieces, piece = i % kPieces;
    if (k >= c.keep || s_from[k] == s_to[k]) continue;
    const uint8_t* src = piece_at(a.kv, s_from[k], piece);
    if (piece < 22) held[j] = *reinterpret_cast<const uint4*>(src);
    else held[j].x = *reinterpret_cast<const uint32_t*>(src);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    const int i = tid + j * kThreads, k = i / kPieces, piece = i % kPieces;
    if (k >= c.keep || s_from[k] == s_to[k]) continue;
    uint8_t* dst = const_cast<uint8_t*>(piece_at(a.kv, s_to[k], piece));
    if (piece < 22) *reinterpret_cast<uint4*>(dst) = held[j];
    else *reinterpret_cast<uint32_t*>(dst) = held[j].x;
  }
}

}  // namespace
}  // namespace csa2

extern "C" size_t csa2_tree_commit_workspace_size(int32_t R) { return R <= 0 || R > 65535 ? 0 : csa2::kWsHeader; }

extern "C" csa2_status csa2_tree_commit(const csa2_kv_planes* kv, const csa2_pages* pages, const csa2_trees* trees,
                                        const int32_t* n_entries, const int32_t* n_accept, const int32_t* path,
                                        int32_t n_path, int32_t* n_new, const uint8_t* draft_e4m3, const int64_t* pos,
                                        uint8_t* ring, int64_t* ring_pos, int32_t n_win, void* ws, size_t ws_bytes,
                                        csa2_stream stream) {
  using namespace csa2;
  if (!trees || !trees->start || !aligned(trees->start, 4) || trees->R <= 0 || trees->R > 65535 || trees->B < 0 ||
      trees->max_tokens < 1 || trees->max_tokens > CSA2_MAX_TREE)
    return CSA2_ERR_INVALID_ARG;
  if (!n_accept || n_path < 0 || (n_path > 0 && !path) || n_win < 0 || !aligned(n_accept, 4) || !aligned(path, 4) ||
      !aligned(n_new, 4))
    return CSA2_ERR_INVALID_ARG;
  if (n_win > 0 && (!draft_e4m3 || !pos || !ring || !ring_pos || !aligned(draft_e4m3, 16) || !aligned(pos, 8) ||
                    !aligned(ring, 16) || !aligned(ring_pos, 8)))
    return CSA2_ERR_INVALID_ARG;
  if (trees->entries) {
    if (!planes_ok(kv) || !pages || pages->max_pages < 0 || pages->n_pages < 0 || kv->seq_stride > INT32_MAX ||
        (pages->max_pages > 0 && !pages->table) || !aligned(pages->table, 4) || !n_entries || !aligned(n_entries, 4))
      return CSA2_ERR_INVALID_ARG;
  }
  if (!ws || !aligned(ws, 256) || ws_bytes < kWsHeader) return CSA2_ERR_WORKSPACE;
  CommitArgs a{};
  if (trees->entries) {
    a.kv = *kv;
    a.table = pages->table;
    a.max_pages = pages->max_pages;
    a.n_pages = pages->n_pages;
  }
  a.trees = *trees;
  a.n_entries = n_entries;
  a.n_accept = n_accept;
  a.path = path;
  a.n_path = n_path;
  a.n_new = n_new;
  a.draft = draft_e4m3;
  a.pos = pos;
  a.ring = ring;
  a.ring_pos = ring_pos;
  a.n_win = n_win;
  a.ws = ws;
  cudaStream_t st = (cudaStream_t)stream;
  KernelTimer timer("k_tree_commit", st);
  a.reporters = (int64_t)trees->R * n_path > kManyPlaces ? kReporters : 1;
  const unsigned ctas = (unsigned)align_up((size_t)(a.reporters + trees->R), (size_t)a.reporters);
  if (a.reporters > 1) launch_clusters(k_tree_commit, dim3(ctas), dim3(kThreads), a.reporters, 1, 0, st, a);
  else launch_pdl(k_tree_commit, dim3(ctas), dim3(kThreads), 0, st, a);
  return launch_status();
}
