// Attention through page tables: for queries by themselves, for a batch whose queries share prefixes, and for trees of
// drafted tokens.
//
// out = softmax(scale q X^T) X over the rows X that a query sees: the entries its table row names, then its
// window.  With z the logits in log2 units, a part of the rows leaves its reference m, l = sum 2^(z - m) and
// O / l = sum 2^(z - m) x / l; parts join by log-sum-exp.  Each call is three launches:
//   k_prefix_prep   the plan (which chunks of rows every CTA runs), the queries' f16 images, and the image:
//                   the shared entries of large groups, widened to f16 once;
//   k_paged_attn    one query to a CTA (without groups, or with small ones), or
//   k_prefix_attn   two queries of a group to a pair of CTAs;
//   k_paged_merge / k_prefix_merge   the join, the sink, the turn back, the output's type.
// All chunks form one list that the CTAs share evenly, whatever the queries' lengths; a query cut between
// CTAs leaves a partial in each, in fp32 for an fp32 output and in f16 for a bf16 one (Vec8).
//
// Pairs.  Two queries of a group make a pair, and their 2 x 64 heads the 128 rows of one MMA, so an entry of
// the shared prefix serves two queries and the tensor cores run at their full rate (64 rows alone run at half
// of it).  A pair of CTAs (one query each) computes with tcgen05.mma.cta_group::2 in chunks of 128 rows:
//   S[128 x 128 rows] = q' X^T   each CTA holds 64 of the rows (all channels), K-major;
//   P = 2^(S c2 - m)             each CTA its own query: thread t head t % 64, rows 64 (t / 64) ..;
//   O[128 x 512] += P X          each CTA holds 256 of the channels (all rows), N-major.
// At M = 128 a CTA's tensor memory holds 64 rows of an accumulator in 128 lanes, so O takes 256
// columns and leaves room for two S buffers; neither operand is exchanged between the CTAs: each holds the
// 64 x 512 values of S and the 128 x 256 of O.  Chunks of the image come as they are by tensor copies (widened
// by every pair for itself 768 us a call on 64 queries of 65,000 shared entries, from the image 451); the rest
// is widened by the row warps.  Shared memory bounds a chunk: 128 KB read by the S MMAs, 96 KB by the O MMAs,
// 128 KB of rows and 16 KB of P written, 368 KB = 2,900 cycles at 128 bytes a cycle, against 2,048 cycles of
// MMA; measured, 3,400 to 3,900, the waits of the odd CTA's arrivals among them.  With one buffer for each operand there is no room for a second chunk, so both
// are handed over in four pieces (128 channels of S's rows, 32 rows of O's).
// Behind the shared entries come the two queries' own (their last entries and windows): chunks whose
// first 64 rows are the first query's and whose last 64 the second's, each query masking the other's; behind
// the shorter's last, 128 rows of the longer.
// Trees of drafted tokens (kTree): a request's queries share all its rows, its context and behind it the drafts' entries,
// its ring and the drafts' window rows, of which each query sees its own path's.  The preparation follows the parents
// (tree_block); whole chunks of context come from the image, the others' rows carry in a bit whether the CTA's query sees
// them (flip_seen), and probabilities of rows that it does not are 0.  Measured: 16 trees of 16 tokens on 8,192 entries,
// normalised and rotated, 281 us (0.99 PFLOP/s), 4 of 64 on 65,000 1,580 us (1.38 PFLOP/s), one of 8 on 4,096 22 us.
// Measured: 64 queries on 65,000 shared entries 405 us, 1.35 PFLOP/s, 71 % of the rate of a library bf16
// product; 32 on 8,192, normalised and rotated, 51 us.
#include <algorithm>
#include <type_traits>

#include "attn.cuh"
#include "index_scan.cuh"
#include "rotary.cuh"

namespace csa2 {
namespace {

constexpr int kPrepThreads = 512;
constexpr int kClusters = 76;    // CTA pairs of a launch: one for every two of the 152 SMs
constexpr int kChunk = 128;      // rows of a chunk
constexpr int kOwnChunk = 64;    // of which each query of a pair has this many in an own chunk
// A group of at least this many queries has its shared entries widened once: 64 queries on 8,192 entries, groups of
// four: 114 us with the image, 94 without; of five 116 and 110, six 100 and 96, eight 92 and 94, sixteen 82 and 94.
// Batches whose groups are smaller than this on average run every query by itself.  Two queries of a pair share every
// row, but an odd group's last query takes a pair's time, and own rows cost a pair more.  In pairs / by themselves, us,
// 64 on 8,192, groups of equal size: one 166 / 100, two 98 / 99, three 115 / 98, four 93 / 97, five 116 / 98, six
// 100 / 100, eight 92 / 97, sixteen 82 / 97; groups and lengths drawn at random: 4 on average 94 / 77, 8 80 / 71,
// 13 92 / 84 to 77 / 85, 20 (101 on 4,001) 68 / 75, 32 65 / 82.  The host knows the average alone: five is about where
// equal groups break even, even ones below and odd ones above it; random ones do so at about thirteen.
constexpr int kImageQueries = 5;
// Queries times shared entries below which every query runs by itself all the same, its ramp being shorter.  In
// pairs / by themselves, us: 8 queries on 8,192 entries 33 / 27, 32 on 2,000 31 / 27, 128 on 500 38 / 36; 16 on 8,192
// 37 / 38, 128 on 1,000 45 / 45, 64 on 2,000 39 / 41; 16 on 16,384 48 / 57, 64 on 4,000 51 / 58.
constexpr int64_t kPairWork = 1 << 17;
constexpr int kTreesPerCta = kPrepThreads / 32;
constexpr int kWidenCtas = 304;    // CTAs that widen, two for every SM,
constexpr int kWidenFirst = 152;   // of which these come before the queries' staging
constexpr int64_t kImageChunks = 8192;  // at most this many chunks (128 KB each) of the workspace

// Two queries of a group (q1 = -1: one), and their rows: the group's shared entries [0, ns), seen
// up to vis by each, then each query's own entries ns .. ns + own - 1 and its window.
// Trees of drafted tokens (kTree): all of a request's rows are shared, its context, its drafts' entries, its ring and
// its drafts' window rows, of which each query sees some (see Sight).  Then first is the request, ns its entries,
// vis0 those of the context, vis1 the tree's tokens, own0 the first of them.
struct Pair {
  int32_t q0, own0;
  int32_t chunk0;  // this pair's first chunk in the order of all pairs' chunks
  int32_t q1, own1;
  int32_t first;  // the query whose table row holds the shared entries
  int32_t ns;
  int32_t vis0, vis1;
  int32_t paired;  // own chunks that hold 64 rows of each query; behind them 128 of the longer one's
  int32_t nshared; // shared chunks; own chunks follow
  int32_t image;   // the shared entries' first chunk in the image, or -1
};

// What one part (a CTA, or a pair of CTAs) of the attention launch runs: chunks [t0, t1) of the order of all
// pairs' chunks, beginning in `pair`, number p, whose chunks end at `end`.  The first item needs no further
// load, and a query by itself no more than the first 32 bytes.
struct __align__(16) Part {
  int32_t p, t0, t1, end;
  Pair pair;
};

// The queries' staging: what it reads, and where it leaves their images.
struct PrefixQuery {
  const uint16_t* q;
  const float* norm_w;
  float eps, scale;
  int rope;
  const int64_t* qpos;
  RopeTheta th;
  uint16_t* image;  // [B + 1][c/8][head][c%8] f16
  float* c2;        // [B + 1][64]
  float2* turn;     // [B][32]
  uint16_t* rest;   // [B][head][c] what the rounding to f16 took from q', in q's scale (f16); null: not kept
};

struct PrefixArgs {
  int32_t B, G;
  const int32_t* n_entries;
  const int32_t* group_start;  // G == 0: null
  const int32_t* n_shared;
  int32_t shared_max, own_max, n_swa;
  int64_t table_cap;  // entries a table row can hold
  Pair* pairs;        // [pairs + 1], the last one holds the number of chunks
  int32_t* gpair;     // [G + 3] first pair of each range of queries
  int32_t* chunk0;    // [pairs + 1] first chunk of each pair (these two where shared memory is too small)
  int2* qpart;        // [B] first partial (see the merges), partials
  Part* parts_of;     // [parts]
  int32_t* gimage;    // [G] first image chunk of each group, or -1
  int2* gshared;      // [G] see shared_of (where shared memory is too small)
  int64_t image_cap;  // chunks the image has room for
  int32_t parts;      // CTAs (one query each) or pairs of CTAs that share the chunks
  void* ws;
  // trees: group_start has their first tokens, n_entries [G] the contexts, shared_max the bound of those
  const int32_t* parent;
  int32_t max_tokens, entries;
  int32_t* cost0;     // [pairs + 1] cost of the pairs before each (where shared memory is too small)
  uint64_t* kin;      // [B] itself and its ancestors, bit t token t of the request
  int32_t* depth;     // [B] how many ancestors; + kBadParent where the parent is none
};
constexpr int32_t kBadParent = INT32_MIN;

// whether a batch runs every query by itself
__host__ __device__ __forceinline__ bool by_itself(int32_t B, int32_t G, int64_t shared_max) {
  return G == 0 || B < (int64_t)kImageQueries * G || B * shared_max < kPairWork;
}
// The same for trees, which share all their rows: the more tokens a tree has, the more a row of the image serves.  In pairs /
// by themselves, us: trees of five on 2,000 (160,000 queries times entries) 54 / 50, on 4,000 80 / 72; of eight on 5,000
// (160,000) 44.7 / 43.5; of nine on 20,000 (180,000) 47 / 45, on 40,000 68 / 73; of 16 on 5,000 (80,000) 32.6 / 32.5, on
// 9,000 38.5 / 40.4; of 32 on 700 (90,000) 39 / 44; of 64 on 700 (45,000) 31.7 / 33.2.
constexpr int64_t kTreeWork = 1 << 21;
__host__ __device__ __forceinline__ bool trees_by_themselves(int32_t B, int32_t R, int64_t n_max) {
  return B < (int64_t)kImageQueries * R || (int64_t)B * B * n_max < kTreeWork * R;
}
template <bool kTree>
__host__ __device__ __forceinline__ bool alone_of(int32_t B, int32_t G, int64_t shared_max) {
  return kTree ? trees_by_themselves(B, G, shared_max) : by_itself(B, G, shared_max);
}
// pairs of a batch, at most
__host__ __device__ __forceinline__ int max_pairs(int32_t B, int32_t G) { return (B + G + 2) / 2; }

// exclusive sum over the block of x (all threads call); total = the block's sum
__device__ __forceinline__ int block_scan(int x, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int w = lane < kPrepThreads / 32 ? s_warp[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  *total = __shfl_sync(0xffffffffu, w, 31);
  __syncthreads();
  return inc - x + (warp > 0 ? before : 0);
}

// The pairs of the batch and the chunks of each, by one CTA.  Ranges of queries: those before the
// first group, the G groups, those behind the last (a range outside the groups shares nothing).
__device__ __forceinline__ int visible(const int32_t* n_entries, int64_t table_cap, int q) {
  return (int)min((long long)max(n_entries[q], 0), (long long)table_cap);
}
__device__ __forceinline__ int visible(const PrefixArgs& a, int q) { return visible(a.n_entries, a.table_cap, q); }
// Of queries [q, end), by a warp, 128 at a time: the first that sees `want` entries, else the longest (of equal ones the
// first), if it sees more than best.y.  Out of line: its registers are not kept for the many calls that need none.
__device__ __noinline__ int2 longest_of(const int32_t* n_entries, int64_t table_cap, int q, int end, int want, int2 best) {
  const int lane = threadIdx.x & 31;
  for (; q < end && best.y < want; q += 4 * 32) {
    int n[4], top = -1, at = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = q + 32 * i + lane < end ? visible(n_entries, table_cap, q + 32 * i + lane) : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = min(n[i], want);
      if (v > top) {
        top = v;
        at = q + 32 * i + lane;
      }
    }
    const int most = __reduce_max_sync(0xffffffffu, top);
    if (most > best.y) best = make_int2(__reduce_min_sync(0xffffffffu, top == most ? at : INT32_MAX), most);
  }
  return best;
}
// A group's shared entries: the query whose table row holds them (the first that is long enough, else the
// longest) and their number.  Every lane of a warp calls it, those with `any` for a group [first, end) of one query at
// least.  Where a group's first query is not long enough (a batch that begins with requests that have ended) its lane
// looks at the next four, and the whole warp at the rest (all by the lane: the preparation of 1,000 queries of which
// the first 900 are short took 126 us, now 36, as with none).
__device__ __forceinline__ int2 shared_of(const PrefixArgs& a, bool any, int g, int first, int end) {
  const int want = any ? min(max(a.n_shared[g], 0), a.shared_max) : 0;
  int2 best = make_int2(first, any && first < end ? visible(a, first) : 0);
  if (__any_sync(0xffffffffu, any && best.y < want)) {
    int n[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = any && first + 1 + i < end ? visible(a, first + 1 + i) : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (best.y < want && n[i] > best.y) best = make_int2(first + 1 + i, n[i]);
    for (unsigned open = __ballot_sync(0xffffffffu, any && first + 5 < end && best.y < want); open; open &= open - 1) {
      const int src = __ffs(open) - 1;
      auto of = [&](int x) { return __shfl_sync(0xffffffffu, x, src); };
      const int2 r = longest_of(a.n_entries, a.table_cap, of(first) + 5, of(end), of(want), make_int2(of(best.x), of(best.y)));
      if ((int)(threadIdx.x & 31) == src) best = r;
    }
  }
  return make_int2(best.x, min(best.y, want));
}
// chunks that the image of a group of n queries takes, if there is room
__device__ __forceinline__ int image_chunks(int n, int ns) {
  return n < kImageQueries ? 0 : (ns + kChunk - 1) / kChunk;
}

// trees: whether a request's first and last token are in order, its context, and chunks of that which are widened once
// (whole ones: every query sees all of them)
__device__ __forceinline__ bool tree_ok(const PrefixArgs& a, int lo, int hi) {
  return lo >= 0 && hi >= lo && hi <= a.B && hi - lo <= a.max_tokens;
}
__device__ __forceinline__ int tree_context(const PrefixArgs& a, int g) { return min(max(a.n_entries[g], 0), a.shared_max); }
__device__ __forceinline__ int tree_image_chunks(int tokens, int n) { return tokens < kImageQueries ? 0 : n / kChunk; }
// Trees share the chunks among the pairs of CTAs by what they cost: a request of few tokens has no image, and of short
// contexts the tails and the change from pair to pair are most.  In units of half an image chunk; a change of 2 / 4 / 8, us:
// ragged 48 of up to 32 on up to 4,001 134 / 135 / 141 (by the number of chunks 184), 64 of up to 48 on up to 900 118 / 123 /
// 129; rows of 3 / 4 with a change of 4 135 / 140 and 123 / 127.
constexpr int kCostImage = 2, kCostRows = 3, kCostPair = 2;
__device__ __forceinline__ int image_chunks_of(const Pair& x) { return x.image >= 0 ? min(x.vis0 / kChunk, x.nshared) : 0; }
__device__ __forceinline__ int cost_of(const Pair& x) {
  const int im = image_chunks_of(x);
  return x.nshared > 0 ? kCostPair + kCostImage * im + kCostRows * (x.nshared - im) : 0;
}
constexpr int kSliceChunks = 512;  // chunks of image (64 MB) to each part of the list that all CTAs work on (tree_slices)
// the largest i in [0, n) with list[i] <= x, list[0] <= x
__device__ __forceinline__ int last_at_most(const int32_t* list, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (list[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <bool kAloneQueries, bool kTree>
__device__ __forceinline__ void plan_block(const PrefixArgs& a, int32_t* smem, int smem_ints) {
  __shared__ int s_warp[kPrepThreads / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  if (tid == 0) {
    s_bad = 0;
    *reinterpret_cast<ErrWord*>(a.ws) = ErrWord{0, 0, 0};  // no other CTA of the launch reports
  }
  __syncthreads();
  // the lists that are searched, in shared memory where they fit: a search is a chain of dependent loads
  int2* const gshared = a.G <= smem_ints / 8 ? reinterpret_cast<int2*>(smem + smem_ints / 4) : a.gshared;
  for (int g0 = 0; g0 < a.G; g0 += kPrepThreads) {
    const int g = g0 + tid;
    const int lo = g < a.G ? a.group_start[g] : 0, hi = g < a.G ? a.group_start[g + 1] : 0;
    const bool bad = kTree ? !tree_ok(a, lo, hi) : lo < 0 || hi < lo || hi > a.B, any = !bad && lo < hi;
    if (bad) {
      s_bad = 1;
      report_error(a.ws, CSA2_ERR_INDEX_RANGE, g);
    }
    int2 sh = make_int2(0, 0);
    if constexpr (!kTree) sh = shared_of(a, any, g, lo, hi);
    else if (any) sh = make_int2(tree_context(a, g), hi - lo);
    if (any) gshared[g] = sh;
  }
  __syncthreads();
  const int G = s_bad ? 0 : a.G;
  const int R = G + 2;  // ranges; without groups the first is empty
  int32_t* const gpair = R + 1 <= smem_ints / 4 ? smem : a.gpair;
  const int most_pairs = kAloneQueries ? a.B : max_pairs(a.B, a.G);
  constexpr bool kCosts = kTree && !kAloneQueries;
  const int room = kCosts ? smem_ints / 4 : smem_ints / 2;
  int32_t* const chunk0 = most_pairs + 1 <= room ? smem + smem_ints / 2 : a.chunk0;
  int32_t* const cost0 = !kCosts ? nullptr : most_pairs + 1 <= room ? smem + 3 * (smem_ints / 4) : a.cost0;
  auto range_lo = [&](int v) { return v == 0 ? 0 : G == 0 ? 0 : a.group_start[v - 1]; };
  auto range_hi = [&](int v) { return v == R - 1 ? a.B : G == 0 ? 0 : a.group_start[v]; };
  int base = 0;
  for (int v0 = 0; !kAloneQueries && v0 < R; v0 += kPrepThreads) {
    const int v = v0 + tid;
    const int n = v < R ? (range_hi(v) - range_lo(v) + 1) / 2 : 0;
    int total;
    const int at = base + block_scan(n, s_warp, &total);
    if (v < R) gpair[v] = at;
    base += total;
  }
  if (tid == 0) gpair[R] = base;
  const int np = kAloneQueries ? a.B : base;
  // a group whose image would end beyond the room has none, and so do all behind it
  int images = 0;
  for (int g0 = 0; !kAloneQueries && g0 < G; g0 += kPrepThreads) {
    const int g = g0 + tid, size = g < G ? a.group_start[g + 1] - a.group_start[g] : 0;
    const int n = size <= 0 ? 0 : kTree ? tree_image_chunks(size, gshared[g].x) : image_chunks(size, gshared[g].y);
    int total;
    const int at = images + block_scan(n, s_warp, &total);
    if (g < G) a.gimage[g] = n > 0 && at + (int64_t)n <= a.image_cap ? at : -1;
    images += total;
  }
  __syncthreads();
  int chunks = 0, costs = 0;
  for (int p0 = 0; p0 < np; p0 += kPrepThreads) {
    const int p = p0 + tid;
    Pair x{};
    int n = 0;
    auto tree_rows = [&](int g) {  // request g's, in chunks
      x.first = g;
      x.own0 = a.group_start[g];
      x.vis0 = gshared[g].x;
      x.vis1 = gshared[g].y;
      x.ns = x.vis0 + (a.entries ? x.vis1 : 0);
      constexpr int kPer = kAloneQueries ? kOwnChunk : kChunk;
      n = x.nshared = (x.ns + (a.n_swa > 0 ? a.n_swa + x.vis1 : 0) + kPer - 1) / kPer;
    };
    if (kTree && kAloneQueries) {
      if (p < np) {
        x.q0 = p;
        x.q1 = x.image = -1;
        if (G > 0 && p >= a.group_start[0] && p < a.group_start[G]) tree_rows(last_at_most(a.group_start, G, p));
      }
    } else if (kAloneQueries && p < np) {  // a query by itself, in chunks of kOwnChunk rows
      x.q0 = x.first = p;
      x.q1 = x.image = -1;
      if (G > 0 && p >= a.group_start[0] && p < a.group_start[G]) {
        int lo = 0, hi = G;  // the group with group_start[g] <= p < group_start[g + 1]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (a.group_start[mid] <= p) lo = mid;
          else hi = mid;
        }
        x.first = gshared[lo].x;
        x.ns = gshared[lo].y;
      }
      const int c = visible(a, p), most = x.ns + a.own_max;
      if (a.G > 0 && c > most) report_error(a.ws, CSA2_ERR_INDEX_RANGE, a.n_entries[p]);
      x.own0 = min(c, most);  // the first ns through the row of `first`
      n = (x.own0 + a.n_swa + kOwnChunk - 1) / kOwnChunk;
    } else if (p < np) {
      int lo = 0, hi = R;  // the range with gpair[v] <= p < gpair[v + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (gpair[mid] <= p) lo = mid;
        else hi = mid;
      }
      const int first = range_lo(lo), end = range_hi(lo);
      x.q0 = first + 2 * (p - gpair[lo]);
      x.q1 = x.q0 + 1 < end ? x.q0 + 1 : -1;
      x.first = first;
      x.image = -1;
      if (lo >= 1 && lo <= G) {
        if (kTree) tree_rows(lo - 1);
        else {
          x.first = gshared[lo - 1].x;
          x.ns = gshared[lo - 1].y;
        }
        x.image = a.gimage[lo - 1];
      }
#pragma unroll
      for (int i = 0; i < (kTree ? 0 : 2); ++i) {
        const int q = i ? x.q1 : x.q0;
        if (q < 0) continue;
        const int c = visible(a, q);
        int own = max(c - x.ns, 0);
        if (own > a.own_max) {
          report_error(a.ws, CSA2_ERR_INDEX_RANGE, a.n_entries[q]);
          own = a.own_max;
        }
        (i ? x.vis1 : x.vis0) = min(x.ns, c);
        (i ? x.own1 : x.own0) = own;
      }
      if (!kTree) {
        x.nshared = (max(x.vis0, x.vis1) + kChunk - 1) / kChunk;
        x.paired = x.q1 >= 0 ? (min(x.own0, x.own1) + a.n_swa + kOwnChunk - 1) / kOwnChunk : 0;
        const int alone = max(x.own0, x.own1) + a.n_swa - x.paired * kOwnChunk;
        n = x.nshared + x.paired + (max(alone, 0) + kChunk - 1) / kChunk;
      }
    }
    int total;
    x.chunk0 = chunks + block_scan(n, s_warp, &total);
    if (p < np) {
      a.pairs[p] = x;
      chunk0[p] = x.chunk0;
    }
    chunks += total;
    if (kCosts) {
      const int at = costs + block_scan(p < np ? cost_of(x) : 0, s_warp, &total);
      if (p < np) cost0[p] = at;
      costs += total;
    }
  }
  if (tid == 0) {
    a.pairs[np].chunk0 = chunk0[np] = chunks;
    if (kCosts) cost0[np] = costs;
  }
  __syncthreads();
  if constexpr (kCosts) {
    // Chunk t, which begins at cost s, belongs to part s parts / costs.  Chunks begin kCostPair + kCostRows apart at
    // most, so no part is empty if it is as long.
    // no more parts than the image needs: tree_slices goes by the bounds
    const long long image = min((long long)images, (long long)a.image_cap);
    const long long most = max((image + kSliceChunks - 1) / kSliceChunks, 1LL) * kClusters;
    const long long parts = min(min((long long)a.parts, most), (long long)costs / (kCostPair + kCostRows));
    for (int p = tid; p < np; p += kPrepThreads) {
      const Pair& x = a.pairs[p];
      int k0 = 0, k1 = 0;
      if (x.nshared > 0) {
        const int last = x.nshared > image_chunks_of(x) ? kCostRows : kCostImage;
        k0 = (int)((cost0[p] + kCostPair) * parts / costs);
        k1 = (int)((cost0[p] + cost_of(x) - last) * parts / costs) + 1;
      }
      a.qpart[x.q0] = make_int2(2 * (p + k0), k1 - k0);
      if (x.q1 >= 0) a.qpart[x.q1] = make_int2(2 * (p + k0) + 1, k1 - k0);
    }
    for (int c = tid; c < a.parts; c += kPrepThreads) {
      if (c >= parts) {
        a.parts_of[c] = Part{};
        continue;
      }
      // the first chunk that begins at cost (costs c / parts) or behind, and its pair
      auto first_of = [&](int c, int& p) {
        const int at = (int)((costs * (long long)c + parts - 1) / parts);
        p = c < parts ? last_at_most(cost0, np, at) : np - 1;
        const Pair& x = a.pairs[p];
        const int im = image_chunks_of(x), off = at - cost0[p] - kCostPair;
        const int j = off <= 0 ? 0 : off <= kCostImage * im ? (off + kCostImage - 1) / kCostImage
                                   : im + (off - kCostImage * im + kCostRows - 1) / kCostRows;
        if (c >= parts || j >= x.nshared) {
          ++p;
          return chunk0[p];
        }
        return chunk0[p] + j;
      };
      int p, next;
      const int t0 = first_of(c, p), t1 = first_of(c + 1, next);
      while (chunk0[p + 1] <= t0) ++p;  // pairs without chunks
      a.parts_of[c] = Part{p, t0, t1, chunk0[p + 1], a.pairs[p]};
    }
    return;
  }
  const int clusters = min(a.parts, chunks);
  for (int p = tid; p < np; p += kPrepThreads) {
    // chunk t belongs to part ceil((t + 1) parts / chunks) - 1; a pair's partial of part c is p + c
    const int s0 = chunk0[p], s1 = chunk0[p + 1];
    const int k0 = s1 > s0 ? (int)(((s0 + 1LL) * clusters + chunks - 1) / chunks) - 1 : 0;
    const int k1 = s1 > s0 ? (int)((s1 * (long long)clusters + chunks - 1) / chunks) : 0;
    if (kAloneQueries) {
      a.qpart[p] = make_int2(p + k0, k1 - k0);
    } else {
      const int q0 = a.pairs[p].q0, q1 = a.pairs[p].q1;
      a.qpart[q0] = make_int2(2 * (p + k0), k1 - k0);
      if (q1 >= 0) a.qpart[q1] = make_int2(2 * (p + k0) + 1, k1 - k0);
    }
  }
  for (int c = tid; c < a.parts; c += kPrepThreads) {
    if (c >= clusters) {
      a.parts_of[c] = Part{};
      continue;
    }
    const int t0 = (int)((long long)chunks * c / clusters), t1 = (int)((long long)chunks * (c + 1) / clusters);
    int lo = 0, hi = np;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (chunk0[mid] <= t0) lo = mid;
      else hi = mid;
    }
    a.parts_of[c] = Part{lo, t0, t1, chunk0[lo + 1], a.pairs[lo]};
  }
}

// ------------------------------------------------------------------ attention

// warps 0-3: softmax, rescaling of O, epilogue; 4-11: rows of S's operand; 12-19: rows of O's; then one
// warp each: S MMAs, O MMAs (even CTA; in the odd one they pass arrivals on), where rows come from; the last one passes
// P's arrivals on (odd CTA)
constexpr int kRowWarp = 4, kSMma = 20, kOMma = 21, kIndexWarp = 22;
constexpr int kThreads = 24 * 32;
// registers of a thread: 80 at launch, which the last warpgroup keeps; the softmax takes what the row
// warpgroups give back
constexpr int kSoftRegs = 104, kRowRegs = 72;
static_assert(kSoftRegs + 4 * kRowRegs + 80 <= 6 * 80, "registers of the launch");
constexpr int kPieces = 4;
constexpr uint32_t kCols = 512;   // tensor memory: O 2 x 128 columns, S 2 x 64
constexpr uint32_t kColS = 256;
constexpr long long kWaitBudget = 1LL << 32;

struct __align__(1024) PrefixSmem {
  uint16_t q[kDMain / 8][kQPlane];          // q' [c/8][head][c%8]
  uint16_t xs[kDMain / 8][kOwnChunk * 8];   // this CTA's 64 rows for S [c/8][row][c%8]
  uint16_t xo[4][kDMain / 16][32 * 8];      // this CTA's 256 channels of all 128 rows [row/32][c/8][row%32][c%8]
  uint16_t p[2][kChunk / 8][kHAtt * 8];     // probabilities [row/8][head][row%8]
  float red[2][kHAtt];                      // of the two threads of a head; at the end their sums of p
  int32_t rows[4][kChunk];                  // where a chunk's rows come from, up to four chunks ahead
  int32_t image[4];                         // its chunk of the image, or -1
  // what the MMA warps wait on counts the even CTA's own warps and one arrival that a warp of the odd CTA
  // passes on for all of that CTA's
  uint64_t q_land, q_peer, q_free;          // q' copied; the odd CTA's q'; S of an item's chunks complete
  uint64_t i_full[4], r_full[4], r_free[4]; // image, rows written (one warp); read (16 row and 4 softmax warps)
  uint64_t x_full[2][kPieces], x_free[2][kPieces];  // [0] S's operand, [1] O's
  uint64_t x_go[2][kPieces];                // the piece is free, where rows are written (see rows_role)
  uint64_t s_full[2], p_full[2], p_free[2];
  uint64_t o_read;                          // epilogue done with O
  uint64_t drained;                         // every MMA issued complete (two warps)
  uint64_t last_o;                          // the last item's O complete, its sums in red (four softmax warps)
  int32_t last_slot;                        // its partial, or -1
  Part part;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(PrefixSmem) <= 232448, "prefix attention shared memory");

struct PrefixKernel {
  const uint8_t *kv_codes, *kv_scales, *swa;
  const uint16_t* q;      // [B + 1][c/8][head][c%8] f16 images of the staged queries, the last one zeros
  const float* c2;        // [B + 1][64] logit (log2 units) per raw S
  const int32_t* table;
  int64_t max_pages;
  int32_t n_pages, page_entries, n_swa, B;
  uint64_t page_div;  // ceil(2^40 / page_entries): e * page_div >> 40 = e / page_entries for e < 2^18
  const int64_t *win_pos, *win_lo;
  const Pair* pairs;
  const Part* parts;
  // trees: kin and depth (PrefixArgs) and position of each query; swa and win_pos, n_ring rows, are the requests' rings,
  // draft the tokens' window rows, which count behind those as window rows n_ring + query
  const uint64_t* kin;
  const int32_t* depth;
  const int64_t* q_pos;
  const uint8_t* draft;
  int32_t n_ring, slices;  // slices: parts of each pair of CTAs
  uint4* part_o;    // [pairs + clusters][2][32 Vec8::kWords][128]: eight channels of thread t of the epilogue, of O / l
  float2* part_ml;  // [pairs + clusters][2][64]
  void* ws;
};

// The image of the shared entries: f16 [chunk][c/8][128 rows][c%8].  A piece of S's operand is 16 planes x
// 64 rows of it (1 KB runs), a piece of O's 32 planes x 32 rows (512-byte runs); both 16 KB.
struct ImageMaps {
  CUtensorMap s, o;
};

// A row of a chunk: the plane row of an entry (>= 0), kNoRow, or a window row (kNoRow - 1 - its index).
constexpr int kNoRow = -1;

// Row i of chunk jc of pair x, in two steps so that the page's load is not waited for at once: the page
// (valid when off >= 0) and the entry's place in it, or kNoRow / a window row as `off`.
struct RowRef {
  int page, off;
};
__device__ __forceinline__ RowRef find_entry(const PrefixKernel& k, int q, int e) {
  const int pi = (int)((uint64_t)e * k.page_div >> 40);
  return RowRef{__ldg(k.table + q * k.max_pages + pi), e - pi * k.page_entries};
}
// row idx of query q's own: entries e0 .. e0 + own - 1, then its window
__device__ __forceinline__ RowRef find_own(const PrefixKernel& k, int q, int own, int idx, int e0 = 0) {
  if (idx < own) return find_entry(k, q, e0 + idx);
  idx -= own;
  if (idx >= k.n_swa) return RowRef{0, kNoRow};
  const int w = q * k.n_swa + idx;
  if (k.win_pos && __ldg(k.win_pos + w) < max(__ldg(k.win_lo + q), (int64_t)0)) return RowRef{0, kNoRow};
  return RowRef{0, kNoRow - 1 - w};
}
__device__ __forceinline__ RowRef find_row(const PrefixKernel& k, const Pair& x, int jc, int i) {
  if (jc < x.nshared) {
    const int e = jc * kChunk + i;
    return e < x.ns ? find_entry(k, x.first, e) : RowRef{0, kNoRow};
  }
  const int jo = jc - x.nshared;
  int idx, h;
  if (jo < x.paired) {
    h = i / kOwnChunk;
    idx = jo * kOwnChunk + i % kOwnChunk;
  } else {
    h = x.own1 > x.own0;
    idx = x.paired * kOwnChunk + (jo - x.paired) * kChunk + i;
  }
  return find_own(k, h ? x.q1 : x.q0, h ? x.own1 : x.own0, idx, x.ns);
}
// row idx of a request's (trees): entries, ring, drafts' window rows
__device__ __forceinline__ RowRef find_tree(const PrefixKernel& k, const Pair& x, int idx) {
  if (idx < x.ns) return find_entry(k, x.first, idx);
  idx -= x.ns;
  if (idx < k.n_swa) return RowRef{0, kNoRow - 1 - (x.first * k.n_swa + idx)};
  idx -= k.n_swa;
  if (k.n_swa == 0 || idx >= x.vis1) return RowRef{0, kNoRow};
  return RowRef{0, kNoRow - 1 - (k.n_ring + x.own0 + idx)};
}
// What a query sees of its request's rows behind the context (trees).
struct Sight {
  uint64_t kin;
  int32_t depth;
  int64_t pos;
};
// of query q, by all lanes of a warp; a parent that is none is reported
__device__ __forceinline__ Sight sight_of(const PrefixKernel& k, int q, int lane) {
  if (q < 0) return Sight{0, 0, 0};
  Sight v{__ldg(k.kin + q), __ldg(k.depth + q), k.q_pos ? __ldg(k.q_pos + q) : 0};
  if (v.depth < 0) {
    if (lane == 0) report_error(k.ws, CSA2_ERR_INDEX_RANGE, q);
    v.depth -= kBadParent;
  }
  return v;
}
// whether it sees row idx, one behind the context
__device__ __forceinline__ bool sees(const PrefixKernel& k, const Pair& x, const Sight& v, int idx) {
  if (idx < x.ns) return (v.kin >> (idx - x.vis0)) & 1u;
  idx -= x.ns;
  if (idx < k.n_swa) {
    const int64_t p = __ldg(k.win_pos + x.first * k.n_swa + idx);
    return p >= max(v.pos - k.n_swa + 1, (int64_t)0) && p < v.pos - v.depth;
  }
  idx -= k.n_swa;
  if (idx >= x.vis1 || !((v.kin >> idx) & 1u)) return false;
  // a window of CSA2_MAX_TREE tokens holds any path
  return k.n_swa >= CSA2_MAX_TREE || v.depth - (__ldg(k.depth + x.own0 + idx) & ~kBadParent) < k.n_swa;
}
// A row's bit 30 tells a CTA of a pair whether its query sees it (trees): as it is, the bit is bit 31's copy (entries
// are fewer than 2^30, window rows than 2^24).
__device__ __forceinline__ int flip_seen(int r) { return r ^ 1 << 30; }
__device__ __forceinline__ bool seen(int r) { return (r ^ (int)((uint32_t)r << 1)) >= 0; }
// whether a row of a chunk counts in the softmax
template <bool kTree>
__device__ __forceinline__ bool counts(int r) {
  return r != kNoRow && (!kTree || seen(r));
}
// window row r (< kNoRow)
template <bool kTree>
__device__ __forceinline__ const uint8_t* window_row(const PrefixKernel& k, int r) {
  const int w = kNoRow - 1 - r;
  if (kTree && w >= k.n_ring) return k.draft + (int64_t)(w - k.n_ring) * kDMain;
  return k.swa + (int64_t)w * kDMain;
}
// a page outside the planes is skipped, and reported by the warp that is told to
__device__ __forceinline__ int resolve(const PrefixKernel& k, RowRef r, bool report) {
  if (r.off < 0) return r.off;
  if (r.page < 0 || r.page >= k.n_pages) {
    if (report) report_error(k.ws, CSA2_ERR_INDEX_RANGE, r.page);
    return kNoRow;
  }
  return r.page * k.page_entries + r.off;
}

// A NaN (a scale or a window value 0x7F, 0xFF) becomes lim, which every finite E4M3 value is at most; a NaN
// lim leaves all as it is.
constexpr uint32_t kAnyValue = 0x7FFF7FFFu, kFinite = 0x5F005F00u;  // 448, E4M3's largest
__device__ __forceinline__ uint32_t min2_u32(uint32_t x, uint32_t lim) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(lim));
  return r;
}
// 32 channels of an entry (16 bytes of codes, two scales) -> four 8-channel vectors of f16
__device__ __forceinline__ void widen_codes(uint4 cw, uint32_t sc, uint32_t lim, uint4 (&v)[4]) {
  const uint32_t s0 = min2_u32(e4m3x2_to_f16x2((sc & 0xFFu) * 0x0101u), lim);
  const uint32_t s1 = min2_u32(e4m3x2_to_f16x2((sc >> 8) * 0x0101u), lim);
  const uint32_t wq[4] = {cw.x, cw.y, cw.z, cw.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t h[4];
    e2m1x8_to_f16(wq[q], h);
    const uint32_t s = q < 2 ? s0 : s1;
    v[q] = make_uint4(hmul2_u32(h[0], s), hmul2_u32(h[1], s), hmul2_u32(h[2], s), hmul2_u32(h[3], s));
  }
}
// 16 channels of a window row
__device__ __forceinline__ void widen_e4m3(uint4 w, uint32_t lim, uint4& a, uint4& b) {
  auto two = [&](uint32_t x) { return min2_u32(e4m3x2_to_f16x2(x), lim); };
  a = make_uint4(two(w.x), two(w.x >> 16), two(w.y), two(w.y >> 16));
  b = make_uint4(two(w.z), two(w.z >> 16), two(w.w), two(w.w >> 16));
}

// The block that lane l (row l % 8 of its eight) begins with, mod 8.  A 128-bit load is served eight lanes at a
// time: with one block for all they would read eight rows at the same bank, 32 accesses for a warp's load
// instead of 4, from the memory that also feeds the MMAs (paged ragged 48 x 65536: 253 us, with the blocks rotated 234).
__device__ __forceinline__ int rotated(int lane) { return (lane & 7) + (lane >> 3); }

// One thread's fetched codes of 32 channels of a row.
struct Fetch {
  uint4 codes, more;  // 16 bytes of codes, or 32 of a window row
  uint32_t scales;
};
// Starts the loads of 32-channel block cb of row r.
template <bool kTree>
__device__ __forceinline__ void fetch(Fetch& f, const PrefixKernel& k, int r, int cb) {
  if (r >= 0) {
    f.codes = __ldg(reinterpret_cast<const uint4*>(k.kv_codes + (int64_t)r * 256) + cb);
    f.scales = __ldg(reinterpret_cast<const uint16_t*>(k.kv_scales + (int64_t)r * 32) + cb);
  } else if (r < kNoRow) {
    const uint4* src = reinterpret_cast<const uint4*>(window_row<kTree>(k, r)) + 2 * cb;
    f.codes = __ldg(src);
    f.more = __ldg(src + 1);
  }
}
// Writes the fetched block of row r to dst: vector q of it at dst + q * stride (f16 elements).
__device__ __forceinline__ void put(const Fetch& f, int r, uint16_t* dst, int stride, uint32_t lim = kAnyValue) {
  uint4 v[4];
  if (r >= 0) {
    widen_codes(f.codes, f.scales, lim, v);
  } else if (r < kNoRow) {
    widen_e4m3(f.codes, lim, v[0], v[1]);
    widen_e4m3(f.more, lim, v[2], v[3]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(dst + q * stride) = v[q];
}

// packed fp32 arithmetic on two neighbouring registers
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Probabilities go to the tensor cores as f16 of p = 2^(z - m), a rounding of 2^-11 at most down to p = 2^-14, and
// an absolute one of 2^-25 below.  A long context behind one strong row lies there: 65,536 rows, each 2^-25.5 of
// the strongest, are a thousandth of the output together, and none of them would be left with m at the largest
// logit.  So a new reference m is kTopExp below the largest logit, and moves when one exceeds it by more than
// kMaxExp (f16 ends below 2^16): what a row loses is 2^-36 of the largest at most.  The 4 bits (2.8 nats) between
// the two are what the running maximum may rise before O has to be scaled.
constexpr float kTopExp = 11.0f, kMaxExp = 15.0f;

// p of 32 rows (exponents s c2 - m), packed in pairs as f16 from the fp32 values whose sum goes to `sum`;
// returns the largest exponent.  Rows that the mask has not are -inf.
__device__ __forceinline__ float probs32(uint64_t (&s)[16], uint32_t mask, float c2, float m, uint32_t (&ph)[16],
                                         float& sum) {
  const uint64_t cc = pack2(__float_as_uint(c2), __float_as_uint(c2));
  const uint64_t mm = pack2(__float_as_uint(-m), __float_as_uint(-m));
#pragma unroll
  for (int u = 0; u < 16; ++u) s[u] = fma2(s[u], cc, mm);
  if (mask != ~0u) {
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      float e0, e1;
      unpack2(s[u], e0, e1);
      if (!((mask >> (2 * u)) & 1u)) e0 = -INFINITY;
      if (!((mask >> (2 * u + 1)) & 1u)) e1 = -INFINITY;
      s[u] = pack2(__float_as_uint(e0), __float_as_uint(e1));
    }
  }
  float top = -INFINITY;
  uint64_t acc = 0;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    float e0, e1;
    unpack2(s[u], e0, e1);
    top = fmaxf(top, fmaxf(e0, e1));
    const float p0 = ptx::ex2(e0), p1 = ptx::ex2(e1);
    acc = add2(acc, pack2(__float_as_uint(p0), __float_as_uint(p1)));
    const __half2 h2 = __floats2half2_rn(p0, p1);
    ph[u] = *reinterpret_cast<const uint32_t*>(&h2);
  }
  float s0, s1;
  unpack2(acc, s0, s1);
  sum = s0 + s1;
  return top;
}

// Copies piece i of operand op from a chunk of the image to this CTA; its bytes count on the even CTA's barrier, whose
// MMA warps read both CTAs'.
constexpr int kPieceBytes = 16 * 1024;
__device__ __forceinline__ void copy_piece(PrefixSmem& S, const ImageMaps& maps, int op, int rank, int i, int image) {
  const int plane0 = image * (kDMain / 8);
  uint64_t* const bar = &S.x_full[op][i];
  if (op) ptx::tma_load_2d_pair(&S.xo[i][0][0], &maps.o, 128 * i, plane0 + 32 * rank, bar, 0);
  else ptx::tma_load_2d_pair(&S.xs[16 * i][0], &maps.s, 256 * rank, plane0 + 16 * i, bar, 0);
}

// The operands of all `chunks` chunks of this pair of CTAs, whatever items they belong to, by the 16 row
// warps: per operand two groups of four, which write every other piece.  Operand 0 (S's, warps 0-7): this
// CTA's 64 rows, handed over by 128 channels: in piece i a thread has one of the blocks (of 32 channels) 4 i .. of
// rows 8 (w % 4) + l % 8 and 32 more.  Operand 1 (O's): its 256 channels of all rows, by 32 rows: a thread
// has two of its eight blocks, four apart, of row 32 i + 8 (w % 4) + l % 8.  Either way a load reads 64
// contiguous bytes of eight rows, and a store writes eight rows of a plane: no bank conflicts.  A step writes
// one piece and fetches the codes of the next (half a chunk ahead); a chunk of the image is copied instead,
// by the first warp of each group, and its bytes count on the even CTA's barrier (x_full).  Only that warp waits for
// x_free; the others go by its x_go, of which rows alone have phases: a warp that takes no part in a copy could miss
// one of x_free.  The odd CTA's x_full too has phases of rows alone, which are passed on.  Both operands run the same code: the
// kernel's loops have to fit the instruction cache (unrolled by piece and operand they waited more for instructions
// than for data).
template <bool kTree>
__device__ __forceinline__ bool rows_role(PrefixSmem& S, const PrefixKernel& k, const ImageMaps& maps, int rank,
                                          int chunks, int w, int lane) {
  const int op = w >> 3, group = (w >> 2) & 1;
  const bool lead = (w & 3) == 0;
  const int rl = 8 * (w & 3) + (lane & 7);
  const int row0 = op ? rl : kOwnChunk * rank + rl, row_step = op ? 32 : 0, row_u = op ? 0 : 32;
  const int b = rotated(lane) & (op ? 7 : 3);
  const int blk0 = op ? 8 * rank + b : b, blk_step = op ? 0 : 4, blk_u = op ? (b ^ 4) - b : 0;
  const int plane = (op ? 32 : kOwnChunk) * 8;  // f16 elements
  uint16_t* const dst = (op ? &S.xo[0][4 * b][0] : &S.xs[4 * b][0]) + rl * 8;
  constexpr int dst_step = 16 * 1024 / 2;  // a piece
  const int dst_u = op ? blk_u * 4 * 32 * 8 : 32 * 8;
  const int steps = chunks * 2;  // step st: chunk st / 2, piece 2 (st % 2) + group
  int r[2], image = -1;
  Fetch f[2];
  int issued = -1;  // last step copied from the image
  uint32_t owns = 0;  // chunks not copied before this one
  bool good = true;
  auto load = [&](int st) {  // this thread's rows and codes of step st
    if (st >= steps) return;
    const uint32_t m = (uint32_t)(st >> 1), slot = m & 3u;
    const int i = 2 * (st & 1) + group;
    if ((st & 1) == 0) {
      good = good && ptx::mbar_wait_warp(&S.i_full[slot], (m >> 2) & 1u, &S.abort_flag, kWaitBudget);
      if (good) image = S.image[slot];
      // rows found; a chunk of the image needs none
      if (image < 0) good = good && ptx::mbar_wait_warp(&S.r_full[slot], (m >> 2) & 1u, &S.abort_flag, kWaitBudget);
    }
    if (!good) return;
    if (image < 0) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        r[u] = S.rows[slot][row0 + row_step * i + row_u * u];
        if (kTree && !seen(r[u])) r[u] = flip_seen(r[u]);
        fetch<kTree>(f[u], k, r[u], blk0 + blk_step * i + blk_u * u);
      }
    }
    if (st & 1) {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.r_free[slot]);
    }
  };
  load(0);
#pragma unroll 1
  for (int st = 0; st < steps && good; ++st) {
    const uint32_t m = (uint32_t)(st >> 1);
    const int i = 2 * (st & 1) + group;
    if (lead && m > 0) good = ptx::mbar_wait_warp(&S.x_free[op][i], (m - 1) & 1u, &S.abort_flag, kWaitBudget);
    if (image >= 0) {
      if (!good) break;
      if (lead) {
        if (rank == 0 && lane < 4) ptx::mbar_arrive(&S.x_full[op][i]);  // for the others, and the odd CTA
        if (rank == 0 && lane == 0) ptx::mbar_arrive_expect_tx(&S.x_full[op][i], 2 * kPieceBytes);
        if (lane == 0) copy_piece(S, maps, op, rank, i, image);
        issued = st;
        __syncwarp();
      }
    } else {
      if (!lead) good = ptx::mbar_wait_warp(&S.x_go[op][i], owns & 1u, &S.abort_flag, kWaitBudget);
      if (!good) break;
      if (lead && lane == 0) ptx::mbar_arrive(&S.x_go[op][i]);
#pragma unroll
      for (int u = 0; u < 2; ++u) put(f[u], r[u], dst + i * dst_step + u * dst_u, plane, op ? kFinite : kAnyValue);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.x_full[op][i]);
      if (st & 1) ++owns;
    }
    load(st + 1);
  }
  // copies in flight write shared memory: they land before anyone leaves (the odd CTA sees it by the MMAs behind
  // them, or the limit)
  if (!good && lead) {
    volatile int keep_waiting = 0;
    for (int st = issued; st >= 0 && st > issued - 2; --st) {
      uint64_t* const landed = (rank ? S.x_free : S.x_full)[op] + 2 * (st & 1) + group;
      ptx::mbar_wait_warp(landed, (uint32_t)(st >> 1) & 1u, &keep_waiting, kWaitBudget);
    }
  }
  return good;
}

// A row's bytes into L2: the row warps fetch half a chunk ahead, which memory's latency exceeds (without this,
// prefix ragged 101 on 4001 took 70.7 us instead of 66.2, 32 on 8192 51.0 instead of 49.4).
template <bool kTree>
__device__ __forceinline__ void prefetch_row(const PrefixKernel& k, int r) {
  if (r == kNoRow) return;
  const uint8_t* at = r >= 0 ? k.kv_codes + (int64_t)r * 256 : window_row<kTree>(k, r);
  ptx::prefetch_l2(at);
  ptx::prefetch_l2(at + 128);
  if (r >= 0) {
    ptx::prefetch_l2(k.kv_scales + (int64_t)r * 32);
  } else {
    ptx::prefetch_l2(at + 256);
    ptx::prefetch_l2(at + 384);
  }
}

// Whether chunk c of a pair is copied from the image, which serves both operands: only where both queries see all of
// the chunk's entries.
template <bool kTree>
__device__ __forceinline__ bool from_image(const Pair& x, int c) {
  if (kTree) return x.image >= 0 && (c + 1) * kChunk <= x.vis0;
  const int seen = x.q1 >= 0 ? min(x.vis0, x.vis1) : x.vis0;
  return x.image >= 0 && c < x.nshared && min((c + 1) * kChunk, x.ns) <= seen;
}

// Where each chunk's rows come from (or its chunk of the image), by one warp (lane l rows l, 32 + l, ..) up to
// four chunks ahead of the row and softmax warps.  Pages outside the planes are reported here.
template <bool kTree>
__device__ __forceinline__ bool index_role(PrefixSmem& S, const PrefixKernel& k, const Pair& x, int rank, int c0,
                                           int nc, int lane, uint32_t n) {
  const bool report = rank == 0;
  bool good = true;
  RowRef r[4];
  const int qme = rank ? x.q1 : x.q0;
  const Sight sight = kTree ? sight_of(k, qme, lane) : Sight{};
  auto find = [&](int j) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = kTree ? find_tree(k, x, (c0 + j) * kChunk + 32 * i + lane) : find_row(k, x, c0 + j, 32 * i + lane);
  };
  find(0);
#pragma unroll 1
  for (int j = 0; j < nc && good; ++j) {
    const uint32_t m = n + (uint32_t)j, slot = m & 3u;
    if (m >= 4) good = ptx::mbar_wait_warp(&S.r_free[slot], ((m >> 2) - 1) & 1u, &S.abort_flag, kWaitBudget);
    if (!good) break;
    if (lane == 0) {
      S.image[slot] = from_image<kTree>(x, c0 + j) ? x.image + c0 + j : -1;
      ptx::mbar_arrive(&S.i_full[slot]);
    }
    int row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = resolve(k, r[i], report);
    if (kTree ? !from_image<kTree>(x, c0 + j) : x.image < 0 || c0 + j >= x.nshared) {  // each CTA half of the rows
      prefetch_row<kTree>(k, rank ? row[1] : row[0]);
      prefetch_row<kTree>(k, rank ? row[3] : row[2]);
    }
    if (kTree) {  // both CTAs have the same rows, each its own query's view of them
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int idx = (c0 + j) * kChunk + 32 * i + lane;
        if (row[i] != kNoRow && !(qme >= 0 && (idx < x.vis0 || sees(k, x, sight, idx)))) row[i] = flip_seen(row[i]);
      }
    }
    if (j + 1 < nc) find(j + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) S.rows[slot][32 * i + lane] = row[i];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.r_full[slot]);
  }
  return good;
}

// Eight values of a part's O / l, as the join reads them: fp32 for an fp32 output.  For a bf16 output f16, times 16:
// |O / l| is at most the largest |x|, 2,688, so 2^-11 of a value or 2^-29 are the most that is rounded off, an
// eighth of the output's own rounding; the smallest entry that is not zero is 2^-10.  The parts are most of what a
// short call moves, in fp32 / f16, us: paged ragged 128 x 2000 52.3 / 44.5, prefix ragged 101 on 4001 67.1 / 61.1,
// paged ragged 48 x 65536 223.7 / 217.6.
template <bool kHalf>
struct Vec8 {
  static constexpr int kWords = kHalf ? 1 : 2;  // 16-byte words
  static constexpr float kScale = kHalf ? 16.0f : 1.0f;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const uint4* p) {  // words 128 apart: a warp's stores are 512 contiguous bytes
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = p[i * 128];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (kHalf) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    } else {
      const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    }
  }
  // value(i) comes scaled by kScale
  template <typename F>
  static __device__ __forceinline__ void store(uint4* p, F value) {
    if constexpr (kHalf) {
      auto two = [&](int i) {
        const __half2 v = __floats2half2_rn(value(i), value(i + 1));
        return *reinterpret_cast<const uint32_t*>(&v);
      };
      p[0] = make_uint4(two(0), two(2), two(4), two(6));
    } else {
      auto one = [&](int i) { return __float_as_uint(value(i)); };
      p[0] = make_uint4(one(0), one(1), one(2), one(3));
      p[128] = make_uint4(one(4), one(5), one(6), one(7));
    }
  }
};

// Columns 32 c0 .. 32 c1 of O / l of thread t's accumulator row.
template <bool kHalf>
__device__ __forceinline__ void store_pair_o(const PrefixKernel& k, uint32_t tmem, int64_t slot, int t, float l, int c0,
                                             int c1) {
  using Vec = Vec8<kHalf>;
  const float inv = l > 0.0f ? Vec::kScale / l : 0.0f;
  uint4* po = k.part_o + slot * (32 * Vec::kWords) * 128 + t;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    uint32_t a[32];
    ptx::tmem_ld_32x32b_x32(tmem + ((uint32_t)(t & ~31) << 16) + 32u * (uint32_t)c, a);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int u = 0; u < 4; ++u)
      Vec::store(po + (c * 4 + u) * Vec::kWords * 128, [&](int i) { return __uint_as_float(a[8 * u + i]) * inv; });
  }
}

template <bool kHalf, bool kTree>
__global__ void __launch_bounds__(kThreads, 1) k_prefix_attn(const __grid_constant__ PrefixKernel k,
                                                                  const __grid_constant__ ImageMaps maps) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  PrefixSmem& S = *reinterpret_cast<PrefixSmem*>(smem_raw);
  volatile int* abort_flag = &S.abort_flag;
  const int rank = (int)ptx::cluster_ctarank();
  const int cluster = blockIdx.x / 2;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  if (warp == kSMma) {
    if (lane == 0) {
      const uint32_t peer = rank == 0 ? 1 : 0;
      ptx::mbar_init(&S.q_peer, 1);
      for (int i = 0; i < 2 * kPieces; ++i) {
        ptx::mbar_init(&S.x_full[0][0] + i, 4 + peer);
        ptx::mbar_init(&S.x_go[0][0] + i, 1);
        ptx::mbar_init(&S.x_free[0][0] + i, 1);
      }
      ptx::mbar_init(&S.q_land, 1);
      ptx::mbar_init(&S.q_free, 1);
      for (int i = 0; i < 4; ++i) {
        ptx::mbar_init(&S.i_full[i], 1);
        ptx::mbar_init(&S.r_full[i], 1);
        ptx::mbar_init(&S.r_free[i], 20);
      }
      for (int i = 0; i < 2; ++i) {
        ptx::mbar_init(&S.s_full[i], 1);
        ptx::mbar_init(&S.p_full[i], 4 + peer);
        ptx::mbar_init(&S.p_free[i], 1);
      }
      ptx::mbar_init(&S.o_read, 4 + peer);
      ptx::mbar_init(&S.last_o, 4);
      ptx::mbar_init(&S.drained, 2);
      S.abort_flag = 0;
      ptx::fence_mbar_init();
    }
    __syncwarp();
    ptx::tmem_alloc_pair(&S.tmem_base, kCols);
  }
  if (warp == kIndexWarp && lane < 2) ptx::prefetch_tensormap(lane ? &maps.o : &maps.s);
  ptx::griddep_launch();
  ptx::tc_fence_before();
  ptx::cluster_sync();  // both CTAs' barriers initialised
  ptx::griddep_wait();
  if (tid < (int)(sizeof(Part) / 4))
    reinterpret_cast<int32_t*>(&S.part)[tid] = reinterpret_cast<const int32_t*>(k.parts + cluster)[tid];
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = S.tmem_base;

  auto wait = [&](uint64_t* bar, uint32_t n) { return ptx::mbar_wait_warp(bar, n & 1u, abort_flag, kWaitBudget); };
  bool good = true;
  int where = 0;
  // this pair of CTAs' parts: one, or (trees) every kClusters-th, so that all work on neighbouring pairs at a time
  const int slices = kTree ? k.slices : 1;
  auto part_of = [&](int i) { return i == 0 ? &S.part : k.parts + cluster + i * kClusters; };
  int chunks = 0;
  for (int i = 0; i < slices; ++i) chunks += part_of(i)->t1 - part_of(i)->t0;
  // Every role runs the same list of items, in a loop of its own: pair x, its chunks c0 .. c0 + nc - 1, and the
  // number of its partial; n counts the chunks before them, items the items.
  auto for_items = [&](auto body) {
    uint32_t n = 0, items = 0;
    for (int i = 0; i < slices && good; ++i) {
      const Part& part = *part_of(i);
      const Pair* px = &part.pair;
      int p = part.p, end = part.end;
      const int t1 = part.t1;
      for (int t = part.t0; t < t1 && good;) {
        const Pair x = *px;
        const int c0 = t - x.chunk0, nc = min(end, t1) - t;
        if (nc > 0) {  // else a pair without chunks
          t += nc;
          body(x, p + cluster + i * kClusters, c0, nc, n, items);
          n += (uint32_t)nc;
          ++items;
        }
        px = k.pairs + ++p;
        if (t < t1) end = k.pairs[p + 1].chunk0;
      }
    }
  };

  if (warp >= kRowWarp && warp < kSMma) {
    ptx::setmaxnreg_dec<kRowRegs>();
    good = rows_role<kTree>(S, k, maps, rank, chunks, warp - kRowWarp, lane);
    // the last item's partial is theirs, a quarter of the columns each four: nothing else is left to do
    if (good && chunks > 0) good = wait(&S.last_o, 0);
    if (good && chunks > 0 && S.last_slot >= 0) {
      ptx::tc_fence_after();
      const int quarter = (warp - kRowWarp) / 4, t = 32 * (warp % 4) + lane;
      store_pair_o<kHalf>(k, tmem, S.last_slot, t, S.red[0][t & 63] + S.red[1][t & 63], 2 * quarter, 2 * quarter + 2);
      ptx::tc_fence_before();
    }
    where = 31;
  } else if (warp >= kSMma) {
    // The odd CTA's MMA warps pass their CTA's arrivals on (and the last warp P's), released here and taken by the even
    // CTA's at cluster scope: the MMAs that read this CTA's rows, P and tensor memory are issued there.
    // Every release waits (ptx.cuh), hence two pieces of rows to one, and copies that count on the even CTA's
    // barriers by themselves: 64 on 65000 takes 405 us, with a release for every piece and copy 733 (at CTA scope,
    // which orders nothing between two CTAs, 370).
    auto wait_pair = [&](uint64_t* bar, uint32_t n) {
      return ptx::mbar_wait_warp<true>(bar, n & 1u, abort_flag, kWaitBudget);
    };
    auto pass = [&](uint64_t* bar, uint32_t ph, int n) {  // n neighbouring barriers
      for (int i = 0; i < n; ++i) good = good && wait(bar + i, ph);
      ptx::tc_fence_after();  // the softmax's tensor-memory stores are among what is passed on
      ptx::tc_fence_before();
      if (good && lane < n) ptx::mbar_arrive_peer(bar + lane, 0);
      __syncwarp();
    };
    // the pair's chunk c, unless it was copied: by the chunks of rows before it
    uint32_t owns = 0;
    auto pass_rows = [&](int op, const Pair& x, int c) {
      if (from_image<kTree>(x, c)) return;
      for (int i = 0; i < kPieces; i += 2) pass(&S.x_full[op][i], owns, 2);
      ++owns;
    };
    if (warp == kIndexWarp) {
      for_items([&](const Pair& x, int, int c0, int nc, uint32_t n, uint32_t) {
        good = index_role<kTree>(S, k, x, rank, c0, nc, lane, n);
      });
      where = 32;
    } else if (warp == kSMma) {
      // ---- S = q' X^T: 32 K steps of 16 channels, four pieces of eight
      constexpr uint32_t idesc_s = ptx::idesc_f16(128, kChunk, 0);
      const uint64_t da = ptx::smem_desc_noswizzle(&S.q[0][0], kQPlane * 2, 128);
      const uint64_t db = ptx::smem_desc_noswizzle(&S.xs[0][0], kOwnChunk * 16, 128);
      for_items([&](const Pair& x, int, int c0, int nc, uint32_t n, uint32_t items) {
        // the item's query, once S of the item before has left q'; the copy lands before anyone leaves
        good = items == 0 || wait(&S.q_free, items - 1);
        if (!good) return;
        if (lane == 0) {
          const int64_t q = rank == 0 ? x.q0 : x.q1 >= 0 ? x.q1 : k.B;
          ptx::mbar_arrive_expect_tx(&S.q_land, kHAtt * kDMain * 2);
          ptx::bulk_g2s(&S.q[0][0], k.q + q * kHAtt * kDMain, kHAtt * kDMain * 2, &S.q_land);
        }
        __syncwarp();
        volatile int keep_waiting = 0;
        good = ptx::mbar_wait_warp(&S.q_land, items & 1u, &keep_waiting, kWaitBudget);
        if (rank == 0) good = good && wait_pair(&S.q_peer, items);
        else if (good && lane == 0) ptx::mbar_arrive_peer(&S.q_peer, 0);
#pragma unroll 1
        for (int j = 0; j < nc && good; ++j) {
          const uint32_t m = n + (uint32_t)j;
          if (rank) {
            pass_rows(0, x, c0 + j);
            continue;
          }
          // the softmax of both CTAs has left this S buffer
          if (m >= 2) good = wait_pair(&S.p_full[m & 1], (m >> 1) - 1);
          const uint32_t dst = tmem + kColS + 64u * (m & 1u);
#pragma unroll 1
          for (int i = 0; i < kPieces && good; ++i) {
            good = wait_pair(&S.x_full[0][i], m);
            if (!good) break;
            ptx::tc_fence_after();
            const uint64_t at = (uint64_t)(i * 1024);  // q'[16 i], xs[16 i]: 16 KB on; a K step 2 KB
            ptx::mma_f16_ss_pair_run_elect<8, 128, 128>(dst, da + at, db + at, idesc_s, i > 0 ? 1u : 0u);
            ptx::mma_commit_pair_elect(&S.x_free[0][i]);
          }
          if (good) ptx::mma_commit_pair_elect(&S.s_full[m & 1]);
        }
        // a barrier of its own: the odd CTA's warp does not follow the chunks, whose phases it would miss
        if (rank == 0 && good) ptx::mma_commit_pair_elect(&S.q_free);
      });
      where = 33;
    } else if (warp == kOMma) {
      // ---- O += P X: eight K steps of 16 rows, four pieces of two; two accumulators of 128 channels a CTA
      constexpr uint32_t idesc_o = ptx::idesc_f16(128, 256, 0) | ptx::kIdescBMajorMN;
      const uint64_t dp = ptx::smem_desc_noswizzle(&S.p[0][0][0], kHAtt * 16, 128);
      const uint64_t dx = ptx::smem_desc_noswizzle(&S.xo[0][0][0], 128, 512);
      for_items([&](const Pair& x, int, int c0, int nc, uint32_t n, uint32_t items) {
#pragma unroll 1
        for (int j = 0; j < nc && good; ++j) {
          const uint32_t m = n + (uint32_t)j;
          if (rank) {
            pass_rows(1, x, c0 + j);
            continue;
          }
          good = wait_pair(&S.p_full[m & 1], m >> 1);
          if (good && j == 0 && items > 0) good = wait_pair(&S.o_read, items - 1);
          const uint64_t dpo = dp + (uint64_t)((m & 1u) * (kChunk / 8 * kHAtt * 16 / 16));
#pragma unroll 1
          for (int i = 0; i < kPieces && good; ++i) {
            good = wait_pair(&S.x_full[1][i], m);
            if (!good) break;
            ptx::tc_fence_after();
            // p[4 i ..]: 2 KB a K step; xo[i], rows 16 ks: 256 bytes a step
#pragma unroll
            for (int h = 0; h < 2; ++h)  // channels 128 h .. of each CTA: xo[i][16 h], 8 KB on
              ptx::mma_f16_ss_pair_run_elect<2, 128, 16>(tmem + 128u * (uint32_t)h, dpo + (uint64_t)(2 * i * 128),
                                                         dx + (uint64_t)(i * 1024 + h * 512), idesc_o,
                                                         (j | i) > 0 ? 1u : 0u);
            ptx::mma_commit_pair_elect(&S.x_free[1][i]);
          }
          if (good) ptx::mma_commit_pair_elect(&S.p_free[m & 1]);
        }
      });
      where = 34;
    } else if (rank) {  // P, and O read
      for_items([&](const Pair&, int, int, int nc, uint32_t n, uint32_t items) {
#pragma unroll 1
        for (int j = 0; j < nc && good; ++j) {
          const uint32_t m = n + (uint32_t)j;
          pass(&S.p_full[m & 1], m >> 1, 1);
          if (j == 0 && items > 0) pass(&S.o_read, items - 1, 1);
        }
      });
      where = 36;
    }
  } else {
    // ---- softmax: thread t head t % 64, chunk rows 64 (t / 64) ..
    ptx::setmaxnreg_inc<kSoftRegs>();
    const int h = tid & 63, half = tid >> 6;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    // An item's partial (reference, sum, O) is written when the next one's first P is on its way, so that the
    // MMAs of both run on meanwhile; the last item's by the row warps.
    bool open = false;
    uint32_t open_last = 0;  // its last chunk
    int open_slot = 0;       // its partial's slot, or -1 - slot without a query
    float open_m = 0.0f, open_l = 0.0f;
    auto finish = [&](bool ends) {
      good = wait(&S.p_free[open_last & 1u], open_last >> 1);
      // the four warps leave together, or none
      good = softmax_vote(false, !good || *abort_flag != 0, lane) < 8;
      if (!good) return;
      ptx::tc_fence_after();
      S.red[half][h] = open_l;
      if (ends && tid == 0) S.last_slot = open_slot;
      softmax_sync();
      const float l = S.red[0][h] + S.red[1][h];
      if (ends) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&S.last_o);
      } else {
        softmax_sync();
      }
      if (open_slot >= 0) {
        if (!ends) store_pair_o<kHalf>(k, tmem, open_slot, tid, l, 0, 8);
        if (half == 0) k.part_ml[(int64_t)open_slot * kHAtt + h] = make_float2(open_m, l);
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.o_read);
    };
    for_items([&](const Pair& x, int slot_of, int c0, int nc, uint32_t n, uint32_t) {
      const int qme = rank ? x.q1 : x.q0, vis = rank ? x.vis1 : x.vis0;
      float m2 = -INFINITY, lsum = 0.0f;
      const float c2 = k.c2[(int64_t)(qme >= 0 ? qme : k.B) * kHAtt + h];
#pragma unroll 1
      for (int j = 0; j < nc; ++j) {
        const uint32_t m = n + (uint32_t)j, slot = m & 1u;
        good = good && wait(&S.r_full[m & 3u], m >> 2) && wait(&S.s_full[slot], m >> 1);
        if (good && m >= 2) good = wait(&S.p_free[slot], (m >> 1) - 1);
        ptx::tc_fence_after();
        uint32_t mk0 = 0u, mk1 = 0u;
        if (kTree) {
          mk0 = mk1 = ~0u;
        } else if (c0 + j < x.nshared) {  // entries below this query's own count
          const int left = vis - (c0 + j) * kChunk - 64 * half;
          mk0 = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1u : 0u;
          mk1 = left >= 64 ? ~0u : left > 32 ? (1u << (left - 32)) - 1u : 0u;
        } else if (c0 + j - x.nshared < x.paired ? half == rank : (x.own1 > x.own0) == (rank == 1)) {
          mk0 = mk1 = ~0u;
        }
        mk0 &= __ballot_sync(0xffffffffu, counts<kTree>(S.rows[m & 3u][64 * half + lane]));
        mk1 &= __ballot_sync(0xffffffffu, counts<kTree>(S.rows[m & 3u][64 * half + 32 + lane]));
        if (good && lane == 0) ptx::mbar_arrive(&S.r_free[m & 3u]);
        // P with the reference so far (0 before the first row); it stands unless some head's logits
        // exceed it by too much (kMaxExp), then once more with that head's new reference
        float alpha = 1.0f, sum, ref = m2 == -INFINITY ? 0.0f : m2;
        uint32_t nv;
#pragma unroll 1
        for (int round = 0;; ++round) {
          float top = -INFINITY;
          sum = 0.0f;
          if (good) {
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              uint32_t a[32], ph[16];
              uint64_t e[16];
              float s1;
              ptx::tmem_ld_32x32b_x32(tmem + lane_base + kColS + 64u * slot + 32u * (uint32_t)i, a);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 16; ++u) e[u] = pack2(a[2 * u], a[2 * u + 1]);
              top = fmaxf(top, probs32(e, i ? mk1 : mk0, c2, ref, ph, s1));
              sum += s1;
#pragma unroll
              for (int u = 0; u < 4; ++u)
                *reinterpret_cast<uint4*>(&S.p[slot][8 * half + 4 * i + u][h * 8]) =
                    make_uint4(ph[4 * u], ph[4 * u + 1], ph[4 * u + 2], ph[4 * u + 3]);
            }
            ptx::fence_proxy_async_smem();
          }
          if (round) break;
          const bool over = m2 == -INFINITY ? top > -INFINITY : top > kMaxExp;
          nv = softmax_vote(__any_sync(0xffffffffu, over), !good || *abort_flag != 0, lane);
          if (nv == 0 || nv >= 8) break;
          S.red[half][h] = top;
          softmax_sync();
          const float cm = fmaxf(S.red[0][h], S.red[1][h]) + ref;  // over both threads' rows
          if (m2 == -INFINITY ? cm > -INFINITY : cm > m2 + kMaxExp) {
            alpha = m2 == -INFINITY ? 0.0f : ptx::ex2(m2 - (cm - kTopExp));
            m2 = cm - kTopExp;
          }
          ref = m2 == -INFINITY ? 0.0f : m2;
        }
        if (nv >= 8) {
          good = false;
          break;
        }
        if (nv != 0 && j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
          // O holds earlier chunks: scale the rows of the heads that moved
          good = wait(&S.p_free[slot ^ 1u], (m - 1) >> 1);
          if (good) {
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 256; c += 32) {
              uint32_t a[32];
              ptx::tmem_ld_32x32b_x32(tmem + lane_base + (uint32_t)c, a);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 32; ++u) a[u] = __float_as_uint(__uint_as_float(a[u]) * alpha);
              ptx::tmem_st_32x32b_x32(tmem + lane_base + (uint32_t)c, a);
            }
            ptx::tmem_wait_st();
          }
        }
        if (good) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&S.p_full[slot]);
        }
        lsum = fmaf(alpha, lsum, sum);
        if (j == 0 && open) {
          finish(false);
          if (!good) break;
        }
      }
      good = softmax_vote(false, !good || *abort_flag != 0, lane) < 8;  // together, or none
      open = true;
      open_last = n + (uint32_t)nc - 1;
      open_slot = slot_of * 2 + rank;
      if (qme < 0) open_slot = -1 - open_slot;
      open_m = m2;
      open_l = lsum;
    });
    if (open && good) finish(true);
    where = 35;
  }
  if (!good && lane == 0 && !*abort_flag) {
    *abort_flag = 1;
    report_error(k.ws, CSA2_ERR_DEVICE_TIMEOUT, where);
  }
  if (warp == kSMma || warp == kOMma) {  // every MMA has completed, for both, before tensor memory is freed
    if (rank == 0) ptx::mma_commit_pair_elect(&S.drained);
    volatile int keep_waiting = 0;
    ptx::mbar_wait_warp(&S.drained, 0, &keep_waiting, kWaitBudget);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // no CTA leaves while the other may still arrive on its barriers
  if (warp == kSMma) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, kCols);
  }
}

// ------------------------------------------------------ preparation and merge

// 16 heads of a query into its f16 image and c2 (attn.cuh, stage_q: the same steps, from global memory, a warp to a
// head, lane l holding channels 16 l ..), and the rotation's cosines and sines.  The image goes through shared
// memory with padded planes, so that its stores are runs of 256 bytes.  Instructions bound it: with a CTA
// for all 64 heads the call on 32 normalised and rotated queries took 63.9 us, with four 58.9.
constexpr int kStageCtas = 4, kStageHeads = kHAtt / kStageCtas;  // of a query; heads of each
static_assert(kStageHeads == kPrepThreads / 32, "a head for each warp");
// CTAs that stage in a call for trees, at most.  A part for each CTA / 304 CTAs for all, us of the preparation: 1,536 queries
// 110 / 93, 664 42 / 36, 256 (with norm, rotation and 128 MB of image) 60 / 57.
constexpr int kStageMost = 304;
constexpr int kQPad = kStageHeads * 16 + 16;  // bytes of a plane
constexpr int kPrepSmem = 64 * 1024;          // this, or the plan's lists
static_assert(kDMain / 8 * kQPad <= kPrepSmem, "shared memory of the staging");
// This thread's channels of a query's part.
struct StageWords {
  uint4 w0, w1;
};
__device__ __forceinline__ StageWords stage_words(const PrefixQuery& a, int b, int part) {
  const int h = kStageHeads * part + (threadIdx.x >> 5);
  const uint4* src = reinterpret_cast<const uint4*>(a.q + ((int64_t)b * kHAtt + h) * kDMain) + 2 * (threadIdx.x & 31);
  return StageWords{src[0], src[1]};
}
// words: read already, or null
__device__ __forceinline__ void stage_block(const PrefixQuery& a, int B, int b, int part, unsigned char* smem,
                                            const StageWords* words = nullptr) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = kStageHeads * part + warp;
  uint4* const img = reinterpret_cast<uint4*>(a.image + (int64_t)b * kHAtt * kDMain) + kStageHeads * part;
  auto image_at = [&](int i) -> uint4& { return img[i / kStageHeads * kHAtt + i % kStageHeads]; };
  if (b == B) {  // the missing second query of an odd group
    for (int i = threadIdx.x; i < kStageHeads * kDMain / 8; i += kPrepThreads) image_at(i) = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0) a.c2[(int64_t)b * kHAtt + h] = 1.0f;
    return;
  }
  const StageWords x = words ? *words : stage_words(a, b, part);
  const uint4 q0 = x.w0, q1 = x.w1;
  float4 g[4];
  if (a.norm_w)
#pragma unroll
    for (int j = 0; j < 4; ++j) g[j] = __ldg(reinterpret_cast<const float4*>(a.norm_w) + 4 * lane + j);
  __shared__ float2 s_turn[32];
  if (a.rope && warp == 0) {  // one warp: the angles are formed in fp64, of which an SM does little
    float c, s;
    rope_cos_sin(a.th.t[lane], (double)a.qpos[b], c, s);
    s_turn[lane] = make_float2(c, s);
    if (part == 0) a.turn[(int64_t)b * 32 + lane] = make_float2(c, s);
  }
  {
    const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
    float v[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
    if (a.norm_w) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = 1.0f / sqrtf(ss / (float)kDMain + a.eps);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[4 * j] = g[j].x * (v[4 * j] * r);
        v[4 * j + 1] = g[j].y * (v[4 * j + 1] * r);
        v[4 * j + 2] = g[j].z * (v[4 * j + 2] * r);
        v[4 * j + 3] = g[j].w * (v[4 * j + 3] * r);
      }
    }
    if (a.rope) {
      __syncthreads();
      if (lane >= 28)  // these hold the pairs 8 (l - 28) ..
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 t = s_turn[8 * (lane - 28) + j];
          rope_pair(v[2 * j], v[2 * j + 1], t.x, t.y);
        }
    }
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) mx = fmaxf(mx, fabsf(v[j]));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const int sig = mx > 0.0f ? min(max(floor_log2_f32(mx) - 14, -126), 126) : 0;
    const float inv = exp2i_f32(-sig);
    uint32_t o[8], rest[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v0 = v[2 * j] * inv, v1 = v[2 * j + 1] * inv;
      const __half2 h2 = __floats2half2_rn(v0, v1);
      const __half2 r2 = __floats2half2_rn(v0 - __low2float(h2), v1 - __high2float(h2));
      o[j] = *reinterpret_cast<const uint32_t*>(&h2);
      rest[j] = *reinterpret_cast<const uint32_t*>(&r2);
    }
    if (a.rest) {
      uint4* rp = reinterpret_cast<uint4*>(a.rest + ((int64_t)b * kHAtt + h) * kDMain) + 2 * lane;
      rp[0] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
      rp[1] = make_uint4(rest[4], rest[5], rest[6], rest[7]);
    }
    *reinterpret_cast<uint4*>(smem + (2 * lane) * kQPad + warp * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(smem + (2 * lane + 1) * kQPad + warp * 16) = make_uint4(o[4], o[5], o[6], o[7]);
    if (lane == 0) a.c2[(int64_t)b * kHAtt + h] = kLog2e * a.scale * exp2i_f32(sig);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kStageHeads * kDMain / 8; i += kPrepThreads)
    image_at(i) = *reinterpret_cast<const uint4*>(smem + (i / kStageHeads) * kQPad + (i % kStageHeads) * 16);
}

// The image's chunks first, first + step, ..: a warp's lane l widens four blocks (of 32 channels), the rotated
// one xor 4 i, of row l % 8 of its eight, and stores 16 bytes to each of the block's four planes, 128 contiguous
// bytes for eight rows.  Bytes bound it: 288 read and 1,024 written an entry (65,000 entries: about 20 us, 12 of
// them the bytes').  The rows of a CTA's next chunk are asked for with this one's (64 on 65000 386.7 us without,
// 384.1 with).
template <bool kTree>
__device__ __forceinline__ void widen_chunks(const PrefixArgs& a, const PrefixKernel& k, uint16_t* image, int first_chunk,
                                             int step) {
  __shared__ int s_warp[kPrepThreads / 32];
  __shared__ int2 s_found;   // the row's query (-1: no such group) and the shared entries
  __shared__ int2 s_chunks;  // the group's first chunk, and the next group's
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b0 = rotated(lane) & 7;
  auto row_of = [&](int first, int e) {  // a page outside the planes is reported by the attention
    const int pi = (int)((uint64_t)e * k.page_div >> 40);
    return resolve(k, RowRef{k.table[first * k.max_pages + pi], e - pi * k.page_entries}, false);
  };
  int2 found = make_int2(-1, 0), chunks = make_int2(0, 0);
  for (int64_t t = first_chunk;; t += step) {
    if (t >= chunks.y) {  // the group whose image holds chunk t
      __syncthreads();
      if (threadIdx.x == 0) s_found.x = -1;
      __syncthreads();
      int base = 0;
      for (int g0 = 0; g0 < a.G && base <= t; g0 += kPrepThreads) {
        const int g = g0 + threadIdx.x;
        const int lo = g < a.G ? a.group_start[g] : 0, hi = g < a.G ? a.group_start[g + 1] : 0;
        const bool any = (kTree ? tree_ok(a, lo, hi) : lo >= 0 && hi <= a.B) && hi - lo >= kImageQueries;
        int2 sh = make_int2(g, 0);
        if constexpr (!kTree) sh = shared_of(a, any, g, lo, hi);
        else if (any) sh.y = tree_context(a, g);
        const int n = !any ? 0 : kTree ? tree_image_chunks(hi - lo, sh.y) : image_chunks(hi - lo, sh.y);
        int total;
        const int at = base + block_scan(n, s_warp, &total);
        if (n > 0 && at + (int64_t)n <= a.image_cap && t >= at && t < at + n) {
          s_found = sh;
          s_chunks = make_int2(at, at + n);
        }
        base += total;
      }
      __syncthreads();
      found = s_found;
      if (found.x < 0) return;
      chunks = s_chunks;
    }
    const int row = 8 * warp + (lane & 7), e = (int)(t - chunks.x) * kChunk + row;
    const int r = e < found.y ? row_of(found.x, e) : kNoRow;
    Fetch f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) fetch<kTree>(f[i], k, r, b0 ^ (4 * i));
    const int64_t next = e + (int64_t)step * kChunk;
    if (lane < 8 && next < found.y) prefetch_row<kTree>(k, row_of(found.x, (int)next));
    uint16_t* dst = image + t * kDMain * kChunk + row * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) put(f[i], r, dst + (b0 ^ (4 * i)) * 4 * kChunk * 8, kChunk * 8);
  }
}

// Ancestors and depths of the tokens of request g (trees), by a warp: lane l has the tokens l and 32 + l, each at first
// itself and its parent, and follows the parents in steps of twice the length: six for 64 tokens.
__device__ __forceinline__ void tree_block(const PrefixArgs& a, int g) {
  const int lane = threadIdx.x & 31, first = a.group_start[g], end = a.group_start[g + 1];
  if (!tree_ok(a, first, end)) return;
  uint32_t lo[2], hi[2];  // tokens 0 .. 31 and 32 .. 63
  int up[2];
  bool bad[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 32 * i + lane;
    up[i] = t < end - first ? a.parent[first + t] : -1;
    bad[i] = up[i] < -1 || up[i] >= t;
    if (bad[i]) up[i] = -1;
    lo[i] = i == 0 ? 1u << lane : 0u;
    hi[i] = i == 0 ? 0u : 1u << lane;
  }
#pragma unroll
  for (int s = 0; s < 6; ++s) {
    uint32_t l[2], h[2];
    int u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int src = up[i] & 31;  // every lane shuffles
      auto of = [&](auto(&v)[2]) {
        const auto v0 = __shfl_sync(0xffffffffu, v[0], src), v1 = __shfl_sync(0xffffffffu, v[1], src);
        return up[i] >= 32 ? v1 : v0;
      };
      l[i] = of(lo);
      h[i] = of(hi);
      u[i] = of(up);
      if (up[i] < 0) {
        l[i] = h[i] = 0u;
        u[i] = -1;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lo[i] |= l[i];
      hi[i] |= h[i];
      up[i] = u[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 32 * i + lane;
    if (t >= end - first) continue;
    a.kin[first + t] = (uint64_t)hi[i] << 32 | lo[i];
    a.depth[first + t] = __popc(lo[i]) + __popc(hi[i]) - 1 + (bad[i] ? kBadParent : 0);
  }
}

// Everything the attention needs, by independent CTAs of one launch: the plan, the queries, the image, of which
// half the CTAs come first (all behind the queries: 53.4 and 75.1 us for prefix 32 on 8192 and 101 on 4001
// instead of 50.9 and 71.2).  Two CTAs on an SM: with the 72 registers it would take, one (ragged 101 on 4001
// 68.5 us instead of 66.0).
template <bool kTree>
__global__ void __launch_bounds__(kPrepThreads, 2) k_prefix_prep(PrefixArgs a, PrefixQuery q,
                                                              const __grid_constant__ PrefixKernel k, uint16_t* image) {
  extern __shared__ __align__(16) unsigned char prep_smem[];
  ptx::griddep_launch();
  ptx::griddep_wait();
  const int trees = kTree ? (a.G + kTreesPerCta - 1) / kTreesPerCta : 0;
  const int parts = kStageCtas * (a.B + 1), stage = kTree ? min(parts, kStageMost) : parts;
  const int widen = (int)gridDim.x - 1 - trees - stage, widen1 = min(widen, kWidenFirst);
  int b = (int)blockIdx.x - 1;
  if (b < 0) {
    int32_t* ints = reinterpret_cast<int32_t*>(prep_smem);
    if (alone_of<kTree>(a.B, a.G, a.shared_max)) plan_block<true, kTree>(a, ints, kPrepSmem / 4);
    else plan_block<false, kTree>(a, ints, kPrepSmem / 4);
    return;
  }
  if (b < trees) {
    const int g = b * kTreesPerCta + (int)(threadIdx.x >> 5);
    if (g < a.G) tree_block(a, g);
    return;
  }
  b -= trees;
  if (b < widen1) return widen_chunks<kTree>(a, k, image, b, widen);
  b -= widen1;
  if (b < stage && stage == parts) return stage_block(q, a.B, b / kStageCtas, b % kStageCtas, prep_smem);
  if (kTree && b < stage) {  // parts b, b + stage, ..: the next one's words are on their way while one is worked on
    StageWords w{}, next{};
    if (b < parts - kStageCtas) w = stage_words(q, b / kStageCtas, b % kStageCtas);  // the last query is none
    for (int i = b; i < parts; i += stage) {
      const int n = i + stage;
      if (n < parts - kStageCtas) next = stage_words(q, n / kStageCtas, n % kStageCtas);
      if (i != b) __syncthreads();  // shared memory is written again
      stage_block(q, a.B, i / kStageCtas, i % kStageCtas, prep_smem, &w);
      w = next;
    }
    return;
  }
  widen_chunks<kTree>(a, k, image, widen1 + b - stage, widen);
}

// kC consecutive output channels at element `at`
template <bool kBf16, int kC>
__device__ __forceinline__ void store_channels(void* out, int64_t at, const float (&v)[kC]) {
  if (kBf16) {
    uint32_t w[kC / 2];
#pragma unroll
    for (int u = 0; u < kC / 2; ++u) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * u], v[2 * u + 1]);
      w[u] = *reinterpret_cast<const uint32_t*>(&x);
    }
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
    for (int u = 0; u < kC / 8; ++u) o[u] = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
  } else {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int u = 0; u < kC / 4; ++u) o[u] = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
  }
}

// The join of a query's partials.  Partial i has reference m_i (log2 units), sum l_i and O_i / l_i:
//   out = sum 2^(m_i - m) l_i (O_i / l_i) / L,  L = sum 2^(m_i - m) l_i  (+ 2^(z - m) of the sink).
// Latency bounds it: a thread reads up to 16 words of partials at once (references and channels in one round
// trip), and for few queries, which are cut into many partials, four slices of a CTA's threads take every fourth
// and the first joins the four.  A call with one slice / four, us: one query of 4,096 entries (66 partials) 31.2 /
// 15.6, eight 24.4 / 21.1, 15 28.2 / 30.8, 32 37.0 / 47.3; 8 queries on 65,000 shared entries 77.0 / 78.1, 15 on
// 20,000 52.7 / 58.0.
constexpr int kSliceQueries = 12;  // below this many queries: four slices

// the running join of one head's kC channels
template <int kC>
struct Join {
  float ref, L, acc[kC];
  __device__ __forceinline__ void start(float z) {  // z: the sink's logit (log2 units) or -inf
    ref = z;
    L = z == -INFINITY ? 0.0f : 1.0f;
#pragma unroll
    for (int u = 0; u < kC; ++u) acc[u] = 0.0f;
  }
  __device__ __forceinline__ void raise(float top) {
    if (!(top > ref)) return;
    const float f = ref > -INFINITY ? ptx::ex2(ref - top) : 0.0f;
    L *= f;
#pragma unroll
    for (int u = 0; u < kC; ++u) acc[u] *= f;
    ref = top;
  }
};

// The logsumexp of queries that were rounded to f16.  With q = q' + r, r of at most 2^-11 |q|, the joins give
// lse(q'), and lse(q) = lse(q') + E + (at most w^2 / 8), E = the mean of scale r x under q's own weights and w the
// width of scale r x over the rows (Hoeffding's lemma): E = scale r o with the output o before it turns back.
// Without it one row of 512 normal channels is off by 2 10^-4, with it by 10^-8.  So a CTA has all channels of its
// heads, or is in a cluster of those that have (a counter in global memory and its fence for the last of a
// query's CTAs instead: 2 to 3 us more a call).
struct LseRest {
  const uint16_t* rest;  // null: q was not rounded, or no logsumexp is asked for
  const float* c2;
};
// ref + log2 L in natural units.  A sum is 2^11 (kTopExp) or more: its exponent joins the reference first, so that
// the logarithm's rounding is that of a number below one.
__device__ __forceinline__ float natural(float ref, float L) {
  const int e = (int)(__float_as_uint(L) >> 23) - 127;
  return (isfinite(L) ? ref + (float)e + log2f(L * exp2i_f32(-e)) : ref + log2f(L)) / kLog2e;
}
__device__ __forceinline__ float corrected(const LseRest& f, int b, int h, float l, float e) {
  // a query without rows may hold anything
  return l > -INFINITY && isfinite(e) ? fmaf(e, f.c2[(int64_t)b * kHAtt + h] / kLog2e, l) : l;
}

// A CTA joins 8 / kSlices heads: thread t of a slice has head t % (8 / kSlices) of them and kVec planes (of eight
// channels): two, which share a weight, or one where slices make for more threads (one for all: 4 us more for
// 101 queries).
// Many queries of trees have two partials or so: two at once leave room for more CTAs on an SM (the join of 256 queries
// 28 us with eight, 19 with two, of 664 39 and 25).
template <int kSlices, bool kHalf, bool kTree>
struct PrefixMerge {
  static constexpr int kVec = kSlices > 1 ? 1 : 2, kHeads = 8 / kSlices, kPer = kHeads * (kDMain / 8) / kVec;
  static constexpr int kAhead = kSlices > 1 ? 8 : kTree ? 2 : kHalf ? 8 : 4;  // partials read at once
  static constexpr int kThreads = kPer * kSlices, kCtas = kTree && kSlices == 1 ? (kHalf ? 5 : 4) : 1;
};
template <int kSlices, bool kHalf, bool kTree>
__global__ void __launch_bounds__(PrefixMerge<kSlices, kHalf, kTree>::kThreads,
                                  PrefixMerge<kSlices, kHalf, kTree>::kCtas)
    k_prefix_merge(const int2* __restrict__ qpart, const uint4* __restrict__ part_o, const float2* __restrict__ part_ml,
                   const float* __restrict__ sink, const float2* __restrict__ turn, void* __restrict__ out,
                   float* __restrict__ lse, LseRest fix) {
  using Form = PrefixMerge<kSlices, kHalf, kTree>;
  using Vec = Vec8<kHalf>;
  constexpr int kVec = Form::kVec, kHeads = Form::kHeads, kPer = Form::kPer, kC = 8 * kVec, kAhead = Form::kAhead;
  __shared__ float s_join[kSlices > 1 ? kSlices - 1 : 1][2 + kC][kSlices > 1 ? kPer : 1];
  __shared__ float s_dot[kPer / 32][kHeads];
  ptx::griddep_wait();
  const int b = blockIdx.x, slice = threadIdx.x / kPer, t = threadIdx.x % kPer, plane = t / kHeads * kVec;
  const int h = blockIdx.y * kHeads + t % kHeads;
  const int2 part = qpart[b];  // twice the first partial's slot, plus the query's place in its pair; partials
  Join<kC> a;
  a.start(slice == 0 && sink ? sink[h] * kLog2e : -INFINITY);
  // the epilogue's thread h + 64 (plane / 32) wrote vector plane % 32
  const uint4* po = part_o + (plane & 31) * Vec::kWords * 128 + 64 * (plane >> 5) + h;
  for (int c0 = slice; c0 < part.y; c0 += kSlices * kAhead) {
    float2 ml[kAhead];
    Vec v[kAhead][kVec];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      ml[i] = make_float2(-INFINITY, 0.0f);
      if (c0 + i * kSlices < part.y) {
        const int64_t slot = part.x + 2 * (int64_t)(c0 + i * kSlices);
        ml[i] = part_ml[slot * kHAtt + h];
#pragma unroll
        for (int u = 0; u < kVec; ++u) v[i][u].load(po + (slot * 32 + u) * Vec::kWords * 128);
      }
    }
    float top = a.ref;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (ml[i].y != 0.0f) top = fmaxf(top, ml[i].x);
    a.raise(top);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (ml[i].y == 0.0f) continue;
      const float f = ptx::ex2(ml[i].x - a.ref) * ml[i].y;
      a.L += f;
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        float x[8];
        v[i][u].get(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) a.acc[8 * u + j] = fmaf(f, x[j], a.acc[8 * u + j]);
      }
    }
  }
  if (kSlices > 1) {
    if (slice > 0) {
      s_join[slice - 1][0][t] = a.ref;
      s_join[slice - 1][1][t] = a.L;
#pragma unroll
      for (int u = 0; u < kC; ++u) s_join[slice - 1][2 + u][t] = a.acc[u];
    }
    __syncthreads();
    if (slice > 0) return;
#pragma unroll
    for (int i = 0; i < kSlices - 1; ++i) {
      const float m = s_join[i][0][t], l = s_join[i][1][t];
      if (l == 0.0f) continue;
      a.raise(m);
      const float f = ptx::ex2(m - a.ref);
      a.L = fmaf(f, l, a.L);
#pragma unroll
      for (int u = 0; u < kC; ++u) a.acc[u] = fmaf(f, s_join[i][2 + u][t], a.acc[u]);
    }
  }
  const float inv = a.L > 0.0f ? 1.0f / (Vec::kScale * a.L) : 0.0f;
#pragma unroll
  for (int u = 0; u < kC; ++u) a.acc[u] *= inv;
  if (lse) {
    float e = 0.0f;
    if (fix.rest) {
      const __half2* r = reinterpret_cast<const __half2*>(fix.rest + ((int64_t)b * kHAtt + h) * kDMain + 8 * plane);
#pragma unroll
      for (int u = 0; u < kC / 2; ++u) {
        const float2 x = __half22float2(r[u]);
        e = fmaf(x.x, a.acc[2 * u], fmaf(x.y, a.acc[2 * u + 1], e));
      }
#pragma unroll
      for (int o = 16; o >= kHeads; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
      if ((t & 31) < kHeads) s_dot[t >> 5][t & 31] = e;
      asm volatile("bar.sync 1, %0;" ::"n"(kPer) : "memory");
      e = 0.0f;
      if (t < kHeads)
        for (int i = 0; i < kPer / 32; ++i) e += s_dot[i][t];
    }
    if (t < kHeads) {
      const float l = a.L == 0.0f ? -INFINITY : natural(a.ref, a.L);
      lse[b * kHAtt + h] = fix.rest ? corrected(fix, b, h, l, e) : l;
    }
  }
  if (turn && plane >= kRopeFirst / 8) {  // turn back by -q_pos
    const float2* cs = turn + (int64_t)b * 32 + 4 * (plane - kRopeFirst / 8);
#pragma unroll
    for (int u = 0; u < kC / 2; ++u) rope_pair(a.acc[2 * u], a.acc[2 * u + 1], cs[u].x, -cs[u].y);
  }
  store_channels<kHalf>(out, ((int64_t)b * kHAtt + h) * kDMain + 8 * plane, a.acc);
}

// ------------------------------------------------------------ queries alone

// Queries that share nothing run one to a CTA (a pair of them in one MMA would multiply each one's rows by
// the other's probabilities): 64 heads, chunks of 64 rows in two slots, every row widened once.
//   S[64 x 64] = q' X^T    heads as M;
//   O^T[512 x 64] += X^T P^T  four tiles of 128 channels, so that the rows serve both products as they are.
// Shared memory bounds a chunk: 128 KB read by the S MMAs, 96 KB by the O MMAs, 64 KB of rows and 8 KB of P
// written, 296 KB = 2,300 cycles at 128 bytes a cycle; the MMAs alone (S at the half rate of M = 64) take
// 1,800; measured, about 2,800, the wait of a slot for its softmax among them.  48 queries of up to 65,536 entries
// take 217 us (0.80 PFLOP/s, 1.8 TB/s of entries), one of 4,096 entries 16 us, three launches.
constexpr int kAlone = 152;
constexpr int kRows = 64;  // rows of a chunk
constexpr int kRing = 8;   // chunks whose rows are found ahead

struct __align__(1024) AloneSmem {
  uint16_t x[2][kDMain / 8][kRows * 8];  // rows [c/8][row][c%8]
  uint16_t q[kDMain / 8][kQPlane];       // q' [c/8][head][c%8]
  uint16_t p[2][kRows / 8][kHAtt * 8];   // probabilities [row/8][head][row%8]
  __align__(16) float alpha[kHAtt];      // factor of O when a head's reference moved; at the end 1 / l (read four at a time)
  int32_t last_slot;                     // the last item's partial
  uint64_t last_o;                       // its O complete, 1 / l in alpha (four softmax warps)
  int32_t rows[kRing][kRows];
  uint64_t q_land;
  uint64_t r_full[kRing], r_free[kRing];
  uint64_t x_full[2][2], x_free[2][2];   // slot, channel half
  uint64_t s_full[2], p_full[2];
  uint64_t o_read, drained;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(AloneSmem) <= 232448, "attention shared memory");

// warps 0-3: softmax and epilogue; 4-19: rows (4-11 channels 0-255, 12-19 the others); then one warp
// each: S MMAs, O MMAs, where rows come from
constexpr int kAloneS = 20, kAloneO = 21, kAloneIndex = 22;

// The rows of all `chunks` chunks of this CTA, whatever queries they belong to: thread's row 8 (w % 8) + l % 8,
// of the blocks (of 32 channels) 8 (w / 8) .. the rotated first and the one four on; codes fetched two chunks ahead.
template <bool kTree>
__device__ __forceinline__ bool alone_rows(AloneSmem& S, const PrefixKernel& k, int chunks, int w, int lane) {
  const int half = w >> 3, rl = 8 * (w & 7) + (lane & 7);
  const int b0 = 8 * half + (rotated(lane) & 7), b1 = b0 ^ 4;
  uint16_t* const dst = &S.x[0][4 * b0][rl * 8];
  const int to_b1 = (b1 - b0) * 4 * kRows * 8;
  bool good = true;
  int ra, rb;
  Fetch fa[2], fb[2];
  auto load = [&](Fetch (&f)[2], int& r, int m) {
    if (m >= chunks) return;
    const uint32_t slot = (uint32_t)m % kRing;
    good = good && ptx::mbar_wait_warp(&S.r_full[slot], ((uint32_t)m / kRing) & 1u, &S.abort_flag, kWaitBudget);
    if (!good) return;
    r = S.rows[slot][rl];
    fetch<kTree>(f[0], k, r, b0);
    fetch<kTree>(f[1], k, r, b1);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.r_free[slot]);
  };
  load(fa, ra, 0);
  load(fb, rb, 1);
  auto step = [&](Fetch (&f)[2], int& r, int m) {
    if (m >= chunks) return;
    const uint32_t slot = (uint32_t)m & 1u;
    if (m >= 2)
      good = good && ptx::mbar_wait_warp(&S.x_free[slot][half], (((uint32_t)m >> 1) - 1) & 1u, &S.abort_flag,
                                         kWaitBudget);
    if (!good) return;
    uint16_t* d = dst + slot * (kDMain * kRows);
    put(f[0], r, d, kRows * 8);
    put(f[1], r, d + to_b1, kRows * 8);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.x_full[slot][half]);
    load(f, r, m + 2);
  };
#pragma unroll 1
  for (int m = 0; m < chunks && good; m += 2) {
    step(fa, ra, m);
    step(fb, rb, m + 1);
  }
  return good;
}

// Tiles' columns 32 c0 .. 32 c1 of O^T / l, thread t's channels; vector (c, u) of thread t holds heads
// 32 (c % 2) + 8 u .. of channel 128 (c / 2) + t.  1 / l comes scaled (Vec8).
template <bool kHalf>
__device__ __forceinline__ void store_alone_o(const AloneSmem& S, const PrefixKernel& k, uint32_t tmem, int64_t slot, int t,
                                              int c0, int c1) {
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    uint32_t a[32];
    ptx::tmem_ld_32x32b_x32(tmem + ((uint32_t)(t & ~31) << 16) + 32u * (uint32_t)c, a);
    ptx::tmem_wait_ld();
    uint4* po = k.part_o + (slot * 32 + 4 * c) * Vec8<kHalf>::kWords * 128 + t;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float4* i8 = reinterpret_cast<const float4*>(&S.alpha[32 * (c & 1) + 8 * u]);
      const float4 f0 = i8[0], f1 = i8[1];
      const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
      Vec8<kHalf>::store(po + u * Vec8<kHalf>::kWords * 128, [&](int i) { return __uint_as_float(a[8 * u + i]) * f[i]; });
    }
  }
}

template <bool kHalf, bool kTree>
__global__ void __launch_bounds__(kThreads, 1) k_paged_attn(const __grid_constant__ PrefixKernel k) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  AloneSmem& S = *reinterpret_cast<AloneSmem*>(smem_raw);
  volatile int* abort_flag = &S.abort_flag;
  const int cta = blockIdx.x;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  if (warp == kAloneS) {
    if (lane == 0) {
      ptx::mbar_init(&S.q_land, 1);
      for (int i = 0; i < kRing; ++i) {
        ptx::mbar_init(&S.r_full[i], 1);
        ptx::mbar_init(&S.r_free[i], 20);
      }
      for (int i = 0; i < 2; ++i) {
        for (int h = 0; h < 2; ++h) {
          ptx::mbar_init(&S.x_full[i][h], 8);
          ptx::mbar_init(&S.x_free[i][h], 1);
        }
        ptx::mbar_init(&S.s_full[i], 1);
        ptx::mbar_init(&S.p_full[i], 4);
      }
      ptx::mbar_init(&S.o_read, 4);
      ptx::mbar_init(&S.last_o, 4);
      ptx::mbar_init(&S.drained, 2);
      S.abort_flag = 0;
      ptx::fence_mbar_init();
    }
    __syncwarp();
    ptx::tmem_alloc(&S.tmem_base, kCols);
  }
  ptx::griddep_launch();
  ptx::griddep_wait();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  const Part& part = k.parts[cta];
  const int t0 = part.t0, t1 = part.t1;
  auto wait = [&](uint64_t* bar, uint32_t n) { return ptx::mbar_wait_warp(bar, n & 1u, abort_flag, kWaitBudget); };
  bool good = true;
  int where = 0;
  auto for_items = [&](auto body) {  // as in k_prefix_attn, over queries
    const Pair* px = &part.pair;
    int p = part.p, end = part.end;
    uint32_t n = 0, items = 0;
    for (int t = t0; t < t1 && good;) {
      const Pair& x = *px;
      const int q = x.q0, c0 = t - x.chunk0, nc = min(end, t1) - t;
      if (nc > 0) {
        t += nc;
        body(q, x, p, c0, nc, n, items);
        n += (uint32_t)nc;
        ++items;
      }
      px = k.pairs + ++p;
      if (t < t1) end = k.pairs[p + 1].chunk0;
    }
  };

  if (warp >= 4 && warp < kAloneS) {
    good = alone_rows<kTree>(S, k, t1 - t0, warp - 4, lane);
    if (good && t1 > t0) {  // as in k_prefix_attn
      good = wait(&S.last_o, 0);
      if (good) {
        ptx::tc_fence_after();
        const int quarter = (warp - 4) / 4;
        store_alone_o<kHalf>(S, k, tmem, S.last_slot, 32 * (warp % 4) + lane, 2 * quarter, 2 * quarter + 2);
        ptx::tc_fence_before();
      }
    }
    where = 41;
  } else if (warp >= kAloneS) {
    if (warp == kAloneIndex) {
      ptx::prefetch_l1(&part.pair.ns);  // the record's second half
      for_items([&](int q, const Pair& x, int, int c0, int nc, uint32_t n, uint32_t) {
        const int own = x.own0, ns = x.ns, first = x.first;
        const Sight sight = kTree ? sight_of(k, q, lane) : Sight{};
        RowRef r[2];
        auto find = [&](int j) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int e = (c0 + j) * kRows + 32 * i + lane;
            if (kTree) r[i] = e < x.vis0 || sees(k, x, sight, e) ? find_tree(k, x, e) : RowRef{0, kNoRow};
            else r[i] = e < ns && e < own ? find_entry(k, first, e) : find_own(k, q, own, e);
          }
        };
        find(0);
#pragma unroll 1
        for (int j = 0; j < nc && good; ++j) {
          const uint32_t m = n + (uint32_t)j, slot = m % kRing;
          const int r0 = resolve(k, r[0], true), r1 = resolve(k, r[1], true);
          prefetch_row<kTree>(k, r0);  // paged ragged 48 x 65536: 219 us without, 217 with
          prefetch_row<kTree>(k, r1);
          if (j + 1 < nc) find(j + 1);
          if (m >= kRing) good = wait(&S.r_free[slot], m / kRing - 1);
          if (!good) break;
          S.rows[slot][lane] = r0;
          S.rows[slot][32 + lane] = r1;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&S.r_full[slot]);
        }
      });
      where = 42;
    } else if (warp == kAloneS) {
      // ---- S: 32 K steps, of each channel half as it comes
      constexpr uint32_t idesc_s = ptx::idesc_f16(64, kRows, 0);
      const uint64_t da = ptx::smem_desc_noswizzle(&S.q[0][0], kQPlane * 2, 128);
      const uint64_t db = ptx::smem_desc_noswizzle(&S.x[0][0][0], kRows * 16, 128);
      for_items([&](int q, const Pair&, int, int, int nc, uint32_t n, uint32_t items) {
        // the item's query, once S of the item before has left q'; it lands before anyone leaves
        good = n == 0 || wait(&S.s_full[(n - 1) & 1u], (n - 1) >> 1);
        if (!good) return;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&S.q_land, kHAtt * kDMain * 2);
          ptx::bulk_g2s(&S.q[0][0], k.q + (int64_t)q * kHAtt * kDMain, kHAtt * kDMain * 2, &S.q_land);
        }
        __syncwarp();
        volatile int keep_waiting = 0;
        good = ptx::mbar_wait_warp(&S.q_land, items & 1u, &keep_waiting, kWaitBudget);
#pragma unroll 1
        for (int j = 0; j < nc && good; ++j) {
          const uint32_t m = n + (uint32_t)j, slot = m & 1u, dst = tmem + kColS + 64u * slot;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            good = good && wait(&S.x_full[slot][half], m >> 1);  // O(m - 2) is done with the slot, so its softmax with S
            if (!good) break;
            ptx::tc_fence_after();
            const uint64_t das = da + (uint64_t)(half * 2048);
            const uint64_t dbs = db + (uint64_t)slot * (kDMain * kRows * 2 / 16) + (uint64_t)(half * 2048);
#pragma unroll
            for (int ks = 0; ks < 16; ks += 8)
              ptx::mma_f16_ss_run_elect<8, 128, 128>(dst, das + (uint64_t)(ks * 128), dbs + (uint64_t)(ks * 128), idesc_s,
                                                     (half | ks) > 0 ? 1u : 0u);
          }
          if (good) ptx::mma_commit_elect(&S.s_full[slot]);
        }
      });
      where = 43;
    } else if (warp == kAloneO) {
      // ---- O^T: per channel half two tiles of 128 channels, four K steps of 16 rows each
      constexpr uint32_t idesc_o = ptx::idesc_f16(128, kHAtt, 0) | (1u << 15);  // A M-major
      const uint64_t da = ptx::smem_desc_noswizzle(&S.x[0][0][0], 128, kRows * 16);
      const uint64_t db = ptx::smem_desc_noswizzle(&S.p[0][0][0], kHAtt * 16, 128);
      for_items([&](int, const Pair&, int, int, int nc, uint32_t n, uint32_t items) {
#pragma unroll 1
        for (int j = 0; j < nc && good; ++j) {
          const uint32_t m = n + (uint32_t)j, slot = m & 1u;
          good = wait(&S.p_full[slot], m >> 1);
          if (good && j == 0 && items > 0) good = wait(&S.o_read, items - 1);
          if (!good) break;
          ptx::tc_fence_after();
          const uint64_t das = da + (uint64_t)slot * (kDMain * kRows * 2 / 16);
          const uint64_t dbs = db + (uint64_t)slot * (kRows * kHAtt * 2 / 16);
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
              ptx::mma_f16_ss_run_elect<kRows / 16, 16, 128>(tmem + 64u * (uint32_t)(2 * half + mt),
                                                             das + (uint64_t)(half * 2048 + mt * 1024), dbs, idesc_o,
                                                             j > 0 ? 1u : 0u);
            ptx::mma_commit_elect(&S.x_free[slot][half]);
          }
        }
      });
      where = 44;
    }
  } else {
    // ---- softmax: lane l of warp w head 16 w + l % 16, chunk rows 32 (l / 16) .. (the rows of an M = 64
    // accumulator lie in lanes 0-15 of each quarter; two lanes share a head's columns)
    const int rh = lane >> 4, h = 16 * warp + (lane & 15);
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    bool open = false;  // as in k_prefix_attn
    uint32_t open_last = 0;
    int open_slot = 0;
    float open_m = 0.0f, open_l = 0.0f;
    auto finish = [&](bool ends) {
      good = wait(&S.x_free[open_last & 1u][0], open_last >> 1) && wait(&S.x_free[open_last & 1u][1], open_last >> 1);
      good = softmax_vote(false, !good || *abort_flag != 0, lane) < 8;
      if (!good) return;
      ptx::tc_fence_after();
      open_l += __shfl_xor_sync(0xffffffffu, open_l, 16);
      if (rh == 0) {
        S.alpha[h] = open_l > 0.0f ? Vec8<kHalf>::kScale / open_l : 0.0f;
        k.part_ml[(int64_t)open_slot * kHAtt + h] = make_float2(open_m, open_l);
      }
      if (ends) {
        if (tid == 0) S.last_slot = open_slot;
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&S.last_o);
        return;
      }
      softmax_sync();
      store_alone_o<kHalf>(S, k, tmem, open_slot, tid, 0, 8);
      softmax_sync();  // alpha is written again
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.o_read);
    };
    for_items([&](int q, const Pair&, int p, int, int nc, uint32_t n, uint32_t) {
      const float c2 = k.c2[(int64_t)q * kHAtt + h];
      float m2 = -INFINITY, lsum = 0.0f;
#pragma unroll 1
      for (int j = 0; j < nc; ++j) {
        const uint32_t m = n + (uint32_t)j, slot = m & 1u, ring = m % kRing;
        good = good && wait(&S.r_full[ring], m / kRing) && wait(&S.s_full[slot], m >> 1);
        ptx::tc_fence_after();
        const uint32_t k0 = __ballot_sync(0xffffffffu, S.rows[ring][lane] != kNoRow);
        const uint32_t k1 = __ballot_sync(0xffffffffu, S.rows[ring][32 + lane] != kNoRow);
        if (good && lane == 0) ptx::mbar_arrive(&S.r_free[ring]);
        const uint32_t mask = rh ? k1 : k0;
        float alpha = 1.0f, sum = 0.0f, ref = m2 == -INFINITY ? 0.0f : m2;
        uint32_t nv;
#pragma unroll 1
        for (int round = 0;; ++round) {
          float top = -INFINITY;
          if (good) {
            uint32_t a[32], ph[16];
            ptx::tmem_ld_16x32bx2_x32<32>(tmem + lane_base + kColS + 64u * slot, a);
            ptx::tmem_wait_ld();
            uint64_t e[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) e[u] = pack2(a[2 * u], a[2 * u + 1]);
            top = probs32(e, mask, c2, ref, ph, sum);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              *reinterpret_cast<uint4*>(&S.p[slot][4 * rh + u][h * 8]) =
                  make_uint4(ph[4 * u], ph[4 * u + 1], ph[4 * u + 2], ph[4 * u + 3]);
            ptx::fence_proxy_async_smem();
          }
          if (round) break;
          const bool over = m2 == -INFINITY ? top > -INFINITY : top > kMaxExp;
          nv = softmax_vote(__any_sync(0xffffffffu, over), !good || *abort_flag != 0, lane);
          if (nv == 0 || nv >= 8) break;
          const float cm = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)) + ref;
          if (m2 == -INFINITY ? cm > -INFINITY : cm > m2 + kMaxExp) {
            alpha = m2 == -INFINITY ? 0.0f : ptx::ex2(m2 - (cm - kTopExp));
            m2 = cm - kTopExp;
          }
          ref = m2 == -INFINITY ? 0.0f : m2;
        }
        if (nv >= 8) {
          good = false;
          break;
        }
        if (nv != 0 && j > 0) {  // O^T holds earlier chunks: scale the columns of the heads that moved
          if (rh == 0) S.alpha[h] = alpha;
          softmax_sync();
          good = wait(&S.x_free[slot ^ 1u][0], (m - 1) >> 1) && wait(&S.x_free[slot ^ 1u][1], (m - 1) >> 1);
          if (good) {
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {  // tile c / 2, heads 32 (c % 2) ..
              const float a32 = S.alpha[32 * (c & 1) + lane];
              if (!__any_sync(0xffffffffu, a32 != 1.0f)) continue;
              uint32_t a[32];
              ptx::tmem_ld_32x32b_x32(tmem + lane_base + 32u * (uint32_t)c, a);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 32; ++u)
                a[u] = __float_as_uint(__uint_as_float(a[u]) * __shfl_sync(0xffffffffu, a32, u));
              ptx::tmem_st_32x32b_x32(tmem + lane_base + 32u * (uint32_t)c, a);
            }
            ptx::tmem_wait_st();
          }
        }
        if (good) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&S.p_full[slot]);
        }
        lsum = fmaf(alpha, lsum, sum);
        if (j == 0 && open) {
          finish(false);
          if (!good) break;
        }
      }
      good = softmax_vote(false, !good || *abort_flag != 0, lane) < 8;
      open = true;
      open_last = n + (uint32_t)nc - 1;
      open_slot = p + cta;
      open_m = m2;
      open_l = lsum;
    });
    if (open && good) finish(true);
    where = 45;
  }
  if (!good && lane == 0 && !*abort_flag) {
    *abort_flag = 1;
    report_error(k.ws, CSA2_ERR_DEVICE_TIMEOUT, where);
  }
  if (warp == kAloneS || warp == kAloneO) {  // every MMA has completed before tensor memory is freed
    ptx::mma_commit_elect(&S.drained);
    volatile int keep_waiting = 0;
    ptx::mbar_wait_warp(&S.drained, 0, &keep_waiting, kWaitBudget);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kAloneS) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kCols);
  }
}

// The join over partials of the epilogue's order: a CTA has eight heads 8 g .. and all channels, thread t of it
// channel t; with four slices the 128 channels of a tile, and four CTAs (a cluster where the logsumexp wants all
// channels) make the heads.  The weights 2^(m_i - m) l_i / L are the same for all channels: the CTA forms them
// once, while the first partials' channels are on their way.  Without slices a query has few partials: four (fp32: two) at
// once, which leaves room for three CTAs on an SM (eight and two: paged ragged 128 x 2000 49.9 us, now 47.9).
constexpr int kMergeThreads = 512;
constexpr int kOneWave = 4;  // queries whose 32 CTAs each fit the GPU one to an SM
// Queries of trees, each by itself, below which slices join them, with two CTAs on an SM from five on.  A call without /
// with slices, us: 12 on 4,096 28.9 / 27.0, 16 30.6 / 30.0, 20 33.1 / 34.2, 32 on 3,000 35.2 / 39.4; with slices one CTA
// to an SM / two: eight on 4,096 23.8 / 22.3, normalised and rotated 29.1 / 25.2.
constexpr int kTreeSliceQueries = 17;
// kTwo: with slices, two CTAs on an SM, for which half as many partials are on their way.
template <int kSlices, bool kHalf, bool kTwo = false>
__global__ void __launch_bounds__(kMergeThreads, kSlices > 1 ? (kTwo ? 2 : 1) : 3) k_paged_merge(const int2* __restrict__ qpart,
                                                               const uint4* __restrict__ part_o,
                                                               const float2* __restrict__ part_ml,
                                                               const float* __restrict__ sink,
                                                               const float2* __restrict__ turn, void* __restrict__ out,
                                                               float* lse, LseRest fix) {
  constexpr int kAhead = kSlices > 1 ? (kTwo ? 4 : 8) : kHalf ? 4 : 2;  // partials on their way
  constexpr int kTiles = 4 / kSlices, kPer = 128 * kTiles;
  static_assert(kSlices == 1 || kTiles == 1, "all channels, or a tile of them");
  __shared__ __align__(16) float s_w[kAlone][8];  // read four at a time
  __shared__ float s_m[kAlone][8], s_dot[4 * kTiles][8], s_part[4][8];
  __shared__ float s_join[kSlices > 1 ? kSlices - 1 : 1][8][kSlices > 1 ? 128 : 1];
  if (kSlices > 1 && fix.rest) ptx::cluster_sync();  // the first CTA's shared memory is there
  ptx::griddep_wait();
  const int b = blockIdx.x, slice = threadIdx.x / kPer, t = threadIdx.x % kPer;
  const int tile = kSlices > 1 ? blockIdx.y & 3 : t >> 7, g = kSlices > 1 ? blockIdx.y >> 2 : blockIdx.y;
  const int h0 = 8 * g, c = kSlices > 1 ? 128 * tile + t : t;
  const int y = 8 * tile + g;  // the epilogue's vector, of its thread c % 128
  const int2 part = qpart[b];  // the first partial's slot, partials (at most one a CTA)
  for (int i = threadIdx.x; i < part.y * 8; i += kMergeThreads) {
    const float2 ml = part_ml[(int64_t)(part.x + i / 8) * kHAtt + h0 + i % 8];
    s_m[i / 8][i % 8] = ml.y == 0.0f ? -INFINITY : ml.x;
    s_w[i / 8][i % 8] = ml.y;
  }
  Vec8<kHalf> v[kAhead];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (k0 + j * kSlices < part.y)
        v[j].load(part_o + ((int64_t)(part.x + k0 + j * kSlices) * 32 + y) * Vec8<kHalf>::kWords * 128 + (t & 127));
  };
  fetch(slice);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < 8; i += kMergeThreads / 32) {  // a warp per head
    const float z = sink ? sink[h0 + i] * kLog2e : -INFINITY;
    float ref = z;
    for (int j = lane; j < part.y; j += 32) ref = fmaxf(ref, s_m[j][i]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    float L = 0.0f;
    for (int j = lane; j < part.y; j += 32) {
      const float w = s_w[j][i] == 0.0f ? 0.0f : ptx::ex2(s_m[j][i] - ref) * s_w[j][i];
      s_w[j][i] = w;
      L += w;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (z != -INFINITY) L += ptx::ex2(z - ref);
    const float inv = L > 0.0f ? 1.0f / (Vec8<kHalf>::kScale * L) : 0.0f;
    for (int j = lane; j < part.y; j += 32) s_w[j][i] *= inv;
    if (lse && (kSlices == 1 || tile == 0) && lane == 0)
      lse[b * kHAtt + h0 + i] = L == 0.0f ? -INFINITY : natural(ref, L);
  }
  __syncthreads();
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int k0 = slice; k0 < part.y; k0 += kSlices * kAhead) {
    if (k0 > slice) fetch(k0);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j * kSlices;
      if (k >= part.y) break;
      const float4 w0 = *reinterpret_cast<const float4*>(&s_w[k][0]), w1 = *reinterpret_cast<const float4*>(&s_w[k][4]);
      const float f[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      float x[8];
      v[j].get(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(f[i], x[i], acc[i]);
    }
  }
  if (kSlices > 1) {
    if (slice > 0)
#pragma unroll
      for (int i = 0; i < 8; ++i) s_join[slice - 1][i][t] = acc[i];
    __syncthreads();
    if (slice > 0) return;
#pragma unroll
    for (int j = 0; j < kSlices - 1; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += s_join[j][i][t];
  }
  if (fix.rest) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float e = __half2float(__ushort_as_half(fix.rest[((int64_t)b * kHAtt + h0 + i) * kDMain + c])) * acc[i];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
      if (lane == 0) s_dot[t >> 5][i] = e;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kPer) : "memory");
    if (t < 8) {
      float e = 0.0f;
      for (int i = 0; i < 4 * kTiles; ++i) e += s_dot[i][t];
      if (kSlices > 1) ptx::st_cluster_f32(&s_part[tile][t], 0, e);
      else lse[b * kHAtt + h0 + t] = corrected(fix, b, h0 + t, lse[b * kHAtt + h0 + t], e);
    }
  }
  const bool rotated = turn && c >= kRopeFirst;  // whole warps
  float cs = 1.0f, sn = 0.0f;
  if (rotated) {  // turn back by -q_pos: x' = x c + y s, y' = y c - x s, pairs in neighbouring lanes
    const float2 r = turn[(int64_t)b * 32 + (c - kRopeFirst) / 2];
    cs = r.x;
    sn = t & 1 ? -r.y : r.y;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float o = acc[i];
    if (rotated) {
      const float partner = __shfl_xor_sync(0xffffffffu, o, 1);
      o = fmaf(o, cs, partner * sn);
    }
    const int64_t at = ((int64_t)b * kHAtt + h0 + i) * kDMain + c;
    if (kHalf) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(o);
    else static_cast<float*>(out)[at] = o;
  }
  if (kSlices > 1 && fix.rest) {
    __syncwarp();
    ptx::cluster_sync();
    if (tile == 0 && t < 8)
      lse[b * kHAtt + h0 + t] = corrected(fix, b, h0 + t, lse[b * kHAtt + h0 + t],
                                          (s_part[0][t] + s_part[1][t]) + (s_part[2][t] + s_part[3][t]));
  }
}

// Parts of each pair of CTAs in a call for trees.  The pairs of CTAs work on neighbouring pairs of queries at a time, whose
// image L2 then holds: one part for every 64 MB of image at most.  One / two / three / four / six / eight parts, us of the
// attention: 4 trees of 64 on 65,000 (254 MB) 1,642 / 1,550 / 1,541 / 1,449 / 1,491 / 1,466, 48 of 32 on 4,001 (192 MB)
// 684 / 667 / 656 / 634 / 639 / 637, 16 of 16 on 8,192 (128 MB) 232 / 219 / 217 / 216 / 223 / 232, 48 of 16 on 2,000
// (96 MB) 200 / 192 / 193 / 198 / 199 / 210.  A part has sixteen chunks at least, by the bounds.
int tree_slices(int32_t B, int32_t G, int64_t n_max) {
  const int64_t image = cdiv(G * cdiv(n_max, kChunk), kSliceChunks), chunks = B * n_max / (2 * kChunk);
  return (int)std::max<int64_t>(1, std::min<int64_t>({8, image, chunks / (16 * kClusters)}));
}

struct PrefixWs {
  Pair* pairs;
  int32_t *gpair, *chunk0, *gimage;
  Part* parts;
  int2 *qpart, *gshared;
  uint16_t *image, *qimage, *rest;
  float* c2;
  float2* turn;
  int64_t image_cap;
  uint4* part_o;
  float2* part_ml;
  int32_t* cost0;
  uint64_t* kin;
  int32_t* depth;
  size_t bytes;
};

PrefixWs prefix_ws(void* ws, int32_t B, int32_t G, int64_t shared_max, bool trees = false) {
  PrefixWs L{};
  size_t off = kWsHeader;
  char* base = (char*)ws;
  auto take = [&](size_t n) {
    char* p = base ? base + off : nullptr;
    off += align_up(n, 256);
    return p;
  };
  // partials: of pairs cut by kClusters pairs of CTAs (two queries each), or of queries cut by kAlone CTAs
  const bool alone = trees ? trees_by_themselves(B, G, shared_max) : by_itself(B, G, shared_max);
  const size_t parts = alone ? kAlone : kClusters * (trees ? tree_slices(B, G, shared_max) : 1);
  const size_t pairs = alone ? B : max_pairs(B, G);
  const size_t slots = (pairs + parts) * (alone ? 1 : 2);
  L.pairs = (Pair*)take((pairs + 1) * sizeof(Pair));
  L.gpair = (int32_t*)take(((size_t)G + 3) * 4);
  L.chunk0 = (int32_t*)take((pairs + 1) * 4);
  L.qpart = (int2*)take((size_t)B * 8);
  L.parts = (Part*)take(parts * sizeof(Part));
  L.gimage = (int32_t*)take((size_t)G * 4);
  L.gshared = (int2*)take((size_t)G * 8);
  L.qimage = (uint16_t*)take(((size_t)B + 1) * kHAtt * kDMain * 2);
  L.c2 = (float*)take(((size_t)B + 1) * kHAtt * 4);
  L.rest = (uint16_t*)take((size_t)B * kHAtt * kDMain * 2);
  L.turn = (float2*)take((size_t)B * 32 * 8);
  L.part_o = (uint4*)take(slots * kHAtt * kDMain * 4);  // room for fp32: the output's type is not known here
  L.part_ml = (float2*)take(slots * kHAtt * 8);
  L.image_cap = alone ? 0 : G * cdiv(shared_max, kChunk);
  if (L.image_cap > kImageChunks) L.image_cap = kImageChunks;
  L.image = (uint16_t*)take((size_t)L.image_cap * kChunk * kDMain * 2);
  if (trees) {
    L.cost0 = (int32_t*)take((pairs + 1) * 4);
    L.kin = (uint64_t*)take((size_t)B * 8);
    L.depth = (int32_t*)take((size_t)B * 4);
  }
  L.bytes = off;
  return L;
}

// f16 image [chunks * 64 planes][128 rows][8 channels] as 32-bit words, boxes of `rows` rows x `planes`
bool image_map(CUtensorMap* map, uint16_t* image, int64_t chunks, uint32_t rows, uint32_t planes) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)kChunk * 4, (cuuint64_t)(chunks > 0 ? chunks : 1) * (kDMain / 8)};
  cuuint64_t strides[1] = {(cuuint64_t)kChunk * 16};
  cuuint32_t box[2] = {rows * 4, planes};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, image, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace csa2

extern "C" size_t csa2_prefix_attn_workspace_size(int32_t B, int32_t G, int64_t n_shared_max, int64_t n_own_max,
                                                  int32_t n_swa) {
  if (B <= 0 || B > 65535 || G <= 0 || G > B || n_shared_max < 0 || n_own_max < 0 || n_shared_max > CSA2_MAX_DENSE ||
      n_own_max > CSA2_MAX_DENSE || n_swa < 0)
    return 0;
  return csa2::prefix_ws(nullptr, B, G, n_shared_max).bytes;
}

namespace csa2 {
namespace {

// Page table of a call over B queries: rows long enough for n entries of each.
bool pages_ok(const csa2_pages* p, const csa2_kv_planes* kv, int64_t n) {
  if (!p || p->max_pages < 0 || p->n_pages < 0 || kv->seq_stride > INT32_MAX) return false;
  if (n > 0 && (!p->table || !aligned(p->table, 4))) return false;
  if ((int64_t)p->n_pages * kv->seq_stride > INT32_MAX) return false;  // plane rows are 32-bit
  return n <= (int64_t)p->max_pages * kv->seq_stride;
}

// The launches of a call: preparation, attention, join.
template <bool kTree>
csa2_status attn_call(const PrefixArgs& a, const PrefixKernel& k, const PrefixWs& L, const AttnExtras& ex, const void* q_bf16,
                      float softmax_scale, const float* sink, void* out, int32_t out_type, float* lse_out, cudaStream_t st) {
  const int32_t B = a.B;
  const bool alone = alone_of<kTree>(B, a.G, a.shared_max);
  // bf16 queries are exact in f16 unless they were normalised or rotated
  uint16_t* const rest = lse_out && (ex.qnorm_w || ex.rope) ? L.rest : nullptr;
  const PrefixQuery pq{(const uint16_t*)q_bf16, ex.qnorm_w, ex.eps, softmax_scale, ex.rope, ex.qpos, ex.th,
                       L.qimage, L.c2, L.turn, rest};
  const LseRest fix{rest, L.c2};
  ImageMaps maps{};
  if (L.image_cap > 0 &&
      (!image_map(&maps.s, L.image, L.image_cap, 64, 16) || !image_map(&maps.o, L.image, L.image_cap, 32, 32)))
    return CSA2_ERR_CUDA;
  const int slices = B < (kTree && alone ? kTreeSliceQueries : kSliceQueries) ? 4 : 1;
  const float2* turn = ex.rope ? L.turn : nullptr;
  auto merge = [&](auto kern, unsigned ctas, unsigned threads, unsigned cluster) {
    launch_clusters(kern, dim3(B, ctas), dim3(threads), 1, cluster, 0, st, (const int2*)L.qpart,
                    (const uint4*)L.part_o, (const float2*)L.part_ml, sink, turn, out, lse_out, fix);
  };
  auto run = [&](auto half) {  // parts in f16 for a bf16 output (Vec8)
    constexpr bool kHalf = decltype(half)::value;
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const auto prep = k_prefix_prep<kTree>;
    if (cudaFuncSetAttribute(prep, attr, kPrepSmem) != cudaSuccess ||
        (alone ? cudaFuncSetAttribute(k_paged_attn<kHalf, kTree>, attr, (int)sizeof(AloneSmem))
               : cudaFuncSetAttribute(k_prefix_attn<kHalf, kTree>, attr, (int)sizeof(PrefixSmem))) != cudaSuccess)
      return launch_status();
    {
      KernelTimer timer("k_prefix_prep", st);
      const int trees = kTree ? (a.G + kTreesPerCta - 1) / kTreesPerCta : 0;
      const int widen = (int)(L.image_cap < kWidenCtas ? L.image_cap : kWidenCtas);
      // without its plan the attention would run whatever one the workspace held, and the join its parts
      const int stage = kTree ? std::min(kStageCtas * (B + 1), kStageMost) : kStageCtas * (B + 1);
      if (launch_pdl(prep, dim3((unsigned)(1 + trees + stage + widen)), dim3(kPrepThreads),
                     (size_t)kPrepSmem, st, a, pq, k, L.image) != cudaSuccess)
        return launch_status();
    }
    if (alone) {
      {
        KernelTimer timer("k_paged_attn", st);
        if (launch_pdl(k_paged_attn<kHalf, kTree>, dim3(kAlone), dim3(kThreads), sizeof(AloneSmem), st, k) != cudaSuccess)
          return launch_status();
      }
      KernelTimer timer("k_paged_merge", st);
      if (kTree && slices > 1 && B > kOneWave) merge(k_paged_merge<4, kHalf, true>, 32, kMergeThreads, rest ? 4 : 1);
      else if (slices > 1) merge(k_paged_merge<4, kHalf>, 32, kMergeThreads, rest ? 4 : 1);
      else merge(k_paged_merge<1, kHalf>, 8, kMergeThreads, 1);
      return launch_status();
    }
    {
      KernelTimer timer("k_prefix_attn", st);
      if (launch_clusters(k_prefix_attn<kHalf, kTree>, dim3(2 * kClusters), dim3(kThreads), 2, 1, sizeof(PrefixSmem), st, k,
                          maps) != cudaSuccess)
        return launch_status();
    }
    KernelTimer timer("k_prefix_merge", st);
    // with slices the forms are the same
    if (slices > 1) merge(k_prefix_merge<4, kHalf, false>, 32, PrefixMerge<4, kHalf, false>::kThreads, 1);
    else merge(k_prefix_merge<1, kHalf, kTree>, 8, PrefixMerge<1, kHalf, kTree>::kThreads, 1);
    return launch_status();
  };
  return out_type == CSA2_OUT_BF16 ? run(std::true_type{}) : run(std::false_type{});
}

// Attention of B queries through page tables, G groups of them sharing prefixes (G = 0: none).
csa2_status prefix_run(const csa2_kv_planes* kv, const csa2_pages* pages, int32_t B, const int32_t* n_entries, int32_t G,
                       const int32_t* group_start, const int32_t* n_shared, int64_t n_shared_max, int64_t n_own_max,
                       const uint8_t* swa_e4m3, int32_t n_swa, const void* q_bf16, float softmax_scale,
                       const csa2_norm_rope* q_nr, const int64_t* q_pos, const float* sink, const csa2_window* win,
                       void* out, int32_t out_type, float* lse_out, void* ws, size_t ws_bytes, csa2_stream stream) {
  if (!n_entries || !aligned(n_entries, 4) || (n_swa > 0 && !swa_e4m3) || !q_bf16 || !out || !aligned(q_bf16, 16) ||
      !aligned(out, 16) || (swa_e4m3 && !aligned(swa_e4m3, 16)) || (lse_out && !aligned(lse_out, 4)))
    return CSA2_ERR_INVALID_ARG;
  if (out_type != CSA2_OUT_F32 && out_type != CSA2_OUT_BF16) return CSA2_ERR_INVALID_ARG;
  AttnExtras ex;
  const csa2_status bad = attn_extras(q_nr, q_pos, sink, win, n_swa, softmax_scale, &ex);
  if (bad != CSA2_OK) return bad;
  if (!ws || !aligned(ws, 256)) return CSA2_ERR_WORKSPACE;
  const bool alone = by_itself(B, G, n_shared_max);
  const PrefixWs L = prefix_ws(ws, B, G, n_shared_max);
  if (ws_bytes < L.bytes) return CSA2_ERR_WORKSPACE;
  const PrefixArgs a{B, G, n_entries, group_start, n_shared, (int32_t)n_shared_max, (int32_t)n_own_max, n_swa,
                     (int64_t)pages->max_pages * kv->seq_stride, L.pairs, L.gpair, L.chunk0, L.qpart, L.parts,
                     L.gimage, L.gshared, L.image_cap, alone ? kAlone : kClusters, ws, nullptr, 0, 0, nullptr, nullptr,
                     nullptr};
  const PrefixKernel k{kv->kv_codes, kv->kv_scales, swa_e4m3, L.qimage, L.c2, pages->table,
                       pages->max_pages, pages->n_pages, (int32_t)kv->seq_stride, n_swa, B,
                       ((1ull << 40) + kv->seq_stride - 1) / kv->seq_stride, ex.win_pos, ex.win_lo,
                       L.pairs, L.parts, nullptr, nullptr, nullptr, nullptr, 0, 1, L.part_o, L.part_ml, ws};
  return attn_call<false>(a, k, L, ex, q_bf16, softmax_scale, sink, out, out_type, lse_out, (cudaStream_t)stream);
}

}  // namespace
}  // namespace csa2

extern "C" size_t csa2_paged_attn_workspace_size(int32_t B, int64_t n_max, int32_t n_swa) {
  if (B <= 0 || B > 65535 || n_max < 0 || n_max > CSA2_MAX_DENSE || n_swa < 0) return 0;
  return csa2::prefix_ws(nullptr, B, 0, 0).bytes;
}

extern "C" csa2_status csa2_paged_attn_decode(const csa2_kv_planes* kv, const csa2_pages* pages, int32_t B,
                                              const int32_t* n_entries, int64_t n_max, const uint8_t* swa_e4m3,
                                              int32_t n_swa, const void* q_bf16, float softmax_scale,
                                              const csa2_norm_rope* q_nr, const int64_t* q_pos, const float* sink,
                                              const csa2_window* win, void* out, int32_t out_type, float* lse_out,
                                              void* ws, size_t ws_bytes, csa2_stream stream) {
  using namespace csa2;
  if (!planes_ok(kv) || B <= 0 || B > 65535 || n_max < 0 || n_max > CSA2_MAX_DENSE || n_swa < 0 ||
      n_swa > CSA2_MAX_SWA || !pages_ok(pages, kv, n_max))
    return CSA2_ERR_INVALID_ARG;
  return prefix_run(kv, pages, B, n_entries, 0, nullptr, nullptr, 0, n_max, swa_e4m3, n_swa, q_bf16, softmax_scale, q_nr,
                    q_pos, sink, win, out, out_type, lse_out, ws, ws_bytes, stream);
}

extern "C" csa2_status csa2_prefix_attn_decode(const csa2_kv_planes* kv, const csa2_pages* pages, int32_t B,
                                               const int32_t* n_entries, int32_t G, const int32_t* group_start,
                                               const int32_t* n_shared, int64_t n_shared_max, int64_t n_own_max,
                                               const uint8_t* swa_e4m3, int32_t n_swa, const void* q_bf16,
                                               float softmax_scale, const csa2_norm_rope* q_nr, const int64_t* q_pos,
                                               const float* sink, const csa2_window* win, void* out, int32_t out_type,
                                               float* lse_out, void* ws, size_t ws_bytes, csa2_stream stream) {
  using namespace csa2;
  if (!planes_ok(kv) || B <= 0 || B > 65535 || G <= 0 || G > B || n_shared_max < 0 || n_own_max < 0 ||
      n_shared_max > CSA2_MAX_DENSE || n_own_max > CSA2_MAX_DENSE || n_swa < 0 || n_swa > CSA2_MAX_SWA ||
      !pages_ok(pages, kv, n_shared_max) || !pages_ok(pages, kv, n_own_max))
    return CSA2_ERR_INVALID_ARG;
  if (!group_start || !n_shared || !aligned(group_start, 4) || !aligned(n_shared, 4)) return CSA2_ERR_INVALID_ARG;
  return prefix_run(kv, pages, B, n_entries, G, group_start, n_shared, n_shared_max, n_own_max, swa_e4m3, n_swa, q_bf16,
                    softmax_scale, q_nr, q_pos, sink, win, out, out_type, lse_out, ws, ws_bytes, stream);
}

extern "C" size_t csa2_tree_attn_workspace_size(int32_t R, int32_t B, int32_t max_tokens, int64_t n_max, int32_t n_swa) {
  if (R <= 0 || R > 65535 || B <= 0 || B > 65535 || max_tokens < 1 || max_tokens > CSA2_MAX_TREE || n_max < 0 ||
      n_max > CSA2_MAX_DENSE || n_swa < 0)
    return 0;
  return csa2::prefix_ws(nullptr, B, R, n_max, true).bytes;
}

extern "C" csa2_status csa2_tree_attn_decode(const csa2_kv_planes* kv, const csa2_pages* pages, const csa2_trees* trees,
                                             const int32_t* n_entries, int64_t n_max, const uint8_t* swa_e4m3,
                                             const int64_t* swa_pos, const uint8_t* draft_e4m3, int32_t n_swa,
                                             const void* q_bf16, const int64_t* q_pos, float softmax_scale,
                                             const csa2_norm_rope* q_nr, const csa2_rope_scaling* scaling,
                                             const float* sink, void* out, int32_t out_type, float* lse_out, void* ws,
                                             size_t ws_bytes, csa2_stream stream) {
  using namespace csa2;
  if (!trees || !trees->start || !trees->parent || !aligned(trees->start, 4) || !aligned(trees->parent, 4) ||
      trees->R <= 0 || trees->R > 65535 || trees->B <= 0 || trees->B > 65535 || trees->max_tokens < 1 ||
      trees->max_tokens > CSA2_MAX_TREE)
    return CSA2_ERR_INVALID_ARG;
  const int32_t R = trees->R, B = trees->B;
  if (!planes_ok(kv) || n_max < 0 || n_max > CSA2_MAX_DENSE || n_swa < 0 || n_swa > CSA2_MAX_SWA ||
      !pages_ok(pages, kv, n_max + (trees->entries ? trees->max_tokens : 0)) ||
      (int64_t)pages->n_pages * kv->seq_stride > 1 << 30)
    return CSA2_ERR_INVALID_ARG;
  if (!n_entries || !aligned(n_entries, 4) || !q_bf16 || !out || !aligned(q_bf16, 16) || !aligned(out, 16) ||
      (lse_out && !aligned(lse_out, 4)) || (out_type != CSA2_OUT_F32 && out_type != CSA2_OUT_BF16))
    return CSA2_ERR_INVALID_ARG;
  if (n_swa > 0 && (!swa_e4m3 || !swa_pos || !draft_e4m3 || !q_pos || !aligned(swa_e4m3, 16) || !aligned(swa_pos, 8) ||
                    !aligned(draft_e4m3, 16)))
    return CSA2_ERR_INVALID_ARG;
  if (!scaling_ok(scaling)) return CSA2_ERR_INVALID_ARG;
  AttnExtras ex;
  const csa2_status bad = attn_extras(q_nr, q_pos, sink, nullptr, n_swa, softmax_scale, &ex);
  if (bad != CSA2_OK) return bad;
  if (ex.rope) make_thetas(ex.th.t, 64, q_nr->rope_base, scaling);
  if (!ws || !aligned(ws, 256)) return CSA2_ERR_WORKSPACE;
  const PrefixWs L = prefix_ws(ws, B, R, n_max, true);
  if (ws_bytes < L.bytes) return CSA2_ERR_WORKSPACE;
  const int slices = tree_slices(B, R, n_max);
  const PrefixArgs a{B, R, n_entries, trees->start, nullptr, (int32_t)n_max, 0, n_swa,
                     (int64_t)pages->max_pages * kv->seq_stride, L.pairs, L.gpair, L.chunk0, L.qpart, L.parts,
                     L.gimage, L.gshared, L.image_cap, trees_by_themselves(B, R, n_max) ? kAlone : kClusters * slices, ws,
                     trees->parent, trees->max_tokens, trees->entries, L.cost0, L.kin, L.depth};
  const PrefixKernel k{kv->kv_codes, kv->kv_scales, swa_e4m3, L.qimage, L.c2, pages->table,
                       pages->max_pages, pages->n_pages, (int32_t)kv->seq_stride, n_swa, B,
                       ((1ull << 40) + kv->seq_stride - 1) / kv->seq_stride, swa_pos, nullptr,
                       L.pairs, L.parts, L.kin, L.depth, n_swa > 0 ? q_pos : nullptr, draft_e4m3, R * n_swa, slices,
                       L.part_o, L.part_ml, ws};
  return attn_call<true>(a, k, L, ex, q_bf16, softmax_scale, sink, out, out_type, lse_out, (cudaStream_t)stream);
}
