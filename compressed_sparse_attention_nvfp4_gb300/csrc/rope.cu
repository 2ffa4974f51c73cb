// Rotary positions by themselves: y[r][h] = x[r][h] with n_rot channels turned by pos[r] (csa2_rope).
//
// Bytes bound it: x is read once and y written once, 3 flops a rotated channel.  A CTA takes a tile of rows and
// heads and forms its cosines and sines once (a row's serve all its heads) in shared memory.  A vector's units are
// its rotated ones, two vectors of kV channels whose kV pairs turn (HALVES: pair k is the k-th channel of the two;
// INTERLEAVED: the neighbouring channels of each), and its copied ones, one vector each.  Threads take units of one kind
// at a time: with both kinds in a warp every warp runs both (32,768 x 32 queries 120 us).  Measured: 32,768 x 32 bf16
// queries of 128 channels, half of them rotated, 82 us, 6.6 TB/s, in fp32 153, 7.0 TB/s; 128 x 32 2.3 us from a graph.
// Where an address, a stride or a number of pairs is no multiple of 16 bytes all units are of one channel: with gaps of 7
// or 4 channels between the rows 271 us (fp32, 7: 273), with 20 pairs 354 (fp32, 18: 362).
#include <algorithm>

#include "ptx.cuh"
#include "rotary.cuh"
#include "timing.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 2;              // units of a kind that a thread has on their way
// Units of a tile, of the kind of which it has more: at most, and at least where the call has them.  512 / 1,024 /
// 1,536 / 2,048 at most, us: 32,768 x 32 queries of 128 channels 87 / 82 / 83 / 84, 16,385 rows of 512 in fp32 17.1 /
// 14.4 / 15.8 / 15.8 (four on their way in three CTAs an SM instead of two in four: 82 and 14.5 at 2,048).
constexpr int kUnits = 4 * kThreads, kFewUnits = 256;
constexpr int kTiles = 608;            // tiles that fill the GPU: four on an SM
constexpr int kTable = 4096;           // cosines of a tile, at most

struct RopeArgs {
  const void* x;
  void* y;
  int64_t x_row, x_head, y_row, y_head;
  const int64_t* pos;
  int64_t n_rows;
  int32_t heads, first, pairs;
  int32_t rot, copies;        // units of a vector
  int32_t rows_of, heads_of;  // of a tile
  float magnitude, sign;
  uint32_t by_heads, by_pairs, by_rot, by_copies;  // reciprocals (see over)
};

// i / d for i, d <= 2^16, by a product with r = ceil(2^32 / d); d = 1 has none
__host__ __device__ __forceinline__ uint32_t reciprocal(uint32_t d) {
  return d > 1 ? (uint32_t)(((1ull << 32) + d - 1) / d) : 0;
}
__device__ __forceinline__ int over(int i, uint32_t r) { return r ? (int)__umulhi((uint32_t)i, r) : i; }

template <typename T, int kV>
struct __align__(sizeof(T) * kV) Vec {
  T v[kV];
};
// kV pairs of two vectors, turned; t: their cosines and sines
template <bool kHalves, typename T, int kV>
struct Turn {
  static __device__ __forceinline__ void run(Vec<T, kV>& p, Vec<T, kV>& q, const float2* t) {
    static_assert(sizeof(T) == 4 || kV == 1, "see the other form");
    constexpr bool kApart = kHalves || kV == 1;
    const Vec<T, kV> x = p, y = q;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const float2 cs = t[k];
      const float m = (float)(kApart ? x.v[k] : 2 * k < kV ? x.v[2 * k] : y.v[2 * k - kV]);
      const float n = (float)(kApart ? y.v[k] : 2 * k < kV ? x.v[2 * k + 1] : y.v[2 * k + 1 - kV]);
      T& g = kApart ? p.v[k] : 2 * k < kV ? p.v[2 * k] : q.v[2 * k - kV];
      T& h = kApart ? q.v[k] : 2 * k < kV ? p.v[2 * k + 1] : q.v[2 * k + 1 - kV];
      g = (T)(m * cs.x - n * cs.y);
      h = (T)(m * cs.y + n * cs.x);
    }
  }
};
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool kHalves>
struct Turn<kHalves, __nv_bfloat16, 8> {  // two channels to a word
  static __device__ __forceinline__ void run(Vec<__nv_bfloat16, 8>& p, Vec<__nv_bfloat16, 8>& q, const float2* t) {
    uint32_t* const a = reinterpret_cast<uint32_t*>(&p);
    uint32_t* const b = reinterpret_cast<uint32_t*>(&q);
    const float4* const t2 = reinterpret_cast<const float4*>(t);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float4 cs = t2[w];  // pairs 2 w, 2 w + 1
      if (kHalves) {
        const float m0 = low(a[w]), m1 = high(a[w]), n0 = low(b[w]), n1 = high(b[w]);
        a[w] = pack(m0 * cs.x - n0 * cs.y, m1 * cs.z - n1 * cs.w);
        b[w] = pack(m0 * cs.y + n0 * cs.x, m1 * cs.w + n1 * cs.z);
      } else {
        uint32_t* const c = w < 2 ? a + 2 * w : b + 2 * w - 4;
        const float m0 = low(c[0]), n0 = high(c[0]), m1 = low(c[1]), n1 = high(c[1]);
        c[0] = pack(m0 * cs.x - n0 * cs.y, m0 * cs.y + n0 * cs.x);
        c[1] = pack(m1 * cs.z - n1 * cs.w, m1 * cs.w + n1 * cs.z);
      }
    }
  }
};

template <typename T, int kV, bool kHalves, int kPairs>
__global__ void __launch_bounds__(kThreads, 4) k_rope(RopeArgs a, const __grid_constant__ Turns<kPairs> turns) {
  extern __shared__ __align__(16) float2 table[];  // [rows][pairs] cosine, sine
  using V = Vec<T, kV>;
  ptx::griddep_launch();
  ptx::griddep_wait();
  const int64_t row0 = (int64_t)blockIdx.x * a.rows_of;
  const int head0 = blockIdx.y * a.heads_of;
  const int rows = (int)min((int64_t)a.rows_of, a.n_rows - row0), heads = min(a.heads_of, a.heads - head0);
  const T* const x = static_cast<const T*>(a.x) + row0 * a.x_row + head0 * a.x_head;
  T* const y = static_cast<T*>(a.y) + row0 * a.y_row + head0 * a.y_head;
  const int vectors = rows * a.heads_of, turned = vectors * a.rot, copied = vectors * a.copies;
  const int second = kHalves ? a.pairs : kV;
  // vector v = row v / heads, its head; -1: there is none
  auto row_of = [&](int v, int& h) {
    const int r = over(v, a.by_heads);
    h = v - r * a.heads_of;
    return v < vectors && h < heads ? r : -1;
  };
  V p[kBatch], q[kBatch];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kThreads, v = over(i, a.by_rot), u = i - v * a.rot;
      int h;
      const int r = row_of(v, h);
      if (r < 0) continue;
      const T* const xs = x + r * a.x_row + h * a.x_head + a.first + (kHalves ? u * kV : 2 * u * kV);
      p[j] = *reinterpret_cast<const V*>(xs);
      q[j] = *reinterpret_cast<const V*>(xs + second);
    }
  };
  if ((int)threadIdx.x < turned) fetch(threadIdx.x);
  for (int i0 = threadIdx.x; i0 < copied; i0 += kBatch * kThreads) {
    V w[kBatch];
    T* to[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kThreads, v = over(i, a.by_copies);
      int h, c = (i - v * a.copies) * kV;
      const int r = row_of(v, h);
      to[j] = nullptr;
      if (r < 0) continue;
      if (c >= a.first) c += 2 * a.pairs;
      w[j] = *reinterpret_cast<const V*>(x + r * a.x_row + h * a.x_head + c);
      to[j] = y + r * a.y_row + h * a.y_head + c;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (to[j]) *reinterpret_cast<V*>(to[j]) = w[j];
  }
  for (int i = threadIdx.x; i < rows * a.pairs; i += kThreads) {
    const int r = over(i, a.by_pairs);
    float c, s;
    turn_cos_sin(turns.f[i - r * a.pairs], a.pos[row0 + r], c, s);
    table[i] = make_float2(a.magnitude * c, a.sign * a.magnitude * s);
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < turned; i0 += kBatch * kThreads) {
    if (i0 >= kBatch * kThreads) fetch(i0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kThreads, v = over(i, a.by_rot), u = i - v * a.rot;
      int h;
      const int r = row_of(v, h);
      if (r < 0) continue;
      Turn<kHalves, T, kV>::run(p[j], q[j], table + r * a.pairs + u * kV);
      T* const ys = y + r * a.y_row + h * a.y_head + a.first + (kHalves ? u * kV : 2 * u * kV);
      *reinterpret_cast<V*>(ys) = p[j];
      *reinterpret_cast<V*>(ys + second) = q[j];
    }
  }
}

template <typename T, int kV, int kPairs>
csa2_status run(RopeArgs a, const csa2_rotary* rot, int32_t dim, cudaStream_t st) {
  Turns<kPairs> turns;
  make_turns(&turns, rot->n_rot, rot->base, &rot->scaling);
  a.rot = a.pairs / kV;
  a.copies = a.x == a.y ? 0 : (dim - rot->n_rot) / kV;
  // units of the kind that is more; over() wants fewer than 2^16
  const int per = std::max(a.rot, a.copies);
  const int64_t all = (int64_t)per * a.heads;
  const int64_t want = std::min<int64_t>(std::max<int64_t>(all * a.n_rows / kTiles, kFewUnits), kUnits);
  a.rows_of = (int)std::min<int64_t>({std::max<int64_t>(want / all, 1), kTable / a.pairs, a.n_rows});
  a.heads_of = (int)std::min<int64_t>(std::max<int64_t>(want / per, 1), a.heads);
  a.by_heads = reciprocal(a.heads_of);
  a.by_pairs = reciprocal(a.pairs);
  a.by_rot = reciprocal(a.rot);
  a.by_copies = reciprocal(a.copies);
  KernelTimer timer("k_rope", st);
  launch_pdl(rot->layout == CSA2_ROPE_HALVES ? k_rope<T, kV, true, kPairs> : k_rope<T, kV, false, kPairs>,
             dim3((unsigned)cdiv(a.n_rows, a.rows_of), (unsigned)cdiv(a.heads, a.heads_of)), dim3(kThreads),
             (size_t)a.rows_of * a.pairs * sizeof(float2), st, a, turns);
  return launch_status();
}
// the angles are the launch's parameters: few of them make it shorter
template <typename T, int kV>
csa2_status run(const RopeArgs& a, const csa2_rotary* rot, int32_t dim, cudaStream_t st) {
  return a.pairs <= 32 ? run<T, kV, 32>(a, rot, dim, st) : run<T, kV, kMaxPairs>(a, rot, dim, st);
}

}  // namespace
}  // namespace csa2

extern "C" csa2_status csa2_rope(const void* x, int64_t x_row, int64_t x_head, void* y, int64_t y_row, int64_t y_head,
                                 int32_t type, int64_t n_rows, int32_t heads, int32_t dim, const int64_t* pos,
                                 const csa2_rotary* rot, int32_t inverse, csa2_stream stream) {
  using namespace csa2;
  if (type != CSA2_F32 && type != CSA2_BF16) return CSA2_ERR_INVALID_ARG;
  if (n_rows < 0 || n_rows > INT32_MAX || heads < 1 || heads > 65535 || dim < 1 || dim > 65536)
    return CSA2_ERR_INVALID_ARG;
  if (!rot || !rotary_ok(rot, dim)) return CSA2_ERR_INVALID_ARG;
  if (n_rows == 0) return CSA2_OK;
  const size_t size = type == CSA2_F32 ? 4 : 2;
  if (!x || !y || !pos || !aligned(x, size) || !aligned(y, size) || !aligned(pos, 8)) return CSA2_ERR_INVALID_ARG;
  if (x == y) {
    if ((n_rows > 1 && x_row != y_row) || (heads > 1 && x_head != y_head)) return CSA2_ERR_INVALID_ARG;
  }
  // the vectors of y lie behind one another, rows of heads or heads of rows
  constexpr int64_t kMost = INT64_MAX >> 20;  // strides whose products stay within 64 bits
  if (x_row > kMost >> 12 || x_row < -(kMost >> 12) || x_head > kMost || x_head < -kMost || y_row > kMost >> 12 ||
      y_head > kMost)
    return CSA2_ERR_INVALID_ARG;
  const int64_t row_of = (heads > 1 ? (heads - 1) * y_head : 0) + dim;
  const int64_t head_of = (n_rows > 1 ? (n_rows - 1) * y_row : 0) + dim;
  const bool by_row = (heads == 1 || y_head >= dim) && (n_rows == 1 || y_row >= row_of);
  const bool by_head = (n_rows == 1 || y_row >= dim) && (heads == 1 || y_head >= head_of);
  if (!by_row && !by_head) return CSA2_ERR_INVALID_ARG;
  const int64_t v = 16 / (int64_t)size;
  const bool wide = aligned(x, 16) && aligned(y, 16) && rot->first % v == 0 && rot->n_rot / 2 % v == 0 && dim % v == 0 &&
                    (n_rows == 1 || (x_row % v == 0 && y_row % v == 0)) &&
                    (heads == 1 || (x_head % v == 0 && y_head % v == 0));
  RopeArgs a{};
  a.x = x;
  a.y = y;
  a.x_row = x_row;
  a.x_head = x_head;
  a.y_row = y_row;
  a.y_head = y_head;
  a.pos = pos;
  a.n_rows = n_rows;
  a.heads = heads;
  a.first = rot->first;
  a.pairs = rot->n_rot / 2;
  a.magnitude = rot->magnitude;
  a.sign = inverse ? -1.0f : 1.0f;
  cudaStream_t st = (cudaStream_t)stream;
  if (type == CSA2_F32) return wide ? run<float, 4>(a, rot, dim, st) : run<float, 1>(a, rot, dim, st);
  return wide ? run<__nv_bfloat16, 8>(a, rot, dim, st) : run<__nv_bfloat16, 1>(a, rot, dim, st);
}
