// Rotary positions by themselves: y[r][h] = x[r][h] with n_rot channels turned by pos[r] (csa2_rope).
//
// Bytes bound it: x is read once and y written once, 3 flops a rotated channel.  A CTA takes a tile of rows and
// heads and forms its cosines and sines once (a row's serve all its heads) in shared memory.  A vector's units are
// its rotated ones, two vectors of kV channels whose kV pairs turn (HALVES: pair k is the k-th channel of the two;
// INTERLEAVED: the neighbouring channels of each), and its copied ones, one vector each; a thread has one unit of every
// so many vectors, so that a warp's loads are contiguous and its loop divides once a vector.
#include <algorithm>

#include "ptx.cuh"
#include "rotary.cuh"
#include "timing.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2048, kFewUnits = 512;  // of a tile, at most (about) and at least
constexpr int kTiles = 608;                    // tiles a call is cut into where it has that many units: four on an SM
constexpr int kTable = 4096;                   // cosines of a tile, at most
constexpr int kBatch = 2;                      // units a thread has on their way

struct RopeArgs {
  const void* x;
  void* y;
  int64_t x_row, x_head, y_row, y_head;
  const int64_t* pos;
  int64_t n_rows;
  int32_t heads, first, pairs;
  int32_t rot, copies;        // units of a vector
  int32_t rows_of, heads_of;  // of a tile
  int32_t lanes;              // vectors that a CTA's threads work on at once
  float magnitude, sign;
  uint32_t by_heads, by_pairs;  // reciprocals (see over)
};

// i / d for i, d <= 2^16, by a product with r = ceil(2^32 / d); d = 1 has none
__host__ __device__ __forceinline__ uint32_t reciprocal(uint32_t d) { return d > 1 ? (uint32_t)(((1ull << 32) + d - 1) / d) : 0; }
__device__ __forceinline__ int over(int i, uint32_t r) { return r ? (int)__umulhi((uint32_t)i, r) : i; }

template <typename T, int kV>
struct __align__(sizeof(T) * kV) Vec {
  T v[kV];
};
__device__ __forceinline__ float load(float x) { return x; }
__device__ __forceinline__ float load(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float& y, float x) { y = x; }
__device__ __forceinline__ void store(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

template <typename T, int kV, bool kHalves, int kPairs>
__global__ void __launch_bounds__(kThreads, 4) k_rope(RopeArgs a, const __grid_constant__ Turns<kPairs> turns) {
  extern __shared__ float2 table[];  // [rows][pairs] cosine, sine
  ptx::griddep_launch();
  ptx::griddep_wait();
  const int64_t row0 = (int64_t)blockIdx.x * a.rows_of;
  const int head0 = blockIdx.y * a.heads_of;
  const int rows = (int)min((int64_t)a.rows_of, a.n_rows - row0), heads = min(a.heads_of, a.heads - head0);
  const T* const x = static_cast<const T*>(a.x) + row0 * a.x_row + head0 * a.x_head;
  T* const y = static_cast<T*>(a.y) + row0 * a.y_row + head0 * a.y_head;
  for (int i = threadIdx.x; i < rows * a.pairs; i += blockDim.x) {
    const int r = over(i, a.by_pairs);
    float c, s;
    turn_cos_sin(turns.f[i - r * a.pairs], a.pos[row0 + r], c, s);
    table[i] = make_float2(a.magnitude * c, a.sign * a.magnitude * s);
  }
  __syncthreads();
  const int per = a.rot + a.copies, vectors = rows * a.heads_of;
  const int lane = a.lanes > 1 ? threadIdx.x / per : 0;
  if (lane >= a.lanes) return;
  for (int u = threadIdx.x - lane * per; u < per; u += a.lanes > 1 ? per : blockDim.x) {
    const bool turned = u < a.rot;
    int c0 = a.first + (kHalves ? u * kV : 2 * u * kV), c1 = c0 + (kHalves ? a.pairs : kV);
    if (!turned) {
      c0 = (u - a.rot) * kV;
      if (c0 >= a.first) c0 += 2 * a.pairs;
    }
    for (int v0 = lane; v0 < vectors; v0 += kBatch * a.lanes) {
      Vec<T, kV> p[kBatch], q[kBatch];
      int r[kBatch], h[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int v = v0 + j * a.lanes;
        r[j] = over(v, a.by_heads);
        h[j] = v - r[j] * a.heads_of;
        if (v >= vectors) h[j] = heads;
        if (h[j] >= heads) continue;
        const T* const xs = x + r[j] * a.x_row + h[j] * a.x_head;
        p[j] = *reinterpret_cast<const Vec<T, kV>*>(xs + c0);
        if (turned) q[j] = *reinterpret_cast<const Vec<T, kV>*>(xs + c1);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (h[j] >= heads) continue;
        T* const ys = y + r[j] * a.y_row + h[j] * a.y_head;
        if (turned) {
          const float2* const t = table + r[j] * a.pairs + u * kV;
          Vec<T, kV> o0, o1;
#pragma unroll
          for (int k = 0; k < kV; ++k) {
            constexpr bool kApart = kHalves || kV == 1;
            const float m = load(kApart ? p[j].v[k] : 2 * k < kV ? p[j].v[2 * k] : q[j].v[2 * k - kV]);
            const float n = load(kApart ? q[j].v[k] : 2 * k < kV ? p[j].v[2 * k + 1] : q[j].v[2 * k + 1 - kV]);
            const float2 cs = t[k];
            store(kApart ? o0.v[k] : 2 * k < kV ? o0.v[2 * k] : o1.v[2 * k - kV], m * cs.x - n * cs.y);
            store(kApart ? o1.v[k] : 2 * k < kV ? o0.v[2 * k + 1] : o1.v[2 * k + 1 - kV], m * cs.y + n * cs.x);
          }
          *reinterpret_cast<Vec<T, kV>*>(ys + c0) = o0;
          *reinterpret_cast<Vec<T, kV>*>(ys + c1) = o1;
        } else {
          *reinterpret_cast<Vec<T, kV>*>(ys + c0) = p[j];
        }
      }
    }
  }
}

template <typename T, int kV, int kPairs>
csa2_status run(RopeArgs a, const csa2_rotary* rot, int32_t dim, cudaStream_t st) {
  Turns<kPairs> turns;
  make_turns(&turns, rot->n_rot, rot->base, &rot->scaling);
  a.rot = a.pairs / kV;
  a.copies = a.x == a.y ? 0 : (dim - rot->n_rot) / kV;
  const int per = a.rot + a.copies;
  const int64_t all = (int64_t)per * a.heads;
  const int64_t want = std::min<int64_t>(std::max<int64_t>(all * a.n_rows / kTiles, kFewUnits), kUnits);
  a.rows_of = (int)std::min<int64_t>({std::max<int64_t>(want / all, 1), kTable / a.pairs, a.n_rows});
  a.heads_of = (int)std::min<int64_t>(std::max<int64_t>(want / per, 1), a.heads);
  a.lanes = std::max(kThreads / per, 1);
  a.by_heads = reciprocal(a.heads_of);
  a.by_pairs = reciprocal(a.pairs);
  const int threads = per >= kThreads ? kThreads : (a.lanes * per + 31) / 32 * 32;
  KernelTimer timer("k_rope", st);
  launch_pdl(rot->layout == CSA2_ROPE_HALVES ? k_rope<T, kV, true, kPairs> : k_rope<T, kV, false, kPairs>,
             dim3((unsigned)cdiv(a.n_rows, a.rows_of), (unsigned)cdiv(a.heads, a.heads_of)), dim3(threads),
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
  const bool by_row = (heads == 1 || y_head >= dim) && (n_rows == 1 || y_row >= (heads - 1) * (heads > 1 ? y_head : 0) + dim);
  const bool by_head = (n_rows == 1 || y_row >= dim) && (heads == 1 || y_head >= (n_rows - 1) * (n_rows > 1 ? y_row : 0) + dim);
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
