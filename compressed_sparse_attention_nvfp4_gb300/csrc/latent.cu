// Append of ready latents to slots or pages, normalised and rotated on the way (csa2_latent_append).
//
// Row r's main copy: y = w x / sqrt(mean(x^2) + eps), the last 64 channels turned by pos, rounded to fp32 once, then
// the cache's codec; its indexer key: turned by pos, then the codec.  The codec's borders make the bytes depend on the
// last bits of y: with y formed in fp32, off by a few 2^-24, one code in five million falls to the other side, several
// in a prefill chunk; formed in pairs of fp32 (rotary.cuh), off by 2^-36, the bytes are those of the definition.
//
// A warp takes a row: lane l holds the channels 16 l .. (a quantization group), and for the rotation pair l of the
// last 64, which lanes 28-31 get back through shared memory; of the key, channels 4 l ...  Bytes bound a long
// call: up to 2,560 read and 356 written a row.
#include "codec.cuh"
#include "ptx.cuh"
#include "rotary.cuh"
#include "timing.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
// CTAs that look at the destinations: a cluster, so that none reports before the word is cleared; one for few rows
constexpr int kCheckers = 8, kManyRows = 4096;

struct LatentArgs {
  const void *x, *key;
  int32_t R, n_slots, checkers;
  const int32_t* slot;
  const int64_t* entry;
  int64_t stride;
  const int64_t* pos;
  const float* norm_w;
  float eps;
  int rope;                            // of the main copy
  int key_pairs, key_first, key_step;  // of the key: pair i is (first + i step, that + other)
  int key_other;
  float key_magnitude;
  uint8_t *kv_codes, *kv_scales, *ix_codes, *ix_scales;
  void* ws;
};
struct LatentTurns {
  Turns<32> kv;
  Turns<64> key;
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
  } else {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xFFFF0000u);
  }
}
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float u[4];
    if constexpr (sizeof(T) == 2) {
      if (i & 1) continue;
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + i / 2);
      const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[4 * i + 2 * j] = __uint_as_float(q[j] << 16);
        v[4 * i + 2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
      }
    } else {
      load4(p + 4 * i, u);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = u[j];
    }
  }
}
__device__ __forceinline__ float2 load2(const float* p) { return __ldg(reinterpret_cast<const float2*>(p)); }
__device__ __forceinline__ float2 load2(const uint16_t* p) {
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// plane row of a destination, -1: padding, -2: outside the planes
__device__ __forceinline__ int64_t place(const LatentArgs& a, int r) {
  const int32_t s = a.slot[r];
  const int64_t e = a.entry[r];
  if (s == -1 && e == -1) return -1;
  return s < 0 || s >= a.n_slots || e < 0 || e >= a.stride ? -2 : s * a.stride + e;
}

// 1 / sqrt(mean(x^2) + eps) of a row of which each lane has 16 values, as a pair of fp32: an estimate and one Newton
// step.  A row far from 1 is first scaled by a power of two, which `scale` says (exact).
__device__ __forceinline__ FF inverse_rms(float (&v)[16], float eps, float& scale) {
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fabsf(v[i]));
  const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));  // of values >= 0 as their bits
  const int e = (int)(top >> 23) - 127;
  scale = 1.0f;
  if (e > 40 || e < -40) {  // squares and their remainders within fp32's range
    const int k = min(max(e, -60), 100);
    scale = exp2i_f32(-k);
    eps = ldexpf(eps, -2 * k);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= scale;
  }
  FF ss{0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const FF p = two_prod(v[i], v[i]), s = two_sum(ss.hi, p.hi);
    ss = FF{s.hi, __fadd_rn(ss.lo, __fadd_rn(s.lo, p.lo))};
  }
  ss = fast_sum(ss.hi, ss.lo);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1)
    ss = add(ss, FF{__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
  const FF m = add(FF{ss.hi * (1.0f / kDMain), ss.lo * (1.0f / kDMain)}, FF{eps, 0.0f});
  const float r = rsqrtf(m.hi);
  const FF t = mul(m, two_prod(r, r));
  const float d = __fsub_rn(__fsub_rn(1.0f, t.hi), t.lo);
  return FF{r, 0.5f * r * d};
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_latent_append(LatentArgs a, const __grid_constant__ LatentTurns turns) {
  __shared__ __align__(16) float s_row[kWarps][kDIdx];
  ptx::griddep_launch();
  ptx::griddep_wait();
  if ((int)blockIdx.x < a.checkers) {  // these report destinations outside the planes: the error word is theirs alone
    if (blockIdx.x == 0 && threadIdx.x == 0) *reinterpret_cast<ErrWord*>(a.ws) = ErrWord{0, 0, 0};
    if (a.checkers > 1) ptx::cluster_sync();
    else __syncthreads();
#pragma unroll 8
    for (int r = blockIdx.x * kThreads + threadIdx.x; r < a.R; r += a.checkers * kThreads)
      if (place(a, r) == -2)
        report_error(a.ws, CSA2_ERR_INDEX_RANGE,
                     a.slot[r] < 0 || a.slot[r] >= a.n_slots ? (long long)a.slot[r] : a.entry[r]);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int r = ((int)blockIdx.x - a.checkers) * kWarps + warp;
  if (r >= a.R) return;
  const int64_t row = place(a, r);
  if (row < 0) return;  // the same for the whole warp
  const uint64_t pos = a.pos ? (uint64_t)a.pos[r] : 0;
  if (a.x) {
    const T* const x = static_cast<const T*>(a.x) + (int64_t)r * kDMain;
    float v[16];
    load16(x + 16 * lane, v);
    FF inv{1.0f, 0.0f};
    float scale = 1.0f;
    if (a.norm_w) {
      inv = inverse_rms(v, a.eps, scale);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 w4 = __ldg(reinterpret_cast<const float4*>(a.norm_w + 16 * lane) + i);
        const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = value(mul(mul(inv, v[4 * i + j]), w[j]));
      }
    }
    if (a.rope) {
      FF c, s;
      turn_cos_sin(pos * turns.kv.f[lane], c, s);
      const float2 p = load2(x + kRopeFirst + 2 * lane);
      FF u{p.x * scale, 0.0f}, w{p.y * scale, 0.0f};
      if (a.norm_w) {
        const float2 g = load2(a.norm_w + kRopeFirst + 2 * lane);
        u = mul(mul(inv, u.hi), g.x);
        w = mul(mul(inv, w.hi), g.y);
      }
      turn_pair(u, w, c, s);
      *reinterpret_cast<float2*>(&s_row[warp][2 * lane]) = make_float2(value(u), value(w));
      __syncwarp();
      if (lane >= 28) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 f = *reinterpret_cast<const float4*>(&s_row[warp][16 * (lane - 28) + 4 * i]);
          v[4 * i] = f.x;
          v[4 * i + 1] = f.y;
          v[4 * i + 2] = f.z;
          v[4 * i + 3] = f.w;
        }
      }
      __syncwarp();
    }
    quantize_main_group_vals(v, a.kv_codes + row * 256 + lane * 8, a.kv_scales + row * 32 + lane);
  }
  if (a.key) {
    float v[4];
    load4(static_cast<const T*>(a.key) + (int64_t)r * kDIdx + 4 * lane, v);
    if (a.key_pairs) {
      *reinterpret_cast<float4*>(&s_row[warp][4 * lane]) = make_float4(v[0], v[1], v[2], v[3]);
      __syncwarp();
      for (int i = lane; i < a.key_pairs; i += 32) {
        FF c, s;
        turn_cos_sin(pos * turns.key.f[i], c, s);
        float* const at = &s_row[warp][a.key_first + i * a.key_step];
        FF u{at[0], 0.0f}, w{at[a.key_other], 0.0f};
        turn_pair(u, w, c, s);
        at[0] = value(mul(u, a.key_magnitude));
        at[a.key_other] = value(mul(w, a.key_magnitude));
      }
      __syncwarp();
      const float4 f = *reinterpret_cast<const float4*>(&s_row[warp][4 * lane]);
      v[0] = f.x;
      v[1] = f.y;
      v[2] = f.z;
      v[3] = f.w;
    }
    // codec.cuh, quantize_index_group_vals: eight lanes have a group
    float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    int e = -127;
    uint32_t codes = 0;
    if (amax > 0.0f) {
      e = floor_log2_f32(amax) - 2;
      e = e < -127 ? -127 : (e > 127 ? 127 : e);
      const float f = exp2i_f32(-e);
      codes = float2_to_e2m1x2(__fmul_rn(v[0], f), __fmul_rn(v[1], f)) |
              float2_to_e2m1x2(__fmul_rn(v[2], f), __fmul_rn(v[3], f)) << 8;
    }
    *reinterpret_cast<uint16_t*>(a.ix_codes + row * 64 + lane * 2) = (uint16_t)codes;
    if (lane % 8 == 0) a.ix_scales[row * 4 + lane / 8] = (uint8_t)(e + 127);
  }
}

}  // namespace
}  // namespace csa2

extern "C" size_t csa2_latent_append_workspace_size(int32_t R) { return R < 0 || R > 1 << 30 ? 0 : csa2::kWsHeader; }

extern "C" csa2_status csa2_latent_append(const void* x, const void* key, int32_t type, int32_t R,
                                          const csa2_kv_planes* dst, int32_t n_slots, const int32_t* slot,
                                          const int64_t* entry, const csa2_norm_rope* kv_nr,
                                          const csa2_rope_scaling* scaling, const int64_t* pos,
                                          const csa2_rotary* key_rot, void* ws, size_t ws_bytes, csa2_stream stream) {
  using namespace csa2;
  if (type != CSA2_F32 && type != CSA2_BF16) return CSA2_ERR_INVALID_ARG;
  if (R < 0 || R > 1 << 30 || n_slots <= 0 || !planes_ok(dst)) return CSA2_ERR_INVALID_ARG;
  if (kv_nr && !norm_rope_ok(kv_nr)) return CSA2_ERR_INVALID_ARG;
  if (!scaling_ok(scaling) || (key_rot && !rotary_ok(key_rot, kDIdx))) return CSA2_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(key, 16) || !aligned(slot, 4) || !aligned(entry, 8) || !aligned(pos, 8))
    return CSA2_ERR_INVALID_ARG;
  const bool rope = x && kv_nr && kv_nr->rope, key_rope = key && key_rot;
  if (R > 0 && (!slot || !entry || ((rope || key_rope) && !pos))) return CSA2_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256) || ws_bytes < kWsHeader) return CSA2_ERR_WORKSPACE;
  const int checkers = R > kManyRows ? kCheckers : 1;
  LatentArgs a{x, key, R, n_slots, checkers, slot, entry, dst->seq_stride, pos, x && kv_nr ? kv_nr->norm_weight : nullptr,
               kv_nr ? kv_nr->norm_eps : 0.0f, rope, 0, 0, 0, 0, 1.0f, dst->kv_codes, dst->kv_scales, dst->ix_codes,
               dst->ix_scales, ws};
  LatentTurns turns{};
  if (rope) make_turns(&turns.kv, 64, kv_nr->rope_base, scaling);
  if (key_rope) {
    const bool halves = key_rot->layout == CSA2_ROPE_HALVES;
    a.key_pairs = key_rot->n_rot / 2;
    a.key_first = key_rot->first;
    a.key_step = halves ? 1 : 2;
    a.key_other = halves ? key_rot->n_rot / 2 : 1;
    a.key_magnitude = key_rot->magnitude;
    make_turns(&turns.key, key_rot->n_rot, key_rot->base, &key_rot->scaling);
  }
  cudaStream_t st = (cudaStream_t)stream;
  KernelTimer timer("k_latent_append", st);
  const auto kern = type == CSA2_F32 ? k_latent_append<float> : k_latent_append<uint16_t>;
  const unsigned ctas = (unsigned)(align_up((size_t)(checkers + cdiv(R, kWarps)), (size_t)checkers));
  launch_clusters(kern, dim3(ctas), dim3(kThreads), checkers, 1, 0, st, a, turns);
  return launch_status();
}
