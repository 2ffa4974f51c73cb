// Pieces that the decode-attention kernels share: the row codec's widening steps, the query's
// staging, the in-layer extras, and the softmax warps' vote.
#pragma once

#include "codec.cuh"
#include "ptx.cuh"
#include "timing.cuh"

namespace csa2 {

constexpr float kLog2e = 1.4426950408889634f;
// the softmax reference (log2 units) moves only when a chunk exceeds it by
// more than 8 nats, so probabilities stay below e^8 (inside f16)
constexpr float kTau2 = 8.0f * kLog2e;
// the reference of a head with no row yet: finite, so that 2^(S c2 - kNoRef) of a
// missing (-inf) row stays 0, and far below any logit, so that a row exceeds it
constexpr float kNoRef = -1.0e30f;
// q' plane stride: 64 heads x 16 bytes, unpadded, so that every core matrix the
// S MMAs read sits on a 128-byte line
constexpr int kQPlane = kHAtt * 8;       // in f16 elements (1024 bytes)

// In-layer extras ("DeepSeek-V4: ...", CSA, other details), each off when null /
// zero: RMSNorm weight of the query heads, RoPE of the query at qpos[b] with the
// output turned back by -qpos[b], per-head sink logits.
struct AttnExtras {
  const float* qnorm_w;
  float eps;
  int rope;
  const int64_t* qpos;
  const float* sink;
  const int64_t* win_pos;  // [B][n_swa] position of each window row (< 0: empty), or null: all visible
  const int64_t* win_lo;   // [B] lowest visible window position
  RopeTheta th;
};

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\tmov.b32 {t0, t1, t2, t3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t0;\n\tcvt.rn.f16x2.e2m1x2 %1, t1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, t2;\n\tcvt.rn.f16x2.e2m1x2 %3, t3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t h;
  uint16_t v = (uint16_t)two;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return h;
}

// q' = q_h 2^-s_h in f16 with 2^s_h bringing the head's largest |q| to
// [2^14, 2^15), clamped so that both 2^s_h and 2^-s_h are normal fp32 values;
// bf16 q keeps q' exact and inside the f16 range (with RMSNorm or RoPE the
// fp32 result is rounded to f16 once).  One bulk copy brings the query's bf16
// rows ([64][512]) into row slot 1; the softmax and MMA warps, idle until the
// first chunk's rows are written, convert them from there while the row warps
// dequantize chunk 0 into slot 0.  Warp 8 + w takes heads 8w .. 8w + 7: lane
// l = 8g + t head 8w + t over the 8-channel planes (t + 4i + g) mod 64, i < 16.
// The eight lanes of a phase then read eight different banks of the bf16 rows
// (their planes differ mod 8) and write eight consecutive head slots of the
// [c/8][head][c%8] image, so neither side conflicts; the values are read again
// for each pass rather than held (a pass holding all 64 registers spills other
// warps' state), and the four lanes of a head combine its maximum (and sum of
// squares) with two shuffles.
template <bool kEx>
__device__ __forceinline__ void stage_q(uint16_t (*sq)[kQPlane], float* c2, const uint16_t* qs, float scale, int w, int lane,
                                        const AttnExtras& ex, int b) {
  const int t = lane & 7, g = lane >> 3, h = 8 * w + t;
  const uint4* src = reinterpret_cast<const uint4*>(qs + h * kDMain);
  const bool norm = kEx && ex.qnorm_w != nullptr;
  const bool rot = kEx && ex.rope;
  float r = 1.0f;  // 1 / RMS of the head
  if (norm) {
    float ss = 0.0f;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const uint4 q4 = src[(t + 4 * i + g) & 63];
      const uint32_t w4[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v0 = __uint_as_float(w4[j] << 16), v1 = __uint_as_float(w4[j] & 0xFFFF0000u);
        ss = fmaf(v0, v0, ss);
        ss = fmaf(v1, v1, ss);
      }
    }
    ss += __shfl_xor_sync(0xffffffffu, ss, 8);
    ss += __shfl_xor_sync(0xffffffffu, ss, 16);
    r = 1.0f / sqrtf(ss / (float)kDMain + ex.eps);
  }
  // RoPE turns planes 56 .. 63 (pairs 4 (p - 56) + pr); lane l keeps the cosine and
  // sine of pair l (every head turns by the same angles)
  float rcos = 1.0f, rsin = 0.0f;
  if (rot) rope_cos_sin(ex.th.t[lane], (double)ex.qpos[b], rcos, rsin);
  // the 8 channels of plane p after RMSNorm and RoPE
  auto plane = [&](int p, float (&v)[8]) {
    const uint4 q4 = src[p];
    const uint32_t w4[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w4[j] << 16);
      v[2 * j + 1] = __uint_as_float(w4[j] & 0xFFFF0000u);
    }
    if (norm) {
      const float4* wv = reinterpret_cast<const float4*>(ex.qnorm_w + 8 * p);
      const float4 a = __ldg(wv), c = __ldg(wv + 1);
      const float wq[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = wq[k] * (v[k] * r);
    }
    if (rot) {
#pragma unroll
      for (int pr = 0; pr < 4; ++pr) {  // every lane shuffles; only planes 56 .. 63 turn
        const int pair = (4 * (p - 56) + pr) & 31;
        const float c = __shfl_sync(0xffffffffu, rcos, pair), sn = __shfl_sync(0xffffffffu, rsin, pair);
        if (p >= 56) rope_pair(v[2 * pr], v[2 * pr + 1], c, sn);
      }
    }
  };
  float mx = 0.0f;
  if (kEx) {
#pragma unroll 2
    for (int i = 0; i < 16; ++i) {
      float v[8];
      plane((t + 4 * i + g) & 63, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(v[k]));
    }
  } else {  // |bf16| orders as its bit pattern: a packed 16-bit maximum over the raw words
    uint32_t m2 = 0;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const uint4 q4 = src[(t + 4 * i + g) & 63];
      const uint32_t w4[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) asm("max.u16x2 %0, %0, %1;" : "+r"(m2) : "r"(w4[j] & 0x7FFF7FFFu));
    }
    mx = __uint_as_float(max(m2 & 0xFFFFu, m2 >> 16) << 16);
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
  const int sig = mx > 0.0f ? min(max(floor_log2_f32(mx) - 14, -126), 126) : 0;
  const float inv = exp2i_f32(-sig);  // exact power of two: q 2^-sig rounds only in the f16 conversion
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int p = (t + 4 * i + g) & 63;
    float v[8];
    plane(p, v);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h2 = __floats2half2_rn(v[2 * j] * inv, v[2 * j + 1] * inv);
      o[j] = *reinterpret_cast<const uint32_t*>(&h2);
    }
    *reinterpret_cast<uint4*>(&sq[p][h * 8]) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (g == 0) c2[h] = kLog2e * scale * exp2i_f32(sig);
}

// Whether some of the four softmax warps (named barrier 2, 128 threads) saw a
// logit above its head's reference (lane 0 of each warp posts `wover`) and
// whether one of them gave up waiting (lanes 1-8 post `wbad`): one barrier, the
// count of posted predicates below 8 for the first, at least 8 for the second.
// Every softmax warp passes it once per chunk, also after a failed wait, so no
// warp is left at the barrier.
__device__ __forceinline__ uint32_t softmax_vote(bool wover, bool wbad, int lane) {
  const uint32_t pred = lane == 0 ? (wover ? 1u : 0u) : (lane <= 8 && wbad ? 1u : 0u);
  uint32_t n;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.popc.u32 %0, 2, 128, p;\n\t}"
      : "=r"(n)
      : "r"(pred)
      : "memory");
  return n;
}
// the four softmax warps (named barrier 2): shared-memory writes before it are seen after it
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 2, 128;" ::: "memory"); }

// Argument checks and kernel form of the in-layer extras of an attention call.
csa2_status attn_extras(const csa2_norm_rope* q_nr, const int64_t* q_pos, const float* sink, const csa2_window* win,
                        int32_t n_swa, float softmax_scale, AttnExtras* ex);

}  // namespace csa2
