// Append of ready latents to slots or pages, normalised and rotated on the way (csa2_latent_append).
//
// Row r's main copy: y = w x / sqrt(mean(x^2) + eps), the last 64 channels turned by pos, rounded to fp32 once, then
// the cache's codec; its indexer key: turned by pos, then the codec.  The codec's borders make the bytes depend on the
// last bits of y: from a y formed in fp32, off by up to 2^-19, a code in some thousand rows falls to the other side.  So
// a row is formed in fp32 first, with every value's code taken at both ends of what it may be; where the ends agree,
// the byte is certain.  Where one does not (one row in fifty after a norm), the row is formed again in pairs of fp32
// (rotary.cuh), to 2^-36, and quantized from that.  In pairs alone: 1,283 warp instructions a row and 47 us for 32,768.
// That goes by dense data: a zero's ends have different codes (8 and 0), so a row with a zero in a group that is normalised or
// rotated is formed twice.  32,768 rows with a channel that is always zero take 50.7 us (bf16 50.3), with zero key pairs 38.0.
//
// A warp takes the main copies of one row or two: lane l reads, normalises and rotates the channels 128 i + 4 l .. (whole
// lines) and quantizes 16 l .. (a group); a row changes hands in shared memory.  Another takes four rows' keys, eight
// lanes to each in the end.  Bytes would bound a long call, up to 2,560 read and 356 written a row; measured, the chain
// from a row's loads to its bytes does, 355 warp instructions for a main copy and 118 for a key, of which a warp issues one in
// eleven cycles: 32,768 rows with keys, normalised and rotated, 24.6 us in fp32 (3.9 TB/s), 23.6 in bf16 (2.3 TB/s); the
// main copies alone 20.4, without norm and rotation 16.1.  Two rows are two chains side by side.
#include "codec.cuh"
#include "ptx.cuh"
#include "rotary.cuh"
#include "timing.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kKeys = 4;  // rows whose keys a warp takes
// CTAs that look at the destinations: a cluster, so that none reports before the word is cleared; one for few rows
// (4,096 rows with one / eight 8.8 / 6.6 us, 2,048 without norm, rotation and keys 4.6 / 2.8).
constexpr int kReporters = 8, kManyRows = 512;
// Rows from which a warp takes two.  One / two, us, normalised and rotated with keys: 8,192 9.4 / 9.5, 12,000 11.9 / 11.7,
// 16,384 14.8 / 14.1, 32,768 25.8 / 23.6, 100,000 73 / 64; bf16 32,768 26.8 / 23.0; 32,768 without any 15.1 / 16.6 in fp32
// (the form that loses by it), 13.8 / 12.4 in bf16.
constexpr int kTwoRows = 12000;

struct LatentArgs {
  const void *x, *key;
  int32_t R, n_slots, reporters, main_ctas;
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
  const int32_t s = __ldg(a.slot + r);
  const int64_t e = __ldg(a.entry + r);
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
  if (e > 40 || e < -40) {  // squares and their remainders within fp32's range, and eps's: 2^61 at most
    const int least = max(((int)(__float_as_uint(eps) >> 23) - 127 - 60) / 2, -60);
    const int k = min(max(e, least), 100);
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

// ------------------------------------------------- in fp32, with both ends

// packed fp32 arithmetic on two neighbouring registers
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

// How far a value formed in fp32 may be off.  A norm: 16 fused steps and five sums of 2^-24 each, halved by the root,
// the root's two units and two products: below 2^-20 of the value.  A rotation: 2^-21 of |a| + |b| of its pair (angle
// 2^-24 pi, sine and cosine 2^-22, three roundings).  A rotated channel of the main copy has its partner in its group, so
// |a| + |b| <= 2 amax, and together 3 2^-20 amax; in units of the scale, of which amax is at most nine, below 2^-15.
// A channel that is normalised alone is off by 2^-20 of itself: below 2^-17 of the scale up to eight of it, beyond which
// its code is the largest anyway.
struct Off {
  float top, code;  // of the group's largest, relatively; of a value, in units of the scale
};
__device__ __forceinline__ Off off_by(bool norm, bool turned) {
  return turned ? Off{0x1p-18f, 0x1p-15f} : norm ? Off{0x1p-19f, 0x1p-17f} : Off{0.0f, 0.0f};
}
constexpr float kTopMost = 2600.0f;  // beyond, the scale saturates and amax may be more than nine of it
// of a key's channel, in units of the row's largest, turned: |a| + |b| is two of it at most
constexpr float kOffTurn = 0x1p-20f;

// The codes of eight values (E2M1, nearest even): value i of v at nibble i.
__device__ __forceinline__ uint32_t codes8(const uint64_t (&t)[4]) {
  uint32_t r;
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2(t[i], f[2 * i], f[2 * i + 1]);
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
      "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// One lane's group: codes and scale, and whether they are certain for values that are off (else exact).
__device__ __forceinline__ bool main_group(const uint64_t (&y)[8], Off by, uint2& codes, uint32_t& scale) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    unpack2(y[i], a, b);
    amax = fmaxf(amax, fmaxf(fabsf(a), fabsf(b)));
  }
  const bool off = by.code > 0.0f;
  const float t = __fdiv_rn(amax, 6.0f);
  // an exact value's ends are itself, an infinity's too
  const float t0 = off ? fmaf(t, -by.top, t) : t, t1 = off ? fmaf(t, by.top, t) : t;
  uint16_t ends;  // low byte: the lower one
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(ends) : "f"(t1), "f"(t0));
  scale = ends & 0xFFu;
  bool sure = !off || (amax < kTopMost && (ends >> 8) == scale);
  const float s = e4m3_to_float(scale);
  codes = make_uint2(0u, 0u);
  if (s == 0.0f) return sure;
  const float r = __frcp_rn(s);
  // the ends; an exact value's are itself, a negative zero's too
  const float e0 = off ? -by.code : -0.0f, e1 = off ? by.code : -0.0f;
  const uint64_t s2 = pack2(-s, -s), r2 = pack2(r, r), m2 = pack2(e0, e0), e2 = pack2(e1, e1);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint64_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // codec.cuh, div_by_e4m3
      const uint64_t x = y[4 * h + i], q0 = mul2(x, r2), q = fma2(fma2(q0, s2, x), r2, q0);
      lo[i] = add2(q, m2);
      hi[i] = add2(q, e2);
    }
    const uint32_t c = codes8(lo);
    sure = sure && c == codes8(hi);
    (h ? codes.y : codes.x) = c;
  }
  return sure;
}

// Sixteen values of a row in shared memory, 64 bytes of it, by chunks of four: lane l's first chunk is l / 2 mod 4, so
// that the eight lanes of an access are at different banks.
__device__ __forceinline__ int first_chunk(int lane) { return lane >> 1 & 3; }
__device__ __forceinline__ void take16(const float* at, int lane, uint64_t (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = *reinterpret_cast<const float4*>(at + 4 * ((i + first_chunk(lane)) & 3));
    y[2 * i] = pack2(f.x, f.y);
    y[2 * i + 1] = pack2(f.z, f.w);
  }
}
// their codes, 16 bits a chunk, put in order
__device__ __forceinline__ uint2 in_order(uint2 c, int lane) {
  const int s = first_chunk(lane);
  if (s & 2) c = make_uint2(c.y, c.x);
  if (s & 1) c = make_uint2(__funnelshift_l(c.y, c.x, 16), __funnelshift_l(c.x, c.y, 16));
  return c;
}

// The main copies of kRows rows (v: this lane's values) to plane rows `row` (< 0: nowhere); returns the rows (bit n: row n)
// that are not certain, of which nothing is written.
template <int kRows>
__device__ __forceinline__ uint32_t append_main(const LatentArgs& a, const LatentTurns& turns, float (&v)[kRows][4][4],
                                                const int64_t (&row)[kRows], const uint64_t (&pos)[kRows], float* s_row,
                                                int lane) {
  uint32_t open = 0;
  float2 turn[kRows];
  if (a.rope) {
    const uint64_t f = turns.kv.f[lane];
#pragma unroll
    for (int n = 0; n < kRows; ++n) turn_cos_sin(f, (int64_t)pos[n], turn[n].x, turn[n].y);
  }
  if (a.norm_w) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const float4*>(a.norm_w) + 32 * i + lane);
    float ss[kRows];
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
      uint64_t sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const uint64_t p = pack2(v[n][i][j], v[n][i][j + 1]);
          sum = fma2(p, p, sum);
        }
      float s0, s1;
      unpack2(sum, s0, s1);
      ss[n] = s0 + s1;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
      for (int n = 0; n < kRows; ++n) ss[n] += __shfl_xor_sync(0xffffffffu, ss[n], o);
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
      // sums whose terms are subnormal, or too large, are another's
      if (!(ss[n] > 0x1p-80f && ss[n] < 0x1p100f)) open |= 1u << n;
      const float inv = rsqrtf(fmaf(ss[n], 1.0f / kDMain, a.eps));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[n][i][0] = v[n][i][0] * inv * w[i].x;
        v[n][i][1] = v[n][i][1] * inv * w[i].y;
        v[n][i][2] = v[n][i][2] * inv * w[i].z;
        v[n][i][3] = v[n][i][3] * inv * w[i].w;
      }
    }
  }
  if (a.rope) {  // the last 64 channels, lanes 16 .. two pairs each; lane l has formed pair l's angle
#pragma unroll
    for (int n = 0; n < kRows; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float c = __shfl_sync(0xffffffffu, turn[n].x, 2 * lane + j);
        const float s = __shfl_sync(0xffffffffu, turn[n].y, 2 * lane + j);
        if (lane >= 16) rope_pair(v[n][3][2 * j], v[n][3][2 * j + 1], c, s);
      }
  }
#pragma unroll
  for (int n = 0; n < kRows; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(s_row + kDMain * n + 128 * i + 4 * lane) =
          make_float4(v[n][i][0], v[n][i][1], v[n][i][2], v[n][i][3]);
  __syncwarp();
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    uint64_t y[8];
    take16(s_row + kDMain * n + 16 * lane, lane, y);
    uint2 codes;
    uint32_t scale;
    const bool sure = main_group(y, off_by(a.norm_w, a.rope && lane >= 28), codes, scale);
    if (!__all_sync(0xffffffffu, sure)) open |= 1u << n;
    if (row[n] < 0 || (open >> n & 1u)) continue;
    *reinterpret_cast<uint2*>(a.kv_codes + row[n] * 256 + lane * 8) = in_order(codes, lane);
    a.kv_scales[row[n] * 32 + lane] = (uint8_t)scale;
  }
  return open;
}

// Exponent of a key's group scale (codec.cuh, quantize_index_group_vals): floor(log2 amax) - 2, -127 at least; the
// exponent field of a subnormal or zero gives that too.
__device__ __forceinline__ int key_exponent(float amax) { return max((int)(__float_as_uint(amax) >> 23) - 129, -127); }

// The keys of rows r .. r + kKeys - 1, eight lanes to each; returns the rows (bit i: row r + i) that are not certain,
// of which nothing is written.
template <typename T>
__device__ __forceinline__ uint32_t append_keys(const LatentArgs& a, const LatentTurns& turns, int r,
                                                float (*s_row)[kDIdx + 4], int lane) {
  const int i = lane / 8, j = lane % 8;  // the row, and of it channels 16 j ..
#pragma unroll
  for (int u = 0; u < kKeys; ++u) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (r + u < a.R) load4(static_cast<const T*>(a.key) + (int64_t)(r + u) * kDIdx + 4 * lane, v);
    *reinterpret_cast<float4*>(s_row[u] + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
  }
  const bool any = r + i < a.R;
  const int64_t pos = any && a.pos ? __ldg(a.pos + r + i) : 0;
  const int64_t row = any ? place(a, r + i) : -1;
  __syncwarp();
  for (int t = j; t < a.key_pairs; t += 8) {
    float c, s;
    turn_cos_sin(turns.key.f[t], pos, c, s);
    float* const at = s_row[i] + a.key_first + t * a.key_step;
    float m = at[0], n = at[a.key_other];
    rope_pair(m, n, c * a.key_magnitude, s * a.key_magnitude);
    at[0] = m;
    at[a.key_other] = n;
  }
  __syncwarp();
  uint64_t v[8];
  take16(s_row[i] + 16 * j, j, v);
  float amax = 0.0f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float x, y;
    unpack2(v[u], x, y);
    amax = fmaxf(amax, fmaxf(fabsf(x), fabsf(y)));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // a group is two lanes'
  float off = 0.0f, err = 0.0f;
  if (a.key_pairs) {
    float most = amax;
#pragma unroll
    for (int o = 4; o >= 2; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    // an infinity in the row, or a NaN that hides behind other values, is another's
    if (16 * j + 15 >= a.key_first && 16 * j < a.key_first + 2 * a.key_pairs) off = kOffTurn * most;
    err = fmaxf(off, __shfl_xor_sync(0xffffffffu, off, 1));
  }
  const int e = key_exponent(amax);
  const float f = exp2i_f32(-e);
  uint2 codes = make_uint2(0u, 0u);
  bool sure = off < INFINITY;  // no NaN either
  if (err != 0.0f) sure = sure && amax - err > 0.0f && key_exponent(amax - err) == e && key_exponent(amax + err) == e;
  if (amax > 0.0f) {
    // the ends; an exact value's are itself, a negative zero's too
    const float by = off * f, lo = off != 0.0f ? -by : -0.0f, hi = off != 0.0f ? by : -0.0f;
    const uint64_t f2 = pack2(f, f), lo2 = pack2(lo, lo), hi2 = pack2(hi, hi);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint64_t x[4], y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        x[u] = fma2(v[4 * h + u], f2, lo2);
        y[u] = fma2(v[4 * h + u], f2, hi2);
      }
      const uint32_t c = codes8(x);
      sure = sure && c == codes8(y);
      (h ? codes.y : codes.x) = c;
    }
  }
  const uint32_t open = __ballot_sync(0xffffffffu, !sure && row >= 0);
  if (row >= 0 && (open >> (8 * i) & 0xFFu) == 0u) {
    *reinterpret_cast<uint2*>(a.ix_codes + row * 64 + j * 8) = in_order(codes, j);
    if (j % 2 == 0) a.ix_scales[row * 4 + j / 2] = (uint8_t)(e + 127);
  }
  uint32_t rows = 0;
#pragma unroll
  for (int u = 0; u < kKeys; ++u) rows |= (open >> (8 * u) & 0xFFu) ? 1u << u : 0u;
  return rows;
}

// --------------------------------------------------------- in pairs of fp32

template <typename T>
__device__ __noinline__ void exact_main(const LatentArgs& a, const LatentTurns& turns, int r, int64_t row, uint64_t pos,
                                        float* s_row, int lane) {
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
    *reinterpret_cast<float2*>(s_row + 2 * lane) = make_float2(value(u), value(w));
    __syncwarp();
    if (lane >= 28) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(s_row + 16 * (lane - 28) + 4 * i);
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

template <typename T>
__device__ __noinline__ void exact_key(const LatentArgs& a, const LatentTurns& turns, int r, int64_t row, uint64_t pos,
                                       float* s_row, int lane) {
  float v[4];
  load4(static_cast<const T*>(a.key) + (int64_t)r * kDIdx + 4 * lane, v);
  if (a.key_pairs) {
    *reinterpret_cast<float4*>(s_row + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
    __syncwarp();
    for (int i = lane; i < a.key_pairs; i += 32) {
      FF c, s;
      turn_cos_sin(pos * turns.key.f[i], c, s);
      float* const at = s_row + a.key_first + i * a.key_step;
      FF u{at[0], 0.0f}, w{at[a.key_other], 0.0f};
      turn_pair(u, w, c, s);
      at[0] = value(mul(u, a.key_magnitude));
      at[a.key_other] = value(mul(w, a.key_magnitude));
    }
    __syncwarp();
    const float4 f = *reinterpret_cast<const float4*>(s_row + 4 * lane);
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
  }
  float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1)  // eight lanes have a group
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = key_exponent(amax);
  const float f = exp2i_f32(-e);
  uint32_t codes = 0;
  if (amax > 0.0f)
    codes = float2_to_e2m1x2(__fmul_rn(v[0], f), __fmul_rn(v[1], f)) |
            float2_to_e2m1x2(__fmul_rn(v[2], f), __fmul_rn(v[3], f)) << 8;
  *reinterpret_cast<uint16_t*>(a.ix_codes + row * 64 + lane * 2) = (uint16_t)codes;
  if (lane % 8 == 0) a.ix_scales[row * 4 + lane / 8] = (uint8_t)(e + 127);
}

template <typename T, int kRows>
__global__ void __launch_bounds__(kThreads, kRows > 1 ? 8 : 9)
    k_latent_append(const __grid_constant__ LatentArgs a, const __grid_constant__ LatentTurns turns) {
  constexpr int kRoom = kRows > 1 ? kRows * kDMain : kKeys * (kDIdx + 4);
  static_assert(kRoom % 4 == 0 && kRoom >= kDMain && kRoom >= kKeys * (kDIdx + 4), "rows, or four keys");
  __shared__ __align__(16) float s_room[kWarps][kRoom];
  ptx::griddep_launch();
  ptx::griddep_wait();
  if ((int)blockIdx.x < a.reporters) {  // these report destinations outside the planes: the error word is theirs alone
    if (blockIdx.x == 0 && threadIdx.x == 0) *reinterpret_cast<ErrWord*>(a.ws) = ErrWord{0, 0, 0};
    if (a.reporters > 1) ptx::cluster_sync();
    else __syncthreads();
#pragma unroll 8
    for (int r = blockIdx.x * kThreads + threadIdx.x; r < a.R; r += a.reporters * kThreads)
      if (place(a, r) == -2)
        report_error(a.ws, CSA2_ERR_INDEX_RANGE,
                     a.slot[r] < 0 || a.slot[r] >= a.n_slots ? (long long)a.slot[r] : a.entry[r]);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, cta = (int)blockIdx.x - a.reporters;
  if (cta >= a.main_ctas) {
    const int r = ((cta - a.main_ctas) * kWarps + warp) * kKeys;
    if (!a.key || r >= a.R) return;
    auto* const s_keys = reinterpret_cast<float(*)[kDIdx + 4]>(s_room[warp]);
    for (uint32_t open = append_keys<T>(a, turns, r, s_keys, lane); open; open &= open - 1) {
      const int i = r + __ffs(open) - 1;
      exact_key<T>(a, turns, i, place(a, i), a.pos ? (uint64_t)a.pos[i] : 0, s_room[warp], lane);
    }
    return;
  }
  const int r = (cta * kWarps + warp) * kRows;
  if (r >= a.R) return;
  // everything the rows need is asked for before the first of it is used
  float v[kRows][4][4];
  uint64_t pos[kRows];
  int64_t row[kRows];
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    const int at = min(r + n, a.R - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) load4(static_cast<const T*>(a.x) + (int64_t)at * kDMain + 128 * i + 4 * lane, v[n][i]);
    pos[n] = a.pos ? (uint64_t)__ldg(a.pos + at) : 0;
    row[n] = r + n < a.R ? place(a, at) : -1;
  }
  uint32_t open = append_main(a, turns, v, row, pos, s_room[warp], lane);
#pragma unroll
  for (int n = 0; n < kRows; ++n)
    if (row[n] < 0) open &= ~(1u << n);
  for (; open; open &= open - 1) {
    const int at = r + __ffs(open) - 1;
    exact_main<T>(a, turns, at, place(a, at), a.pos ? (uint64_t)a.pos[at] : 0, s_room[warp], lane);
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
  const int reporters = R > kManyRows ? kReporters : 1;
  const int rows = R >= kTwoRows ? 2 : 1;
  const int main_ctas = x ? (int)cdiv(R, kWarps * rows) : 0, key_ctas = key ? (int)cdiv(R, kWarps * kKeys) : 0;
  LatentArgs a{x, key, R, n_slots, reporters, main_ctas, slot, entry, dst->seq_stride, pos,
               x && kv_nr ? kv_nr->norm_weight : nullptr, kv_nr ? kv_nr->norm_eps : 0.0f, rope, 0, 0, 0, 0, 1.0f,
               dst->kv_codes, dst->kv_scales, dst->ix_codes, dst->ix_scales, ws};
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
  const auto kern = type == CSA2_F32 ? (rows > 1 ? k_latent_append<float, 2> : k_latent_append<float, 1>)
                                     : (rows > 1 ? k_latent_append<uint16_t, 2> : k_latent_append<uint16_t, 1>);
  const unsigned ctas = (unsigned)align_up((size_t)reporters + main_ctas + key_ctas, (size_t)reporters);
  if (reporters > 1) launch_clusters(kern, dim3(ctas), dim3(kThreads), reporters, 1, 0, st, a, turns);
  else launch_pdl(kern, dim3(ctas), dim3(kThreads), 0, st, a, turns);
  return launch_status();
}
