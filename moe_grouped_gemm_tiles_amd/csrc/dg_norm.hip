// dg_norm.hip -- residual addition, RMS norm and the per-token FP8 cast in one
// pass, and the gradient of the norm, on gfx950.
//
// Forward, per row of K values (all in FP32, every output rounded once):
//     s = x + residual,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s * rstd * w,
//     per 128 values:  sf = amax(|y|) / 448 (or the UE8M0 form),  q = E4M3(y / sf),
// the same scale rule and quotient as the plain cast (dg_cast.hpp).
//
// Backward, with xhat = s * rstd and g = dy * w:
//     dx = rstd * (g - xhat * mean(g * xhat)) + dresidual,   dw = sum over rows of dy * xhat
// (the cast passes its gradient through unchanged).
//
// Both are bound by HBM: every operand is read once and every result written
// once, a row staying in registers from its loads to its stores.  What that
// takes on this chip (a plain device copy reaches 5.0 to 6.1 TB/s):
//   * the next row's loads are in flight while a row is reduced, cast and stored,
//     and nothing in between waits for them: no branch stands around a memory
//     access (buffer descriptors drop what is out of range), and lanes exchange
//     values on the VALU (DPP, permlane swaps), not through LDS;
//   * accesses past the L2s' capacity are streaming: with them 33280 x 7168 BF16
//     takes 363 us, without 448 us (before the prefetch);
//   * workgroups run through memory together.  With one or two rows per workgroup
//     the forward takes 276 us, with 4 297 us, with 16 336 us: the more regions are
//     being read at once, the less HBM delivers.  The backward, whose workgroups
//     persist to keep their column sums, is best with a few MiB of rows in flight: 208
//     workgroups for rows of 8 KiB and more (316 us; 256 331 us, 512 354 us, 1024
//     357 us), a multiple of 208 for shorter ones (bwd_grid), up to 1664 for 128 columns;
//   * FP32 rows are split so that every load instruction reads 256 adjacent bytes per
//     16 lanes: 29000 x 4096 backward 343 -> 306 us, 4099 x 4096 forward 34 -> 29.5 us.
// 33280 x 7168 BF16 now: forward 274 us, 6.1 TB/s; backward 313 us, 6.1 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "dg.h"
#include "dg_cast.hpp"
#include "dg_common.hpp"

namespace {

namespace norm {

using namespace dg::cast;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kMaxK = 16384;
// Threads of the longest rows and 8-value chunks that each holds: forward 1024 and two (3695 x 11264: 60 us, with
// 512 and four 70 us), backward 512 and four (14560 x 16384: 318 us, the other way 327 us).
constexpr int kFwdThreads = 1024, kFwdChunks = 2;
constexpr int kBwdThreads = 512, kBwdChunks = 4;
constexpr uint32_t kNowhere = 0xffffffffu;           // a buffer offset past every operand: the access is dropped

// Rows go through buffer descriptors of exactly their length: lanes past the
// row's end load zeros and store nothing, and an operand that is not there is a
// descriptor of length 0.  So the row loop has no branch around a memory access,
// and the compiler can count what is in flight: with branches it has to wait for
// everything before each use.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// Cache policy of the row accesses: 2 marks them as streaming (not kept in the
// caches), 0 does not.
template <bool NT>
constexpr int kPolicy = NT ? 2 : 0;

// Where a thread's eight values of chunk ch lie in a row, in elements: BF16 rows
// give it eight adjacent ones (16 bytes), FP32 rows four in each half of the
// 128-value block, so that 16 lanes always read 256 adjacent bytes.
template <bool BF16>
__device__ __forceinline__ uint32_t place(int ch, int half) {
  return BF16 ? ch * 8 + half * 4 : (ch >> 4) * 128 + half * 64 + (ch & 15) * 4;
}

// Rows of 128 and 256 values take 16 and 32 lanes, so a wave works on four and two of them at a
// time (ROWS): a lane's offset in its operand is then its row's distance from the wave's first row,
// or kNoRow past the last row, and a descriptor reaches over the wave's rows.  (Longer rows: 0.)
constexpr uint32_t kNoRow = 0x80000000u;
template <int ROWS>
__device__ __forceinline__ uint32_t row_off(int sub, bool valid, int64_t ld) {
  if constexpr (ROWS == 1) return 0;
  return valid ? (uint32_t)sub * (uint32_t)ld : kNoRow;
}
template <int ROWS>
__device__ __forceinline__ uint32_t reach(uint32_t bytes, int64_t ld) {
  return bytes == 0 ? 0 : (uint32_t)(ROWS - 1) * (uint32_t)ld + bytes;
}

// Raw bits of a thread's chunks of one row.
template <bool BF16, int C>
struct Raw {
  u32x4 d[C][BF16 ? 1 : 2];
};

template <bool BF16, bool NT, int C>
__device__ __forceinline__ void load_row(__amdgpu_buffer_rsrc_t r, uint32_t off, int tid, int nt, Raw<BF16, C>& o) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h)
      o.d[c][h] = __builtin_amdgcn_raw_buffer_load_b128(r, off + place<BF16>(c * nt + tid, h) * (BF16 ? 2 : 4), 0,
                                                        kPolicy<NT>);
}

template <bool BF16, int C>
__device__ __forceinline__ void unpack(const Raw<BF16, C>& o, int c, float (&v)[8]) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(o.d[c][0][i] << 16);
      v[2 * i + 1] = __uint_as_float(o.d[c][0][i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(o.d[c][i >> 2][i & 3]);
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};  // round to nearest even
  return __builtin_bit_cast(uint32_t, v);
}

// Eight values of chunk ch, laid out as rows of type BF16, to FP32 memory.
template <bool BF16, bool NT>
__device__ __forceinline__ void store8_fp32(__amdgpu_buffer_rsrc_t r, uint32_t off, int ch, const float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const u32x4 o = {__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                     __float_as_uint(v[4 * h + 3])};
    __builtin_amdgcn_raw_buffer_store_b128(o, r, off + place<BF16>(ch, h) * 4, 0, kPolicy<NT>);
  }
}

// Eight values of chunk ch to a row, rounded to the row's type.
template <bool BF16, bool NT>
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t r, uint32_t off, int ch, const float (&v)[8]) {
  if constexpr (BF16) {
    const u32x4 o = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    __builtin_amdgcn_raw_buffer_store_b128(o, r, off + ch * 16, 0, kPolicy<NT>);
  } else {
    store8_fp32<false, NT>(r, off, ch, v);
  }
}

// A thread's chunks of the norm's weight (BF16 or FP32), as FP32, laid out as rows of type BF16.
template <bool BF16, int C>
__device__ __forceinline__ void load_weight(const uint8_t* w, int bf16, int k, int tid, int nt, float (&v)[C][8]) {
  const __amdgpu_buffer_rsrc_t r = make_rsrc(w, (uint32_t)k * (bf16 ? 2 : 4));
  if (bf16) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x2 o = __builtin_amdgcn_raw_buffer_load_b64(r, place<BF16>(c * nt + tid, h) * 2, 0, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          v[c][4 * h + 2 * i] = __uint_as_float(o[i] << 16);
          v[c][4 * h + 2 * i + 1] = __uint_as_float(o[i] & 0xffff0000u);
        }
      }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 o = __builtin_amdgcn_raw_buffer_load_b128(r, place<BF16>(c * nt + tid, h) * 4, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][4 * h + i] = __uint_as_float(o[i]);
      }
  }
}

// Lane permutations on the VALU: 0xB1 and 0x4E swap neighbours and pairs in
// each four lanes, 0x141 and 0x140 mirror eight and sixteen.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}

// Largest of 16 adjacent lanes.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, dpp<0xB1>(v));
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  return max(v, dpp<0x140>(v));
}

// Sum of lanes l, l ^ 16 (or l ^ 32).
__device__ __forceinline__ float add_xor16(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float add_xor32(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Sum of 16 adjacent lanes.
__device__ __forceinline__ float sum16(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  return v + dpp<0x140>(v);
}

// Sum over the row, the same on every thread of it and in a fixed order: over its 64 / ROWS
// lanes, and then over the waves of the workgroup.  `slot` holds one float per wave (zeros past
// the last); calls in turn use different slots, so one barrier per call is enough.
constexpr int kSlots = 16;
static_assert(kSlots * 64 >= std::max(kFwdThreads, kBwdThreads), "one slot per wave, read by 16 lanes");
template <int ROWS>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = sum16(v);
  if (ROWS < 4) v = add_xor16(v);
  if (ROWS < 2) v = add_xor32(v);
  if (ROWS > 1 || blockDim.x == 64) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  return sum16(slot[threadIdx.x & 15]);
}

// A value that is the same on every lane, kept in a scalar register.
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}
// ss / k with 1/k given, the quotient's error corrected once.
__device__ __forceinline__ float mean(float ss, float k, float inv_k) {
  const float q = ss * inv_k;
  return __builtin_fmaf(__builtin_fmaf(-q, k, ss), inv_k, q);
}
// 1 / sqrt(t) for normal t: the hardware's estimate r (1 ulp) and one Newton step r + r (1 - t r^2) / 2, with the
// rounding error of t r carried along, so that only the last addition rounds.  Every code of a row depends on this
// one value: with the estimate alone one row in ten is off by an ulp.
__device__ __forceinline__ float rsqrt(float t) {
  const float r = __builtin_amdgcn_rsqf(t), a = t * r, e = __builtin_fmaf(t, r, -a);
  const float d = __builtin_fmaf(-e, r, __builtin_fmaf(-a, r, 1.0f));
  return __builtin_fmaf(0.5f * r, d, r);
}

// Codes of eight values of a block whose amax has the bits `amax` (compared as
// an unsigned integer, so that a NaN is the largest).  The common case takes
// amax / 448 and x / s with the steps of the correctly rounded division
// (dg_cast.hpp), written so that a zero keeps its sign and without a clamp:
// |x / s| <= 448 * (1 + 2^-23), which rounds to 448.  Zero blocks and scales
// outside the range of those steps take the general form, and a block with an
// Inf or NaN keeps it: its scale is not finite, and neither are the codes of
// such elements.
__device__ __forceinline__ float quotient(float x, float s, float y) {
  const float q0 = x * y;
  const float q1 = __builtin_fmaf(-__builtin_fmaf(s, q0, -x), y, q0);
  return __builtin_fmaf(-__builtin_fmaf(s, q1, -x), y, q1);
}

template <bool UE8M0>
__device__ __forceinline__ u32x2 codes8(const float (&v)[8], uint32_t amax, float& s, uint32_t& byte) {
  const float a = __uint_as_float(amax);
  const float t = quotient(a, kE4M3Max, 1.0f / kE4M3Max);
  if (plain_div_range(t)) {
    float y[8];
    if constexpr (UE8M0) {
      byte = (__float_as_uint(t) + 0x7fffffu) >> 23;  // the exponent, one more unless t is a power of two
      s = __uint_as_float(byte << 23);
      const float inv = __uint_as_float((254 - byte) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = v[i] * inv;
    } else {
      byte = 0;
      s = t;
      const float r = refined_recip(s);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = quotient(v[i], s, r);
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
    return u32x2{(uint32_t)lo, (uint32_t)hi};
  }
  if (amax >= 0x7f800000u) {
    byte = 255;
    s = amax > 0x7f800000u ? __builtin_nanf("") : __builtin_inff();
    u32x2 c = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i >> 2] |= (fabsf(v[i]) < __builtin_inff() ? 0u : 0x7fu) << (8 * (i & 3));
    return c;
  }
  if constexpr (UE8M0) {
    byte = ue8m0_byte(a);
    s = ue8m0_value(byte);
  } else {
    byte = 0;
    s = fp32_scale(a);
  }
  const uint2 c = quant8<UE8M0>(v, s);
  return u32x2{c.x, c.y};
}

struct FwdParams {
  const uint8_t* x;
  const uint8_t* res;
  uint8_t* res_out;
  const uint8_t* w;
  uint8_t* q;
  uint8_t* sf;
  uint8_t* y;
  float* rstd;
  int64_t ldx, ldr, ldro, ldq, ld_sf, ldy;  // bytes
  float eps;
  int m, k, rows_per_wg;
  int w_bf16;
};

// One workgroup takes rows_per_wg rows in turn (ROWS at a time), the next row's operands being
// loaded while a row is worked on; a thread holds chunks c * blockDim + tid of
// eight values of a row, so 16 adjacent lanes hold one 128-value block and a
// wave four adjacent ones (one packed UE8M0 word).
template <bool BF16, bool UE8M0, bool NT, int C, int ROWS>
__global__ void __launch_bounds__(ROWS > 1 ? 64 : C == 1 ? 512 : kFwdThreads, C == 1 ? 7 : BF16 ? 6 : 4)
    fwd_kernel(const FwdParams p) {
  __shared__ float s_sum[2][2][kSlots];  // [scaled again][row parity]
  constexpr int ES = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63, sub = ROWS > 1 ? lane / (64 / ROWS) : 0;
  const int tid = ROWS > 1 ? lane % (64 / ROWS) : threadIdx.x, nt = blockDim.x;
  const int chunks = p.k >> 3;
  const uint32_t bytes = (uint32_t)p.k * ES, res_bytes = p.res != nullptr ? bytes : 0;
  // Workgroups go to the eight XCDs in turn.  Each XCD takes runs of 32 adjacent rows, so that
  // the scales of a run, one 128-byte line per K block, meet in its L2 and are written once.
  const int run = max(1, 32 / p.rows_per_wg), whole = (int)gridDim.x / (8 * run) * (8 * run);
  int wg = blockIdx.x;
  if (wg < whole) {
    const int slot = wg >> 3;
    wg = (slot / run * 8 + (wg & 7)) * run + slot % run;
  }
  const int row0 = wg * p.rows_per_wg;
  const int row1 = min(row0 + p.rows_per_wg, p.m);
  if (ROWS == 1) {
    if (tid < 4 * kSlots) (&s_sum[0][0][0])[tid] = 0.f;
  }
  float w[C][8];
  load_weight<BF16, C>(p.w, p.w_bf16, p.k, tid, nt, w);
  Raw<BF16, C> x, r;
  const auto load = [&](int row) __attribute__((always_inline)) {
    const bool valid = ROWS == 1 || row + sub < row1;
    load_row<BF16, NT, C>(make_rsrc(p.x + row * p.ldx, reach<ROWS>(bytes, p.ldx)), row_off<ROWS>(sub, valid, p.ldx),
                          tid, nt, x);
    load_row<BF16, NT, C>(make_rsrc(p.res + row * p.ldr, reach<ROWS>(res_bytes, p.ldr)),
                          row_off<ROWS>(sub, valid, p.ldr), tid, nt, r);
  };
  load(row0);
  const float k = uniform((float)p.k), inv_k = uniform(1.0f / (float)p.k);
  if (ROWS == 1) __syncthreads();
  for (int row = row0; row < row1; row += ROWS) {
    const bool valid = ROWS == 1 || row + sub < row1;
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(p.res_out + row * p.ldro, reach<ROWS>(res_bytes, p.ldro));
    float v[C][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float t[8];
      unpack<BF16, C>(x, c, v[c]);
      unpack<BF16, C>(r, c, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] += t[i];
        ss = __builtin_fmaf(v[c][i], v[c][i], ss);
      }
    }
    if (row + ROWS < row1) load(row + ROWS);
#pragma unroll
    for (int c = 0; c < C; ++c) store8<BF16, NT>(ro, row_off<ROWS>(sub, valid, p.ldro), c * nt + tid, v[c]);
    ss = row_sum<ROWS>(ss, s_sum[0][row & 1]);
    const float arg = mean(ss, k, inv_k) + p.eps;
    float rstd = rsqrt(arg), rstd_out = rstd;  // what multiplies the row, and what is stored
    const bool again = !(ss >= 0x1p-100f && arg < __builtin_inff());
    if (ROWS > 1 ? __any(again) : again) {
      // Squares (or the argument) past FP32's range on either side (the same branch on every thread): again,
      // scaled.  A sum that overflowed has a value of 2^57 or more, so 2^-80 brings the largest to between 2^-23 and
      // 2^48; below 2^-100 all values are below 2^-50, and 2^100 brings even the smallest denormal to 2^-49.
      const float f = ss < 1.0f ? 0x1p100f : 0x1p-80f;
      ss = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += (v[c][i] * f) * (v[c][i] * f);
      ss = row_sum<ROWS>(ss, s_sum[1][row & 1]);
      const double exact = 1.0 / sqrt((double)ss / ((double)f * (double)f) / p.k + (double)p.eps);
      // a row so small that 1/rms nears or passes FP32's range is scaled itself
      const float up = again && exact >= 0x1p100 ? 0x1p100f : 1.0f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= up;
      rstd = again ? (float)(exact / up) : rstd;
      rstd_out = again ? (float)exact : rstd;
    }
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(rstd_out),
                                          make_rsrc(p.rstd + row, p.rstd != nullptr ? 4 * ROWS : 0),
                                          tid == 0 && valid ? sub * 4 : kNowhere, 0, 0);
    const __amdgpu_buffer_rsrc_t ry = make_rsrc(p.y + row * p.ldy, p.y != nullptr ? reach<ROWS>(bytes, p.ldy) : 0);
    const __amdgpu_buffer_rsrc_t rq = make_rsrc(p.q + row * p.ldq, reach<ROWS>((uint32_t)p.k, p.ldq));
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.sf + (int64_t)row * 4, 0xfffffffeu);
    const uint32_t q_off = row_off<ROWS>(sub, valid, p.ldq);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = c * nt + tid;
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] = v[c][i] * rstd * w[c][i];
        amax = max(amax, __float_as_uint(v[c][i]) & 0x7fffffffu);
      }
      store8<BF16, NT>(ry, row_off<ROWS>(sub, valid, p.ldy), ch, v[c]);
      amax = max16(amax);
      float s;
      uint32_t byte;
      const u32x2 q = codes8<UE8M0>(v[c], amax, s, byte);
      if constexpr (BF16) {
        __builtin_amdgcn_raw_buffer_store_b64(q, rq, q_off + ch * 8, 0, kPolicy<NT>);
      } else {
        __builtin_amdgcn_raw_buffer_store_b32(q[0], rq, q_off + place<false>(ch, 0), 0, kPolicy<NT>);
        __builtin_amdgcn_raw_buffer_store_b32(q[1], rq, q_off + place<false>(ch, 1), 0, kPolicy<NT>);
      }
      if constexpr (UE8M0) {
        byte = ch < chunks ? byte : 127u;
        uint32_t word;
        if constexpr (ROWS == 1)
          word = __builtin_amdgcn_readlane(byte, 0) | __builtin_amdgcn_readlane(byte, 16) << 8 |
                 __builtin_amdgcn_readlane(byte, 32) << 16 | __builtin_amdgcn_readlane(byte, 48) << 24;
        else if constexpr (ROWS == 2)
          word = (sub == 0 ? __builtin_amdgcn_readlane(byte, 0) | __builtin_amdgcn_readlane(byte, 16) << 8
                           : __builtin_amdgcn_readlane(byte, 32) | __builtin_amdgcn_readlane(byte, 48) << 8) |
                 0x7f7f0000u;
        else
          word = byte | 0x7f7f7f00u;
        const uint32_t at = (ROWS == 1 ? lane : tid) == 0 && ch < chunks && valid
                                ? (uint32_t)(ch >> 6) * (uint32_t)p.ld_sf + sub * 4 : kNowhere;
        __builtin_amdgcn_raw_buffer_store_b32(word, rs, at, 0, 0);
      } else {
        const uint32_t at =
            (lane & 15) == 0 && ch < chunks && valid ? (uint32_t)(ch >> 4) * (uint32_t)p.ld_sf + sub * 4 : kNowhere;
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), rs, at, 0, 0);
      }
    }
  }
}

struct BwdParams {
  const uint8_t* dy;
  const uint8_t* s;
  const uint8_t* w;
  const uint8_t* dres;
  const float* rstd;
  uint8_t* dx;
  float* part;
  int64_t lddy, lds, lddres, lddx;  // bytes
  int m, k;
  int w_bf16;
};

// One workgroup takes rows (ROWS at a time) blockIdx, blockIdx + gridDim, ... (the next ones'
// operands in flight) and keeps its sum of dy * xhat per column in registers;
// it leaves that as one row of `part`.
template <bool BF16, bool NT, int C, int ROWS>
__global__ void __launch_bounds__(ROWS > 1 ? 64 : kBwdThreads) bwd_kernel(const BwdParams p) {
  __shared__ float s_sum[2][kSlots];
  constexpr int ES = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63, sub = ROWS > 1 ? lane / (64 / ROWS) : 0;
  const int tid = ROWS > 1 ? lane % (64 / ROWS) : threadIdx.x, nt = blockDim.x;
  const uint32_t bytes = (uint32_t)p.k * ES, res_bytes = p.dres != nullptr ? bytes : 0;
  if (ROWS == 1) {
    if (tid < 2 * kSlots) (&s_sum[0][0])[tid] = 0.f;
  }
  float w[C][8], dw[C][8];
  load_weight<BF16, C>(p.w, p.w_bf16, p.k, tid, nt, w);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.f;
  Raw<BF16, C> dy, s, dr;
  float rstd = 0.f;
  const auto load = [&](int row) __attribute__((always_inline)) {
    const bool valid = ROWS == 1 || row + sub < p.m;
    load_row<BF16, NT, C>(make_rsrc(p.dy + row * p.lddy, reach<ROWS>(bytes, p.lddy)), row_off<ROWS>(sub, valid, p.lddy),
                          tid, nt, dy);
    load_row<BF16, NT, C>(make_rsrc(p.s + row * p.lds, reach<ROWS>(bytes, p.lds)), row_off<ROWS>(sub, valid, p.lds),
                          tid, nt, s);
    load_row<BF16, NT, C>(make_rsrc(p.dres + row * p.lddres, reach<ROWS>(res_bytes, p.lddres)),
                          row_off<ROWS>(sub, valid, p.lddres), tid, nt, dr);
  };
  const auto load_rstd = [&](int row) __attribute__((always_inline)) {
    if constexpr (ROWS == 1)
      rstd = p.rstd[row];
    else
      rstd = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          make_rsrc(p.rstd + row, 4 * (uint32_t)min(ROWS, p.m - row)), sub * 4, 0, 0));
  };
  int row = blockIdx.x * ROWS;
  load_rstd(row);
  constexpr bool kAhead = BF16 || C < 4;  // (else the next row's operands would not fit in registers)
  if (kAhead) load(row);
  const float inv_k = 1.0f / (float)p.k;
  if (ROWS == 1) __syncthreads();
  for (int turn = 0; row < p.m; turn ^= 1) {
    if (!kAhead) load(row);
    float g[C][8], xh[C][8], d[C][8];
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      unpack<BF16, C>(dy, c, g[c]);
      unpack<BF16, C>(s, c, xh[c]);
      unpack<BF16, C>(dr, c, d[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[c][i] *= rstd;
        dw[c][i] = __builtin_fmaf(g[c][i], xh[c][i], dw[c][i]);
        g[c][i] *= w[c][i];
        dot = __builtin_fmaf(g[c][i], xh[c][i], dot);
      }
    }
    const float r = rstd;
    const int here = row;
    row += gridDim.x * ROWS;
    if (row < p.m) {
      load_rstd(row);
      if (kAhead) load(row);
    }
    dot = row_sum<ROWS>(dot, s_sum[turn]) * inv_k;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.dx + here * p.lddx, reach<ROWS>(bytes, p.lddx));
    const uint32_t off = row_off<ROWS>(sub, here + sub < p.m, p.lddx);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[c][i] = __builtin_fmaf(r, __builtin_fmaf(-xh[c][i], dot, g[c][i]), d[c][i]);
      store8<BF16, NT>(rx, off, c * nt + tid, d[c]);
    }
  }
  if constexpr (ROWS > 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[0][i] = add_xor32(dw[0][i]);
      if (ROWS > 2) dw[0][i] = add_xor16(dw[0][i]);
    }
  }
  const __amdgpu_buffer_rsrc_t rp = make_rsrc(p.part + (int64_t)blockIdx.x * p.k, (uint32_t)p.k * 4);
#pragma unroll
  for (int c = 0; c < C; ++c) store8_fp32<BF16, false>(rp, sub == 0 ? 0 : kNoRow, c * nt + tid, dw[c]);
}

constexpr int kDwCols = 32;   // columns of one workgroup of the column sum
constexpr int kDwWaves = 16;  // its waves; eight lanes take 32 columns of a row, a wave eight rows

// Sum of v over the lanes l, l + 8, l + 16, ... of the wave.
__device__ __forceinline__ float sum_every8(float v) {
  v += dpp<0x128>(v);  // rotated by eight in each 16 lanes
  return add_xor32(add_xor16(v));
}

// dw[col] (+)= sum over rows of part[row][col], in a fixed order.
__global__ void __launch_bounds__(kDwWaves * 64) dw_kernel(const float* part, int rows, int k, float* dw,
                                                           int accumulate) {
  __shared__ float t[kDwWaves][kDwCols];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c4 = (tid & 7) * 4, col = blockIdx.x * kDwCols + c4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kStep = kDwWaves * 8, kUnroll = 4;
  int i = tid >> 3;
  for (; i + (kUnroll - 1) * kStep < rows; i += kUnroll * kStep) {
    float4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      v[u] = *reinterpret_cast<const float4*>(part + (int64_t)(i + u * kStep) * k + col);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) { a.x += v[u].x; a.y += v[u].y; a.z += v[u].z; a.w += v[u].w; }
  }
  for (; i < rows; i += kStep) {
    const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)i * k + col);
    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
  }
  a = make_float4(sum_every8(a.x), sum_every8(a.y), sum_every8(a.z), sum_every8(a.w));
  if (lane < 8) *reinterpret_cast<float4*>(&t[wave][c4]) = a;
  __syncthreads();
  if (tid < kDwCols) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kDwWaves; ++w) sum += t[w][tid];
    float* o = dw + blockIdx.x * kDwCols + tid;
    *o = accumulate ? *o + sum : sum;
  }
}

// Threads and chunks per thread for rows of k values: as many threads as there are chunks up to
// 512, then more chunks per thread, no more than `most`.
struct Shape {
  int threads, chunks;
};
Shape shape_for(int k, int most) {
  const int n = k / 8;
  int c = 1;
  while (c < most && (n + c - 1) / c > 512) c *= 2;
  return {((n + c - 1) / c + 63) / 64 * 64, c};
}

// Rows a wave takes at a time.  (A million rows of 128: forward 150 us with four, 325 us with one;
// backward 170 and 249 us.  500000 of 256: 150 and 188 us with two and one, 171 and 184 us.)
int rows_of(int k) { return k == 128 ? 4 : k == 256 ? 2 : 1; }
// Whether so many rows of an operand lie within 32-bit offsets.
bool near(int64_t ld) { return ld < (int64_t)1 << 28; }

// Rows one workgroup of the forward takes: one where a row keeps a CU's load queue busy by itself,
// more for shorter rows (a million of 128 columns: 150 us with 8, 156 us with 4; 333000 of 384:
// 160 us with 4, 167 us with 8; 500000 of 256: 148.5 and 150 us).  The longest BF16 rows, of which no more
// than two workgroups share a CU, need the prefetch (20000 x 8320: 212 us with 4, 228 us with 2, 281 us
// with 1; 14560 x 16384: 298, 284 and 305 us) and a full last round (4339 x 11520: 65 us with 3, 71 us with
// 4); FP32 ones do not (7000 x 16384: 250, 249 and 240 us).  With neither residual nor y there is less
// traffic for the same arithmetic, and the prefetch decides (33280 x 7168: 154 us with 6, 158 us with 4, 175 us
// with 2, 206 us with 1; 33280 x 4096: 92 us with 4, 101 us with 2; with y, 20000 x 4096 FP32: 131 and 122 us).
int fwd_rows(int m, int k, bool bf16, bool codes_only) {
  const int step = rows_of(k);
  int rows = std::max(1, std::min(k > 4096 ? 1 : k > 512 ? 2 : k > 128 ? 4 : 8, m / 2048));
  if (codes_only && k > 512) rows = std::max(1, std::min(k > 4096 ? 6 : 4, m / 1024));
  rows = std::max(step, rows / step * step);
  if (k > 8192 && bf16) {
    const int at_once = 256 * (24 / ((k / 16 + 63) / 64));  // 24 waves to a CU
    const auto turns = [&](int r) { return ((int64_t)m + r * at_once - 1) / (r * at_once) * r; };
    for (int r = 2; r <= (k > 12288 ? 2 : 4); ++r)
      if (turns(r) * 15 <= turns(rows) * 16) rows = r;
  }
  while (m / rows > 1 << 21) rows *= 2;  // (a launch holds fewer than 2^32 threads)
  return rows;
}

// Workgroups of the backward's row loop, each of which leaves a row of partial sums: 208 for rows
// of 8 KiB and more, else a multiple of 208 that comes to about as many bytes in flight (a number between one
// and two per CU leaves some CUs twice the work of others: 20000 x 2560 FP32 136 us with 208, 167 us with 332).
// 20741 x 2176 BF16: 63 us with 416, 81 us with 208; 30000 x 1024 FP32: 82 us with 416, 91 us with 832;
// a million x 128 BF16: 170 us with 1664, 181 us with half as many more, 186 us with a quarter less.
// Few rows: one turn each up to 64 workgroups (49 x 11264 FP32: 8.0 us, with two turns 9.3 us), then three
// turns, because the column sum has to read what each of them leaves (1000 x 1024: 7.0 us, two turns 7.8,
// six 7.7; 333 x 1536 FP32: 6.0, 6.0 and 6.8 us).
int bwd_grid(int m, int k, bool bf16) {
  const int rows = rows_of(k), full = bf16 ? 4096 : 2048;
  const int most = 208 * std::max(1, (3 * full + 2 * k) / (3 * k)) / rows;
  const int turns = (m + rows - 1) / rows;
  return turns <= 64 ? turns : std::max(64, std::min(most, (turns + 2) / 3));
}

inline bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A row-major operand: rows 16-byte aligned and at least k elements apart.
inline bool rows_ok(const void* p, int64_t ld, int64_t es, int k) {
  return p != nullptr && aligned_to(p, 16) && ld >= k && (ld * es) % 16 == 0;
}

// Operands past the L2s' 32 MiB are marked as streaming; smaller ones stay for whoever
// reads them next.  (2048 x 7168 BF16 forward, 103 MB: 21.0 us streaming, 22.8 us not.)
bool streams(int64_t bytes) { return bytes > (int64_t)32 << 20; }

template <bool BF16, bool UE8M0, bool NT>
void launch_fwd(const FwdParams& p, Shape s, int rows, dim3 grid, hipStream_t stream) {
  const dim3 block(s.threads);
  if (rows == 4) hipLaunchKernelGGL((fwd_kernel<BF16, UE8M0, NT, 1, 4>), grid, block, 0, stream, p);
  else if (rows == 2) hipLaunchKernelGGL((fwd_kernel<BF16, UE8M0, NT, 1, 2>), grid, block, 0, stream, p);
  else if (s.chunks == 1) hipLaunchKernelGGL((fwd_kernel<BF16, UE8M0, NT, 1, 1>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((fwd_kernel<BF16, UE8M0, NT, 2, 1>), grid, block, 0, stream, p);
}
template <bool BF16, bool UE8M0>
void launch_fwd(const FwdParams& p, Shape s, int rows, bool nt, dim3 grid, hipStream_t stream) {
  if (nt) launch_fwd<BF16, UE8M0, true>(p, s, rows, grid, stream);
  else launch_fwd<BF16, UE8M0, false>(p, s, rows, grid, stream);
}

template <bool BF16, bool NT>
void launch_bwd(const BwdParams& p, Shape s, int rows, dim3 grid, hipStream_t stream) {
  const dim3 block(s.threads);
  if (rows == 4) hipLaunchKernelGGL((bwd_kernel<BF16, NT, 1, 4>), grid, block, 0, stream, p);
  else if (rows == 2) hipLaunchKernelGGL((bwd_kernel<BF16, NT, 1, 2>), grid, block, 0, stream, p);
  else if (s.chunks == 1) hipLaunchKernelGGL((bwd_kernel<BF16, NT, 1, 1>), grid, block, 0, stream, p);
  else if (s.chunks == 2) hipLaunchKernelGGL((bwd_kernel<BF16, NT, 2, 1>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((bwd_kernel<BF16, NT, 4, 1>), grid, block, 0, stream, p);
}
template <bool BF16>
void launch_bwd(const BwdParams& p, Shape s, int rows, bool nt, dim3 grid, hipStream_t stream) {
  if (nt) launch_bwd<BF16, true>(p, s, rows, grid, stream);
  else launch_bwd<BF16, false>(p, s, rows, grid, stream);
}

dg_status launch_status() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_SUCCESS : dg::record_hip_error(e);
}

}  // namespace norm

}  // namespace

extern "C" {

dg_status dg_add_rms_norm_cast_to_fp8(const void* x, int64_t ldx, const void* residual, int64_t ld_residual,
                                      void* residual_out, int64_t ld_residual_out, dg_dtype dtype,
                                      const void* weight, dg_dtype weight_dtype, float eps, void* q, int64_t ldq,
                                      void* sf, int64_t ld_sf, int ue8m0, void* y, int64_t ldy, float* rstd, int m,
                                      int k, hipStream_t stream) {
  using namespace norm;
  if (m < 0 || k < 0 || (dtype != DG_DTYPE_BF16 && dtype != DG_DTYPE_FP32) ||
      (weight_dtype != DG_DTYPE_BF16 && weight_dtype != DG_DTYPE_FP32) || !(eps >= 0.f))
    return DG_ERROR_INVALID_VALUE;
  if (k % 128 != 0 || k > kMaxK) return DG_ERROR_NOT_SUPPORTED;
  if (m == 0 || k == 0) return DG_SUCCESS;
  const int64_t es = dtype == DG_DTYPE_BF16 ? 2 : 4;
  if (!rows_ok(x, ldx, es, k)) return DG_ERROR_INVALID_VALUE;
  if ((residual == nullptr) != (residual_out == nullptr)) return DG_ERROR_INVALID_VALUE;
  if (residual != nullptr && (!rows_ok(residual, ld_residual, es, k) || !rows_ok(residual_out, ld_residual_out, es, k)))
    return DG_ERROR_INVALID_VALUE;
  if (y != nullptr && !rows_ok(y, ldy, es, k)) return DG_ERROR_INVALID_VALUE;
  if (weight == nullptr || !aligned_to(weight, 16)) return DG_ERROR_INVALID_VALUE;
  if (q == nullptr || !aligned_to(q, 8) || ldq < k || ldq % 8 != 0) return DG_ERROR_INVALID_VALUE;
  if (sf == nullptr || !aligned_to(sf, 16) || ld_sf < m || ld_sf % 4 != 0) return DG_ERROR_INVALID_VALUE;
  if (ld_sf > (int64_t)0xfffffff0 / 4 / (k / 128)) return DG_ERROR_NOT_SUPPORTED;  // 32-bit offsets into sf
  if (!aligned_to(rstd, 4)) return DG_ERROR_INVALID_VALUE;
  FwdParams p{static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(residual),
              static_cast<uint8_t*>(residual_out), static_cast<const uint8_t*>(weight), static_cast<uint8_t*>(q),
              static_cast<uint8_t*>(sf), static_cast<uint8_t*>(y), rstd, ldx * es, ld_residual * es,
              ld_residual_out * es, ldq, ld_sf * 4, ldy * es, eps, m, k,
              fwd_rows(m, k, dtype == DG_DTYPE_BF16, residual == nullptr && y == nullptr),
              weight_dtype == DG_DTYPE_BF16};
  const Shape s = shape_for(k, kFwdChunks);
  const bool nt = streams((int64_t)m * k * (es * (residual != nullptr ? 3 : 1) + 1));
  const dim3 grid((m + p.rows_per_wg - 1) / p.rows_per_wg);
  const int rows = near(p.ldx) && near(p.ldr) && near(p.ldro) && near(p.ldy) && near(ldq) ? rows_of(k) : 1;
  if (dtype == DG_DTYPE_BF16) {
    if (ue8m0) launch_fwd<true, true>(p, s, rows, nt, grid, stream);
    else launch_fwd<true, false>(p, s, rows, nt, grid, stream);
  } else {
    if (ue8m0) launch_fwd<false, true>(p, s, rows, nt, grid, stream);
    else launch_fwd<false, false>(p, s, rows, nt, grid, stream);
  }
  return launch_status();
}

size_t dg_get_rms_norm_backward_workspace_size(int m, int k) {
  if (m <= 0 || k <= 0 || k % 128 != 0 || k > norm::kMaxK) return 0;
  // (BF16 rows have the most workgroups)
  return (size_t)norm::bwd_grid(m, k, true) * (size_t)k * sizeof(float);
}

dg_status dg_rms_norm_backward(const void* dy, int64_t ld_dy, const void* s, int64_t ld_s, dg_dtype dtype,
                               const void* weight, dg_dtype weight_dtype, const float* rstd, const void* dresidual,
                               int64_t ld_dresidual, void* dx, int64_t ld_dx, float* dw, int accumulate_dw, int m,
                               int k, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace norm;
  if (m < 0 || k < 0 || (dtype != DG_DTYPE_BF16 && dtype != DG_DTYPE_FP32) ||
      (weight_dtype != DG_DTYPE_BF16 && weight_dtype != DG_DTYPE_FP32))
    return DG_ERROR_INVALID_VALUE;
  if (k % 128 != 0 || k > kMaxK) return DG_ERROR_NOT_SUPPORTED;
  if (k == 0) return DG_SUCCESS;
  if (dw == nullptr || !aligned_to(dw, 16)) return DG_ERROR_INVALID_VALUE;
  const int grid = m > 0 ? bwd_grid(m, k, dtype == DG_DTYPE_BF16) : 0;
  if (m > 0) {
    const int64_t es = dtype == DG_DTYPE_BF16 ? 2 : 4;
    if (!rows_ok(dy, ld_dy, es, k) || !rows_ok(s, ld_s, es, k) || !rows_ok(dx, ld_dx, es, k))
      return DG_ERROR_INVALID_VALUE;
    if (dresidual != nullptr && !rows_ok(dresidual, ld_dresidual, es, k)) return DG_ERROR_INVALID_VALUE;
    if (weight == nullptr || !aligned_to(weight, 16) || rstd == nullptr || !aligned_to(rstd, 4))
      return DG_ERROR_INVALID_VALUE;
    if (workspace == nullptr || !aligned_to(workspace, 256) ||
        workspace_bytes < dg_get_rms_norm_backward_workspace_size(m, k))
      return DG_ERROR_WORKSPACE;
    const BwdParams p{static_cast<const uint8_t*>(dy), static_cast<const uint8_t*>(s),
                      static_cast<const uint8_t*>(weight), static_cast<const uint8_t*>(dresidual), rstd,
                      static_cast<uint8_t*>(dx), static_cast<float*>(workspace), ld_dy * es, ld_s * es,
                      ld_dresidual * es, ld_dx * es, m, k, weight_dtype == DG_DTYPE_BF16};
    const Shape sh = shape_for(k, kBwdChunks);
    const bool nt = streams((int64_t)m * k * es * (dresidual != nullptr ? 4 : 3));
    const int rows = near(p.lddy) && near(p.lds) && near(p.lddres) && near(p.lddx) ? rows_of(k) : 1;
    if (dtype == DG_DTYPE_BF16) launch_bwd<true>(p, sh, rows, nt, dim3(grid), stream);
    else launch_bwd<false>(p, sh, rows, nt, dim3(grid), stream);
    const dg_status st = launch_status();
    if (st != DG_SUCCESS) return st;
  }
  hipLaunchKernelGGL(dw_kernel, dim3(k / kDwCols), dim3(kDwWaves * 64), 0, stream,
                     static_cast<const float*>(workspace), grid, k, dw, accumulate_dw != 0);
  return launch_status();
}

}  // extern "C"
