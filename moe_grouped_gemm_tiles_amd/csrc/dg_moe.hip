// dg_moe.hip -- a whole gated expert layer for a few tokens in two kernels, on
// gfx950.
//
// For token t with experts ids[t][j] and weights tw[t][j], j < top_k:
//     h = x_t @ W13[e]^T  (2I values: gate, then up),
//     a = silu(h[:I]) * h[I:],
//     out_t = sum_j tw[t][j] * (a_j @ W2[e_j]^T).
// x, W13 and W2 are E4M3 with the GEMMs' scales (per row and 128 K for x, per
// 128 x 128 block for the weights).  With a few tokens each touched expert's
// weights are used for a handful of rows, so the layer is the reading of them
// once; everything else is arranged around that.
//
//   * gate/up kernel: a workgroup owns 16 gate and the matching 16 up rows of
//     one touched expert, its four waves split K, and every wave streams the
//     rows straight into registers as the first operand of
//     v_mfma_f32_16x16x128_f8f6f4 (one MFMA = one 128-K scale block); the
//     expert's tokens, up to 16 per MFMA, are the second operand.  The K
//     partial sums meet in LDS, and a is written once per (token, slot), in
//     BF16: the second product's MFMA takes BF16, and one rounding of a to 8
//     more bits than the E4M3 that the composed path would store costs the
//     result no more than the rounding of the output does.
//   * down kernel: a workgroup owns 16 output columns of all tokens; its waves
//     take (expert, K range) pieces in turn.  E4M3 is exact in BF16, so W2
//     fragments are converted in registers and the block scale is applied to
//     the FP32 sum of each 128 K values.  Each (token, slot) leaves its own
//     16 sums in LDS, and the slots are added in the order of j: no atomics,
//     the same bits every time.
//
// Which tokens go to which expert is worked out by every workgroup from ids
// (at most kPairs (token, slot) pairs per chunk of tokens; larger batches are
// further grid rows), so there is no planning kernel and no host work.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "dg.h"
#include "dg_common.hpp"

namespace {

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kPairs = 512;       // (token, slot) pairs a workgroup plans for
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kUpWaves = 4;
constexpr int kDownWaves = 8;

struct Params {
  const uint8_t* x;
  const void* sfx;
  const uint8_t* w13;
  const void* sf13;
  const uint8_t* w2;
  const void* sf2;
  const int32_t* ids;
  const float* tw;
  __bf16* act;  // [m * top_k][inter]
  uint16_t* out;
  int64_t ldx, ld_sfx, ld_out;
  int m, top_k, experts, hidden, inter;
  int tokens;  // tokens per chunk
  int slots;   // down kernel: most K ranges whose sums fit in LDS
};

// The pairs of one chunk by expert: expert of the i-th touched one, its first
// place in `order` and, in `order`, the pairs (token in chunk * top_k + slot).
// Pairs whose id is outside [0, experts) are in no list.
struct Plan {
  int16_t id[kPairs];
  uint16_t order[kPairs];
  uint16_t expert[kPairs];
  uint16_t start[kPairs + 1];
  int touched;
};

// Sorts the chunk's pairs by expert.  `count` holds kMaxExperts words of
// scratch.  The order of an expert's own pairs depends on timing, but no
// result does: a pair's place only says which MFMA column computes it.
__device__ __forceinline__ void make_plan(const Params& p, int t0, int pairs, Plan& plan, uint32_t* count) {
  const int tid = threadIdx.x, nt = blockDim.x;
  for (int e = tid; e < p.experts; e += nt) count[e] = 0;
  __syncthreads();
  for (int i = tid; i < pairs; i += nt) {
    const int e = p.ids[(int64_t)t0 * p.top_k + i];
    const bool ok = e >= 0 && e < p.experts;
    plan.id[i] = (int16_t)(ok ? e : -1);
    if (ok) atomicAdd(&count[e], 1u);
  }
  __syncthreads();
  if (tid < 64) {  // one wave: touched experts in order of their number, and where their pairs start
    int touched = 0, start = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
      const int e = e0 + tid;
      const int c = e < p.experts ? (int)count[e] : 0;
      const uint64_t mask = __ballot(c > 0);
      int before = c;  // inclusive sum of counts over the lanes
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(before, off);
        if (tid >= off) before += v;
      }
      if (c > 0) {
        const int i = touched + __popcll(mask & ((1ull << tid) - 1));
        plan.expert[i] = (uint16_t)e;
        plan.start[i] = (uint16_t)(start + before - c);
        count[e] = (uint32_t)(start + before - c);  // next free place of this expert
      }
      touched += __popcll(mask);
      start += __shfl(before, 63);
    }
    if (tid == 0) {
      plan.touched = touched;
      plan.start[touched] = (uint16_t)start;
    }
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += nt) {
    const int e = plan.id[i];
    if (e >= 0) plan.order[atomicAdd(&count[e], 1u)] = (uint16_t)i;
  }
  __syncthreads();
}

// 2^(byte - 127); byte 255 is NaN, byte 0 the denormal 2^-127.
__device__ __forceinline__ float e8m0(uint32_t byte) {
  return byte == 255 ? __builtin_nanf("") : __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}
template <bool UE8M0>
__device__ __forceinline__ float row_scale(const void* sf, int64_t ld, int64_t row, int kb) {
  if constexpr (UE8M0)
    return e8m0((static_cast<const uint32_t*>(sf)[(int64_t)(kb >> 2) * ld + row] >> (8 * (kb & 3))) & 255);
  else
    return static_cast<const float*>(sf)[(int64_t)kb * ld + row];
}
// Scale of K block kb in row block nb of a weight with nkb K blocks.
template <bool UE8M0>
__device__ __forceinline__ float block_scale(const void* sf, int64_t nb, int nkb, int kb) {
  if constexpr (UE8M0)
    return e8m0((static_cast<const uint32_t*>(sf)[nb * ((nkb + 3) >> 2) + (kb >> 2)] >> (8 * (kb & 3))) & 255);
  else
    return static_cast<const float*>(sf)[nb * nkb + kb];
}

// Operand fragment of a 16-row x 128-byte block: lane (r16, q4) takes the 16-byte
// chunks q4 and q4 + 4 of row r16.  Both operands of an MFMA are read this way, so
// the order of K inside the block does not matter.
__device__ __forceinline__ i32x8 load_frag(const uint8_t* p) {
  const i32x4 lo = *reinterpret_cast<const i32x4*>(p);
  const i32x4 hi = *reinterpret_cast<const i32x4*>(p + 64);
  return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

__device__ __forceinline__ f32x4 mfma_fp8(i32x8 a, i32x8 b) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// Eight E4M3 values as BF16 (exact).
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

// grid: (inter / 16, most touched experts, chunks).
template <bool UE8M0>
__global__ void __launch_bounds__(kUpWaves * 64) gate_up_kernel(const Params p) {
  __shared__ Plan plan;
  __shared__ uint32_t count[kMaxExperts];
  __shared__ float red[kUpWaves][8][64];
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, q4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.z * p.tokens;
  const int pairs = min(p.tokens, p.m - t0) * p.top_k;
  make_plan(p, t0, pairs, plan, count);
  const int i = blockIdx.y;
  if (i >= plan.touched) return;
  const int e = plan.expert[i], first = plan.start[i], n = plan.start[i + 1] - first;
  const int col0 = blockIdx.x * 16;
  const int nkb = p.hidden >> 7, nb = p.inter >> 7;
  const uint8_t* wg = p.w13 + ((int64_t)e * 2 * p.inter + col0 + r16) * p.hidden + 16 * q4;
  const uint8_t* wu = wg + (int64_t)p.inter * p.hidden;
  const int64_t sb = (int64_t)e * 2 * nb + (col0 >> 7);
  for (int g0 = 0; g0 < n; g0 += 16) {
    const int pair = plan.order[first + min(g0 + r16, n - 1)];
    const int64_t tok = t0 + pair / p.top_k;
    const uint8_t* x = p.x + tok * p.ldx + 16 * q4;
    f32x4 ag = {0.f, 0.f, 0.f, 0.f}, au = {0.f, 0.f, 0.f, 0.f};
    for (int kb = wave; kb < nkb; kb += kUpWaves) {
      const i32x8 fg = load_frag(wg + kb * 128), fu = load_frag(wu + kb * 128), fx = load_frag(x + kb * 128);
      const float sx = row_scale<UE8M0>(p.sfx, p.ld_sfx, tok, kb);
      const float sg = sx * block_scale<UE8M0>(p.sf13, sb, nkb, kb);
      const float su = sx * block_scale<UE8M0>(p.sf13, sb + nb, nkb, kb);
      const f32x4 pg = mfma_fp8(fg, fx), pu = mfma_fp8(fu, fx);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        ag[r] = __builtin_fmaf(pg[r], sg, ag[r]);
        au[r] = __builtin_fmaf(pu[r], su, au[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      red[wave][r][lane] = ag[r];
      red[wave][4 + r][lane] = au[r];
    }
    __syncthreads();
    if (wave == 0 && g0 + r16 < n) {
      __bf16 a[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float g = red[0][r][lane], u = red[0][4 + r][lane];
#pragma unroll
        for (int w = 1; w < kUpWaves; ++w) {
          g += red[w][r][lane];
          u += red[w][4 + r][lane];
        }
        a[r] = (__bf16)(silu(g) * u);
      }
      __bf16* o = p.act + ((int64_t)t0 * p.top_k + pair) * p.inter + col0 + 4 * q4;
      typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
      *reinterpret_cast<bf16x4*>(o) = bf16x4{a[0], a[1], a[2], a[3]};
    }
    __syncthreads();
  }
}

// grid: (hidden / 16, chunks).  Dynamic LDS: slots * pairs * 16 floats.
template <bool UE8M0>
__global__ void __launch_bounds__(kDownWaves * 64) down_kernel(const Params p) {
  __shared__ Plan plan;
  __shared__ uint32_t count[kMaxExperts];
  extern __shared__ float sums[];  // [K range][pair][16]
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, q4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.y * p.tokens;
  const int tokens = min(p.tokens, p.m - t0), pairs = tokens * p.top_k;
  make_plan(p, t0, pairs, plan, count);
  const int col0 = blockIdx.x * 16;
  const int nkb = p.inter >> 7;
  // K is split into ranges until there are two pieces for each wave
  int split = 1;
  while (2 * split <= p.slots && 2 * split <= nkb && plan.touched * split < 2 * kDownWaves) split *= 2;
  for (int u = wave; u < plan.touched * split; u += kDownWaves) {
    const int i = u / split, s = u % split;
    const int e = plan.expert[i], first = plan.start[i], n = plan.start[i + 1] - first;
    const int kb0 = nkb * s / split, kb1 = nkb * (s + 1) / split;
    const uint8_t* w = p.w2 + ((int64_t)e * p.hidden + col0 + r16) * p.inter + 16 * q4;
    const int64_t sb = (int64_t)e * (p.hidden >> 7) + (col0 >> 7);
    for (int g0 = 0; g0 < n; g0 += 16) {
      const int pair = plan.order[first + min(g0 + r16, n - 1)];
      const __bf16* a = p.act + ((int64_t)t0 * p.top_k + pair) * p.inter + 16 * q4;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      for (int kb = kb0; kb < kb1; ++kb) {
        const i32x8 f = load_frag(w + kb * 128);
        f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bf16x8 b = *reinterpret_cast<const bf16x8*>(a + kb * 128 + (c >> 1) * 64 + (c & 1) * 8);
          part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(f[2 * c], f[2 * c + 1]), b, part, 0, 0, 0);
        }
        const float sc = block_scale<UE8M0>(p.sf2, sb, nkb, kb);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(part[r], sc, acc[r]);
      }
      if (g0 + r16 < n)
        *reinterpret_cast<f32x4*>(&sums[((int64_t)s * pairs + pair) * 16 + 4 * q4]) = acc;
    }
  }
  __syncthreads();
  for (int o = tid; o < tokens * 16; o += kDownWaves * 64) {
    const int t = o >> 4, c = o & 15;
    float v = 0.f;
    for (int j = 0; j < p.top_k; ++j) {
      const int pair = t * p.top_k + j;
      if (plan.id[pair] < 0) continue;
      float y = 0.f;
      for (int s = 0; s < split; ++s) y += sums[((int64_t)s * pairs + pair) * 16 + c];
      v = __builtin_fmaf(p.tw[(int64_t)(t0 + t) * p.top_k + j], y, v);
    }
    const __bf16 b = (__bf16)v;
    p.out[(int64_t)(t0 + t) * p.ld_out + col0 + c] = __builtin_bit_cast(uint16_t, b);
  }
}

inline bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int kSumBytes = 32 * 1024;  // LDS for the pairs' sums: kPairs * 64 bytes

dg_status run(const void* x, int64_t ldx, const void* sfx, int64_t ld_sfx, const void* w13, const void* sf13,
              const void* w2, const void* sf2, const int32_t* ids, const float* tw, void* out, int64_t ld_out, int m,
              int top_k, int experts, int hidden, int inter, bool ue8m0, void* workspace, size_t workspace_bytes,
              hipStream_t stream) {
  if (m < 0 || top_k < 0 || experts < 0 || hidden < 0 || inter < 0) return DG_ERROR_INVALID_VALUE;
  if (hidden % 128 != 0 || inter % 128 != 0 || inter == 0 || top_k == 0 || top_k > kMaxTopK || experts == 0 ||
      experts > kMaxExperts)
    return DG_ERROR_NOT_SUPPORTED;
  if (m == 0 || hidden == 0) return DG_SUCCESS;
  for (const void* q : {x, sfx, w13, w2, static_cast<const void*>(out)})
    if (q == nullptr || !aligned_to(q, 16)) return DG_ERROR_INVALID_VALUE;
  for (const void* q : {sf13, sf2, static_cast<const void*>(ids), static_cast<const void*>(tw)})
    if (q == nullptr || !aligned_to(q, 4)) return DG_ERROR_INVALID_VALUE;
  if (ldx < hidden || ldx % 16 != 0 || ld_out < hidden || ld_out % 8 != 0 || ld_sfx < m || ld_sfx % 4 != 0)
    return DG_ERROR_INVALID_VALUE;
  if (workspace == nullptr || !aligned_to(workspace, 256) ||
      workspace_bytes < dg_get_moe_workspace_size(m, top_k, inter))
    return DG_ERROR_WORKSPACE;
  Params p{static_cast<const uint8_t*>(x), sfx, static_cast<const uint8_t*>(w13), sf13,
           static_cast<const uint8_t*>(w2), sf2, ids, tw, static_cast<__bf16*>(workspace),
           static_cast<uint16_t*>(out), ldx, ld_sfx, ld_out, m, top_k, experts, hidden, inter, kPairs / top_k, 1};
  const int chunks = (m + p.tokens - 1) / p.tokens;
  if (chunks > 65535) return DG_ERROR_NOT_SUPPORTED;
  const int pairs = (m < p.tokens ? m : p.tokens) * top_k;
  p.slots = kSumBytes / (pairs * 64);
  const int most = pairs < experts ? pairs : experts;
  const dim3 up(inter / 16, most, chunks), down(hidden / 16, chunks);
  if (ue8m0) hipLaunchKernelGGL(gate_up_kernel<true>, up, dim3(kUpWaves * 64), 0, stream, p);
  else hipLaunchKernelGGL(gate_up_kernel<false>, up, dim3(kUpWaves * 64), 0, stream, p);
  if (ue8m0) hipLaunchKernelGGL(down_kernel<true>, down, dim3(kDownWaves * 64), kSumBytes, stream, p);
  else hipLaunchKernelGGL(down_kernel<false>, down, dim3(kDownWaves * 64), kSumBytes, stream, p);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_SUCCESS : dg::record_hip_error(e);
}

}  // namespace moe

}  // namespace

extern "C" {

size_t dg_get_moe_workspace_size(int m, int top_k, int inter) {
  if (m <= 0 || top_k <= 0 || inter <= 0) return 0;
  return ((size_t)m * (size_t)top_k * (size_t)inter * 2 + 255) / 256 * 256;
}

dg_status dg_fp8_moe_few_tokens(const void* x, int64_t ldx, const float* sfx, int64_t ld_sfx, const void* w13,
                                const float* sf13, const void* w2, const float* sf2, const int32_t* topk_ids,
                                const float* topk_weights, void* out, int64_t ld_out, int m, int top_k,
                                int num_experts, int hidden, int inter, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  return moe::run(x, ldx, sfx, ld_sfx, w13, sf13, w2, sf2, topk_ids, topk_weights, out, ld_out, m, top_k,
                  num_experts, hidden, inter, false, workspace, workspace_bytes, stream);
}

dg_status dg_fp8_moe_few_tokens_ue8m0(const void* x, int64_t ldx, const int32_t* sfx, int64_t ld_sfx, const void* w13,
                                      const int32_t* sf13, const void* w2, const int32_t* sf2,
                                      const int32_t* topk_ids, const float* topk_weights, void* out, int64_t ld_out,
                                      int m, int top_k, int num_experts, int hidden, int inter, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
  return moe::run(x, ldx, sfx, ld_sfx, w13, sf13, w2, sf2, topk_ids, topk_weights, out, ld_out, m, top_k,
                  num_experts, hidden, inter, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
