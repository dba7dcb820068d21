#ifndef UPD
#define UPD 2
#endif
#ifndef UPG
#define UPG 2
#endif
#ifndef RH
#define RH 6144
#endif
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

#include <algorithm>
#include <cstdint>

#include "dg.h"
#include "dg_common.hpp"

namespace {

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kPairs = 512;       // (token, slot) pairs a workgroup plans for
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kUpWaves = 4;

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
  uint16_t order[kPairs];
  uint16_t expert[kPairs];
  uint16_t start[kPairs + 1];
  int touched;
};

// Sorts the chunk's pairs by expert; id[pair] becomes the pair's expert or -1.
// `count` holds kMaxExperts words of scratch.  The order of an expert's own pairs depends on timing, but no
// result does: a pair's place only says which MFMA column computes it.
__device__ __forceinline__ void make_plan(const Params& p, int t0, int pairs, Plan& plan, int16_t* id,
                                          uint32_t* count) {
  const int tid = threadIdx.x, nt = blockDim.x;
  for (int e = tid; e < p.experts; e += nt) count[e] = 0;
  __syncthreads();
  for (int i = tid; i < pairs; i += nt) {
    const int e = p.ids[(int64_t)t0 * p.top_k + i];
    const bool ok = e >= 0 && e < p.experts;
    id[i] = (int16_t)(ok ? e : -1);
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
    const int e = id[i];
    if (e >= 0) plan.order[atomicAdd(&count[e], 1u)] = (uint16_t)i;
  }
  __syncthreads();
}

// 2^(byte - 127); byte 255 is NaN, byte 0 the denormal 2^-127.
__device__ __forceinline__ float e8m0(uint32_t byte) {
  return byte == 255 ? __builtin_nanf("") : __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}
// Scale of K block kb from the word that holds it (FP32, or four packed bytes).
template <bool UE8M0>
__device__ __forceinline__ float scale_of(uint32_t word, int kb) {
  return UE8M0 ? e8m0((word >> (8 * (kb & 3))) & 255) : __uint_as_float(word);
}
template <bool UE8M0>
__device__ __forceinline__ int words(int nkb) { return UE8M0 ? (nkb + 3) >> 2 : nkb; }
template <bool UE8M0>
__device__ __forceinline__ int word_of(int kb) { return UE8M0 ? kb >> 2 : kb; }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
// The same from an address that is the same on every lane: into scalar registers, which the asm below needs.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a), hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return make_rsrc(reinterpret_cast<const void*>(((uint64_t)hi << 32) | lo), __builtin_amdgcn_readfirstlane(bytes));
}
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every operand here: the load gives zeros

// A wave streams its operands through a ring of stages of its own in LDS, one
// stage per 128-K block, with direct global->LDS loads: nothing is held in
// registers while it is on its way, and no other wave is waited for.  The loads
// are inline asm so that the compiler, which would wait for all of them before
// any LDS read, does not see them; they write no register.  The waits are
// counted below: a wave's vector loads complete in order, so "at most N
// outstanding" means that all but the last N loads have arrived, whatever
// stores are in flight besides.  s_nop 4 covers the wait states between a
// scalar write of m0 or of the descriptor and its use, which the compiler does
// not add inside asm.  NT: streaming, the weights are read once.
template <int BYTES, bool NT>
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t off) {
  if constexpr (BYTES == 16 && NT)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds" : : "v"(off), "s"(r), "s"(lds)
                 : "memory", "m0");
  else if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(off), "s"(r), "s"(lds)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds" : : "v"(off), "s"(r), "s"(lds)
                 : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  asm volatile("" ::: "memory");
}
// The wave's LDS reads have returned (their place may be loaded into again).
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((0xF) | (0x3 << 14) | (0x7 << 4) | (0x0 << 8));
  asm volatile("" ::: "memory");
}

// 16-row x 128-byte tiles lie in LDS row by row, the 16-byte chunk c of row r at
// chunk c ^ (r & 7); one load instruction brings eight whole rows.  An operand
// fragment: lane (r16, q4) takes chunks q4 and q4 + 4 of row r16.  Both operands of
// an MFMA are read this way, so the order of K inside a block does not matter.
__device__ __forceinline__ i32x8 read_frag(const uint8_t* tile, int r16, int q4) {
  const uint8_t* row = tile + r16 * 128;
  const i32x4 lo = *reinterpret_cast<const i32x4*>(row + ((q4 ^ (r16 & 7)) << 4));
  const i32x4 hi = *reinterpret_cast<const i32x4*>(row + (((q4 + 4) ^ (r16 & 7)) << 4));
  return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}
// Chunk of its row that a lane loads (row = 8 h + lane / 8).
__device__ __forceinline__ uint32_t tile_chunk(int lane) { return ((lane & 7) ^ (lane >> 3)) << 4; }

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

// Stage of the gate/up kernel: gate tile, up tile, NG token tiles, the tokens' scales
// (one per lane), the two block scales.
template <int NG>
struct UpStage {
  static constexpr int kX = 4096, kSx = kX + 2048 * NG, kSw = kSx + 256, kBytes = kSw + 256;
  static constexpr int kLoads = 6 + 2 * NG;
};

// A unit is one touched expert's tile of 16 columns of a; workgroups take contiguous
// ranges of units.  An expert with more than 16 * NG tokens takes several passes.
// grid: (workgroups, chunks).
template <bool UE8M0, int NG, int D>
__global__ void __launch_bounds__(kUpWaves * 64) gate_up_kernel(const Params p) {
  using S = UpStage<NG>;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kUpWaves * D * S::kBytes];
  __shared__ __attribute__((aligned(16))) float red[kUpWaves * 8 * 64];
  __shared__ Plan plan;
  static_assert(sizeof(red) >= sizeof(uint32_t) * kMaxExperts, "the plan's scratch shares red");
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, q4 = lane >> 4;
  const int wave = uniform(tid >> 6);
  const int t0 = blockIdx.y * p.tokens;
  const int tokens = min(p.tokens, p.m - t0);
  make_plan(p, t0, tokens * p.top_k, plan, reinterpret_cast<int16_t*>(ring), reinterpret_cast<uint32_t*>(red));
  const int tiles = p.inter >> 4, nkb = p.hidden >> 7, nb = p.inter >> 7, nw = words<UE8M0>(nkb);
  const int rounds = (nkb + kUpWaves - 1) / kUpWaves;
  const int units = uniform(plan.touched) * tiles;
  const int u0 = uniform((int)((int64_t)units * blockIdx.x / gridDim.x));
  const int u1 = uniform((int)((int64_t)units * (blockIdx.x + 1) / gridDim.x));
  if (u0 >= u1) return;

  uint8_t* my_ring = ring + wave * D * S::kBytes;
  const uint32_t my_lds = (uint32_t)uniform((int)(uintptr_t)(lds_ptr_t)my_ring);
  const __amdgpu_buffer_rsrc_t rx = uniform_rsrc(p.x + (int64_t)t0 * p.ldx, (uint32_t)((tokens - 1) * p.ldx + p.hidden));
  const __amdgpu_buffer_rsrc_t rsx =
      uniform_rsrc(static_cast<const uint32_t*>(p.sfx) + t0, (uint32_t)(((nw - 1) * p.ld_sfx + tokens) * 4));
  const uint32_t w_off = (uint32_t)(lane >> 3) * p.hidden + tile_chunk(lane);

  // Where the next stage to load is: pass (expert i, tile t, first token g0), round it.
  int li = uniform(u0 / tiles), lt = u0 - li * tiles, lg0 = 0, lit = 0, left = u1 - u0, ln = 0, slot = 0;
  const uint8_t* lw = nullptr;
  const uint32_t* lsw = nullptr;
  uint32_t x_off[NG][2], sx_off;
  auto pass = [&]() __attribute__((always_inline)) {
    const int e = uniform((int)plan.expert[li]), first = uniform((int)plan.start[li]);
    ln = uniform((int)plan.start[li + 1]) - first;
    lw = p.w13 + ((int64_t)e * 2 * p.inter + lt * 16) * p.hidden;
    lsw = static_cast<const uint32_t*>(p.sf13) + ((int64_t)e * 2 * nb + (lt >> 3)) * nw;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = lg0 + 16 * g + 8 * h + (lane >> 3);
        x_off[g][h] = c < ln ? (uint32_t)(plan.order[first + c] / p.top_k) * (uint32_t)p.ldx + tile_chunk(lane) : kNowhere;
      }
    const int c = lg0 + lane;
    sx_off = lane < 16 * NG && c < ln ? (uint32_t)(plan.order[first + c] / p.top_k) * 4 : kNowhere;
  };
  auto load = [&]() __attribute__((always_inline)) {
    const int kb = wave + lit * kUpWaves;
    const uint32_t k = kb < nkb ? (uint32_t)kb * 128 : kNowhere;
    const uint32_t lds = (uint32_t)uniform((int)(my_lds + slot * S::kBytes));
    const __amdgpu_buffer_rsrc_t rg = uniform_rsrc(lw, 16u * p.hidden);
    const __amdgpu_buffer_rsrc_t ru = uniform_rsrc(lw + (int64_t)p.inter * p.hidden, 16u * p.hidden);
    const __amdgpu_buffer_rsrc_t rsw = uniform_rsrc(lsw, (uint32_t)((nb + 1) * nw * 4));
    to_lds<16, true>(rg, lds, w_off + k);
    to_lds<16, true>(rg, lds + 1024, w_off + 8u * p.hidden + k);
    to_lds<16, true>(ru, lds + 2048, w_off + k);
    to_lds<16, true>(ru, lds + 3072, w_off + 8u * p.hidden + k);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) to_lds<16, false>(rx, lds + S::kX + 2048 * g + 1024 * h, x_off[g][h] + k);
    const uint32_t wd = kb < nkb ? (uint32_t)word_of<UE8M0>(kb) : kNowhere;
    to_lds<4, false>(rsx, lds + S::kSx, kb < nkb && sx_off != kNowhere ? sx_off + wd * (uint32_t)p.ld_sfx * 4 : kNowhere);
    to_lds<4, false>(rsw, lds + S::kSw, kb < nkb && lane < 2 ? (lane * nb * nw + wd) * 4 : kNowhere);
    slot = slot + 1 == D ? 0 : slot + 1;
    if (++lit < rounds) return;
    lit = 0;
    lg0 += 16 * NG;
    if (lg0 >= ln) {
      lg0 = 0;
      --left;
      if (++lt == tiles) lt = 0, ++li;
    }
    if (left > 0) pass();
  };
  pass();
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (left > 0) load();

  int at = 0;
  for (int u = u0; u < u1; ++u) {
    const int i = uniform(u / tiles), col0 = (u - i * tiles) * 16;
    const int first = uniform((int)plan.start[i]), n = uniform((int)plan.start[i + 1]) - first;
    for (int g0 = 0; g0 < n; g0 += 16 * NG) {
      f32x4 ag[NG], au[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) ag[g] = au[g] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int it = 0; it < rounds; ++it) {
        if (left > 0) wait_loads<(D - 1) * S::kLoads>();
        else wait_loads<0>();
        const uint8_t* st = my_ring + at * S::kBytes;
        const int kb = wave + it * kUpWaves;
        const i32x8 fg = read_frag(st, r16, q4), fu = read_frag(st + 2048, r16, q4);
        const uint32_t* sw = reinterpret_cast<const uint32_t*>(st + S::kSw);
        const float sg = scale_of<UE8M0>(sw[0], kb), su = scale_of<UE8M0>(sw[1], kb);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (g > 0 && g0 + 16 * g >= n) break;
          const i32x8 fx = read_frag(st + S::kX + 2048 * g, r16, q4);
          const float sx = scale_of<UE8M0>(reinterpret_cast<const uint32_t*>(st + S::kSx)[16 * g + r16], kb);
          const f32x4 pg = mfma_fp8(fg, fx), pu = mfma_fp8(fu, fx);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            ag[g][r] = __builtin_fmaf(pg[r], sx * sg, ag[g][r]);
            au[g][r] = __builtin_fmaf(pu[r], sx * su, au[g][r]);
          }
        }
        wait_lds();
        if (left > 0) load();
        at = at + 1 == D ? 0 : at + 1;
      }
      // the waves' sums meet group by group: red[wave][gate 0..3, up 0..3][lane]
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (g > 0 && g0 + 16 * g >= n) break;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          red[(wave * 8 + r) * 64 + lane] = ag[g][r];
          red[(wave * 8 + 4 + r) * 64 + lane] = au[g][r];
        }
        __syncthreads();
        if (g % kUpWaves == wave && g0 + 16 * g + r16 < n) {
          bf16x4 a;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float vg = 0.f, vu = 0.f;
#pragma unroll
            for (int k = 0; k < kUpWaves; ++k) {
              vg += red[(k * 8 + r) * 64 + lane];
              vu += red[(k * 8 + 4 + r) * 64 + lane];
            }
            a[r] = (__bf16)(silu(vg) * vu);
          }
          const int pair = plan.order[first + g0 + 16 * g + r16];
          *reinterpret_cast<bf16x4*>(p.act + ((int64_t)t0 * p.top_k + pair) * p.inter + col0 + 4 * q4) = a;
        }
        __syncthreads();
      }
    }
  }
}

// Stage of the down kernel: R weight tiles, NG tiles of 16 tokens x 128 BF16 values of a,
// the block scale.
template <int R, int NG>
struct DownStage {
  static constexpr int kA = 2048 * R, kSw = kA + 4096 * NG, kBytes = kSw + 256;
  static constexpr int kLoads = 2 * R + 4 * NG + 1;
};

// grid: (hidden / (16 * R), chunks).  Dynamic LDS: the sums, slots * pairs * 16 * R floats.
template <bool UE8M0, int R, int NG, int W, int D>
__global__ void __launch_bounds__(W * 64) down_kernel(const Params p) {
  using S = DownStage<R, NG>;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[W * D * S::kBytes];
  __shared__ Plan plan;
  __shared__ int16_t id[kPairs];
  extern __shared__ __attribute__((aligned(16))) float sums[];  // [K range][pair][16 * R]
  static_assert(sizeof(ring) >= sizeof(uint32_t) * kMaxExperts, "the plan's scratch shares the ring");
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, q4 = lane >> 4;
  const int wave = uniform(tid >> 6);
  const int t0 = blockIdx.y * p.tokens;
  const int tokens = min(p.tokens, p.m - t0), pairs = tokens * p.top_k;
  make_plan(p, t0, pairs, plan, id, reinterpret_cast<uint32_t*>(ring));
  const int col0 = blockIdx.x * 16 * R;
  const int nkb = p.inter >> 7, nw = words<UE8M0>(nkb);
  const int touched = uniform(plan.touched);
  // K ranges per expert: as many as balance the waves best, a piece costing two K blocks beside its own
  int split = 1, best = 0x7fffffff;
  for (int s = 1; s <= p.slots && s <= nkb; s *= 2) {
    const int cost = ((touched * s + W - 1) / W) * ((nkb + s - 1) / s + 2);
    if (cost < best) best = cost, split = s;
  }
  const int pieces = touched * split;

  uint8_t* my_ring = ring + wave * D * S::kBytes;
  const uint32_t my_lds = (uint32_t)uniform((int)(uintptr_t)(lds_ptr_t)my_ring);
  const __amdgpu_buffer_rsrc_t ra =
      uniform_rsrc(p.act + (int64_t)t0 * p.top_k * p.inter, (uint32_t)pairs * p.inter * 2);
  const uint32_t w_off = (uint32_t)(lane >> 3) * p.inter + tile_chunk(lane);

  // Where the next stage to load is: piece lu (expert, K range), first token lg0, K block lkb.
  int lu = wave, lg0 = 0, lkb = 0, lkb0 = 0, lkb1 = 0, ln = 0, slot = 0;
  const uint8_t* lw = nullptr;
  const uint32_t* lsw = nullptr;
  uint32_t a_off[NG][4];
  auto pass = [&]() __attribute__((always_inline)) {
    const int i = uniform(lu / split), s = lu - i * split;
    const int e = uniform((int)plan.expert[i]), first = uniform((int)plan.start[i]);
    ln = uniform((int)plan.start[i + 1]) - first;
    lkb0 = lkb = uniform(nkb * s / split);
    lkb1 = uniform(nkb * (s + 1) / split);
    lw = p.w2 + ((int64_t)e * p.hidden + col0) * p.inter;
    lsw = static_cast<const uint32_t*>(p.sf2) + ((int64_t)e * (p.hidden >> 7) + (col0 >> 7)) * nw;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int row = 4 * h + (lane >> 4), c = lg0 + 16 * g + row;
        a_off[g][h] = c < ln ? (uint32_t)plan.order[first + c] * (uint32_t)p.inter * 2 + (((lane & 15) ^ row) << 4) : kNowhere;
      }
  };
  auto load = [&]() __attribute__((always_inline)) {
    const uint32_t lds = (uint32_t)uniform((int)(my_lds + slot * S::kBytes));
    const __amdgpu_buffer_rsrc_t rw = uniform_rsrc(lw, (uint32_t)(16 * R) * p.inter);
    const __amdgpu_buffer_rsrc_t rsw = uniform_rsrc(lsw, (uint32_t)nw * 4);
#pragma unroll
    for (int r = 0; r < 2 * R; ++r) to_lds<16, true>(rw, lds + 1024 * r, w_off + (uint32_t)(8 * r) * p.inter + lkb * 128);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < 4; ++h) to_lds<16, false>(ra, lds + S::kA + 4096 * g + 1024 * h, a_off[g][h] + lkb * 256);
    to_lds<4, false>(rsw, lds + S::kSw, lane == 0 ? word_of<UE8M0>(lkb) * 4 : kNowhere);
    slot = slot + 1 == D ? 0 : slot + 1;
    if (++lkb < lkb1) return;
    lg0 += 16 * NG;
    if (lg0 >= ln) lg0 = 0, lu += W;
    if (lu < pieces) pass();
  };
  if (lu < pieces) pass();
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (lu < pieces) load();

  int at = 0;
  for (int u = wave; u < pieces; u += W) {
    const int i = uniform(u / split), s = u - i * split;
    const int first = uniform((int)plan.start[i]), n = uniform((int)plan.start[i + 1]) - first;
    const int kb0 = uniform(nkb * s / split), kb1 = uniform(nkb * (s + 1) / split);
    for (int g0 = 0; g0 < n; g0 += 16 * NG) {
      f32x4 acc[NG][R];
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[g][r] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int kb = kb0; kb < kb1; ++kb) {
        if (lu < pieces) wait_loads<(D - 1) * S::kLoads>();
        else wait_loads<0>();
        const uint8_t* st = my_ring + at * S::kBytes;
        const float f = scale_of<UE8M0>(*reinterpret_cast<const uint32_t*>(st + S::kSw), kb);
        bf16x8 b[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const i32x8 w = read_frag(st + 2048 * r, r16, q4);
#pragma unroll
          for (int c = 0; c < 4; ++c) b[r][c] = widen(w[2 * c], w[2 * c + 1]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (g > 0 && g0 + 16 * g >= n) break;
          const uint8_t* row = st + S::kA + 4096 * g + r16 * 256;
          bf16x8 a[4];  // K chunks in the order of the weight fragment's
#pragma unroll
          for (int c = 0; c < 4; ++c)
            a[c] = *reinterpret_cast<const bf16x8*>(row + (((2 * q4 + (c & 1) + 8 * (c >> 1)) ^ r16) << 4));
#pragma unroll
          for (int r = 0; r < R; ++r) {
            f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[r][c], a[c], part, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[g][r][k] = __builtin_fmaf(part[k], f, acc[g][r][k]);
          }
        }
        wait_lds();
        if (lu < pieces) load();
        at = at + 1 == D ? 0 : at + 1;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (g0 + 16 * g + r16 >= n) continue;
        const int pair = plan.order[first + g0 + 16 * g + r16];
#pragma unroll
        for (int r = 0; r < R; ++r)
          *reinterpret_cast<f32x4*>(&sums[((s * pairs + pair) * R + r) * 16 + 4 * q4]) = acc[g][r];
      }
    }
  }
  __syncthreads();
  for (int o = tid; o < tokens * 16 * R; o += W * 64) {
    const int t = o / (16 * R), c = o % (16 * R);
    float v = 0.f;
    for (int j = 0; j < p.top_k; ++j) {
      const int pair = t * p.top_k + j;
      if (id[pair] < 0) continue;
      float y = 0.f;
      for (int s = 0; s < split; ++s) y += sums[(s * pairs + pair) * 16 * R + c];
      v = __builtin_fmaf(p.tw[(int64_t)(t0 + t) * p.top_k + j], y, v);
    }
    const __bf16 b = (__bf16)v;
    p.out[(int64_t)(t0 + t) * p.ld_out + col0 + c] = __builtin_bit_cast(uint16_t, b);
  }
}

inline bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int kLds = 160 * 1024;  // LDS of a CU

template <bool UE8M0, int NG, int D>
void launch_up(const Params& p, dim3 grid, hipStream_t stream) {
  hipLaunchKernelGGL((gate_up_kernel<UE8M0, NG, D>), grid, dim3(kUpWaves * 64), 0, stream, p);
}

// Tries R * 16 columns per workgroup; false where the sums of `pairs` pairs do not fit in LDS.
template <bool UE8M0, int R, int NG, int W, int D>
bool launch_down(Params p, int chunks, int pairs, hipStream_t stream) {
  const int room = kLds - W * D * DownStage<R, NG>::kBytes - (int)sizeof(Plan) - 2 * kPairs - 1024;
  p.slots = std::min(16, room / (pairs * 64 * R));
  if (p.slots < 1) return false;
  const dim3 grid(p.hidden / (16 * R), chunks);
  hipLaunchKernelGGL((down_kernel<UE8M0, R, NG, W, D>), grid, dim3(W * 64), p.slots * pairs * 64 * R, stream, p);
  return true;
}

template <bool UE8M0>
void launch(const Params& p, int chunks, int pairs, hipStream_t stream) {
  // tokens per expert if all ids are of this device: how many groups of 16 a pass takes
  const int cus = dg_get_num_cus() > 0 ? dg_get_num_cus() : 256;
  const int64_t units = (int64_t)std::min(pairs, p.experts) * (p.inter / 16);
  const int each = pairs / p.experts;
  const auto grid = [&](int per_cu) { return dim3((unsigned)std::min<int64_t>(units, (int64_t)cus * per_cu), chunks); };
  if (each <= 8) launch_up<UE8M0, 1, UPD>(p, grid(UPG), stream);
  else if (each <= 20) launch_up<UE8M0, 2, 2>(p, grid(2), stream);
  else launch_up<UE8M0, 4, 2>(p, grid(1), stream);
  const bool wide = p.hidden >= RH;
  if (each <= 8) {
    if (!(wide && launch_down<UE8M0, 2, 1, 8, 2>(p, chunks, pairs, stream))) launch_down<UE8M0, 1, 1, 8, 2>(p, chunks, pairs, stream);
  } else {
    if (!(wide && launch_down<UE8M0, 2, 2, 4, 2>(p, chunks, pairs, stream))) launch_down<UE8M0, 1, 2, 4, 2>(p, chunks, pairs, stream);
  }
}

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
  // offsets inside a chunk of tokens are 32-bit
  const int64_t chunk_tokens = std::min(m, kPairs / top_k);
  if (chunk_tokens * ldx >= kNowhere || (int64_t)(hidden / 128) * ld_sfx * 4 >= kNowhere ||
      (int64_t)32 * hidden >= kNowhere || (int64_t)kPairs * inter * 2 >= kNowhere)
    return DG_ERROR_NOT_SUPPORTED;
  if (workspace == nullptr || !aligned_to(workspace, 256) ||
      workspace_bytes < dg_get_moe_workspace_size(m, top_k, inter))
    return DG_ERROR_WORKSPACE;
  Params p{static_cast<const uint8_t*>(x), sfx, static_cast<const uint8_t*>(w13), sf13,
           static_cast<const uint8_t*>(w2), sf2, ids, tw, static_cast<__bf16*>(workspace),
           static_cast<uint16_t*>(out), ldx, ld_sfx, ld_out, m, top_k, experts, hidden, inter, kPairs / top_k, 1};
  const int chunks = (m + p.tokens - 1) / p.tokens;
  if (chunks > 65535) return DG_ERROR_NOT_SUPPORTED;
  const int pairs = (m < p.tokens ? m : p.tokens) * top_k;
  if (ue8m0) launch<true>(p, chunks, pairs, stream);
  else launch<false>(p, chunks, pairs, stream);
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
