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
// once from HBM, and everything else is arranged around that.
//
//   * gate/up kernel: a workgroup takes 16 gate and the matching 16 up rows of a
//     touched expert at a time (a unit; 32 and 32 with more than 16 tokens, whose tiles are
//     then read half as often: 64 tokens 76 us, 83 us), its four waves split K, and one
//     v_mfma_f32_16x16x128_f8f6f4 covers 16 rows, 16 tokens and one 128-K scale
//     block.  The waves' partial sums meet in LDS and a is written once per (token,
//     slot) in BF16.  (The second product then takes BF16; the composed path would
//     store a in E4M3, 4 bits less.  The rounding costs the result as much as the
//     rounding of the output itself.)
//   * down kernel: a workgroup owns 8, 16 or 32 output columns of all tokens; its
//     waves take (expert, K range) pieces in turn.  E4M3 is exact in BF16, so W2
//     fragments are widened in registers and the block scale is applied to the
//     FP32 sum of each 128 K values.  Each (token, slot) leaves its own sums in
//     LDS, and the slots are added in the order of j: no atomics on results, the
//     same bits every time.
//   * both kernels bring their operands with direct global->LDS loads into rings of
//     K-block stages, one ring per wave, the next stages on their way while one is
//     multiplied.  A load instruction brings whole 128-byte lines (8 rows), which is
//     what lets the weights be marked as streaming: reading 235 MB of gate/up weights
//     takes 35 us that way, 40 us unmarked; fragments loaded straight into registers, 64
//     bytes of a line at a time, took 43 us unmarked and 50 us marked.
//   * which tokens go to which expert is worked out by every workgroup from ids (at
//     most kPairs (token, slot) pairs per chunk of tokens; larger batches are further
//     grid rows), about 1.5 us, so there is no planning kernel and no host work.
//
// Measured (both kernels, weights not in any cache; reads alone reach 7.0 TB/s):
//     1 token, 8 of 16 experts of 7168 x 2048       60 us   5.9 TB/s (38 + 22 us of kernels)
//     9 tokens, top 8 of 64 experts of 4096 x 1024  92 us   6.1 TB/s
//     64 tokens, top 4 of 16 experts of 7168 x 2048 128 us  5.5 TB/s (a's tiles fill the down
//                                                   kernel's rings: fewer stages in flight)
//     37 tokens, 32 of 128 experts of 2048 x 1408   47 us   4.9 TB/s (the down kernel 3.9: a
//                                                   workgroup's 8 columns bring in half as much
//                                                   of a as of W2)
// Where every workgroup's rows of a outweigh its columns of W2 (small layers, or few experts with
// many tokens each) the layer is far from its bytes: 20 tokens, top 8 of 10 experts of 1280 x 1152
// take 27 us (13 + 16 us of kernels) for 6 us of weights.
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
constexpr int kDownWaves = 16;

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
  int ring;    // down kernel: bytes of LDS for the rings
};

// The pairs of one chunk by expert: expert of the i-th touched one, its first
// place in `order` and, in `order`, the pairs (token in chunk, slot).
// Pairs whose id is outside [0, experts) are in no list.
struct Plan {
  uint16_t order[kPairs];  // token << 6 | slot
  uint16_t expert[kPairs];
  uint16_t start[kPairs + 1];
  int touched;
  int most;                // tokens of the fullest expert
  int passes24, passes32;  // over all experts' tokens, 24 or 32 at a time
};

static_assert(kPairs <= 1 << 10 && kMaxTopK <= 64, "order[] packs a token and a slot into 16 bits");
__device__ __forceinline__ int pair_of(const Params& p, int place) { return (place >> 6) * p.top_k + (place & 63); }

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, true);
}
// Sum of v over this lane and those below it: shifts of 1, 2, 4 and 8 inside each 16 lanes, then
// the last lane of each 16 to the next, and of the lower half to the upper.
__device__ __forceinline__ int scan(int v) {
  v += dpp<0x111, 0xf>(v);
  v += dpp<0x112, 0xf>(v);
  v += dpp<0x114, 0xf>(v);
  v += dpp<0x118, 0xf>(v);
  v += dpp<0x142, 0xa>(v);
  return v + dpp<0x143, 0xc>(v);
}

// Sorts the chunk's pairs by expert; id[pair] becomes the pair's expert or -1.
// `count` holds kMaxExperts words of scratch.  The order of an expert's own
// pairs depends on timing, but no result does: a pair's place only says which
// MFMA column computes it.
template <int THREADS>
__device__ __forceinline__ void make_plan(const Params& p, int t0, int pairs, Plan& plan, int16_t* id,
                                          uint32_t* count) {
  const int tid = threadIdx.x;
  constexpr int PER = (kPairs + THREADS - 1) / THREADS;
  int mine[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = j * THREADS + tid;
    const int e = i < pairs ? p.ids[(int64_t)t0 * p.top_k + i] : -1;
    mine[j] = e >= 0 && e < p.experts ? e : -1;
  }
  for (int e = tid; e < p.experts; e += THREADS) count[e] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = j * THREADS + tid;
    if (i < pairs) id[i] = (int16_t)mine[j];
    if (mine[j] >= 0) atomicAdd(&count[mine[j]], 1u);
  }
  __syncthreads();
  if (tid < 64) {  // one wave: touched experts in order of their number, and where their pairs start
    int touched = 0, start = 0, most = 0, passes24 = 0, passes32 = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
      const int e = e0 + tid;
      const int c = e < p.experts ? (int)count[e] : 0;
      const uint64_t mask = __ballot(c > 0);
      const int before = scan(c);
      if (c > 0) {
        const int i = touched + __popcll(mask & ((1ull << tid) - 1));
        plan.expert[i] = (uint16_t)e;
        plan.start[i] = (uint16_t)(start + before - c);
        count[e] = (uint32_t)(start + before - c);  // next free place of this expert
      }
      touched += __popcll(mask);
      start += __builtin_amdgcn_readlane(before, 63);
      most = max(most, c);
      passes24 += (int)((uint32_t)(c + 23) / 24u);
      passes32 += (c + 31) >> 5;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) most = max(most, __shfl_xor(most, off));
    passes24 = scan(passes24);
    passes32 = scan(passes32);
    if (tid == 63) {
      plan.touched = touched;
      plan.most = most;
      plan.passes24 = passes24;
      plan.passes32 = passes32;
      plan.start[touched] = (uint16_t)start;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (mine[j] >= 0) {
      const int pair = j * THREADS + tid, token = pair / p.top_k;
      plan.order[atomicAdd(&count[mine[j]], 1u)] = (uint16_t)(token << 6 | (pair - token * p.top_k));
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
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
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
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds"
                 : : "v"(off), "s"(r), "s"(lds) : "memory", "m0");
  else if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 : : "v"(off), "s"(r), "s"(lds) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 : : "v"(off), "s"(r), "s"(lds) : "memory", "m0");
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

// Stage of the gate/up kernel: RT gate tiles, RT up tiles, NG token tiles, and a word per
// lane: the tokens' scales, and in the last two the block scales (with 64 tokens, whose
// scales take them all, in words of their own).
template <int NG, int RT>
struct UpStage {
  static constexpr int kUp = 2048 * RT, kX = 2 * kUp, kSx = kX + 2048 * NG, kSw = kSx + (NG < 4 ? 248 : 256);
  static constexpr int kBytes = kSx + (NG < 4 ? 256 : 512);
  static constexpr int kLoads = 4 * RT + 2 * NG + 2;
};

// A unit is one touched expert's tile of 16 * RT columns of a; workgroups take contiguous
// ranges of units.  An expert with more than 16 * NG tokens takes several passes.
// D: stages of a ring.  grid: (workgroups, chunks).
template <bool UE8M0, int NG, int RT, int D>
__global__ void __launch_bounds__(kUpWaves * 64) gate_up_kernel(const Params p) {
  using S = UpStage<NG, RT>;
  constexpr int XG = NG * RT <= kUpWaves ? NG : 1;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kUpWaves * D * S::kBytes];
  // the waves' sums, XG token groups at a time: [wave][token group, row tile][gate, up][lane]
  __shared__ __attribute__((aligned(16))) f32x4 red[kUpWaves * XG * RT * 2 * 64];
  __shared__ Plan plan;
  static_assert(sizeof(red) >= sizeof(uint32_t) * kMaxExperts, "the plan's scratch shares red");
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, q4 = lane >> 4;
  const int wave = uniform(tid >> 6);
  const int t0 = blockIdx.y * p.tokens;
  const int tokens = min(p.tokens, p.m - t0);
  make_plan<kUpWaves * 64>(p, t0, tokens * p.top_k, plan, reinterpret_cast<int16_t*>(ring),
                           reinterpret_cast<uint32_t*>(red));
  const int tiles = p.inter / (16 * RT), nkb = p.hidden >> 7, nb = p.inter >> 7, nw = words<UE8M0>(nkb);
  const int rounds = (nkb + kUpWaves - 1) / kUpWaves;
  const int units = uniform(plan.touched) * tiles;
  const int each = units / (int)gridDim.x, more = units - each * (int)gridDim.x;  // the first `more` take one more
  const int u0 = uniform((int)blockIdx.x * each + min((int)blockIdx.x, more));
  const int u1 = u0 + each + ((int)blockIdx.x < more ? 1 : 0);
  if (u0 >= u1) return;

  uint8_t* my_ring = ring + wave * D * S::kBytes;
  const uint32_t my_lds = (uint32_t)uniform((int)(uintptr_t)(lds_ptr_t)my_ring);
  const __amdgpu_buffer_rsrc_t rx =
      uniform_rsrc(p.x + (int64_t)t0 * p.ldx, (uint32_t)((tokens - 1) * p.ldx + p.hidden));
  const __amdgpu_buffer_rsrc_t rsx =
      uniform_rsrc(static_cast<const uint32_t*>(p.sfx) + t0, (uint32_t)(((nw - 1) * p.ld_sfx + tokens) * 4));
  const uint32_t w_off = (uint32_t)(lane >> 3) * p.hidden + tile_chunk(lane);

  // Where the next stage to load is: pass (expert i, tile t, first token g0), round it.
  const int i0 = uniform(u0 / tiles);
  int li = i0, lt = u0 - i0 * tiles, lg0 = 0, lit = 0, left = u1 - u0, ln = 0, slot = 0;
  const uint8_t* lw = nullptr;
  const uint32_t* lsw = nullptr;
  uint32_t x_off[NG][2], sx_off;
  auto pass = [&]() __attribute__((always_inline)) {
    const int e = uniform((int)plan.expert[li]), first = uniform((int)plan.start[li]);
    ln = uniform((int)plan.start[li + 1]) - first;
    lw = p.w13 + ((int64_t)e * 2 * p.inter + lt * 16 * RT) * p.hidden;
    lsw = static_cast<const uint32_t*>(p.sf13) + ((int64_t)e * 2 * nb + (lt * RT >> 3)) * nw;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = lg0 + 16 * g + 8 * h + (lane >> 3);
        x_off[g][h] = c < ln ? (uint32_t)(plan.order[first + c] >> 6) * (uint32_t)p.ldx + tile_chunk(lane) : kNowhere;
      }
    const int c = lg0 + lane;
    sx_off = lane < 16 * NG && c < ln ? (uint32_t)(plan.order[first + c] >> 6) * 4 : kNowhere;
  };
  auto load = [&]() __attribute__((always_inline)) {
    const int kb = wave + lit * kUpWaves;
    const uint32_t k = kb < nkb ? (uint32_t)kb * 128 : kNowhere;
    const uint32_t lds = (uint32_t)uniform((int)(my_lds + slot * S::kBytes));
    const __amdgpu_buffer_rsrc_t rg = uniform_rsrc(lw, 16u * RT * p.hidden);
    const __amdgpu_buffer_rsrc_t ru = uniform_rsrc(lw + (int64_t)p.inter * p.hidden, 16u * RT * p.hidden);
    const __amdgpu_buffer_rsrc_t rsw = uniform_rsrc(lsw, (uint32_t)((nb + 1) * nw * 4));
#pragma unroll
    for (int h = 0; h < 2 * RT; ++h) to_lds<16, true>(rg, lds + 1024 * h, w_off + 8u * h * p.hidden + k);
#pragma unroll
    for (int h = 0; h < 2 * RT; ++h) to_lds<16, true>(ru, lds + S::kUp + 1024 * h, w_off + 8u * h * p.hidden + k);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) to_lds<16, false>(rx, lds + S::kX + 2048 * g + 1024 * h, x_off[g][h] + k);
    const uint32_t wd = kb < nkb ? (uint32_t)word_of<UE8M0>(kb) : kNowhere;
    // (a lane's word lies at the address given and four bytes per lane, whichever lanes take part)
    const uint32_t sx_at = kb < nkb && sx_off != kNowhere ? sx_off + wd * (uint32_t)p.ld_sfx * 4 : kNowhere;
    if constexpr (NG < 4) {
      if (lane < 62) to_lds<4, false>(rsx, lds + S::kSx, sx_at);
      else to_lds<4, false>(rsw, lds + S::kSx, kb < nkb ? ((lane - 62) * nb * nw + wd) * 4 : kNowhere);
    } else {
      to_lds<4, false>(rsx, lds + S::kSx, sx_at);
      to_lds<4, false>(rsw, lds + S::kSw, kb < nkb && lane < 2 ? (lane * nb * nw + wd) * 4 : kNowhere);
    }
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

  int at = 0, i = i0, t = u0 - i0 * tiles;
  for (int u = u0; u < u1; ++u) {
    const int col0 = t * 16 * RT;
    const int first = uniform((int)plan.start[i]), n = uniform((int)plan.start[i + 1]) - first;
    for (int g0 = 0; g0 < n; g0 += 16 * NG) {
      f32x4 ag[NG][RT], au[NG][RT];
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int v = 0; v < RT; ++v) ag[g][v] = au[g][v] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int it = 0; it < rounds; ++it) {
        if (left > 0) wait_loads<(D - 1) * S::kLoads>();
        else wait_loads<0>();
        const uint8_t* st = my_ring + at * S::kBytes;
        const int kb = wave + it * kUpWaves;
        i32x8 fg[RT], fu[RT];
#pragma unroll
        for (int v = 0; v < RT; ++v) {
          fg[v] = read_frag(st + 2048 * v, r16, q4);
          fu[v] = read_frag(st + S::kUp + 2048 * v, r16, q4);
        }
        const uint32_t* sw = reinterpret_cast<const uint32_t*>(st + S::kSw);
        const float sg = scale_of<UE8M0>(sw[0], kb), su = scale_of<UE8M0>(sw[1], kb);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (g > 0 && g0 + 16 * g >= n) break;
          const i32x8 fx = read_frag(st + S::kX + 2048 * g, r16, q4);
          const float sx = scale_of<UE8M0>(reinterpret_cast<const uint32_t*>(st + S::kSx)[16 * g + r16], kb);
#pragma unroll
          for (int v = 0; v < RT; ++v) {
            const f32x4 pg = mfma_fp8(fg[v], fx), pu = mfma_fp8(fu[v], fx);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              ag[g][v][r] = __builtin_fmaf(pg[r], sx * sg, ag[g][v][r]);
              au[g][v][r] = __builtin_fmaf(pu[r], sx * su, au[g][v][r]);
            }
          }
        }
        wait_lds();
        if (left > 0) load();
        at = at + 1 == D ? 0 : at + 1;
      }
      // the waves' sums meet in LDS, where one wave adds each tile's
#pragma unroll
      for (int x0 = 0; x0 < NG; x0 += XG) {
        if (x0 > 0 && g0 + 16 * x0 >= n) break;
#pragma unroll
        for (int g = 0; g < XG; ++g)
#pragma unroll
          for (int v = 0; v < RT; ++v) {
            if (g > 0 && g0 + 16 * g >= n) break;
            red[((wave * XG + g) * RT + v) * 128 + lane] = ag[x0 + g][v];
            red[((wave * XG + g) * RT + v) * 128 + 64 + lane] = au[x0 + g][v];
          }
        __syncthreads();
#pragma unroll
        for (int g = 0; g < XG; ++g)
#pragma unroll
          for (int v = 0; v < RT; ++v) {
            const int c = g0 + 16 * (x0 + g) + r16;
            if (((x0 + g) * RT + v) % kUpWaves != wave || c >= n) continue;
            f32x4 vg = {0.f, 0.f, 0.f, 0.f}, vu = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kUpWaves; ++k) {
              vg += red[((k * XG + g) * RT + v) * 128 + lane];
              vu += red[((k * XG + g) * RT + v) * 128 + 64 + lane];
            }
            bf16x4 a;
#pragma unroll
            for (int r = 0; r < 4; ++r) a[r] = (__bf16)(silu(vg[r]) * vu[r]);
            const int pair = pair_of(p, plan.order[first + c]);
            *reinterpret_cast<bf16x4*>(p.act + ((int64_t)t0 * p.top_k + pair) * p.inter + col0 + 16 * v + 4 * q4) = a;
          }
        __syncthreads();
      }
    }
    if (++t == tiles) t = 0, ++i;
  }
}

// Down kernel.  A stage holds the 128-K block of RB weight rows, 4 * AL tokens x 128 BF16
// values of a, and the block scale.
template <int RB, int AL>
struct DownStage {
  static constexpr int kA = 128 * RB, kSw = kA + 1024 * AL, kBytes = kSw + 16;
  static constexpr int kLoads = RB / 8 + AL + 1;
};

struct DownWork {
  int t0, pairs, col0;
  int split;         // log2 of the K ranges per expert
  int waves, depth;  // waves that stream, stages of their rings
};

// What the waves do between the plan and the weighted sum: wave w takes pieces (expert, K
// range) w, w + waves, ..., each for 4 * AL of the expert's tokens at a time.
template <bool UE8M0, int RB, int AL>
__device__ __forceinline__ void down_stream(const Params& p, const Plan& plan, const DownWork& k, uint8_t* ring,
                                            float* sums) {
  using S = DownStage<RB, AL>;
  constexpr int T = 4 * AL, R = (RB + 15) / 16, NG = (T + 15) / 16;
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, q4 = lane >> 4;
  const int wave = uniform(tid >> 6);
  const int nkb = p.inter >> 7, nw = words<UE8M0>(nkb);
  const int pieces = uniform(plan.touched) << k.split;
  if (wave >= k.waves) return;
  uint8_t* my_ring = ring + wave * k.depth * S::kBytes;
  const uint32_t my_lds = (uint32_t)uniform((int)(uintptr_t)(lds_ptr_t)my_ring);
  const __amdgpu_buffer_rsrc_t ra =
      uniform_rsrc(p.act + (int64_t)k.t0 * p.top_k * p.inter, (uint32_t)k.pairs * p.inter * 2);
  const uint32_t w_off = (uint32_t)(lane >> 3) * p.inter + tile_chunk(lane);

  // Where the next stage to load is: piece lu, first token lg0, K block lkb.
  int lu = wave, lg0 = 0, lkb = 0, lkb1 = 0, ln = 0, slot = 0;
  const uint8_t* lw = nullptr;
  const uint32_t* lsw = nullptr;
  uint32_t a_off[AL];
  auto pass = [&]() __attribute__((always_inline)) {
    const int i = lu >> k.split, s = lu - (i << k.split);
    const int e = uniform((int)plan.expert[i]), first = uniform((int)plan.start[i]);
    ln = uniform((int)plan.start[i + 1]) - first;
    lkb = nkb * s >> k.split;
    lkb1 = nkb * (s + 1) >> k.split;
    lw = p.w2 + ((int64_t)e * p.hidden + k.col0) * p.inter;
    lsw = static_cast<const uint32_t*>(p.sf2) + ((int64_t)e * (p.hidden >> 7) + (k.col0 >> 7)) * nw;
#pragma unroll
    for (int h = 0; h < AL; ++h) {
      const int row = 4 * h + (lane >> 4), c = lg0 + row;
      a_off[h] = c < ln ? (uint32_t)pair_of(p, plan.order[first + c]) * (uint32_t)p.inter * 2 +
                              (((lane ^ row) & 15) << 4)
                        : kNowhere;
    }
  };
  auto load = [&]() __attribute__((always_inline)) {
    const uint32_t lds = (uint32_t)uniform((int)(my_lds + slot * S::kBytes));
    const __amdgpu_buffer_rsrc_t rw = uniform_rsrc(lw, (uint32_t)RB * p.inter);
    const __amdgpu_buffer_rsrc_t rsw = uniform_rsrc(lsw, (uint32_t)nw * 4);
#pragma unroll
    for (int r = 0; r < RB / 8; ++r)
      to_lds<16, true>(rw, lds + 1024 * r, w_off + (uint32_t)(8 * r) * p.inter + lkb * 128);
#pragma unroll
    for (int h = 0; h < AL; ++h) to_lds<16, false>(ra, lds + S::kA + 1024 * h, a_off[h] + lkb * 256);
    if (lane == 0) to_lds<4, false>(rsw, lds + S::kSw, word_of<UE8M0>(lkb) * 4);
    slot = slot + 1 == k.depth ? 0 : slot + 1;
    if (++lkb < lkb1) return;
    lg0 += T;
    if (lg0 >= ln) lg0 = 0, lu += k.waves;
    if (lu < pieces) pass();
  };
  if (lu < pieces) pass();
  for (int d = 0; d < k.depth; ++d)
    if (lu < pieces) load();

  int at = 0;
  for (int u = wave; u < pieces; u += k.waves) {
    const int i = u >> k.split, s = u - (i << k.split);
    const int first = uniform((int)plan.start[i]), n = uniform((int)plan.start[i + 1]) - first;
    const int kb0 = nkb * s >> k.split, kb1 = nkb * (s + 1) >> k.split;
    for (int g0 = 0; g0 < n; g0 += T) {
      f32x4 acc[NG][R];
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[g][r] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int kb = kb0; kb < kb1; ++kb) {
        if (lu >= pieces) wait_loads<0>();
        else if (k.depth == 2) wait_loads<S::kLoads>();
        else if (k.depth == 3) wait_loads<2 * S::kLoads>();
        else wait_loads<3 * S::kLoads>();
        const uint8_t* st = my_ring + at * S::kBytes;
        const float f = scale_of<UE8M0>(*reinterpret_cast<const uint32_t*>(st + S::kSw), kb);
        bf16x8 b[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const i32x8 w = read_frag(st + 2048 * r, RB == 8 ? r16 & 7 : r16, q4);
#pragma unroll
          for (int c = 0; c < 4; ++c) b[r][c] = widen(w[2 * c], w[2 * c + 1]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (g > 0 && g0 + 16 * g >= n) break;
          // rows past the last token held repeat earlier ones: their columns are not stored
          const int row = 16 * g + (T - 16 * g >= 16 ? r16 : r16 & ((T & 15) - 1));
          const uint8_t* arow = st + S::kA + row * 256;
          bf16x8 a[4];  // K chunks in the order of the weight fragment's
#pragma unroll
          for (int c = 0; c < 4; ++c)
            a[c] = *reinterpret_cast<const bf16x8*>(arow + (((2 * q4 + (c & 1) + 8 * (c >> 1)) ^ (row & 15)) << 4));
#pragma unroll
          for (int r = 0; r < R; ++r) {
            f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[r][c], a[c], part, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[g][r][j] = __builtin_fmaf(part[j], f, acc[g][r][j]);
          }
        }
        wait_lds();
        if (lu < pieces) load();
        at = at + 1 == k.depth ? 0 : at + 1;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int c = 16 * g + r16;
        if (c >= T || g0 + c >= n || (RB == 8 && q4 >= 2)) continue;
        const int pair = pair_of(p, plan.order[first + g0 + c]);
#pragma unroll
        for (int r = 0; r < R; ++r)
          *reinterpret_cast<f32x4*>(&sums[(s * k.pairs + pair) * RB + 16 * r + 4 * q4]) = acc[g][r];
      }
    }
  }
}

// grid: (hidden / RB, chunks).  Dynamic LDS: the rings, then the sums ([K range][pair][RB]).
template <bool UE8M0, int RB>
__global__ void __launch_bounds__(kDownWaves * 64) down_kernel(const Params p) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  __shared__ Plan plan;
  __shared__ int16_t id[kPairs];
  __shared__ float tw[kPairs];
  static_assert(kDownWaves * 64 >= kPairs, "a thread for every pair");
  const int tid = threadIdx.x;
  float* sums = reinterpret_cast<float*>(lds + p.ring);
  DownWork k;
  k.t0 = blockIdx.y * p.tokens;
  const int tokens = min(p.tokens, p.m - k.t0);
  k.pairs = tokens * p.top_k;
  k.col0 = blockIdx.x * RB;
  const float my_tw = tid < k.pairs ? p.tw[(int64_t)k.t0 * p.top_k + tid] : 0.f;
  make_plan<kDownWaves * 64>(p, k.t0, k.pairs, plan, id, reinterpret_cast<uint32_t*>(lds));
  if (tid < kPairs) tw[tid] = my_tw;
  const int nkb = p.inter >> 7, touched = uniform(plan.touched), most = uniform(plan.most);
  // How many tokens' rows of a a stage holds: the fullest expert's, up to 32; past that 24 or 32, whichever
  // brings fewer bytes into LDS, each pass over an expert's tokens reading its weights and costing about
  // 3 KiB's time besides (8 experts with 43 tokens on average: 23 us with 24, 27 us with 32; 16 with 32: 144 and
  // 140 us).  (Several passes for few tokens: 32 experts with 3 on average 63 us, 59 us with one.)  The stage's
  // size decides how many waves have rings of at least two stages.  (Any number of waves: 64 tokens
  // 133 us, 136 us with powers of two.)
  const bool less = uniform(plan.passes24) * (128 * RB + 9216) < uniform(plan.passes32) * (128 * RB + 11264);
  const int al = most <= 4 ? 1 : most <= 8 ? 2 : most <= 16 ? 4 : most <= 24 || (most > 32 && less) ? 6 : 8;
  const int bytes = 128 * RB + 1024 * al + 16;
  const int stages = p.ring / bytes;
  k.waves = min(kDownWaves, stages / 2);
  k.depth = min(4, stages / k.waves);
  // K ranges per expert: as many as balance the waves best, a piece costing two K blocks beside its own
  k.split = 0;
  int best = 0x7fffffff;
  for (int s = 0; 1 << s <= p.slots && 1 << s <= nkb; ++s) {
    const int cost = (((touched << s) + k.waves - 1) / k.waves) * (((nkb + (1 << s) - 1) >> s) + 2);
    if (cost < best) best = cost, k.split = s;
  }
  switch (al) {
    case 1: down_stream<UE8M0, RB, 1>(p, plan, k, lds, sums); break;
    case 2: down_stream<UE8M0, RB, 2>(p, plan, k, lds, sums); break;
    case 4: down_stream<UE8M0, RB, 4>(p, plan, k, lds, sums); break;
    case 6: down_stream<UE8M0, RB, 6>(p, plan, k, lds, sums); break;
    default: down_stream<UE8M0, RB, 8>(p, plan, k, lds, sums); break;
  }
  __syncthreads();
  for (int o = tid; o < tokens * RB; o += kDownWaves * 64) {
    const int t = o / RB, c = o % RB;
    float v = 0.f;
    for (int j = 0; j < p.top_k; ++j) {
      const int pair = t * p.top_k + j;
      if (id[pair] < 0) continue;
      float y = 0.f;
      for (int s = 0; s < 1 << k.split; ++s) y += sums[(s * k.pairs + pair) * RB + c];
      v = __builtin_fmaf(tw[pair], y, v);
    }
    const __bf16 b = (__bf16)v;
    p.out[(int64_t)(k.t0 + t) * p.ld_out + k.col0 + c] = __builtin_bit_cast(uint16_t, b);
  }
}

inline bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int kLds = 160 * 1024;  // LDS of a CU

template <bool UE8M0, int NG, int RT, int D>
void launch_up(const Params& p, dim3 grid, hipStream_t stream) {
  hipLaunchKernelGGL((gate_up_kernel<UE8M0, NG, RT, D>), grid, dim3(kUpWaves * 64), 0, stream, p);
}

template <bool UE8M0, int RB>
void launch_down(Params p, int chunks, int pairs, hipStream_t stream) {
  const int room = (kLds - (int)sizeof(Plan) - 6 * kPairs - 512) / 1024 * 1024;
  p.slots = std::max(1, std::min(16, 16 * 1024 / (pairs * RB * 4)));
  const int sum_bytes = (p.slots * pairs * RB * 4 + 1023) / 1024 * 1024;
  p.ring = room - sum_bytes;
  const dim3 grid(p.hidden / RB, chunks);
  hipLaunchKernelGGL((down_kernel<UE8M0, RB>), grid, dim3(kDownWaves * 64), room, stream, p);
}

template <bool UE8M0>
void launch(const Params& p, int chunks, int pairs, hipStream_t stream) {
  const int usable = dg_get_num_cus(), cus = usable > 0 ? usable : 256;
  const auto units = [&](int columns) { return (int64_t)std::min(pairs, p.experts) * (p.inter / columns); };
  const auto grid = [&](int columns, int per_cu) {
    return dim3((unsigned)std::min<int64_t>(units(columns), (int64_t)cus * per_cu), chunks);
  };
  // Tokens of an expert per pass: no more than 16 can come where there are no more tokens;
  // else 32, with room for an uneven routing, until the average (pairs / experts, if all ids are
  // of this device) comes close to that: 16 experts of 4096 x 2048 with 24 on average 100 us, 111 us
  // with 64 tokens per pass; with 28 126 and 121 us.  An expert with more takes further passes.
  // 64 tokens with 32 columns of a per unit where that leaves every CU two units (16 experts with 32 tokens on
  // average, 7168 x 2048: 205 us, with 16 columns 228 us; 8 with 43, 1664 x 512: 25.4 and 23.6 us).
  if (std::min(p.m, p.tokens) <= 16) launch_up<UE8M0, 1, 1, 2>(p, grid(16, 2), stream);
  else if (pairs / p.experts <= 26) launch_up<UE8M0, 2, 2, 2>(p, grid(32, 1), stream);
  else if (units(32) >= 2 * cus) launch_up<UE8M0, 4, 2, 2>(p, grid(32, 1), stream);
  else launch_up<UE8M0, 4, 1, 2>(p, grid(16, 1), stream);
  // Columns per workgroup by the time they take, in bytes at the 45 B/ns that a CU brings in (of HBM's
  // 7 TB/s its share is 3/5 of that): every round over the CUs costs 4 us, and each workgroup reads its
  // rows of the weights and all of a.  (64 tokens, 7168 columns: 32 133 us, 16 154 us, 8 197 us; 27 tokens, 5
  // experts, 4224 columns, 640 values: 23, 30 and 37 us; 24 tokens, 32 experts, 2048 columns: 77, 66 and 62 us.)
  const auto cost = [&](int rb) {
    const int64_t wgs = (int64_t)(p.hidden / rb) * chunks, last = wgs % cus;
    const int64_t weights = (int64_t)rb * std::min(pairs, p.experts) * p.inter;
    const int64_t all = weights + (int64_t)pairs * p.inter * 2;
    const int64_t round = 180000 + std::max(weights * 5 / 3, all);
    return wgs / cus * round + (last == 0 ? 0 : 180000 + std::max(weights * 5 / 3 * last / cus, all));
  };
  const int64_t c8 = cost(8), c16 = cost(16), c32 = cost(32);
  if (c32 <= c16 && c32 <= c8) launch_down<UE8M0, 32>(p, chunks, pairs, stream);
  else if (c16 <= c8) launch_down<UE8M0, 16>(p, chunks, pairs, stream);
  else launch_down<UE8M0, 8>(p, chunks, pairs, stream);
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
      (int64_t)32 * hidden >= kNowhere || (int64_t)kPairs * inter * 2 >= kNowhere ||
      ((int64_t)inter / 128 + 1) * (hidden / 128) * 4 >= kNowhere)
    return DG_ERROR_NOT_SUPPORTED;
  if (workspace == nullptr || !aligned_to(workspace, 256) ||
      workspace_bytes < dg_get_moe_workspace_size(m, top_k, inter))
    return DG_ERROR_WORKSPACE;
  Params p{static_cast<const uint8_t*>(x), sfx, static_cast<const uint8_t*>(w13), sf13,
           static_cast<const uint8_t*>(w2), sf2, ids, tw, static_cast<__bf16*>(workspace),
           static_cast<uint16_t*>(out), ldx, ld_sfx, ld_out, m, top_k, experts, hidden, inter, kPairs / top_k, 1, 0};
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
