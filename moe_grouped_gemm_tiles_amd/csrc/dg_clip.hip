// dg_clip.hip -- global norm over many gradient tensors and clipping by it, on
// gfx950.
//
//     norm = sqrt(sum over all tensors and elements of g^2)
//     out  = g * min(1, max_norm / (norm + 1e-6))
//
// Two passes, each one launch for up to kTensors tensors: the first leaves one
// FP64 partial sum per workgroup, the second adds the partial sums (every
// workgroup for itself, in the same order, so there is neither an atomic nor a
// third launch) and scales.  Squares are summed in FP64, which neither
// overflows for large gradients nor loses small ones; reading the gradients
// takes longer than the FP64 adds.
//
// The tensors' addresses and sizes travel in the kernel arguments: the library
// allocates no device memory and keeps no table between calls.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "dg.h"
#include "dg_common.hpp"

namespace {

namespace clip {

constexpr int kTensors = 128;      // tensors per launch (their descriptors fit in 4 KiB of arguments)
constexpr int kPartials = 2048;    // workgroups of the first pass, over all its launches
constexpr int kThreads = 256;
constexpr int kVec = 8;            // elements a thread takes at once

struct Group {
  const void* in[kTensors];
  void* out[kTensors];
  int64_t n[kTensors];
  int32_t first[kTensors];  // first chunk of each tensor
  uint32_t bf16[kTensors / 32];
  int tensors;
  int chunks;
  int64_t chunk;  // elements per chunk, a multiple of kThreads * kVec
  double* partial;
  int partials;  // of all launches (second pass)
  float max_norm;
  float* norm;
  int in_place;
};

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else return static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (BF16) {
    const __bf16 b = (__bf16)v;
    static_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, b);
  } else {
    static_cast<float*>(p)[i] = v;
  }
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
template <bool BF16>
__device__ __forceinline__ void store8(void* p, const float (&v)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                                              bf16_pair(v[6], v[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Sum over the workgroup on every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double t[kThreads / 64];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  if ((threadIdx.x & 63) == 0) t[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) s += t[i];
  return s;
}

// Tensor of a chunk: the last one whose first chunk is not after it (a tensor
// without elements has no chunk and shares its place with the next one).
__device__ __forceinline__ int tensor_of(const Group& g, int chunk) {
  int lo = 0, hi = g.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Elements [begin, end) of one tensor: f8(element) on whole 16-byte-aligned
// vectors, f1(element) on what is before and after them.
template <bool BF16, typename F8, typename F1>
__device__ __forceinline__ void each(const void* in, const void* out, int64_t begin, int64_t end, F8 f8, F1 f1) {
  constexpr int ES = BF16 ? 2 : 4;
  const uintptr_t a = reinterpret_cast<uintptr_t>(in) + begin * ES;
  int64_t head = ((16 - (a & 15)) & 15) / ES;
  const bool vec = ((a ^ (reinterpret_cast<uintptr_t>(out) + begin * ES)) & 15) == 0;
  if (!vec || head > end - begin) head = end - begin;
  const int64_t body = begin + head, vecs = (end - body) / kVec;
  for (int64_t i = begin + threadIdx.x; i < body; i += kThreads) f1(i);
  for (int64_t i = threadIdx.x; i < vecs; i += kThreads) f8(body + i * kVec);
  for (int64_t i = body + vecs * kVec + threadIdx.x; i < end; i += kThreads) f1(i);
}

template <bool BF16>
__device__ __forceinline__ double square_sum(const void* in, int64_t begin, int64_t end) {
  constexpr int ES = BF16 ? 2 : 4;
  double s0 = 0.0, s1 = 0.0;
  each<BF16>(in, in, begin, end,
             [&](int64_t i) {
               float v[8];
               load8<BF16>(static_cast<const uint8_t*>(in) + i * ES, v);
#pragma unroll
               for (int k = 0; k < 8; k += 2) {
                 s0 += (double)v[k] * (double)v[k];
                 s1 += (double)v[k + 1] * (double)v[k + 1];
               }
             },
             [&](int64_t i) {
               const double v = (double)load1<BF16>(in, i);
               s0 += v * v;
             });
  return s0 + s1;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const Group g) {
  double s = 0.0;
  for (int c = blockIdx.x; c < g.chunks; c += gridDim.x) {
    const int t = tensor_of(g, c);
    const int64_t begin = (int64_t)(c - g.first[t]) * g.chunk, end = min(begin + g.chunk, g.n[t]);
    s += (g.bf16[t >> 5] >> (t & 31) & 1) ? square_sum<true>(g.in[t], begin, end)
                                          : square_sum<false>(g.in[t], begin, end);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) g.partial[blockIdx.x] = s;
}

template <bool BF16>
__device__ __forceinline__ void scale(const void* in, void* out, int64_t begin, int64_t end, float c) {
  constexpr int ES = BF16 ? 2 : 4;
  each<BF16>(in, out, begin, end,
             [&](int64_t i) {
               float v[8];
               load8<BF16>(static_cast<const uint8_t*>(in) + i * ES, v);
#pragma unroll
               for (int k = 0; k < 8; ++k) v[k] *= c;
               store8<BF16>(static_cast<uint8_t*>(out) + i * ES, v);
             },
             [&](int64_t i) { store1<BF16>(out, i, load1<BF16>(in, i) * c); });
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const Group g) {
  double s = 0.0;
  for (int i = threadIdx.x; i < g.partials; i += kThreads) s += g.partial[i];
  const float norm = (float)sqrt(block_sum(s));
  if (blockIdx.x == 0 && threadIdx.x == 0) *g.norm = norm;
  const float q = g.max_norm / (norm + 1e-6f);
  const float c = g.max_norm == __builtin_inff() || q > 1.0f ? 1.0f : q;  // a NaN stays one
  if (g.in_place && c == 1.0f) return;
  // from the last chunk back: the first pass read those last, so they are the ones still in the caches
  for (int k = g.chunks - 1 - (int)blockIdx.x; k >= 0; k -= gridDim.x) {
    const int t = tensor_of(g, k);
    const int64_t begin = (int64_t)(k - g.first[t]) * g.chunk, end = min(begin + g.chunk, g.n[t]);
    if (g.bf16[t >> 5] >> (t & 31) & 1) scale<true>(g.in[t], g.out[t], begin, end, c);
    else scale<false>(g.in[t], g.out[t], begin, end, c);
  }
}

}  // namespace clip

}  // namespace

extern "C" {

size_t dg_get_clip_workspace_size(void) { return clip::kPartials * sizeof(double); }

dg_status dg_clip_grad_norm(const dg_tensor* grads, const dg_tensor* out, int num_tensors, float max_norm, float* norm,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace clip;
  if (num_tensors < 0 || !(max_norm >= 0.f) || norm == nullptr || reinterpret_cast<uintptr_t>(norm) % 4 != 0)
    return DG_ERROR_INVALID_VALUE;
  if (num_tensors > 0 && grads == nullptr) return DG_ERROR_INVALID_VALUE;
  int64_t total = 0;
  for (int i = 0; i < num_tensors; ++i) {
    const dg_tensor& t = grads[i];
    if (t.numel < 0 || (t.dtype != DG_DTYPE_BF16 && t.dtype != DG_DTYPE_FP32)) return DG_ERROR_INVALID_VALUE;
    const dg_tensor& o = out != nullptr ? out[i] : t;
    if (o.numel != t.numel || o.dtype != t.dtype) return DG_ERROR_INVALID_VALUE;
    const uintptr_t es = t.dtype == DG_DTYPE_BF16 ? 2 : 4;
    if (t.numel > 0 && (t.data == nullptr || o.data == nullptr || reinterpret_cast<uintptr_t>(t.data) % es != 0 ||
                        reinterpret_cast<uintptr_t>(o.data) % es != 0))
      return DG_ERROR_INVALID_VALUE;
    if (t.numel > (int64_t)1 << 44 || (total += t.numel) > (int64_t)1 << 44) return DG_ERROR_NOT_SUPPORTED;
  }
  if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
      workspace_bytes < dg_get_clip_workspace_size())
    return DG_ERROR_WORKSPACE;
  const int groups = num_tensors > 0 ? (num_tensors + kTensors - 1) / kTensors : 1;
  if (groups > kPartials) return DG_ERROR_NOT_SUPPORTED;
  // chunks: about four for each workgroup of a full round, from 8 Ki elements (one
  // pass of four vectors per thread) to where their number fits 31 bits
  int64_t chunk = 8192;
  while (chunk < (int64_t)1 << 40 && total / chunk > 4 * kPartials) chunk *= 2;
  Group g;
  g.chunk = chunk;
  g.partial = static_cast<double*>(workspace);
  g.max_norm = max_norm;
  g.norm = norm;
  g.in_place = 1;
  for (int pass = 0; pass < 2; ++pass) {
    int used = 0;
    for (int k = 0; k < groups; ++k) {
      const int lo = k * kTensors, n = num_tensors - lo < kTensors ? num_tensors - lo : kTensors;
      int chunks = 0;
      for (uint32_t& b : g.bf16) b = 0;
      g.in_place = 1;
      for (int i = 0; i < n; ++i) {
        const dg_tensor& t = grads[lo + i];
        g.in[i] = t.data;
        g.out[i] = out != nullptr ? out[lo + i].data : t.data;
        if (g.out[i] != g.in[i]) g.in_place = 0;
        g.n[i] = t.numel;
        g.first[i] = chunks;
        if (t.dtype == DG_DTYPE_BF16) g.bf16[i >> 5] |= 1u << (i & 31);
        chunks += (int)((t.numel + chunk - 1) / chunk);
      }
      g.tensors = n;
      g.chunks = chunks;
      const int most = kPartials / groups;
      const int grid = chunks < 1 ? 1 : (chunks < most ? chunks : most);
      if (pass == 0) {
        hipLaunchKernelGGL(norm_kernel, dim3(grid), dim3(kThreads), 0, stream, g);
        g.partial += grid;
      } else {
        hipLaunchKernelGGL(scale_kernel, dim3(grid), dim3(kThreads), 0, stream, g);
      }
      used += grid;
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return dg::record_hip_error(e);
    }
    g.partials = used;
    g.partial = static_cast<double*>(workspace);
  }
  return DG_SUCCESS;
}

}  // extern "C"
