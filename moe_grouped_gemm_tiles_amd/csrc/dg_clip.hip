// dg_clip.hip -- global norm over many gradient tensors and clipping by it, on
// gfx950.
//
//     norm = sqrt(sum over all tensors and elements of g^2)
//     out  = g * min(1, max_norm / (norm + 1e-6))
//
// Two passes over the gradients, one launch each for up to kTensors tensors.  The
// first leaves one FP64 partial sum per workgroup; they are added in a fixed order
// (no atomics).  Squares are summed in FP64, which neither overflows for large
// gradients nor loses small ones, and costs less time than reading them.
//
// The tensors' addresses and sizes travel in the kernel arguments: the library
// allocates no device memory and keeps no table between calls.
//
// Both passes are bound by HBM.  Measured on eight FP32 tensors of 117 MB (940 MB):
//   * first pass 141 us, 6.7 TB/s: persistent workgroups, four 16-byte loads in
//     flight per thread, streaming (not streaming: 158 us);
//   * second pass, out of place, 281 us, 6.7 TB/s: one 16-byte vector per thread and one
//     4 KiB chunk per workgroup, which a launch of its own with the factor makes
//     possible; persistent workgroups, which work the factor out for themselves, take 312
//     to 350 us.  They stay where that launch costs more than it gives (up to 32 MiB:
//     21.2 us against 22.2 us; 64 MiB: 43.0 us against 37.7 us) and in place, where they
//     end at once when nothing is to be clipped;
//   * the second pass begins with what the first read last: the last 256 MiB, the
//     size of the last-level cache, are not marked as streaming (12 us less).
// Together 435 us; 48 ragged tensors of 3.4 MB in all take 8.4 us, two launches.  In place the eight
// tensors take 464 us, and 151 us where nothing is to be clipped; in BF16 (470 MB) 221 and 83 us, out of
// place 224 us.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "dg.h"
#include "dg_common.hpp"

namespace {

namespace clip {

constexpr int kTensors = 128;      // tensors per launch (their descriptors fit in 4 KiB of arguments)
constexpr int kPartials = 2048;    // workgroups of the first pass, over all its launches
constexpr int kThreads = 256;
constexpr int64_t kLarge = (int64_t)32 << 20;  // gradients past this are streamed
constexpr int64_t kKept = (int64_t)256 << 20;  // but for the last ones of the first pass
constexpr int64_t kMostBytes = (int64_t)1 << 42;

struct Group {
  const void* in[kTensors];
  void* out[kTensors];
  int64_t n[kTensors];
  int32_t first[kTensors];  // first chunk of each tensor
  uint32_t bf16[kTensors / 32];
  int tensors;
  int chunks;
  int64_t chunk;  // bytes per chunk
  int keep;       // first pass: chunks from here on may stay in the caches
  int in_place;
  double* partial;
  int partials;   // of all launches (second pass)
  float max_norm;
  float* norm;
  float* factor;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A 16-byte vector: 4 FP32 or 8 BF16 elements.
template <bool BF16>
constexpr int kVec = BF16 ? 8 : 4;

template <bool NT>
__device__ __forceinline__ u32x4 load_vec(const void* p) {
  const u32x4* v = reinterpret_cast<const u32x4*>(p);
  return NT ? __builtin_nontemporal_load(v) : *v;
}
template <bool NT>
__device__ __forceinline__ void store_vec(void* p, u32x4 x) {
  u32x4* v = reinterpret_cast<u32x4*>(p);
  if (NT) __builtin_nontemporal_store(x, v);
  else *v = x;
}
// Element i of a vector as FP32.
template <bool BF16>
__device__ __forceinline__ float element(u32x4 v, int i) {
  if constexpr (BF16) return __uint_as_float(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16);
  else return __uint_as_float(v[i]);
}
template <bool BF16>
__device__ __forceinline__ u32x4 times(u32x4 v, float c) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
      const bf16x2 r = {(__bf16)(element<true>(v, 2 * i) * c), (__bf16)(element<true>(v, 2 * i + 1) * c)};
      o[i] = __builtin_bit_cast(uint32_t, r);
    } else {
      o[i] = __float_as_uint(element<false>(v, i) * c);
    }
  }
  return o;
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

// Elements [begin, end) of one tensor: whole 16-byte-aligned vectors, kUnroll of them in
// flight per thread, and single elements before and after them.
struct Span {
  int64_t body, vecs;  // first element of the vectors, how many vectors
};
template <bool BF16>
__device__ __forceinline__ Span span_of(const void* in, const void* out, int64_t begin, int64_t end) {
  constexpr int ES = BF16 ? 2 : 4;
  const uintptr_t a = reinterpret_cast<uintptr_t>(in) + begin * ES;
  int64_t head = ((16 - (a & 15)) & 15) / ES;
  const bool same = ((a ^ (reinterpret_cast<uintptr_t>(out) + begin * ES)) & 15) == 0;
  if (!same || head > end - begin) head = end - begin;
  return {begin + head, (end - begin - head) / kVec<BF16>};
}

constexpr int kUnroll = 4;

template <bool BF16, bool NT>
__device__ __forceinline__ double square_sum(const void* in, int64_t begin, int64_t end) {
  constexpr int V = kVec<BF16>;
  const int tid = threadIdx.x;
  const Span s = span_of<BF16>(in, in, begin, end);
  const uint8_t* body = static_cast<const uint8_t*>(in) + s.body * (16 / V);
  double sum[2] = {0.0, 0.0};
  const auto add = [&](u32x4 v) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double e = (double)element<BF16>(v, i);
      sum[i & 1] = __builtin_fma(e, e, sum[i & 1]);
    }
  };
  int64_t i = tid;
  for (; i + (kUnroll - 1) * kThreads < s.vecs; i += kUnroll * kThreads) {
    u32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = load_vec<NT>(body + (i + u * kThreads) * 16);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) add(v[u]);
  }
  for (; i < s.vecs; i += kThreads) add(load_vec<NT>(body + i * 16));
  const auto one = [&](int64_t k) {
    const double e = (double)load1<BF16>(in, k);
    sum[0] = __builtin_fma(e, e, sum[0]);
  };
  for (int64_t k = begin + tid; k < s.body; k += kThreads) one(k);
  for (int64_t k = s.body + s.vecs * V + tid; k < end; k += kThreads) one(k);
  return sum[0] + sum[1];
}

// Elements [begin, end) of tensor t that chunk c holds.
struct Part {
  int t;
  bool bf16;
  int64_t begin, end;
};
__device__ __forceinline__ Part part_of(const Group& g, int c) {
  Part p;
  p.t = tensor_of(g, c);
  p.bf16 = g.bf16[p.t >> 5] >> (p.t & 31) & 1;
  const int64_t n = g.chunk >> (p.bf16 ? 1 : 2);
  p.begin = (c - g.first[p.t]) * n;
  p.end = min(p.begin + n, g.n[p.t]);
  return p;
}

template <bool NT>
__device__ __forceinline__ double square_sum(const Group& g, int c) {
  const Part p = part_of(g, c);
  return p.bf16 ? square_sum<true, NT>(g.in[p.t], p.begin, p.end) : square_sum<false, NT>(g.in[p.t], p.begin, p.end);
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const Group g) {
  double s = 0.0;
  int c = blockIdx.x;
  for (; c < g.keep; c += gridDim.x) s += square_sum<true>(g, c);
  for (; c < g.chunks; c += gridDim.x) s += square_sum<false>(g, c);
  s = block_sum(s);
  if (threadIdx.x == 0) g.partial[blockIdx.x] = s;
}

// The norm and the factor, on every thread of a workgroup.
__device__ __forceinline__ float factor_of(const Group& g, float& norm) {
  double s = 0.0;
  for (int i = threadIdx.x; i < g.partials; i += kThreads) s += g.partial[i];
  norm = (float)sqrt(block_sum(s));
  const float q = g.max_norm / (norm + 1e-6f);
  return g.max_norm == __builtin_inff() || q > 1.0f ? 1.0f : q;  // a NaN stays one
}

__global__ void __launch_bounds__(kThreads) factor_kernel(const Group g) {
  float norm;
  const float c = factor_of(g, norm);
  if (threadIdx.x == 0) {
    *g.norm = norm;
    *g.factor = c;
  }
}

template <bool BF16, bool NT>
__device__ __forceinline__ void scale(const void* in, void* out, int64_t begin, int64_t end, float c) {
  constexpr int V = kVec<BF16>;
  const int tid = threadIdx.x;
  const Span s = span_of<BF16>(in, out, begin, end);
  const uint8_t* from = static_cast<const uint8_t*>(in) + s.body * (16 / V);
  uint8_t* to = static_cast<uint8_t*>(out) + s.body * (16 / V);
  int64_t i = tid;
  for (; i + (kUnroll - 1) * kThreads < s.vecs; i += kUnroll * kThreads) {
    u32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = load_vec<NT>(from + (i + u * kThreads) * 16);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) store_vec<NT>(to + (i + u * kThreads) * 16, times<BF16>(v[u], c));
  }
  for (; i < s.vecs; i += kThreads) store_vec<NT>(to + i * 16, times<BF16>(load_vec<NT>(from + i * 16), c));
  for (int64_t k = begin + tid; k < s.body; k += kThreads) store1<BF16>(out, k, load1<BF16>(in, k) * c);
  for (int64_t k = s.body + s.vecs * V + tid; k < end; k += kThreads) store1<BF16>(out, k, load1<BF16>(in, k) * c);
}

template <bool NT>
__device__ __forceinline__ void scale(const Group& g, int c, float f) {
  const Part p = part_of(g, c);
  if (p.bf16) scale<true, NT>(g.in[p.t], g.out[p.t], p.begin, p.end, f);
  else scale<false, NT>(g.in[p.t], g.out[p.t], p.begin, p.end, f);
}

// Persistent: every workgroup works out the factor, then takes chunks in turn.
template <bool NT>
__global__ void __launch_bounds__(kThreads) scale_kernel(const Group g) {
  float norm;
  const float f = factor_of(g, norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *g.norm = norm;
  if (g.in_place && f == 1.0f) return;
  for (int c = g.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) scale<NT>(g, c, f);
}

// One chunk per workgroup, from the last one back: the first pass left those in the caches.
__global__ void __launch_bounds__(kThreads) scale_once_kernel(const Group g) {
  scale<true>(g, g.chunks - 1 - (int)blockIdx.x, *g.factor);
}

}  // namespace clip

}  // namespace

extern "C" {

size_t dg_get_clip_workspace_size(void) { return clip::kPartials * sizeof(double) + 256; }

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
    if (t.numel > kMostBytes / 4 || (total += t.numel * (int64_t)es) > kMostBytes) return DG_ERROR_NOT_SUPPORTED;
  }
  if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
      workspace_bytes < dg_get_clip_workspace_size())
    return DG_ERROR_WORKSPACE;
  const int groups = num_tensors > 0 ? (num_tensors + kTensors - 1) / kTensors : 1;
  if (groups > kPartials) return DG_ERROR_NOT_SUPPORTED;
  const int64_t bytes = total;
  // bytes per chunk: 8 KiB (two vectors per thread) for the smallest sets, so that they too reach most
  // CUs (3.4 MB: 8.4 us, with 32 KiB 9.2 us), 32 KiB from 16 MiB on (16 MiB: 13.9 us, with 8 KiB 17.0 us),
  // and so many that a workgroup of a full round takes at most four
  int64_t chunk = 8 << 10;
  while (chunk < 32 << 10 && bytes / chunk > 512) chunk *= 2;
  while (bytes / chunk > 4 * kPartials) chunk *= 2;
  // one vector per thread, more where a launch would pass 2^31 threads
  int64_t once = kThreads * 16;
  while (bytes / once > 1 << 22) once *= 2;
  const bool large = bytes > kLarge;
  Group g;
  g.partial = static_cast<double*>(workspace);
  g.factor = reinterpret_cast<float*>(g.partial + kPartials);
  g.max_norm = max_norm;
  g.norm = norm;
  const int most = kPartials / groups;  // workgroups of a launch
  int used = 0;
  // Tensors of launch k in chunks of `chunk` bytes.
  const auto fill = [&](int k, int64_t chunk) {
    const int lo = k * kTensors, n = num_tensors - lo < kTensors ? num_tensors - lo : kTensors;
    g.tensors = n;
    g.chunk = chunk;
    g.chunks = 0;
    g.in_place = 1;
    for (uint32_t& b : g.bf16) b = 0;
    for (int i = 0; i < n; ++i) {
      const dg_tensor& t = grads[lo + i];
      g.in[i] = t.data;
      g.out[i] = out != nullptr ? out[lo + i].data : t.data;
      if (g.out[i] != g.in[i]) g.in_place = 0;
      g.n[i] = t.numel;
      g.first[i] = g.chunks;
      if (t.dtype == DG_DTYPE_BF16) g.bf16[i >> 5] |= 1u << (i & 31);
      g.chunks += (int)((t.numel * (t.dtype == DG_DTYPE_BF16 ? 2 : 4) + chunk - 1) / chunk);
    }
  };
  const auto grid_of = [&] { return dim3(g.chunks < 1 ? 1 : (g.chunks < most ? g.chunks : most)); };
  int64_t done = 0;  // bytes of the launches so far
  for (int k = 0; k < groups; ++k) {
    fill(k, chunk);
    // everything may stay in the caches of a small set; of a large one its last kKept bytes
    const int64_t past = bytes - kKept - done;
    g.keep = !large ? 0 : past <= 0 ? 0 : past / chunk >= g.chunks ? g.chunks : (int)(past / chunk);
    done += (int64_t)g.chunks * chunk;
    const dim3 grid = grid_of();
    hipLaunchKernelGGL(norm_kernel, grid, dim3(kThreads), 0, stream, g);
    g.partial += grid.x;
    used += grid.x;
  }
  g.partial = static_cast<double*>(workspace);
  g.partials = used;
  bool factor_known = false;
  for (int k = groups - 1; k >= 0; --k) {
    fill(k, chunk);
    if (!large) {
      hipLaunchKernelGGL(scale_kernel<false>, grid_of(), dim3(kThreads), 0, stream, g);
    } else if (g.in_place) {
      hipLaunchKernelGGL(scale_kernel<true>, grid_of(), dim3(kThreads), 0, stream, g);
    } else {
      if (!factor_known) hipLaunchKernelGGL(factor_kernel, dim3(1), dim3(kThreads), 0, stream, g);
      factor_known = true;
      fill(k, once);
      if (g.chunks > 0) hipLaunchKernelGGL(scale_once_kernel, dim3(g.chunks), dim3(kThreads), 0, stream, g);
    }
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_SUCCESS : dg::record_hip_error(e);
}

}  // extern "C"
