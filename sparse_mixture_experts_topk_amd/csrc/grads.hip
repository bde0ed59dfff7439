// Norm over a list of gradients, and the list scaled to a bound.
//
//   S = sum over all elements of x^2,  norm = sqrt(S),  out = x min(1, max_norm / norm)
//
// Squares and sums are fp64: bf16 and fp32 gradients reach 1e38 and 1e-38, whose
// squares leave fp32, and a sum of 10^9 terms loses digits there; the products hide
// under the reads.  Workgroup b sums one chunk of one tensor; a second kernel adds
// the chunks' sums in a fixed order, so S depends on the list's sizes, alignments and values alone.
// Both passes are HBM-bound: the norm has to be known before the first element is
// written, so the list is read twice and written once.
//
// A list goes to a kernel by value, kListed tensors a launch.  Chunks are cut at
// 16-byte boundaries of memory, so a tensor may begin and end at any element.
#include <algorithm>
#include <cmath>

#include "device_common.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kListed = 140;                     // a kernel's arguments are under 4 KiB
constexpr int64_t kChunkBytes = 32 << 10;        // at least
constexpr int64_t kMaxChunks = 8192;             // about, of all lists

struct Listed {
  const void* p;
  void* o;                // clip: output
  int64_t n2;             // elements, doubled, + 1 for fp32
};
struct List {
  Listed t[kListed];
  int32_t first[kListed + 1];      // first chunk of each tensor
  int32_t count;
  int64_t chunk;                   // 16-byte vectors
};
static_assert(sizeof(List) + 32 <= 4096, "a launch's arguments");

// The tensor of chunk b and the vectors [v0, v1) of it; vector v holds the elements
// v V - head .. + V - 1 of the tensor.
struct Span {
  const uint8_t* base;
  int64_t v0, v1, n;
  int tensor, head;
  bool f32;
};
__device__ __forceinline__ Span span_of(const List& l, int b) {
  // How many tensors begin at b or before: every lane looks at one of each 64, for a search
  // step by step waits for the arguments' memory at each (norm and clipping replayed from a
  // graph, 1000 tensors of 4096: 52.3 -> 47.0 us in bf16, 74.1 -> 60.0 in fp32).
  constexpr int N = (kListed + kWave - 1) / kWave;
  int32_t first[N];
#pragma unroll
  for (int i = 0; i < N; ++i) first[i] = l.first[min(i * kWave + (int)(threadIdx.x & 63), kListed)];
  int lo = -1;
#pragma unroll
  for (int i = 0; i < N; ++i)
    lo += __popcll(__ballot(i * kWave + (int)(threadIdx.x & 63) < l.count && first[i] <= b));
  lo = __builtin_amdgcn_readfirstlane(lo);
  Span s;
  s.tensor = lo;
  s.f32 = l.t[lo].n2 & 1;
  s.n = l.t[lo].n2 >> 1;
  const uintptr_t p = reinterpret_cast<uintptr_t>(l.t[lo].p);
  const int es = s.f32 ? 4 : 2, V = 16 / es;
  s.head = (int)(p & 15) / es;
  s.base = reinterpret_cast<const uint8_t*>(p & ~(uintptr_t)15);
  s.v0 = (int64_t)(b - l.first[lo]) * l.chunk;
  const int64_t end = (s.head + s.n + V - 1) / V;
  s.v1 = s.v0 + l.chunk < end ? s.v0 + l.chunk : end;
  return s;
}

template <bool F32>
__device__ __forceinline__ double square_sum(uint4 u, double acc) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      const double v = __uint_as_float(w[i]);
      acc = fma(v, v, acc);
    } else {
      const double a = bf16_lo(w[i]), b = bf16_hi(w[i]);
      acc = fma(a, a, acc);
      acc = fma(b, b, acc);
    }
  }
  return acc;
}

// A vector at the tensor's edge: the elements outside it are zero.
template <bool F32>
__device__ __forceinline__ uint4 load_edge(const Span& s, int64_t v) {
  constexpr int V = F32 ? 4 : 8;
  uint32_t w[4] = {0, 0, 0, 0};
  const int64_t e0 = v * V - s.head;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (e0 + i < 0 || e0 + i >= s.n) continue;
    if constexpr (F32) w[i] = reinterpret_cast<const uint32_t*>(s.base)[v * V + i];
    else w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(s.base)[v * V + i] << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whole vectors of the span [i0, i1): those that hold elements of the tensor only.
template <bool F32>
__device__ __forceinline__ void inner(const Span& s, int64_t& i0, int64_t& i1) {
  constexpr int V = F32 ? 4 : 8;
  const int64_t whole0 = s.head > 0 ? 1 : 0, whole1 = (s.head + s.n) / V;
  i0 = s.v0 > whole0 ? s.v0 : whole0;
  i1 = s.v1 < whole1 ? s.v1 : whole1;
}

constexpr int kUnroll = 8;

template <bool F32>
__device__ __forceinline__ double chunk_sum(const Span& s) {
  int64_t i0, i1;
  inner<F32>(s, i0, i1);
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  const uint4* p = reinterpret_cast<const uint4*>(s.base);
  int64_t v = i0 + threadIdx.x;
  for (; v + (kUnroll - 1) * kThreads < i1; v += kUnroll * kThreads) {
    uint4 u[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) u[k] = p[v + k * kThreads];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) acc[k & 3] = square_sum<F32>(u[k], acc[k & 3]);
  }
  for (; v < i1; v += kThreads) acc[0] = square_sum<F32>(p[v], acc[0]);
  // the edges: at most the first and the last vector of the tensor
  if (threadIdx.x == 0 && s.v0 < i0) acc[1] = square_sum<F32>(load_edge<F32>(s, s.v0), acc[1]);
  if (threadIdx.x == 1 && s.v1 > i1 && s.v1 - 1 >= i0) acc[1] = square_sum<F32>(load_edge<F32>(s, s.v1 - 1), acc[1]);
  return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

template <int THREADS>
__device__ __forceinline__ double workgroup_sum(double v, double (&part)[THREADS / kWave]) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v += __shfl_xor(v, m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / kWave; ++w) s += part[w];
  return s;
}

__device__ __forceinline__ void store_norm(double sum, double* sum_squares, float* norm) {
  *sum_squares = sum;
  if (norm != nullptr) *norm = (float)sqrt(sum);
}

// A list of one chunk ends here: sum_squares and norm are given.
__global__ __launch_bounds__(kThreads) void norm_chunks_kernel(const List l, double* __restrict__ part,
                                                               double* __restrict__ sum_squares,
                                                               float* __restrict__ norm) {
  __shared__ double waves[kThreads / kWave];
  const Span s = span_of(l, blockIdx.x);
  const double v = s.f32 ? chunk_sum<true>(s) : chunk_sum<false>(s);
  const double sum = workgroup_sum<kThreads>(v, waves);
  if (threadIdx.x != 0) return;
  if (sum_squares != nullptr) store_norm(sum, sum_squares, norm);
  else part[blockIdx.x] = sum;
}

constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void norm_join_kernel(const double* __restrict__ part, int chunks,
                                                                 double* __restrict__ sum_squares,
                                                                 float* __restrict__ norm) {
  __shared__ double waves[kJoinThreads / kWave];
  double v = 0.0;
  for (int i = threadIdx.x; i < chunks; i += kJoinThreads) v += part[i];
  const double sum = workgroup_sum<kJoinThreads>(v, waves);
  if (threadIdx.x == 0) store_norm(sum, sum_squares, norm);
}

// An fp64 product in bf16, rounded once: over fp32 one next to the middle between two bf16
// values would land on it and go to the even one, whichever side it was on.
__device__ __forceinline__ uint16_t to_bf16(double v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// x scale: in fp64, so that the one rounding is the result's.
template <bool F32>
__device__ __forceinline__ uint4 scaled(uint4 u, double scale) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) w[i] = __float_as_uint((float)(__uint_as_float(w[i]) * scale));
    else w[i] = to_bf16(bf16_lo(w[i]) * scale) | (uint32_t)to_bf16(bf16_hi(w[i]) * scale) << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements [first, end) one by one.
template <bool F32>
__device__ __forceinline__ void clip_elements(const void* p, void* o, int64_t first, int64_t end, double scale) {
  for (int64_t e = first + threadIdx.x; e < end; e += kThreads) {
    if constexpr (F32) static_cast<float*>(o)[e] = (float)(static_cast<const float*>(p)[e] * scale);
    else static_cast<uint16_t*>(o)[e] = to_bf16(bf16_bits_to_f32(static_cast<const uint16_t*>(p)[e]) * scale);
  }
}

template <bool F32>
__device__ __forceinline__ void clip_chunk(const Span& s, const void* p, void* o, double scale) {
  constexpr int V = F32 ? 4 : 8;
  const int64_t e0 = s.v0 * V - s.head > 0 ? s.v0 * V - s.head : 0;
  const int64_t e1 = s.v1 * V - s.head < s.n ? s.v1 * V - s.head : s.n;
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) != 0) {   // no common vectors
    clip_elements<F32>(p, o, e0, e1, scale);
    return;
  }
  int64_t i0, i1;
  inner<F32>(s, i0, i1);
  if (i0 >= i1) {
    clip_elements<F32>(p, o, e0, e1, scale);
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(s.base);
  uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(o) & ~(uintptr_t)15);
  int64_t v = i0 + threadIdx.x;
  for (; v + (kUnroll - 1) * kThreads < i1; v += kUnroll * kThreads) {
    uint4 u[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) u[k] = src[v + k * kThreads];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) dst[v + k * kThreads] = scaled<F32>(u[k], scale);
  }
  for (; v < i1; v += kThreads) dst[v] = scaled<F32>(src[v], scale);
  clip_elements<F32>(p, o, e0, i0 * V - s.head, scale);
  clip_elements<F32>(p, o, i1 * V - s.head, e1, scale);
}

// The factor: 1 for a norm within the bound, and for one that is not finite as store_norm
// gives it to the caller, in fp32 (fp32 and bf16 elements near 1e38 have one that leaves it).
__device__ __forceinline__ double clip_scale(double sum_squares, float max_norm) {
  const double norm = sqrt(sum_squares);
  return norm > (double)max_norm && (float)norm < INFINITY ? (double)max_norm / norm : 1.0;
}

__global__ __launch_bounds__(kThreads) void clip_kernel(const List l, const double* __restrict__ sum_squares,
                                                        float max_norm) {
  const double scale = clip_scale(*sum_squares, max_norm);
  // from the end: what the norm's pass read last may still be in the memory-side cache
  const Span s = span_of(l, gridDim.x - 1 - blockIdx.x);
  const void* p = l.t[s.tensor].p;
  void* o = l.t[s.tensor].o;
  if (scale == 1.0 && p == o) return;
  if (s.f32) clip_chunk<true>(s, p, o, scale);
  else clip_chunk<false>(s, p, o, scale);
}

int64_t vectors_of(const moe_tensor_t& t) {
  if (t.n == 0) return 0;
  const int es = t.dtype == MOE_F32 ? 4 : 2, V = 16 / es;
  const int head = (int)(reinterpret_cast<uintptr_t>(t.data) & 15) / es;
  return (head + t.n + V - 1) / V;
}

// 16-byte vectors of a chunk: 32 KiB, more where that would make over kMaxChunks of them.
int64_t chunk_vectors(const moe_tensor_t* tensors, int count) {
  int64_t total = 0;
  for (int i = 0; i < count; ++i) total += vectors_of(tensors[i]);
  int64_t chunk = kChunkBytes / 16;
  while (total / chunk > kMaxChunks) chunk *= 2;
  return chunk;
}

// Calls run(list, chunks in it) for the tensors, kListed at a time; empty ones are passed over.
template <class F>
hipError_t each_list(const moe_tensor_t* tensors, const moe_tensor_t* outs, int count, F&& run) {
  List l;
  l.chunk = chunk_vectors(tensors, count);
  l.count = 0;
  l.first[0] = 0;
  for (int i = 0; i < count; ++i) {
    if (tensors[i].n > 0) {
      l.t[l.count] = {tensors[i].data, outs != nullptr ? outs[i].data : tensors[i].data,
                      tensors[i].n * 2 + (tensors[i].dtype == MOE_F32 ? 1 : 0)};
      l.first[l.count + 1] = l.first[l.count] + (int32_t)((vectors_of(tensors[i]) + l.chunk - 1) / l.chunk);
      ++l.count;
    }
    if (l.count == kListed || (i == count - 1 && l.count > 0)) {
      const hipError_t e = run(l, l.first[l.count]);
      if (e != hipSuccess) return e;
      l.count = 0;
    }
  }
  return hipSuccess;
}

int64_t total_chunks(const moe_tensor_t* tensors, int count) {
  const int64_t chunk = chunk_vectors(tensors, count);
  int64_t n = 0;
  for (int i = 0; i < count; ++i) n += (vectors_of(tensors[i]) + chunk - 1) / chunk;
  return n;
}

}  // namespace

size_t grad_norm_workspace_bytes(const moe_tensor_t* tensors, int count) {
  return (size_t)total_chunks(tensors, count) * sizeof(double);
}

hipError_t launch_grad_norm(const moe_tensor_t* tensors, int count, double* sum_squares, float* norm, void* workspace,
                            hipStream_t st) {
  double* part = static_cast<double*>(workspace);
  const bool one = total_chunks(tensors, count) == 1;
  int chunks = 0;
  hipError_t e = each_list(tensors, nullptr, count, [&](const List& l, int n) {
    hipLaunchKernelGGL(norm_chunks_kernel, dim3((unsigned)n), dim3(kThreads), 0, st, l, part + chunks,
                       one ? sum_squares : nullptr, norm);
    chunks += n;
    return hipGetLastError();
  });
  if (e != hipSuccess || one) return e;
  hipLaunchKernelGGL(norm_join_kernel, dim3(1), dim3(kJoinThreads), 0, st, part, chunks, sum_squares, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const moe_tensor_t* tensors, const moe_tensor_t* outs, int count,
                            const double* sum_squares, float max_norm, hipStream_t st) {
  return each_list(tensors, outs, count, [&](const List& l, int n) {
    hipLaunchKernelGGL(clip_kernel, dim3((unsigned)n), dim3(kThreads), 0, st, l, sum_squares, max_norm);
    return hipGetLastError();
  });
}

}  // namespace moe
