// Slices and products of the fp32 matrix-core tiles (v_mfma_f32_16x16x4_f32).
//
// out[r][c] = sum_t P(r, t) Q(c, t), an operand stored [r][t] or, SLOW, [t][r].  The
// contraction advances 16 terms at a time: the next slice is loaded into registers
// while this one is multiplied from LDS.  An LDS row holds the 16 terms of one operand
// row; lane (i, g) reads row i's terms 4 g .. 4 g + 3 at once and instruction s takes
// term 4 g + s of both operands (any order of the terms will do, as long as it is the
// same one).  16-byte chunk c of row r sits at c ^ ((r >> 2) & 3): the 16 rows of a
// read phase cover all banks.
#pragma once
#include "device_common.hpp"

namespace moe {

constexpr int kTerms = 16;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// This thread's parts of an operand's slice (rows x 16 terms, 16 bytes each).
template <bool SLOW, int ROWS>
struct SliceF32 {
  static constexpr int N = ROWS * kTerms / 4 / 256;
  float4 v[N];

  __device__ __forceinline__ void load(const float* p, int64_t ld, int r0, int rows, int t0, int end) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + 256 * k;
      const int r = r0 + (SLOW ? i % (ROWS / 4) * 4 : i / 4), t = t0 + (SLOW ? i / (ROWS / 4) : i % 4 * 4);
      v[k] = r < rows && t < end
                 ? load4(SLOW ? p + (int64_t)t * ld + r : p + (int64_t)r * ld + t)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  // Blocks of 16 rows of two operands in turn: rows r0 .. of p, the same of q.
  __device__ __forceinline__ void load_pair(const float* p, const float* q, int64_t ld, int r0, int rows, int t0, int end) {
    static_assert(!SLOW, "rows as they lie");
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + 256 * k, row = i / 4;
      const int r = r0 + (row >> 5) * 16 + (row & 15), t = t0 + i % 4 * 4;
      v[k] = r < rows && t < end ? load4((row & 16 ? q : p) + (int64_t)r * ld + t) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void store(float* lds) const {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + 256 * k;
      if constexpr (SLOW) {
        const int r = i % (ROWS / 4) * 4, t = i / (ROWS / 4);       // 4 rows r .., one swizzle key
        const int at = (((t >> 2) ^ ((r >> 2) & 3)) << 2) + (t & 3);
        lds[(r + 0) * kTerms + at] = v[k].x;
        lds[(r + 1) * kTerms + at] = v[k].y;
        lds[(r + 2) * kTerms + at] = v[k].z;
        lds[(r + 3) * kTerms + at] = v[k].w;
      } else {
        const int r = i / 4, c = i % 4;
        *reinterpret_cast<float4*>(lds + r * kTerms + ((c ^ ((r >> 2) & 3)) << 2)) = v[k];
      }
    }
  }
};

// acc[x][y] += the slice's products: B column blocks (of Q, from row wc) x B row
// blocks (of P, from row wr).
template <int B>
__device__ __forceinline__ void multiply_f32(const float* ps, const float* qs, int wr, int wc, int i, int g,
                                             f32x4_t (&acc)[B][B]) {
  float4 fa[B], fb[B];
#pragma unroll
  for (int x = 0; x < B; ++x) {
    const int c = wc + x * 16 + i, r = wr + x * 16 + i;
    fa[x] = *reinterpret_cast<const float4*>(&qs[c * kTerms + ((g ^ ((c >> 2) & 3)) << 2)]);
    fb[x] = *reinterpret_cast<const float4*>(&ps[r * kTerms + ((g ^ ((r >> 2) & 3)) << 2)]);
  }
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int x = 0; x < B; ++x)
#pragma unroll
      for (int y = 0; y < B; ++y)
        acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x4f32(reinterpret_cast<const float*>(&fa[x])[s],
                                                         reinterpret_cast<const float*>(&fb[y])[s], acc[x][y], 0, 0, 0);
}

}  // namespace moe
