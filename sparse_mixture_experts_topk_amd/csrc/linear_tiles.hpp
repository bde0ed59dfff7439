// Tiled dense product on the gfx950 matrix cores: out[r][c] = sum_t P(r, t) Q(c, t).
//
// P has `rows` rows, Q `cols` rows, the contraction `len` terms.  An operand is
// stored [r][t] (its contraction contiguous) or, SLOW, [t][r]; nothing is
// transposed in memory.  The matrix-core operand A is Q, B is P, so an
// accumulator block is [c][r]: a lane holds one row r and runs of 4
// consecutive c.
//
// A tile is TA x TB (c x r).  The contraction advances BK at a time through a
// ring of NS LDS stages, filled by buffer loads that write LDS directly.  A
// stage of an operand:
//   [r][t]: 128-byte rows of BK = 64 terms; fragments are one 16-byte read per
//           lane.  16-byte chunk c of row r sits at c ^ key(r), so that the 16
//           rows of a read phase cover all banks.
//   [t][r]: BK rows of the tile's width; fragments are two transposing 8-byte
//           reads (ds_read_b64_tr_b16: 16 lanes read 4 rows x 16 columns and
//           each gets one column).  Chunk c of row t sits at c ^ slow_key(t):
//           the 4 rows of a read go to different 64-byte quarters of the 256
//           bytes that the banks cover, rows t and t + 8 to different halves
//           of one, so no two of the lanes served together share a bank.
// Buffer descriptors are bounded to the operand's valid part and a chunk past
// the end of a [r][t] row is sent past it: such loads write zeros to LDS, on
// both operands, so a NaN next to the end cannot come in.
//
// The kernel is persistent (one workgroup per CU): workgroup b takes tiles of
// XCD b % 8's contiguous share of the tile list, and the slices of all its
// tiles form one stream through the ring, so the next tile's first slices load
// while this one's results are stored.  The last, partial round of tiles is cut
// along the contraction over all workgroups (TileSplit): their fp32 partial
// tiles are summed in order by a second kernel, which applies the epilogue.
#pragma once
#include "device_common.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"
#include "lds_stream.hpp"
#include "persistent_tiles.hpp"

namespace moe {

struct ProductArgs {
  const uint16_t* P;
  const uint16_t* Q;
  int64_t ldp, ldq;         // elements
  int rows, cols, len;
  int row_tiles, col_tiles;
  float* partials;
  Epilogue ep;
};

// Consecutive tiles run side by side on one XCD; a near-square patch of them
// shares the most operand bytes in its L2: column tiles are taken in bands of 8,
// the tiles of a band row by row.
constexpr int kBand = 8;
__device__ __forceinline__ void tile_at(int t, int row_tiles, int col_tiles, int& rt, int& ct) {
  const int per_band = kBand * row_tiles;
  const int band = t / per_band, in = t - band * per_band;
  const int width = min(kBand, col_tiles - band * kBand);
  rt = in / width;
  ct = band * kBand + in - rt * width;
}

template <int BK, int NS, int WR, int WC, int WA, int WB>
struct ProductGeom {
  static_assert(BK == 64, "128-byte rows of the [r][t] layout");
  static constexpr int NW = WR * WC, THREADS = 64 * NW;
  static constexpr int TA = 32 * WR * WA, TB = 32 * WC * WB;
  static constexpr int A_BYTES = TA * BK * 2, B_BYTES = TB * BK * 2, STAGE = A_BYTES + B_BYTES;
  static constexpr int SUB = BK / 16;
  static constexpr int JA = A_BYTES / 1024 / NW, JB = B_BYTES / 1024 / NW, LOADS = JA + JB;
  static_assert(JA * NW * 1024 == A_BYTES && JB * NW * 1024 == B_BYTES, "whole loads per wavefront");
  static_assert(NS * STAGE <= 160 * 1024, "LDS");
  static constexpr int64_t PARTIAL = (int64_t)TA * TB;      // floats of a partial tile
};

__device__ __forceinline__ int fast_key(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int slow_key(int t) { return ((t & 3) << 2) | (((t >> 3) & 1) << 1); }

// This lane's byte offset in memory of an operand's first load of a slice (loads
// are whole swizzle periods of rows apart) and the step to the next.
template <bool SLOW, int TX, int NW>
struct LoadMap {
  static constexpr int CPR = SLOW ? TX / 8 : 8;            // chunks per LDS row
  static constexpr int RPI = 64 / CPR;                     // LDS rows per load
  static_assert(64 % CPR == 0 && (NW * RPI) % 16 == 0, "loads are whole swizzle periods apart");
  __device__ static __forceinline__ int chunk(int wave, int lane) {
    const int row = wave * RPI + lane / CPR;
    return (lane % CPR) ^ (SLOW ? slow_key(row) : fast_key(row));
  }
  __device__ static __forceinline__ int first(int wave, int lane, int rowbytes) {
    return (wave * RPI + lane / CPR) * rowbytes + chunk(wave, lane) * 16;
  }
  __device__ static __forceinline__ int step(int rowbytes) { return NW * RPI * rowbytes; }
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// Fragment of 32 operand rows x 16 terms for v_mfma_f32_32x32x16_bf16: lane
// (fi, fg) holds row fi, terms 8 fg .. 8 fg + 7.
template <bool SLOW, int TX>
__device__ __forceinline__ bf16x8_t read_fragment(const uint8_t* stage, int row0, int s, int lane) {
  const int fg = lane >> 5;
  if constexpr (!SLOW) {
    const int fi = lane & 31;
    return as_bf16x8(*reinterpret_cast<const uint4*>(stage + (row0 + fi) * 128 + (((2 * s + fg) ^ fast_key(fi)) << 4)));
  } else {
    const int i = lane & 15, t0 = 16 * s + 8 * fg + (i >> 2);
    const int x = row0 + 16 * ((lane >> 4) & 1) + 4 * (i & 3);     // first of the 4 columns read
    s16x4_t v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = t0 + 4 * j;
      const uint8_t* p = stage + t * (TX * 2) + (((x >> 3) ^ slow_key(t)) << 4) + (x & 4) * 2;
      v[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
    }
    typedef short s16x8_t __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8_t, s16x8_t{v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w});
  }
}

template <bool PSLOW, bool QSLOW, int ACT, int BK, int NS, int WR, int WC, int WA, int WB>
__global__ __launch_bounds__(64 * WR * WC, 1) void linear_product_kernel(const ProductArgs a) {
  using G = ProductGeom<BK, NS, WR, WC, WA, WB>;
  using MA = LoadMap<QSLOW, G::TA, G::NW>;
  using MB = LoadMap<PSLOW, G::TB, G::NW>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * G::STAGE];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC;
  const int KT = (a.len + BK - 1) / BK;
  const int slots = gridDim.x >> 3, xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  const TileSplit sp = TileSplit::of(a.row_tiles * a.col_tiles, xcd, slots, KT);
  const int n_whole = sp.R + (sp.whole_tail && slot < sp.tail ? 1 : 0);
  const int run0 = slot * sp.P, run1 = min(run0 + sp.P, sp.tail * KT);
  const int n_runs = run0 < run1 ? (run1 - 1) / KT - run0 / KT + 1 : 0;
  const int n_items = n_whole + n_runs;
  if (n_items == 0) return;

  // Item i: a whole tile, or a run [kb, ke) of slices of tail tile j (partial tile slot + j of the XCD's).
  struct Item { int r0, c0, kb, ke, part; };
  auto item = [&](int i) __attribute__((always_inline)) -> Item {
    Item it{0, 0, 0, KT, -1};
    int t;
    if (i < n_whole) {
      t = sp.share_begin + slot + i * slots;
    } else {
      const int j = run0 / KT + (i - n_whole);
      t = sp.share_begin + sp.R * slots + j;
      it.kb = max(run0 - j * KT, 0);
      it.ke = min(run1 - j * KT, KT);
      it.part = xcd * 2 * slots + slot + j;
    }
    int rt, ct;
    tile_at(t, a.row_tiles, a.col_tiles, rt, ct);
    it.r0 = __builtin_amdgcn_readfirstlane(rt * G::TB);
    it.c0 = __builtin_amdgcn_readfirstlane(ct * G::TA);
    it.kb = __builtin_amdgcn_readfirstlane(it.kb);
    it.ke = __builtin_amdgcn_readfirstlane(it.ke);
    it.part = __builtin_amdgcn_readfirstlane(it.part);
    return it;
  };

  // ---- loads ----
  const uint32_t lds_base = (uint32_t)(uintptr_t)smem;
  const int qrow = (int)a.ldq * 2, prow = (int)a.ldp * 2;          // bytes
  int li = 0, lkt = 0, lke = 0;
  const uint8_t *qbase = nullptr, *pbase = nullptr;                 // operand's first byte of the cursor's slice
  int64_t qleft = 0, pleft = 0;                                     // valid bytes from there
  auto load_item = [&]() __attribute__((always_inline)) {
    if (li >= n_items) {                                            // past the last slice: nothing is in range
      qleft = pleft = 0;
      return;
    }
    const Item it = item(li);
    lkt = it.kb;
    lke = it.ke;
    if constexpr (QSLOW) {
      qbase = reinterpret_cast<const uint8_t*>(a.Q + (int64_t)it.kb * BK * a.ldq + it.c0);
      qleft = ((int64_t)(a.len - it.kb * BK) * a.ldq - it.c0) * 2;
    } else {
      qbase = reinterpret_cast<const uint8_t*>(a.Q + (int64_t)it.c0 * a.ldq + it.kb * BK);
      qleft = ((int64_t)min(G::TA, a.cols - it.c0) * a.ldq - it.kb * BK) * 2;
    }
    if constexpr (PSLOW) {
      pbase = reinterpret_cast<const uint8_t*>(a.P + (int64_t)it.kb * BK * a.ldp + it.r0);
      pleft = ((int64_t)(a.len - it.kb * BK) * a.ldp - it.r0) * 2;
    } else {
      pbase = reinterpret_cast<const uint8_t*>(a.P + (int64_t)it.r0 * a.ldp + it.kb * BK);
      pleft = ((int64_t)min(G::TB, a.rows - it.r0) * a.ldp - it.kb * BK) * 2;
    }
  };
  // this lane's offsets of the first load of each operand (chunk of a [r][t] row past the contraction: out of range)
  const int qchunk = MA::chunk(wave, lane), pchunk = MB::chunk(wave, lane);
  const int qfirst = MA::first(wave, lane, qrow), pfirst = MB::first(wave, lane, prow);
  constexpr int kPast = (int)0x80000000u;
  auto load = [&](int ls, int j) __attribute__((always_inline)) {
    const uint32_t sb = lds_base + (uint32_t)((ls % NS) * G::STAGE);
    if (j < G::JA) {
      const int off = !QSLOW && lkt * BK + qchunk * 8 >= a.len ? kPast : qfirst;
      dma_to_lds(make_desc(qbase, qleft), off + j * MA::step(qrow), 0,
                 __builtin_amdgcn_readfirstlane(sb + (G::NW * j + wave) * 1024));
    } else {
      const int q = j - G::JA;
      const int off = !PSLOW && lkt * BK + pchunk * 8 >= a.len ? kPast : pfirst;
      dma_to_lds(make_desc(pbase, pleft), off + q * MB::step(prow), 0,
                 __builtin_amdgcn_readfirstlane(sb + G::A_BYTES + (G::NW * q + wave) * 1024));
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {
    if (++lkt >= lke) {
      ++li;
      load_item();
    } else {
      const int64_t qs = QSLOW ? (int64_t)BK * a.ldq * 2 : BK * 2, ps = PSLOW ? (int64_t)BK * a.ldp * 2 : BK * 2;
      qbase += qs; qleft -= qs;
      pbase += ps; pleft -= ps;
    }
  };

  // ---- fragments and products ----
  f32x16_t acc[WA][WB];
  bf16x8_t fa[WA], fb[2][WB];
  auto read_a = [&](int g, int s, int i) __attribute__((always_inline)) {
    return read_fragment<QSLOW, G::TA>(smem + (g % NS) * G::STAGE, (wr * WA + i) * 32, s, lane);
  };
  auto read_b = [&](int g, int s, int i) __attribute__((always_inline)) {
    return read_fragment<PSLOW, G::TB>(smem + (g % NS) * G::STAGE + G::A_BYTES, (wc * WB + i) * 32, s, lane);
  };
  // One substep: the WA x WB products of the held fragments; `reads` brings
  // substep (gn, sn)'s fragments, each A fragment right after its last use, B
  // into the other buffer; `loads` spreads the cursor's loads over the products.
  auto substep = [&](int cur, int gn, int sn, bool reads, bool loads, int ls) __attribute__((always_inline)) {
    constexpr int NI = WA * WB, PER = (G::LOADS + NI - 1) / NI;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int x = i / WB, y = i % WB;
      acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[x], fb[cur][y], acc[x][y], 0, 0, 0);
      if (reads && i < WB) fb[cur ^ 1][i] = read_b(gn, sn, i);
      if (reads && y == WB - 1) fa[x] = read_a(gn, sn, x);
      if (loads) {
#pragma unroll
        for (int q = 0; q < PER; ++q)
          if (i * PER + q < G::LOADS) load(ls, i * PER + q);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  auto epilogue = [&](const Item& it) __attribute__((always_inline)) {
    int fi = lane & 31, fg = lane >> 5;
    asm volatile("" : "+v"(fi), "+v"(fg));            // offsets formed here, not kept through the product loop
    float* part = it.part >= 0 ? a.partials + (int64_t)it.part * G::PARTIAL : nullptr;
#pragma unroll
    for (int y = 0; y < WB; ++y) {
      const int rl = (wc * WB + y) * 32 + fi, r = it.r0 + rl;
#pragma unroll
      for (int x = 0; x < WA; ++x) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int cl = (wr * WA + x) * 32 + q * 8 + fg * 4, c = it.c0 + cl;
          const float4 v = make_float4(acc[x][y][4 * q], acc[x][y][4 * q + 1], acc[x][y][4 * q + 2], acc[x][y][4 * q + 3]);
          if (part != nullptr) *reinterpret_cast<float4*>(part + rl * G::TA + cl) = v;
          else if (r < a.rows && c < a.cols) a.ep.template store4<ACT>(r, c, a.cols, v);
        }
        acc[x][y] = f32x16_t{};                       // the next item starts from zero
      }
    }
  };

  // Slice g of the stream lives in stage g % NS.  The first substep of slice g
  // issues the loads of slice g + NS - 1 into the stage that slice g - 1 left
  // (every wavefront was past it at the last barrier).  Before the last
  // substep: this wavefront's loads of slice g + 1 are in, its LDS reads done,
  // barrier; the last substep reads the first fragments of slice g + 1.
  load_item();
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
#pragma unroll
    for (int j = 0; j < G::LOADS; ++j) load(s, j);
    advance();
  }
  wait_vmcnt<G::LOADS * (NS - 2)>();
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int x = 0; x < WA; ++x)
#pragma unroll
    for (int y = 0; y < WB; ++y) acc[x][y] = f32x16_t{};
  int g = 0;
#pragma unroll
  for (int x = 0; x < WA; ++x) fa[x] = read_a(0, 0, x);
#pragma unroll
  for (int y = 0; y < WB; ++y) fb[0][y] = read_b(0, 0, y);
  for (int ci = 0; ci < n_items; ++ci) {
    const Item it = item(ci);
    for (int kt = it.kb; kt < it.ke; ++kt, ++g) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < G::SUB - 1; ++s) substep(s & 1, g, s + 1, true, s == 0, g + NS - 1);
      advance();
      wait_vmcnt<G::LOADS * (NS - 2)>();
      wait_lgkmcnt0();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      // (slice g + 1 may be the next item's first, or after the last item one that is never used)
      substep((G::SUB - 1) & 1, g + 1, 0, true, false, 0);
    }
    epilogue(it);
  }
  wait_vmcnt<0>();
}

// Sums the partial tiles of the split tail tiles in contraction order and applies
// the epilogue.  One workgroup per (XCD, tail tile, 32 rows of it).
template <int ACT, int TA, int TB>
__global__ __launch_bounds__(256) void linear_join_kernel(const ProductArgs a, int slots, int KT) {
  constexpr int RG = TB / 32;
  const int rg = blockIdx.x % RG, xcd = (blockIdx.x / RG) & 7, j = blockIdx.x / RG >> 3;
  const TileSplit sp = TileSplit::of(a.row_tiles * a.col_tiles, xcd, slots, KT);
  if (sp.whole_tail || j >= sp.tail) return;
  int rt, ct;
  tile_at(sp.share_begin + sp.R * slots + j, a.row_tiles, a.col_tiles, rt, ct);
  const int s_lo = j * KT / sp.P, s_hi = min(((j + 1) * KT - 1) / sp.P, slots - 1);
  const float* base = a.partials + (int64_t)(xcd * 2 * slots + j) * (TA * TB);
  for (int i = threadIdx.x; i < 32 * TA / 4; i += 256) {
    const int rl = rg * 32 + i / (TA / 4), cl = i % (TA / 4) * 4;
    const int r = rt * TB + rl, c = ct * TA + cl;
    if (r >= a.rows || c >= a.cols) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = s_lo; s <= s_hi; ++s) {
      const float4 p = *reinterpret_cast<const float4*>(base + (int64_t)s * (TA * TB) + rl * TA + cl);
      v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
    }
    a.ep.template store4<ACT>(r, c, a.cols, v);
  }
}

}  // namespace moe
