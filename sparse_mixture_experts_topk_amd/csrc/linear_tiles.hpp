// Tiled dense product on the gfx950 matrix cores: out[r][c] = sum_t P(r, t) Q(c, t).
//
// P has `rows` rows, Q `cols` rows, the contraction `len` terms.  An operand is
// stored [r][t] (its contraction contiguous) or, SLOW, [t][r]; nothing is
// transposed in memory.  The matrix-core operand A is Q, B is P, so an
// accumulator block is [c][r]: a lane holds one row r and 4 consecutive c.
// v_mfma_f32_16x16x32_bf16 rather than 32x32x16: from registers, on random
// data, the card sustains 2080 against 1830 TFLOP/s (power sets its clock).
//
// A tile is TA x TB (c x r).  The contraction advances BK = 64 at a time
// through a ring of NS LDS stages, filled by buffer loads that write LDS
// directly.  A stage of an operand:
//   [r][t]: 128-byte rows of 64 terms; a fragment is one 16-byte read per lane.
//           16-byte chunk c of row r sits at c ^ fast_key(r), so that the 16
//           rows of a read phase cover all banks.
//   [t][r]: 64 rows of the tile's width; a fragment is two transposing 8-byte
//           reads (ds_read_b64_tr_b16: 16 lanes read 4 rows x 16 columns and
//           each gets one column).  Chunk c of row t sits at c ^ slow_key(t):
//           the 4 rows of a read go to different 64-byte quarters of the 256
//           bytes that the banks cover, rows t and t + 8 to different halves
//           of one (64-wide tiles: to the same effect), so no two of the lanes
//           served together share a bank.
// Neither has bank conflicts (SQ_LDS_BANK_CONFLICT 0).  Buffer descriptors are
// bounded to the operand's valid part and a chunk past the end of a [r][t] row
// is sent past it: such loads write zeros to LDS, on both operands, so a NaN
// next to the end cannot come in.
//
// The kernel is persistent (one workgroup per CU): workgroup b takes tiles of
// XCD b % 8's contiguous share of the tile list, and the slices of all its
// tiles form one stream through the ring, so the next tile's first slices load
// while this one's results are stored.  The last, partial round of tiles may be
// cut along the contraction over all workgroups (TileShare): their fp32 partial
// tiles are summed in order by a second kernel, which applies the epilogue.  The
// two products of a backward pass share one launch of each.
#pragma once
#include "device_common.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"
#include "lds_stream.hpp"
#include "persistent_tiles.hpp"

namespace moe {

// The tile list in 8 contiguous shares, one per XCD; the `slots` workgroups of
// an XCD take its full rounds of tiles, then the last `tail` < slots tiles either
// whole (the other workgroups idle) or, split, cut along the contraction into
// near-equal runs of P slices, one per workgroup, each covering parts of at most
// two tiles.  Which of the two is the plan's choice.
struct TileShare {
  int begin, R, tail, P;
  __host__ __device__ static TileShare of(int total, int xcd, int slots, int KT, bool split) {
    TileShare t;
    const int per_xcd = (total + 7) >> 3;
    t.begin = xcd * per_xcd;
    const int end = t.begin + per_xcd < total ? t.begin + per_xcd : total;
    const int len = end > t.begin ? end - t.begin : 0;
    t.R = len / slots;
    t.tail = len - t.R * slots;
    t.P = split ? (t.tail * KT + slots - 1) / slots : 0;
    return t;
  }
};

struct ProductArgs {
  const uint16_t* P;
  const uint16_t* Q;
  int64_t ldp, ldq;         // elements
  int rows, cols, len;
  int row_tiles, col_tiles;
  bool split;
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

// WR x WC wavefronts (c x r), each with WA x WB blocks of 16 x 16.
template <int NS, int WR, int WC, int WA_, int WB_>
struct ProductGeom {
  static constexpr int BK = 64, WA = WA_, WB = WB_;
  static constexpr int NW = WR * WC, THREADS = 64 * NW;
  static constexpr int TA = 16 * WR * WA, TB = 16 * WC * WB;
  static constexpr int A_BYTES = TA * BK * 2, B_BYTES = TB * BK * 2, STAGE = A_BYTES + B_BYTES;
  static constexpr int JA = A_BYTES / 1024 / NW, JB = B_BYTES / 1024 / NW, LOADS = JA + JB;
  static_assert(JA * NW * 1024 == A_BYTES && JB * NW * 1024 == B_BYTES && LOADS * (NS - 1) < 64,
                "whole loads per wavefront, counted by vmcnt");
  static_assert(NS >= 2 && NS * STAGE <= 160 * 1024, "LDS");
  static_assert(WA % 2 == 0, "the epilogue joins pairs of blocks");
  static constexpr int64_t PARTIAL = (int64_t)TA * TB;      // floats of a partial tile
  // The largest tile's outputs are large: stored past L2 (8192 x 14336 x 4096 with
  // pre kept 825 -> 735 us, the rows' pieces stored in order included).
  static constexpr bool STREAM = TA * TB >= 256 * 256;
};

__device__ __forceinline__ int fast_key(int row) { return (row >> 1) & 7; }
template <int TX>
__device__ __forceinline__ int slow_key(int t) {
  static_assert(TX >= 64 && TX % 64 == 0, "rows of at least 8 chunks");
  if constexpr (TX == 64) return (((t >> 1) & 1) << 1) | (((t >> 3) & 1) << 2);   // 128-byte rows: t's parity picks the half
  else return ((t & 3) << 2) | (((t >> 3) & 1) << 1);
}

// Which chunk of the operand this lane fetches in the wavefront's load j of a
// slice, and its byte offset in memory.  Load j covers LDS rows (NW j + wave)
// RPI ...; the swizzle repeats every PERIOD loads, so PERIOD offsets and a step
// give all of them.
template <bool SLOW, int TX, int NW>
struct LoadMap {
  static constexpr int CPR = SLOW ? TX / 8 : 8;            // chunks per LDS row
  static constexpr int RPI = 64 / CPR;                     // LDS rows per load
  static constexpr int PERIOD = NW * RPI >= 16 ? 1 : 16 / (NW * RPI);
  static_assert(64 % CPR == 0 && (NW * RPI * PERIOD) % 16 == 0, "whole swizzle periods");
  __device__ static __forceinline__ int chunk(int wave, int lane, int j) {
    const int row = (NW * j + wave) * RPI + lane / CPR;
    return (lane % CPR) ^ (SLOW ? slow_key<TX>(row) : fast_key(row));
  }
  __device__ static __forceinline__ int offset(int wave, int lane, int j, int rowbytes) {
    return (wave * RPI + lane / CPR) * rowbytes + chunk(wave, lane, j) * 16;   // + j * step
  }
  __device__ static __forceinline__ int step(int rowbytes) { return NW * RPI * rowbytes; }
  // Of two operands in turn, 16 rows of each: LDS rows (NW j + wave) 8 .. are rows 32 j +
  // 16 (wave / 4) + 8 (wave % 2) .. of operand wave / 2 % 2.
  __device__ static __forceinline__ int pair_offset(int wave, int lane, int rowbytes) {
    static_assert(SLOW || (NW == 8 && RPI == 8 && PERIOD == 1), "a wavefront's rows are all from one operand");
    return ((wave >> 2) * 16 + (wave & 1) * 8 + lane / CPR) * rowbytes + chunk(wave, lane, 0) * 16;
  }
  __device__ static __forceinline__ int pair_step(int rowbytes) { return 32 * rowbytes; }
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// Fragments of 16 operand rows x 32 terms for v_mfma_f32_16x16x32_bf16: lane
// (i, g) holds row i, terms 8 g .. 8 g + 7.  `lane_base` is this lane's byte
// offset in a stage for block 0 of the wavefront (first row row0, a multiple
// of the N blocks' rows), terms 0 .. 31; `read` adds block n and the half s.  In
// the [t][r] layout a block moves chunk bits that the swizzle also moves, so it
// enters by exclusive or (rows of the tile are a power of two of bytes).
template <bool SLOW, int TX, int N>
struct Fragments {
  static_assert((N & (N - 1)) == 0 && (!SLOW || (TX & (TX - 1)) == 0), "blocks and rows by bits");
  __device__ static __forceinline__ int lane_base(int row0, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (!SLOW) {
      return (row0 + i) * 128 + ((g ^ fast_key(i)) << 4);
    } else {
      const int t = 8 * g + (i >> 2), x = row0 + 4 * (i & 3);          // this lane's part of the 4 x 16 block
      return t * (TX * 2) + (((x >> 3) ^ slow_key<TX>(t)) << 4) + (x & 4) * 2;
    }
  }
  __device__ static __forceinline__ bf16x8_t read(const uint8_t* stage, int base, int n, int s) {
    if constexpr (!SLOW) {
      return as_bf16x8(*reinterpret_cast<const uint4*>(stage + (base ^ (s << 6)) + n * 16 * 128));
    } else {
      const uint8_t* p = stage + (base ^ (n << 5)) + s * 32 * (TX * 2);
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * (TX * 2)));
      return __builtin_bit_cast(bf16x8_t, s16x8_t{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w});
    }
  }
};

// Blocks x and x + 1 (16 columns each) of a row, 4 columns to a lane group of
// 16, become 8 consecutive columns per lane: group g of the result holds
// columns 8 g .. 8 g + 7 of the 32 (the half swap brings each block to one half
// of the wavefront, the row swap puts neighbouring fours together).
__device__ __forceinline__ void join_blocks(f32x4_t a, f32x4_t b, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(a[k]), __float_as_uint(b[k]), false, false);
    const auto q = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
    v[k] = __uint_as_float(q[0]);
    v[4 + k] = __uint_as_float(q[1]);
  }
}

// The stream of one workgroup's tiles.  The job says which they are, where their
// operands' slices lie and what becomes of the products:
//   n_items                 tiles, or runs of slices of one, of this workgroup
//   load_item(i), tile_item(i)   item i, slices [kb, ke), ke > kb: the first for the loads,
//                           the second for the products, each called with ascending i
//   descs(item, kt, first, dq, dp)   operands at slice kt of the item: a [t][r] operand's
//                           descriptor is of that slice (its rows may lie more than 2^31
//                           bytes apart), a [r][t] operand's of the tile (or a half of
//                           it, if the contraction has halves) and set when that begins
//   row_slice(kt), row_terms()   slice kt's place in a [r][t] operand's row, and the row's length
//   kPair                   Q is 16 rows of one operand and 16 of another in turn, both [r][t]
//                           (descs gives the one that this wavefront loads)
//   epilogue(item, acc, wr, wc, lane)   stores a tile's products and clears them, by
//                           kStores vector-memory instructions at least of every wavefront
template <bool PSLOW, bool QSLOW, int NS, int WR, int WC, int WA, int WB, class Job>
__device__ __forceinline__ void tile_stream(Job& job, int64_t ldp, int64_t ldq, uint8_t* smem) {
  using G = ProductGeom<NS, WR, WC, WA, WB>;
  using MA = LoadMap<QSLOW, G::TA, G::NW>;
  using MB = LoadMap<PSLOW, G::TB, G::NW>;
  constexpr int BK = G::BK;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC;

  // ---- loads ----
  // Load cursor: slice lkt of item li.  A [r][t] operand moves along its rows by the scalar offset.
  const uint32_t lds_base = (uint32_t)(uintptr_t)smem;
  const int qrow = (int)ldq * 2, prow = (int)ldp * 2;          // bytes
  int li = 0, lkt = 0;
  typename Job::Item lit{};
  i32x4_t dq, dp;
  auto load_item = [&]() __attribute__((always_inline)) {
    if (li < job.n_items) {
      lit = job.load_item(li);
      lkt = lit.kb;
      job.descs(lit, lkt, true, dq, dp);
    } else {                                       // past the last slice nothing is in range: zeros, no memory read
      dq = make_desc(job.base(), 0);
      dp = make_desc(job.base(), 0);
      lit.ke = 0x7fffffff;
    }
  };
  int qoff[MA::PERIOD], poff[MB::PERIOD], qch[MA::PERIOD], pch[MB::PERIOD];
#pragma unroll
  for (int j = 0; j < MA::PERIOD; ++j) {
    qoff[j] = Job::kPair ? MA::pair_offset(wave, lane, qrow) : MA::offset(wave, lane, j, qrow);
    qch[j] = MA::chunk(wave, lane, j) * 8;
  }
#pragma unroll
  for (int j = 0; j < MB::PERIOD; ++j) {
    poff[j] = MB::offset(wave, lane, j, prow);
    pch[j] = MB::chunk(wave, lane, j) * 8;
  }
  const int qstep = Job::kPair ? MA::pair_step(qrow) : MA::step(qrow);
  // a chunk of a [r][t] row past the contraction's end goes out of range
  constexpr int kPast = (int)0x80000000u;
  auto load = [&](int ls, int j) __attribute__((always_inline)) {
    const uint32_t sb = lds_base + (uint32_t)((ls % NS) * G::STAGE);
    const int k0 = job.row_slice(lkt) * BK;
    if (j < G::JA) {
      int off = qoff[j % MA::PERIOD];
      if constexpr (!QSLOW) off = k0 + qch[j % MA::PERIOD] >= job.row_terms() ? kPast : off;
      dma_to_lds(dq, off + j * qstep, QSLOW ? 0 : k0 * 2,
                 __builtin_amdgcn_readfirstlane(sb + (G::NW * j + wave) * 1024));
    } else {
      const int q = j - G::JA;
      int off = poff[q % MB::PERIOD];
      if constexpr (!PSLOW) off = k0 + pch[q % MB::PERIOD] >= job.row_terms() ? kPast : off;
      dma_to_lds(dp, off + q * MB::step(prow), PSLOW ? 0 : k0 * 2,
                 __builtin_amdgcn_readfirstlane(sb + G::A_BYTES + (G::NW * q + wave) * 1024));
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {
    if (++lkt >= lit.ke) {
      ++li;
      load_item();
    } else if (li < job.n_items) {
      job.descs(lit, lkt, false, dq, dp);
    }
  };

  // ---- fragments and products ----
  f32x4_t acc[WA][WB];
  bf16x8_t fa[2][WA], fb[WB];
  using FA = Fragments<QSLOW, G::TA, WA>;
  using FB = Fragments<PSLOW, G::TB, WB>;
  const int abase = FA::lane_base(wr * WA * 16, lane), bbase = FB::lane_base(wc * WB * 16, lane);
  auto read_a = [&](int g, int s, int i) __attribute__((always_inline)) {
    return FA::read(smem + (g % NS) * G::STAGE, abase, i, s);
  };
  auto read_b = [&](int g, int s, int i) __attribute__((always_inline)) {
    return FB::read(smem + (g % NS) * G::STAGE + G::A_BYTES, bbase, i, s);
  };
  // One half slice: the WA x WB products of the held fragments, B outermost.  The
  // next half's fragments (gn, sn) are read meanwhile: A into the other buffer
  // (from the second quarter on, clear of the barrier), each B right after its
  // last use.  `loads` spreads the cursor's loads over the products.  The
  // wavefront has priority meanwhile, so that of the two on a SIMD one runs
  // ahead and its waits fall under the other's products (dx 764 -> 704 us).
  auto half = [&](int cur, int gn, int sn, bool loads, int ls) __attribute__((always_inline)) {
    constexpr int NI = WA * WB, RA = NI / 4, GAP = NI / G::LOADS > 0 ? NI / G::LOADS : 1, PER = (G::LOADS + NI - 1) / NI;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int y = i / WA, x = i % WA;
      acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[cur][x], fb[y], acc[x][y], 0, 0, 0);
      if (i >= RA && i < RA + WA) fa[cur ^ 1][i - RA] = read_a(gn, sn, i - RA);
      if (x == WA - 1) fb[y] = read_b(gn, sn, y);
      if (loads && i % GAP == 0) {
#pragma unroll
        for (int q = 0; q < PER; ++q)
          if (i / GAP * PER + q < G::LOADS) load(ls, i / GAP * PER + q);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
  };

  // Slice g of the stream lives in stage g % NS.  Its first half reads the second
  // half's fragments; then this wavefront's loads of slice g + 1 are in, its LDS
  // reads done, barrier: slice g + 1 is whole and stage g % NS is no longer read.
  // The second half reads the first fragments of slice g + 1 and issues the loads
  // of slice g + NS into the freed stage, a whole slice (NS = 2) before their wait.
  load_item();
#pragma unroll
  for (int s = 0; s < NS; ++s) {
#pragma unroll
    for (int j = 0; j < G::LOADS; ++j) load(s, j);
    advance();
  }
  wait_vmcnt<G::LOADS * (NS - 1)>();
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int x = 0; x < WA; ++x)
#pragma unroll
    for (int y = 0; y < WB; ++y) acc[x][y] = f32x4_t{};
  // The wait is for the loads of slice g + 1 alone.  In the NS - 1 slices after an
  // epilogue these lie before its stores, which then may stay on their way.
  int g = 0, stored = -NS;
  for (int ci = 0; ci < job.n_items; ++ci) {
    const typename Job::Item it = job.tile_item(ci);
    // (read again after the last item's read ahead: no fragment lives through the epilogue)
#pragma unroll
    for (int x = 0; x < WA; ++x) fa[0][x] = read_a(g, 0, x);
#pragma unroll
    for (int y = 0; y < WB; ++y) fb[y] = read_b(g, 0, y);
    for (int kt = it.kb; kt < it.ke; ++kt, ++g) {
      __builtin_amdgcn_sched_barrier(0);
      half(0, g, 1, false, 0);
      if (Job::kStores > 0 && g - stored < NS - 1) wait_vmcnt<G::LOADS * (NS - 2) + Job::kStores>();
      else wait_vmcnt<G::LOADS * (NS - 2)>();
      wait_lgkmcnt0();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      half(1, g + 1, 0, true, g + NS);
      advance();
    }
    job.epilogue(it, acc, wr, wc, lane);
    stored = g;
  }
  wait_vmcnt<0>();   // the zero loads past the end land before the workgroup's LDS is released
}

// The job of workgroup `block` of the `blocks` (a multiple of 8) that share a dense product.
template <bool PSLOW, bool QSLOW, int ACT, class G>
struct DenseJob {
  static constexpr bool kPair = false;
  static constexpr int kStores = 0;      // (a wavefront without rows stores nothing)
  struct Item { int r0, c0, kb, ke, part; };
  const ProductArgs& a;
  TileShare sp;
  int KT, slots, xcd, slot, n_whole, run0, run1, n_items;

  __device__ __forceinline__ DenseJob(const ProductArgs& args, int block, int blocks) : a(args) {
    KT = (a.len + G::BK - 1) / G::BK;
    slots = blocks >> 3;
    xcd = block & 7;
    slot = block >> 3;
    sp = TileShare::of(a.row_tiles * a.col_tiles, xcd, slots, KT, a.split);
    n_whole = sp.R + (!a.split && slot < sp.tail ? 1 : 0);
    run0 = slot * sp.P;
    run1 = min(run0 + sp.P, sp.tail * KT);
    n_items = n_whole + (run0 < run1 ? (run1 - 1) / KT - run0 / KT + 1 : 0);
  }
  // Item i: a whole tile, or a run [kb, ke) of slices of tail tile j (partial tile slot + j of the XCD's).
  __device__ __forceinline__ Item item(int i) const {
    Item it{0, 0, 0, KT, -1};
    int t;
    if (i < n_whole) {
      t = sp.begin + slot + i * slots;
    } else {
      const int j = run0 / KT + (i - n_whole);
      t = sp.begin + sp.R * slots + j;
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
  }
  __device__ __forceinline__ Item load_item(int i) const { return item(i); }
  __device__ __forceinline__ Item tile_item(int i) const { return item(i); }
  __device__ __forceinline__ const void* base() const { return a.Q; }
  __device__ __forceinline__ int row_slice(int kt) const { return kt; }
  __device__ __forceinline__ int row_terms() const { return a.len; }
  __device__ __forceinline__ void descs(const Item& it, int kt, bool first, i32x4_t& dq, i32x4_t& dp) const {
    const int64_t t0 = (int64_t)kt * G::BK;
    if constexpr (QSLOW) dq = make_desc(a.Q + t0 * a.ldq + it.c0, ((a.len - t0) * a.ldq - it.c0) * 2);
    else if (first) dq = make_desc(a.Q + it.c0 * a.ldq, min(G::TA, a.cols - it.c0) * a.ldq * 2);
    if constexpr (PSLOW) dp = make_desc(a.P + t0 * a.ldp + it.r0, ((a.len - t0) * a.ldp - it.r0) * 2);
    else if (first) dp = make_desc(a.P + it.r0 * a.ldp, min(G::TB, a.rows - it.r0) * a.ldp * 2);
  }
  template <int WA, int WB>
  __device__ __forceinline__ void epilogue(const Item& it, f32x4_t (&acc)[WA][WB], int wr, int wc, int lane) const {
    int i = lane & 15, g = lane >> 4;
    float* part = it.part >= 0 ? a.partials + (int64_t)it.part * G::PARTIAL : nullptr;
    Epilogue ep = a.ep;
#pragma unroll
    for (int o = 0; o < WA * WB / 2; ++o) {
      const int x = o % (WA / 2) * 2, y = o / (WA / 2);          // a row's 64-byte pieces one after the other
      // Addresses are formed here and the choices made anew for every piece: kept in
      // registers, or followed through one copy of the epilogue per combination,
      // they would cost the product loop registers (spills: 0.7 -> 2.8 ms).
      asm volatile("" : "+v"(i), "+v"(g), "+s"(part), "+s"(ep.bias), "+s"(ep.residual), "+s"(ep.pre), "+s"(ep.f32));
      const int cl = (wr * WA + x) * 16 + 8 * g, c = it.c0 + cl;
      const int rl = (wc * WB + y) * 16 + i, r = it.r0 + rl;
      float v[8];
      join_blocks(acc[x][y], acc[x + 1][y], v);
      if (part != nullptr) store8f(part + rl * G::TA + cl, v);
      else if (r < a.rows && c < a.cols) ep.template store8<ACT, G::STREAM>(r, c, a.cols, v);
      acc[x][y] = acc[x + 1][y] = f32x4_t{};          // the next item starts from zero
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

template <bool PSLOW, bool QSLOW, int ACT, int NS, int WR, int WC, int WA, int WB>
__device__ __forceinline__ void product_workgroup(const ProductArgs& a, uint8_t* smem, int block, int blocks) {
  DenseJob<PSLOW, QSLOW, ACT, ProductGeom<NS, WR, WC, WA, WB>> job(a, block, blocks);
  if (job.n_items > 0) tile_stream<PSLOW, QSLOW, NS, WR, WC, WA, WB>(job, a.ldp, a.ldq, smem);
}

template <bool PSLOW, bool QSLOW, int ACT, int NS, int WR, int WC, int WA, int WB>
__global__ __launch_bounds__(64 * WR * WC, 1) void linear_product_kernel(const ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * ProductGeom<NS, WR, WC, WA, WB>::STAGE];
  product_workgroup<PSLOW, QSLOW, ACT, NS, WR, WC, WA, WB>(a, smem, blockIdx.x, gridDim.x);
}

// Sums the partial tiles of the split tail tiles in contraction order and applies
// the epilogue.  One workgroup per (XCD, tail tile, kJoinRows rows of it), 8
// columns of a row to a lane; four partials are in flight at a time.
template <int TA> constexpr int kJoinRows = 256 * 8 / TA;

template <int ACT, int TA, int TB>
__device__ __forceinline__ void join_workgroup(const ProductArgs& a, int slots, int block) {
  constexpr int RG = TB / kJoinRows<TA>;
  const int KT = (a.len + 63) / 64;
  const int rg = block % RG, xcd = (block / RG) & 7, j = block / RG >> 3;
  const TileShare sp = TileShare::of(a.row_tiles * a.col_tiles, xcd, slots, KT, true);
  if (j >= sp.tail) return;
  int rt, ct;
  tile_at(sp.begin + sp.R * slots + j, a.row_tiles, a.col_tiles, rt, ct);
  const int s_lo = j * KT / sp.P, s_hi = min(((j + 1) * KT - 1) / sp.P, slots - 1);
  const int rl = rg * kJoinRows<TA> + threadIdx.x / (TA / 8), cl = threadIdx.x % (TA / 8) * 8;
  const int r = rt * TB + rl, c = ct * TA + cl;
  if (r >= a.rows || c >= a.cols) return;
  const float* base = a.partials + (int64_t)(xcd * 2 * slots + j) * (TA * TB) + rl * TA + cl;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = s_lo; s <= s_hi; s += 4) {
    float p[4][8];
#pragma unroll
    for (int q = 0; q < 4; ++q) load8f(base + (int64_t)min(s + q, s_hi) * (TA * TB), p[q]);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += s + q <= s_hi ? p[q][k] : 0.0f;
  }
  a.ep.template store8<ACT>(r, c, a.cols, v);
}

template <int ACT, int TA, int TB>
__global__ __launch_bounds__(256) void linear_join_kernel(const ProductArgs a, int slots) {
  join_workgroup<ACT, TA, TB>(a, slots, blockIdx.x);
}

}  // namespace moe
