// Gated feed-forward block and its gradients on the fp32 matrix cores
// (v_mfma_f32_16x16x4_f32, f32_tiles.hpp): nothing is rounded below fp32.
//
// The products are those of FfnKind.  A workgroup of 4 wavefronts (2 x 2) has a tile
// of 32 B x 32 B of one group, each wavefront B x B blocks of 16 x 16.  kGateUp takes
// 16 channels of w1 and the same 16 of w3 in turn as column blocks, so that a lane
// holds g and u of the same elements; kDx walks dg, w1 and then du, w3.
// Where the tiles leave CUs idle the contraction is cut into runs whose results
// are summed in order by a second kernel, which has the same lanes and epilogue.
//
// A matrix core adds its terms to an fp32 sum one after the other, and what is added
// to a sum 2^n times as large loses n bits: of 2^20 rows of one sign dw2 lost 2.6e-4, of
// 2^24 3.3e-2.  LONG: results that may be sums of more than kLong terms are taken in
// chains of kChain, each joined to the sum of those before it in memory, where the
// result goes, which costs the loop no registers (2.4e-7 and 9e-7 are left).  All
// gradients, ms, without / with: 40000 rows of 4096 x 1024 22.7 / 19.8, 2^17 rows in 3
// groups of 1024 x 2048 39.5 / 38.4, 2^20 in one of 257 groups of 64 x 64 4.6 / 4.5,
// 40000 rows in 64 groups of 1024 x 1024, none of them long, 4.83 / 5.20 (two
// workgroups on a CU for three).
#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "f32_tiles.hpp"
#include "ffn_groups.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"

namespace moe {
namespace {

constexpr int kChain = 1 << 12, kLong = 1 << 15;
// Kinds whose sums are results themselves: over rows, and the two halves of kDx.
constexpr bool ffn_long_sums(int kind) { return ffn_over_rows(kind) || kind == kDx; }

struct FfnArgsF32 {
  const float *P0, *P1, *Q0, *Q1;      // P1, Q1: the second half where there are two
  const int32_t* offsets;
  int M, groups;
  int rows, cols, len;             // weight rows (kDw13, kDw2), columns (channels), terms of a half (else)
  int col_tiles, runs;
  int64_t group_tiles;             // kDw13, kDw2: tiles per group
  float* partials;
  const float *g, *u;              // kDh: pre-activations
  float *o0, *o1, *o2;
  int act;
};

template <int B>
struct FfnLdsF32 {
  float ps[2][32 * B * kTerms];
  float qs[2][32 * B * kTerms];
  FfnGroups groups;
};

template <int KIND, int B, bool JOIN, bool LONG>
__device__ __forceinline__ void ffn_f32_workgroup(const FfnArgsF32& a, FfnLdsF32<B>& lds, int block) {
  constexpr int T = 32 * B;
  constexpr bool OVER_ROWS = ffn_over_rows(KIND), PAIR = KIND == kGateUp, TWO = KIND == kDx;
  constexpr bool PSLOW = OVER_ROWS, QSLOW = KIND != kGateUp, CHAINS = LONG && ffn_long_sums(KIND);
  auto &ps = lds.ps, &qs = lds.qs;
  FfnGroups& groups = lds.groups;
  groups.load(a.offsets, a.groups, a.M, [](int rows) { return (rows + T - 1) / T; });
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int64_t tile = JOIN ? block : block / a.runs;
  const int run = JOIN ? 0 : block % a.runs;

  // the tile's group, first row and column, rows' end, and the operands there
  int e, r0, r_end, c0, len = a.len;
  const float *P0 = a.P0, *P1 = a.P1, *Q0 = a.Q0, *Q1 = a.Q1;
  float *o0 = a.o0, *o1 = a.o1;
  int64_t ldp, ldq;
  if constexpr (OVER_ROWS) {
    e = (int)(tile / a.group_tiles);
    int in = (int)(tile % a.group_tiles);
    if constexpr (KIND == kDw13) {
      const int half = (int)(a.group_tiles / 2);
      if (in >= half) {
        in -= half;
        P0 = P1;
        o0 = o1;
      }
    }
    r0 = in / a.col_tiles * T;
    c0 = in % a.col_tiles * T;
    r_end = a.rows;
    ldp = a.rows;
    ldq = a.cols;
    const int64_t first = groups.first(e);
    len = groups.first(e + 1) - groups.first(e);
    P0 += first * ldp;
    Q0 += first * ldq;
    o0 += (int64_t)e * a.rows * a.cols;
  } else {
    const int t = (int)(tile / a.col_tiles);
    if (t >= groups.before(a.groups)) return;                // the whole workgroup
    e = groups.of(t, a.groups);
    r0 = groups.first(e) + (t - groups.before(e)) * T;
    r_end = groups.first(e + 1);
    c0 = (int)(tile % a.col_tiles) * (PAIR ? T / 2 : T);     // kGateUp: channels
    ldp = a.len;
    ldq = PAIR ? a.len : a.cols;
    const int64_t w = (int64_t)e * a.cols * a.len;
    Q0 += w;
    if constexpr (PAIR || TWO) Q1 += w;
  }

  const int wr = (wave >> 1) * 16 * B, wc = (wave & 1) * 16 * B;
  f32x4_t acc[B][B];
#pragma unroll
  for (int x = 0; x < B; ++x)
#pragma unroll
    for (int y = 0; y < B; ++y) acc[x][y] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto partial = [&](int64_t r, int x, int y) __attribute__((always_inline)) {
    return a.partials + (((tile * a.runs + r) * 4 + wave) * (B * B) + x * B + y) * 256 + lane * 4;
  };

  if constexpr (!JOIN) {
    const int half_slices = (len + kTerms - 1) / kTerms, slices = TWO ? 2 * half_slices : half_slices;
    const int per = (slices + a.runs - 1) / a.runs, s0 = run * per, s1 = min(slices, s0 + per);
    SliceF32<PSLOW, T> p;
    SliceF32<QSLOW, T> q;
    auto load = [&](int s) __attribute__((always_inline)) {
      const bool second = TWO && s >= half_slices;
      const int t = (second ? s - half_slices : s) * kTerms;
      p.load(second ? P1 : P0, ldp, r0, r_end, t, len);
      if constexpr (PAIR) q.load_pair(Q0, Q1, ldq, c0, a.cols, t, len);
      else q.load(second ? Q1 : Q0, ldq, c0, a.cols, t, len);
    };
    for (int s = s0, stage = 0;;) {
      const bool more = s != s0;
      const int end = CHAINS ? min(s1, s + kChain / kTerms) : s1;
      if (s < end) load(s);
      for (; s < end; ++s, stage ^= 1) {
        p.store(ps[stage]);
        q.store(qs[stage]);
        __syncthreads();      // (the other stage's readers were past it at the last barrier)
        if (s + 1 < end) load(s + 1);
        multiply_f32<B>(ps[stage], qs[stage], wr, wc, i, g, acc);
      }
      if constexpr (!CHAINS) break;
#pragma unroll
      for (int y = 0; y < B; ++y)
#pragma unroll
        for (int x = 0; x < B; ++x) {
          const int r = r0 + wr + y * 16 + i, c = c0 + wc + x * 16 + 4 * g;
          f32x4_t* at = reinterpret_cast<f32x4_t*>(a.runs > 1 ? partial(run, x, y) : o0 + (int64_t)r * a.cols + c);
          if (a.runs > 1 || (r < r_end && c < a.cols)) {
            f32x4_t v = acc[x][y];
            if (more) v += *at;
            *at = v;
          }
          acc[x][y] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          __builtin_amdgcn_sched_barrier(0);
        }
      if (s >= s1) return;
    }
    if (a.runs > 1) {
#pragma unroll
      for (int y = 0; y < B; ++y)
#pragma unroll
        for (int x = 0; x < B; ++x) *reinterpret_cast<f32x4_t*>(partial(run, x, y)) = acc[x][y];
      return;
    }
  } else {
    for (int r = 0; r < a.runs; ++r) {
      f32x4_t v[B][B];
#pragma unroll
      for (int x = 0; x < B; ++x)
#pragma unroll
        for (int y = 0; y < B; ++y) v[x][y] = *reinterpret_cast<const f32x4_t*>(partial(r, x, y));
#pragma unroll
      for (int x = 0; x < B; ++x)
#pragma unroll
        for (int y = 0; y < B; ++y)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[x][y][k] += v[x][y][k];
    }
  }

  // lane (i, g): row y 16 + i, columns x 16 + 4 g .. + 3
#pragma unroll
  for (int y = 0; y < B; ++y) {
    const int r = r0 + wr + y * 16 + i;
    if (r >= r_end) continue;
    if constexpr (PAIR) {
#pragma unroll
      for (int x = 0; x < B; x += 2) {
        const int c = c0 + (wc + x * 16) / 2 + 4 * g;
        if (c >= a.cols) continue;
        const int64_t at = (int64_t)r * a.cols + c;
        const f32x4_t vg = acc[x][y], vu = acc[x + 1][y];
        float h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = act_value<true>(vg[k], a.act) * vu[k];
        store4(a.o0 + at, make_float4(h[0], h[1], h[2], h[3]));
        if (a.o1 != nullptr) {
          store4(a.o1 + at, make_float4(vg[0], vg[1], vg[2], vg[3]));
          store4(a.o2 + at, make_float4(vu[0], vu[1], vu[2], vu[3]));
        }
      }
    } else {
#pragma unroll
      for (int x = 0; x < B; ++x) {
        const int c = c0 + wc + x * 16 + 4 * g;
        if (c >= a.cols) continue;
        const int64_t at = (int64_t)r * a.cols + c;
        const float4 v = make_float4(acc[x][y][0], acc[x][y][1], acc[x][y][2], acc[x][y][3]);
        if constexpr (KIND == kDh) {
          const float4 pg = load4(a.g + at), pu = load4(a.u + at);
          const float vg[4] = {pg.x, pg.y, pg.z, pg.w}, vu[4] = {pu.x, pu.y, pu.z, pu.w}, d[4] = {v.x, v.y, v.z, v.w};
          float dg[4], du[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float value, slope;
            act_both<true>(vg[k], a.act, value, slope);
            dg[k] = d[k] * vu[k] * slope;
            du[k] = d[k] * value;
          }
          store4(a.o0 + at, make_float4(dg[0], dg[1], dg[2], dg[3]));
          store4(a.o1 + at, make_float4(du[0], du[1], du[2], du[3]));
        } else {
          store4(o0 + at, v);
        }
      }
    }
  }
}

// A's product (or join) on the first a_blocks workgroups, B's (another kind) on the others.
template <int KA, int KB, int B, bool JOIN, bool LONG>
__global__ __launch_bounds__(256) void ffn_f32_kernel(const FfnArgsF32 a, const FfnArgsF32 b, int a_blocks) {
  __shared__ __attribute__((aligned(16))) FfnLdsF32<B> lds;
  const int i = blockIdx.x;
  if (KA == KB || i < a_blocks) ffn_f32_workgroup<KA, B, JOIN, LONG>(a, lds, i);
  else ffn_f32_workgroup<KB, B, JOIN, LONG>(b, lds, i - a_blocks);
}

// 128 x 128 tiles where they give every CU one and the groups fill their rows, 64 x 64
// otherwise (257 groups of 4 rows, 2936 x 248, gate/up: 853 us in the large, 427 in the
// small); the contraction in
// as many runs as give each CU two workgroups, of 16 slices at least (a join is a
// launch more).
struct FfnPlanF32 {
  int T, col_tiles, runs;
  int64_t tiles, group_tiles;      // tiles: all that any offsets can give
  bool is_long;                    // a run may have sums of more than kLong terms (any group all rows)
  static FfnPlanF32 of(const moe_ffn_t& f, int kind) {
    FfnPlanF32 p{};
    const int64_t cus = device_cu_count();
    const bool over_rows = ffn_over_rows(kind);
    const int rows = kind == kDw2 ? f.d_model : f.d_ff, halves = kind == kDw13 ? 2 : 1;
    const int cols = kind == kGateUp ? 2 * f.d_ff : kind == kDh || kind == kDw2 ? f.d_ff : f.d_model;
    const int64_t len = over_rows ? (f.M + f.groups - 1) / f.groups
                        : kind == kDx ? 2 * (int64_t)f.d_ff : f.d_model;
    const int64_t most = over_rows ? f.M : len;
    for (p.T = 128;; p.T = 64) {
      p.col_tiles = (cols + p.T - 1) / p.T;
      p.group_tiles = over_rows ? (int64_t)halves * ((rows + p.T - 1) / p.T) * p.col_tiles : 0;
      const int64_t row_tiles = (f.M + p.T - 1) / p.T + f.groups - 1;
      p.tiles = over_rows ? p.group_tiles * f.groups : std::min<int64_t>(row_tiles, f.M) * p.col_tiles;
      const int64_t usual = over_rows ? p.tiles : std::max<int64_t>(p.tiles - (int64_t)(f.groups - 1) / 2 * p.col_tiles, 1);
      p.runs = (int)std::max<int64_t>(1, std::min<int64_t>({64, 2 * cus / usual, len / (16 * kTerms)}));
      p.is_long = ffn_long_sums(kind) && most > (int64_t)kLong * p.runs;
      if ((usual >= cus && (over_rows || f.M > 64 * (int64_t)f.groups)) || p.T == 64) return p;
    }
  }
  size_t workspace() const { return runs > 1 ? (size_t)tiles * runs * T * T * 4 : 0; }
};

FfnArgsF32 planned(const moe_ffn_t& f, const FfnPlanF32& p, FfnArgsF32 a, void* partials) {
  a.M = f.M;
  a.groups = f.groups;
  a.act = f.act;
  a.col_tiles = p.col_tiles;
  a.runs = p.runs;
  a.group_tiles = p.group_tiles;
  a.partials = static_cast<float*>(partials);
  return a;
}

// Two products that need nothing of each other: one launch where they have one tile
// size.  (A product alone: has_b false; KB is then not run.)
template <int KA, int KB>
hipError_t launch_pair(const moe_ffn_t& f, const FfnArgsF32& args_a, const FfnArgsF32& args_b, bool has_a, bool has_b,
                       void* partials, hipStream_t st) {
  const FfnPlanF32 pa = FfnPlanF32::of(f, KA), pb = FfnPlanF32::of(f, KB);
  if (has_a && has_b && pa.T != pb.T) {
    const hipError_t e = launch_pair<KA, KB>(f, args_a, args_b, true, false, partials, st);
    return e != hipSuccess ? e : launch_pair<KA, KB>(f, args_a, args_b, false, true, partials, st);
  }
  const FfnArgsF32 a = planned(f, pa, args_a, partials);
  const FfnArgsF32 b = planned(f, pb, args_b, static_cast<uint8_t*>(partials) + (has_a ? pa.workspace() : 0));
  auto run = [&](auto product, auto join) {
    const int64_t na = has_a ? pa.tiles * pa.runs : 0, nb = has_b ? pb.tiles * pb.runs : 0;
    hipLaunchKernelGGL(product, dim3((unsigned)(na + nb)), dim3(256), 0, st, a, b, (int)na);
    const hipError_t e = hipGetLastError();
    const int64_t ja = has_a && pa.runs > 1 ? pa.tiles : 0, jb = has_b && pb.runs > 1 ? pb.tiles : 0;
    if (e != hipSuccess || ja + jb == 0) return e;
    hipLaunchKernelGGL(join, dim3((unsigned)(ja + jb)), dim3(256), 0, st, a, b, (int)ja);
    return hipGetLastError();
  };
  const auto with = [&](auto b) {
    constexpr int B = decltype(b)::value;
    const auto join = ffn_f32_kernel<KA, KB, B, true, false>;
    if constexpr (ffn_long_sums(KA) || ffn_long_sums(KB))
      if ((has_a && pa.is_long) || (has_b && pb.is_long)) return run(ffn_f32_kernel<KA, KB, B, false, true>, join);
    return run(ffn_f32_kernel<KA, KB, B, false, false>, join);
  };
  return (has_a ? pa : pb).T == 128 ? with(std::integral_constant<int, 4>{}) : with(std::integral_constant<int, 2>{});
}

}  // namespace

size_t ffn_gate_up_bytes_f32(const moe_ffn_t& f) { return FfnPlanF32::of(f, kGateUp).workspace(); }

size_t ffn_backward_product_bytes_f32(const moe_ffn_t& f) {
  auto of = [&](int kind) { return FfnPlanF32::of(f, kind).workspace(); };
  return std::max(of(kDh) + of(kDw2), of(kDx) + of(kDw13));
}

hipError_t launch_ffn_gate_up_f32(const moe_ffn_t& f, const FfnTensors<float>& t, void* workspace, hipStream_t st) {
  FfnArgsF32 a{};
  a.P0 = t.x; a.Q0 = t.w1; a.Q1 = t.w3; a.offsets = t.offsets; a.cols = f.d_ff; a.len = f.d_model;
  a.o0 = t.h_out; a.o1 = t.g_out; a.o2 = t.u_out;
  return launch_pair<kGateUp, kGateUp>(f, a, a, true, false, workspace, st);
}

// dh and dw2, which need nothing of each other, then dx and dw1, dw3, which need dh's dg and du.
hipError_t launch_ffn_backward_f32(const moe_ffn_t& f, const FfnTensors<float>& t, void* partials, hipStream_t st) {
  FfnArgsF32 dh{}, dw2{}, dx{}, dw13{};
  dh.offsets = dw2.offsets = dx.offsets = dw13.offsets = t.offsets;
  dh.P0 = t.dy; dh.Q0 = t.w2; dh.cols = f.d_ff; dh.len = f.d_model; dh.g = t.g; dh.u = t.u; dh.o0 = t.dg; dh.o1 = t.du;
  dw2.P0 = t.dy; dw2.Q0 = t.h; dw2.rows = f.d_model; dw2.cols = f.d_ff; dw2.o0 = t.dw2;
  dx.P0 = t.dg; dx.P1 = t.du; dx.Q0 = t.w1; dx.Q1 = t.w3; dx.cols = f.d_model; dx.len = f.d_ff; dx.o0 = t.dx;
  dw13.P0 = t.dg; dw13.P1 = t.du; dw13.Q0 = t.x; dw13.rows = f.d_ff; dw13.cols = f.d_model; dw13.o0 = t.dw1;
  dw13.o1 = t.dw3;
  const bool inner = t.dx != nullptr || t.dw1 != nullptr;
  const hipError_t e = launch_pair<kDh, kDw2>(f, dh, dw2, inner, t.dw2 != nullptr, partials, st);
  if (e != hipSuccess || !inner) return e;
  return launch_pair<kDx, kDw13>(f, dx, dw13, t.dx != nullptr, t.dw1 != nullptr, partials, st);
}

}  // namespace moe
