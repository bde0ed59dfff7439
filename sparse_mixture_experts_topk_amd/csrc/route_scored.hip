// Scored top-k routing from given logits, and its gradient at the logits.
//
// Pages: "How Mixtral 8x7B uses mixture of experts", the simplified forward
// pass (softmax over all experts, top-k, renormalise); "Mixtral 8x7B"
// interview page, section on how MoE design changed since Mixtral (256
// fine-grained experts, balanced without an auxiliary loss).
//
// Forward, per token: scores s = softmax(l) or sigmoid(l); choice c = s + b
// (b the balance bias); the score of a group of consecutive experts is its
// largest c or the sum of its two largest; the best `topk_groups` groups stay
// open and the k largest c of their experts are chosen, ties to the lower
// index.  The weights come from s alone: w_j = scale * s_j, or scale * s_j /
// (sum of the chosen s), the latter formed as e^(l_j - m) / sum e^(l_i - m)
// (softmax) or with every e^l taken relative to the largest chosen one
// (sigmoid), so that it holds where every score underflows.
//
// One wavefront per token.  The 64 lanes are cut into as many equal parts as
// there are groups (rounded up to a power of two), a group's experts lying in
// index order over its part's lanes, PER to a lane: a lane position, then a
// position within the lane, orders experts by index, so "the lowest lane that
// holds the maximum" settles ties.  Keys are the choices mapped to ordered
// unsigned integers (0: not a candidate), which also orders -inf (an expert
// that is only chosen when nothing else is left; a NaN choice counts as one), so
// k distinct experts always come out.  A NaN logit is read as -inf (usable), so
// that its rank, score, weight and gradient are those of a masked expert, in
// fp32 as in fp64; +inf is read as the largest number.
//
// The choice must not depend on how fp32 rounds the scores.  Without a
// balance bias the order of c is that of the logits and the keys are the
// logits themselves.  Otherwise the wavefront works in fp32 and looks at
// every gap that decided something (between consecutive chosen experts, the
// last chosen and the first left out, the last open group and the first closed):
// one within the fp32 error of the two values (k...Err) sends the token through
// the same steps in fp64, where scores of distinct fp32 logits are distinct until
// they saturate.  With 256 experts and N(0,1) logits about one token in 1500 goes
// that way.
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kRouteWaves = 4;     // tokens per workgroup
// Errors of a difference of two fp32 scores.  Sigmoid: 2.2e-7 each (exp and the
// reciprocal to 1 ulp, three roundings).  Softmax, of the largest score: the
// denominator's 8.5e-7 (a sum of depth 10 of exps), which both share, and 2e-7
// each.  c = s + b rounds once more, 2^-24 of its value.  A group's score has two
// scores' errors, its choices' roundings and that of their sum, 2^-24 (|c1| + |c2| +
// |c1 + c2|): of the choices' own sizes, which two of opposite sign do not show in
// their sum.  kGroupErr (|c1| + |c2|) holds these and the rounding of the score's end.
constexpr float kSoftmaxErr = 1.5e-6f;
constexpr float kSigmoidErr = 5e-7f;
constexpr float kSumErr = 1.25e-7f;
constexpr float kGroupErr = 1.9e-7f;
constexpr float kLargest = 3.402823466e38f;

// Order-preserving map of a value that is no NaN to unsigned integers; 0 is kept
// for "no candidate".
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);          // -0 -> +0
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ double from_ordered(uint64_t u) {
  return __longlong_as_double((long long)(u ^ ((u >> 63) ? 0x8000000000000000ull : ~0ull)));
}
// NaN becomes -inf (the maximum of a number and NaN is the number).
__device__ __forceinline__ float no_nan(float v) { return fmaxf(v, -INFINITY); }
__device__ __forceinline__ double no_nan(double v) { return fmax(v, -(double)INFINITY); }
// A logit as the router takes it: NaN as -inf, +inf as the largest number (differences
// of logits are then numbers or -inf).
__device__ __forceinline__ float usable(float v) { return fminf(no_nan(v), kLargest); }

// Reductions over the wavefront by DPP: row shifts within 16 lanes, then the two
// row broadcasts, leave the result in lane 63, read back as a uniform value.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_or(uint32_t none, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROW_MASK, 0xF, false);
}
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t none, Op op) {
  v = op(v, dpp_or<0x111, 0xF>(none, v));
  v = op(v, dpp_or<0x112, 0xF>(none, v));
  v = op(v, dpp_or<0x114, 0xF>(none, v));
  v = op(v, dpp_or<0x118, 0xF>(none, v));
  v = op(v, dpp_or<0x142, 0xA>(none, v));
  v = op(v, dpp_or<0x143, 0xC>(none, v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {       // the upper halves, then the lower ones of their largest
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  const uint32_t lo = wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
// (as ordered integers: one instruction a step, where fp32 maxima quiet their operands first)
__device__ __forceinline__ float wave_max_value(float v) { return from_ordered(wave_max(ordered(v))); }      // no NaN
__device__ __forceinline__ uint32_t lane_read(uint32_t v, int lane) { return (uint32_t)__shfl((int)v, lane); }
__device__ __forceinline__ uint64_t lane_read(uint64_t v, int lane) { return (uint64_t)__shfl((long long)v, lane); }
// A reduction's partner in step 0, 1, 2 over 8 lanes: lane ^ 1, lane ^ 2 (by quad),
// then the mirror within 8, whose quads already agree; step 3: the mirror within 16.
__device__ __forceinline__ uint32_t partner(uint32_t v, int step) {
  if (step == 0) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);
  if (step == 1) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);
  if (step == 2) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false);
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false);
}
__device__ __forceinline__ float xor_lane(float v, int step) {
  return __uint_as_float(partner(__float_as_uint(v), step));
}
// Sum and maximum over the 8 lanes that hold the chosen experts (equal in all 8).
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int i = 0; i < 3; ++i) v += xor_lane(v, i);
  return v;
}
__device__ __forceinline__ float max8(float v) {
#pragma unroll
  for (int i = 0; i < 3; ++i) v = fmaxf(v, xor_lane(v, i));
  return v;
}

// The renormalised weight of each of the 8 lanes' chosen logits: e^l (softmax) or
// sigmoid(l) over their sum, every term taken relative to the largest e^l, so that
// it holds where all scores underflow; 0 where every chosen logit is -inf.
__device__ __forceinline__ float chosen_weight(float lj, bool mine, bool softmax) {
  float m = fmaxf(max8(lj), -kLargest);
  float w;
  if (softmax) {
    w = exp_r(lj - m);
  } else {
    m = fminf(m, 0.0f);
    w = exp_r(fminf(lj, 0.0f) - m) * rcp_r(1.0f + exp_r(-fabsf(lj)));
  }
  if (!mine) w = 0.0f;
  const float sum = sum8(w);
  return sum > 0.0f ? w / sum : 0.0f;
}

struct RouteArgs {
  int T, E, k;
  int n_groups, group_size, lanes_per_group, group_shift, topk_groups, group_top;
  bool renormalize, vector;
  float scale;
  const float* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  float* scores;
  int32_t* next_ids;
};

// Scores of the lane's experts (0 at positions past the group), in R; returns a
// bound of the largest score of the token.
template <class R, int PER, bool SOFTMAX>
__device__ __forceinline__ R lane_scores(const float (&l)[PER], const bool (&in)[PER], float lmax, R (&s)[PER]) {
  if constexpr (!SOFTMAX) {
#pragma unroll
    for (int p = 0; p < PER; ++p) s[p] = sigmoid<R>((R)l[p]);       // past the group: l = -inf
    return R(1);
  }
  R z = 0;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const R e = exp_r((R)l[p] - (R)lmax);
    s[p] = in[p] ? e : R(0);
    z += s[p];
  }
  z = wave_sum(z);
  const R inv = z > 0 ? R(1) / z : R(0);           // every logit -inf: no score
#pragma unroll
  for (int p = 0; p < PER; ++p) s[p] *= inv;
  return inv;
}

// The `rounds` <= 16 best experts of the open groups into lanes 0 .. rounds - 1 of
// `chosen` (-1: no candidate left).  Returns whether fp32 could have decided
// any step wrongly (always false in fp64).
template <class R, int PER, bool SOFTMAX, bool BIAS, bool GROUPED>
__device__ __forceinline__ bool choose(const RouteArgs& a, const float (&l)[PER], const bool (&in)[PER],
                                       const float (&b)[PER], float lmax, bool need_scores, int lane, int rounds,
                                       R (&s)[PER], int& chosen) {
  using Key = std::conditional_t<sizeof(R) == 4, uint32_t, uint64_t>;
  constexpr bool CHECK = sizeof(R) == 4;
  const int lig = lane & (a.lanes_per_group - 1), grp = lane >> a.group_shift;
  bool near = false;
  float score_tol = 0;
  R smax = 0;
  if (BIAS || need_scores) {
    smax = lane_scores<R, PER, SOFTMAX>(l, in, lmax, s);
    score_tol = (SOFTMAX ? kSoftmaxErr : kSigmoidErr) * (float)smax;
  }
  // the lane's keys in descending order (equal ones by index), each with its position
  Key key[PER];
  int pos[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const Key k = ordered(BIAS ? no_nan(s[p] + (R)b[p]) : (R)l[p]);
    key[p] = in[p] ? k : Key(0);
    pos[p] = p;
  }
#pragma unroll
  for (int i = 1; i < PER; ++i)
#pragma unroll
    for (int j = i; j > 0; --j) {
      const bool up = key[j] > key[j - 1];
      const Key k0 = key[j - 1];
      const int p0 = pos[j - 1];
      key[j - 1] = up ? key[j] : k0;
      pos[j - 1] = up ? pos[j] : p0;
      key[j] = up ? k0 : key[j];
      pos[j] = up ? p0 : pos[j];
    }
  if constexpr (GROUPED) {
    // the group's two largest choices, merged over the part's lanes
    Key h1 = key[0], h2 = PER > 1 ? key[PER > 1 ? 1 : 0] : Key(0);
    auto merge = [&](Key o1, Key o2) __attribute__((always_inline)) {
      const Key lo = min(h1, o1), hi = max(h2, o2);
      h1 = max(h1, o1);
      h2 = max(lo, hi);
    };
    if constexpr (CHECK) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (a.lanes_per_group > (1 << i)) merge(partner(h1, i), partner(h2, i));
      if (a.lanes_per_group > 16) merge((Key)__shfl_xor((int)h1, 16), (Key)__shfl_xor((int)h2, 16));
    } else {
      for (int m = 1; m < a.lanes_per_group; m <<= 1)
        merge((Key)__shfl_xor((long long)h1, m), (Key)__shfl_xor((long long)h2, m));
    }
    // the group's score; without a bias the two logits' scores, unless one logit orders the groups
    const bool by_logit = !BIAS && a.group_top == 1;
    auto value = [&](Key h) __attribute__((always_inline)) -> R {
      const R v = from_ordered(h);
      if (BIAS || by_logit) return v;
      if constexpr (SOFTMAX) return no_nan(exp_r(v - (R)lmax) * smax);
      else return sigmoid<R>(v);
    };
    R gs = -(R)INFINITY, sizes = 0;                          // sizes: |c1| + |c2|
    if (h1 != 0) {
      const R c1 = value(h1), c2 = a.group_top == 1 ? R(0) : value(h2);
      gs = c1 + c2;
      sizes = fabs(c1) + fabs(c2);
    }
    const Key gk = ordered(no_nan(gs));
    const bool group = grp < a.n_groups;
    // groups ahead of the lane's own: lane i of a part looks at group i, i + lanes, ...
    int rank = 0;
    for (int base = 0; base < a.n_groups; base += a.lanes_per_group) {
      const int o = base + lig;
      const Key ok = lane_read(gk, o << a.group_shift);
      const uint64_t ahead = __ballot(o < a.n_groups && (ok > gk || (ok == gk && o < grp)));
      rank += __popc((uint32_t)(ahead >> (lane - lig)) & (uint32_t)((1ull << a.lanes_per_group) - 1));
    }
    const bool open = group && rank < a.topk_groups;
    if (!open) key[0] = 0;                                   // never the owner: the others need not go
    if constexpr (CHECK) {
      // every open group, at the lower end of its error, above every closed one at its upper end
      if (!by_logit) {
        const float err = kGroupErr * (float)sizes;
        const float kept = from_ordered(~wave_max(open ? ~ordered(no_nan(gs - err)) : 0u));
        const float shut = from_ordered(wave_max(group && !open ? ordered(no_nan(gs + err)) : 0u));
        near = !(kept - shut > 2 * score_tol);
      }
    }
  }
  const int first = grp * a.group_size + lig * PER;
#pragma unroll
  for (int p = 0; p < PER; ++p) pos[p] += first;
  chosen = -1;
  Key value = 0;                                             // lane r: the r-th chosen key
  for (int r = 0; r < rounds; ++r) {
    const Key top = wave_max(key[0]);
    if (top == 0) break;                                   // uniform: no candidate left
    const int owner = (int)__builtin_ctzll(__ballot(key[0] == top));       // the lowest index of equals
    const int e = __builtin_amdgcn_readlane(pos[0], owner);
    const bool slot = __builtin_amdgcn_inverse_ballot_w64(1ull << r);      // lane == r
    chosen = slot ? e : chosen;
    if constexpr (CHECK && BIAS) value = slot ? top : value;
    if (__builtin_amdgcn_inverse_ballot_w64(1ull << owner)) {              // its next one moves up
#pragma unroll
      for (int p = 0; p + 1 < PER; ++p) {
        key[p] = key[p + 1];
        pos[p] = pos[p + 1];
      }
      key[PER - 1] = 0;
    }
  }
  if constexpr (CHECK && BIAS) {
    const Key after = (Key)__builtin_amdgcn_mov_dpp((int)value, 0x101, 0xF, 0xF, false);     // lane r + 1's
    const float v = from_ordered(value), n = from_ordered(after);
    if (lane + 1 < rounds && after != 0)
      near |= !(v - n > score_tol + kSumErr * fmaxf(fabsf(v), fabsf(n)));
  }
  return CHECK && __ballot(near) != 0;
}

// The lane's PER consecutive values (those of in[]); vector: whole groups of 4 at 16-byte aligned places.
template <int PER>
__device__ __forceinline__ void load_lane(const float* p, const bool (&in)[PER], bool vector, float (&v)[PER]) {
  if constexpr (PER % 4 == 0) {
    if (vector) {
#pragma unroll
      for (int q = 0; q < PER; q += 4)
        if (in[q]) {
          const float4 f = *reinterpret_cast<const float4*>(p + q);
          v[q] = f.x; v[q + 1] = f.y; v[q + 2] = f.z; v[q + 3] = f.w;
        }
      return;
    }
  }
#pragma unroll
  for (int q = 0; q < PER; ++q)
    if (in[q]) v[q] = p[q];
}
template <int PER>
__device__ __forceinline__ void load_logits(const float* p, const bool (&in)[PER], bool vector, float (&l)[PER]) {
  load_lane<PER>(p, in, vector, l);
#pragma unroll
  for (int q = 0; q < PER; ++q) l[q] = usable(l[q]);
}

// Bound by instruction issue: 495 vector instructions per token, 20 of them in each
// of the k + 1 selection rounds (16384 tokens of 256 experts, sigmoid, 4 of 8
// groups, top 8, MI355X: 15.4-16.6 us; its 17.8 MB need 3.6).
template <int PER, bool SOFTMAX, bool BIAS, bool GROUPED>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_scored_kernel(const RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kRouteWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  const int lig = lane & (a.lanes_per_group - 1), grp = lane >> a.group_shift;
  const int first = grp * a.group_size + lig * PER;          // the lane's first expert
  const float* row = a.logits + (int64_t)t * a.E;
  float l[PER], b[PER];
  bool in[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    in[p] = grp < a.n_groups && lig * PER + p < a.group_size;
    l[p] = -INFINITY;
    b[p] = 0.0f;
  }
  load_logits<PER>(row + first, in, a.vector, l);
  if constexpr (BIAS) load_lane<PER>(a.bias + first, in, a.vector, b);
  // the softmax of all experts is not needed where the weights are
  // renormalised over the chosen ones and nothing else looks at scores
  const bool need_scores = BIAS || (GROUPED && a.group_top > 1) || a.scores != nullptr || (SOFTMAX && !a.renormalize);
  float lmax = -INFINITY;
  if (SOFTMAX && need_scores) {
#pragma unroll
    for (int p = 0; p < PER; ++p) lmax = fmaxf(lmax, l[p]);
    lmax = fmaxf(wave_max_value(lmax), -kLargest);    // all -inf: every term e^-inf
  }
  const int want = a.k + (a.next_ids != nullptr ? 2 : 0);
  float s[PER];
  int chosen;
  if (choose<float, PER, SOFTMAX, BIAS, GROUPED>(a, l, in, b, lmax, need_scores, lane, BIAS ? want + 1 : want, s, chosen)) {
    double s64[PER];
    choose<double, PER, SOFTMAX, BIAS, GROUPED>(a, l, in, b, lmax, need_scores, lane, want, s64, chosen);
  }
  if (a.scores != nullptr) {
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if (in[p]) a.scores[(int64_t)t * a.E + first + p] = s[p];
  }
  // weights: lane j < k holds the j-th chosen expert
  const bool mine = lane < a.k;
  const float lj = mine ? usable(row[chosen]) : -INFINITY;
  float w;
  if (a.renormalize) {
    w = chosen_weight(lj, mine, SOFTMAX);
  } else if (SOFTMAX) {
    // the token's softmax, its denominator from the lanes' experts again
    float z = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p) z += in[p] ? exp_r(l[p] - lmax) : 0.0f;
    z = wave_sum(z);
    w = z > 0.0f ? exp_r(lj - lmax) / z : 0.0f;
  } else {
    w = sigmoid(lj);
  }
  if (mine) {
    a.ids[(int64_t)t * a.k + lane] = chosen;
    a.weights[(int64_t)t * a.k + lane] = w * a.scale;
  }
  if (a.next_ids != nullptr && lane >= a.k && lane < a.k + 2)
    a.next_ids[(int64_t)t * 2 + lane - a.k] = chosen;
}

struct RouteBackArgs {
  int T, E, k;
  bool softmax, renormalize, vector;
  float scale;
  const float* logits;
  const int32_t* ids;
  const float* dweights;
  const float* dscores;
  float* dlogits;
};

// Gradient at the logits, one wavefront per token.  With D the gradient that
// arrives at the scores (0 without one), g the one at the weights and, when
// renormalised, w' = s / (sum of the chosen s) and
//   q_j = scale w'_j sum_i w'_i (g_j - g_i),
//   softmax:  dl_e = q_e + s_e (D_e - sum_i D_i s_i)
//   sigmoid:  dl_e = q_e (1 - s_e) + D_e s_e (1 - s_e)
// else, with a_e = D_e + scale g_e,
//   softmax:  dl_e = s_e (a_e - sum_i a_i s_i)
//   sigmoid:  dl_e = a_e s_e (1 - s_e).
// The differences g_j - g_i are taken before they are weighted: they hold
// where the g are near each other.  1 - sigmoid(l) is sigmoid(-l).
// HBM-bound: reads 4 E bytes (8 E with D) and writes 4 E per token (16384 x 256,
// sigmoid, MI355X: 9.7 us, 3.6 TB/s).
template <int PER>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_scored_backward_kernel(const RouteBackArgs a) {
  __shared__ __attribute__((aligned(16))) float at_chosen[kRouteWaves][kWave * PER];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= a.T) return;
  const int64_t base = (int64_t)t * a.E;
  float l[PER], d[PER];
  bool in[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    in[p] = lane * PER + p < a.E;
    l[p] = -INFINITY;
    d[p] = 0.0f;
  }
  // renormalised softmax weights do not see the other experts' logits
  const bool need = !(a.softmax && a.renormalize) || a.dscores != nullptr;
  if (need) load_logits<PER>(a.logits + base + lane * PER, in, a.vector, l);
  if (a.dscores != nullptr) load_lane<PER>(a.dscores + base + lane * PER, in, a.vector, d);
  // lanes j < k: the j-th chosen expert (an id outside the row adds nothing)
  int id = lane < a.k ? a.ids[(int64_t)t * a.k + lane] : -1;
  if (id >= a.E) id = -1;
  const float g = id >= 0 ? a.dweights[(int64_t)t * a.k + lane] : 0.0f;
  float q = a.scale * g;
  if (a.renormalize) {
    const float lj = id >= 0 ? usable(a.logits[base + id]) : -INFINITY;
    const float w = chosen_weight(lj, id >= 0, a.softmax);
    float c = 0.0f;
#pragma unroll
    for (int x = 1; x < 8; ++x) c += __shfl_xor(w, x) * (g - __shfl_xor(g, x));
    q = a.scale * w * c;
  }
  // q to the lanes that hold the chosen experts, through the wavefront's own LDS
  // row (LDS operations of one wavefront execute in order)
  float* row = at_chosen[wave];
#pragma unroll
  for (int p = 0; p < PER; ++p) row[lane * PER + p] = 0.0f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (id >= 0) atomicAdd(&row[id], q);       // (an expert named twice gets both)
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  float sel[PER], out[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) sel[p] = row[lane * PER + p];
  if (a.softmax) {
    if (need) {
      float lmax = -INFINITY;
#pragma unroll
      for (int p = 0; p < PER; ++p) lmax = fmaxf(lmax, l[p]);
      lmax = fmaxf(wave_max_value(lmax), -kLargest);
      float s[PER], z = 0.0f, dot = 0.0f;
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        s[p] = exp_r(l[p] - lmax);
        z += s[p];
        if (!a.renormalize) d[p] += sel[p];
        dot += d[p] * s[p];
      }
      z = wave_sum(z);
      dot = wave_sum(dot);
      const float inv = z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
      for (int p = 0; p < PER; ++p)
        out[p] = (a.renormalize ? sel[p] : 0.0f) + s[p] * inv * (d[p] - dot * inv);
    } else {
#pragma unroll
      for (int p = 0; p < PER; ++p) out[p] = sel[p];
    }
  } else {
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      float s, below;                                          // below: 1 - s
      sigmoids(l[p], s, below);
      out[p] = a.renormalize ? sel[p] * below + d[p] * s * below : (d[p] + sel[p]) * s * below;
    }
  }
  float* o = a.dlogits + base + lane * PER;
  if constexpr (PER % 4 == 0) {
    if (a.vector) {
      if (in[0]) *reinterpret_cast<float4*>(o) = make_float4(out[0], out[1], out[2], out[3]);
      return;
    }
  }
#pragma unroll
  for (int p = 0; p < PER; ++p)
    if (in[p]) o[p] = out[p];
}

}  // namespace

hipError_t launch_route_scored(const moe_shape_t& s, const moe_router_t& r, const float* logits, const float* bias,
                               int32_t* ids, float* weights, float* scores, int32_t* next_ids, hipStream_t st) {
  RouteArgs a{};
  a.T = s.T; a.E = s.n_experts; a.k = s.top_k;
  a.n_groups = r.n_groups;
  a.group_size = s.n_experts / r.n_groups;
  int parts = 1;
  while (parts < r.n_groups) parts *= 2;
  a.lanes_per_group = kWave / parts;
  a.group_shift = 6;
  while ((1 << a.group_shift) > a.lanes_per_group) --a.group_shift;
  a.vector = a.group_size % 4 == 0;
  a.topk_groups = r.topk_groups;
  a.group_top = r.group_top;
  a.renormalize = r.renormalize != 0;
  a.scale = r.scale;
  a.logits = logits; a.bias = bias; a.ids = ids; a.weights = weights; a.scores = scores; a.next_ids = next_ids;
  const int per = (a.group_size + a.lanes_per_group - 1) / a.lanes_per_group;
  const dim3 grid((unsigned)((s.T + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * kWave);
  // groups that are all open decide nothing, but keep the lanes' layout
  const bool softmax = r.score == MOE_SCORE_SOFTMAX, biased = bias != nullptr, grouped = r.topk_groups < r.n_groups;
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, st, a);
    return hipGetLastError();
  };
  auto by_per = [&](auto sm, auto bi, auto gr) {
    constexpr bool S = decltype(sm)::value, B = decltype(bi)::value, G = decltype(gr)::value;
    if (per <= 1) return run(route_scored_kernel<1, S, B, G>);
    if (per <= 2) return run(route_scored_kernel<2, S, B, G>);
    if (per <= 4) return run(route_scored_kernel<4, S, B, G>);
    return run(route_scored_kernel<8, S, B, G>);
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  if (softmax && biased) return grouped ? by_per(yes, yes, yes) : by_per(yes, yes, no);
  if (softmax) return grouped ? by_per(yes, no, yes) : by_per(yes, no, no);
  if (biased) return grouped ? by_per(no, yes, yes) : by_per(no, yes, no);
  return grouped ? by_per(no, no, yes) : by_per(no, no, no);
}

hipError_t launch_route_scored_backward(const moe_shape_t& s, const moe_router_t& r, const float* logits,
                                        const int32_t* ids, const float* dweights, const float* dscores,
                                        float* dlogits, hipStream_t st) {
  RouteBackArgs a{s.T, s.n_experts, s.top_k, r.score == MOE_SCORE_SOFTMAX, r.renormalize != 0, s.n_experts % 4 == 0,
                  r.scale, logits, ids, dweights, dscores, dlogits};
  const dim3 grid((unsigned)((s.T + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * kWave);
  if (a.E <= 64) hipLaunchKernelGGL(route_scored_backward_kernel<1>, grid, block, 0, st, a);
  else if (a.E <= 128) hipLaunchKernelGGL(route_scored_backward_kernel<2>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(route_scored_backward_kernel<4>, grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace moe
