// Routing of tokens to experts and its gradient (gfx950).
//
//   s = softmax(l) or sigmoid(l) over the E logits of a token;  key = s + bias (without a bias: l orders)
//   an expert with l = -inf or key = -inf is never chosen
//   groups: the score of a group of E / G neighbouring experts is the sum of its two highest keys (s where there is
//   no bias; the highest where it has one); the experts of all but the best top_groups groups are not chosen
//   chosen: the highest keys, descending, ties to the lowest index; slots left over get id -1 and weight 0
//   w_j = scale s_j / sum_i s_i (renormalised; 0 where the sum is 0) or scale s_j
//   a token with a NaN key (or softmax of +inf): ids 0 .. top - 1, weights NaN
//
// One wave a token, lane l holding experts l, l + 64, ..  Keys are formed in 64 bits: two experts' scores lie within
// a 32-bit rounding of each other every few thousand tokens, and the choice must not depend on how exp is rounded.
// As unsigned integers that order as the keys do, their upper halves alone nearly always single out one lane:
// an arg max is a 32-bit maximum by DPP and a ballot, the lower halves and the index only decide where more than
// one lane has it.
//   Few tokens are bound by the chain of dependent steps: 16 tokens of 256 experts with a bias and 8 groups take 6.2 us (8.4
// with exchanges through LDS and keys searched again for every choice), 2.2 of them an empty launch.  Many are bound by
// the vector instructions of the choices: 16384 tokens of 128 experts, bf16, 12.4 us and 10.1 for the gradient, where
// their 4 and 8 MB would take 1 and 2.
#include <hip/hip_runtime.h>

#include <cmath>

#include "aq_device.h"
#include "aq_kernels.h"

namespace aq {

namespace {

constexpr int kTokens = 4;   // waves of a workgroup, a token each

__device__ __forceinline__ uint32_t lane_id() { return threadIdx.x & 63; }

// Exchanges within the wave by DPP and lane swaps (a fifth of the time of exchanges through LDS).  A value that is the
// same in all lanes of a quad, half row, row or half wave meets its partner's there, so that after the steps up to
// `lanes` all of them hold f over the lanes, from operands that only change places: the same bits in every lane.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 | dpp<CTRL>((uint32_t)u));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;   // quad_perm [1,0,3,2], [2,3,0,1]

// f(value of the lane's half, of the other half) where the halves are rows (32 lanes) or half waves
template <bool ROWS, class F>
__device__ __forceinline__ double across(double v, F f) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t h = (uint32_t)(u >> 32), l = (uint32_t)u;
  const auto a = ROWS ? __builtin_amdgcn_permlane16_swap(h, h, false, false) : __builtin_amdgcn_permlane32_swap(h, h, false, false);
  const auto b = ROWS ? __builtin_amdgcn_permlane16_swap(l, l, false, false) : __builtin_amdgcn_permlane32_swap(l, l, false, false);
  return f(__builtin_bit_cast(double, (uint64_t)a[0] << 32 | b[0]), __builtin_bit_cast(double, (uint64_t)a[1] << 32 | b[1]));
}

// max over the wave, in every lane
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  v = max(v, dpp<kMirror>(v));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

__device__ __forceinline__ double wave_sum64(double v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  const auto plus = [](double a, double b) { return a + b; };
  return across<false>(across<true>(v, plus), plus);
}

__device__ __forceinline__ double readlane64(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t h = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane), l = __builtin_amdgcn_readlane((uint32_t)u, lane);
  return __builtin_bit_cast(double, (uint64_t)h << 32 | l);
}

// integers that order as the numbers do, above 0 (0: never chosen; -inf gives 0x000F.. in 64 bits, above 0 too)
__device__ __forceinline__ uint64_t order(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);   // (-0 as 0)
  return u >> 63 ? ~u : u | (uint64_t(1) << 63);
}
__device__ __forceinline__ uint32_t order(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float wave_max(float v) {   // (not NaN)
  const uint32_t h = wave_umax(order(v));
  return __uint_as_float(h >> 31 ? h & 0x7FFFFFFFu : ~h);
}

template <bool BF16>
__device__ __forceinline__ float logit(const void* L, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(L)[i]);
  else return static_cast<const float*>(L)[i];
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// The lane and index of the largest key; keys of 32 or 64 bits in two halves.  `best` is this lane's largest key's
// halves and `index` its expert, the lowest of its equals; a lane without one has zero.
struct Winner {
  int lane;
  uint32_t index;
};
template <bool WIDE>
__device__ __forceinline__ bool wave_best(uint32_t hi, uint32_t lo, uint32_t index, Winner& out) {
  const uint32_t top = wave_umax(hi);
  if (top == 0) return false;
  uint64_t who = __ballot(hi == top);
  if (who & (who - 1)) {
    if constexpr (WIDE) {
      const uint32_t low = wave_umax(hi == top ? lo : 0u);
      who = __ballot(hi == top && lo == low);
    }
    if (who & (who - 1)) {
      const bool in = who >> lane_id() & 1;
      const uint32_t first = ~wave_umax(in ? ~index : 0u);
      who = __ballot(in && index == first);
    }
  }
  out.lane = __builtin_ctzll(who);
  out.index = __builtin_amdgcn_readlane(index, out.lane);
  return true;
}

// P: experts a lane; BIAS: keys are 64-bit scores plus bias, else the logits themselves
template <int P, bool BF16, bool BIAS>
__global__ __launch_bounds__(64 * kTokens) void route_kernel(RouteArgs a) {
  extern __shared__ double keys[];   // groups: [kTokens][E]
  const int wave = threadIdx.x >> 6;
  const int lane = lane_id();
  const int64_t t = (int64_t)blockIdx.x * kTokens + wave;
  if (t >= a.T) return;
  const int64_t row = t * a.ld;
  float l[P];
  bool wrong = false;
  float high = -INFINITY;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < a.E ? logit<BF16>(a.logits, row + e) : -INFINITY;
    wrong |= l[i] != l[i] || (!a.sigmoid && l[i] == INFINITY);
    high = fmaxf(high, l[i]);
  }
  // scores where they are needed: for keys with a bias, for the groups' sums, for shares of the whole softmax
  const bool grouped = a.groups > 1;
  const bool whole = !a.sigmoid && (BIAS || grouped || !a.renormalize);
  double total = 1.0, top_l = 0.0;
  double s[P];
  if (whole) {
    const float hf = wave_max(high);
    top_l = hf == -INFINITY ? 0.0 : hf;
    total = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      s[i] = exp((double)l[i] - top_l);
      total += s[i];
    }
    total = wave_sum64(total);
    if (total == 0.0) total = 1.0;   // every expert masked
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] /= total;
  } else if (BIAS || grouped) {
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = sigmoid64(l[i]);
  }
  uint32_t hi[P], lo[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    double k = 0.0;
    if constexpr (BIAS) {
      k = s[i] + (e < a.E ? (double)a.bias[e] : 0.0);
      wrong |= k != k;
      const uint64_t u = l[i] == -INFINITY || k == -INFINITY ? 0 : order(k);
      hi[i] = (uint32_t)(u >> 32);
      lo[i] = (uint32_t)u;
    } else {
      hi[i] = l[i] == -INFINITY ? 0 : order(l[i]);
      lo[i] = 0;
      if (grouped) k = s[i];
    }
    if (grouped && e < a.E) keys[wave * a.E + e] = hi[i] ? k : -INFINITY;
  }
  wrong = __any(wrong);
  if (wrong) {
    if (lane < a.top) {
      a.ids[t * a.top + lane] = lane;
      a.weights[t * a.top + lane] = __builtin_nanf("");
    }
    return;
  }

  if (grouped) {
    wave_order();   // (lanes read keys that others wrote)
    // q lanes a group, each over every q-th of its experts; then the group's two highest by exchanges
    const int q = a.lanes, size = a.E / a.groups, g = lane / q;
    double one = -INFINITY, two = -INFINITY;
    if (g < a.groups)
      for (int i = lane % q; i < size; i += q) {
        const double k = keys[wave * a.E + g * size + i];
        two = fmax(two, fmin(one, k));
        one = fmax(one, k);
      }
    // the two highest of this lane's and its partner's two
    auto meet = [&](double x, double y) {
      two = fmax(fmax(two, y), fmin(one, x));
      one = fmax(one, x);
    };
    if (q > 1) meet(dpp<kXor1>(one), dpp<kXor1>(two));
    if (q > 2) meet(dpp<kXor2>(one), dpp<kXor2>(two));
    if (q > 4) meet(dpp<kHalfMirror>(one), dpp<kHalfMirror>(two));
    if (q > 8) meet(dpp<kMirror>(one), dpp<kMirror>(two));
    if (q > 16) {   // (two groups: 32 lanes each)
      const bool odd = lane >> 4 & 1;
      double x[2], y[2];
      across<true>(one, [&](double a, double b) { return x[0] = a, x[1] = b, a; });
      across<true>(two, [&](double a, double b) { return y[0] = a, y[1] = b, a; });
      meet(odd ? x[0] : x[1], odd ? y[0] : y[1]);
    }
    const double score = two == -INFINITY ? one : one + two;
    int rank = 0;   // groups ahead of this lane's
    for (int j = 0; j < a.groups; ++j) {
      const double other = readlane64(score, j * q);
      rank += other > score || (other == score && j < g);
    }
    const uint64_t stay = __ballot(g < a.groups && lane % q == 0 && rank < a.top_groups);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane + 64 * i, group = (int)((uint32_t)e * a.magic >> 20);   // e / size
      if (e < a.E && !(stay >> (group * q) & 1)) hi[i] = lo[i] = 0;
    }
  }

  // the choices, one after the other; lane j keeps the j-th
  int id = -1;
  if constexpr (P <= 4) {
    // a lane's keys in order, the winner's move up
    uint32_t at[P];
#pragma unroll
    for (int i = 0; i < P; ++i) at[i] = lane + 64 * i;
    auto sort2 = [&](int i, int j) {
      const bool swap = hi[j] > hi[i] || (hi[j] == hi[i] && (lo[j] > lo[i] || (lo[j] == lo[i] && at[j] < at[i])));
      const uint32_t h = hi[i], l = lo[i], x = at[i];
      hi[i] = swap ? hi[j] : h, lo[i] = swap ? lo[j] : l, at[i] = swap ? at[j] : x;
      hi[j] = swap ? h : hi[j], lo[j] = swap ? l : lo[j], at[j] = swap ? x : at[j];
    };
    if constexpr (P == 2) sort2(0, 1);
    if constexpr (P == 4) sort2(0, 1), sort2(2, 3), sort2(0, 2), sort2(1, 3), sort2(1, 2);
    for (int j = 0; j < a.top; ++j) {
      Winner w;
      if (!wave_best<BIAS>(hi[0], lo[0], at[0], w)) break;
      if (lane == j) id = (int)w.index;
      const bool mine = lane == w.lane;
#pragma unroll
      for (int i = 0; i + 1 < P; ++i) {
        hi[i] = mine ? hi[i + 1] : hi[i];
        lo[i] = mine ? lo[i + 1] : lo[i];
        at[i] = mine ? at[i + 1] : at[i];
      }
      hi[P - 1] = mine ? 0 : hi[P - 1];
    }
  } else {
    // the winner's lane looks through its keys again (8 or 16: ordering them all would cost more than eight choices)
    uint32_t bh = 0, bl = 0, bi = 0;
    auto local = [&]() {
      bh = bl = 0;
      bi = lane;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const bool more = BIAS ? hi[i] > bh || (hi[i] == bh && lo[i] > bl) : hi[i] > bh;
        if (more) {
          bh = hi[i];
          bl = lo[i];
          bi = lane + 64 * i;
        }
      }
    };
    local();
    for (int j = 0; j < a.top; ++j) {
      Winner w;
      if (!wave_best<BIAS>(bh, bl, bi, w)) break;
      if (lane == j) id = (int)w.index;
      if (lane == w.lane) {
#pragma unroll
        for (int i = 0; i < P; ++i)
          if ((int)w.index == lane + 64 * i) hi[i] = lo[i] = 0;
        local();
      }
    }
  }

  // their scores again, from the logits
  double share = 0.0;
  const float chosen = id >= 0 ? logit<BF16>(a.logits, row + id) : -INFINITY;
  const double mine = chosen;
  if (a.sigmoid) {
    if (id >= 0) share = sigmoid64(mine);
  } else if (a.renormalize) {
    // relative to the chosen ones' highest: their sum is at least 1
    const float h = wave_max(chosen);
    if (id >= 0) share = exp(mine - h);
  } else if (id >= 0) {
    share = exp(mine - top_l) / total;
  }
  if (a.renormalize) {
    const double sum = wave_sum64(share);
    share = sum > 0.0 ? share / sum : 0.0;
  }
  if (lane < a.top) {
    a.ids[t * a.top + lane] = id;
    a.weights[t * a.top + lane] = (float)(a.scale * share);
  }
}

// With a_j the share w_j / scale and d_j = scale dL/dw_j, m = sum_j a_j d_j:
//   softmax, renormalised   dl_j = a_j (d_j - m)                      (chosen experts only)
//   softmax                 dl_e = p_e (d_e - m), d_e = 0 where e is not chosen
//   sigmoid, renormalised   dl_j = (d_j - m) / sum s  s_j (1 - s_j)   sigmoid  dl_j = d_j s_j (1 - s_j)
// in 64 bits, rounded once; 1 - s as sigmoid(-l).  Moves bytes: a lane's experts are written whether chosen or not.
template <int P, bool BF16>
__global__ __launch_bounds__(64 * kTokens) void route_backward_kernel(RouteArgs a, const float* __restrict__ grad,
                                                                       void* __restrict__ dlogits) {
  const int lane = lane_id();
  const int64_t t = (int64_t)blockIdx.x * kTokens + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int64_t row = t * a.ld;
  int id = -1;
  double d = 0.0, mine = -INFINITY;
  bool nan = false;
  if (lane < a.top) {
    id = a.ids[t * a.top + lane];
    if (id < 0 || id >= a.E) id = -1;
    if (id >= 0) {
      d = (double)a.scale * grad[t * a.top + lane];
      mine = logit<BF16>(a.logits, row + id);
      nan = a.weights[t * a.top + lane] != a.weights[t * a.top + lane];
    }
  }
  double p[P];
  double v = 0.0, m = 0.0;
  const bool whole = !a.sigmoid && !a.renormalize;
  if (whole) {
    float l[P], high = -INFINITY;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane + 64 * i;
      l[i] = e < a.E ? logit<BF16>(a.logits, row + e) : -INFINITY;
      high = fmaxf(high, l[i]);
    }
    const float hf = wave_max(high);
    const double top_l = hf == -INFINITY ? 0.0 : hf;
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      p[i] = exp((double)l[i] - top_l);
      total += p[i];
    }
    total = wave_sum64(total);
    if (total == 0.0) total = 1.0;
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] /= total;
    v = id >= 0 ? exp(mine - top_l) / total * d : 0.0;   // p_j d_j, added to the chosen expert's
    m = wave_sum64(v);
  } else if (!a.sigmoid) {
    const float h = wave_max((float)mine);
    const double s = id >= 0 ? exp(mine - h) : 0.0;
    const double sum = wave_sum64(s);
    const double share = sum > 0.0 ? s / sum : 0.0;
    m = wave_sum64(share * d);
    v = share * (d - m);
  } else {
    const double s = id >= 0 ? sigmoid64(mine) : 0.0;
    double f = d;
    if (a.renormalize) {
      const double sum = wave_sum64(s);
      m = sum > 0.0 ? wave_sum64(s / sum * d) : 0.0;
      f = sum > 0.0 ? (d - m) / sum : 0.0;
    }
    v = id >= 0 ? f * s * sigmoid64(-mine) : 0.0;
  }
  if (nan) v = __builtin_nan("");
  double out[P];
#pragma unroll
  for (int i = 0; i < P; ++i) out[i] = whole ? -p[i] * m : 0.0;
  for (int j = 0; j < a.top; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const double x = readlane64(v, j);
    if (e >= 0 && (e & 63) == lane) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i == e >> 6) out[i] += x;
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    if (e < a.E) {
      if constexpr (BF16) static_cast<__bf16*>(dlogits)[t * a.E + e] = (__bf16)(float)out[i];
      else static_cast<float*>(dlogits)[t * a.E + e] = (float)out[i];
    }
  }
}

// f(integral_constant P) for the smallest P of 1, 2, 4, 8, 16 whose 64 P lanes' experts hold E
template <class F>
hipError_t with_experts(int E, F f) {
  if (E <= 64) return f(std::integral_constant<int, 1>{});
  if (E <= 128) return f(std::integral_constant<int, 2>{});
  if (E <= 256) return f(std::integral_constant<int, 4>{});
  if (E <= 512) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_moe_route(RouteArgs a, bool l_bf16, hipStream_t stream) {
  a.lanes = 1;
  while (2 * a.lanes * a.groups <= 64) a.lanes *= 2;
  // e / size for e <= 1023: the multiplier is off by less than size, e times that by less than 2^20
  const int size = a.E / a.groups;
  a.magic = ((1u << 20) + size - 1) / size;
  const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(64 * kTokens);
  const size_t lds = a.groups > 1 ? sizeof(double) * kTokens * a.E : 0;
  return with_experts(a.E, [&](auto p) {
    constexpr int P = decltype(p)::value;
    auto* kernel = l_bf16 ? a.bias ? route_kernel<P, true, true> : route_kernel<P, true, false>
                          : a.bias ? route_kernel<P, false, true> : route_kernel<P, false, false>;
    hipLaunchKernelGGL(kernel, grid, block, lds, stream, a);
    return hipGetLastError();
  });
}

hipError_t launch_moe_route_backward(const RouteArgs& a, bool l_bf16, const float* grad, void* dlogits, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(64 * kTokens);
  return with_experts(a.E, [&](auto p) {
    constexpr int P = decltype(p)::value;
    auto* kernel = l_bf16 ? route_backward_kernel<P, true> : route_backward_kernel<P, false>;
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, grad, dlogits);
    return hipGetLastError();
  });
}

}  // namespace aq
