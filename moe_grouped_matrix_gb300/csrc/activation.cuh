// The experts' gated activations in fp32: silu(g) = g / (1 + exp(-g)), and gelu in its
// tanh form, g / 2 (1 + tanh(i)) = g / (1 + exp(-2 i)) with i = sqrt(2 / pi) (g + 0.044715 g^3).
#pragma once

#include "../../include/libgmm_experts.h"

namespace gmmk {

constexpr float kGeluCube = 0.044715f;
constexpr float kGeluTwice = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// The argument x of act(g) = g / (1 + exp(-x)).
template <int kAct>
__device__ __forceinline__ float act_inner(float g) {
  return kAct == GMM_ACT_SILU ? g : kGeluTwice * (g + kGeluCube * g * g * g);
}

// kFast: for results in bf16, an exponential and a quotient of few instructions, off by 2 + |1.173 x| and 2
// units of their last place (CUDA's bounds): 2^-15 at exp(-90), for bf16's half step of 2^-9.
template <bool kFast>
__device__ __forceinline__ float act_exp(float x) {
  return kFast ? __expf(x) : expf(x);
}
template <bool kFast>
__device__ __forceinline__ float act_over(float a, float b) {
  return kFast ? __fdividef(a, b) : a / b;
}

// exp(-|x|) does not overflow, so what it scales keeps its precision down to fp32's least numbers.
template <int kAct, bool kFast>
__device__ __forceinline__ float act_value(float g) {
  const float x = act_inner<kAct>(g), e = act_exp<kFast>(-fabsf(x));
  return act_over<kFast>(x < 0.f ? g * e : g, 1.f + e);
}

// act(g) and its derivative s + g s (1 - s) x'(g), s = 1 / (1 + exp(-x)).  With e = exp(-|x|) both s and
// s (1 - s) = e / (1 + e)^2 keep their relative precision where s is next to 0 or 1.
template <int kAct, bool kFast>
__device__ __forceinline__ float act_value(float g, float& slope) {
  const float x = act_inner<kAct>(g), e = act_exp<kFast>(-fabsf(x)), inv = act_over<kFast>(1.f, 1.f + e);
  const float s = x < 0.f ? e * inv : inv, rest = e * inv * inv;
  const float dx = kAct == GMM_ACT_SILU ? 1.f : kGeluTwice * (1.f + 3.f * kGeluCube * g * g);
  slope = rest == 0.f ? s : s + g * rest * dx;  // far out gelu's x' may be infinite
  return g * s;
}

}  // namespace gmmk
