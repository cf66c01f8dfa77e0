// act.h — the gated feed-forward's activations, included inside an anonymous
// namespace of a kernel file.

// The gate's activation and its derivative at g. FAST (bf16 results, half a
// step 2^-8 of the value): the hardware exponential and reciprocal, each
// within a few 2^-23 of exact, and a fitted erfc; otherwise the library
// functions.
template <bool FAST>
__device__ __forceinline__ float sigmoid_of(float g) {
  if (FAST) return __builtin_amdgcn_rcpf(1.f + __expf(-g));
  return 1.f / (1.f + expf(-g));
}

constexpr float kInvSqrt2 = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// The normal distribution function. Through erfc, which keeps the relative
// precision of the lower tail. FAST: erfc(z) = t exp(-z^2 + P(t)), t = 1 / (1 + z/2),
// z >= 0, the Chebyshev fit of Numerical Recipes in C, section 6.2 (relative
// error 1.2e-7), a few instructions where the library's erfc is a long
// branching function that made the epilogues spill.
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float g) {
  if (!FAST) return 0.5f * erfcf(-g * kInvSqrt2);
  const float z = fabsf(g) * kInvSqrt2;
  const float t = __builtin_amdgcn_rcpf(1.f + 0.5f * z);
  float p = 0.17087277f;
  p = fmaf(p, t, -0.82215223f);
  p = fmaf(p, t, 1.48851587f);
  p = fmaf(p, t, -1.13520398f);
  p = fmaf(p, t, 0.27886807f);
  p = fmaf(p, t, -0.18628806f);
  p = fmaf(p, t, 0.09678418f);
  p = fmaf(p, t, 0.37409196f);
  p = fmaf(p, t, 1.00002368f);
  p = fmaf(p, t, -1.26551223f);
  const float h = 0.5f * t * __expf(fmaf(-z, z, p));
  return g < 0.f ? h : 1.f - h;
}

template <bool FAST>
__device__ __forceinline__ float act_of(float g, int act) {
  switch (act) {
    case MOE_ACT_SILU: return g * sigmoid_of<FAST>(g);
    case MOE_ACT_GELU: return g * normal_cdf<FAST>(g);
    case MOE_ACT_RELU: return g > 0.f ? g : g == g ? 0.f : g;
    default: return g;
  }
}

// act(g) in a, act'(g) in d.
template <bool FAST>
__device__ __forceinline__ void act_grad_of(float g, int act, float& a, float& d) {
  switch (act) {
    case MOE_ACT_SILU: {
      const float s = sigmoid_of<FAST>(g);
      a = g * s;
      d = s * (1.f + g * sigmoid_of<FAST>(-g));
      return;
    }
    case MOE_ACT_GELU: {
      const float c = normal_cdf<FAST>(g);
      a = g * c;
      d = c + g * kInvSqrt2Pi * (FAST ? __expf(-0.5f * g * g) : expf(-0.5f * g * g));
      return;
    }
    case MOE_ACT_RELU:
      a = g > 0.f ? g : g == g ? 0.f : g;
      d = g > 0.f ? 1.f : 0.f;
      return;
    default:
      a = g;
      d = 1.f;
  }
}
