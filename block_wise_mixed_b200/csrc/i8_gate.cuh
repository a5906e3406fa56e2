// i8_gate.cuh -- the gate functions and their derivatives, in fp32.
//
// Both gates are a * sigmoid(t): silu with t = a, gelu_tanh with t = 2 u,
// u = sqrt(2 / pi) (a + 0.044715 a^3), since (1 + tanh u) / 2 = sigmoid(2u).
// sigmoid(t) and 1 - sigmoid(t) both come from e = exp(-|t|), so neither
// cancels and neither overflows.
#pragma once
#include "../../include/mpq.h"

namespace mpq {

struct Gate {
    float act, grad;   // act(a), act'(a)
};

template <int ACT>
__device__ __forceinline__ Gate gate_eval(float a) {
    float t = a, dt = 1.f;
    if (ACT == MPQ_ACT_GELU_TANH) {
        // |t| > 300 beyond |a| = 16: sigmoid is 0 or 1 there in fp32, and
        // the clamp keeps a^3 finite.  NaN goes on through act and grad.
        const float c = fminf(fmaxf(a, -16.f), 16.f), c2 = c * c;
        t = 1.5957691216057308f * c * fmaf(0.044715f, c2, 1.f);
        dt = 1.5957691216057308f * fmaf(0.134145f, c2, 1.f);
    }
    const float e = expf(-fabsf(t));
    const float r = __fdividef(1.f, 1.f + e), er = e * r;   // 1 + e in [1, 2]
    const float sig = t >= 0.f ? r : er, cosig = t >= 0.f ? er : r;
    Gate g;
    g.act = a * sig;
    g.grad = fmaf(g.act * cosig, dt, sig);
    return g;
}

}  // namespace mpq
