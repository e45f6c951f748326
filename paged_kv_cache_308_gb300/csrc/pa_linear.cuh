// The decay of linear attention's states, shared by the kernels that go token by
// token (pa_linear.cu) and by blocks of tokens (pa_linear_prefix.cu).
#pragma once

namespace pa {
namespace {

// What a state is multiplied by: S -> exp(y) S = S * whole + S * rest, the sum
// rounded once (a fused sum over the product with rest).  Next to 1 the two hold
// what exp(y) alone loses there: rest is what 1 + expm1(y) has below whole's last
// place.  Both are positive unless exp(y) is 0 or the smallest number in 32 bits, so
// that an infinite entry stays one instead of meeting itself with the other sign, or a 0.
struct Decay {
    float whole, rest;
};
__device__ __forceinline__ Decay decay_of(float y) {
    if (y > -0.5f) {
        const float less = expm1f(y);  // > -0.4
        Decay d;
        d.whole = __fadd_rd(1.f, less);
        d.rest = (1.f - d.whole) + less;  // exact but for less above -2^-24
        if (!(d.rest > 0.f)) {  // (0.5 to 1: the next number down is 2^-24 away)
            d.whole -= 0x1p-24f;
            d.rest += 0x1p-24f;
        }
        return d;
    }
    // So little that next to no rounding sees it, down to the smallest number: that is no more than 2^-24 of exp(y)
    // from 2^-125 on, and below whole is a multiple of it.
    const float whole = expf(y), rest = whole > 0.f ? fmaxf(whole * 0x1p-64f, 0x1p-149f) : 0.f;
    return {whole < 0x1p-125f ? whole - rest : whole, rest};
}

}  // namespace
}  // namespace pa
