// Device helpers shared by the state-space mixer's kernels (ssm*.cu).
#pragma once

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace ssm {

// Tokens [begin, end) of sequence n: from cu_seqlens, clamped to [0, n_tok] and to
// begin <= end so that a bad offset reads and writes nothing out of range, or
// equal lengths.
__device__ __forceinline__ void seq_range(const int32_t *__restrict__ cu, int n_seq, int n_tok, int n, int &begin,
                                          int &end) {
    if (cu) {
        begin = min(max(__ldg(cu + n), 0), n_tok);
        end = min(max(__ldg(cu + n + 1), begin), n_tok);
    } else {
        const int L = n_tok / n_seq;
        begin = n * L;
        end = begin + L;
    }
}

// 4 consecutive elements as floats (8 bytes of bf16 or 16 bytes of fp32).
__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ float4 load4(const bf16 *p) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
    return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}

// SiLU with the full-precision exponential: the state takes its inputs from here
// and is held to fp32 accuracy.  x = -inf gives 0 * inf = NaN as in the formula.
__device__ __forceinline__ float silu(float x) { return x / (1.0f + expf(-x)); }

// e^{-t} as hi + lo.  Near 1, where a state remembers thousands of tokens, the rounding of
// one fp32 decay is the same at every like step and adds up (738 tokens: 6.6e-6 of the
// state), so its remainder, from e^{-t} - 1, is not dropped.  Below 1/2 the memory is short.
__device__ __forceinline__ float2 decay_pair(float t) {
    if (t < 0.69f) {
        const float e = expm1f(-t), hi = 1.f + e;
        return make_float2(hi, e - (hi - 1.f));
    }
    return make_float2(expf(-t), 0.f);
}
__device__ __forceinline__ float relative_rest(float2 a) { return a.y == 0.f ? 0.f : a.y / a.x; }

// a (1 + carry) as one fp32 factor d; carry becomes what that rounding leaves, for the next
// factor.  So a product of decays stays within a rounding or two of the true one however
// long it is.  (What is left of a (1 + carry) is a (1 + carry) - d, and relative to d that
// over a: the division is left out, for it changes carry by 1 - a of itself, and a state
// remembers 1 / (1 - a) decays.)  A remainder added to the state instead, S + rest S, is
// rounded in its turn, and where rest S is a few units of S the same way thousands of times
// (1e-4 of a state after 32768 tokens); it would also make NaN of an infinite state.
__device__ __forceinline__ float next_decay(float a, float &carry) {
    const float d = fmaf(carry, a, a);
    carry = fmaf(carry, a, a - d);
    return d;
}

// The mixer's channels [x (H P) | B (G N) | C (G N)] and their three raw sources.
template <typename T> struct Raw {
    const T *x, *B, *C;
    long long ld_x, ld_B, ld_C;
    int hp, gn;
    // the raw row element of channel c of token t; vector loads of channels stay
    // inside one source because hp and gn are multiples of 64
    __device__ __forceinline__ const T *at(long long t, int c) const {
        if (c < hp) return x + t * ld_x + c;
        if (c < hp + gn) return B + t * ld_B + (c - hp);
        return C + t * ld_C + (c - hp - gn);
    }
};

}  // namespace ssm
}  // namespace gdn
