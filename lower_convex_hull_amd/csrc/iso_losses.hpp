// What the post-training loss kernels (iso_logp.hip, iso_losses.hip) share:
// workgroup sums, sequences of tokens, and the clipped policy loss's terms.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

namespace iso {

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Sum over the workgroup (NT threads), the same value in every thread.
template <int NT>
__device__ __forceinline__ double wg_sum(double v, double* red) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < NT / 64; ++k) s += red[k];
    __syncthreads();
    return s;
}

// Sequences of tokens: packed by offsets (held inside [0, tokens]), or all of
// one length.
struct Seqs {
    const int32_t* off;
    int64_t n;       // sequences
    int64_t tokens;
    int64_t len;     // common length (off == NULL)
    __device__ __forceinline__ int64_t begin(int64_t q) const {
        if (!off) return q * len;
        const int64_t b = off[q];
        return b < 0 ? 0 : b > tokens ? tokens : b;
    }
    __device__ __forceinline__ int64_t end(int64_t q) const {
        const int64_t b = begin(q), e = begin(q + 1);
        return e < b ? b : e;
    }
};

// The clipped policy loss of one token.  With d = logp - old (exact in f64 for
// f32 inputs), the clip is decided on d against the logarithms of the bounds:
// no rounding of exp(d) can put a token on the other side.
struct Policy {
    const float* old_logp;
    const float* ref_logp;  // or NULL
    const float* adv;       // per sequence, or per token
    int token_adv;
    int seq_mean;
    double up, low;            // log(1 + clip_hi), log(1 - clip_lo)
    double edge_hi, edge_lo;   // 1 + clip_hi, 1 - clip_lo
    double kl_coef;
    double norm;               // > 0: in place of the count of tokens or sequences
    double grad_scale;
};
struct PolicyTerm {
    double pg, kl, slope;  // slope: derivative of pg + kl_coef kl in logp
    bool over;             // held by the clip
};
__device__ __forceinline__ PolicyTerm policy_term(const Policy& p, double lp, double old, double ref, double a) {
    const double d = lp - old;
    PolicyTerm o;
    o.over = a > 0.0 ? d > p.up : a < 0.0 ? d < p.low : false;
    const double ra = exp(d) * a;
    o.pg = o.over ? -(a > 0.0 ? p.edge_hi : p.edge_lo) * a : -ra;
    o.slope = o.over ? 0.0 : -ra;
    o.kl = 0.0;
    if (p.ref_logp) {
        const double u = ref - lp;
        const double em = expm1(u);
        o.kl = em - u;
        o.slope -= p.kl_coef * em;
    }
    return o;
}

// The policy loss over tokens' log-probabilities (LP: f32, or f64 from the
// logits), live where mask is NULL or non-zero and target is NULL or >= 0.
size_t policy_workspace(int64_t tokens, int64_t seqs);
template <typename LP>
hipError_t launch_policy(const Policy& p, const LP* logp, const uint8_t* mask, const int32_t* target,
                         const Seqs& sq, float* loss, int32_t* counts, float* grad, void* workspace,
                         hipStream_t st);

// Argument checks of the policy loss that do not depend on where logp comes from.
bool policy_args_ok(const float* old_logp, const float* ref_logp, const float* adv, const int32_t* seq_off,
                    int64_t seqs, int64_t tokens, double clip_lo, double clip_hi, double kl_coef, double norm,
                    double grad_scale, uint32_t flags);
Policy make_policy(const float* old_logp, const float* ref_logp, const float* adv, double clip_lo,
                   double clip_hi, double kl_coef, double norm, double grad_scale, uint32_t flags);

// A byte range of an argument, for the overlap checks.
struct Span {
    const void* p;
    size_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}
// No output overlaps an input or another output.
template <int NO, int NI>
bool disjoint(const Span (&out)[NO], const Span (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int k = 0; k < NI; ++k)
            if (overlap(out[i], in[k])) return false;
        for (int k = 0; k < i; ++k)
            if (overlap(out[i], out[k])) return false;
    }
    return true;
}
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace iso
