// What the post-training loss kernels (iso_logp.hip, iso_losses.hip) share:
// workgroup sums, sequences of tokens, and the clipped policy loss's terms.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

namespace iso {

// A value of another lane by data-parallel primitive (row_shr and the row
// broadcasts of a wave scan, shifts by one lane); lanes without a source keep `old`.
template <int CTRL, int RM>
__device__ __forceinline__ int dpp(int old, int v) {
    return __builtin_amdgcn_update_dpp(old, v, CTRL, RM, 0xf, false);
}
template <int CTRL, int RM>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)dpp<CTRL, RM>(0, (int)(uint32_t)u);
    const uint32_t hi = (uint32_t)dpp<CTRL, RM>(0, (int)(uint32_t)(u >> 32));
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
constexpr int kShl1 = 0x130, kShr1 = 0x138;  // by one lane, over the whole wave

// f.template step<CTRL, ROW_MASK>() for each step of an inclusive scan over a wave.
template <typename F>
__device__ __forceinline__ void wave_scan(F& f) {
    f.template step<0x111, 0xf>();  // row_shr 1, 2, 4, 8 within rows of 16 lanes
    f.template step<0x112, 0xf>();
    f.template step<0x114, 0xf>();
    f.template step<0x118, 0xf>();
    f.template step<0x142, 0xa>();  // lane 15 of rows 0, 2 to rows 1, 3
    f.template step<0x143, 0xc>();  // lane 31 to rows 2, 3
}

__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)lane_value((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)lane_value((int)(uint32_t)(u >> 32), lane);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// Sums over the wave, the same value in every lane (all lanes active).
struct SumStep {
    double v;
    template <int CTRL, int RM>
    __device__ __forceinline__ void step() { v += dpp<CTRL, RM>(v); }
};
__device__ __forceinline__ double wave_sum(double v) {
    SumStep s{v};
    wave_scan(s);
    return lane_value(s.v, 63);
}
struct IntSumStep {
    int v;
    template <int CTRL, int RM>
    __device__ __forceinline__ void step() { v += dpp<CTRL, RM>(0, v); }
};
__device__ __forceinline__ int wave_sum(int v) {
    IntSumStep s{v};
    wave_scan(s);
    return lane_value(s.v, 63);
}

// Sum over the workgroup (NT threads), the same value in every thread.
template <int NT, typename T>
__device__ __forceinline__ T wg_sum(T v, T* red) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    T s = 0;
#pragma unroll
    for (int k = 0; k < NT / 64; ++k) s += red[k];
    __syncthreads();
    return s;
}

// Sequences of tokens: packed by offsets (held inside [0, tokens]), or all of
// one length.  Tokens and sequences are below 2^31.
struct Seqs {
    const int32_t* off;
    uint32_t n;  // sequences
    uint32_t tokens;
    uint32_t len;  // common length (off == NULL)
    __device__ __forceinline__ uint32_t begin(uint32_t q) const {
        if (!off) return q * len;
        const int32_t b = off[q];
        return b < 0 ? 0u : min((uint32_t)b, tokens);
    }
    __device__ __forceinline__ uint32_t end(uint32_t q) const { return max(begin(q), begin(q + 1)); }
};
inline Seqs make_seqs(const int32_t* off, int64_t seqs, int64_t tokens) {
    return Seqs{off, (uint32_t)seqs, (uint32_t)tokens, seqs ? (uint32_t)(tokens / seqs) : 0u};
}

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
    // w_t of a sequence's tokens (ISO_POLICY_SEQ_MEAN), from those that take part in it
    __device__ __forceinline__ double seq_weight(uint32_t seqs, double count) const {
        return 1.0 / ((norm > 0.0 ? norm : (double)seqs) * fmax(count, 1.0));
    }
    // every token's w_t where they are alike
    __device__ __forceinline__ double token_weight(int count) const {
        return 1.0 / (norm > 0.0 ? norm : fmax((double)count, 1.0));
    }
};
// exp(x), exp(x) - 1 and exp(x) - 1 - x in f64.  Cody and Waite's reduction
// x = k ln 2 + r with |r| <= ln(2)/2, then Taylor's series q of exp(r) - 1 - r
// to r^11 (the rest is below 7e-15 of 1).  With s = 2^k the small differences
// are s q + (s r + (s - 1) - x): for k = 0 that is q, with its relative
// accuracy.  A third of the instructions of the library's exp and expm1, whose
// last bits an f32 output does not show.  The coefficients are held in scalar
// registers: as literals each would be copied to a vector register before its
// multiply-add, twice the instructions.
struct ExpTerms {
    double e, m1, m2;  // exp(x), exp(x) - 1, exp(x) - 1 - x
};
struct ExpSeries {
    double c[9], log2e, ln2, ln2_rest;
    static constexpr double kFar = 700.0;  // s is a normal number up to here
    __device__ __forceinline__ ExpSeries() {
        double f = 6.0;
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            c[i] = 1.0 / f;  // 1/3!, ..., 1/11!
            f *= i + 4.0;
            asm("" : "+s"(c[i]));
        }
        log2e = 1.4426950408889634;
        ln2 = -0x1.62e42fefa39efp-1;  // ln 2 in f64, and the rest of it
        ln2_rest = -0x1.abc9e3b39803fp-56;
        asm("" : "+s"(log2e), "+s"(ln2), "+s"(ln2_rest));
    }
    // for |x| <= kFar (NaN stays NaN); else far() makes it right
    __device__ __forceinline__ ExpTerms operator()(double x) const {
        constexpr double kRound = 0x1.8p52;  // adding it rounds to a whole number, held in the low bits
        const double t = fma(x, log2e, kRound);
        const double kd = t - kRound;
        const uint32_t k = (uint32_t)__double_as_longlong(t);
        double r = fma(kd, ln2, x);
        r = fma(kd, ln2_rest, r);
        double q = fma(c[8], r, c[7]);
#pragma unroll
        for (int i = 6; i >= 0; --i) q = fma(q, r, c[i]);
        q = fma(q, r, 0.5) * (r * r);
        const double s = __hiloint2double((int)((k + 1023u) << 20), 0);
        ExpTerms o;
        o.e = fma(s, r + q, s);
        o.m2 = fma(s, q, fma(s, r, s - 1.0) - x);
        o.m1 = o.m2 + x;
        return o;
    }
    // for any x
    __device__ __forceinline__ ExpTerms any(double x) const {
        ExpTerms o = (*this)(x);
        far(x, o);
        return o;
    }
    // Beyond kFar: infinity or 0, which is what f32 outputs make of it.
    __device__ __forceinline__ static void far(double x, ExpTerms& o) {
        if (fabs(x) > kFar) {
            o.e = x > 0.0 ? INFINITY : 0.0;
            o.m1 = o.e - 1.0;
            o.m2 = x > 0.0 ? INFINITY : o.m1 - x;  // also at x = infinity
        }
    }
};

struct PolicyTerm {
    double pg, kl, slope;  // slope: derivative of pg + kl_coef kl in logp
    bool over;             // held by the clip
};
// The terms of N tokens, d = logp - old, u = ref_logp - logp (0 without a
// reference), a the advantage; no branches but for what is far off, so that the
// tokens' chains overlap.
template <bool REF, int N>
__device__ __forceinline__ void policy_terms(const Policy& p, const ExpSeries& ex, const double (&d)[N],
                                             const double (&u)[N], const float (&a)[N], PolicyTerm (&o)[N]) {
    ExpTerms r[N], k[N];
    bool far = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        r[i] = ex(d[i]);
        k[i] = REF ? ex(u[i]) : ExpTerms{1.0, 0.0, 0.0};
        far |= !((REF ? fabs(d[i]) + fabs(u[i]) : fabs(d[i])) <= ExpSeries::kFar);  // NaN too
    }
    if (far) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            ExpSeries::far(d[i], r[i]);
            if (a[i] == 0.0f && fabs(d[i]) < INFINITY) r[i].e = 1.0;  // r A is 0, also where r is beyond f64
            if (REF) {
                ExpSeries::far(u[i], k[i]);
                // a reference that is only watched: no infinity or NaN times 0 into the slope
                if (p.kl_coef == 0.0) k[i].m1 = 0.0;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        o[i].over = (a[i] > 0.0f && d[i] > p.up) || (a[i] < 0.0f && d[i] < p.low);
        const double f = o[i].over ? (a[i] > 0.0f ? p.edge_hi : p.edge_lo) : r[i].e;
        o[i].pg = -f * (double)a[i];
        o[i].slope = o[i].over ? 0.0 : o[i].pg;
        if (REF) o[i].slope = fma(-p.kl_coef, k[i].m1, o[i].slope);
        o[i].kl = k[i].m2;
    }
}

// Sums over tokens: w pg, w kl; tokens that take part, tokens held by the clip.
struct PolicySums {
    double pg, kl;
    int live, over;
};

// A row's part in the policy loss from logits: its weight w_t (0: it takes no
// part) and its advantage.
struct RowTerm {
    double w;
    float adv, pad;
};
// Row r's, by a workgroup of NT threads that each look at some sequences and
// targets.
template <int NT>
__device__ __forceinline__ RowTerm own_row_term(const Policy& p, const int32_t* __restrict__ target, const Seqs& sq,
                                                uint32_t r) {
    uint32_t q = 0;
    if (sq.off) {
        for (uint32_t k = 1; k < sq.n; k += NT)
            q += (uint32_t)__syncthreads_count(k + threadIdx.x < sq.n && sq.begin(k + threadIdx.x) <= r);
    } else {
        q = r / sq.len;
    }
    const uint32_t b = p.seq_mean ? sq.begin(q) : 0u, e = p.seq_mean ? sq.end(q) : sq.tokens;
    int count = 0;
    for (uint32_t t = b; t < e; t += NT) count += __syncthreads_count(t + threadIdx.x < e && target[t + threadIdx.x] >= 0);
    return RowTerm{p.seq_mean ? p.seq_weight(sq.n, (double)count) : p.token_weight(count), p.adv[p.token_adv ? r : q], 0.0f};
}
// Every row's, from the rows' targets (negative: no part) and the sequences.
size_t row_terms_workspace(int64_t rows, int64_t seqs);
hipError_t launch_row_terms(const Policy& p, const int32_t* target, const Seqs& sq, RowTerm* terms, void* workspace,
                            hipStream_t st);
// The loss and the counts from `parts` sums.
hipError_t launch_policy_out(const Policy& p, const PolicySums* part, int parts, float* loss, int32_t* counts,
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
