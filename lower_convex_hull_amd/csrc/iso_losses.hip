// Losses over tokens' log-probabilities, with their gradients: the paired
// preference loss and the clipped policy loss with a KL term (formulas in
// iso.h).  Both are sums over sequences of tokens followed by one value per
// token; every sum is f64, without atomics.
#include "../../include/iso.h"
#include "iso_losses.hpp"

namespace iso {
namespace {

constexpr int kLossNT = 256;       // threads of a workgroup over many tokens: four waves, a span each
constexpr int kSpan = 1024;        // tokens of a wave at a time: 16 a lane, in four groups of four
constexpr int kOneNT = 1024;       // the one workgroup of a small call
constexpr int64_t kOneMax = 16384;  // tokens (and sequences) up to which one workgroup takes the whole call

// A lane's 16 tokens of a span: group g holds tokens at(g) .. at(g)+3.
struct Place {
    int64_t p0, p1;  // the span's tokens
    int lane;
    __device__ __forceinline__ Place(int64_t span, int64_t tokens) {
        lane = threadIdx.x & 63;
        p0 = span * kSpan;
        p1 = min(p0 + kSpan, tokens);
    }
    __device__ __forceinline__ int64_t at(int g) const { return p0 + g * 256 + lane * 4; }
};

typedef float Float4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ void load16(const float* __restrict__ p, const Place& w, float (&v)[16]) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int64_t t = w.at(g);
        if (t + 4 <= w.p1) {
            const Float4 x = *reinterpret_cast<const Float4*>(p + t);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * g + i] = x[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * g + i] = t + i < w.p1 ? p[t + i] : 0.0f;
        }
    }
}

__device__ __forceinline__ void store16(float* __restrict__ p, const Place& w, const float (&v)[16]) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int64_t t = w.at(g);
        if (t + 4 <= w.p1) {
            Float4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = v[4 * g + i];
            *reinterpret_cast<Float4*>(p + t) = x;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t + i < w.p1) p[t + i] = v[4 * g + i];
        }
    }
}

// Which tokens take part: a mask, or rows' targets (negative: not), or all.
struct Live {
    const uint8_t* mask;
    const int32_t* target;
    __device__ __forceinline__ bool all() const { return !mask && !target; }
    // bit k: the lane's token k takes part
    __device__ __forceinline__ uint32_t bits(const Place& w) const {
        uint32_t b = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int64_t t = w.at(g);
            if (t + 4 <= w.p1) {
                if (mask) {
                    uint32_t x;
                    __builtin_memcpy(&x, mask + t, 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) b |= ((x >> (8 * i)) & 255u) ? 1u << (4 * g + i) : 0u;
                } else if (target) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) b |= target[t + i] >= 0 ? 1u << (4 * g + i) : 0u;
                } else {
                    b |= 15u << (4 * g);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t + i < w.p1 && (!mask || mask[t + i]) && (!target || target[t + i] >= 0))
                        b |= 1u << (4 * g + i);
            }
        }
        return b;
    }
};

// The bits of a lane's tokens in [a, b).
__device__ __forceinline__ uint32_t inside(const Place& w, int64_t a, int64_t b) {
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int lo = (int)max((int64_t)0, min((int64_t)4, a - w.at(g)));
        const int hi = (int)max((int64_t)0, min((int64_t)4, b - w.at(g)));
        m |= (((1u << hi) - 1u) & ~((1u << lo) - 1u)) << (4 * g);
    }
    return m;
}

// The sequence that holds token p: the last one that begins at or before it.
// All lanes of a wave together: 64 places are looked at in each round.
__device__ __forceinline__ int64_t find_seq(const Seqs& sq, int64_t p) {
    if (!sq.off) return p / sq.len;
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, hi = sq.n;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 63) / 64;
        const int64_t k = lo + (lane + 1) * step;
        const int c = __popcll(__ballot(k < hi && sq.begin(k) <= p));
        lo += c * step;
        hi = min(lo + step, hi);
    }
    return lo;
}

// f(q, a, b) for each piece [a, b) of a span that lies in one sequence q, in
// order.  Offsets that are not non-decreasing end a piece at the span's end.
template <typename F>
__device__ __forceinline__ void each_piece(const Seqs& sq, const Place& w, F f) {
    int64_t p = w.p0;
    int64_t q = p < w.p1 ? find_seq(sq, p) : 0;
    while (p < w.p1) {
        int64_t e = sq.end(q);
        if (e <= p || e > w.p1) e = w.p1;
        f(q, p, e);
        p = e;
        if (p < w.p1) {
            ++q;
            if (q >= sq.n || sq.begin(q) > p || sq.end(q) <= p) q = find_seq(sq, p);
        }
    }
}

// Sums by sequence of what spans hold.  A span's piece that holds its first
// token goes to head, one that holds its last token (and not the first) to
// tail, one between is a whole sequence's sum and goes to whole.
struct PartSums {
    double2 *head, *tail, *whole;
    __device__ __forceinline__ void put(const Place& w, int64_t span, int64_t q, int64_t a, int64_t b, double2 v) const {
        if (w.lane == 0) (a == w.p0 ? head[span] : b == w.p1 ? tail[span] : whole[q]) = v;
    }
    // The sum of sequence q; all lanes of a wave together.
    __device__ __forceinline__ double2 get(const Seqs& sq, int64_t q) const {
        const int64_t b = sq.begin(q), e = sq.end(q);
        double2 v = make_double2(0.0, 0.0);
        if (e <= b) return v;
        const int64_t s0 = b / kSpan, s1 = (e - 1) / kSpan;
        for (int64_t s = s0 + (threadIdx.x & 63); s <= s1; s += 64) {
            const double2 x = b <= s * kSpan                                   ? head[s]
                              : e >= min((s + 1) * (int64_t)kSpan, sq.tokens) ? tail[s]
                                                                               : whole[q];
            v.x += x.x;
            v.y += x.y;
        }
        return make_double2(wave_sum(v.x), wave_sum(v.y));
    }
};

int64_t spans_of(int64_t tokens) { return (tokens + kSpan - 1) / kSpan; }

// Workgroups for `waves` waves' work, at most 65536 (each then takes more).
dim3 wave_grid(int64_t waves) {
    const int64_t g = (waves + kLossNT / 64 - 1) / (kLossNT / 64);
    return dim3((unsigned)(g < 1 ? 1 : g > 65536 ? 65536 : g));
}

// A wave's number among all of a launch, and their number.
struct Wave {
    int64_t id, count;
    __device__ __forceinline__ Wave() {
        const int nw = blockDim.x >> 6;
        id = (int64_t)blockIdx.x * nw + (threadIdx.x >> 6);
        count = (int64_t)gridDim.x * nw;
    }
};

// ---- preference loss ----

struct Pref {
    const float* logp;
    const float* ref;  // or NULL
    Live live;
    Seqs sq;
    int64_t pairs;
    double beta, smooth;
    int mean, squared;
    double grad_scale;
    float *loss, *pair_loss, *reward, *grad;
    PartSums sums;   // (sum of ratios, tokens)
    double* each;    // pair losses
    float* coef;     // a sequence's gradient
};

// -log sigma(h), without overflow for either sign.
__device__ __forceinline__ double softplus_neg(double h) { return fmax(-h, 0.0) + log1p(exp(-fabs(h))); }

__device__ __forceinline__ void pref_sums(const Pref& p, int64_t span) {
    const Place w(span, p.sq.tokens);
    float x[16], y[16];
    load16(p.logp, w, x);
    if (p.ref) load16(p.ref, w, y);
    const uint32_t live = p.live.bits(w);
    each_piece(p.sq, w, [&](int64_t q, int64_t a, int64_t b) {
        const uint32_t m = live & inside(w, a, b);
        double v = 0.0;
#pragma unroll
        for (int k = 0; k < 16; ++k) v += (m >> k) & 1u ? (double)x[k] - (p.ref ? (double)y[k] : 0.0) : 0.0;
        p.sums.put(w, span, q, a, b, make_double2(wave_sum(v), wave_sum((double)__popc(m))));
    });
}

__device__ __forceinline__ void pref_pair(const Pref& p, int64_t i) {
    double2 c = p.sums.get(p.sq, 2 * i), r = p.sums.get(p.sq, 2 * i + 1);
    const double fc = p.mean ? 1.0 / fmax(c.y, 1.0) : 1.0, fr = p.mean ? 1.0 / fmax(r.y, 1.0) : 1.0;
    c.x *= fc;
    r.x *= fr;
    const double delta = c.x - r.x;
    double loss, slope;
    if (p.squared) {
        const double z = delta - 0.5 / p.beta;
        loss = z * z;
        slope = 2.0 * z;
    } else {
        const double h = p.beta * delta;
        loss = (1.0 - p.smooth) * softplus_neg(h) + (p.smooth > 0.0 ? p.smooth * softplus_neg(-h) : 0.0);
        slope = p.beta * (p.smooth / (1.0 + exp(-h)) - (1.0 - p.smooth) / (1.0 + exp(h)));
    }
    if ((threadIdx.x & 63) != 0) return;
    slope *= p.grad_scale / (double)p.pairs;
    p.each[i] = loss;
    p.coef[2 * i] = (float)(slope * fc);
    p.coef[2 * i + 1] = (float)(-slope * fr);
    p.pair_loss[i] = (float)loss;
    p.reward[2 * i] = (float)(p.beta * c.x);
    p.reward[2 * i + 1] = (float)(p.beta * r.x);
}

__device__ __forceinline__ void pref_grad(const Pref& p, int64_t span) {
    const Place w(span, p.sq.tokens);
    float g[16] = {};
    const uint32_t live = p.live.bits(w);
    each_piece(p.sq, w, [&](int64_t q, int64_t a, int64_t b) {
        const uint32_t m = live & inside(w, a, b);
        const float c = p.coef[q];
#pragma unroll
        for (int k = 0; k < 16; ++k) g[k] = (m >> k) & 1u ? c : g[k];
    });
    store16(p.grad, w, g);
}

template <int NT>
__device__ __forceinline__ void pref_mean(const Pref& p) {
    __shared__ double red[NT / 64];
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < p.pairs; i += NT) v += p.each[i];
    v = wg_sum<NT>(v, red);
    if (threadIdx.x == 0) *p.loss = p.pairs ? (float)(v / (double)p.pairs) : 0.0f;
}

__global__ __launch_bounds__(kLossNT) void k_pref_sums(Pref p, int64_t spans) {
    const Wave w;
    for (int64_t s = w.id; s < spans; s += w.count) pref_sums(p, s);
}
__global__ __launch_bounds__(kLossNT) void k_pref_pairs(Pref p) {
    const Wave w;
    for (int64_t i = w.id; i < p.pairs; i += w.count) pref_pair(p, i);
}
// The first workgroup takes the mean of the pair losses, the others the tokens.
__global__ __launch_bounds__(kLossNT) void k_pref_grad(Pref p, int64_t spans) {
    if (blockIdx.x == 0) {
        pref_mean<kLossNT>(p);
        return;
    }
    const Wave w;
    const int64_t first = kLossNT / 64;
    for (int64_t s = w.id - first; s < spans; s += w.count - first) pref_grad(p, s);
}
// A small call whole: the three steps by one workgroup.
__global__ __launch_bounds__(kOneNT) void k_pref_one(Pref p, int64_t spans) {
    const Wave w;
    for (int64_t s = w.id; s < spans; s += w.count) pref_sums(p, s);
    __syncthreads();
    for (int64_t i = w.id; i < p.pairs; i += w.count) pref_pair(p, i);
    __syncthreads();
    if (p.grad)
        for (int64_t s = w.id; s < spans; s += w.count) pref_grad(p, s);
    pref_mean<kOneNT>(p);
}

struct PrefPlan {
    size_t off_head, off_tail, off_whole, off_each, off_coef, bytes;
};
PrefPlan pref_plan(int64_t tokens, int64_t pairs) {
    PrefPlan p;
    size_t at = 0;
    auto take = [&](int64_t n, size_t size) {
        const size_t o = at;
        at += ((size_t)n * size + 255) / 256 * 256;
        return o;
    };
    p.off_head = take(spans_of(tokens), sizeof(double2));
    p.off_tail = take(spans_of(tokens), sizeof(double2));
    p.off_whole = take(2 * pairs, sizeof(double2));
    p.off_each = take(pairs, sizeof(double));
    p.off_coef = take(2 * pairs, sizeof(float));
    p.bytes = at;
    return p;
}

// ---- policy loss ----

template <typename LP>
struct PolicyCall {
    Policy p;
    const LP* logp;
    Live live;
    Seqs sq;
    float* loss;
    int32_t* counts;
    float* grad;      // or NULL
    PartSums sums;    // (tokens that take part, 0)
    double* weight;   // a sequence's w_t (ISO_POLICY_SEQ_MEAN)
    double* part;     // a wave's sums of w pg, w kl; tokens, clipped
    double2* total;   // tokens that take part in all, w_t
};

// Tokens that take part, by sequence.
template <typename LP>
__device__ __forceinline__ void policy_count(const PolicyCall<LP>& c, int64_t span) {
    const Place w(span, c.sq.tokens);
    const uint32_t live = c.live.bits(w);
    if (!c.p.seq_mean) {
        const double n = wave_sum((double)__popc(live));
        if (w.lane == 0) c.sums.head[span] = make_double2(n, 0.0);
        return;
    }
    each_piece(c.sq, w, [&](int64_t q, int64_t a, int64_t b) {
        c.sums.put(w, span, q, a, b, make_double2(wave_sum((double)__popc(live & inside(w, a, b))), 0.0));
    });
}

// A sequence's weight, from its count.
template <typename LP>
__device__ __forceinline__ void policy_weight(const PolicyCall<LP>& c, int64_t q) {
    const double n = c.sums.get(c.sq, q).x;
    if ((threadIdx.x & 63) == 0) c.weight[q] = 1.0 / ((c.p.norm > 0.0 ? c.p.norm : (double)c.sq.n) * fmax(n, 1.0));
}

// Every token's weight where they are alike, by one workgroup.
template <typename LP, int NT>
__device__ __forceinline__ void policy_total(const PolicyCall<LP>& c, int64_t spans) {
    __shared__ double red[NT / 64];
    double n = 0.0;
    for (int64_t s = threadIdx.x; s < spans; s += NT) n += c.sums.head[s].x;
    n = wg_sum<NT>(n, red);
    if (threadIdx.x == 0) *c.total = make_double2(n, 1.0 / (c.p.norm > 0.0 ? c.p.norm : fmax(n, 1.0)));
}

struct Four {
    double pg, kl, live, over;
};

// The terms of a span's tokens, summed into s by lane; their gradient is written.
template <typename LP>
__device__ __forceinline__ void policy_span(const PolicyCall<LP>& c, int64_t span, Four& s) {
    const Place w(span, c.sq.tokens);
    const Policy& p = c.p;
    float old[16], ref[16], adv[16], f[16];
    double lp[16];
    if constexpr (sizeof(LP) == 4) {
        load16(c.logp, w, f);
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int64_t t = w.at(k / 4) + k % 4;
            lp[k] = t < w.p1 ? c.logp[t] : 0.0;
        }
    }
    load16(p.old_logp, w, old);
    if (p.ref_logp) load16(p.ref_logp, w, ref);
    const uint32_t live = c.live.bits(w);
    double wt[16];
    if (p.token_adv) load16(p.adv, w, adv);
    if (!p.token_adv || p.seq_mean) {
#pragma unroll
        for (int k = 0; k < 16; ++k) wt[k] = 0.0;
        each_piece(c.sq, w, [&](int64_t q, int64_t a, int64_t b) {
            const uint32_t m = inside(w, a, b);
            const float av = p.token_adv ? 0.0f : p.adv[q];
            const double wq = p.seq_mean ? c.weight[q] : 0.0;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (!p.token_adv) adv[k] = (m >> k) & 1u ? av : adv[k];
                wt[k] = (m >> k) & 1u ? wq : wt[k];
            }
        });
    }
    const double all = p.seq_mean ? 0.0 : c.total->y;
    float g[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        g[k] = 0.0f;
        if ((live >> k) & 1u) {
            const double x = sizeof(LP) == 4 ? (double)f[k] : lp[k];
            const PolicyTerm o = policy_term(p, x, (double)old[k], p.ref_logp ? (double)ref[k] : 0.0, (double)adv[k]);
            const double wk = p.seq_mean ? wt[k] : all;
            s.pg += wk * o.pg;
            s.kl += wk * o.kl;
            s.over += o.over ? 1.0 : 0.0;
            s.live += 1.0;
            g[k] = (float)(o.slope * (wk * p.grad_scale));
        }
    }
    if (c.grad) store16(c.grad, w, g);
}

// A workgroup's sums into its part; or, from the parts, the outputs.
template <typename LP, int NT>
__device__ __forceinline__ void policy_part(const PolicyCall<LP>& c, const Four& s) {
    __shared__ double red[NT / 64];
    const double pg = wg_sum<NT>(s.pg, red), kl = wg_sum<NT>(s.kl, red);
    const double live = wg_sum<NT>(s.live, red), over = wg_sum<NT>(s.over, red);
    if (threadIdx.x == 0) {
        double* o = c.part + 4 * (int64_t)blockIdx.x;
        o[0] = pg;
        o[1] = kl;
        o[2] = live;
        o[3] = over;
    }
}
template <typename LP>
__device__ __forceinline__ void policy_out(const PolicyCall<LP>& c, const Four& s) {
    if (threadIdx.x != 0) return;
    c.loss[0] = (float)(c.p.kl_coef != 0.0 ? s.pg + c.p.kl_coef * s.kl : s.pg);
    c.loss[1] = (float)s.pg;
    c.loss[2] = (float)s.kl;
    c.counts[0] = (int32_t)s.live;
    c.counts[1] = (int32_t)s.over;
}

template <typename LP>
__global__ __launch_bounds__(kLossNT) void k_policy_count(PolicyCall<LP> c, int64_t spans) {
    const Wave w;
    for (int64_t s = w.id; s < spans; s += w.count) policy_count(c, s);
}
template <typename LP>
__global__ __launch_bounds__(kLossNT) void k_policy_weights(PolicyCall<LP> c, int64_t spans) {
    if (!c.p.seq_mean) {  // one workgroup
        policy_total<LP, kLossNT>(c, spans);
        return;
    }
    const Wave w;
    for (int64_t q = w.id; q < c.sq.n; q += w.count) policy_weight(c, q);
}
template <typename LP>
__global__ __launch_bounds__(kLossNT) void k_policy_tokens(PolicyCall<LP> c, int64_t spans) {
    const Wave w;
    Four s{};
    for (int64_t k = w.id; k < spans; k += w.count) policy_span(c, k, s);
    policy_part<LP, kLossNT>(c, s);
}
template <typename LP>
__global__ __launch_bounds__(kOneNT) void k_policy_sum(PolicyCall<LP> c, int64_t parts) {
    __shared__ double red[kOneNT / 64];
    Four s{};
    for (int64_t k = threadIdx.x; k < parts; k += kOneNT) {
        const double* o = c.part + 4 * k;
        s.pg += o[0];
        s.kl += o[1];
        s.live += o[2];
        s.over += o[3];
    }
    s.pg = wg_sum<kOneNT>(s.pg, red);
    s.kl = wg_sum<kOneNT>(s.kl, red);
    s.live = wg_sum<kOneNT>(s.live, red);
    s.over = wg_sum<kOneNT>(s.over, red);
    policy_out(c, s);
}
// A small call whole.
template <typename LP>
__global__ __launch_bounds__(kOneNT) void k_policy_one(PolicyCall<LP> c, int64_t spans) {
    __shared__ double red[kOneNT / 64];
    const Wave w;
    for (int64_t s = w.id; s < spans; s += w.count) policy_count(c, s);
    __syncthreads();
    if (c.p.seq_mean)
        for (int64_t q = w.id; q < c.sq.n; q += w.count) policy_weight(c, q);
    else
        policy_total<LP, kOneNT>(c, spans);
    __syncthreads();
    Four s{};
    for (int64_t k = w.id; k < spans; k += w.count) policy_span(c, k, s);
    s.pg = wg_sum<kOneNT>(s.pg, red);
    s.kl = wg_sum<kOneNT>(s.kl, red);
    s.live = wg_sum<kOneNT>(s.live, red);
    s.over = wg_sum<kOneNT>(s.over, red);
    policy_out(c, s);
}

struct PolicyPlan {
    size_t off_total, off_head, off_tail, off_whole, off_weight, off_part, bytes;
};
PolicyPlan policy_plan(int64_t tokens, int64_t seqs) {
    PolicyPlan p;
    size_t at = 0;
    auto take = [&](int64_t n, size_t size) {
        const size_t o = at;
        at += ((size_t)n * size + 255) / 256 * 256;
        return o;
    };
    p.off_total = take(1, sizeof(double2));
    p.off_head = take(spans_of(tokens), sizeof(double2));
    p.off_tail = take(spans_of(tokens), sizeof(double2));
    p.off_whole = take(seqs, sizeof(double2));
    p.off_weight = take(seqs, sizeof(double));
    p.off_part = take(4 * (int64_t)wave_grid(spans_of(tokens)).x, sizeof(double));
    p.bytes = at;
    return p;
}

bool seqs_ok(const int32_t* off, int64_t seqs, int64_t tokens) {
    if (seqs < 0 || tokens < 0 || tokens > 0x7fffffffLL || seqs > 0x7fffffffLL) return false;
    if (!aligned(off, 4)) return false;
    if (seqs == 0) return tokens == 0;  // tokens have to belong to a sequence
    return off || tokens % seqs == 0;
}

}  // namespace

bool policy_args_ok(const float* old_logp, const float* ref_logp, const float* adv, const int32_t* seq_off,
                    int64_t seqs, int64_t tokens, double clip_lo, double clip_hi, double kl_coef, double norm,
                    double grad_scale, uint32_t flags) {
    if (flags & ~(uint32_t)(ISO_POLICY_SEQ_MEAN | ISO_POLICY_ADV_TOKEN)) return false;
    if (!seqs_ok(seq_off, seqs, tokens)) return false;
    if (tokens && (!old_logp || !adv)) return false;
    if (!(clip_lo >= 0.0 && clip_lo <= 1.0) || !(clip_hi >= 0.0)) return false;
    if (!isfinite(kl_coef) || !isfinite(norm) || norm < 0.0 || !isfinite(grad_scale)) return false;
    if (kl_coef != 0.0 && !ref_logp && tokens) return false;
    return aligned(old_logp, 4) && aligned(ref_logp, 4) && aligned(adv, 4);
}

Policy make_policy(const float* old_logp, const float* ref_logp, const float* adv, double clip_lo,
                   double clip_hi, double kl_coef, double norm, double grad_scale, uint32_t flags) {
    Policy p;
    p.old_logp = old_logp;
    p.ref_logp = ref_logp;
    p.adv = adv;
    p.token_adv = (flags & ISO_POLICY_ADV_TOKEN) != 0;
    p.seq_mean = (flags & ISO_POLICY_SEQ_MEAN) != 0;
    p.up = log1p(clip_hi);
    p.low = log1p(-clip_lo);
    p.edge_hi = 1.0 + clip_hi;
    p.edge_lo = 1.0 - clip_lo;
    p.kl_coef = kl_coef;
    p.norm = norm;
    p.grad_scale = grad_scale;
    return p;
}

size_t policy_workspace(int64_t tokens, int64_t seqs) {
    if (tokens < 0 || seqs < 0 || tokens > 0x7fffffffLL || seqs > 0x7fffffffLL) return 0;
    return policy_plan(tokens, seqs).bytes;
}

template <typename LP>
hipError_t launch_policy(const Policy& p, const LP* logp, const uint8_t* mask, const int32_t* target,
                         const Seqs& sq, float* loss, int32_t* counts, float* grad, void* workspace,
                         hipStream_t st) {
    const PolicyPlan pl = policy_plan(sq.tokens, sq.n);
    char* ws = static_cast<char*>(workspace);
    PolicyCall<LP> c;
    c.p = p;
    c.logp = logp;
    c.live = Live{mask, target};
    c.sq = sq;
    c.loss = loss;
    c.counts = counts;
    c.grad = grad;
    c.total = reinterpret_cast<double2*>(ws + pl.off_total);
    c.sums = PartSums{reinterpret_cast<double2*>(ws + pl.off_head), reinterpret_cast<double2*>(ws + pl.off_tail),
                      reinterpret_cast<double2*>(ws + pl.off_whole)};
    c.weight = reinterpret_cast<double*>(ws + pl.off_weight);
    c.part = reinterpret_cast<double*>(ws + pl.off_part);
    const int64_t spans = spans_of(sq.tokens);
    if (sq.tokens <= kOneMax && sq.n <= kOneMax) {
        hipLaunchKernelGGL((k_policy_one<LP>), dim3(1), dim3(kOneNT), 0, st, c, spans);
        return hipGetLastError();
    }
    const dim3 grid = wave_grid(spans), nt(kLossNT);
    hipLaunchKernelGGL((k_policy_count<LP>), grid, nt, 0, st, c, spans);
    hipLaunchKernelGGL((k_policy_weights<LP>), p.seq_mean ? wave_grid(sq.n) : dim3(1), nt, 0, st, c, spans);
    hipLaunchKernelGGL((k_policy_tokens<LP>), grid, nt, 0, st, c, spans);
    hipLaunchKernelGGL((k_policy_sum<LP>), dim3(1), dim3(kOneNT), 0, st, c, (int64_t)grid.x);
    return hipGetLastError();
}
template hipError_t launch_policy<float>(const Policy&, const float*, const uint8_t*, const int32_t*, const Seqs&,
                                         float*, int32_t*, float*, void*, hipStream_t);
template hipError_t launch_policy<double>(const Policy&, const double*, const uint8_t*, const int32_t*, const Seqs&,
                                          float*, int32_t*, float*, void*, hipStream_t);

}  // namespace iso

extern "C" {

size_t iso_pref_loss_workspace_bytes(int64_t tokens, int64_t pairs) {
    if (tokens < 0 || pairs < 0 || tokens > 0x7fffffffLL || pairs > 0x3fffffffLL) return 0;
    return iso::pref_plan(tokens, pairs).bytes;
}

int iso_pref_loss(const float* logp, const float* ref_logp, const uint8_t* mask, const int32_t* seq_off,
                  int64_t pairs, int64_t tokens, double beta, double label_smoothing, float* loss,
                  float* pair_loss, float* reward, float* grad, double grad_scale, void* workspace,
                  size_t workspace_bytes, void* stream, uint32_t flags) {
    using namespace iso;
    if (flags & ~(uint32_t)(ISO_PREF_MEAN | ISO_PREF_SQUARED)) return ISO_ERR_ARG;
    if (pairs < 0 || pairs > 0x3fffffffLL || !seqs_ok(seq_off, 2 * pairs, tokens)) return ISO_ERR_ARG;
    if (!loss || (pairs && (!pair_loss || !reward)) || (tokens && !logp)) return ISO_ERR_ARG;
    if (!(beta > 0.0) || !isfinite(beta) || !isfinite(grad_scale)) return ISO_ERR_ARG;
    if (!(label_smoothing >= 0.0 && label_smoothing <= 0.5)) return ISO_ERR_ARG;
    if ((flags & ISO_PREF_SQUARED) && label_smoothing != 0.0) return ISO_ERR_ARG;
    const size_t tb = (size_t)tokens * 4;
    const Span out[] = {{loss, 4}, {pair_loss, (size_t)pairs * 4}, {reward, (size_t)pairs * 8}, {grad, tb}};
    const Span in[] = {{logp, tb}, {ref_logp, tb}, {mask, (size_t)tokens}, {seq_off, (size_t)(2 * pairs + 1) * 4}};
    if (!disjoint(out, in)) return ISO_ERR_ARG;
    if (!aligned(logp, 4) || !aligned(ref_logp, 4) || !aligned(loss, 4) || !aligned(pair_loss, 4) ||
        !aligned(reward, 4) || !aligned(grad, 4))
        return ISO_ERR_ARG;
    const size_t need = iso_pref_loss_workspace_bytes(tokens, pairs);
    if (need && (!workspace || workspace_bytes < need)) return ISO_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return ISO_ERR_ARG;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const PrefPlan pl = pref_plan(tokens, pairs);
    char* ws = static_cast<char*>(workspace);
    Pref p;
    p.logp = logp;
    p.ref = ref_logp;
    p.live = Live{mask, nullptr};
    p.sq = Seqs{seq_off, 2 * pairs, tokens, pairs ? tokens / (2 * pairs) : 0};
    p.pairs = pairs;
    p.beta = beta;
    p.smooth = label_smoothing;
    p.mean = (flags & ISO_PREF_MEAN) != 0;
    p.squared = (flags & ISO_PREF_SQUARED) != 0;
    p.grad_scale = grad_scale;
    p.loss = loss;
    p.pair_loss = pair_loss;
    p.reward = reward;
    p.grad = grad;
    p.sums = PartSums{reinterpret_cast<double2*>(ws + pl.off_head), reinterpret_cast<double2*>(ws + pl.off_tail),
                      reinterpret_cast<double2*>(ws + pl.off_whole)};
    p.each = reinterpret_cast<double*>(ws + pl.off_each);
    p.coef = reinterpret_cast<float*>(ws + pl.off_coef);
    const int64_t spans = pairs ? spans_of(tokens) : 0;
    if (tokens <= kOneMax && pairs <= kOneMax) {
        hipLaunchKernelGGL(k_pref_one, dim3(1), dim3(kOneNT), 0, st, p, spans);
        return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
    }
    const dim3 nt(kLossNT);
    hipLaunchKernelGGL(k_pref_sums, wave_grid(spans), nt, 0, st, p, spans);
    hipLaunchKernelGGL(k_pref_pairs, wave_grid(pairs), nt, 0, st, p);
    hipLaunchKernelGGL(k_pref_grad, dim3(grad ? wave_grid(spans).x + 1 : 1), nt, 0, st, p, spans);
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

size_t iso_policy_loss_workspace_bytes(int64_t tokens, int64_t seqs) { return iso::policy_workspace(tokens, seqs); }

int iso_policy_loss(const float* logp, const float* old_logp, const float* ref_logp, const float* adv,
                    const uint8_t* mask, const int32_t* seq_off, int64_t seqs, int64_t tokens, double clip_lo,
                    double clip_hi, double kl_coef, double norm, float* loss, int32_t* counts, float* grad,
                    double grad_scale, void* workspace, size_t workspace_bytes, void* stream, uint32_t flags) {
    using namespace iso;
    if (!policy_args_ok(old_logp, ref_logp, adv, seq_off, seqs, tokens, clip_lo, clip_hi, kl_coef, norm,
                        grad_scale, flags))
        return ISO_ERR_ARG;
    if (!loss || !counts || (tokens && !logp)) return ISO_ERR_ARG;
    const size_t tb = (size_t)tokens * 4;
    const size_t ab = (flags & ISO_POLICY_ADV_TOKEN) ? tb : (size_t)seqs * 4;
    const Span out[] = {{loss, 12}, {counts, 8}, {grad, tb}};
    const Span in[] = {{logp, tb}, {old_logp, tb}, {ref_logp, tb}, {adv, ab}, {mask, (size_t)tokens},
                       {seq_off, (size_t)(seqs + 1) * 4}};
    if (!disjoint(out, in)) return ISO_ERR_ARG;
    if (!aligned(logp, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(grad, 4)) return ISO_ERR_ARG;
    const size_t need = iso_policy_loss_workspace_bytes(tokens, seqs);
    if (!workspace || workspace_bytes < need) return ISO_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return ISO_ERR_ARG;
    const Policy p = make_policy(old_logp, ref_logp, adv, clip_lo, clip_hi, kl_coef, norm, grad_scale, flags);
    const Seqs sq{seq_off, seqs, tokens, seqs ? tokens / seqs : 0};
    const hipError_t e = launch_policy<float>(p, logp, mask, nullptr, sq, loss, counts, grad, workspace,
                                              static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

}  // extern "C"
