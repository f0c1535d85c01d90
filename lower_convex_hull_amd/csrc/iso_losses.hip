// Losses over tokens' log-probabilities, with their gradients: the paired
// preference loss and the clipped policy loss with a KL term (formulas in
// iso.h).  Both are sums over sequences of tokens followed by one value per
// token; every sum of values is f64, in a fixed order, without atomics (the one
// atomic is a maximum of whole numbers in LDS, whose order does not matter).
#include "../../include/iso.h"
#include "iso_losses.hpp"

#include <type_traits>

namespace iso {
namespace {

constexpr int kLossNT = 256;  // threads of a workgroup over many tokens: four waves
// A wave's span, in groups of 256 tokens (4 a lane in each): 1 for the sums and
// the preference gradient (64 pairs of 20000 tokens: 12.0 us, 13.1 with 2), 2 for the
// policy's terms, whose registers leave no room for more.
constexpr int kSpanG = 1, kTermG = 2;
// Workgroups over spans, eight a CU, four where they take more registers
// (policy loss of 8e6 tokens: 58 us, 60 with four throughout, 66 with one span a wave).
constexpr int64_t kGrid = 2048, kTermGrid = 1024;
constexpr int kTermWaves = 4;  // waves a SIMD holds of them
// Pairs or sequences up to which each has a workgroup for its spans, else a wave:
// few can be long (2 pairs of 2e6 tokens: 17 us, 22 with waves).
constexpr int64_t kWideSeqs = 256;
// Up to this many tokens and sequences one workgroup takes the whole call, in
// spans of one group (6000 tokens in 16 pairs: 10.1 us, 12.1 in three launches; at
// 12000 13.1 and 12.3).
constexpr int kOneNT = 1024;
constexpr int64_t kOneMax = 8192;

// A span of G groups and a lane's tokens of it: group g holds tokens at(g) .. at(g)+3.
template <int G>
struct Place {
    uint32_t p0, p1;  // the span's tokens
    int lane;
    __device__ __forceinline__ Place(uint32_t span, uint32_t tokens) {
        lane = threadIdx.x & 63;
        p0 = span * (256u * G);
        p1 = min(p0 + 256u * G, tokens);
    }
    __device__ __forceinline__ uint32_t at(int g) const { return p0 + g * 256u + lane * 4u; }
};

typedef float Float4 __attribute__((ext_vector_type(4), aligned(4)));

// A lane's four values of each group, those at or past the span's end 0.
// Whole spans (all but a call's last) take one wide load a group.
template <int G>
__device__ __forceinline__ void load_span(const float* __restrict__ p, const Place<G>& w, float* v) {
    if (w.p1 - w.p0 == 256u * G) {
        const float* b = p + w.p0;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const Float4 x = *reinterpret_cast<const Float4*>(b + (g * 256u + w.lane * 4u));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * g + i] = x[i];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4 * G; ++k) {
            const uint32_t t = w.at(k / 4) + k % 4;
            v[k] = t < w.p1 ? p[t] : 0.0f;
        }
    }
}
__device__ __forceinline__ void load4(const float* __restrict__ p, uint32_t t, uint32_t end, float* v) {
    if (t + 4 <= end) {
        const Float4 x = *reinterpret_cast<const Float4*>(p + t);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = x[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = t + i < end ? p[t + i] : 0.0f;
    }
}
__device__ __forceinline__ void store4(float* __restrict__ p, uint32_t t, uint32_t end, const float* v) {
    if (t + 4 <= end) {
        Float4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = v[i];
        __builtin_nontemporal_store(x, reinterpret_cast<Float4*>(p + t));  // not left to the kernel end to write back
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t + i < end) p[t + i] = v[i];
    }
}

// Which tokens take part: a mask, or rows' targets (negative: not), or all.
struct Live {
    const uint8_t* mask;
    const int32_t* target;
    __host__ __device__ __forceinline__ bool all() const { return !mask && !target; }
    // bit i: token t + i takes part
    __device__ __forceinline__ uint32_t bits4(uint32_t t, uint32_t end) const {
        uint32_t b = 0;
        if (t + 4 <= end) {
            if (all()) return 15u;
            if (mask) {
                uint32_t x;
                __builtin_memcpy(&x, mask + t, 4);
                // the top bit of each byte that is not 0, moved to its lowest; bytes 1, 2, 4, 8 times them summed
                x = ((((x & 0x7f7f7f7fu) + 0x7f7f7f7fu) | x) & 0x80808080u) >> 7;
                return __builtin_amdgcn_udot4(x, 0x08040201u, 0u, false);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) b |= target[t + i] >= 0 ? 1u << i : 0u;
            }
            return b;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t + i < end && (!mask || mask[t + i]) && (!target || target[t + i] >= 0)) b |= 1u << i;
        return b;
    }
    // bit 4g + i: the lane's token i of group g
    template <int G>
    __device__ __forceinline__ uint32_t bits(const Place<G>& w) const {
        uint32_t b = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) b |= bits4(w.at(g), w.p1) << (4 * g);
        return b;
    }
};

// The sequence that holds token p: the last one that begins at or before it.
// All lanes of a wave together: 64 places are looked at in each round.
__device__ __forceinline__ uint32_t find_seq(const Seqs& sq, uint32_t p) {
    if (!sq.off) return p / sq.len;
    const uint32_t lane = threadIdx.x & 63;
    uint32_t lo = 0, hi = sq.n;
    while (hi - lo > 1) {
        const uint32_t step = (hi - lo + 63) / 64;
        const uint32_t k = lo + (lane + 1) * step;
        const uint32_t c = (uint32_t)__popcll(__ballot(k < hi && sq.begin(k) <= p));
        lo += c * step;
        hi = min(lo + step, hi);
    }
    return lo;
}

// A wave's LDS writes before its LDS reads: one wave's are in order, the
// compiler has to leave them so.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The sequence of each of a lane's tokens, as a distance id >= 0 to the
// sequence q0 of the span's first token; the ids never fall along the span.
template <int G>
struct Ids {
    uint32_t q0;
    bool one;  // all tokens in q0
    int id[4 * G];
};
struct MaxStep {
    int v;
    template <int CTRL, int RM>
    __device__ __forceinline__ void step() { v = max(v, dpp<CTRL, RM>(0, v)); }
};
// A wave takes spans that follow each other.  Its lanes hold where the 64
// sequences after q begin, in which a span's first sequence and those that begin
// inside it are looked up; the window moves on when the spans have passed it.
struct Cursor {
    uint32_t q = 0xffffffffu;  // one that begins at or before the next span, or none known
    uint32_t b = 0;            // where sequence q + 1 + lane begins (none: 2^32 - 1)
    __device__ __forceinline__ void look(const Seqs& sq, uint32_t at) {
        q = at;
        const uint32_t k = q + 1 + (threadIdx.x & 63);
        b = k < sq.n ? sq.begin(k) : 0xffffffffu;
    }
};
// Each sequence that begins inside the span marks its first token in `map`
// (G * 256 words of the wave's own in LDS; the last one where some are empty);
// a running maximum then tells every token's.  The cost does not depend on how
// many sequences there are, and offsets that are not non-decreasing give some
// sequences below n.
template <int G>
__device__ __forceinline__ Ids<G> seq_ids(const Seqs& sq, const Place<G>& w, int* map, Cursor& cur) {
    if (!sq.off) cur.look(sq, w.p0 / sq.len);
    else if (cur.q == 0xffffffffu) cur.look(sq, sq.n <= 64 ? 0u : find_seq(sq, w.p0));
    uint32_t passed = (uint32_t)__popcll(__ballot(cur.b <= w.p0));
    if (passed == 64) {
        cur.look(sq, cur.q + 64);
        passed = (uint32_t)__popcll(__ballot(cur.b <= w.p0));
        if (passed == 64) {
            cur.look(sq, find_seq(sq, w.p0));
            passed = (uint32_t)__popcll(__ballot(cur.b <= w.p0));
        }
    }
    Ids<G> s;
    s.q0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)(cur.q + passed));
#pragma unroll
    for (int i = 0; i < 4 * G; ++i) s.id[i] = 0;
    s.one = !__any(cur.b > w.p0 && cur.b < w.p1) && !__all(cur.b < w.p1);
    if (s.one) return s;
    int4* m = reinterpret_cast<int4*>(map);
#pragma unroll
    for (int g = 0; g < G; ++g) m[g * 64 + w.lane] = make_int4(0, 0, 0, 0);
    wave_order();
    for (;;) {
        if (cur.b > w.p0 && cur.b < w.p1) atomicMax(map + (cur.b - w.p0), (int)(cur.q + 1 + w.lane - s.q0));
        if (!__all(cur.b < w.p1)) break;
        cur.look(sq, cur.q + 64);
    }
    wave_order();
    int before = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int4 v = m[g * 64 + w.lane];
        int* id = s.id + 4 * g;
        id[0] = v.x;
        id[1] = max(id[0], v.y);
        id[2] = max(id[1], v.z);
        id[3] = max(id[2], v.w);
        MaxStep x{id[3]};
        wave_scan(x);
        const int low = max(before, dpp<kShr1, 0xf>(0, x.v));
#pragma unroll
        for (int i = 0; i < 4; ++i) id[i] = max(id[i], low);
        before = max(before, lane_value(x.v, 63));
    }
    return s;
}

// A sequence's sum (or a part of it): of values, and of tokens that take part.
struct Part {
    double sum, count;
};

// Sums by sequence of what spans hold.  The first sequence of a span puts its
// part into head, one that holds the span's last token (and not its first)
// into tail, one between is whole.
struct PartSums {
    Part *head, *tail, *whole;
    // The sum of sequence q over spans of `size` tokens, by N lanes of which this
    // is number i: the first span's part by where the sequence begins and ends in
    // it, the others are their spans' first.
    __device__ __forceinline__ Part some(const Seqs& sq, uint32_t q, uint32_t size, uint32_t i, uint32_t n) const {
        const uint32_t b = sq.begin(q), e = sq.end(q);
        Part v{0.0, 0.0};
        if (e <= b) return v;
        const uint32_t s0 = b / size, s1 = (e - 1) / size;
        if (i == 0) v = b <= s0 * size ? head[s0] : e >= min((s0 + 1) * size, sq.tokens) ? tail[s0] : whole[q];
#pragma unroll 4
        for (uint32_t s = s0 + 1 + i; s <= s1; s += n) {
            v.sum += head[s].sum;
            v.count += head[s].count;
        }
        return v;
    }
    // by a wave, all lanes together
    __device__ __forceinline__ Part by_wave(const Seqs& sq, uint32_t q, uint32_t size) const {
        const Part v = some(sq, q, size, threadIdx.x & 63, 64);
        return Part{wave_sum(v.sum), wave_sum(v.count)};
    }
    // by a workgroup, all threads together
    template <int NT>
    __device__ __forceinline__ Part by_group(const Seqs& sq, uint32_t q, uint32_t size, double* red) const {
        const Part v = some(sq, q, size, threadIdx.x, NT);
        return Part{wg_sum<NT>(v.sum, red), wg_sum<NT>(v.count, red)};
    }
    // by one thread: where a sequence has a few spans at most
    __device__ __forceinline__ Part by_lane(const Seqs& sq, uint32_t q, uint32_t size) const {
        return some(sq, q, size, 0, 1);
    }
};

// A step of the scan by sequence: the lane's running sum takes another's where
// that one ends in the same sequence (ids do not fall, so nothing between differs).
template <bool VALUE>
struct SeqStep {
    double x;
    int n, key;
    template <int CTRL, int RM>
    __device__ __forceinline__ void step() {
        const int k = dpp<CTRL, RM>(-1, key), m = dpp<CTRL, RM>(0, n);
        const double y = VALUE ? dpp<CTRL, RM>(x) : 0.0;
        if (k == key) {
            n += m;
            if (VALUE) x += y;
        }
    }
};

// A span's sums by sequence: of v (VALUE; 0 at tokens that take no part) and of
// live's bits.  A NaN or infinity stays in its own sequence.
template <int G, bool VALUE>
__device__ __forceinline__ void sum_span(const Place<G>& w, uint32_t span, const Ids<G>& s, const double* v,
                                         uint32_t live, const PartSums& out) {
    if (s.one) {
        double x = 0.0;
        if (VALUE) {
#pragma unroll
            for (int k = 0; k < 4 * G; ++k) x += v[k];
            x = wave_sum(x);
        }
        const int n = wave_sum((int)__popc(live));
        if (w.lane == 0) out.head[span] = Part{x, (double)n};
        return;
    }
    double cx = 0.0;  // the sum that the group before left open, and its sequence
    int cn = 0, ckey = -1;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int* id = s.id + 4 * g;
        double x[4];
        int n[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = VALUE ? v[4 * g + i] : 0.0;
            n[i] = (int)((live >> (4 * g + i)) & 1u);
            if (i == 0 ? w.lane == 0 && id[0] == ckey : id[i] == id[i > 0 ? i - 1 : 0]) {
                if (VALUE) x[i] += i == 0 ? cx : x[i > 0 ? i - 1 : 0];
                n[i] += i == 0 ? cn : n[i > 0 ? i - 1 : 0];
            }
        }
        SeqStep<VALUE> t{x[3], n[3], id[3]};
        wave_scan(t);
        const int pk = dpp<kShr1, 0xf>(-1, t.key), pn = dpp<kShr1, 0xf>(0, t.n);
        const double px = VALUE ? dpp<kShr1, 0xf>(t.x) : 0.0;
        // the sequence of the token after the lane's last one
        int next = dpp<kShl1, 0xf>(-1, id[0]);
        if (g + 1 < G) {
            const int first = lane_value(s.id[4 * (g + 1 < G ? g + 1 : g)], 0);
            if (w.lane == 63) next = first;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (pk == id[i]) {
                if (VALUE) x[i] += px;
                n[i] += pn;
            }
            const uint32_t at = w.at(g) + i;
            const bool last = at + 1 == w.p1;
            if (at < w.p1 && (last || id[i] != (i < 3 ? id[i < 3 ? i + 1 : 3] : next)))
                (id[i] == 0 ? out.head[span] : last ? out.tail[span] : out.whole[s.q0 + id[i]]) = Part{x[i], (double)n[i]};
        }
        cx = VALUE ? lane_value(t.x, 63) : 0.0;
        cn = lane_value(t.n, 63);
        ckey = lane_value(t.key, 63);
    }
}

// f(i, sequence) for a lane's tokens i of group g: once for all four, then
// f.same(), where they are in one sequence (nearly all lanes).
template <int G, typename F>
__device__ __forceinline__ void by_token(const Ids<G>& s, int g, F f) {
    const int* id = s.id + 4 * g;
    f(0, s.q0 + (uint32_t)id[0]);
    f.same();
    if (id[0] != id[3]) {
#pragma unroll
        for (int i = 1; i < 4; ++i) f(i, s.q0 + (uint32_t)id[i]);
    }
}

uint32_t spans_of(int64_t tokens, int g) { return (uint32_t)((tokens + 256 * g - 1) / (256 * g)); }

// Workgroups for `waves` waves' work, at most `most` (each then takes more).
dim3 wave_grid(int64_t waves, int64_t most = kGrid) {
    const int64_t g = (waves + kLossNT / 64 - 1) / (kLossNT / 64);
    return dim3((unsigned)(g < 1 ? 1 : g > most ? most : g));
}

// A wave's number among all of a launch, and their number; its share of n
// items, which follow each other.
struct Wave {
    uint32_t id, count;
    __device__ __forceinline__ explicit Wave(uint32_t first_block = 0) {
        const uint32_t nw = blockDim.x >> 6;
        id = (blockIdx.x - first_block) * nw + (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        count = (gridDim.x - first_block) * nw;
    }
    template <typename F>
    __device__ __forceinline__ void each(uint32_t n, F f) const {
        const uint32_t part = (n + count - 1) / count;
        const uint32_t e = min((id + 1) * part, n);
        for (uint32_t i = id * part; i < e; ++i) f(i);
    }
};

// A wave's own map for the sequences of its tokens.
template <int NT, int G>
struct Maps {
    int word[NT / 64][256 * G];
    __device__ __forceinline__ int* mine() { return word[__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6))]; }
};

struct Taker {  // places in a workspace, 256-byte aligned
    size_t at = 0;
    size_t take(int64_t n, size_t size) {
        const size_t o = at;
        at += ((size_t)n * size + 255) / 256 * 256;
        return o;
    }
};
// Span sums take as many places as the smaller spans need.
struct SumsPlan {
    size_t head, tail, whole;
    SumsPlan(Taker& t, int64_t tokens, int64_t seqs) {
        const int g = tokens <= kOneMax ? 1 : kSpanG;
        head = t.take(spans_of(tokens, g), sizeof(Part));
        tail = t.take(spans_of(tokens, g), sizeof(Part));
        whole = t.take(seqs, sizeof(Part));
    }
    PartSums at(char* ws) const {
        return PartSums{reinterpret_cast<Part*>(ws + head), reinterpret_cast<Part*>(ws + tail),
                        reinterpret_cast<Part*>(ws + whole)};
    }
};

// ---- preference loss ----

struct Pref {
    const float* logp;
    const float* ref;  // or NULL
    Live live;
    Seqs sq;
    uint32_t pairs;
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

template <int G>
__device__ __forceinline__ void pref_sums(const Pref& p, uint32_t span, int* map, Cursor& cur) {
    const Place<G> w(span, p.sq.tokens);
    float x[4 * G], y[4 * G];
    double v[4 * G];
    const uint32_t live = p.live.bits(w);
    load_span(p.logp, w, x);
    if (p.ref) {
        load_span(p.ref, w, y);
    } else {
#pragma unroll
        for (int k = 0; k < 4 * G; ++k) y[k] = 0.0f;
    }
    const Ids<G> s = seq_ids(p.sq, w, map, cur);
#pragma unroll
    for (int k = 0; k < 4 * G; ++k) v[k] = (live >> k) & 1u ? (double)x[k] - (double)y[k] : 0.0;
    sum_span<G, true>(w, span, s, v, live, p.sums);
}

// Pair i, of the sums c and r of its sequences.
__device__ __forceinline__ void pref_pair(const Pref& p, uint32_t i, Part c, Part r) {
    const double fc = p.mean ? 1.0 / fmax(c.count, 1.0) : 1.0, fr = p.mean ? 1.0 / fmax(r.count, 1.0) : 1.0;
    c.sum *= fc;
    r.sum *= fr;
    const double delta = c.sum - r.sum;
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
    slope *= p.grad_scale / (double)p.pairs;
    p.each[i] = loss;
    p.coef[2 * i] = (float)(slope * fc);
    p.coef[2 * i + 1] = (float)(-slope * fr);
    p.pair_loss[i] = (float)loss;
    p.reward[2 * i] = (float)(p.beta * c.sum);
    p.reward[2 * i + 1] = (float)(p.beta * r.sum);
}

struct Coefs {
    const float* coef;
    float* c;
    __device__ __forceinline__ void operator()(int i, uint32_t q) const { c[i] = coef[q]; }
    __device__ __forceinline__ void same() const { c[1] = c[2] = c[3] = c[0]; }
};
template <int G>
__device__ __forceinline__ void pref_grad(const Pref& p, uint32_t span, int* map, Cursor& cur) {
    const Place<G> w(span, p.sq.tokens);
    const uint32_t live = p.live.bits(w);
    const Ids<G> s = seq_ids(p.sq, w, map, cur);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float c[4];
        by_token(s, g, Coefs{p.coef, c});
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = (live >> (4 * g + i)) & 1u ? c[i] : 0.0f;
        store4(p.grad, w.at(g), w.p1, c);
    }
}

template <int NT>
__device__ __forceinline__ void pref_mean(const Pref& p) {
    __shared__ double red[NT / 64];
    double v = 0.0;
    for (uint32_t i = threadIdx.x; i < p.pairs; i += NT) v += p.each[i];
    v = wg_sum<NT>(v, red);
    if (threadIdx.x == 0) *p.loss = p.pairs ? (float)(v / (double)p.pairs) : 0.0f;
}

__global__ __launch_bounds__(kLossNT) void k_pref_sums(Pref p, uint32_t spans) {
    __shared__ Maps<kLossNT, kSpanG> maps;
    const Wave w;
    Cursor cur;
    w.each(spans, [&](uint32_t s) { pref_sums<kSpanG>(p, s, maps.mine(), cur); });
}
// 4e6 tokens in 1000 pairs: sums 11 us (28 MB read), pairs 5, gradient 7 (16 MB
// written), each launch about 3 of them.
// A wave a pair, or (WIDE) a workgroup: few pairs can be long.
template <bool WIDE>
__global__ __launch_bounds__(kLossNT) void k_pref_pairs(Pref p) {
    __shared__ double red[kLossNT / 64];
    const Wave w;
    for (uint32_t i = WIDE ? blockIdx.x : w.id; i < p.pairs; i += WIDE ? gridDim.x : w.count) {
        Part v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            v[k] = WIDE ? p.sums.by_group<kLossNT>(p.sq, 2 * i + k, 256 * kSpanG, red)
                        : p.sums.by_wave(p.sq, 2 * i + k, 256 * kSpanG);
        if ((WIDE ? threadIdx.x : threadIdx.x & 63) == 0) pref_pair(p, i, v[0], v[1]);
    }
}
// The first workgroup takes the mean of the pair losses, the others the tokens.
__global__ __launch_bounds__(kLossNT) void k_pref_grad(Pref p, uint32_t spans) {
    __shared__ Maps<kLossNT, kSpanG> maps;
    if (blockIdx.x == 0) {
        pref_mean<kLossNT>(p);
        return;
    }
    const Wave w(1);
    Cursor cur;
    w.each(spans, [&](uint32_t s) { pref_grad<kSpanG>(p, s, maps.mine(), cur); });
}
// A small call whole: the three steps by one workgroup.
__global__ __launch_bounds__(kOneNT) void k_pref_one(Pref p, uint32_t spans) {
    __shared__ Maps<kOneNT, 1> maps;
    const Wave w;
    Cursor first, second;
    w.each(spans, [&](uint32_t s) { pref_sums<1>(p, s, maps.mine(), first); });
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < p.pairs; i += kOneNT)
        pref_pair(p, i, p.sums.by_lane(p.sq, 2 * i, 256), p.sums.by_lane(p.sq, 2 * i + 1, 256));
    __syncthreads();
    if (p.grad) w.each(spans, [&](uint32_t s) { pref_grad<1>(p, s, maps.mine(), second); });
    pref_mean<kOneNT>(p);
}

struct PrefPlan {
    Taker t;
    SumsPlan sums;
    size_t off_each, off_coef, bytes;
    PrefPlan(int64_t tokens, int64_t pairs) : sums(t, tokens, 2 * pairs) {
        off_each = t.take(pairs, sizeof(double));
        off_coef = t.take(2 * pairs, sizeof(float));
        bytes = t.at;
    }
};

// ---- policy loss ----

// Weights of tokens: what the loss, and the rows' terms, take of a policy call.
struct Weights {
    Policy p;
    Live live;
    Seqs sq;
    PartSums sums;    // (0, tokens that take part)
    double* weight;   // a sequence's w_t (ISO_POLICY_SEQ_MEAN)
    int* counted;     // a workgroup's tokens that take part (else)
    uint32_t parts;   // how many of them
    __device__ __forceinline__ bool by_seq() const { return p.seq_mean != 0; }
};

// What tokens take from their sequence: its advantage, its weight.
template <bool ADV, bool WEIGHT>
struct SeqTerms {
    const Weights& c;
    float* adv;
    double* wt;
    __device__ __forceinline__ void operator()(int i, uint32_t q) const {
        if (ADV) adv[i] = c.p.adv[q];
        if (WEIGHT) wt[i] = c.weight[q];
    }
    __device__ __forceinline__ void same() const {
        if (ADV) adv[1] = adv[2] = adv[3] = adv[0];
        if (WEIGHT) wt[1] = wt[2] = wt[3] = wt[0];
    }
};

// Tokens that take part, by sequence.
template <int G>
__device__ __forceinline__ void count_by_seq(const Weights& c, uint32_t span, int* map, Cursor& cur) {
    const Place<G> w(span, c.sq.tokens);
    const uint32_t live = c.live.bits(w);
    const Ids<G> s = seq_ids(c.sq, w, map, cur);
    sum_span<G, false>(w, span, s, nullptr, live, c.sums);
}
// Sequence q's weight, from the count of its tokens that take part.
__device__ __forceinline__ void weigh_seq(const Weights& c, uint32_t q, double count) {
    c.weight[q] = c.p.seq_weight(c.sq.n, c.live.all() ? (double)(c.sq.end(q) - c.sq.begin(q)) : count);
}

// The weight that all tokens share, for every thread of a workgroup: from the
// workgroups' counts.
template <int NT>
__device__ __forceinline__ double shared_weight(const Weights& c) {
    __shared__ int red[NT / 64];
    if (c.by_seq()) return 0.0;
    if (c.live.all()) return c.p.token_weight((int)c.sq.tokens);
    int n = 0;
    for (uint32_t k = threadIdx.x; k < c.parts; k += NT) n += c.counted[k];
    return c.p.token_weight(wg_sum<NT>(n, red));
}
// The weights of a small call, by one workgroup: every token's if they are alike.
template <int NT>
__device__ __forceinline__ double small_weights(const Weights& c, uint32_t spans, int* map) {
    __shared__ int red[NT / 64];
    const Wave w;
    if (c.by_seq()) {
        if (!c.live.all()) {
            Cursor cur;
            w.each(spans, [&](uint32_t s) { count_by_seq<1>(c, s, map, cur); });
            __syncthreads();
        }
        for (uint32_t q = threadIdx.x; q < c.sq.n; q += NT)
            weigh_seq(c, q, c.live.all() ? 0.0 : c.sums.by_lane(c.sq, q, 256).count);
        __syncthreads();
        return 0.0;
    }
    if (c.live.all()) return c.p.token_weight((int)c.sq.tokens);
    int n = 0;
    for (uint32_t s = w.id; s < spans; s += w.count) n += (int)__popc(c.live.bits(Place<1>(s, c.sq.tokens)));
    return c.p.token_weight(wg_sum<NT>(n, red));
}

__global__ __launch_bounds__(kLossNT) void k_count_by_seq(Weights c, uint32_t spans) {
    __shared__ Maps<kLossNT, kSpanG> maps;
    const Wave w;
    Cursor cur;
    w.each(spans, [&](uint32_t s) { count_by_seq<kSpanG>(c, s, maps.mine(), cur); });
}
// A thread a sequence where every token takes part, else a wave, or (WIDE) a workgroup.
template <bool WIDE>
__global__ __launch_bounds__(kLossNT) void k_weigh_seqs(Weights c) {
    __shared__ double red[kLossNT / 64];
    if (c.live.all()) {
        for (uint32_t q = blockIdx.x * kLossNT + threadIdx.x; q < c.sq.n; q += gridDim.x * kLossNT) weigh_seq(c, q, 0.0);
        return;
    }
    const Wave w;
    for (uint32_t q = WIDE ? blockIdx.x : w.id; q < c.sq.n; q += WIDE ? gridDim.x : w.count) {
        const double n = WIDE ? c.sums.by_group<kLossNT>(c.sq, q, 256 * kSpanG, red).count
                              : c.sums.by_wave(c.sq, q, 256 * kSpanG).count;
        if ((WIDE ? threadIdx.x : threadIdx.x & 63) == 0) weigh_seq(c, q, n);
    }
}
__global__ __launch_bounds__(kLossNT) void k_count(Weights c, uint32_t spans) {
    __shared__ int red[kLossNT / 64];
    const Wave w;
    int n = 0;
    for (uint32_t s = w.id; s < spans; s += w.count) n += (int)__popc(c.live.bits(Place<kSpanG>(s, c.sq.tokens)));
    n = wg_sum<kLossNT>(n, red);
    if (threadIdx.x == 0) c.counted[blockIdx.x] = n;
}

struct PolicyCall {
    Weights c;
    const float* logp;
    float* loss;
    int32_t* counts;
    float* grad;       // or NULL
    PolicySums* part;  // a workgroup's sums
};

// What a policy call has: advantages by token, weights by sequence, a
// reference.  The kernels over tokens are made for each combination: asked at
// run time, the questions are a third of the instructions (67 -> 61 us at 8e6 tokens).
template <bool TOKEN_ADV, bool BY_SEQ, bool REF>
struct Kind {
    static constexpr bool token_adv = TOKEN_ADV, by_seq = BY_SEQ, ref = REF;
};
template <typename F>
void by_kind(const Policy& p, F f) {
    auto third = [&](auto t, auto s) {
        if (p.ref_logp) f(Kind<decltype(t)::value, decltype(s)::value, true>{});
        else f(Kind<decltype(t)::value, decltype(s)::value, false>{});
    };
    auto second = [&](auto t) {
        if (p.seq_mean) third(t, std::true_type{});
        else third(t, std::false_type{});
    };
    if (p.token_adv) second(std::true_type{});
    else second(std::false_type{});
}

// The terms of a span's tokens, summed into s by lane; their gradient is written.
template <typename K, int G>
__device__ __forceinline__ void policy_span(const PolicyCall& f, uint32_t span, double all, const ExpSeries& ex,
                                            PolicySums& s, int* map, Cursor& cur) {
    const Weights& c = f.c;
    const Policy& p = c.p;
    const Place<G> w(span, c.sq.tokens);
    float lp[4 * G], old[4 * G], ref[4 * G], adv[4 * G];
    const uint32_t live = c.live.bits(w);
    load_span(f.logp, w, lp);
    load_span(p.old_logp, w, old);
    if (K::ref) load_span(p.ref_logp, w, ref);
    if (K::token_adv) load_span(p.adv, w, adv);
    Ids<G> ids;
    constexpr bool need_ids = !K::token_adv || K::by_seq;
    if (need_ids) ids = seq_ids(c.sq, w, map, cur);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        double wt[4] = {all, all, all, all};
        if (need_ids) by_token(ids, g, SeqTerms<!K::token_adv, K::by_seq>{c, adv + 4 * g, wt});
        float o4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t on = (live >> (4 * g)) & 15u;
        if (__any(on)) {
            double d[4], u[4];
            float a[4];
            PolicyTerm o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = adv[4 * g + i];
            if (on != 15u) {
                // a token that takes no part: d, u and a are 0 whatever it holds, and so are its terms
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = 4 * g + i;
                    const bool in = (on >> i) & 1u;
                    lp[k] = in ? lp[k] : 0.0f;
                    old[k] = in ? old[k] : 0.0f;
                    if (K::ref) ref[k] = in ? ref[k] : 0.0f;
                    a[i] = in ? a[i] : 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = 4 * g + i;
                d[i] = (double)lp[k] - (double)old[k];
                u[i] = K::ref ? (double)ref[k] - (double)lp[k] : 0.0;
            }
            policy_terms<K::ref>(p, ex, d, u, a, o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s.pg += wt[i] * o[i].pg;
                s.kl += wt[i] * o[i].kl;
                s.over += o[i].over ? 1 : 0;
                o4[i] = (float)(o[i].slope * (wt[i] * p.grad_scale));
            }
            s.live += (int)__popc(on);
        }
        if (f.grad) store4(f.grad, w.at(g), w.p1, o4);
    }
}

// The workgroup's sums, in thread 0.
template <int NT>
__device__ __forceinline__ PolicySums wg_policy(const PolicySums& s) {
    __shared__ PolicySums red[NT / 64];
    PolicySums o{wave_sum(s.pg), wave_sum(s.kl), wave_sum(s.live), wave_sum(s.over)};
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = o;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int k = 1; k < NT / 64; ++k) {
            o.pg += red[k].pg;
            o.kl += red[k].kl;
            o.live += red[k].live;
            o.over += red[k].over;
        }
    return o;
}
__device__ __forceinline__ void policy_out(double kl_coef, const PolicySums& s, float* loss, int32_t* counts) {
    loss[0] = (float)(kl_coef != 0.0 ? s.pg + kl_coef * s.kl : s.pg);
    loss[1] = (float)s.pg;
    loss[2] = (float)s.kl;
    counts[0] = s.live;
    counts[1] = s.over;
}

// Bound by its f64 instructions: 8e6 tokens take 10.9e6 wave instructions (18 of
// 36 us of every SIMD's issue at 2.4 GHz; two thirds of the time that waves live)
// for 105 MB read and 32 MB written.  More waves (5, 6, 8 a SIMD) spill, spans
// of 256 or 1024 tokens were 7 and 12 % slower, and loads issued a span ahead
// brought nothing.
template <typename K>
__global__ __launch_bounds__(kLossNT, kTermWaves) void k_policy_tokens(PolicyCall f, uint32_t spans) {
    __shared__ Maps<kLossNT, kTermG> maps;
    const double all = shared_weight<kLossNT>(f.c);
    const Wave w;
    const ExpSeries ex;
    PolicySums s{};
    Cursor cur;
    w.each(spans, [&](uint32_t k) { policy_span<K, kTermG>(f, k, all, ex, s, maps.mine(), cur); });
    s = wg_policy<kLossNT>(s);
    if (threadIdx.x == 0) f.part[blockIdx.x] = s;
}
__global__ __launch_bounds__(kOneNT) void k_policy_out(double kl_coef, const PolicySums* __restrict__ part, int parts,
                                                       float* loss, int32_t* counts) {
    PolicySums s{};
    for (int k = threadIdx.x; k < parts; k += kOneNT) {
        const PolicySums o = part[k];
        s.pg += o.pg;
        s.kl += o.kl;
        s.live += o.live;
        s.over += o.over;
    }
    s = wg_policy<kOneNT>(s);
    if (threadIdx.x == 0) policy_out(kl_coef, s, loss, counts);
}
// A small call whole.
template <typename K>
__global__ __launch_bounds__(kOneNT) void k_policy_one(PolicyCall f, uint32_t spans) {
    __shared__ Maps<kOneNT, 1> maps;
    const double all = small_weights<kOneNT>(f.c, spans, maps.mine());
    const Wave w;
    const ExpSeries ex;
    PolicySums s{};
    Cursor cur;
    w.each(spans, [&](uint32_t k) { policy_span<K, 1>(f, k, all, ex, s, maps.mine(), cur); });
    s = wg_policy<kOneNT>(s);
    if (threadIdx.x == 0) policy_out(f.c.p.kl_coef, s, f.loss, f.counts);
}

// Rows' terms of the loss from logits.
template <int G>
__device__ __forceinline__ void row_span(const Weights& c, uint32_t span, double all, RowTerm* terms, int* map,
                                         Cursor& cur) {
    const Place<G> w(span, c.sq.tokens);
    const uint32_t live = c.live.bits(w);
    Ids<G> ids;
    const bool need_ids = !c.p.token_adv || c.by_seq();
    if (need_ids) ids = seq_ids(c.sq, w, map, cur);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float adv[4];
        double wt[4] = {all, all, all, all};
        if (c.p.token_adv) load4(c.p.adv, w.at(g), w.p1, adv);
        if (need_ids) {
            if (!c.p.token_adv) by_token(ids, g, SeqTerms<true, false>{c, adv, wt});
            if (c.by_seq()) by_token(ids, g, SeqTerms<false, true>{c, adv, wt});
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (w.at(g) + i < w.p1)
                terms[w.at(g) + i] = RowTerm{(live >> (4 * g + i)) & 1u ? wt[i] : 0.0, adv[i], 0.0f};
    }
}
__global__ __launch_bounds__(kLossNT) void k_row_terms(Weights c, uint32_t spans, RowTerm* terms) {
    __shared__ Maps<kLossNT, kSpanG> maps;
    const double all = shared_weight<kLossNT>(c);
    const Wave w;
    Cursor cur;
    w.each(spans, [&](uint32_t k) { row_span<kSpanG>(c, k, all, terms, maps.mine(), cur); });
}
__global__ __launch_bounds__(kOneNT) void k_row_terms_one(Weights c, uint32_t spans, RowTerm* terms) {
    __shared__ Maps<kOneNT, 1> maps;
    const double all = small_weights<kOneNT>(c, spans, maps.mine());
    const Wave w;
    Cursor cur;
    w.each(spans, [&](uint32_t k) { row_span<1>(c, k, all, terms, maps.mine(), cur); });
}

constexpr int kCountGrid = 512;  // workgroups that count, their counts read by every later workgroup

struct WeightsPlan {
    Taker t;
    SumsPlan sums;
    size_t off_weight, off_counted, bytes;
    WeightsPlan(int64_t tokens, int64_t seqs) : sums(t, tokens, seqs) {
        off_weight = t.take(seqs, sizeof(double));
        off_counted = t.take(kCountGrid, sizeof(int));
        bytes = t.at;
    }
};

Weights make_weights(const Policy& p, const Live& live, const Seqs& sq, const WeightsPlan& pl, char* ws) {
    return Weights{p, live, sq, pl.sums.at(ws), reinterpret_cast<double*>(ws + pl.off_weight),
                   reinterpret_cast<int*>(ws + pl.off_counted), 0};
}
bool small_call(const Seqs& sq) { return sq.tokens <= kOneMax && sq.n <= kOneMax; }

// What the weights of a larger call take: tokens counted (if not all take
// part), by sequence or by workgroup, and each sequence's weight.
void start_weights(Weights& c, hipStream_t st) {
    const uint32_t spans = spans_of(c.sq.tokens, kSpanG);
    const dim3 nt(kLossNT);
    if (c.p.seq_mean) {
        if (!c.live.all()) hipLaunchKernelGGL(k_count_by_seq, wave_grid(spans), nt, 0, st, c, spans);
        if (c.sq.n <= kWideSeqs) hipLaunchKernelGGL((k_weigh_seqs<true>), dim3(c.sq.n ? c.sq.n : 1), nt, 0, st, c);
        else hipLaunchKernelGGL((k_weigh_seqs<false>), wave_grid(c.sq.n, 65536), nt, 0, st, c);
    } else if (!c.live.all()) {
        const dim3 grid = wave_grid(spans, kCountGrid);
        c.parts = grid.x;
        hipLaunchKernelGGL(k_count, grid, nt, 0, st, c, spans);
    }
}

struct PolicyPlan {
    WeightsPlan w;
    size_t off_part, bytes;
    PolicyPlan(int64_t tokens, int64_t seqs) : w(tokens, seqs) {
        off_part = w.t.take((int64_t)wave_grid(spans_of(tokens, kTermG), kTermGrid).x, sizeof(PolicySums));
        bytes = w.t.at;
    }
};

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

size_t row_terms_workspace(int64_t rows, int64_t seqs) { return WeightsPlan(rows, seqs).bytes; }

hipError_t launch_row_terms(const Policy& p, const int32_t* target, const Seqs& sq, RowTerm* terms, void* workspace,
                            hipStream_t st) {
    Weights c = make_weights(p, Live{nullptr, target}, sq, WeightsPlan(sq.tokens, sq.n), static_cast<char*>(workspace));
    if (small_call(sq)) {
        hipLaunchKernelGGL(k_row_terms_one, dim3(1), dim3(kOneNT), 0, st, c, spans_of(sq.tokens, 1), terms);
        return hipGetLastError();
    }
    start_weights(c, st);
    const uint32_t spans = spans_of(sq.tokens, kSpanG);
    hipLaunchKernelGGL(k_row_terms, wave_grid(spans), dim3(kLossNT), 0, st, c, spans, terms);
    return hipGetLastError();
}

hipError_t launch_policy_out(const Policy& p, const PolicySums* part, int parts, float* loss, int32_t* counts,
                             hipStream_t st) {
    hipLaunchKernelGGL(k_policy_out, dim3(1), dim3(kOneNT), 0, st, p.kl_coef, part, parts, loss, counts);
    return hipGetLastError();
}

}  // namespace iso

extern "C" {

size_t iso_pref_loss_workspace_bytes(int64_t tokens, int64_t pairs) {
    if (tokens < 0 || pairs < 0 || tokens > 0x7fffffffLL || pairs > 0x3fffffffLL) return 0;
    return iso::PrefPlan(tokens, pairs).bytes;
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
    const PrefPlan pl(tokens, pairs);
    char* ws = static_cast<char*>(workspace);
    Pref p;
    p.logp = logp;
    p.ref = ref_logp;
    p.live = Live{mask, nullptr};
    p.sq = make_seqs(seq_off, 2 * pairs, tokens);
    p.pairs = (uint32_t)pairs;
    p.beta = beta;
    p.smooth = label_smoothing;
    p.mean = (flags & ISO_PREF_MEAN) != 0;
    p.squared = (flags & ISO_PREF_SQUARED) != 0;
    p.grad_scale = grad_scale;
    p.loss = loss;
    p.pair_loss = pair_loss;
    p.reward = reward;
    p.grad = grad;
    p.sums = pl.sums.at(ws);
    p.each = reinterpret_cast<double*>(ws + pl.off_each);
    p.coef = reinterpret_cast<float*>(ws + pl.off_coef);
    if (small_call(p.sq)) {
        hipLaunchKernelGGL(k_pref_one, dim3(1), dim3(kOneNT), 0, st, p, spans_of(tokens, 1));
        return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
    }
    const dim3 nt(kLossNT);
    const uint32_t spans = spans_of(tokens, kSpanG);
    hipLaunchKernelGGL(k_pref_sums, wave_grid(spans), nt, 0, st, p, spans);
    if (pairs <= kWideSeqs) hipLaunchKernelGGL((k_pref_pairs<true>), dim3((unsigned)(pairs ? pairs : 1)), nt, 0, st, p);
    else hipLaunchKernelGGL((k_pref_pairs<false>), wave_grid(pairs, 65536), nt, 0, st, p);
    hipLaunchKernelGGL(k_pref_grad, dim3(grad ? wave_grid(spans).x + 1 : 1), nt, 0, st, p, spans);
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

size_t iso_policy_loss_workspace_bytes(int64_t tokens, int64_t seqs) {
    if (tokens < 0 || seqs < 0 || tokens > 0x7fffffffLL || seqs > 0x7fffffffLL) return 0;
    return iso::PolicyPlan(tokens, seqs).bytes;
}

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
    hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const PolicyPlan pl(tokens, seqs);
    const Policy p = make_policy(old_logp, ref_logp, adv, clip_lo, clip_hi, kl_coef, norm, grad_scale, flags);
    PolicyCall f{make_weights(p, Live{mask, nullptr}, make_seqs(seq_off, seqs, tokens), pl.w, ws), logp, loss, counts,
                 grad, reinterpret_cast<PolicySums*>(ws + pl.off_part)};
    if (small_call(f.c.sq)) {
        by_kind(p, [&](auto k) {
            hipLaunchKernelGGL((k_policy_one<decltype(k)>), dim3(1), dim3(kOneNT), 0, st, f, spans_of(tokens, 1));
        });
        return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
    }
    start_weights(f.c, st);
    const uint32_t spans = spans_of(tokens, kTermG);
    const dim3 grid = wave_grid(spans, kTermGrid);
    by_kind(p, [&](auto k) {
        hipLaunchKernelGGL((k_policy_tokens<decltype(k)>), grid, dim3(kLossNT), 0, st, f, spans);
    });
    return launch_policy_out(p, f.part, (int)grid.x, loss, counts, st) == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

}  // extern "C"
