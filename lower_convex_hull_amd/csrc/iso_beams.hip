// Beam search: the selection over beams and vocabulary from logits, and the
// states of beams brought into the order of their parents (formulas in iso.h).
#include "iso_logits.hpp"
#include "iso_states.hpp"

#include <type_traits>

namespace iso {
namespace {

constexpr int kMaxBeams = 128, kMaxTake = 128;
constexpr int64_t kMaxGrid = 1 << 20;

// f32 values as whole numbers in the same order; -0 is 0.  Nothing but NaN is 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}

// A token of a row: the higher logit first, then the lower token.  0: none.
__device__ __forceinline__ uint64_t token_key(float x, int v) {
    return x > -INFINITY ? ((uint64_t)ordered(x) << 32) | (uint32_t)~v : 0;
}
__device__ __forceinline__ float key_logit(uint64_t k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_token(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)v, d);
        v = o > v ? o : v;
    }
    return v;
}

// A piece of a row: its maximum and the sum of exp2((x - m) c).
struct PieceSum {
    double m, s;
};

// Keys of a batch item: place i of list l at i * stride + (l + i * turn) mod stride.
// The best keys are the first ones of a few lists; a stride that is odd and a turn
// of 5/8 of it spread them over the threads of the join, whose maxima bound little
// where few threads hold them all (without the turn 128 x 32000 bf16, 128 of them,
// went through the rounds of a maximum: 4377 us).
__host__ __device__ __forceinline__ uint32_t key_stride(uint32_t lists) { return lists | 1u; }
__device__ __forceinline__ uint32_t key_turn(uint32_t stride) { return stride * 5u / 8u; }  // strides are below 2^25
__device__ __forceinline__ int64_t key_at(uint32_t i, uint32_t list, uint32_t stride) {
    return (int64_t)i * stride + (list + i * key_turn(stride)) % stride;
}

struct Beams {
    const float* score;
    const float* weight;   // or NULL
    const uint8_t* ended;  // or NULL
    int beams, take;
    int32_t end_token;
    // Row r: 0 no candidates, 1 its tokens, 2 itself.  The three are read at once.
    __device__ __forceinline__ int state(int64_t r) const {
        const float s = score[r], w = weight ? weight[r] : 1.0f;
        const uint8_t e = ended ? ended[r] : (uint8_t)0;
        const bool counts = (fabsf(s) < INFINITY) & (w > 0.0f) & (w < INFINITY);
        return counts ? e ? 2 : 1 : 0;
    }
};

// A value t >= 1 that at least n of a wave's values (V a lane) reach, and few
// more; 1 if less than n of them are not 0.  Bits below LOW tell no two apart.
template <int LOW, int V>
__device__ __forceinline__ uint32_t reached_by(const uint32_t (&v)[V], int n) {
    uint32_t t = 0;
    for (int bit = 31; bit >= LOW; --bit) {
        const uint32_t c = t | (1u << bit);
        int count = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) count += __popcll(__ballot(v[i] >= c));
        if (count >= n) {
            t = c;
            if (count <= n + n / 4) break;
        }
    }
    return t ? t : 1u;
}
// The bits of ordered() that a type's values leave alike.
template <typename T>
constexpr int kLowBits = std::is_same<T, float>::value ? 0 : std::is_same<T, __bf16>::value ? 16 : 13;

// Room for the candidates that reach a bound (in a piece: 4 a thread); where more
// do, a round of a maximum each finds the best.  That is slow, and masks of a finite
// value come to it where a piece holds little else (64 x 8 x 131072 bf16, 16 each, all but
// 100 tokens at the lowest value: 1278 us; at -infinity, which reaches no bound, 40).
constexpr int kRoom = 1024;

// How many of `found` keys in LDS are above k; the next 7 places hold keys that
// are above none.
template <typename K, typename F>
__device__ __forceinline__ int rank_of(const K* room, int found, F above) {
    int rank = 0;
    for (int j = 0; j < found; j += 8)
#pragma unroll
        for (int i = 0; i < 8; ++i) rank += above(room[j + i]);
    return rank;
}

// The larger of three; what it makes of a NaN does not matter here.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
    return d;
}

// The terms exp2((x - m) c) of a piece's sum, m its maximum.  Vectors with a term
// above 1/2 take the difference first, so that the largest term is 1, and are
// summed in f64: where it is nearly all, logp is what the others add to it.
// Other vectors take x c - b with b = fl(m c), one instruction for two, and their
// few terms are summed in f32, which is off by no more than 2^-22 of themselves;
// what b's rounding leaves is a factor of them all, near 1 while b is below 2^10:
// two terms of its series do.  Past that every vector goes the first way.
struct PieceTerms {
    float base, cf, b, edge;
    double rest;
    __device__ __forceinline__ PieceTerms(float m, const Scale& sc) : base(m), cf(sc.cf) {
        const double exact = (double)m * (double)cf;
        const bool large = !(fabs(exact) < 0x1p10);
        b = large ? 0.0f : (float)exact;
        edge = large ? -INFINITY : -1.0f;
        const double d = ((double)b - exact) * kLn2;  // below 2^-15
        rest = large ? 0.0 : fma(0.5 * d, d, d) + 1.0;
    }
    __device__ __forceinline__ float near(float x) const { return __builtin_amdgcn_exp2f((x - base) * cf); }
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N], float top, double& s, double& far) const {
        if ((top - base) * cf >= edge) {
#pragma unroll
            for (int j = 0; j < N; ++j) s += (double)near(x[j]);
        } else {
            float e[N];
#pragma unroll
            for (int j = 0; j < N; ++j) e[j] = __builtin_amdgcn_exp2f(fmaf(x[j], cf, -b));
#pragma unroll
            for (int d = N / 2; d > 0; d >>= 1)
#pragma unroll
                for (int j = 0; j < d; ++j) e[j] += e[j + d];
            far += (double)e[0];
        }
    }
};

// 512 rows x 131072 bf16 (134 MB, read once) take 35 us: 3.8 TB/s and 69 % of the SIMDs'
// issue cycles, neither at its limit; waves wait at the barriers around the bound, which
// one of them seeks.  f32 at 128 x 8 x 200000 is bound by HBM (133 us, 6.1 TB/s), few rows
// by the latency of one piece (6 us).
// A workgroup takes a piece of a row, held in its registers: the piece's maximum
// and sum, and its `take` best tokens.  A value that `take` threads' maxima reach
// bounds the take-th best token from below.  The few vectors that reach it go
// through LDS, where a thread looks at each of their values; the values that
// reach it are brought into order by counting.  A row with a NaN has no
// candidates (its sum is NaN), whatever is found in it.
template <typename T, int NT, int U, bool STREAM>
__global__ __launch_bounds__(NT, U >= 16 ? 4 : 5) void k_beam_pieces(const T* __restrict__ logits, uint32_t rows, int vocab, int64_t ld,
                                                    Beams b, Scale sc, uint32_t splits, uint64_t* __restrict__ keys,
                                                    PieceSum* __restrict__ sums) {
    typedef typename Wide<T>::A Vec;
    constexpr int N = Wide<T>::N, kWaves = NT / 64, kPlaces = NT * 4, kVectors = NT * 2;
    static_assert(kPlaces <= kRoom, "");
    __shared__ uint64_t room[kPlaces + 8];
    __shared__ Vec vec[kVectors];
    __shared__ int at[kVectors];
    __shared__ uint32_t most[NT];
    __shared__ double red_sum[kWaves];
    __shared__ float red[kWaves];
    __shared__ uint32_t bound;
    __shared__ int vectors, count;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (uint32_t r = blockIdx.x; r < rows; r += gridDim.x) {
        if (b.state(r) != 1) continue;
        for (uint32_t split = blockIdx.y; split < splits; split += gridDim.y) {
            const T* x = logits + r * ld;
            const Piece<T> w(x, (int)split, Chunk<T, NT, U>::kSize, vocab);
            Chunk<T, NT, U> c;
            c.template load<STREAM>(x, w.from, w.to);
            const int ke = w.edge();
            const float xe = ke >= 0 ? (float)x[ke] : -INFINITY;
            float top[U], m = xe;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                top[u] = max3((float)c.v[u][0], (float)c.v[u][1], (float)c.v[u][2]);
                if (N == 8) top[u] = max3(top[u], (float)c.v[u][N - 5], (float)c.v[u][N - 4]);
                if (N == 8) top[u] = max3(top[u], (float)c.v[u][N - 3], (float)c.v[u][N - 2]);
                top[u] = fmaxf(top[u], (float)c.v[u][N - 1]);
                m = fmaxf(m, top[u]);
            }
            c.forget();
            most[threadIdx.x] = m > -INFINITY ? ordered(m) : 0;
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
            if (lane == 0) red[wave] = m;
            if (threadIdx.x == 0) vectors = count = 0;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kWaves; ++k) m = fmaxf(m, red[k]);
            if (wave == 0) {
                uint32_t v[kWaves];
#pragma unroll
                for (int k = 0; k < kWaves; ++k) v[k] = most[k * 64 + lane];
                const uint32_t t = reached_by<kLowBits<T>>(v, b.take);
                if (lane == 0) bound = t;
            }
            const float base = base_of(m);
            const PieceTerms terms(base, sc);
            double s = (double)terms.near(xe), far = 0.0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float y[N];
#pragma unroll
                for (int j = 0; j < N; ++j) y[j] = (float)c.v[u][j];
                terms.add(y, top[u], s, far);
            }
            s += far * terms.rest;
            c.forget();
            s = wg_sum<NT>(s, red_sum);
            const uint32_t stride = key_stride((uint32_t)b.beams * splits), item = r / (uint32_t)b.beams;
            const uint32_t list = (r - item * (uint32_t)b.beams) * splits + split;
            if (threadIdx.x == 0) sums[(int64_t)r * splits + split] = PieceSum{(double)m, s};
            // every number reaches the lowest one
            const float low = bound == 1u ? -3.402823466e38f : unordered(bound);
            int n = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) n += __popcll(__ballot(top[u] >= low));
            n += __popcll(__ballot(xe >= low));
            if (n) {
                int p = 0;
                if (lane == 0) p = atomicAdd(&vectors, n);
                p = __builtin_amdgcn_readfirstlane(p);
#pragma unroll
                for (int u = 0; u <= U; ++u) {
                    const bool mine = (u < U ? top[u < U ? u : 0] : xe) >= low;
                    const uint64_t mask = __ballot(mine);
                    const int place = p + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
                    p += __popcll(mask);
                    if (mine && place < kVectors) {
                        if (u < U) vec[place] = c.v[u < U ? u : 0];
                        at[place] = u < U ? c.at(w.from, u) : -1 - ke;  // a value of its own: its place is kept alone
                    }
                }
            }
            __syncthreads();
            const int held = vectors;
            if (held <= kVectors) {
                for (int i = threadIdx.x; i < held * N; i += NT) {
                    const int first = at[i / N];
                    const int k = first < 0 ? -1 - first : first + i % N;
                    // (a value of its own is looked at once)
                    const float v = first >= 0 ? (float)vec[i / N][i % N] : i % N ? -INFINITY : (float)x[k];
                    if (v >= low) {
                        const int p = atomicAdd(&count, 1);
                        if (p < kPlaces) room[p] = token_key(v, k);
                    }
                }
            }
            __syncthreads();
            const int found = held <= kVectors ? count : kPlaces + 1;
            uint64_t* out = keys + (int64_t)item * stride * b.take;
            if (found <= kPlaces) {
                if (threadIdx.x < 8) room[found + threadIdx.x] = 0;
                __syncthreads();
                for (int i = threadIdx.x; i < found; i += NT) {
                    const uint64_t k = room[i];
                    const int rank = rank_of(room, found, [&](uint64_t o) { return o > k; });
                    if (rank < b.take) out[key_at(rank, list, stride)] = k;
                }
                for (int i = found + threadIdx.x; i < b.take; i += NT) out[key_at(i, list, stride)] = 0;
            } else {
                uint64_t last = ~0ull;
                for (int i = 0; i < b.take; ++i) {
                    uint64_t best = token_key(xe, ke);
                    if (best >= last) best = 0;
#pragma unroll 1
                    for (int k = w.from + (int)threadIdx.x; k < w.to; k += NT) {
                        const uint64_t y = token_key((float)x[k], k);
                        best = y < last && y > best ? y : best;
                    }
                    best = wave_max(best);
                    __syncthreads();
                    if (lane == 0) room[wave] = best;
                    __syncthreads();
#pragma unroll
                    for (int k = 0; k < kWaves; ++k) best = room[k] > best ? room[k] : best;
                    if (threadIdx.x == 0) out[key_at(i, list, stride)] = best;
                    last = best;  // 0: nothing is below it
                }
            }
            __syncthreads();  // the shared arrays are used again
        }
    }
}

// A row's lists of keys into one, of its `take` best tokens, found as in a piece.
// Bound by latency: 6 us for 224 rows of 7 lists of 64.
constexpr int kMergeNT = 256;
__global__ __launch_bounds__(kMergeNT) void k_beam_merge(uint32_t rows, Beams b, uint32_t splits,
                                                         const uint64_t* __restrict__ keys, uint64_t* __restrict__ merged) {
    constexpr int kWaves = kMergeNT / 64;
    __shared__ uint64_t room[kRoom + 8];
    __shared__ uint32_t most[kMergeNT];
    __shared__ uint32_t bound;
    __shared__ int count;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint32_t stride = key_stride((uint32_t)b.beams * splits), all = splits * (uint32_t)b.take;
    const uint32_t row_stride = key_stride((uint32_t)b.beams);
    const Divide by_splits(splits);
    for (uint32_t r = blockIdx.x; r < rows; r += gridDim.x) {
        if (b.state(r) != 1) continue;
        const uint32_t item = r / (uint32_t)b.beams, k = r - item * (uint32_t)b.beams;
        const uint64_t* key = keys + (int64_t)item * stride * b.take;
        uint64_t* out = merged + (int64_t)item * row_stride * b.take;
        auto at = [&](uint32_t e) {
            const uint32_t i = by_splits(e);
            return key[key_at(i, k * splits + (e - i * splits), stride)];
        };
        uint32_t mine = 0;
#pragma unroll 4
        for (uint32_t e = threadIdx.x; e < all; e += kMergeNT) mine = max(mine, (uint32_t)(at(e) >> 32));
        most[threadIdx.x] = mine;
        if (threadIdx.x == 0) count = 0;
        __syncthreads();
        if (wave == 0) {
            uint32_t v[kWaves];
#pragma unroll
            for (int i = 0; i < kWaves; ++i) v[i] = most[i * 64 + lane];
            const uint32_t t = reached_by<0>(v, b.take);
            if (lane == 0) bound = t;
        }
        __syncthreads();
        if (mine >= bound) {
#pragma unroll 4
            for (uint32_t e = threadIdx.x; e < all; e += kMergeNT) {
                const uint64_t x = at(e);
                if ((uint32_t)(x >> 32) >= bound) {
                    const int p = atomicAdd(&count, 1);
                    if (p < kRoom) room[p] = x;
                }
            }
        }
        __syncthreads();
        const int found = count;
        if (found <= kRoom) {
            if (threadIdx.x < 8) room[found + threadIdx.x] = 0;
            __syncthreads();
            for (int i = threadIdx.x; i < found; i += kMergeNT) {
                const uint64_t x = room[i];
                const int rank = rank_of(room, found, [&](uint64_t o) { return o > x; });
                if (rank < b.take) out[key_at(rank, k, row_stride)] = x;
            }
            for (int i = found + threadIdx.x; i < b.take; i += kMergeNT) out[key_at(i, k, row_stride)] = 0;
        } else {
            uint64_t last = ~0ull;
            for (int i = 0; i < b.take; ++i) {
                uint64_t best = 0;
                for (uint32_t e = threadIdx.x; e < all; e += kMergeNT) {
                    const uint64_t x = at(e);
                    best = x < last && x > best ? x : best;
                }
                best = wave_max(best);
                __syncthreads();
                if (lane == 0) room[wave] = best;
                __syncthreads();
#pragma unroll
                for (int j = 0; j < kWaves; ++j) best = room[j] > best ? room[j] : best;
                if (threadIdx.x == 0) out[key_at(i, k, row_stride)] = best;
                last = best;
            }
        }
        __syncthreads();  // the shared arrays are used again
    }
}

// A batch item: its rows' log-sums, then its best candidates by (rank, lower
// beam; logit, lower token), found as in a piece.
struct Cand {
    uint64_t hi, lo;
    __device__ __forceinline__ bool over(const Cand& o) const { return hi > o.hi || (hi == o.hi && lo > o.lo); }
};
struct RowSum {
    double m, log_s, score, weight;
    int state;  // 0: no candidates, 1: its tokens, 2: itself
    __device__ __forceinline__ double logp(uint64_t key, double inv_t) const {
        return state == 2 ? 0.0 : ((double)key_logit(key) - m) * inv_t - log_s;
    }
};
struct SelectOut {
    float *score, *logp;
    int32_t *parent, *token;
};
// Bound by the latency of its steps, one workgroup an item: 7 to 9 us at 8 beams of 8
// pieces and 16 keys each, 13 us at 32 beams of 64.  With 512 threads, or more of a
// thread's keys or ranks in registers, small calls took 0.5 to 5 us longer.
// Keys lie by place in their lists, so that the best of all are spread over the threads.
constexpr int kJoinNT = 1024, kJoinKeep = 2;
__global__ __launch_bounds__(kJoinNT) void k_beam_join(int64_t batch, Beams b, Scale sc, int splits, int per,
                                                       const uint64_t* __restrict__ keys,
                                                       const PieceSum* __restrict__ sums, SelectOut o) {
    constexpr int kWaves = kJoinNT / 64, kGroups = kJoinNT / 4;
    __shared__ RowSum row[kMaxBeams];
    __shared__ Cand room[kRoom + 8];
    __shared__ uint32_t most[kJoinNT];
    __shared__ uint32_t bound;
    __shared__ int count;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // `per` lists of keys a beam: a list a piece, or one
    const uint32_t lists = (uint32_t)b.beams * (uint32_t)per, stride = key_stride(lists), all = stride * (uint32_t)b.take;
    const uint32_t turn = key_turn(stride);
    const Divide by_stride(stride), by_per((uint32_t)per);
    for (int64_t item = blockIdx.x; item < batch; item += gridDim.x) {
        const uint64_t* key = keys + item * all;
        uint64_t kept[kJoinKeep];
#pragma unroll
        for (int i = 0; i < kJoinKeep; ++i) {
            const uint32_t e = threadIdx.x + i * kJoinNT;
            kept[i] = e < all ? key[e] : 0;
        }
        for (int k = wave; k < b.beams; k += kWaves) {
            const int64_t r = item * b.beams + k;
            const PieceSum none{-INFINITY, 0.0};
            // read whether the row counts or not (what is there is not used then): one latency for all
            const PieceSum head = lane < splits ? sums[r * splits + lane] : none;
            const int state = b.state(r);
            RowSum a{0.0, 0.0, (double)b.score[r], b.weight ? (double)b.weight[r] : 1.0, state == 2 ? 2 : 0};
            if (state == 1) {
                double m = head.m;
                for (int p = lane + 64; p < splits; p += 64) m = fmax(m, sums[r * splits + p].m);
#pragma unroll
                for (int d = 32; d > 0; d >>= 1) m = fmax(m, __shfl_xor(m, d));
                double s = 0.0;
                for (int p = lane; p < splits; p += 64) {
                    const PieceSum q = p < 64 ? head : sums[r * splits + p];
                    s += q.m == -INFINITY ? q.s : q.s * exp((q.m - m) * sc.inv_t);
                }
                s = wave_sum(s);
                if (s > 0.0 && s < INFINITY) {
                    a.m = m;
                    a.log_s = log(s);
                    a.state = 1;
                }
            }
            if (lane == 0) row[k] = a;
        }
        if (threadIdx.x == 0) count = 0;
        __syncthreads();
        // candidate e with its key; hi is 0 where there is none
        auto cand = [&](uint32_t e, uint64_t x) {
            const uint32_t i = by_stride(e), turned = i * turn, off = turned - by_stride(turned) * stride;
            const uint32_t place = e - i * stride + (e - i * stride < off ? stride : 0u) - off;
            const uint32_t list = min(place, lists - 1), k = by_per(list);
            const RowSum a = row[k];
            // no branches: a row's values come from LDS at once
            const bool token = a.state == 1;
            const float rank = (float)((a.score + a.logp(x, sc.inv_t)) * a.weight);
            const bool some = place < lists && (token ? x != 0 : a.state == 2 && e == k * (uint32_t)per) && rank > -INFINITY;
            return Cand{some ? ((uint64_t)ordered(rank) << 32) | (uint32_t)(kMaxBeams - k) : 0, some && token ? x : 0};
        };
        auto each = [&](auto f) {
#pragma unroll
            for (int i = 0; i < kJoinKeep; ++i) {
                const uint32_t e = threadIdx.x + i * kJoinNT;
                if (e < all) f(cand(e, kept[i]));
            }
            for (uint32_t e = threadIdx.x + kJoinKeep * kJoinNT; e < all; e += kJoinNT) f(cand(e, key[e]));
        };
        auto write = [&](int i, const Cand& c) {
            const int64_t at = item * b.take + i;
            const bool none = !c.hi;
            const int k = none ? 0 : kMaxBeams - (int)(uint32_t)c.hi;
            const RowSum& a = row[k];
            const double logp = a.logp(c.lo, sc.inv_t);
            o.score[at] = none ? -INFINITY : (float)(a.score + logp);
            o.logp[at] = none ? -INFINITY : (float)logp;
            o.parent[at] = none ? -1 : (int32_t)(item * b.beams + k);
            o.token[at] = none ? -1 : a.state == 2 ? b.end_token : key_token(c.lo);
        };
        uint32_t mine = 0;
        each([&](const Cand& c) { mine = max(mine, (uint32_t)(c.hi >> 32)); });
        most[threadIdx.x] = mine;
        __syncthreads();
        if (wave == 0) {
            // maxima of four threads each, that are not neighbours
            uint32_t v[kGroups / 64];
#pragma unroll
            for (int k = 0; k < kGroups / 64; ++k) {
                v[k] = most[k * 64 + lane];
#pragma unroll
                for (int j = 1; j < 4; ++j) v[k] = max(v[k], most[j * kGroups + k * 64 + lane]);
            }
            const uint32_t t = reached_by<0>(v, b.take);
            if (lane == 0) bound = t;
        }
        __syncthreads();
        const uint32_t low = bound;
        if (mine >= low) {
            each([&](const Cand& c) {
                if ((uint32_t)(c.hi >> 32) >= low) {
                    const int p = atomicAdd(&count, 1);
                    if (p < kRoom) room[p] = c;
                }
            });
        }
        __syncthreads();
        const int found = count;
        if (found <= kRoom) {
            if (threadIdx.x < 8) room[found + threadIdx.x] = Cand{0, 0};
            __syncthreads();
            for (int i = threadIdx.x; i < found; i += kJoinNT) {
                const Cand c = room[i];
                const int rank = rank_of(room, found, [&](const Cand& o) { return o.over(c); });
                if (rank < b.take) write(rank, c);
            }
            for (int i = found + threadIdx.x; i < b.take; i += kJoinNT) write(i, Cand{0, 0});
        } else {
            Cand last{~0ull, ~0ull};
            for (int i = 0; i < b.take; ++i) {
                Cand best{0, 0};
                for (uint32_t e = threadIdx.x; e < all; e += kJoinNT) {
                    const Cand c = cand(e, key[e]);
                    if (last.over(c) && c.over(best)) best = c;
                }
#pragma unroll
                for (int d = 32; d > 0; d >>= 1) {
                    const Cand c{(uint64_t)__shfl_xor((unsigned long long)best.hi, d),
                                 (uint64_t)__shfl_xor((unsigned long long)best.lo, d)};
                    if (c.over(best)) best = c;
                }
                __syncthreads();
                if (lane == 0) room[wave] = best;
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kWaves; ++k)
                    if (room[k].over(best)) best = room[k];
                if (threadIdx.x == 0) write(i, best);
                last = best;
            }
        }
        __syncthreads();  // the shared arrays are used again
    }
}

// A piece's workgroup.  Long rows in pieces of 32 KB (256 threads of 8 vectors) where
// there are enough to fill the GPU (64 x 8 x 32000 bf16, 1024 pieces: 20.6 us, 22.8 in
// pieces of 16 KB; 32 x 4 x 200000 f32 31.4 and 36.6), else of 16 KB (4 x 8 x 131072 bf16:
// 13.8 us, 14.4 in pieces of 32; 8 x 4 x 32768 12.4 and 13.2; they meet at 360 pieces).
// Rows of at most 8 KB by single waves, 4 KB each (256 x 8 x 2000 bf16: 14.2 us, 19.4 with
// 256 threads), but where `take` is not well below a wave's lanes: their maxima would
// bound little.  Counted by the bytes of a row, not by its type's elements.
// Logits past half of the last-level cache are streamed (128 x 8 x 200000 f32: 149 us,
// 172 through the caches; bf16 94 and 102), then by 128 threads of 16 vectors, half the
// waves for the same piece (f32 137, bf16 86; on chip they fill the GPU less evenly: 64 x 8
// x 32000 bf16 21.7 us, 20.1 with 256 x 8).
constexpr int64_t kWaveRow = 8 << 10, kManyPieces = 360;
constexpr int kWaveTake = 32;
// A row's lists are merged first where an item has many keys, which its join ranks in
// f64 in one workgroup (1 x 16 x 200000 bf16, 64 of them, 13312 keys: 24.9 us, 40.7 by the
// join alone; 40 x 16 x 50000, 2048 keys, 36.7 and 33.7; they meet at 4000 to 6000).
constexpr size_t kMergedKeys = 6144;
struct SelectPlan {
    int threads, vectors;  // of a piece: 128 x 16, 256 x 8, 256 x 4, 64 x 4
    bool stream;
    int splits;
    bool merge;
    size_t off_merged, off_sums, bytes;
};
SelectPlan select_plan(int64_t batch, int64_t beams, int64_t vocab, int64_t take, int dtype) {
    const int64_t size = (int64_t)size_of(dtype), row = vocab * size, rows = batch * beams;
    SelectPlan p;
    const bool wave = row <= kWaveRow && take <= kWaveTake;
    p.threads = wave ? 64 : 256;
    p.vectors = !wave && rows * ((row + (32 << 10) - 1) / (32 << 10)) > kManyPieces ? 8 : 4;
    p.stream = p.vectors == 8 && rows * row > kStreamed;
    if (p.stream && take <= kWaveTake) {
        p.threads = 128;
        p.vectors = 16;
    }
    const int64_t chunk = (int64_t)p.threads * p.vectors * 16 / size;
    p.splits = (int)((vocab + chunk - 1) / chunk);
    const size_t items = (size_t)rows * (size_t)p.splits;
    const size_t stride = key_stride((uint32_t)(beams * p.splits));
    p.off_merged = align_up((size_t)batch * stride * (size_t)take * sizeof(uint64_t));
    p.merge = p.splits > 1 && stride * (size_t)take > kMergedKeys;
    p.off_sums = p.off_merged + (p.merge ? align_up((size_t)batch * key_stride((uint32_t)beams) * (size_t)take * sizeof(uint64_t)) : 0);
    p.bytes = p.off_sums + align_up(items * sizeof(PieceSum));
    return p;
}

// (An item's keys are 2^31 at most, and one place of padding.)
bool select_sizes_ok(int64_t batch, int64_t beams, int64_t vocab, int64_t take, int dtype) {
    return batch >= 0 && beams >= 1 && beams <= kMaxBeams && take >= 1 && take <= kMaxTake && vocab >= 1 &&
           vocab <= (1LL << 30) && batch <= 0x7fffffffLL / beams && dtype >= ISO_DT_F32 && dtype <= ISO_DT_BF16;
}

// Bound by HBM: what moved rows come from read, they written, 2344 MB in 424 to 454 us,
// 5.2 to 5.5 TB/s (a copy reaches 4.7 to 5.1).  Rows held in arrays of registers instead
// spilled from 8 rows on (835 us with scratch).
// A workgroup takes 2^`shift` columns of 16 bytes through all rows of a batch
// item: it reads what the moved rows come from, waits until all of it has come,
// and only then writes.  No other workgroup reads or writes there, so rows may
// come from each other.  What 16 bytes leave over of each block is a last
// column, taken apart: its width is the same for all.
constexpr int kReorderNT = 256, kReorderU = 8;
struct Moves {
    int32_t to[kMaxBeams], from[kMaxBeams];
    int n;
};
template <bool TAIL, int U, bool STREAM>
__device__ __forceinline__ void reorder_columns(const iso_blocks& s, char* base, const Moves& mv, int shift) {
    const uint32_t whole = (uint32_t)(s.inner / 16), cols = TAIL ? 1 : whole, all = (uint32_t)s.mid * cols;
    const int width = TAIL ? (int)(s.inner % 16) : 16;
    if (TAIL) base += (int64_t)whole * 16;
    const Divide by_cols(cols);
    for (uint32_t first = blockIdx.x << shift; first < all; first += gridDim.x << shift) {
        Quad v[U];
        char* put[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t unit = u * kReorderNT + threadIdx.x, k = unit >> shift;
            const uint32_t col = first + (unit & ((1u << shift) - 1));
            put[u] = nullptr;
            if ((int)k < mv.n && col < all) {
                const uint32_t m = TAIL ? col : by_cols(col), c = TAIL ? 0 : col - m * cols;
                char* at = base + m * s.mid_stride + (int64_t)c * 16;
                put[u] = at + mv.to[k] * s.row_stride;
                const char* got = at + mv.from[k] * s.row_stride;
                v[u] = TAIL ? load_bytes(got, width) : load_quad<STREAM>(got);
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (put[u]) TAIL ? store_bytes(put[u], width, v[u]) : store_quad<STREAM>(put[u], v[u]);
    }
}
template <bool STREAM>
__global__ __launch_bounds__(kReorderNT) void k_beam_reorder(States st, const int32_t* __restrict__ parent,
                                                             uint32_t batch, int beams, int shift) {
    __shared__ Moves mv;
    __shared__ int count[2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = 0; i < st.count; ++i) {
        const iso_blocks s = st.b[i];
        const uint32_t outer = (uint32_t)s.outer, all = (uint32_t)s.mid * (uint32_t)((s.inner + 15) / 16);
        if (blockIdx.x << (shift - 3) >= all) continue;  // no column of either kind
        for (uint32_t item = blockIdx.y; item < batch * outer; item += gridDim.y) {
            const uint32_t b = item / outer, o = item - b * outer;
            // the rows that move
            int64_t p = -1;
            if ((int)threadIdx.x < beams) p = (int64_t)parent[b * (uint32_t)beams + threadIdx.x] - (int64_t)b * beams;
            const bool moves = p >= 0 && p < beams && p != (int)threadIdx.x;
            const uint64_t mask = __ballot(moves);
            if (lane == 0 && wave < 2) count[wave] = __popcll(mask);
            __syncthreads();
            if (moves) {
                const int at = (wave ? count[0] : 0) + __popcll(mask & ((1ull << lane) - 1));
                mv.to[at] = (int32_t)threadIdx.x;
                mv.from[at] = (int32_t)p;
            }
            if (threadIdx.x == 0) mv.n = count[0] + count[1];
            __syncthreads();
            if (mv.n) {
                char* base = static_cast<char*>(s.base) + o * s.outer_stride + (int64_t)b * beams * s.row_stride;
                reorder_columns<false, kReorderU, STREAM>(s, base, mv, shift);
                if (s.inner % 16) reorder_columns<true, 1, false>(s, base, mv, shift - 3);
            }
            __syncthreads();  // the list is used again
        }
    }
}

}  // namespace
}  // namespace iso

extern "C" {

size_t iso_beam_select_workspace_bytes(int64_t batch, int64_t beams, int64_t vocab, int64_t take, int dtype) {
    if (!iso::select_sizes_ok(batch, beams, vocab, take, dtype)) return 0;
    return iso::select_plan(batch, beams, vocab, take, dtype).bytes;
}

int iso_beam_select(const void* logits, int dtype, int64_t batch, int64_t beams, int64_t vocab, int64_t ld,
                    const float* score, const float* weight, const uint8_t* ended, int32_t end_token,
                    double temperature, int64_t take, float* out_score, float* out_logp, int32_t* out_parent,
                    int32_t* out_token, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace iso;
    if (!select_sizes_ok(batch, beams, vocab, take, dtype)) return ISO_ERR_ARG;
    const int64_t rows = batch * beams;
    if (batch > (1LL << 40) / take || !logits_ok(logits, dtype, rows, vocab, ld, temperature)) return ISO_ERR_ARG;
    if (batch == 0) return ISO_OK;
    if (!logits || !score || !out_score || !out_logp || !out_parent || !out_token) return ISO_ERR_ARG;
    const size_t rb = (size_t)rows * 4, ob = (size_t)(batch * take) * 4;
    const Span out[] = {{out_score, ob}, {out_logp, ob}, {out_parent, ob}, {out_token, ob}};
    const Span in[] = {{logits, matrix_bytes(dtype, rows, vocab, ld)}, {score, rb}, {weight, rb}, {ended, (size_t)rows}};
    if (!disjoint(out, in)) return ISO_ERR_ARG;
    if (!aligned(score, 4) || !aligned(weight, 4) || !aligned(out_score, 4) || !aligned(out_logp, 4) ||
        !aligned(out_parent, 4) || !aligned(out_token, 4))
        return ISO_ERR_ARG;
    const SelectPlan pl = select_plan(batch, beams, vocab, take, dtype);
    if (!workspace || workspace_bytes < pl.bytes) return ISO_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return ISO_ERR_ARG;
    hipStream_t st = static_cast<hipStream_t>(stream);
    uint64_t* keys = static_cast<uint64_t*>(workspace);
    PieceSum* sums = reinterpret_cast<PieceSum*>(static_cast<char*>(workspace) + pl.off_sums);
    const Beams b{score, weight, ended, (int)beams, (int)take, end_token};
    const Scale sc = scale_of(temperature);
    const dim3 grid((unsigned)(rows < kMaxGrid ? rows : kMaxGrid), (unsigned)(pl.splits < 65535 ? pl.splits : 65535));
    by_dtype(dtype, [&](auto v) {
        typedef decltype(v) T;
        auto start = [&](auto nt, auto u, auto stream) {
            constexpr int NT = decltype(nt)::value, U = decltype(u)::value;
            hipLaunchKernelGGL((k_beam_pieces<T, NT, U, decltype(stream)::value>), grid, dim3(NT), 0, st,
                               static_cast<const T*>(logits), (uint32_t)rows, (int)vocab, ld, b, sc, (uint32_t)pl.splits,
                               keys, sums);
        };
        typedef std::integral_constant<int, 256> Wg;
        typedef std::integral_constant<int, 64> Wave;
        typedef std::integral_constant<int, 4> Four;
        typedef std::integral_constant<int, 8> Eight;
        typedef std::integral_constant<int, 16> Sixteen;
        typedef std::integral_constant<int, 128> Half;
        if (pl.vectors == 16) start(Half{}, Sixteen{}, std::true_type{});
        else if (pl.threads == 64) start(Wave{}, Four{}, std::false_type{});
        else if (pl.vectors == 4) start(Wg{}, Four{}, std::false_type{});
        else if (pl.stream) start(Wg{}, Eight{}, std::true_type{});
        else start(Wg{}, Eight{}, std::false_type{});
    });
    uint64_t* merged = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + pl.off_merged);
    if (pl.merge)
        hipLaunchKernelGGL(k_beam_merge, dim3((unsigned)(rows < kMaxGrid ? rows : kMaxGrid)), dim3(kMergeNT), 0, st,
                           (uint32_t)rows, b, (uint32_t)pl.splits, keys, merged);
    hipLaunchKernelGGL(k_beam_join, dim3((unsigned)(batch < kMaxGrid ? batch : kMaxGrid)), dim3(kJoinNT), 0, st, batch, b,
                       sc, pl.splits, pl.merge ? 1 : pl.splits, pl.merge ? merged : keys, sums, SelectOut{out_score, out_logp, out_parent, out_token});
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

int iso_beam_reorder(const iso_blocks* states, int count, const int32_t* parent, int64_t batch, int64_t beams,
                     void* stream) {
    using namespace iso;
    if (batch < 0 || beams < 1 || beams > kMaxBeams || batch > 0x7fffffffLL / beams) return ISO_ERR_ARG;
    const int64_t rows = batch * beams;
    const Span other[] = {{parent, (size_t)rows * 4}};
    Arrays all;
    if (!take_states(states, count, rows, other, all)) return ISO_ERR_ARG;
    if (rows && !parent) return ISO_ERR_ARG;
    if (!aligned(parent, 4)) return ISO_ERR_ARG;
    if (!all.count) return ISO_OK;
    int shift = 0;  // a workgroup's loads go over the rows first
    while (shift < 11 && (beams << (shift + 1)) <= kReorderNT * kReorderU) ++shift;
    // columns of an array's rows, rows over its outer blocks: 31 bits each
    for (int i = 0; i < all.count; ++i) {
        const iso_blocks& s = all.b[i];
        if ((s.inner + 15) / 16 > 0x7fffffffLL / s.mid || s.outer > 0x7fffffffLL / batch) return ISO_ERR_ARG;
    }
    hipStream_t hs = static_cast<hipStream_t>(stream);
    const bool stream_all = streamed(all, rows);
    all.each_launch([&](const States& st, bool) {
        int64_t tiles = 1, items = 1;
        for (int i = 0; i < st.count; ++i) {
            const iso_blocks& s = st.b[i];
            const int64_t t = ((s.mid * ((s.inner + 15) / 16) - 1) >> shift) + 1;
            tiles = t > tiles ? t : tiles;
            items = batch * s.outer > items ? batch * s.outer : items;
        }
        const dim3 grid((unsigned)(tiles < 65536 ? tiles : 65536), (unsigned)(items < 16384 ? items : 16384));
        auto start = [&](auto big) {
            hipLaunchKernelGGL(k_beam_reorder<decltype(big)::value>, grid, dim3(kReorderNT), 0, hs, st, parent,
                               (uint32_t)batch, (int)beams, shift);
        };
        if (stream_all) start(std::true_type{});
        else start(std::false_type{});
    });
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

}  // extern "C"
