// Token log-probabilities from logits, their backward pass, and the policy loss
// taken from the logits (formulas in iso.h).  A row of logits is one token's;
// logits are f32, f16 or bf16; terms are computed in f32 from the difference to
// the maximum (exact, or nearly, in f32), and summed in f64.
#include "../../include/iso.h"
#include "iso_losses.hpp"

#include <type_traits>

namespace iso {
namespace {

constexpr double kLog2e = 1.4426950408889634;
constexpr double kLn2 = 0.6931471805599453;

// 16 bytes of logits at element alignment: logits and their gradient can have
// strides that no shift aligns both of, and global loads and stores need none.
template <typename T>
struct Wide {
    static constexpr int N = 16 / sizeof(T);
    typedef T V __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
    typedef T A __attribute__((ext_vector_type(16 / sizeof(T))));  // aligned, in LDS
};

// STREAM: without a place in the caches, for logits that do not fit them anyway
// (8192 x 65536 bf16 forward 145 -> 133 us; in workgroups of 64 threads 40000 x 2000
// f32 56.4 -> 55.5, of 512 515 x 99991 f32 48.3 -> 39.4, of 1024 200 x 200000 f32
// 30.3 -> 28.3); smaller ones may still be there from the call before (300 x 30000
// f32 backward: 12.3 us, streamed 13.8).
template <bool STREAM, typename T>
__device__ __forceinline__ typename Wide<T>::V load_wide(const T* p) {
    const auto* v = reinterpret_cast<const typename Wide<T>::V*>(p);
    if constexpr (STREAM) return __builtin_nontemporal_load(v);
    else return *v;
}

// exp((x - m)/T) = exp2((x - m) c), c = log2(e)/T.  The difference to the
// maximum m of what a sum covers comes first: it is exact, or nearly, where the
// term counts, the largest term is exactly 1, and no finite logit overflows.
struct Scale {
    double inv_t, c;
    float cf;  // c in f32
};

// The maximum that differences are taken to: 0 where everything so far is
// -infinity, so that no -infinity minus -infinity arises.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

// An exponent as a factor of the entropy's sum: a masked entry's -infinity is
// held finite, its product with exp2(-infinity) = 0 is then 0.
__device__ __forceinline__ float held(float a) { return fmaxf(a, -1e30f); }

// Part of a row: its maximum m, the sum s of e = exp2((x - m) c) and the sum h
// of e times its exponent.  m = -infinity: nothing but -infinity, sums 0.
struct Stat {
    double m, s, h;
};

// a brought to the maximum m of more: its sums scaled.
template <bool ENT>
__device__ __forceinline__ void rebase(Stat& a, double m, const Scale& sc) {
    // an infinite or NaN maximum's sums are NaN, and stay
    const float d = a.m == -INFINITY ? 0.0f : held((float)((a.m - m) * sc.c));
    const double f = (double)__builtin_amdgcn_exp2f(d);
    if (ENT) a.h = (a.h + a.s * (double)d) * f;
    a.s *= f;
    a.m = m;
}

// Every lane's statistics joined (the same in every lane): the maximum first,
// then one scaling each, then plain sums.
template <bool ENT>
__device__ __forceinline__ Stat wave_join(Stat a, const Scale& sc) {
    float m = (float)a.m;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    rebase<ENT>(a, (double)m, sc);
    a.s = wave_sum(a.s);
    if (ENT) a.h = wave_sum(a.h);
    return a;
}

// Piece number s of a row, of `chunk` elements from the first 16-byte aligned
// one on: whole vectors from..to, and the elements at the row's ends that no
// aligned vector holds, one a thread (N - 1 at each end at most).  Rows of an
// odd length begin anywhere; vectors that straddle cache lines cost 5 us of 90
// at 515 x 99991 f32.  Positions in a row are below 2^30.
template <typename T>
struct Piece {
    int head, from, to, k1;
    __device__ __forceinline__ Piece(const T* aligned_to, int s, int chunk, int vocab) {
        constexpr int N = Wide<T>::N;
        const int skew = (int)((0u - (unsigned)(uintptr_t)aligned_to) & 15u) / (int)sizeof(T);
        head = min(skew, vocab);
        from = min(head + s * chunk, vocab);
        k1 = chunk >= vocab - from ? vocab : from + chunk;
        to = from + (k1 - from) / N * N;
        if (s > 0) head = 0;
    }
    // the thread's own element, -1 if it has none
    __device__ __forceinline__ int edge() const {
        const int t = (int)threadIdx.x, k = to + t - head;
        return t < head ? t : k < k1 ? k : -1;
    }
    // element j is the thread's, of NT that take the vectors in turn from `base` on
    template <int NT>
    __device__ __forceinline__ bool mine(int j, int base) const {
        return j >= from && j < to ? (j - base) / Wide<T>::N % NT == (int)threadIdx.x : j == edge();
    }
};

// A chunk of a row: U vectors a thread of NT, those past k1 filled with
// -infinity (they add nothing).
template <typename T, int NT, int U>
struct Chunk {
    static constexpr int N = Wide<T>::N;
    static constexpr int kSize = NT * U * N;
    typename Wide<T>::V v[U];
    __device__ __forceinline__ static int at(int k, int u) { return k + u * NT * N + (int)threadIdx.x * N; }
    template <bool STREAM = false>
    __device__ __forceinline__ void load(const T* x, int k, int k1) {
        const T* b = x + k;
        if (k1 - k >= kSize) {
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = load_wide<STREAM>(b + u * NT * N + threadIdx.x * N);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < N; ++i) v[u][i] = (T)-INFINITY;
                if (at(k, u) < k1) v[u] = load_wide<STREAM>(b + u * NT * N + threadIdx.x * N);
            }
        }
    }
    // The thread's own vectors to LDS and back.
    __device__ __forceinline__ void put(typename Wide<T>::A* keep) const {
#pragma unroll
        for (int u = 0; u < U; ++u) keep[u * NT + threadIdx.x] = v[u];
    }
    __device__ __forceinline__ void take(const typename Wide<T>::A* keep) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = keep[u * NT + threadIdx.x];
    }
    // What was computed of the values so far is not kept in registers, only
    // the values: their f32 forms take twice the room and are made again.
    __device__ __forceinline__ void forget() {
        typedef int Raw __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Raw r = __builtin_bit_cast(Raw, v[u]);
            asm volatile("" : "+v"(r));
            v[u] = __builtin_bit_cast(typename Wide<T>::V, r);
        }
    }
};

// A thread's running statistics.  A chunk adds its maximum first, then its sums,
// to those so far, which are scaled when the maximum rises.  Terms are f32, their
// sum f64: where one term is nearly all, logp is what the small ones add to its
// 1, and f32 additions to 1 lost up to 2e-5 of it (3e-7 is left).  The extra
// instruction an element costs 2 % where rows stay on chip and nothing elsewhere.
// LEAN: the chunk's values are kept on (a row's gradient takes them again), and
// their f32 forms are made twice rather than held; else held (8192 x 65536 bf16:
// 127 us, 132 lean).
template <typename T, bool ENT, int NT, int U, bool LEAN>
struct Running {
    float m = -INFINITY;
    double s = 0.0, h = 0.0;
    __device__ __forceinline__ void add(Chunk<T, NT, U>& c, const Scale& sc) {
        constexpr int N = Wide<T>::N;
        float bm = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i) bm = fmaxf(bm, (float)c.v[u][i]);
        if (bm > m) {
            if (m != -INFINITY) {
                const float d = held((m - bm) * sc.cf), f = __builtin_amdgcn_exp2f(d);
                if (ENT) h = (h + s * (double)d) * (double)f;
                s *= (double)f;
            }
            m = bm;
        }
        const float base = base_of(m);
        double fs = 0.0;
        float fh = 0.0f;
        if (LEAN) c.forget();
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float a = ((float)c.v[u][i] - base) * sc.cf;
                const float e = __builtin_amdgcn_exp2f(a);
                fs += (double)e;
                if (ENT) fh = fmaf(e, held(a), fh);
            }
        s += fs;
        if (ENT) h += (double)fh;
    }
    // One more value, of those that whole vectors leave over.
    __device__ __forceinline__ void add_one(float x, const Scale& sc) {
        Stat a{(double)m, s, h};
        if (x > m) {
            rebase<ENT>(a, (double)x, sc);
            m = x;
        }
        const float d = (x - base_of(m)) * sc.cf, e = __builtin_amdgcn_exp2f(d);
        s = a.s + (double)e;
        if (ENT) h = a.h + (double)(e * held(d));
    }
    // The workgroup's, in thread 0.
    __device__ __forceinline__ Stat join(const Scale& sc, Stat* part) const {
        Stat a = wave_join<ENT>(Stat{(double)m, s, h}, sc);
        if (NT == 64) return a;
        const int lane = threadIdx.x & 63;
        if (lane == 0) part[threadIdx.x >> 6] = a;
        __syncthreads();
        if (threadIdx.x < 64) a = wave_join<ENT>(lane < NT / 64 ? part[lane] : Stat{-INFINITY, 0.0, 0.0}, sc);
        return a;
    }
};

// The statistics of a piece of a row by a workgroup of NT threads; thread 0 has them.
template <bool STREAM, typename T, bool ENT, int NT, int U>
__device__ __forceinline__ Stat row_stat(const T* __restrict__ x, const Piece<T>& w, const Scale& sc, Stat* part) {
    Running<T, ENT, NT, U, false> run;
    for (int k = w.from; k < w.to; k += Chunk<T, NT, U>::kSize) {
        Chunk<T, NT, U> c;
        c.template load<STREAM>(x, k, w.to);
        run.add(c, sc);
    }
    const int k = w.edge();
    if (k >= 0) run.add_one((float)x[k], sc);
    return run.join(sc, part);
}

// A row's log-sum and its target's log-probability from its statistics and the
// target's logit; NaN where nothing but -infinity is in the row, or (logp) the
// target is outside it.
struct RowLogp {
    double lse, logp, entropy;
};
template <typename T>
__device__ __forceinline__ RowLogp row_logp(T xj, int32_t j, int vocab, double inv_t, const Stat& a) {
    const double ls = log(a.s);
    const bool none = a.m == -INFINITY;
    return RowLogp{none ? __builtin_nan("") : a.m * inv_t + ls,
                   none || j >= vocab ? __builtin_nan("") : ((double)(float)xj - a.m) * inv_t - ls,
                   none ? __builtin_nan("") : ls - kLn2 * (a.h / a.s)};
}

// Where the forward pass's results go (ent may be NULL).
struct LogpOut {
    float *logp, *lse, *ent;
};
template <typename T>
__device__ __forceinline__ void write_row(const LogpOut& o, int64_t r, const T* x, int32_t j, int vocab,
                                          double inv_t, const Stat& a) {
    const RowLogp v = j >= 0 ? row_logp(x[j < vocab ? j : 0], j, vocab, inv_t, a) : RowLogp{0.0, 0.0, 0.0};
    o.logp[r] = (float)v.logp;
    o.lse[r] = (float)v.lse;
    if (o.ent) o.ent[r] = (float)v.entropy;
}

// Items of a grid: `count` of them, each taken by one workgroup; the grid is
// capped and its workgroups then take several.
constexpr int64_t kMaxGrid = 1 << 20;
inline dim3 grid_of(int64_t items) { return dim3((unsigned)(items < kMaxGrid ? items : kMaxGrid)); }

// Vectors of a thread at a time: 4, but 2 of streamed f32 logits.  16 bits: 8192 x
// 65536 bf16 166 us with 4, 168 with 2; 2000 x 131072 92 and 98.  f32 goes by how a
// call's rows fill the CUs: 2 is faster at 515 x 99991 (38.6 us, 42.6 with 4), 1111 x
// 50021 (39.5, 42.0) and 1500 x 99991 (95, 99), 4 at 700 x 131072 (57, 62 with 2), 2000 x
// 50021 (67, 74) and 2000 x 131072 (162, 185); from 3000 rows on they are within 2 %.
template <typename T, bool STREAM>
constexpr int kLogpU = STREAM && sizeof(T) == 4 ? 2 : 4;

// Bound by HBM: 8192 x 65536 bf16, a quarter ignored, is read at 6.1 to 6.4 TB/s
// (126 to 133 us); few rows by the launches and the latency of one read and join.
// Item = (row, part of it).  With one part a row its outputs are written, else
// the part's statistics.
template <typename T, bool ENT, int NT, bool STREAM>
__global__ __launch_bounds__(NT) void k_token_logp(const T* __restrict__ logits, int64_t rows, int vocab,
                                                   int64_t ld, const int32_t* __restrict__ target, Scale sc,
                                                   int splits, int chunk, LogpOut o, Stat* __restrict__ parts) {
    __shared__ Stat part[NT / 64];
    for (int64_t item = blockIdx.x; item < rows * splits; item += gridDim.x) {
        const int64_t r = item / splits;
        const int32_t j = target[r];
        const T* x = logits + r * ld;
        Stat a{};
        if (j >= 0) {
            a = row_stat<STREAM, T, ENT, NT, kLogpU<T, STREAM>>(x, Piece<T>(x, (int)(item - r * splits), chunk, vocab), sc, part);
        }
        if (threadIdx.x == 0) {
            if (splits == 1) write_row(o, r, x, j, vocab, sc.inv_t, a);
            else parts[item] = a;
        }
        __syncthreads();  // part is used again
    }
}

// A wave a row: the parts' statistics joined (in a fixed order), the outputs written.
constexpr int kJoinNT = 256;
template <typename T, bool ENT>
__global__ __launch_bounds__(kJoinNT) void k_token_logp_join(const T* __restrict__ logits, int64_t rows, int vocab,
                                                             int64_t ld,
                                                             const int32_t* __restrict__ target, Scale sc,
                                                             int splits, const Stat* __restrict__ parts, LogpOut o) {
    const int lane = threadIdx.x & 63;
    for (int64_t r = (int64_t)blockIdx.x * (kJoinNT / 64) + (threadIdx.x >> 6); r < rows;
         r += (int64_t)gridDim.x * (kJoinNT / 64)) {
        Stat a{-INFINITY, 0.0, 0.0};
        for (int k = lane; k < splits; k += 64) {
            Stat b = parts[r * splits + k];
            const double m = a.m > b.m ? a.m : b.m;
            rebase<ENT>(a, m, sc);
            rebase<ENT>(b, m, sc);
            a.s += b.s;
            if (ENT) a.h += b.h;
        }
        a = wave_join<ENT>(a, sc);
        if (lane == 0) write_row(o, r, logits + r * ld, target[r], vocab, sc.inv_t, a);
    }
}

// What a row's gradient takes: p = exp(x/T - lse) as exp2((x - mh) c) times a
// factor of the row, folded into a, b: gradient p (a + b y), y = (x - mh) c.  y is
// held at -200, where p is 0: a masked entry's, -infinity or huge, times b would
// be infinite, and its gradient 0 times that.  The target's entry, g (1 - p)/T and
// the entropy's part, is formed apart in f64: in f32 the difference kept nothing
// of 1 - p below 1e-7, and lost bf16's half step at 1e-5.
struct RowGrad {
    float mh, a, b;
};
// From a given log-sum: mh = lse T rounded to f32, the factor is what that
// rounding leaves off.
__device__ __forceinline__ RowGrad row_grad(double lse, double g, double ent, double g_ent, double inv_t,
                                            double temperature) {
    RowGrad o;
    o.mh = (float)(lse * temperature);
    const double off = (double)o.mh * inv_t - lse;  // x/T - lse = (x - mh)/T + off
    const double f = (double)__builtin_amdgcn_exp2f((float)(off * kLog2e)) * inv_t;
    o.a = (float)(-(g + g_ent * (ent + off)) * f);
    o.b = (float)(-g_ent * kLn2 * f);
    return o;
}
// The target's entry at the given log-sum, xj its logit.
template <bool ENT>
__device__ __forceinline__ float target_grad(double xj, double lse, double g, double ent, double g_ent, double inv_t) {
    const double z = xj * inv_t - lse;
    const ExpTerms p = ExpSeries().any(z);
    double v = -g * p.m1;
    if (ENT && p.e > 0.0) v -= g_ent * p.e * (z + ent);
    return (float)(v * inv_t);
}

// From the row's own maximum and sum: 1/sum is the factor.  A log-sum of a row
// of one huge value (a mask's lowest one) does not show log V any more.  The
// target's 1 - p is (sum - e)/sum: its term e is 1 where it is the maximum, and
// at most half of the sum elsewhere.
struct RowShare {
    float m;
    double p, rest;  // 1/sum and the target's 1 - p, over T
    __device__ __forceinline__ RowShare(const Stat& a, float xj, const Scale& sc) : m((float)a.m) {
        p = sc.inv_t / a.s;
        rest = p * (a.s - (double)__builtin_amdgcn_exp2f((xj - m) * sc.cf));
    }
    __device__ __forceinline__ RowGrad grad(double g) const { return RowGrad{m, (float)(-g * p), 0.0f}; }
    __device__ __forceinline__ float target(double g) const { return (float)(g * rest); }
};

// An element's gradient (not the target's).
template <bool ENT>
__device__ __forceinline__ float grad_one(float x, const RowGrad& q, float cf) {
    const float y = (x - q.mh) * cf;
    const float p = __builtin_amdgcn_exp2f(y);
    return ENT ? p * fmaf(q.b, fmaxf(y, -200.0f), q.a) : p * q.a;
}
// The target's place in a row and its entry.  Put into its vector before that is
// stored, or (Later) stored over it at the end by the same thread: the loss from
// logits, whose vectors wait in registers, takes 375 us that way and 378 with the
// entry put in (4096 x 131072 bf16); the backward pass 94.6 us with it put in and 97.6
// with another store (3000 x 50021 f16).
struct Target {
    int j;
    float v;
};
struct Later {};

// N elements of a row's gradient from position k on.
template <typename T, bool ENT, typename AT>
__device__ __forceinline__ typename Wide<T>::V grad_wide(const typename Wide<T>::V& x, int k, const AT& at, const RowGrad& q,
                                                         float cf) {
    constexpr int N = Wide<T>::N;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = grad_one<ENT>((float)x[i], q, cf);
    if constexpr (std::is_same<AT, Target>::value) {
        if ((unsigned)(at.j - k) < (unsigned)N) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (at.j - k == i) v[i] = at.v;
        }
    }
    typename Wide<T>::V o;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = (T)v[i];
    return o;
}

template <typename T>
__device__ __forceinline__ void store_wide(T* p, const typename Wide<T>::V& v) {
    __builtin_nontemporal_store(v, reinterpret_cast<typename Wide<T>::V*>(p));
}

// A chunk's gradient written, from position k on.
template <typename T, bool ENT, int NT, int U, typename AT>
__device__ __forceinline__ void store_grads(const Chunk<T, NT, U>& c, T* o, int k, int k1, const AT& at, const RowGrad& q,
                                            float cf) {
    typedef Chunk<T, NT, U> C;
    T* b = o + k;
    if (k1 - k >= C::kSize) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            store_wide<T>(b + u * NT * C::N + threadIdx.x * C::N, grad_wide<T, ENT>(c.v[u], C::at(k, u), at, q, cf));
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (C::at(k, u) < k1)
                store_wide<T>(b + u * NT * C::N + threadIdx.x * C::N, grad_wide<T, ENT>(c.v[u], C::at(k, u), at, q, cf));
    }
}

// A row's gradient where it is one value: 0 (ignored) or NaN.
template <typename T, int NT>
__device__ __forceinline__ void fill_row(T* o, const Piece<T>& w, T v) {
    constexpr int N = Wide<T>::N;
    typename Wide<T>::V x;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = v;
    for (int k = w.from + (int)threadIdx.x * N; k < w.to; k += NT * N) store_wide<T>(o + k, x);
    const int k = w.edge();
    if (k >= 0) o[k] = v;
}

constexpr int kVjpNT = 256, kVjpU = 2;

// Bound by HBM: 4096 x 65536 bf16 moves 0.94 GB in 151 us, 6.2 TB/s.  One chunk a
// workgroup (a second, read after the first is written, cost 7 %), of two
// vectors a thread (151 us; 1: 176, 3: 159, 4: 156, 8: 165).
// Item = (row, chunk of it).
template <typename T, bool ENT, bool STREAM>
__global__ __launch_bounds__(kVjpNT) void k_logp_vjp(const T* logits, int64_t rows, int vocab, int64_t ld,
                                                     const int32_t* __restrict__ target, double inv_t,
                                                     double temperature, float cf, int splits, int chunk,
                                                     const float* __restrict__ lse, const float* __restrict__ ent,
                                                     const float* __restrict__ g_logp,
                                                     const float* __restrict__ g_ent, T* grad, int64_t ldg) {
    for (int64_t item = blockIdx.x; item < rows * splits; item += gridDim.x) {
        const int64_t r = item / splits;
        const int32_t j = target[r];
        const T* x = logits + r * ld;
        T* o = grad + r * ldg;
        const Piece<T> w(o, (int)(item - r * splits), chunk, vocab);
        if (j < 0 || j >= vocab) {
            fill_row<T, kVjpNT>(o, w, j < 0 ? (T)0.0f : (T)__builtin_nanf(""));
            continue;
        }
        const double ls = (double)lse[r], g = (double)g_logp[r], h = ENT ? (double)ent[r] : 0.0,
                     gh = ENT ? (double)g_ent[r] : 0.0;
        Chunk<T, kVjpNT, kVjpU> c;
        if (w.from < w.to) c.template load<STREAM>(x, w.from, w.to);
        const RowGrad q = row_grad(ls, g, h, gh, inv_t, temperature);
        // by the thread that writes the entry, which may be in its logit's place
        Target at{j, 0.0f};
        if (w.template mine<kVjpNT>(j, w.from)) at.v = target_grad<ENT>((double)(float)x[j], ls, g, h, gh, inv_t);
        if (w.from < w.to) store_grads<T, ENT>(c, o, w.from, w.to, at, q, cf);
        const int edge = w.edge();
        if (edge >= 0) o[edge] = (T)(edge == j ? at.v : grad_one<ENT>((float)x[edge], q, cf));
    }
}

// The policy loss from the logits, a row of a workgroup at a time: its
// statistics, its token's terms, and its gradient.  The last chunk of the row
// stays in registers and the one before in LDS between the two; what a longer
// row has before them is read again while the last-level cache may still have
// it.  Bound by HBM: 4096 x 131072 bf16 reads each logit once (862 MB by the
// counters) and writes 1.07 GB in 375 us, 5.2 TB/s, with 60 % of the issue cycles
// spent on VALU instructions; three passes over the logits took 596.  Every
// row's weight and advantage depend on the targets alone and are known before
// (terms), or (NULL; few rows) are found here, which saves a launch.
template <typename T, int NT, int U>
__global__ __launch_bounds__(NT, 4) void k_policy_rows(const T* logits, int64_t rows, int vocab, int64_t ld,
                                                       const int32_t* __restrict__ target, Scale sc, Policy p,
                                                       const RowTerm* __restrict__ terms, Seqs sq,
                                                       float* __restrict__ logp, T* grad, int64_t ldg,
                                                       PolicySums* __restrict__ sums) {
    typedef Chunk<T, NT, U> C;
    __shared__ Stat part[NT / 64];
    __shared__ RowGrad of_row;
    __shared__ float of_target;
    __shared__ PolicySums total;  // thread 0's
    constexpr bool kKeep = NT * U >= 1024;
    __shared__ typename Wide<T>::A keep[kKeep ? NT * U : 1];
    if (threadIdx.x == 0) total = PolicySums{0.0, 0.0, 0, 0};
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int32_t j = target[r];
        const T* x = logits + r * ld;
        T* o = grad + r * ldg;
        const Piece<T> w(x, 0, vocab, vocab);  // by the logits, with or without a gradient: the same sums
        if (j < 0) {
            if (threadIdx.x == 0) logp[r] = 0.0f;
            if (grad) fill_row<T, NT>(o, w, (T)0.0f);
            continue;
        }
        const RowTerm t = terms ? terms[r] : own_row_term<NT>(p, target, sq, (uint32_t)r);
        const float old = p.old_logp[r], ref = p.ref_logp ? p.ref_logp[r] : 0.0f;
        const T xj = x[j < vocab ? j : 0];
        C c;
        Running<T, false, NT, U, true> run;
        // the first chunk is what whole chunks leave over
        const int after = w.to > w.from ? (w.to - w.from - 1) / C::kSize : 0;
        int k = w.from, e = w.to - after * C::kSize;
        do {
            c.load(x, k, e);
            run.add(c, sc);
            if (kKeep && e + C::kSize == w.to) c.put(keep);
            k = e;
            e += C::kSize;
        } while (k < w.to);
        const int edge = w.edge();
        if (edge >= 0) run.add_one((float)x[edge], sc);
        c.forget();
        const Stat a = run.join(sc, part);
        if (threadIdx.x == 0) {
            const RowShare share(a, (float)xj, sc);  // before the terms, whose chain it would lengthen
            const RowLogp v = row_logp(xj, j, vocab, sc.inv_t, a);
            const double d[1] = {v.logp - (double)old}, u[1] = {p.ref_logp ? (double)ref - v.logp : 0.0};
            const float adv[1] = {t.adv};
            PolicyTerm o1[1];
            if (p.ref_logp) policy_terms<true>(p, ExpSeries(), d, u, adv, o1);
            else policy_terms<false>(p, ExpSeries(), d, u, adv, o1);
            const PolicyTerm& k1 = o1[0];
            logp[r] = (float)v.logp;
            total.pg += t.w * k1.pg;
            total.kl += t.w * k1.kl;
            total.live += 1;
            total.over += k1.over ? 1 : 0;
            const double g = k1.slope * (t.w * p.grad_scale);
            of_row = share.grad(g);
            of_target = share.target(g);
        }
        __syncthreads();
        if (grad && j < vocab) {
            const RowGrad q = of_row;
            if (edge >= 0) o[edge] = (T)grad_one<false>((float)x[edge], q, sc.cf);
            // the last chunk is still in registers, the others follow backwards
            for (e = w.to;;) {
                k = max(e - C::kSize, w.from);
                store_grads<T, false>(c, o, k, e, Later{}, q, sc.cf);
                if (k == w.from) break;
                e = k;
                if (kKeep && e + C::kSize == w.to) c.take(keep);
                else c.load(x, max(e - C::kSize, w.from), e);
            }
            const int whole = w.to - after * C::kSize;  // where whole chunks begin
            if (w.template mine<NT>(j, j < whole ? w.from : whole)) o[j] = (T)of_target;
        } else if (grad) {
            fill_row<T, NT>(o, w, (T)__builtin_nanf(""));
        }
        __syncthreads();  // part and of_row are used again
    }
    if (threadIdx.x == 0) sums[blockIdx.x] = total;
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

size_t size_of(int dtype) { return dtype == ISO_DT_F32 ? 4 : 2; }

// log2(e)/T and lse T (up to 21 T past the largest logit) stay inside f32.
constexpr double kTempMin = 1e-28, kTempMax = 1e28;

bool logits_ok(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld, double temperature) {
    if (dtype != ISO_DT_F32 && dtype != ISO_DT_F16 && dtype != ISO_DT_BF16) return false;
    if (rows < 0 || rows > 0x7fffffffLL || vocab < 1 || vocab > (1LL << 30) || ld < vocab) return false;
    if (rows && ld > INT64_MAX / 16 / rows) return false;
    if (!(temperature >= kTempMin && temperature <= kTempMax)) return false;
    return aligned(logits, size_of(dtype));
}

// Bytes from the first to the last element of `rows` rows.
size_t matrix_bytes(int dtype, int64_t rows, int64_t vocab, int64_t ld) {
    return rows ? ((size_t)(rows - 1) * (size_t)ld + (size_t)vocab) * size_of(dtype) : 0;
}

// grad is apart from the logits, or is the logits.
bool grad_ok(const void* logits, void* grad, int dtype, int64_t rows, int64_t vocab, int64_t ld, int64_t ldg) {
    if (ldg < vocab || (rows && ldg > INT64_MAX / 16 / rows) || !aligned(grad, size_of(dtype))) return false;
    if (grad == logits) return ld == ldg || rows <= 1;
    return !overlap({grad, matrix_bytes(dtype, rows, vocab, ldg)}, {logits, matrix_bytes(dtype, rows, vocab, ld)});
}

// How a row is split over workgroups, and how many threads take a piece.
// Few rows of many bytes are split (1 x 131072 bf16: 10.4 us whole, 6.2 in
// pieces of 16 KB; 96 x 131072 f16 14.4 and 12.5), others not: the pieces are
// joined by a second launch (1 x 32768 bf16: 4.9 us whole, 6.1 split; 256 x
// 131072 14.9 and 17.8, 150 x 65536 7.7 and 10.6).  Threads are as many as one chunk of the piece takes
// (900 x 4000 bf16: 5.1 us with 64, 6.6 with 256, 20.6 with 1024), at most 256 where there
// are workgroups enough to fill the GPU without.
struct LogpPlan {
    int splits, threads;
    int64_t chunk;
    size_t bytes;
};
constexpr int64_t kFewRows = 128, kWholeRow = 96 << 10;  // split below / above
constexpr int64_t kPart = 16 << 10, kPartsMax = 2048;     // bytes of a piece, pieces wanted at most
constexpr int64_t kFullPieces = 256, kManyPieces = 640;  // more than a CU's share of one, of two pieces
LogpPlan logp_plan(int64_t rows, int64_t vocab, int dtype) {
    const int64_t size = (int64_t)size_of(dtype), step = kPart / size;
    int64_t chunk = vocab;
    if (rows && rows < kFewRows && vocab * size > kWholeRow) {
        const int64_t most = kPartsMax / rows;
        const int64_t parts = (vocab + step - 1) / step;
        chunk = (parts + most - 1) / most * step;
    }
    const int64_t splits = (vocab + chunk - 1) / chunk, bytes = chunk * size;
    LogpPlan p;
    p.splits = (int)splits;
    p.chunk = chunk;
    const int64_t pieces = rows * splits;
    p.threads = bytes <= 8 << 10                             ? 64
                : bytes <= 16 << 10 || pieces > kManyPieces ? 256
                : bytes <= 32 << 10 || pieces > kFullPieces ? 512
                                                            : 1024;
    p.bytes = splits > 1 ? (size_t)rows * (size_t)splits * sizeof(Stat) : 0;
    return p;
}

// Logits past half of the last-level cache (256 MB).
template <typename T>
bool streamed(int64_t rows, int64_t vocab) { return rows * vocab * (int64_t)sizeof(T) > 128 << 20; }

Scale scale_of(double temperature) {
    const double c = kLog2e / temperature;
    return Scale{1.0 / temperature, c, (float)c};
}

template <typename T, bool ENT>
void start_logp_t(const T* x, int64_t rows, int64_t vocab, int64_t ld, const int32_t* target, double temperature,
                  const LogpOut& o, const LogpPlan& pl, void* workspace, hipStream_t st) {
    const Scale sc = scale_of(temperature);
    Stat* parts = static_cast<Stat*>(workspace);
    auto start = [&](auto nt, auto stream) {
        constexpr int NT = decltype(nt)::value;
        hipLaunchKernelGGL((k_token_logp<T, ENT, NT, decltype(stream)::value>), grid_of(rows * pl.splits), dim3(NT), 0, st, x, rows, (int)vocab,
                           ld, target, sc, pl.splits, (int)pl.chunk, o, parts);
    };
    auto by_threads = [&](auto stream) {
        if (pl.threads == 64) start(std::integral_constant<int, 64>{}, stream);
        else if (pl.threads == 256) start(std::integral_constant<int, 256>{}, stream);
        else if (pl.threads == 512) start(std::integral_constant<int, 512>{}, stream);
        else start(std::integral_constant<int, 1024>{}, stream);
    };
    if (streamed<T>(rows, vocab)) by_threads(std::true_type{});
    else by_threads(std::false_type{});
    if (pl.splits > 1)
        hipLaunchKernelGGL((k_token_logp_join<T, ENT>), grid_of((rows + kJoinNT / 64 - 1) / (kJoinNT / 64)),
                           dim3(kJoinNT), 0, st, x, rows, (int)vocab, ld, target, sc, pl.splits, parts, o);
}

template <typename T>
void start_logp(const void* logits, int64_t rows, int64_t vocab, int64_t ld, const int32_t* target,
                double temperature, const LogpOut& o, const LogpPlan& pl, void* workspace, hipStream_t st) {
    const T* x = static_cast<const T*>(logits);
    if (o.ent) start_logp_t<T, true>(x, rows, vocab, ld, target, temperature, o, pl, workspace, st);
    else start_logp_t<T, false>(x, rows, vocab, ld, target, temperature, o, pl, workspace, st);
}

template <typename T>
void start_vjp(const void* logits, int64_t rows, int64_t vocab, int64_t ld, const int32_t* target,
               double temperature, const float* lse, const float* ent, const float* g_logp, const float* g_ent,
               void* grad, int64_t ldg, hipStream_t st) {
    const Scale sc = scale_of(temperature);
    const T* x = static_cast<const T*>(logits);
    T* o = static_cast<T*>(grad);
    const int chunk = kVjpU * kVjpNT * Wide<T>::N;
    const int splits = (int)((vocab + chunk - 1) / chunk);
    const dim3 grid = grid_of(rows * splits), nt(kVjpNT);
    auto start = [&](auto ent_on, auto stream) {
        hipLaunchKernelGGL((k_logp_vjp<T, decltype(ent_on)::value, decltype(stream)::value>), grid, nt, 0, st, x, rows,
                           (int)vocab, ld, target, sc.inv_t, temperature, sc.cf, splits, chunk, lse, ent, g_logp,
                           g_ent, o, ldg);
    };
    auto by_ent = [&](auto stream) {
        if (g_ent) start(std::true_type{}, stream);
        else start(std::false_type{}, stream);
    };
    if (streamed<T>(rows, vocab)) by_ent(std::true_type{});
    else by_ent(std::false_type{});
}

// f called with a value of the logits' type.
template <typename F>
void by_dtype(int dtype, F f) {
    if (dtype == ISO_DT_F32) f(float{});
    else if (dtype == ISO_DT_F16) f(_Float16{});
    else f(__bf16{});
}

// Workspace and grid of iso_policy_loss_logits.
constexpr int64_t kHeadGrid = 8192;
constexpr int64_t kOwnTerms = 256;  // rows and sequences up to which a row's workgroup finds its term itself
// A row's workgroup, by the bytes of a row.  A workgroup holds two chunks on
// chip (registers and LDS); the fewer threads it has, the more rows a CU has in
// flight, one reading while another writes.
//   1024 x 8 vectors (2 x 128 KB, one row a CU): 4096 x 131072 bf16, a fifth of the rows
//     ignored, 375 us, 385 with 512; 256 x 131072 33 and 38; 2000 x 65536 f32 204 and 213
//   512 x 8 (2 x 64 KB, two rows): 3000 x 101574 f16 253 us, 288 with 1024, 286 with 256;
//     2000 x 118000 bf16 206 and 217
//     Where they meet goes by more than the bytes, from 160 to 340 KB: f32 is faster
//     with 1024 below the border (2000 x 58001, 227 KB: 199 us, 212 with 512), 16 bits with
//     512 above it where no row is ignored (4096 x 131072, 256 KB: 417 us, 436 with 1024; at
//     2000 x 170003, 332 KB, 312 and 305).
//   256 x 8 (2 x 32 KB, four rows), many rows: 2000 x 25000 bf16 51 us, 57 with 512
//     (37 x 32003 f16: 14.7 us, 12.9 with 512)
//   256 x 4 (2 x 16 KB): 4096 x 16384 bf16 61 us, 72 with 512 x 8
//   64 x 4: 4000 x 1500 bf16 19 us, 30 with 256 x 4
constexpr int64_t kHeadWide = 232 << 10, kHeadFull = 96 << 10, kHeadMid = 40 << 10, kHeadNarrow = 8 << 10;
constexpr int64_t kHeadRows = 512;  // many rows: two a CU
struct HeadPlan {
    int grid;
    size_t off_terms, off_sums, off_weights, bytes;
};
HeadPlan head_plan(int64_t rows, int64_t seqs) {
    HeadPlan p;
    p.grid = (int)(rows < kHeadGrid ? rows : kHeadGrid);
    p.off_terms = 0;
    p.off_sums = align_up((size_t)rows * sizeof(RowTerm));
    p.off_weights = p.off_sums + align_up((size_t)p.grid * sizeof(PolicySums));
    p.bytes = p.off_weights + row_terms_workspace(rows, seqs);
    return p;
}

template <typename T>
void start_rows(const void* logits, int64_t rows, int64_t vocab, int64_t ld, const int32_t* target,
                double temperature, const Policy& p, const RowTerm* terms, const Seqs& sq, float* logp, void* grad, int64_t ldg,
                PolicySums* sums, int grid, hipStream_t st) {
    const T* x = static_cast<const T*>(logits);
    T* o = static_cast<T*>(grad);
    const Scale sc = scale_of(temperature);
    const int64_t bytes = vocab * (int64_t)sizeof(T);
    auto start = [&](auto nt, auto u) {
        constexpr int NT = decltype(nt)::value, U = decltype(u)::value;
        hipLaunchKernelGGL((k_policy_rows<T, NT, U>), dim3(grid), dim3(NT), 0, st, x, rows, (int)vocab, ld, target, sc, p,
                           terms, sq, logp, o, ldg, sums);
    };
    typedef std::integral_constant<int, 4> Four;
    typedef std::integral_constant<int, 8> Eight;
    if (bytes > kHeadWide) start(std::integral_constant<int, 1024>{}, Eight{});
    else if (bytes > kHeadFull || (bytes > kHeadMid && rows <= kHeadRows)) start(std::integral_constant<int, 512>{}, Eight{});
    else if (bytes > kHeadMid) start(std::integral_constant<int, 256>{}, Eight{});
    else if (bytes > kHeadNarrow) start(std::integral_constant<int, 256>{}, Four{});
    else start(std::integral_constant<int, 64>{}, Four{});
}

}  // namespace
}  // namespace iso

extern "C" {

size_t iso_token_logp_workspace_bytes(int64_t rows, int64_t vocab, int dtype) {
    if (rows < 0 || rows > 0x7fffffffLL || vocab < 1 || vocab > (1LL << 30) || dtype < ISO_DT_F32 || dtype > ISO_DT_BF16)
        return 0;
    return iso::logp_plan(rows, vocab, dtype).bytes;
}

int iso_token_logp(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld, const int32_t* target,
                   double temperature, float* logp, float* lse, float* entropy, void* workspace,
                   size_t workspace_bytes, void* stream) {
    using namespace iso;
    if (!logits_ok(logits, dtype, rows, vocab, ld, temperature)) return ISO_ERR_ARG;
    if (rows == 0) return ISO_OK;
    if (!logits || !target || !logp || !lse) return ISO_ERR_ARG;
    const size_t rb = (size_t)rows * 4;
    const Span out[] = {{logp, rb}, {lse, rb}, {entropy, rb}};
    const Span in[] = {{logits, matrix_bytes(dtype, rows, vocab, ld)}, {target, rb}};
    if (!disjoint(out, in)) return ISO_ERR_ARG;
    if (!aligned(target, 4) || !aligned(logp, 4) || !aligned(lse, 4) || !aligned(entropy, 4)) return ISO_ERR_ARG;
    const size_t need = iso_token_logp_workspace_bytes(rows, vocab, dtype);
    if (need && (!workspace || workspace_bytes < need)) return ISO_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return ISO_ERR_ARG;
    hipStream_t st = static_cast<hipStream_t>(stream);
    by_dtype(dtype, [&](auto v) {
        start_logp<decltype(v)>(logits, rows, vocab, ld, target, temperature, {logp, lse, entropy},
                                logp_plan(rows, vocab, dtype), workspace, st);
    });
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

int iso_token_logp_vjp(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                       const int32_t* target, double temperature, const float* lse, const float* entropy,
                       const float* g_logp, const float* g_entropy, void* grad, int64_t ld_grad, void* stream) {
    using namespace iso;
    if (!logits_ok(logits, dtype, rows, vocab, ld, temperature)) return ISO_ERR_ARG;
    if (rows == 0) return ISO_OK;
    if (!logits || !target || !lse || !g_logp || !grad || (g_entropy && !entropy)) return ISO_ERR_ARG;
    if (!grad_ok(logits, grad, dtype, rows, vocab, ld, ld_grad)) return ISO_ERR_ARG;
    const size_t rb = (size_t)rows * 4;
    const Span out[] = {{grad, matrix_bytes(dtype, rows, vocab, ld_grad)}};
    const Span in[] = {{target, rb}, {lse, rb}, {entropy, rb}, {g_logp, rb}, {g_entropy, rb}};
    if (!disjoint(out, in)) return ISO_ERR_ARG;
    if (!aligned(target, 4) || !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(g_logp, 4) ||
        !aligned(g_entropy, 4))
        return ISO_ERR_ARG;
    by_dtype(dtype, [&](auto v) {
        start_vjp<decltype(v)>(logits, rows, vocab, ld, target, temperature, lse, entropy, g_logp, g_entropy, grad,
                               ld_grad, static_cast<hipStream_t>(stream));
    });
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

size_t iso_policy_loss_logits_workspace_bytes(int64_t rows, int64_t vocab, int64_t seqs, int dtype) {
    if (rows < 0 || rows > 0x7fffffffLL || vocab < 1 || vocab > (1LL << 30) || seqs < 0 || seqs > 0x7fffffffLL ||
        dtype < ISO_DT_F32 || dtype > ISO_DT_BF16)
        return 0;
    return iso::head_plan(rows, seqs).bytes;
}

int iso_policy_loss_logits(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                           const int32_t* target, double temperature, const float* old_logp,
                           const float* ref_logp, const float* adv, const int32_t* seq_off, int64_t seqs,
                           double clip_lo, double clip_hi, double kl_coef, double norm, float* loss,
                           int32_t* counts, float* logp, void* grad, int64_t ld_grad, double grad_scale,
                           void* workspace, size_t workspace_bytes, void* stream, uint32_t flags) {
    using namespace iso;
    if (!logits_ok(logits, dtype, rows, vocab, ld, temperature)) return ISO_ERR_ARG;
    if (!policy_args_ok(old_logp, ref_logp, adv, seq_off, seqs, rows, clip_lo, clip_hi, kl_coef, norm, grad_scale,
                        flags))
        return ISO_ERR_ARG;
    if (!loss || !counts || (rows && (!logits || !target || !logp))) return ISO_ERR_ARG;
    if (grad && !grad_ok(logits, grad, dtype, rows, vocab, ld, ld_grad)) return ISO_ERR_ARG;
    const size_t rb = (size_t)rows * 4;
    const size_t ab = (flags & ISO_POLICY_ADV_TOKEN) ? rb : (size_t)seqs * 4;
    const Span out[] = {{loss, 12}, {counts, 8}, {logp, rb}, {grad, grad ? matrix_bytes(dtype, rows, vocab, ld_grad) : 0}};
    const Span in[] = {{target, rb}, {old_logp, rb}, {ref_logp, rb}, {adv, ab}, {seq_off, (size_t)(seqs + 1) * 4}};
    if (!disjoint(out, in)) return ISO_ERR_ARG;
    const Span lg{logits, matrix_bytes(dtype, rows, vocab, ld)};
    if (overlap(lg, out[0]) || overlap(lg, out[1]) || overlap(lg, out[2])) return ISO_ERR_ARG;
    if (!aligned(target, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(logp, 4)) return ISO_ERR_ARG;
    const HeadPlan pl = head_plan(rows, seqs);
    if (!workspace || workspace_bytes < pl.bytes) return ISO_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return ISO_ERR_ARG;
    hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    RowTerm* terms = reinterpret_cast<RowTerm*>(ws + pl.off_terms);
    PolicySums* sums = reinterpret_cast<PolicySums*>(ws + pl.off_sums);
    const Policy p = make_policy(old_logp, ref_logp, adv, clip_lo, clip_hi, kl_coef, norm, grad_scale, flags);
    if (rows) {
        const Seqs sq = make_seqs(seq_off, seqs, rows);
        const bool own = rows <= kOwnTerms && seqs <= kOwnTerms;
        if (!own && launch_row_terms(p, target, sq, terms, ws + pl.off_weights, st) != hipSuccess) return ISO_ERR_HIP;
        by_dtype(dtype, [&](auto v) {
            start_rows<decltype(v)>(logits, rows, vocab, ld, target, temperature, p, own ? nullptr : terms, sq, logp, grad,
                                    ld_grad, sums, pl.grid, st);
        });
    }
    return launch_policy_out(p, sums, pl.grid, loss, counts, st) == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

}  // extern "C"
