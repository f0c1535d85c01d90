// What the kernels over rows of logits (iso_logp.hip, iso_beams.hip) share: wide
// loads, pieces of a row, the softmax's scale, and their argument checks.
#pragma once

#include "../../include/iso.h"
#include "iso_losses.hpp"

namespace iso {

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

inline size_t size_of(int dtype) { return dtype == ISO_DT_F32 ? 4 : 2; }

// log2(e)/T and lse T (up to 21 T past the largest logit) stay inside f32.
constexpr double kTempMin = 1e-28, kTempMax = 1e28;

inline bool logits_ok(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld, double temperature) {
    if (dtype != ISO_DT_F32 && dtype != ISO_DT_F16 && dtype != ISO_DT_BF16) return false;
    if (rows < 0 || rows > 0x7fffffffLL || vocab < 1 || vocab > (1LL << 30) || ld < vocab) return false;
    if (rows && ld > INT64_MAX / 16 / rows) return false;
    if (!(temperature >= kTempMin && temperature <= kTempMax)) return false;
    return aligned(logits, size_of(dtype));
}

// Bytes from the first to the last element of `rows` rows.
inline size_t matrix_bytes(int dtype, int64_t rows, int64_t vocab, int64_t ld) {
    return rows ? ((size_t)(rows - 1) * (size_t)ld + (size_t)vocab) * size_of(dtype) : 0;
}

// Logits past half of the last-level cache (256 MB).
template <typename T>
bool streamed(int64_t rows, int64_t vocab) { return rows * vocab * (int64_t)sizeof(T) > 128 << 20; }

inline Scale scale_of(double temperature) {
    const double c = kLog2e / temperature;
    return Scale{1.0 / temperature, c, (float)c};
}

// f called with a value of the logits' type.
template <typename F>
void by_dtype(int dtype, F f) {
    if (dtype == ISO_DT_F32) f(float{});
    else if (dtype == ISO_DT_F16) f(_Float16{});
    else f(__bf16{});
}

}  // namespace iso
