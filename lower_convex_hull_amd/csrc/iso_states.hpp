// Arrays of states (iso_blocks in iso.h) as the kernels take them, their checks,
// and bytes moved between blocks of any alignment.
#pragma once

#include "../../include/iso.h"
#include "iso_losses.hpp"

#include <algorithm>

namespace iso {

// What one launch takes, as an argument of 900 bytes.
struct States {
    iso_blocks b[16];
    int count;
};
// A call's arrays, those without bytes left out, and their launches: one for every
// sixteen, and at least one.
struct Arrays {
    static constexpr int kLaunch = sizeof(States::b) / sizeof(iso_blocks);
    iso_blocks b[ISO_MAX_BLOCKS];
    int count;
    template <typename F>
    void each_launch(F f) const {
        for (int i = 0; i == 0 || i < count; i += kLaunch) {
            States st{};
            for (; st.count < kLaunch && i + st.count < count; ++st.count) st.b[st.count] = b[i + st.count];
            f(st, i == 0);
        }
    }
};

// Bytes from the first to the last of `rows` rows' blocks, 0 for none, or -1:
// counts or strides that are negative or too large, or blocks that overlap.
inline int64_t blocks_extent(const iso_blocks& b, int64_t rows) {
    if (b.outer < 0 || b.mid < 0 || b.inner < 0 || rows < 0) return -1;
    if (b.outer > 0x7fffffffLL || b.mid > 0x7fffffffLL || b.inner > (1LL << 40)) return -1;
    struct Dim {
        int64_t n, stride;
    } d[3] = {{b.outer, b.outer_stride}, {rows, b.row_stride}, {b.mid, b.mid_stride}};
    for (const Dim& x : d)
        if (x.n > 1 && x.stride < 0) return -1;
    if (!b.outer || !b.mid || !b.inner || !rows) return 0;
    // from the smallest stride on, each holds what is inside it
    for (int i = 0; i < 2; ++i)
        for (int k = 0; k < 2; ++k)
            if (d[k].stride > d[k + 1].stride) {
                const Dim t = d[k];
                d[k] = d[k + 1];
                d[k + 1] = t;
            }
    int64_t extent = b.inner;
    for (const Dim& x : d) {
        if (x.n <= 1) continue;
        int64_t far;
        if (x.stride < extent || __builtin_mul_overflow(x.stride, x.n - 1, &far) ||
            __builtin_add_overflow(far, extent, &extent))
            return -1;
    }
    return extent < (1LL << 62) ? extent : -1;
}

// The arrays of a call, those without bytes left out; false if one is not
// right, or two overlap, or one overlaps one of `other`.
template <int N>
bool take_states(const iso_blocks* from, int count, int64_t rows, const Span (&other)[N], Arrays& to) {
    if (count < 0 || count > ISO_MAX_BLOCKS || (count && !from)) return false;
    to.count = 0;
    Span at[ISO_MAX_BLOCKS];
    for (int i = 0; i < count; ++i) {
        const int64_t bytes = blocks_extent(from[i], rows);
        if (bytes < 0) return false;
        if (!bytes) continue;
        const Span s{from[i].base, (size_t)bytes};
        if (!s.p) return false;
        for (int k = 0; k < N; ++k)
            if (overlap(s, other[k])) return false;
        at[to.count] = s;
        to.b[to.count++] = from[i];
    }
    // by their first bytes: where any two overlap, two neighbours do
    std::sort(at, at + to.count, [](const Span& a, const Span& b) { return (uintptr_t)a.p < (uintptr_t)b.p; });
    for (int k = 1; k < to.count; ++k)
        if (overlap(at[k - 1], at[k])) return false;
    return true;
}

// x / n of 32 bits by a product, a sixth of a division's instructions: it is off by
// less than 2^-51 of itself, and its distance from a whole number is at least
// 0.5 / n.
struct Divide {
    double part;
    __device__ __forceinline__ explicit Divide(uint32_t n) : part(1.0 / (double)n) {}
    __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return (uint32_t)(((double)x + 0.5) * part); }
};

// 16 bytes at any address: global loads and stores need no alignment.
typedef uint32_t Quad __attribute__((ext_vector_type(4)));
typedef uint32_t Wide16 __attribute__((ext_vector_type(4), aligned(1), may_alias));
typedef uint64_t Wide8 __attribute__((aligned(1), may_alias));
typedef uint32_t Wide4 __attribute__((aligned(1), may_alias));
typedef uint16_t Wide2 __attribute__((aligned(1), may_alias));

// STREAM: without a place in the caches, for arrays that do not fit them anyway and
// are reordered or moved together as a whole: past half of the last-level cache (reordering 2.3 GB 471 -> 438 us, half of a pool of
// 2.3 GB moved together 320 -> 302; 40 MB reordered again and again 9.8 -> 11.3).
constexpr int64_t kStreamed = 128 << 20;
template <bool STREAM>
__device__ __forceinline__ Quad load_quad(const char* at) {
    const Wide16* p = reinterpret_cast<const Wide16*>(at);
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool STREAM>
__device__ __forceinline__ void store_quad(char* at, const Quad& v) {
    Wide16* p = reinterpret_cast<Wide16*>(at);
    if constexpr (STREAM) __builtin_nontemporal_store((Wide16)v, p);
    else *p = v;
}
// Whether the arrays' rows, of which there are `rows`, come to more than that.
inline bool streamed(const Arrays& st, int64_t rows) {
    double bytes = 0.0;
    for (int i = 0; i < st.count; ++i) bytes += (double)rows * st.b[i].outer * st.b[i].mid * st.b[i].inner;
    return bytes > kStreamed;
}

// The first `left` of 16 bytes, fewer than 16, as 8, 4, 2 and 1 of them.
__device__ __forceinline__ Quad load_bytes(const char* at, int left) {
    Quad v = {0, 0, 0, 0};
    if (left & 8) {
        const uint64_t x = *reinterpret_cast<const Wide8*>(at);
        v.x = (uint32_t)x;
        v.y = (uint32_t)(x >> 32);
    }
    if (left & 4) v.z = *reinterpret_cast<const Wide4*>(at + (left & 8));
    if (left & 2) v.w = *reinterpret_cast<const Wide2*>(at + (left & 12));
    if (left & 1) v.w |= (uint32_t) * reinterpret_cast<const uint8_t*>(at + (left & 14)) << 16;
    return v;
}
__device__ __forceinline__ void store_bytes(char* at, int left, const Quad& v) {
    if (left & 8) *reinterpret_cast<Wide8*>(at) = (uint64_t)v.y << 32 | v.x;
    if (left & 4) *reinterpret_cast<Wide4*>(at + (left & 8)) = v.z;
    if (left & 2) *reinterpret_cast<Wide2*>(at + (left & 12)) = (uint16_t)v.w;
    if (left & 1) *reinterpret_cast<uint8_t*>(at + (left & 14)) = (uint8_t)(v.w >> 16);
}

}  // namespace iso
