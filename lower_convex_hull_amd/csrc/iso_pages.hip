// Pages of a cache: a step in which sequences are forked, grown, begun and
// freed, and the live pages moved together (definitions in iso.h).
#include "iso_states.hpp"

namespace iso {
namespace {

inline size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

constexpr int kNT = 256, kWaves = kNT / 64;
constexpr int64_t kMaxSeqs = 1 << 20;

// Exclusive prefix of v over the workgroup, and its total.
__device__ __forceinline__ int wg_prefix(int v, int* red, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    IntSumStep s{v};
    wave_scan(s);
    if (lane == 63) red[wave] = s.v;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
        before += k < wave ? red[k] : 0;
        total += red[k];
    }
    __syncthreads();
    return before + s.v - v;
}

// Sums of the first `upto` and of all n values (below 2^63), by the workgroup.
struct Prefix {
    int64_t before, total;
};
__device__ __forceinline__ int64_t wg_sum64(int64_t v, int64_t* red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += (int64_t)__shfl_xor((long long)v, d);
    if (lane == 0) red[wave] = v;
    __syncthreads();
    int64_t s = 0;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) s += red[k];
    __syncthreads();
    return s;
}
template <typename T>
__device__ __forceinline__ Prefix prefix_of(const T* v, int64_t n, int64_t upto, int64_t* red) {
    int64_t a = 0, t = 0;
    for (int64_t i = threadIdx.x; i < n; i += kNT) {
        const int64_t x = v[i];
        t += x;
        a += i < upto ? x : 0;
    }
    return Prefix{wg_sum64(a, red), wg_sum64(t, red)};
}

// Pages are taken in blocks, one a workgroup, children in blocks of kNT.
struct Blocks {
    int64_t pages, per;  // pages in all, in a block
    int64_t count;
};
constexpr int64_t kPageBlock = 2048, kPageBlocks = 1024;
Blocks page_blocks(int64_t pages) {
    Blocks b{pages, kPageBlock, 0};
    if (pages > kPageBlock * kPageBlocks) b.per = ((pages + kPageBlocks - 1) / kPageBlocks + kNT - 1) / kNT * kNT;
    b.count = (pages + b.per - 1) / b.per;
    return b;
}

// What growing children do with the page that their parent's tokens end in.
struct Mark {
    int32_t writers, first;
};
struct Copy {
    int32_t from, to, tokens, pad;
};

struct Fork {
    const int32_t *table, *length, *refs, *parent, *grow;
    int32_t grow_all;
    int64_t seqs, max_pages, pages, page_size, children;
    int32_t *new_table, *new_length, *new_refs, *status;
    // workspace
    Mark* mark;         // [pages]
    int32_t* kids;      // [seqs]
    int32_t* list;      // [pages] the pages taken, in order
    int32_t* need;      // [children] pages a child takes
    int64_t* start;     // [children] places in the list before its own
    int64_t* need_sum;  // [blocks of children]
    int32_t* copy_sum;  // [blocks of children]
    int32_t* long_sum;  // [blocks of children]
    int32_t* free_sum;  // [blocks of pages]
    Copy* copies;       // [children]
    int32_t* plan;      // [2]: done or not, copies
    bool counts_left;   // k_fork_write takes the copied pages' counts down

    __device__ __forceinline__ int64_t tokens_of(int64_t s) const {
        const int64_t n = length[s], most = max_pages * page_size;
        return n < 0 ? 0 : n < most ? n : most;
    }
    __device__ __forceinline__ int64_t pages_for(int64_t n) const { return (n + page_size - 1) / page_size; }
    __device__ __forceinline__ bool is_page(int32_t q) const { return q >= 0 && q < pages; }
    __device__ __forceinline__ int64_t grown(int64_t i) const {
        const int32_t g = grow ? grow[i] : grow_all;
        return g > 0 ? g : 0;
    }
};
struct Child {
    int64_t parent;  // -1: none
    int64_t before, after;  // tokens
    int32_t edge;           // the page it goes on to write, -1: none
};
__device__ __forceinline__ Child child_of(const Fork& f, int64_t i) {
    Child c;
    const int64_t p = f.parent[i], g = f.grown(i);
    c.parent = p >= 0 && p < f.seqs ? p : -1;
    c.before = c.parent >= 0 ? f.tokens_of(c.parent) : 0;
    c.after = c.before + g;
    c.edge = -1;
    if (g > 0 && c.before % f.page_size) {
        const int32_t q = f.table[c.parent * f.max_pages + c.before / f.page_size];
        if (f.is_page(q)) c.edge = q;
    }
    return c;
}

__global__ __launch_bounds__(kNT) void k_fork_begin(Fork f) {
    const int64_t t = (int64_t)blockIdx.x * kNT + threadIdx.x, step = (int64_t)gridDim.x * kNT;
    for (int64_t p = t; p < f.pages; p += step) {
        const int32_t n = f.refs[p];
        f.new_refs[p] = n > 0 ? n : 0;
        f.mark[p] = Mark{0, INT32_MAX};
    }
    for (int64_t s = t; s < f.seqs; s += step) f.kids[s] = 0;
}

__global__ __launch_bounds__(kNT) void k_fork_count(Fork f) {
    for (int64_t i = (int64_t)blockIdx.x * kNT + threadIdx.x; i < f.children; i += (int64_t)gridDim.x * kNT) {
        const Child c = child_of(f, i);
        if (c.parent >= 0) atomicAdd(&f.kids[c.parent], 1);
        if (c.edge >= 0) {
            atomicAdd(&f.mark[c.edge].writers, 1);
            atomicMin(&f.mark[c.edge].first, (int32_t)i);
        }
    }
}

// A sequence's pages have a holder less for it and one more for each child.
__global__ __launch_bounds__(kNT) void k_fork_refs(Fork f) {
    for (int64_t s = blockIdx.x; s < f.seqs; s += gridDim.x) {
        const int32_t more = f.kids[s] - 1;
        if (!more) continue;
        const int64_t held = f.pages_for(f.tokens_of(s));
        for (int64_t j = threadIdx.x; j < held; j += kNT) {
            const int32_t q = f.table[s * f.max_pages + j];
            if (f.is_page(q)) atomicAdd(&f.new_refs[q], more);
        }
    }
}

// Blocks of children: the pages each takes.  Blocks of pages: the free ones.
__global__ __launch_bounds__(kNT) void k_fork_need(Fork f, Blocks pb, int64_t child_blocks) {
    __shared__ int64_t red[kWaves];
    for (int64_t b = blockIdx.x; b < child_blocks + pb.count; b += gridDim.x) {
        if (b < child_blocks) {
            const int64_t i = b * kNT + threadIdx.x;
            int64_t need = 0;
            int copies = 0, too_long = 0;
            if (i < f.children) {
                const Child c = child_of(f, i);
                const int64_t want = f.pages_for(c.after);
                if (c.edge >= 0) {
                    const Mark m = f.mark[c.edge];
                    copies = !(f.new_refs[c.edge] == m.writers && m.first == i);
                }
                too_long = want > f.max_pages || c.after > INT32_MAX;
                need = too_long ? 0 : want - f.pages_for(c.before) + copies;
                f.need[i] = (int32_t)need | (copies << 31);
            }
            need = wg_sum64(need, red);
            const int64_t both = wg_sum64(((int64_t)too_long << 32) | copies, red);
            if (threadIdx.x == 0) {
                f.need_sum[b] = need;
                f.copy_sum[b] = (int32_t)both;
                f.long_sum[b] = (int32_t)(both >> 32);
            }
        } else {
            const int64_t k = b - child_blocks, to = (k + 1) * pb.per < f.pages ? (k + 1) * pb.per : f.pages;
            int64_t n = 0;
            for (int64_t p = k * pb.per + threadIdx.x; p < to; p += kNT) n += f.new_refs[p] <= 0;
            n = wg_sum64(n, red);
            if (threadIdx.x == 0) f.free_sum[k] = (int32_t)n;
        }
    }
}

// Blocks of children: where each one's pages begin in the list, and the copies.
// Blocks of pages: the list of the free ones, as many as are taken.
__global__ __launch_bounds__(kNT) void k_fork_list(Fork f, Blocks pb, int64_t child_blocks) {
    __shared__ int64_t red64[kWaves];
    __shared__ int red[kWaves];
    const int64_t need = prefix_of(f.need_sum, child_blocks, 0, red64).total;
    const int64_t room = prefix_of(f.free_sum, pb.count, 0, red64).total;
    const int64_t late = prefix_of(f.long_sum, child_blocks, 0, red64).total;
    const int64_t copied = prefix_of(f.copy_sum, child_blocks, 0, red64).total;
    const bool done = need <= room && !late;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        const int64_t lack = need - room;
        f.status[0] = lack <= 0 ? 0 : lack < INT32_MAX ? (int32_t)lack : INT32_MAX;
        f.status[1] = (int32_t)late;
        f.status[2] = f.plan[1] = done ? (int32_t)copied : 0;
        f.status[3] = done ? (int32_t)need : 0;
        f.status[4] = done ? (int32_t)(room - need) : 0;
        f.plan[0] = done;
    }
    for (int64_t b = blockIdx.x; b < child_blocks + pb.count; b += gridDim.x) {
        if (b < child_blocks) {
            const int64_t need_before = prefix_of(f.need_sum, child_blocks, b, red64).before;
            const int64_t copies_before = prefix_of(f.copy_sum, child_blocks, b, red64).before;
            const int64_t i = b * kNT + threadIdx.x;
            const int32_t n = i < f.children ? f.need[i] : 0;
            const int own = n & INT32_MAX, copy = (uint32_t)n >> 31;
            int sum;
            // a block's needs can pass 2^31 only where nothing is done
            const int at = wg_prefix(own, red, sum);
            const int64_t start = need_before + at;
            const int64_t place = copies_before + wg_prefix(copy, red, sum);
            if (i < f.children) f.start[i] = start;
            if (copy && done) {
                const Child c = child_of(f, i);
                f.copies[place] = Copy{c.edge, (int32_t)start, (int32_t)(c.before % f.page_size), 0};
            }
        } else {
            const int64_t k = b - child_blocks, to = (k + 1) * pb.per < f.pages ? (k + 1) * pb.per : f.pages;
            int64_t rank = prefix_of(f.free_sum, pb.count, k, red64).before;
            for (int64_t p0 = k * pb.per; p0 < to; p0 += kNT) {
                const int64_t p = p0 + threadIdx.x;
                if (!done) {  // the counts as they were
                    if (p < to) f.new_refs[p] = f.refs[p] > 0 ? f.refs[p] : 0;
                    continue;
                }
                const bool open = p < to && f.new_refs[p] <= 0;
                int sum;
                const int64_t at = rank + wg_prefix(open, red, sum);
                if (open) {
                    f.new_refs[p] = at < need;
                    if (at < need) f.list[at] = (int32_t)p;
                }
                rank += sum;
            }
        }
    }
}

// 16-byte columns of what one block of an array holds, `bytes` of each of its mid
// runs, by the workgroup: kCopyU of them a thread are on their way at a time.
constexpr int kCopyU = 8;
struct CopyTile {
    uint32_t cols, all;  // columns of a run, of all of them
    __device__ __forceinline__ CopyTile(const iso_blocks& s, int64_t bytes)
        : cols((uint32_t)((bytes + 15) / 16)), all((uint32_t)s.mid * cols) {}
    __device__ __forceinline__ uint32_t tiles() const { return (all + kNT * kCopyU - 1) / (kNT * kCopyU); }
};
__device__ __forceinline__ void copy_tile(const iso_blocks& s, const CopyTile& c, int64_t bytes, const char* from, char* to,
                                          uint32_t tile) {
    const Divide by_cols(c.cols);
    const int rest = (int)(bytes - (int64_t)(c.cols - 1) * 16);
    Quad v[kCopyU];
    int64_t at[kCopyU];
#pragma unroll
    for (int u = 0; u < kCopyU; ++u) {
        const uint32_t col = (tile * kCopyU + u) * kNT + threadIdx.x;
        at[u] = -1;
        if (col < c.all) {
            const uint32_t m = by_cols(col), k = col - m * c.cols;
            at[u] = m * s.mid_stride + (int64_t)k * 16;
            if (k + 1 < c.cols || rest == 16) {
                v[u] = *reinterpret_cast<const Wide16*>(from + at[u]);
            } else {  // the end of a run, taken at once
                store_bytes(to + at[u], rest, load_bytes(from + at[u], rest));
                at[u] = -1;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kCopyU; ++u)
        if (at[u] >= 0) *reinterpret_cast<Wide16*>(to + at[u]) = v[u];
}

// The children's tables and lengths, then the copies.
__global__ __launch_bounds__(kNT) void k_fork_write(Fork f, States st) {
    const bool done = f.plan[0];
    for (int64_t i = blockIdx.x; i < f.children; i += gridDim.x) {
        const Child c = child_of(f, i);
        const int64_t held = f.pages_for(c.before), want = done ? f.pages_for(c.after) : 0;
        const bool copy = f.need[i] < 0;
        const int64_t edge = copy ? held - 1 : -1, start = f.start[i];
        for (int64_t j = threadIdx.x; j < f.max_pages; j += kNT) {
            int32_t q = -1;
            if (j < want) {
                if (j >= held) q = f.list[start + copy + j - held];
                else if (j == edge) q = f.list[start];
                else {
                    q = f.table[c.parent * f.max_pages + j];
                    if (!f.is_page(q)) q = -1;
                }
            }
            f.new_table[i * f.max_pages + j] = q;
        }
        if (threadIdx.x == 0) {
            f.new_length[i] = done ? (int32_t)c.after : 0;
            if (f.counts_left && copy && done) atomicAdd(&f.new_refs[c.edge], -1);
        }
    }
    // items are tiles of a whole block; those past a copy's tokens have nothing to do
    const int64_t copies = f.plan[1];
    for (int u = 0; u < st.count; ++u) {
        const iso_blocks& s = st.b[u];
        const int64_t token = s.inner / f.page_size;
        const uint32_t tiles = CopyTile(s, s.inner).tiles();
        const int64_t per = s.outer * tiles;
        for (int64_t item = blockIdx.x; item < copies * per; item += gridDim.x) {
            const int64_t n = item / per, o = (item - n * per) / tiles;
            const uint32_t tile = (uint32_t)(item - n * per - o * tiles);
            const Copy c = f.copies[n];
            const CopyTile ct(s, c.tokens * token);
            if (tile >= ct.tiles()) continue;
            char* base = static_cast<char*>(s.base) + o * s.outer_stride;
            copy_tile(s, ct, c.tokens * token, base + c.from * s.row_stride, base + f.list[c.to] * s.row_stride, tile);
        }
    }
}

// A step in one workgroup but for what k_fork_write does: the counts are in LDS.
// Up to kOnePages pages, kOneNT children and sequences, kOneEntries entries of
// tables (their counting is this workgroup's).
constexpr int kOneNT = 1024, kOnePages = 12288;
constexpr int64_t kOneEntries = 1 << 16;
__global__ __launch_bounds__(kOneNT) void k_fork_one(Fork f) {
    constexpr int kOneWaves = kOneNT / 64, kEach = kOnePages / kOneNT;
    __shared__ int32_t refs[kOnePages];
    __shared__ int32_t kids[kOneNT];
    __shared__ int32_t edges[kOneNT];
    __shared__ int64_t red[kOneWaves];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    // exclusive prefix over the workgroup of two counts in the halves of 64 bits, and the total
    auto prefix = [&](int64_t v, int64_t& total) {
        int64_t s = v;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t o = (int64_t)__shfl_up((long long)s, d);
            s += lane >= d ? o : 0;
        }
        if (lane == 63) red[wave] = s;
        __syncthreads();
        int64_t before = 0;
        total = 0;
#pragma unroll
        for (int k = 0; k < kOneWaves; ++k) {
            before += k < wave ? red[k] : 0;
            total += red[k];
        }
        __syncthreads();
        return before + s - v;
    };
    for (int p = t; p < (int)f.pages; p += kOneNT) {
        const int32_t n = f.refs[p];
        refs[p] = n > 0 ? n : 0;
    }
    kids[t] = 0;
    Child c{-1, 0, 0, -1};
    const bool is_child = t < f.children;
    if (is_child) c = child_of(f, t);
    edges[t] = c.edge;
    __syncthreads();
    if (c.parent >= 0) atomicAdd(&kids[c.parent], 1);
    __syncthreads();
    for (int s = wave; s < (int)f.seqs; s += kOneWaves) {
        const int32_t more = kids[s] - 1;
        if (!more) continue;
        const int held = (int)f.pages_for(f.tokens_of(s));
        for (int j = lane; j < held; j += 64) {
            const int32_t q = f.table[s * f.max_pages + j];
            if (f.is_page(q)) atomicAdd(&refs[q], more);
        }
    }
    __syncthreads();
    // who goes on to write the same page
    int writers = 0, earlier = 0;
    if (c.edge >= 0) {
        for (int k = 0; k < (int)f.children; ++k) {
            const int same = edges[k] == c.edge;
            writers += same;
            earlier += same && k < t;
        }
    }
    const int copy = c.edge >= 0 && !(refs[c.edge] == writers && !earlier);
    const int64_t want = f.pages_for(c.after);
    const bool too_long = want > f.max_pages || c.after > INT32_MAX;
    const int64_t need = too_long ? 0 : want - f.pages_for(c.before) + copy;
    int64_t all_need, all_copies, all_free;
    // a need is below 2^31, the sum of all below 2^41
    const int64_t start = prefix(need, all_need);
    const int64_t place = prefix(((int64_t)too_long << 32) | copy, all_copies);
    int64_t open = 0;
    const int first = t * kEach;
#pragma unroll
    for (int i = 0; i < kEach; ++i) open += first + i < f.pages && refs[first + i] <= 0;
    int64_t at = prefix(open, all_free);
    const int32_t late = (int32_t)(all_copies >> 32), copies = (int32_t)all_copies;
    const bool done = all_need <= all_free && !late;
    if (is_child) {
        f.need[t] = (int32_t)need | (copy << 31);
        f.start[t] = start;
        if (done && copy) f.copies[(int32_t)place] = Copy{c.edge, (int32_t)start, (int32_t)(c.before % f.page_size), 0};
    }
    if (t == 0) {
        const int64_t lack = all_need - all_free;
        f.status[0] = lack <= 0 ? 0 : lack < INT32_MAX ? (int32_t)lack : INT32_MAX;
        f.status[1] = late;
        f.status[2] = f.plan[1] = done ? copies : 0;
        f.status[3] = done ? (int32_t)all_need : 0;
        f.status[4] = done ? (int32_t)(all_free - all_need) : 0;
        f.plan[0] = done;
    }
    if (done) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int p = first + i;
            if (p < f.pages && refs[p] <= 0) {
                refs[p] = at < all_need;
                if (at < all_need) f.list[at] = p;
                ++at;
            }
        }
        __syncthreads();
        if (copy) atomicAdd(&refs[c.edge], -1);
    }
    __syncthreads();
    for (int p = t; p < (int)f.pages; p += kOneNT) {
        const int32_t n = f.refs[p];
        f.new_refs[p] = done ? refs[p] : n > 0 ? n : 0;
    }
}

struct ForkPlan {
    Blocks pb;
    int64_t child_blocks;
    size_t mark, kids, list, need, start, need_sum, copy_sum, long_sum, free_sum, copies, plan, bytes;
};
ForkPlan fork_plan(int64_t seqs, int64_t children, int64_t pages) {
    ForkPlan p;
    p.pb = page_blocks(pages);
    p.child_blocks = (children + kNT - 1) / kNT;
    size_t at = 0;
    auto room = [&](int64_t n, size_t size) {
        const size_t here = at;
        at += align_up((size_t)n * size);
        return here;
    };
    p.mark = room(pages, sizeof(Mark));
    p.kids = room(seqs, 4);
    p.list = room(pages, 4);
    p.need = room(children, 4);
    p.start = room(children, 8);
    p.need_sum = room(p.child_blocks, 8);
    p.copy_sum = room(p.child_blocks, 4);
    p.long_sum = room(p.child_blocks, 4);
    p.free_sum = room(p.pb.count, 4);
    p.copies = room(children, sizeof(Copy));
    p.plan = room(2, 4);
    p.bytes = at;
    return p;
}

// ---- live pages moved together ----

struct Compact {
    const int32_t *table, *refs;
    int64_t entries, pages;
    int32_t *new_table, *new_refs, *moved, *status;
    int32_t* live_sum;  // [blocks]
    int32_t* place;     // [pages]: a page that stays: itself; one that moves: -2 - its number; a free one: -1
    int32_t *holes, *movers;  // [pages / 2]
    int32_t* plan;            // [2]: live pages, moves
};

__global__ __launch_bounds__(kNT) void k_compact_count(Compact f, Blocks pb) {
    __shared__ int64_t red[kWaves];
    for (int64_t b = blockIdx.x; b < pb.count; b += gridDim.x) {
        const int64_t to = (b + 1) * pb.per < f.pages ? (b + 1) * pb.per : f.pages;
        int64_t n = 0;
        for (int64_t p = b * pb.per + threadIdx.x; p < to; p += kNT) n += f.refs[p] > 0;
        n = wg_sum64(n, red);
        if (threadIdx.x == 0) f.live_sum[b] = (int32_t)n;
    }
}

// With n live pages, `in` of them below n: the page at p < n that is free is hole
// number p - (live before p), one at p >= n that lives moves as number
// (live before p) - in; there are n - in of each.
__global__ __launch_bounds__(kNT) void k_compact_map(Compact f, Blocks pb) {
    __shared__ int64_t red64[kWaves];
    __shared__ int red[kWaves];
    const int64_t n = prefix_of(f.live_sum, pb.count, 0, red64).total, border = n / pb.per;
    int64_t in = 0;
    for (int64_t p = border * pb.per + threadIdx.x; p < n; p += kNT) in += f.refs[p] > 0;
    in = prefix_of(f.live_sum, pb.count, border, red64).before + wg_sum64(in, red64);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        f.status[0] = f.plan[0] = (int32_t)n;
        f.status[1] = f.plan[1] = (int32_t)(n - in);
    }
    for (int64_t b = blockIdx.x; b < pb.count; b += gridDim.x) {
        const int64_t to = (b + 1) * pb.per < f.pages ? (b + 1) * pb.per : f.pages;
        int64_t rank = prefix_of(f.live_sum, pb.count, b, red64).before;
        for (int64_t p0 = b * pb.per; p0 < to; p0 += kNT) {
            const int64_t p = p0 + threadIdx.x;
            const bool lives = p < to && f.refs[p] > 0;
            int sum;
            const int64_t before = rank + wg_prefix(lives, red, sum);
            if (p < to) {
                if (lives && p >= n) f.movers[before - in] = (int32_t)p;
                if (!lives && p < n) f.holes[p - before] = (int32_t)p;
                f.place[p] = !lives ? -1 : p < n ? (int32_t)p : (int32_t)(-2 - (before - in));
            }
            rank += sum;
        }
    }
}

__global__ __launch_bounds__(kNT) void k_compact_write(Compact f, States st) {
    const int64_t n = f.plan[0], moves = f.plan[1];
    const int64_t t = (int64_t)blockIdx.x * kNT + threadIdx.x, step = (int64_t)gridDim.x * kNT;
    auto where = [&](int32_t q) {
        const int32_t at = q >= 0 && q < f.pages ? f.place[q] : -1;
        return at < -1 ? f.holes[-2 - at] : at;
    };
    for (int64_t i = t; i < f.entries; i += step) f.new_table[i] = where(f.table[i]);
    for (int64_t p = t; p < f.pages; p += step) {
        f.moved[p] = where((int32_t)p);
        if (p >= n) f.new_refs[p] = 0;
        else if (f.place[p] >= 0) f.new_refs[p] = f.refs[p];
    }
    for (int64_t k = t; k < moves; k += step) f.new_refs[f.holes[k]] = f.refs[f.movers[k]];
    for (int u = 0; u < st.count; ++u) {
        const iso_blocks& s = st.b[u];
        const CopyTile ct(s, s.inner);
        const uint32_t tiles = ct.tiles();
        const int64_t per = s.outer * tiles;
        for (int64_t item = blockIdx.x; item < moves * per; item += gridDim.x) {
            const int64_t k = item / per, o = (item - k * per) / tiles;
            char* base = static_cast<char*>(s.base) + o * s.outer_stride;
            copy_tile(s, ct, s.inner, base + f.movers[k] * s.row_stride, base + f.holes[k] * s.row_stride,
                      (uint32_t)(item - k * per - o * tiles));
        }
    }
}

struct CompactPlan {
    Blocks pb;
    size_t live_sum, place, holes, movers, plan, bytes;
};
CompactPlan compact_plan(int64_t pages) {
    CompactPlan p;
    p.pb = page_blocks(pages);
    size_t at = 0;
    auto room = [&](int64_t n) {
        const size_t here = at;
        at += align_up((size_t)n * 4);
        return here;
    };
    p.live_sum = room(p.pb.count);
    p.place = room(pages);
    p.holes = room(pages / 2 + 1);
    p.movers = room(pages / 2 + 1);
    p.plan = room(2);
    p.bytes = at;
    return p;
}

constexpr int kGrid = 2048;
inline dim3 grid_of(int64_t items) { return dim3((unsigned)(items < 1 ? 1 : items < kGrid ? items : kGrid)); }

// A block's columns of 16 bytes fit 31 bits, items of a copy of every page 64.
bool pools_ok(const States& st, int64_t pages, int64_t page_size) {
    for (int i = 0; i < st.count; ++i) {
        const iso_blocks& s = st.b[i];
        if (s.inner % page_size) return false;
        if ((s.inner + 15) / 16 > 0x7fffffffLL / s.mid || s.outer > (1LL << 30)) return false;
        if (s.outer * ((s.inner * s.mid >> 15) + 1) > (1LL << 61) / pages) return false;
    }
    return true;
}
// Runs that follow each other without a gap are one.
void join_runs(States& st) {
    for (int i = 0; i < st.count; ++i) {
        iso_blocks& s = st.b[i];
        if (s.mid > 1 && s.mid_stride == s.inner) {
            s.inner *= s.mid;
            s.mid = 1;
        }
    }
}

}  // namespace
}  // namespace iso

extern "C" {

size_t iso_pages_fork_workspace_bytes(int64_t seqs, int64_t children, int64_t pages) {
    if (seqs < 0 || seqs > iso::kMaxSeqs || children < 0 || children > iso::kMaxSeqs || pages < 0 || pages > 0x7fffffffLL)
        return 0;
    return iso::fork_plan(seqs, children, pages).bytes;
}

int iso_pages_fork(const int32_t* table, const int32_t* length, int64_t seqs, int64_t max_pages, const int32_t* refs,
                   int64_t pages, int64_t page_size, const int32_t* parent, const int32_t* grow, int32_t grow_all,
                   int64_t children, const iso_blocks* pools, int count, int32_t* new_table, int32_t* new_length,
                   int32_t* new_refs, int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace iso;
    if (seqs < 0 || seqs > kMaxSeqs || children < 0 || children > kMaxSeqs || pages < 0 || pages > 0x7fffffffLL ||
        max_pages < 0 || max_pages > 0x7fffffffLL || page_size < 1 || page_size > 0x7fffffffLL)
        return ISO_ERR_ARG;
    if ((seqs && (!length || (max_pages && !table))) || (pages && (!refs || !new_refs)) || !status ||
        (children && (!parent || !new_length || (max_pages && !new_table))))
        return ISO_ERR_ARG;
    const size_t tb = (size_t)seqs * (size_t)max_pages * 4, nb = (size_t)children * (size_t)max_pages * 4;
    const size_t pb = (size_t)pages * 4, cb = (size_t)children * 4;
    const Span out[] = {{new_table, nb}, {new_length, cb}, {new_refs, pb}, {status, 20}};
    const Span in[] = {{table, tb}, {length, (size_t)seqs * 4}, {refs, pb}, {parent, cb}, {grow, cb}};
    if (!disjoint(out, in)) return ISO_ERR_ARG;
    const Span all[] = {out[0], out[1], out[2], out[3], in[0], in[1], in[2], in[3], in[4]};
    for (const Span& s : all)
        if (!aligned(s.p, 4)) return ISO_ERR_ARG;
    States st;
    if (!take_states(pools, count, pages, all, st) || !pools_ok(st, pages, page_size)) return ISO_ERR_ARG;
    const ForkPlan pl = fork_plan(seqs, children, pages);
    if (!workspace || workspace_bytes < pl.bytes) return ISO_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return ISO_ERR_ARG;
    char* ws = static_cast<char*>(workspace);
    Fork f{table, length, refs, parent, grow, grow_all, seqs, max_pages, pages, page_size, children,
           new_table, new_length, new_refs, status,
           reinterpret_cast<Mark*>(ws + pl.mark), reinterpret_cast<int32_t*>(ws + pl.kids),
           reinterpret_cast<int32_t*>(ws + pl.list), reinterpret_cast<int32_t*>(ws + pl.need),
           reinterpret_cast<int64_t*>(ws + pl.start), reinterpret_cast<int64_t*>(ws + pl.need_sum),
           reinterpret_cast<int32_t*>(ws + pl.copy_sum), reinterpret_cast<int32_t*>(ws + pl.long_sum),
           reinterpret_cast<int32_t*>(ws + pl.free_sum), reinterpret_cast<Copy*>(ws + pl.copies),
           reinterpret_cast<int32_t*>(ws + pl.plan), true};
    hipStream_t hs = static_cast<hipStream_t>(stream);
    const int64_t blocks = pl.child_blocks + pl.pb.count;
    const int64_t sweep = (pages > seqs ? pages : seqs) / kNT + 1;
    if (pages <= kOnePages && children <= kOneNT && seqs <= kOneNT && seqs * max_pages <= kOneEntries) {
        f.counts_left = false;
        hipLaunchKernelGGL(k_fork_one, dim3(1), dim3(kOneNT), 0, hs, f);
        if (children) hipLaunchKernelGGL(k_fork_write, dim3(kGrid), dim3(kNT), 0, hs, f, st);
        return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
    }
    hipLaunchKernelGGL(k_fork_begin, grid_of(sweep), dim3(kNT), 0, hs, f);
    if (children) hipLaunchKernelGGL(k_fork_count, grid_of(pl.child_blocks), dim3(kNT), 0, hs, f);
    if (seqs) hipLaunchKernelGGL(k_fork_refs, grid_of(seqs), dim3(kNT), 0, hs, f);
    hipLaunchKernelGGL(k_fork_need, grid_of(blocks), dim3(kNT), 0, hs, f, pl.pb, pl.child_blocks);
    hipLaunchKernelGGL(k_fork_list, grid_of(blocks), dim3(kNT), 0, hs, f, pl.pb, pl.child_blocks);
    if (children) hipLaunchKernelGGL(k_fork_write, dim3(kGrid), dim3(kNT), 0, hs, f, st);
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

size_t iso_pages_compact_workspace_bytes(int64_t pages) {
    if (pages < 0 || pages > 0x7fffffffLL) return 0;
    return iso::compact_plan(pages).bytes;
}

int iso_pages_compact(const int32_t* table, int64_t entries, const int32_t* refs, int64_t pages,
                      const iso_blocks* pools, int count, int32_t* new_table, int32_t* new_refs, int32_t* moved,
                      int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace iso;
    if (entries < 0 || entries > (1LL << 50) || pages < 0 || pages > 0x7fffffffLL) return ISO_ERR_ARG;
    if ((entries && (!table || !new_table)) || (pages && (!refs || !new_refs || !moved)) || !status) return ISO_ERR_ARG;
    const size_t tb = (size_t)entries * 4, pb = (size_t)pages * 4;
    const Span out[] = {{new_table, tb}, {new_refs, pb}, {moved, pb}, {status, 8}};
    const Span in[] = {{table, tb}, {refs, pb}};
    if (!disjoint(out, in)) return ISO_ERR_ARG;
    const Span all[] = {out[0], out[1], out[2], out[3], in[0], in[1]};
    for (const Span& s : all)
        if (!aligned(s.p, 4)) return ISO_ERR_ARG;
    States st;
    if (!take_states(pools, count, pages, all, st) || !pools_ok(st, pages, 1)) return ISO_ERR_ARG;
    join_runs(st);
    const CompactPlan pl = compact_plan(pages);
    if (!workspace || workspace_bytes < pl.bytes) return ISO_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return ISO_ERR_ARG;
    char* ws = static_cast<char*>(workspace);
    auto at = [&](size_t o) { return reinterpret_cast<int32_t*>(ws + o); };
    Compact f{table, refs, entries, pages, new_table, new_refs, moved, status,
              at(pl.live_sum), at(pl.place), at(pl.holes), at(pl.movers), at(pl.plan)};
    hipStream_t hs = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(k_compact_count, grid_of(pl.pb.count), dim3(kNT), 0, hs, f, pl.pb);
    hipLaunchKernelGGL(k_compact_map, grid_of(pl.pb.count), dim3(kNT), 0, hs, f, pl.pb);
    hipLaunchKernelGGL(k_compact_write, dim3(kGrid), dim3(kNT), 0, hs, f, st);
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

}  // extern "C"
