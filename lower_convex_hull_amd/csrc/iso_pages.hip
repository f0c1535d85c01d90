// Pages of a cache: a step in which sequences are forked, grown, begun and
// freed, and the live pages moved together (definitions in iso.h).
#include "iso_states.hpp"

namespace iso {
namespace {

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

// N sums over the workgroup at once, the same in every thread.
template <int N>
__device__ __forceinline__ void wg_sums(int64_t (&v)[N], int64_t (*red)[kWaves]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) v[n] += (int64_t)__shfl_xor((long long)v[n], d);
        if (lane == 0) red[n][wave] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        v[n] = 0;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) v[n] += red[n][k];
    }
    __syncthreads();
}

// Pages are taken in blocks, one a workgroup, children in blocks of kNT.
struct Blocks {
    int64_t pages, per;  // pages in all, in a block
    int64_t count;
};
constexpr int64_t kPageBlock = 4 * kNT, kPageBlocks = 4096;
Blocks page_blocks(int64_t pages) {
    Blocks b{pages, kPageBlock, 0};
    if (pages > kPageBlock * kPageBlocks) b.per = ((pages + kPageBlocks - 1) / kPageBlocks + kPageBlock - 1) / kPageBlock * kPageBlock;
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
    double part;  // 1 / page_size
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
    int32_t* gap;       // [children] what a kept page's count lacks, or NULL: k_fork_write adds it
    int32_t* plan;      // [4]: done or not, copies, pages taken, counts below 0 or none
    bool counts_left;   // k_fork_write brings the counts up to date

    __device__ __forceinline__ int64_t tokens_of(int64_t s) const {
        const int64_t n = length[s], most = max_pages * page_size;
        return n < 0 ? 0 : n < most ? n : most;
    }
    // Whole pages of n < 2^32 tokens, and pages that hold them (Divide's product).
    __device__ __forceinline__ uint32_t whole(int64_t n) const { return (uint32_t)(((double)n + 0.5) * part); }
    __device__ __forceinline__ int64_t past(int64_t n) const { return n - (int64_t)whole(n) * page_size; }
    __device__ __forceinline__ int64_t pages_for(int64_t n) const { return (int64_t)whole(n) + (past(n) > 0); }
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
    if (g > 0 && f.past(c.before)) {
        const int32_t q = f.table[c.parent * f.max_pages + f.whole(c.before)];
        if (f.is_page(q)) c.edge = q;
    }
    return c;
}

// All but the copies is bound by launches and latency: a step of 1024 sequences over 84000
// pages moves 1.2 MB, its four kernels take 3.4, 6.4, 10.0 and 5.1 us.
// A step of any size takes six launches: the counts copied and the free pages
// counted by block; each sequence's children counted, and who goes on to write
// which page; the counts of the pages of sequences with other than one child;
// what each child takes; where it begins in the list of the taken pages, and the
// list; tables and copies.  Where children are few the second and the fourth are
// done by each workgroup of their neighbours for itself.
__global__ __launch_bounds__(kNT) void k_fork_begin(Fork f, Blocks pb) {
    __shared__ int64_t red[1][kWaves];
    const int64_t t = (int64_t)blockIdx.x * kNT + threadIdx.x, step = (int64_t)gridDim.x * kNT;
    for (int64_t b = blockIdx.x; b < pb.count; b += gridDim.x) {
        const int64_t to = (b + 1) * pb.per < f.pages ? (b + 1) * pb.per : f.pages;
        int64_t open[1] = {0};
        for (int64_t p0 = b * pb.per + threadIdx.x; p0 < to; p0 += kPageBlock)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t p = p0 + i * kNT;
                if (p >= to) break;
                const int32_t n = f.refs[p];
                f.new_refs[p] = n > 0 ? n : 0;
                open[0] += n <= 0;
                if (f.mark) f.mark[p] = Mark{0, INT32_MAX};
            }
        wg_sums(open, red);
        if (threadIdx.x == 0) f.free_sum[b] = (int32_t)open[0];
    }
    if (f.kids)
        for (int64_t s = t; s < f.seqs; s += step) f.kids[s] = 0;
    if (t == 0) f.plan[3] = 0;
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

// A sequence's pages have a holder less for it and one more for each child;
// those that nobody holds any more are free.
__global__ __launch_bounds__(kNT) void k_fork_refs(Fork f, Blocks pb) {
    for (int64_t s = blockIdx.x; s < f.seqs; s += gridDim.x) {
        int32_t more = -1;
        if (f.kids) {
            more += f.kids[s];
        } else {
            for (int64_t i0 = 0; i0 < f.children; i0 += 4 * kNT) {
                int own = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t k = i0 + i * kNT + threadIdx.x;
                    own += k < f.children && f.parent[k] == s;
                }
                // own is 4 at most: three counts of its bits
                more += __syncthreads_count(own & 1) + 2 * __syncthreads_count(own & 2) + 4 * __syncthreads_count(own & 4);
            }
        }
        if (!more) continue;
        const int64_t held = f.pages_for(f.tokens_of(s));
        for (int64_t j = threadIdx.x; j < held; j += kNT) {
            const int32_t q = f.table[s * f.max_pages + j];
            if (!f.is_page(q)) continue;
            // past 32 bits as the count in memory: the free pages stay those that are counted
            const int32_t was = atomicAdd(&f.new_refs[q], more), is = (int32_t)((uint32_t)was + (uint32_t)more);
            if ((was <= 0) != (is <= 0)) atomicAdd(&f.free_sum[q / pb.per], is <= 0 ? 1 : -1);
            if (is < 0) f.plan[3] = 1;  // fewer holders counted than the tables have
        }
    }
}

// What the step comes to.
struct Total {
    int64_t need, room, late, copies;
    __device__ __forceinline__ bool done() const { return need <= room && !late; }
};
__device__ __forceinline__ void write_status(const Fork& f, const Total& t) {
    const int64_t lack = t.need - t.room;
    const bool done = t.done();
    f.status[0] = lack <= 0 ? 0 : lack < INT32_MAX ? (int32_t)lack : INT32_MAX;
    f.status[1] = (int32_t)t.late;
    f.status[2] = f.plan[1] = done ? (int32_t)t.copies : 0;
    f.status[3] = f.plan[2] = done ? (int32_t)t.need : 0;
    f.status[4] = done ? (int32_t)(t.room - t.need) : 0;
    f.plan[0] = done;
}

// Blocks of children: the pages each takes.  A page that children go on to write
// has them as holders at least, however few are counted (the first of them brings
// its count up, the others find it no larger than themselves before and after): it
// is not free, so that nobody's copy goes where another is read.
__global__ __launch_bounds__(kNT) void k_fork_need(Fork f, Blocks pb, int64_t child_blocks) {
    __shared__ int64_t red[2][kWaves];
    for (int64_t b = blockIdx.x; b < child_blocks; b += gridDim.x) {
        const int64_t i = b * kNT + threadIdx.x;
        int64_t need = 0;
        int copies = 0, too_long = 0;
        if (i < f.children) {
            const Child c = child_of(f, i);
            const int64_t want = f.pages_for(c.after);
            if (c.edge >= 0) {
                const Mark m = f.mark[c.edge];
                const int32_t held = f.new_refs[c.edge];
                copies = !(held <= m.writers && m.first == i);
                if (held < m.writers && m.first == i) {
                    f.new_refs[c.edge] = m.writers;
                    if (held <= 0) atomicAdd(&f.free_sum[c.edge / pb.per], -1);
                }
            }
            too_long = want > f.max_pages || c.after > INT32_MAX;
            need = too_long ? 0 : want - f.pages_for(c.before) + copies;
            f.need[i] = (int32_t)need | (copies << 31);
        }
        int64_t v[2] = {need, ((int64_t)too_long << 32) | copies};
        wg_sums(v, red);
        if (threadIdx.x == 0) {
            f.need_sum[b] = v[0];
            f.copy_sum[b] = (int32_t)v[1];
            f.long_sum[b] = (int32_t)(v[1] >> 32);
        }
    }
}

// The list of the taken pages, the lowest free ones: a block's part, by a
// workgroup of NT threads.  The counts stay as they are: other workgroups of the
// launch go by them (k_fork_write brings them up to date), but that those below 0
// (is there one: `below`) of pages nobody goes on to write become 0.  Pages for
// which `kept` are not free though their count may say so (does one: `some`).
template <int NT, typename K>
__device__ __forceinline__ void list_block(const Fork& f, const Blocks& pb, int64_t b, int64_t rank, const Total& total,
                                           int* red, bool below, bool some, K kept) {
    constexpr int kW = NT / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t to = (b + 1) * pb.per < f.pages ? (b + 1) * pb.per : f.pages;
    if (!total.done()) return;
    if (below)
        for (int64_t p = b * pb.per + threadIdx.x; p < to; p += NT)
            if (f.new_refs[p] < 0 && !kept(p)) f.new_refs[p] = 0;
    for (int64_t p0 = b * pb.per; p0 < to && rank < total.need; p0 += NT) {
        const int64_t p = p0 + threadIdx.x;
        const bool open = p < to && f.new_refs[p] <= 0 && !(some && kept(p));
        const uint64_t mask = __ballot(open);
        if (lane == 0) red[wave] = __popcll(mask);
        __syncthreads();
        int64_t at = rank + __popcll(mask & ((1ull << lane) - 1));
#pragma unroll
        for (int k = 0; k < kW; ++k) {
            at += k < wave ? red[k] : 0;
            rank += red[k];
        }
        __syncthreads();
        if (open && at < total.need) f.list[at] = (int32_t)p;
    }
}

// Blocks of children: where each one's pages begin in the list, and the copies.
// Blocks of pages: the list.
__global__ __launch_bounds__(kNT) void k_fork_list(Fork f, Blocks pb, int64_t child_blocks) {
    __shared__ int64_t red64[6][kWaves];
    __shared__ int red[kWaves];
    const bool below = f.plan[3];
    for (int64_t b = blockIdx.x; b < child_blocks + pb.count; b += gridDim.x) {
        // need, late, copies, free; need and copies, or free, of the blocks before
        int64_t v[6] = {0, 0, 0, 0, 0, 0};
        for (int64_t k = threadIdx.x; k < child_blocks; k += kNT) {
            const int64_t need = f.need_sum[k], copies = f.copy_sum[k];
            v[0] += need;
            v[1] += f.long_sum[k];
            v[2] += copies;
            v[4] += k < b ? need : 0;
            v[5] += k < b ? copies : 0;
        }
        if (b >= child_blocks) v[4] = 0;
        for (int64_t k = threadIdx.x; k < pb.count; k += kNT) {
            const int64_t open = f.free_sum[k];
            v[3] += open;
            v[4] += child_blocks + k < b ? open : 0;
        }
        wg_sums(v, red64);
        const Total total{v[0], v[3], v[1], v[2]};
        if (b == 0 && threadIdx.x == 0) write_status(f, total);
        if (b < child_blocks) {
            const int64_t i = b * kNT + threadIdx.x;
            const int32_t n = i < f.children ? f.need[i] : 0;
            const int own = n & INT32_MAX, copy = (uint32_t)n >> 31;
            int sum;
            // a block's needs can pass 2^31 only where nothing is done
            const int64_t start = v[4] + wg_prefix(own, red, sum);
            const int64_t place = v[5] + wg_prefix(copy, red, sum);
            if (i < f.children) f.start[i] = start;
            if (copy && total.done()) {
                const Child c = child_of(f, i);
                f.copies[place] = Copy{c.edge, (int32_t)start, (int32_t)f.past(c.before), 0};
            }
        } else {
            list_block<kNT>(f, pb, b - child_blocks, v[4], total, red, below, false, [](int64_t) { return false; });
        }
    }
}

// One workgroup's view of few children, one a thread.
constexpr int kOneNT = 1024, kOneWaves = kOneNT / 64;
struct Few {
    Child c;
    int64_t start, place;  // pages and copies before its own
    int64_t need;
    int copy;
    int32_t gap;  // what the count of its edge page lacks, at the first of the page's writers
    bool lost;    // such a page was counted as free
    int losts;    // how many were
    Total total;
};
// Exclusive prefixes of N values over the workgroup, and their totals.
template <int N>
__device__ __forceinline__ void one_prefix(int64_t (&v)[N], int64_t (&total)[N], int64_t (*red)[kOneWaves]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t s[N];
#pragma unroll
    for (int n = 0; n < N; ++n) s[n] = v[n];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int64_t o = (int64_t)__shfl_up((long long)s[n], d);
            s[n] += lane >= d ? o : 0;
        }
#pragma unroll
    for (int n = 0; n < N; ++n)
        if (lane == 63) red[n][wave] = s[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        int64_t before = 0;
        total[n] = 0;
#pragma unroll
        for (int k = 0; k < kOneWaves; ++k) {
            before += k < wave ? red[n][k] : 0;
            total[n] += red[n][k];
        }
        v[n] = before + s[n] - v[n];
    }
    __syncthreads();
}
// Who goes on to write which page: a table in LDS by open addressing, with twice
// as many places as there can be pages in it.
struct Edges {
    static constexpr int kPlaces = 2 * kOneNT;
    int32_t page[kPlaces], writers[kPlaces], first[kPlaces];
    __device__ __forceinline__ void clear() {
        for (int i = threadIdx.x; i < kPlaces; i += kOneNT) {
            page[i] = -1;
            writers[i] = 0;
            first[i] = INT32_MAX;
        }
    }
    __device__ __forceinline__ int add(int32_t q) {
        uint32_t at = (uint32_t)q * 2654435761u >> 21;
        static_assert(kPlaces == 1 << 11, "");
        for (;;) {
            const int32_t there = atomicCAS(&page[at], -1, q);
            if (there == -1 || there == q) break;
            at = (at + 1) & (kPlaces - 1);
        }
        atomicAdd(&writers[at], 1);
        atomicMin(&first[at], (int32_t)threadIdx.x);
        return (int)at;
    }
    __device__ __forceinline__ bool has(int32_t q) const {
        uint32_t at = (uint32_t)q * 2654435761u >> 21;
        while (page[at] != -1 && page[at] != q) at = (at + 1) & (kPlaces - 1);
        return page[at] == q;
    }
};
// Every thread's child, its edge page (if any) at place `at` of the table and held
// by `count`, its writers at least (as in k_fork_need); `room` the free pages it has
// counted, such a page among them where `count` is not above 0, then those before
// them.  After a barrier.
__device__ __forceinline__ Few few_children(const Fork& f, const Child& c, const Edges& edges, int at, int32_t count,
                                            int64_t& room, int64_t (*red)[kOneWaves]) {
    Few o;
    o.c = c;
    const int32_t writers = edges.writers[at];
    const bool first = c.edge >= 0 && edges.first[at] == (int32_t)threadIdx.x;
    o.copy = c.edge >= 0 && !(count <= writers && first);
    o.gap = first && count < writers ? (int32_t)((uint32_t)writers - (uint32_t)count) : 0;
    o.lost = o.gap && count <= 0;
    const int64_t want = f.pages_for(c.after);
    const bool too_long = want > f.max_pages || c.after > INT32_MAX;
    o.need = too_long ? 0 : want - f.pages_for(c.before) + o.copy;
    // a need is below 2^31, the sum of all below 2^41; children too long and copies share a sum, free pages and lost ones
    int64_t v[3] = {o.need, ((int64_t)too_long << 32) | o.copy, ((int64_t)o.lost << 32) | room}, total[3];
    one_prefix(v, total, red);
    o.start = v[0];
    o.place = (int32_t)v[1];
    room = (uint32_t)v[2];
    o.losts = (int)(total[2] >> 32);
    o.total = Total{total[0], (int64_t)(uint32_t)total[2] - o.losts, total[1] >> 32, (int32_t)total[1]};
    return o;
}
__device__ __forceinline__ void write_few(const Fork& f, const Few& o, bool done) {
    const int64_t i = threadIdx.x;
    if (i >= f.children) return;
    f.need[i] = (int32_t)o.need | (o.copy << 31);
    f.start[i] = o.start;
    f.gap[i] = o.gap;
    if (done && o.copy) f.copies[o.place] = Copy{o.c.edge, (int32_t)o.start, (int32_t)f.past(o.c.before), 0};
}

// What few children take, by every workgroup, and each one's part of the list.
__global__ __launch_bounds__(kOneNT) void k_fork_few(Fork f, Blocks pb) {
    __shared__ Edges edges;
    __shared__ int64_t red[3][kOneWaves];
    __shared__ int red32[kOneWaves];
    Child c{-1, 0, 0, -1};
    const bool below = f.plan[3];
    edges.clear();
    if (threadIdx.x < f.children) c = child_of(f, threadIdx.x);
    const int32_t count = c.edge >= 0 ? f.new_refs[c.edge] : 0;
    __syncthreads();
    const int at = c.edge >= 0 ? edges.add(c.edge) : 0;
    __syncthreads();
    int64_t open = 0;
    for (int64_t k = threadIdx.x; k < pb.count; k += kOneNT) open += f.free_sum[k];
    const Few o = few_children(f, c, edges, at, count, open, red);
    if (blockIdx.x == 0) {
        write_few(f, o, o.total.done());
        if (threadIdx.x == 0) write_status(f, o.total);
    }
    for (int64_t b = blockIdx.x; b < pb.count; b += gridDim.x) {
        int64_t before[1] = {0}, rank[1];
        for (int64_t k = threadIdx.x; k < b; k += kOneNT) before[0] += f.free_sum[k];
        before[0] -= o.lost && c.edge / pb.per < b;
        one_prefix(before, rank, red);
        list_block<kOneNT>(f, pb, b, rank[0], o.total, red32, below, o.losts > 0, [&](int64_t p) { return edges.has((int32_t)p); });
    }
}

// A step in one workgroup but for what k_fork_write does: the counts are in LDS.  Bound by
// the latency of its steps: 7.7 us for four sequences, 14.2 for 256 over 12280 pages, 16
// where a step's copies came before and the tables are not in the caches (with each
// child's page compared with every other's 27).
// Up to kOnePages pages: a step in which every sequence goes on by itself then takes what
// four launches take (with k_fork_write, 64 sequences: 8192 pages 13.1 us and 14.3, 12288
// 14.6 and 14.1; 1024 sequences 14.8 and 16.5, 16.5 and 16.5), one whose beams all change
// parents less (12288 pages 15.2 and 28.0); room for 16384 would cost every step 3 us.
// Up to kOneEntries entries of tables, which this workgroup alone walks: 256 sequences of
// 96, 24576 in all, 15.4 us and 15.7, of 128 17.3 and 15.7, of 192 17.8 and 15.7; beams
// 16.3 and 25.1, 18.5 and 25.1, 18.6 and 25.1 (6000 pages).  Up to kOneNT children and
// sequences, one a thread.
constexpr int kOnePages = 12288;
constexpr int64_t kOneEntries = 1 << 15;
__global__ __launch_bounds__(kOneNT) void k_fork_one(Fork f) {
    constexpr int kEach = kOnePages / kOneNT, kAhead = 8;
    __shared__ int32_t refs[kOnePages];
    __shared__ int32_t kids[kOneNT], held[kOneNT];
    __shared__ Edges edges;
    __shared__ int64_t red[3][kOneWaves];
    const int t = threadIdx.x;
    const uint32_t entries = (uint32_t)(f.seqs * f.max_pages);
    // entries of the tables, whether they count or not: the first are on their way with all else
    int32_t page[kAhead];
    auto load = [&](uint32_t e0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const uint32_t e = e0 + i * kOneNT;
            page[i] = e < entries ? f.table[e] : -1;
        }
    };
    load(t);
    int32_t own[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int p = i * kOneNT + t;
        own[i] = p < (int)f.pages ? max(f.refs[p], 0) : 1;
    }
    held[t] = t < f.seqs ? (int32_t)f.pages_for(f.tokens_of(t)) : 0;
    Child c{-1, 0, 0, -1};
    if (t < f.children) c = child_of(f, t);
#pragma unroll
    for (int i = 0; i < kEach; ++i) refs[i * kOneNT + t] = own[i];  // a place behind the last page: held
    edges.clear();
    kids[t] = 0;
    __syncthreads();
    if (c.parent >= 0) atomicAdd(&kids[c.parent], 1);
    const int place = c.edge >= 0 ? edges.add(c.edge) : 0;
    __syncthreads();
    const Divide by_row((uint32_t)f.max_pages);
    for (uint32_t e0 = t; e0 < entries; e0 += kOneNT * kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const uint32_t e = e0 + i * kOneNT;
            if (e >= entries || !f.is_page(page[i])) continue;
            const uint32_t s = by_row(e);
            const int32_t more = kids[s] - 1;
            if (more && (int32_t)(e - s * (uint32_t)f.max_pages) < held[s]) atomicAdd(&refs[page[i]], more);
        }
        load(e0 + kOneNT * kAhead);
    }
    __syncthreads();
    if (c.edge >= 0) atomicMax(&refs[c.edge], edges.writers[place]);
    __syncthreads();
    int64_t at = 0;
    const int first = t * kEach;
#pragma unroll
    for (int i = 0; i < kEach; ++i) at += refs[first + i] <= 0;
    const Few o = few_children(f, c, edges, place, c.edge >= 0 ? refs[c.edge] : 0, at, red);
    const bool done = o.total.done();
    write_few(f, o, done);
    if (t == 0) write_status(f, o.total);
    if (done) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int p = first + i;
            if (refs[p] <= 0) {
                refs[p] = at < o.total.need;
                if (at < o.total.need) f.list[at] = p;
                ++at;
            }
        }
        __syncthreads();
        if (o.copy) atomicAdd(&refs[c.edge], -1);
    }
    __syncthreads();
    for (int p = t; p < (int)f.pages; p += kOneNT) f.new_refs[p] = done ? refs[p] : max(f.refs[p], 0);
}

// 16-byte columns of what one block of an array holds, `bytes` of each of its mid
// runs, by the workgroup: kCopyU of them a thread are on their way at a time (half of a
// 2.3 GB pool, 1562 MB moved: 294 us, 5.3 TB/s; with 4 on their way 389 us, with a quarter
// of the workgroups 395, byte by byte 822).
constexpr int kCopyU = 8;
struct CopyTile {
    uint32_t cols, all;  // columns of a run, of all of them
    __device__ __forceinline__ CopyTile(const iso_blocks& s, int64_t bytes)
        : cols((uint32_t)((bytes + 15) / 16)), all((uint32_t)s.mid * cols) {}
    __device__ __forceinline__ uint32_t tiles() const { return (all + kNT * kCopyU - 1) / (kNT * kCopyU); }
};
template <bool STREAM_LOADS, bool STREAM_STORES>
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
                v[u] = load_quad<STREAM_LOADS>(from + at[u]);
            } else {  // the end of a run, taken at once
                store_bytes(to + at[u], rest, load_bytes(from + at[u], rest));
                at[u] = -1;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kCopyU; ++u)
        if (at[u] >= 0) store_quad<STREAM_STORES>(to + at[u], v[u]);
}

// The children's tables and lengths, then the copies: their loads through the caches,
// their stores past them, however large the pool is.  Cold, with a read of the copied
// pages behind them: 14.7 MB 33.1 and 44.0 us (both through the caches 33.0 and 43.0, both
// past them 34.9 and 45.9), 235 MB 156 and 253 (152 and 258, 169 and 271), 470 MB 252 and
// 449 (249 and 461, 274 and 478); one after another the same 22 MB a step leave the tables
// in the caches (25.2 us a step, 26.4, 25.1).
__global__ __launch_bounds__(kNT) void k_fork_write(Fork f, States st) {
    const bool done = f.plan[0];
    for (int64_t i = blockIdx.x; i < f.children; i += gridDim.x) {
        const Child c = child_of(f, i);
        const int64_t held = f.pages_for(c.before), want = done ? f.pages_for(c.after) : 0;
        const bool copy = f.need[i] < 0;
        const int32_t gap = f.gap ? f.gap[i] : 0;
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
            const int32_t more = f.counts_left && done ? gap - copy : 0;
            if (more) atomicAdd(&f.new_refs[c.edge], more);
        }
    }
    if (f.counts_left) {
        const int64_t t = (int64_t)blockIdx.x * kNT + threadIdx.x, step = (int64_t)gridDim.x * kNT, taken = f.plan[2];
        for (int64_t k = t; k < taken; k += step) f.new_refs[f.list[k]] = 1;
        for (int64_t p = t; p < f.pages && !done; p += step) f.new_refs[p] = max(f.refs[p], 0);  // as they were
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
            copy_tile<false, true>(s, ct, c.tokens * token, base + c.from * s.row_stride, base + f.list[c.to] * s.row_stride, tile);
        }
    }
}

struct ForkPlan {
    Blocks pb;
    int64_t child_blocks;
    size_t mark, kids, list, need, start, need_sum, copy_sum, long_sum, free_sum, copies, gap, plan, bytes;
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
    p.gap = room(children, 4);
    p.plan = room(4, 4);
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
    __shared__ int64_t red[1][kWaves];
    for (int64_t b = blockIdx.x; b < pb.count; b += gridDim.x) {
        const int64_t to = (b + 1) * pb.per < f.pages ? (b + 1) * pb.per : f.pages;
        int64_t n[1] = {0};
        for (int64_t p0 = b * pb.per + threadIdx.x; p0 < to; p0 += kPageBlock)
#pragma unroll
            for (int i = 0; i < 4; ++i) n[0] += p0 + i * kNT < to && f.refs[p0 + i * kNT] > 0;
        wg_sums(n, red);
        if (threadIdx.x == 0) f.live_sum[b] = (int32_t)n[0];
    }
}

// With n live pages, `in` of them below n: the page at p < n that is free is hole
// number p - (live before p), one at p >= n that lives moves as number
// (live before p) - in; there are n - in of each.
__global__ __launch_bounds__(kNT) void k_compact_map(Compact f, Blocks pb) {
    __shared__ int64_t red64[2][kWaves];
    __shared__ int red[kWaves];
    for (int64_t b = blockIdx.x; b < pb.count; b += gridDim.x) {
        int64_t v[2] = {0, 0};  // live pages, those in the blocks before
        for (int64_t k = threadIdx.x; k < pb.count; k += kNT) {
            const int64_t live = f.live_sum[k];
            v[0] += live;
            v[1] += k < b ? live : 0;
        }
        wg_sums(v, red64);
        const int64_t n = v[0], border = n / pb.per;
        int64_t rank = v[1];
        int64_t in[1] = {0};  // of the whole blocks below n, and of its own block
        for (int64_t k = threadIdx.x; k < border; k += kNT) in[0] += f.live_sum[k];
        for (int64_t p0 = border * pb.per + threadIdx.x; p0 < n; p0 += kPageBlock)
#pragma unroll
            for (int i = 0; i < 4; ++i) in[0] += p0 + i * kNT < n && f.refs[p0 + i * kNT] > 0;
        wg_sums(in, red64);
        if (b == 0 && threadIdx.x == 0) {
            f.status[0] = f.plan[0] = (int32_t)n;
            f.status[1] = f.plan[1] = (int32_t)(n - in[0]);
        }
        const int64_t to = (b + 1) * pb.per < f.pages ? (b + 1) * pb.per : f.pages;
        for (int64_t p0 = b * pb.per; p0 < to; p0 += kNT) {
            const int64_t p = p0 + threadIdx.x;
            const bool lives = p < to && f.refs[p] > 0;
            int sum;
            const int64_t before = rank + wg_prefix(lives, red, sum);
            if (p < to) {
                if (lives && p >= n) f.movers[before - in[0]] = (int32_t)p;
                if (!lives && p < n) f.holes[p - before] = (int32_t)p;
                f.place[p] = !lives ? -1 : p < n ? (int32_t)p : (int32_t)(-2 - (before - in[0]));
            }
            rank += sum;
        }
    }
}

// The same in one workgroup, up to kCompactPages pages: with k_compact_write 6.2 us for
// 165 pages, 7.7 for 2048 and 8.6 for 4096, as three launches 7.0, 10.4 and 10.5.  Room for
// 8192 would cost small pools a microsecond (7.1, 8.5 and 9.9) and lose at 8192 (12.4 and
// 10.8).
constexpr int kCompactPages = 4096;
__global__ __launch_bounds__(kOneNT) void k_compact_one(Compact f) {
    constexpr int kEach = kCompactPages / kOneNT;
    __shared__ uint8_t lives[kCompactPages];
    __shared__ int64_t red[1][kOneWaves];
    const int t = threadIdx.x, first = t * kEach;
    int32_t own[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) own[i] = i * kOneNT + t < f.pages ? f.refs[i * kOneNT + t] : 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) lives[i * kOneNT + t] = own[i] > 0;
    __syncthreads();
    int64_t rank[1] = {0}, n[1], in[1] = {0}, all[1];
#pragma unroll
    for (int i = 0; i < kEach; ++i) rank[0] += lives[first + i];
    one_prefix(rank, n, red);
#pragma unroll
    for (int i = 0; i < kEach; ++i) in[0] += first + i < n[0] && lives[first + i];
    one_prefix(in, all, red);
    int32_t before = (int32_t)rank[0];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int p = first + i;
        if (p >= f.pages) break;
        const bool live = lives[p];
        if (live && p >= n[0]) f.movers[before - all[0]] = p;
        if (!live && p < n[0]) f.holes[p - before] = p;
        f.place[p] = !live ? -1 : p < n[0] ? p : (int32_t)(-2 - (before - all[0]));
        before += live;
    }
    if (t == 0) {
        f.status[0] = f.plan[0] = (int32_t)n[0];
        f.status[1] = f.plan[1] = (int32_t)(n[0] - all[0]);
    }
}

template <bool STREAM>
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
            copy_tile<STREAM, STREAM>(s, ct, s.inner, base + f.movers[k] * s.row_stride, base + f.holes[k] * s.row_stride,
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

constexpr int kGrid = 2048, kCopyGrid = 8192, kFewGrid = 64;
inline dim3 grid_of(int64_t items) { return dim3((unsigned)(items < 1 ? 1 : items < kGrid ? items : kGrid)); }

// A block's columns of 16 bytes fit 31 bits, items of a copy of every page 64.
bool pools_ok(const Arrays& st, int64_t pages, int64_t page_size) {
    for (int i = 0; i < st.count; ++i) {
        const iso_blocks& s = st.b[i];
        if (s.inner % page_size) return false;
        if ((s.inner + 15) / 16 > 0x7fffffffLL / s.mid || s.outer > (1LL << 30)) return false;
        if (s.outer * ((s.inner * s.mid >> 15) + 1) > (1LL << 61) / pages) return false;
    }
    return true;
}
// Runs that follow each other without a gap are one.
void join_runs(Arrays& st) {
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
    Arrays arrays;
    if (!take_states(pools, count, pages, all, arrays) || !pools_ok(arrays, pages, page_size)) return ISO_ERR_ARG;
    const ForkPlan pl = fork_plan(seqs, children, pages);
    if (!workspace || workspace_bytes < pl.bytes) return ISO_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return ISO_ERR_ARG;
    char* ws = static_cast<char*>(workspace);
    Fork f{table, length, refs, parent, grow, grow_all, seqs, max_pages, pages, page_size, children,
           1.0 / (double)page_size, new_table, new_length, new_refs, status,
           reinterpret_cast<Mark*>(ws + pl.mark), reinterpret_cast<int32_t*>(ws + pl.kids),
           reinterpret_cast<int32_t*>(ws + pl.list), reinterpret_cast<int32_t*>(ws + pl.need),
           reinterpret_cast<int64_t*>(ws + pl.start), reinterpret_cast<int64_t*>(ws + pl.need_sum),
           reinterpret_cast<int32_t*>(ws + pl.copy_sum), reinterpret_cast<int32_t*>(ws + pl.long_sum),
           reinterpret_cast<int32_t*>(ws + pl.free_sum), reinterpret_cast<Copy*>(ws + pl.copies),
           reinterpret_cast<int32_t*>(ws + pl.gap), reinterpret_cast<int32_t*>(ws + pl.plan), true};
    hipStream_t hs = static_cast<hipStream_t>(stream);
    const bool few = children <= kOneNT;
    if (few && pages <= kOnePages && seqs <= kOneNT && seqs * max_pages <= kOneEntries) {
        f.counts_left = false;
        hipLaunchKernelGGL(k_fork_one, dim3(1), dim3(kOneNT), 0, hs, f);
    } else {
        if (few) {
            f.mark = nullptr;
            f.kids = nullptr;
        } else {
            f.gap = nullptr;
        }
        const int64_t rows = few ? 0 : (seqs + kNT - 1) / kNT;
        hipLaunchKernelGGL(k_fork_begin, grid_of(pl.pb.count > rows ? pl.pb.count : rows), dim3(kNT), 0, hs, f, pl.pb);
        if (!few) hipLaunchKernelGGL(k_fork_count, grid_of(pl.child_blocks), dim3(kNT), 0, hs, f);
        if (seqs) hipLaunchKernelGGL(k_fork_refs, grid_of(seqs), dim3(kNT), 0, hs, f, pl.pb);
        if (few) {
            hipLaunchKernelGGL(k_fork_few, dim3((unsigned)(pl.pb.count < 1 ? 1 : pl.pb.count < kFewGrid ? pl.pb.count : kFewGrid)),
                               dim3(kOneNT), 0, hs, f, pl.pb);
        } else {
            hipLaunchKernelGGL(k_fork_need, grid_of(pl.child_blocks), dim3(kNT), 0, hs, f, pl.pb, pl.child_blocks);
            hipLaunchKernelGGL(k_fork_list, grid_of(pl.child_blocks + pl.pb.count), dim3(kNT), 0, hs, f, pl.pb, pl.child_blocks);
        }
    }
    if (children) arrays.each_launch([&](const States& st, bool first) {
        if (!first) {  // copies only: tables and counts are written
            f.children = 0;
            f.counts_left = false;
        }
        int64_t items = f.children;  // a child's table; a tile of an array's block of a copied page
        for (int i = 0; i < st.count; ++i) items += children * st.b[i].outer * ((st.b[i].inner * st.b[i].mid >> 15) + 1);
        const dim3 grid((unsigned)(items < kCopyGrid ? items : kCopyGrid));
        hipLaunchKernelGGL(k_fork_write, grid, dim3(kNT), 0, hs, f, st);
    });
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
    Arrays arrays;
    if (!take_states(pools, count, pages, all, arrays) || !pools_ok(arrays, pages, 1)) return ISO_ERR_ARG;
    join_runs(arrays);
    const CompactPlan pl = compact_plan(pages);
    if (!workspace || workspace_bytes < pl.bytes) return ISO_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return ISO_ERR_ARG;
    char* ws = static_cast<char*>(workspace);
    auto at = [&](size_t o) { return reinterpret_cast<int32_t*>(ws + o); };
    Compact f{table, refs, entries, pages, new_table, new_refs, moved, status,
              at(pl.live_sum), at(pl.place), at(pl.holes), at(pl.movers), at(pl.plan)};
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (pages <= kCompactPages) {
        hipLaunchKernelGGL(k_compact_one, dim3(1), dim3(kOneNT), 0, hs, f);
    } else {
        hipLaunchKernelGGL(k_compact_count, grid_of(pl.pb.count), dim3(kNT), 0, hs, f, pl.pb);
        hipLaunchKernelGGL(k_compact_map, grid_of(pl.pb.count), dim3(kNT), 0, hs, f, pl.pb);
    }
    const bool stream_all = streamed(arrays, pages);
    arrays.each_launch([&](const States& st, bool first) {
        if (!first) f.entries = f.pages = 0;  // moves only: tables are written (the moved counts once more)
        int64_t items = (f.entries + kNT - 1) / kNT + (f.pages + kNT - 1) / kNT;
        for (int i = 0; i < st.count; ++i) items += pages / 2 * st.b[i].outer * ((st.b[i].inner * st.b[i].mid >> 15) + 1);
        const dim3 grid((unsigned)(items < 1 ? 1 : items < kCopyGrid ? items : kCopyGrid));
        if (stream_all) hipLaunchKernelGGL(k_compact_write<true>, grid, dim3(kNT), 0, hs, f, st);
        else hipLaunchKernelGGL(k_compact_write<false>, grid, dim3(kNT), 0, hs, f, st);
    });
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

}  // extern "C"
