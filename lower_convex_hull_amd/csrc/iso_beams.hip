// Beam search: the selection over beams and vocabulary from logits, and the
// states of beams brought into the order of their parents (formulas in iso.h).
#include "iso_logits.hpp"
#include "iso_states.hpp"

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

struct Beams {
    const float* score;
    const float* weight;   // or NULL
    const uint8_t* ended;  // or NULL
    int beams, take;
    int32_t end_token;
    __device__ __forceinline__ bool counts(int64_t r) const {
        const float w = weight ? weight[r] : 1.0f;
        return fabsf(score[r]) < INFINITY && w > 0.0f && w < INFINITY;
    }
    __device__ __forceinline__ bool has_ended(int64_t r) const { return ended && ended[r]; }
};

// Item = (row, piece of it), held in the registers of a workgroup: the piece's
// maximum and sum, and its `take` best tokens, one round of a maximum each.
template <typename T, int NT, int U>
__global__ __launch_bounds__(NT) void k_beam_pieces(const T* __restrict__ logits, int64_t rows, int vocab, int64_t ld,
                                                    Beams b, Scale sc, int splits, uint64_t* __restrict__ keys,
                                                    PieceSum* __restrict__ sums) {
    constexpr int N = Wide<T>::N, kWaves = NT / 64;
    __shared__ uint64_t red[kWaves];
    __shared__ double red_sum[kWaves];
    const int wave = threadIdx.x >> 6;
    for (int64_t item = blockIdx.x; item < rows * splits; item += gridDim.x) {
        const int64_t r = item / splits;
        if (!b.counts(r) || b.has_ended(r)) continue;
        const T* x = logits + r * ld;
        const Piece<T> w(x, (int)(item - r * splits), Chunk<T, NT, U>::kSize, vocab);
        Chunk<T, NT, U> c;
        c.load(x, w.from, w.to);
        const int ke = w.edge();
        const float xe = ke >= 0 ? (float)x[ke] : -INFINITY;
        uint64_t last = ~0ull;
        float m = -INFINITY;
        for (int i = 0; i < b.take; ++i) {
            uint64_t best = token_key(xe, ke);
            if (best >= last) best = 0;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const uint64_t k = token_key((float)c.v[u][j], c.at(w.from, u) + j);
                    best = k < last && k > best ? k : best;
                }
            best = wave_max(best);
            if ((threadIdx.x & 63) == 0) red[wave] = best;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kWaves; ++k) best = red[k] > best ? red[k] : best;
            __syncthreads();
            if (i == 0 && best) m = key_logit(best);
            if (threadIdx.x == 0) keys[item * b.take + i] = best;
            last = best;  // 0: nothing is below it
        }
        const float base = m == -INFINITY ? 0.0f : m;
        double s = (double)__builtin_amdgcn_exp2f((xe - base) * sc.cf);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < N; ++j) s += (double)__builtin_amdgcn_exp2f(((float)c.v[u][j] - base) * sc.cf);
        s = wg_sum<NT>(s, red_sum);
        if (threadIdx.x == 0) sums[item] = PieceSum{(double)m, s};
    }
}

// A batch item: its rows' log-sums, then its best candidates, one round of a
// maximum each, by (rank, lower beam; logit, lower token).
struct Cand {
    uint64_t hi, lo;
    __device__ __forceinline__ bool over(const Cand& o) const { return hi > o.hi || (hi == o.hi && lo > o.lo); }
};
struct RowSum {
    double m, log_s, score, weight;
    int state;  // 0: no candidates, 1: its tokens, 2: itself
};
constexpr int kJoinNT = 256;
__global__ __launch_bounds__(kJoinNT) void k_beam_join(int64_t batch, Beams b, Scale sc, int splits,
                                                       const uint64_t* __restrict__ keys,
                                                       const PieceSum* __restrict__ sums, float* __restrict__ out_score,
                                                       float* __restrict__ out_logp, int32_t* __restrict__ out_parent,
                                                       int32_t* __restrict__ out_token) {
    __shared__ RowSum row[kMaxBeams];
    __shared__ Cand red[kJoinNT / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t item = blockIdx.x; item < batch; item += gridDim.x) {
        for (int k = wave; k < b.beams; k += kJoinNT / 64) {
            const int64_t r = item * b.beams + k;
            RowSum o{0.0, 0.0, (double)b.score[r], b.weight ? (double)b.weight[r] : 1.0, 0};
            if (b.counts(r) && b.has_ended(r)) o.state = 2;
            else if (b.counts(r)) {
                double m = -INFINITY;
                for (int p = lane; p < splits; p += 64) m = fmax(m, sums[r * splits + p].m);
#pragma unroll
                for (int d = 32; d > 0; d >>= 1) m = fmax(m, __shfl_xor(m, d));
                double s = 0.0;
                for (int p = lane; p < splits; p += 64) {
                    const PieceSum a = sums[r * splits + p];
                    s += a.m == -INFINITY ? a.s : a.s * exp((a.m - m) * sc.inv_t);
                }
                s = wave_sum(s);
                if (s > 0.0 && s < INFINITY) {
                    o.m = m;
                    o.log_s = log(s);
                    o.state = 1;
                }
            }
            if (lane == 0) row[k] = o;
        }
        __syncthreads();
        Cand last{~0ull, ~0ull};
        const int each = splits * b.take;
        for (int i = 0; i < b.take; ++i) {
            Cand best{0, 0};
            for (int64_t e = threadIdx.x; e < (int64_t)b.beams * each; e += kJoinNT) {
                const int k = (int)(e / each);
                const RowSum& o = row[k];
                if (o.state == 0 || (o.state == 2 && e - (int64_t)k * each)) continue;
                const uint64_t key = o.state == 2 ? 0 : keys[item * b.beams * each + e];
                if (o.state == 1 && !key) continue;
                const double logp = o.state == 2 ? 0.0 : ((double)key_logit(key) - o.m) * sc.inv_t - o.log_s;
                const float rank = (float)((o.score + logp) * o.weight);
                if (!(rank > -INFINITY)) continue;
                const Cand c{((uint64_t)ordered(rank) << 32) | (uint32_t)(kMaxBeams - k), key};
                if (last.over(c) && c.over(best)) best = c;
            }
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) {
                const Cand o{(uint64_t)__shfl_xor((unsigned long long)best.hi, d),
                             (uint64_t)__shfl_xor((unsigned long long)best.lo, d)};
                if (o.over(best)) best = o;
            }
            if (lane == 0) red[wave] = best;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kJoinNT / 64; ++k)
                if (red[k].over(best)) best = red[k];
            __syncthreads();
            if (threadIdx.x == 0) {
                const int64_t at = item * b.take + i;
                if (best.hi) {
                    const int k = kMaxBeams - (int)(uint32_t)best.hi;
                    const RowSum& o = row[k];
                    const double logp = o.state == 2 ? 0.0 : ((double)key_logit(best.lo) - o.m) * sc.inv_t - o.log_s;
                    out_score[at] = (float)(o.score + logp);
                    out_logp[at] = (float)logp;
                    out_parent[at] = (int32_t)(item * b.beams + k);
                    out_token[at] = o.state == 2 ? b.end_token : key_token(best.lo);
                } else {
                    out_score[at] = out_logp[at] = -INFINITY;
                    out_parent[at] = out_token[at] = -1;
                }
            }
            last = best;
        }
        __syncthreads();  // row is used again
    }
}

constexpr int kPieceNT = 256, kPieceU = 4;
struct SelectPlan {
    int splits;
    size_t off_sums, bytes;
};
SelectPlan select_plan(int64_t batch, int64_t beams, int64_t vocab, int64_t take, int dtype) {
    const int64_t chunk = (int64_t)kPieceNT * kPieceU * 16 / (int64_t)size_of(dtype);
    SelectPlan p;
    p.splits = (int)((vocab + chunk - 1) / chunk);
    const size_t items = (size_t)(batch * beams) * (size_t)p.splits;
    p.off_sums = align_up(items * (size_t)take * sizeof(uint64_t));
    p.bytes = p.off_sums + align_up(items * sizeof(PieceSum));
    return p;
}

bool select_sizes_ok(int64_t batch, int64_t beams, int64_t vocab, int64_t take, int dtype) {
    return batch >= 0 && beams >= 1 && beams <= kMaxBeams && take >= 1 && take <= kMaxTake && vocab >= 1 &&
           vocab <= (1LL << 30) && batch <= 0x7fffffffLL / beams && dtype >= ISO_DT_F32 && dtype <= ISO_DT_BF16;
}

// Item = (array, batch item, outer, 256 vectors of 16 bytes): a thread has one
// column of them through all rows of the item, and reads what rows come from
// before it writes any.
constexpr int kReorderNT = 256;
template <typename V>
__device__ void reorder_column(char* at, int64_t row_stride, const int32_t* from, int beams) {
    V v[kMaxBeams];
    for (int k = 0; k < beams; ++k)
        if (from[k] >= 0) v[k] = *reinterpret_cast<const V*>(at + from[k] * row_stride);
    for (int k = 0; k < beams; ++k)
        if (from[k] >= 0) *reinterpret_cast<V*>(at + k * row_stride) = v[k];
}
__global__ __launch_bounds__(kReorderNT) void k_beam_reorder(States st, const int32_t* __restrict__ parent,
                                                             int64_t batch, int beams) {
    __shared__ int32_t from[kMaxBeams];
    for (int i = 0; i < st.count; ++i) {
        const iso_blocks& s = st.b[i];
        const int64_t cols = (s.inner + 15) / 16, tiles = (s.mid * cols + kReorderNT - 1) / kReorderNT;
        const int64_t items = batch * s.outer * tiles;
        for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
            const int64_t b = item / (s.outer * tiles), o = item / tiles % s.outer, t = item % tiles;
            __syncthreads();
            if (threadIdx.x < beams) {
                const int64_t p = (int64_t)parent[b * beams + threadIdx.x] - b * beams;
                from[threadIdx.x] = p >= 0 && p < beams && p != (int)threadIdx.x ? (int32_t)p : -1;
            }
            __syncthreads();
            const int64_t col = t * kReorderNT + threadIdx.x;
            if (col >= s.mid * cols) continue;
            const int64_t m = col / cols, c = col % cols;
            char* at = static_cast<char*>(s.base) + o * s.outer_stride + b * beams * s.row_stride + m * s.mid_stride + c * 16;
            const int left = (int)(s.inner - c * 16 < 16 ? s.inner - c * 16 : 16);
            if (left == 16) {
                reorder_column<Wide16>(at, s.row_stride, from, beams);
                continue;
            }
            if (left & 8) reorder_column<Wide8>(at, s.row_stride, from, beams);
            if (left & 4) reorder_column<Wide4>(at + (left & 8), s.row_stride, from, beams);
            if (left & 2) reorder_column<Wide2>(at + (left & 12), s.row_stride, from, beams);
            if (left & 1) reorder_column<uint8_t>(at + (left & 14), s.row_stride, from, beams);
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
    const int64_t items = rows * pl.splits;
    by_dtype(dtype, [&](auto v) {
        typedef decltype(v) T;
        hipLaunchKernelGGL((k_beam_pieces<T, kPieceNT, kPieceU>), dim3((unsigned)(items < kMaxGrid ? items : kMaxGrid)),
                           dim3(kPieceNT), 0, st, static_cast<const T*>(logits), rows, (int)vocab, ld, b, sc, pl.splits,
                           keys, sums);
    });
    hipLaunchKernelGGL(k_beam_join, dim3((unsigned)(batch < kMaxGrid ? batch : kMaxGrid)), dim3(kJoinNT), 0, st, batch, b,
                       sc, pl.splits, keys, sums, out_score, out_logp, out_parent, out_token);
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

int iso_beam_reorder(const iso_blocks* states, int count, const int32_t* parent, int64_t batch, int64_t beams,
                     void* stream) {
    using namespace iso;
    if (batch < 0 || beams < 1 || beams > kMaxBeams || batch > 0x7fffffffLL / beams) return ISO_ERR_ARG;
    const int64_t rows = batch * beams;
    const Span other[] = {{parent, (size_t)rows * 4}};
    States st;
    if (!take_states(states, count, rows, other, st)) return ISO_ERR_ARG;
    if (rows && !parent) return ISO_ERR_ARG;
    if (!aligned(parent, 4)) return ISO_ERR_ARG;
    if (!st.count) return ISO_OK;
    int64_t most = 1;
    for (int i = 0; i < st.count; ++i) {
        const iso_blocks& s = st.b[i];
        const int64_t cols = (s.inner + 15) / 16;
        if (s.mid > (1LL << 40) / cols) return ISO_ERR_ARG;
        const int64_t tiles = (s.mid * cols + kReorderNT - 1) / kReorderNT;
        if (s.outer > (1LL << 40) / tiles || batch > (1LL << 60) / (s.outer * tiles)) return ISO_ERR_ARG;
        const int64_t items = batch * s.outer * tiles;
        most = items > most ? items : most;
    }
    hipLaunchKernelGGL(k_beam_reorder, dim3((unsigned)(most < kMaxGrid ? most : kMaxGrid)), dim3(kReorderNT), 0,
                       static_cast<hipStream_t>(stream), st, parent, batch, (int)beams);
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

}  // extern "C"
