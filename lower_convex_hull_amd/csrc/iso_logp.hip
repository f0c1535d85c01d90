// Token log-probabilities from logits, their backward pass, and the policy loss
// taken from the logits (formulas in iso.h).  A row of logits is one token's;
// logits are f32, f16 or bf16 and everything is computed in f32 from the
// difference to the row's maximum (exact, or nearly, in f32), joined in f64.
#include "../../include/iso.h"
#include "iso_losses.hpp"

namespace iso {
namespace {

constexpr int kRowNT = 256;
constexpr double kLog2e = 1.4426950408889634;

// Per-row statistics of x over some of its entries: the maximum m, s = sum
// exp((x - m)/T) and h = sum exp((x - m)/T) (x - m)/T.
struct Stat {
    float m;
    double s, h;
};

// exp((x - m)/T) with c = log2(e)/T.  m is finite or +infinity (base_of).
__device__ __forceinline__ float exp_of(float d, float c) { return __builtin_amdgcn_exp2f(d * c); }

// The maximum that differences are taken to: 0 where everything so far is
// -infinity, so that no -infinity minus -infinity arises.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

// A difference to the maximum as a factor of h: a masked entry's -infinity is
// held finite, its product with exp(-infinity) = 0 is then 0.
__device__ __forceinline__ float held(float d) { return fmaxf(d, -1e30f); }

// a and b of the same row joined.
template <bool ENT>
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, double inv_t) {
    Stat o;
    o.m = fmaxf(a.m, b.m);
    const float base = base_of(o.m);
    // where one side holds nothing but -infinity, its sums are 0
    const double da = (double)held(base_of(a.m) - base) * inv_t, db = (double)held(base_of(b.m) - base) * inv_t;
    const double fa = a.m == -INFINITY ? 1.0 : exp(da), fb = b.m == -INFINITY ? 1.0 : exp(db);
    o.s = a.s * fa + b.s * fb;
    o.h = ENT ? (a.h + (a.m == -INFINITY ? 0.0 : a.s * da)) * fa + (b.h + (b.m == -INFINITY ? 0.0 : b.s * db)) * fb
              : 0.0;
    return o;
}

template <typename T>
__device__ __forceinline__ T nan_of() {
    return (T)__builtin_nanf("");
}

// A row's outputs from its statistics: lse and entropy.
__device__ __forceinline__ void finish_row(const Stat& r, double inv_t, double& lse, double& ent) {
    // nothing but -infinity: s = 0 against base 0
    const bool none = r.m == -INFINITY;
    const double ls = log(r.s);
    lse = none ? __builtin_nan("") : (double)r.m * inv_t + ls;
    ent = none ? __builtin_nan("") : ls - r.h / r.s;
}

// One workgroup a row.
template <typename T, bool ENT>
__global__ __launch_bounds__(kRowNT) void k_token_logp(const T* __restrict__ logits, int64_t vocab, int64_t ld,
                                                       const int32_t* __restrict__ target, double inv_t, float c,
                                                       float* __restrict__ logp, float* __restrict__ lse,
                                                       float* __restrict__ ent, double* __restrict__ logp64,
                                                       double* __restrict__ lse64) {
    __shared__ Stat part[kRowNT / 64];
    const int64_t r = blockIdx.x;
    const int32_t j = target[r];
    if (j < 0) {
        if (threadIdx.x == 0) {
            logp[r] = 0.0f;
            if (lse) lse[r] = 0.0f;
            if (ENT) ent[r] = 0.0f;
            if (logp64) logp64[r] = 0.0, lse64[r] = 0.0;
        }
        return;
    }
    const T* x = logits + r * ld;
    float m = -INFINITY;
    bool bad = false;
    for (int64_t k = threadIdx.x; k < vocab; k += kRowNT) {
        const float v = (float)x[k];
        m = fmaxf(m, v);
        bad |= v != v;
    }
    const float base = base_of(m);
    double s = 0.0, h = 0.0;
    for (int64_t k = threadIdx.x; k < vocab; k += kRowNT) {
        const float d = (float)x[k] - base;
        const float e = exp_of(d, c);
        s += (double)e;
        if (ENT) h += (double)(e * held(d)) * inv_t;
    }
    Stat a{m, bad ? (double)__builtin_nanf("") : s, h};
    for (int d = 32; d > 0; d >>= 1) {
        const Stat b{__shfl_xor(a.m, d), __shfl_xor(a.s, d), __shfl_xor(a.h, d)};
        a = join<ENT>(a, b, inv_t);
    }
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < kRowNT / 64; ++k) a = join<ENT>(a, part[k], inv_t);
        double l, en;
        finish_row(a, inv_t, l, en);
        const double lp = j < vocab ? (double)(float)x[j] * inv_t - l : __builtin_nan("");
        logp[r] = (float)lp;
        if (lse) lse[r] = (float)l;
        if (ENT) ent[r] = (float)en;
        if (logp64) logp64[r] = lp, lse64[r] = l;
    }
}

// One workgroup a row of the gradient.  With z = x/T - lse: p = exp(z), taken
// as exp((x - mh)/T) times a factor of the row, mh = lse T rounded to f32.
template <typename T, bool ENT, typename LSE>
__global__ __launch_bounds__(kRowNT) void k_logp_vjp(const T* logits, int64_t vocab, int64_t ld,
                                                     const int32_t* __restrict__ target, double inv_t, float c,
                                                     const LSE* __restrict__ lse, const float* __restrict__ ent,
                                                     const float* __restrict__ g_logp,
                                                     const float* __restrict__ g_ent, T* grad, int64_t ldg) {
    const int64_t r = blockIdx.x;
    const int32_t j = target[r];
    const T* x = logits + r * ld;
    T* o = grad + r * ldg;
    if (j < 0 || j >= vocab) {
        const T v = j < 0 ? (T)0.0f : nan_of<T>();
        for (int64_t k = threadIdx.x; k < vocab; k += kRowNT) o[k] = v;
        return;
    }
    const double l = (double)lse[r], g = (double)g_logp[r];
    const float mh = (float)(l / inv_t);
    const double off = (double)mh * inv_t - l;  // x/T - lse = (x - mh)/T + off
    const double f = exp(off) * inv_t;
    const double gh = ENT ? (double)g_ent[r] : 0.0;
    const float a = (float)(-(g + (ENT ? gh * ((double)ent[r] + off) : 0.0)) * f);
    const float b = ENT ? (float)(-gh * inv_t * f) : 0.0f;
    const float hot = (float)(g * inv_t);
    for (int64_t k = threadIdx.x; k < vocab; k += kRowNT) {
        const float d = (float)x[k] - mh;
        const float p = exp_of(d, c);
        float v = ENT ? p * (a + b * held(d)) : p * a;
        if (k == j) v += hot;
        o[k] = (T)v;
    }
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

size_t size_of(int dtype) { return dtype == ISO_DT_F32 ? 4 : 2; }

bool logits_ok(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld, double temperature) {
    if (dtype != ISO_DT_F32 && dtype != ISO_DT_F16 && dtype != ISO_DT_BF16) return false;
    if (rows < 0 || rows > 0x7fffffffLL || vocab < 1 || vocab > (1LL << 30) || ld < vocab) return false;
    if (rows && ld > INT64_MAX / 16 / rows) return false;
    if (!(temperature > 0.0) || !isfinite(temperature)) return false;
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

template <typename T>
void start_logp(const void* logits, int64_t rows, int64_t vocab, int64_t ld, const int32_t* target,
                double temperature, float* logp, float* lse, float* ent, double* logp64, double* lse64,
                hipStream_t st) {
    const double inv_t = 1.0 / temperature;
    const float c = (float)(kLog2e * inv_t);
    const T* x = static_cast<const T*>(logits);
    const dim3 grid((unsigned)rows), nt(kRowNT);
    if (ent)
        hipLaunchKernelGGL((k_token_logp<T, true>), grid, nt, 0, st, x, vocab, ld, target, inv_t, c, logp, lse, ent,
                           logp64, lse64);
    else
        hipLaunchKernelGGL((k_token_logp<T, false>), grid, nt, 0, st, x, vocab, ld, target, inv_t, c, logp, lse, ent,
                           logp64, lse64);
}

template <typename T, typename LSE>
void start_vjp(const void* logits, int64_t rows, int64_t vocab, int64_t ld, const int32_t* target,
               double temperature, const LSE* lse, const float* ent, const float* g_logp, const float* g_ent,
               void* grad, int64_t ldg, hipStream_t st) {
    const double inv_t = 1.0 / temperature;
    const float c = (float)(kLog2e * inv_t);
    const T* x = static_cast<const T*>(logits);
    T* o = static_cast<T*>(grad);
    const dim3 grid((unsigned)rows), nt(kRowNT);
    if (g_ent)
        hipLaunchKernelGGL((k_logp_vjp<T, true, LSE>), grid, nt, 0, st, x, vocab, ld, target, inv_t, c, lse, ent,
                           g_logp, g_ent, o, ldg);
    else
        hipLaunchKernelGGL((k_logp_vjp<T, false, LSE>), grid, nt, 0, st, x, vocab, ld, target, inv_t, c, lse, ent,
                           g_logp, g_ent, o, ldg);
}

// f called with a value of the logits' type.
template <typename F>
void by_dtype(int dtype, F f) {
    if (dtype == ISO_DT_F32) f(float{});
    else if (dtype == ISO_DT_F16) f(_Float16{});
    else f(__bf16{});
}

// Workspace of iso_policy_loss_logits.
struct HeadPlan {
    size_t off_lp, off_lse, off_g, off_policy, bytes;
};
HeadPlan head_plan(int64_t rows, int64_t seqs) {
    HeadPlan p;
    const size_t n = (size_t)rows;
    p.off_lp = 0;
    p.off_lse = align_up(n * 8);
    p.off_g = p.off_lse + align_up(n * 8);
    p.off_policy = p.off_g + align_up(n * 4);
    p.bytes = p.off_policy + policy_workspace(rows, seqs);
    return p;
}

}  // namespace
}  // namespace iso

extern "C" {

size_t iso_token_logp_workspace_bytes(int64_t rows, int64_t vocab, int dtype) {
    (void)rows;
    (void)vocab;
    (void)dtype;
    return 0;
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
        start_logp<decltype(v)>(logits, rows, vocab, ld, target, temperature, logp, lse, entropy, nullptr, nullptr,
                                st);
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
    (void)vocab;
    (void)dtype;
    if (rows < 0 || seqs < 0) return 0;
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
    double* lp64 = reinterpret_cast<double*>(ws + pl.off_lp);
    double* lse64 = reinterpret_cast<double*>(ws + pl.off_lse);
    float* g = reinterpret_cast<float*>(ws + pl.off_g);
    const Policy p = make_policy(old_logp, ref_logp, adv, clip_lo, clip_hi, kl_coef, norm, grad_scale, flags);
    const Seqs sq{seq_off, seqs, rows, seqs ? rows / seqs : 0};
    if (rows)
        by_dtype(dtype, [&](auto v) {
            start_logp<decltype(v)>(logits, rows, vocab, ld, target, temperature, logp, nullptr, nullptr, lp64, lse64,
                                    st);
        });
    if (launch_policy<double>(p, lp64, nullptr, target, sq, loss, counts, grad ? g : nullptr, ws + pl.off_policy,
                              st) != hipSuccess)
        return ISO_ERR_HIP;
    if (rows && grad)
        by_dtype(dtype, [&](auto v) {
            start_vjp<decltype(v)>(logits, rows, vocab, ld, target, temperature, lse64, nullptr, g, nullptr, grad,
                                   ld_grad, st);
        });
    return hipGetLastError() == hipSuccess ? ISO_OK : ISO_ERR_HIP;
}

}  // extern "C"
