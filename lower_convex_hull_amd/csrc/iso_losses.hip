// Losses over tokens' log-probabilities, with their gradients: the paired
// preference loss and the clipped policy loss with a KL term (formulas in
// iso.h).  Both are sums over sequences of tokens followed by one value per
// token; every sum is f64, without atomics.
#include "../../include/iso.h"
#include "iso_losses.hpp"

namespace iso {
namespace {

constexpr int kLossNT = 256;

__device__ __forceinline__ bool live_at(const uint8_t* mask, const int32_t* target, int64_t t) {
    return (!mask || mask[t] != 0) && (!target || target[t] >= 0);
}

// ---- preference loss ----

struct Pref {
    const float* logp;
    const float* ref;  // or NULL
    const uint8_t* mask;
    double beta, smooth;
    bool mean, squared;
    double grad_scale;
};

// -log sigma(h), without overflow for either sign.
__device__ __forceinline__ double softplus_neg(double h) { return fmax(-h, 0.0) + log1p(exp(-fabs(h))); }

// One workgroup a pair: the two sums, the pair's loss, then its tokens' gradient.
__global__ __launch_bounds__(kLossNT) void k_pref_pairs(Pref p, Seqs sq, int64_t pairs, float* pair_loss,
                                                        float* reward, float* grad, double* part) {
    __shared__ double red[kLossNT / 64];
    const int64_t i = blockIdx.x;
    double s[2], share[2];
    for (int k = 0; k < 2; ++k) {
        const int64_t b = sq.begin(2 * i + k), e = sq.end(2 * i + k);
        double v = 0.0, c = 0.0;
        for (int64_t t = b + threadIdx.x; t < e; t += kLossNT) {
            if (live_at(p.mask, nullptr, t)) {
                v += (double)p.logp[t] - (p.ref ? (double)p.ref[t] : 0.0);
                c += 1.0;
            }
        }
        s[k] = wg_sum<kLossNT>(v, red);
        c = wg_sum<kLossNT>(c, red);
        share[k] = p.mean ? 1.0 / fmax(c, 1.0) : 1.0;
        s[k] *= share[k];
    }
    const double delta = s[0] - s[1];
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
    if (threadIdx.x == 0) {
        part[i] = loss;
        pair_loss[i] = (float)loss;
        reward[2 * i] = (float)(p.beta * s[0]);
        reward[2 * i + 1] = (float)(p.beta * s[1]);
    }
    if (!grad) return;
    slope *= p.grad_scale / (double)pairs;
    for (int k = 0; k < 2; ++k) {
        const int64_t b = sq.begin(2 * i + k), e = sq.end(2 * i + k);
        const float c = (float)((k ? -slope : slope) * share[k]);
        for (int64_t t = b + threadIdx.x; t < e; t += kLossNT) grad[t] = live_at(p.mask, nullptr, t) ? c : 0.0f;
    }
}

__global__ __launch_bounds__(kLossNT) void k_pref_mean(const double* __restrict__ part, int64_t pairs, float* loss) {
    __shared__ double red[kLossNT / 64];
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < pairs; i += kLossNT) v += part[i];
    v = wg_sum<kLossNT>(v, red);
    if (threadIdx.x == 0) *loss = pairs ? (float)(v / (double)pairs) : 0.0f;
}

// ---- policy loss ----

struct PolicyPart {
    double pg, kl;
    int64_t live, over;
};

// Live tokens of each sequence.
__global__ __launch_bounds__(kLossNT) void k_policy_count(const uint8_t* mask, const int32_t* target, Seqs sq,
                                                          PolicyPart* part) {
    __shared__ double red[kLossNT / 64];
    const int64_t q = blockIdx.x;
    const int64_t b = sq.begin(q), e = sq.end(q);
    double c = 0.0;
    for (int64_t t = b + threadIdx.x; t < e; t += kLossNT) c += live_at(mask, target, t) ? 1.0 : 0.0;
    c = wg_sum<kLossNT>(c, red);
    if (threadIdx.x == 0) part[q].live = (int64_t)c;
}

__global__ __launch_bounds__(kLossNT) void k_policy_total(const PolicyPart* part, int64_t seqs, int64_t* total) {
    __shared__ double red[kLossNT / 64];
    double c = 0.0;
    for (int64_t q = threadIdx.x; q < seqs; q += kLossNT) c += (double)part[q].live;
    c = wg_sum<kLossNT>(c, red);
    if (threadIdx.x == 0) *total = (int64_t)c;
}

template <typename LP>
__global__ __launch_bounds__(kLossNT) void k_policy_tokens(Policy p, const LP* logp, const uint8_t* mask,
                                                           const int32_t* target, Seqs sq, const int64_t* total,
                                                           PolicyPart* part, float* grad) {
    __shared__ double red[kLossNT / 64];
    const int64_t q = blockIdx.x;
    const int64_t b = sq.begin(q), e = sq.end(q);
    double w;
    if (p.seq_mean) w = 1.0 / ((p.norm > 0.0 ? p.norm : (double)sq.n) * fmax((double)part[q].live, 1.0));
    else w = 1.0 / (p.norm > 0.0 ? p.norm : fmax((double)*total, 1.0));
    double pg = 0.0, kl = 0.0, over = 0.0;
    for (int64_t t = b + threadIdx.x; t < e; t += kLossNT) {
        float g = 0.0f;
        if (live_at(mask, target, t)) {
            const PolicyTerm o = policy_term(p, (double)logp[t], t, (double)p.adv[p.token_adv ? t : q]);
            pg += o.pg;
            kl += o.kl;
            over += o.over ? 1.0 : 0.0;
            g = (float)(o.slope * w * p.grad_scale);
        }
        if (grad) grad[t] = g;
    }
    pg = wg_sum<kLossNT>(pg, red);
    kl = wg_sum<kLossNT>(kl, red);
    over = wg_sum<kLossNT>(over, red);
    if (threadIdx.x == 0) {
        part[q].pg = pg * w;
        part[q].kl = kl * w;
        part[q].over = (int64_t)over;
    }
}

__global__ __launch_bounds__(kLossNT) void k_policy_sum(const PolicyPart* part, const int64_t* total, int64_t seqs,
                                                        double kl_coef, float* loss, int32_t* counts) {
    __shared__ double red[kLossNT / 64];
    double pg = 0.0, kl = 0.0, over = 0.0;
    for (int64_t q = threadIdx.x; q < seqs; q += kLossNT) {
        pg += part[q].pg;
        kl += part[q].kl;
        over += (double)part[q].over;
    }
    pg = wg_sum<kLossNT>(pg, red);
    kl = wg_sum<kLossNT>(kl, red);
    over = wg_sum<kLossNT>(over, red);
    if (threadIdx.x == 0) {
        loss[0] = (float)(kl_coef != 0.0 ? pg + kl_coef * kl : pg);
        loss[1] = (float)pg;
        loss[2] = (float)kl;
        counts[0] = (int32_t)*total;
        counts[1] = (int32_t)over;
    }
}

bool seqs_ok(const int32_t* off, int64_t seqs, int64_t tokens) {
    if (seqs < 0 || tokens < 0 || tokens > 0x7fffffffLL || seqs > 0x7fffffffLL) return false;
    if (!aligned(off, 4)) return false;
    if (!off && (seqs ? tokens % seqs != 0 : tokens != 0)) return false;
    return true;
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
    if (tokens < 0 || seqs < 0) return 0;
    return 256 + (size_t)seqs * sizeof(PolicyPart);
}

template <typename LP>
hipError_t launch_policy(const Policy& p, const LP* logp, const uint8_t* mask, const int32_t* target,
                         const Seqs& sq, float* loss, int32_t* counts, float* grad, void* workspace,
                         hipStream_t st) {
    int64_t* total = static_cast<int64_t*>(workspace);
    PolicyPart* part = reinterpret_cast<PolicyPart*>(static_cast<char*>(workspace) + 256);
    const dim3 nt(kLossNT);
    if (sq.n) hipLaunchKernelGGL(k_policy_count, dim3((unsigned)sq.n), nt, 0, st, mask, target, sq, part);
    hipLaunchKernelGGL(k_policy_total, dim3(1), nt, 0, st, part, sq.n, total);
    if (sq.n)
        hipLaunchKernelGGL((k_policy_tokens<LP>), dim3((unsigned)sq.n), nt, 0, st, p, logp, mask, target, sq, total,
                           part, grad);
    hipLaunchKernelGGL(k_policy_sum, dim3(1), nt, 0, st, part, total, sq.n, p.kl_coef, loss, counts);
    return hipGetLastError();
}
template hipError_t launch_policy<float>(const Policy&, const float*, const uint8_t*, const int32_t*, const Seqs&,
                                         float*, int32_t*, float*, void*, hipStream_t);
template hipError_t launch_policy<double>(const Policy&, const double*, const uint8_t*, const int32_t*, const Seqs&,
                                          float*, int32_t*, float*, void*, hipStream_t);

}  // namespace iso

extern "C" {

size_t iso_pref_loss_workspace_bytes(int64_t tokens, int64_t pairs) {
    if (tokens < 0 || pairs < 0) return 0;
    return (size_t)pairs * sizeof(double);
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
    const Pref p{logp, ref_logp, mask, beta, label_smoothing, (flags & ISO_PREF_MEAN) != 0,
                 (flags & ISO_PREF_SQUARED) != 0, grad_scale};
    const Seqs sq{seq_off, 2 * pairs, tokens, pairs ? tokens / (2 * pairs) : 0};
    double* part = static_cast<double*>(workspace);
    if (pairs)
        hipLaunchKernelGGL(k_pref_pairs, dim3((unsigned)pairs), dim3(kLossNT), 0, st, p, sq, pairs, pair_loss,
                           reward, grad, part);
    hipLaunchKernelGGL(k_pref_mean, dim3(1), dim3(kLossNT), 0, st, part, pairs, loss);
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
