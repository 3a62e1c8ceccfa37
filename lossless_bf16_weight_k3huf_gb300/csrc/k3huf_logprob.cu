// Log probabilities of given tokens with entropy and top alternatives, and
// their gradient with respect to the logits.
//
// With z = s x the scaled logits of a row, m its largest and e_j = exp(z_j - m):
//   lse  = m + log sum_j e_j
//   logprob = (z_token - m) - log sum_j e_j
//   entropy = log sum_j e_j - (sum_j e_j (z_j - m)) / sum_j e_j
//   top: the largest logits, ties to the lower index
// and, for upstream gradients g of logprob and h of entropy, p_j = exp(z_j - lse):
//   dx_j = s (g (1[j = token] - p_j) - h p_j (log p_j + entropy))
// Logits of -infinity take no part (p_j = 0).  One CTA takes a row.
#include <cmath>

#include "k3huf_ops.h"

namespace k3huf {
namespace {

constexpr int kThreads = 256;

// (value, index) order of the top alternatives: larger values first, ties to
// the lower index.  A value's order as a whole number; +0 and -0 are equal
// and a NaN sorts by its bits.
__device__ __forceinline__ int32_t order_of(float x) {
    const int32_t b = __float_as_int(x + 0.f);
    return b < 0 ? b ^ 0x7FFFFFFF : b;
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t j) {
    return (uint64_t(uint32_t(order_of(x)) ^ 0x80000000u) << 32) | (0xFFFFFFFFu - j);
}

struct LogprobParams {
    const void *x;
    const void *tokens;
    float *logprob, *entropy, *lse, *top_logprobs;
    int32_t *top_ids;
    uint32_t *status;
    uint64_t stride;
    uint32_t n, vocab, id_bytes, top;
    float scale;
};

template <typename T, typename F>
__device__ T block_reduce(T v, F f, T *buf) {
    __syncthreads();
    buf[threadIdx.x] = v;
    __syncthreads();
    for (int d = kThreads / 2; d; d >>= 1) {
        if (threadIdx.x < d) buf[threadIdx.x] = f(buf[threadIdx.x], buf[threadIdx.x + d]);
        __syncthreads();
    }
    return buf[0];
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_kernel(const LogprobParams P) {
    __shared__ float s_f[kThreads];
    __shared__ uint64_t s_k[kThreads];
    const uint32_t row = blockIdx.x;
    const T *x = static_cast<const T *>(P.x) + uint64_t(row) * P.stride;
    float m = -INFINITY;
    for (uint32_t j = threadIdx.x; j < P.vocab; j += kThreads) m = fmaxf(m, ld_f32(x + j) * P.scale);
    m = block_reduce(m, [](float a, float b) { return fmaxf(a, b); }, s_f);
    float sum = 0.f, dot = 0.f;
    const float shift = m == -INFINITY ? 0.f : m;          // (a row with no finite logit: every e is 0)
    for (uint32_t j = threadIdx.x; j < P.vocab; j += kThreads) {
        const float z = ld_f32(x + j) * P.scale, e = expf(z - shift);
        sum += e;
        dot += e == 0.f ? 0.f : e * (z - shift);           // (0 times infinity)
    }
    auto add = [](float a, float b) { return a + b; };
    sum = block_reduce(sum, add, s_f);
    dot = block_reduce(dot, add, s_f);
    const float logsum = logf(sum), lse = shift + logsum;  // (-infinity for such a row)
    if (threadIdx.x == 0) {
        const int64_t t = ld_id(P.tokens, P.id_bytes, row);
        float lp = 0.f;
        if (t >= int64_t(P.vocab)) atomicOr(P.status, K3HUF_ST_TOKEN);
        else if (t >= 0) {
            const float z = ld_f32(x + t) * P.scale;
            lp = z == -INFINITY ? z : (z - shift) - logsum;
        }
        P.logprob[row] = lp;
        if (P.entropy) P.entropy[row] = sum > 0.f ? logsum - dot / sum : sum;
        if (P.lse) P.lse[row] = lse;
    }
    uint64_t below = ~0ull;
    for (uint32_t k = 0; k < P.top; ++k) {
        uint64_t best = 0;
        for (uint32_t j = threadIdx.x; j < P.vocab; j += kThreads) {
            const uint64_t key = key_of(ld_f32(x + j), j);
            if (key < below && key > best) best = key;
        }
        below = block_reduce(best, [](uint64_t a, uint64_t b) { return a > b ? a : b; }, s_k);
        if (threadIdx.x == 0) {
            const uint32_t j = 0xFFFFFFFFu - uint32_t(below);
            const float z = ld_f32(x + j) * P.scale;
            P.top_ids[uint64_t(row) * P.top + k] = int32_t(j);
            P.top_logprobs[uint64_t(row) * P.top + k] = z == -INFINITY ? z : (z - shift) - logsum;
        }
    }
}

struct GradParams {
    const void *x;
    void *dx;
    const void *tokens;
    const float *lse, *entropy, *g_logprob, *g_entropy;
    uint32_t *status;
    uint64_t stride, dx_stride;
    uint32_t n, vocab, id_bytes;
    float scale;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_grad_kernel(const GradParams P) {
    const uint32_t row = blockIdx.x;
    const T *x = static_cast<const T *>(P.x) + uint64_t(row) * P.stride;
    T *dx = static_cast<T *>(P.dx) + uint64_t(row) * P.dx_stride;
    const int64_t t = ld_id(P.tokens, P.id_bytes, row);
    if (t >= int64_t(P.vocab) && threadIdx.x == 0) atomicOr(P.status, K3HUF_ST_TOKEN);
    const float g = t >= 0 && t < int64_t(P.vocab) ? P.g_logprob[row] : 0.f;
    const float h = P.g_entropy ? P.g_entropy[row] : 0.f, ent = P.g_entropy ? P.entropy[row] : 0.f, lse = P.lse[row];
    for (uint32_t j = threadIdx.x; j < P.vocab; j += kThreads) {
        const float z = ld_f32(x + j) * P.scale, lp = z == -INFINITY ? z : z - lse, p = expf(lp);
        const float d = p == 0.f ? 0.f : -p * (g + h * (lp + ent));   // (0 times infinity)
        st_f32(dx + j, P.scale * (d + (int64_t(j) == t ? g : 0.f)));
    }
}

}  // namespace
}  // namespace k3huf

using namespace k3huf;

extern "C" int k3huf_token_logprobs(const void *d_logits, uint32_t type, uint64_t stride, uint64_t n, uint32_t vocab, float scale,
                                    const void *d_tokens, uint32_t id_bytes, float *d_logprob, float *d_entropy, float *d_lse,
                                    uint32_t top, int32_t *d_top_ids, float *d_top_logprobs, uint32_t *d_status, void *stream) {
    if (!elem_ok(type) || (id_bytes != 4 && id_bytes != 8) || vocab == 0 || vocab > 0x7FFFFFFFu || stride < vocab || !d_status ||
        !(scale > 0.f) || !std::isfinite(scale) || top > K3HUF_MAX_TOP || top > vocab || n > 0x7FFFFFFFull)
        return K3HUF_E_ARG;
    if (!aligned_to(d_logits, elem_bytes(type)) || !aligned_to(d_tokens, id_bytes) || !aligned_to(d_logprob, 4) ||
        !aligned_to(d_entropy, 4) || !aligned_to(d_lse, 4) || !aligned_to(d_top_ids, 4) || !aligned_to(d_top_logprobs, 4) || !aligned_to(d_status, 4))
        return K3HUF_E_ARG;
    if (n == 0) return K3HUF_OK;
    if (!d_logits || !d_tokens || !d_logprob || (top && (!d_top_ids || !d_top_logprobs))) return K3HUF_E_ARG;
    LogprobParams P{d_logits, d_tokens, d_logprob, d_entropy, d_lse, d_top_logprobs, d_top_ids, d_status, stride, uint32_t(n), vocab, id_bytes, top, scale};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (type == K3HUF_BF16) logprob_kernel<__nv_bfloat16><<<uint32_t(n), kThreads, 0, st>>>(P);
    else logprob_kernel<float><<<uint32_t(n), kThreads, 0, st>>>(P);
    return cuda_rc(cudaGetLastError());
}

extern "C" int k3huf_token_logprobs_grad(const void *d_logits, uint32_t type, uint64_t stride, uint64_t n, uint32_t vocab, float scale,
                                         const void *d_tokens, uint32_t id_bytes, const float *d_lse, const float *d_entropy,
                                         const float *d_g_logprob, const float *d_g_entropy, void *d_dlogits, uint64_t out_stride,
                                         uint32_t *d_status, void *stream) {
    if (!elem_ok(type) || (id_bytes != 4 && id_bytes != 8) || vocab == 0 || vocab > 0x7FFFFFFFu || stride < vocab || out_stride < vocab ||
        !d_status || !(scale > 0.f) || !std::isfinite(scale) || n > 0x7FFFFFFFull || (d_g_entropy && !d_entropy))
        return K3HUF_E_ARG;
    if (!aligned_to(d_logits, elem_bytes(type)) || !aligned_to(d_dlogits, elem_bytes(type)) || !aligned_to(d_tokens, id_bytes) || !aligned_to(d_lse, 4) ||
        !aligned_to(d_entropy, 4) || !aligned_to(d_g_logprob, 4) || !aligned_to(d_g_entropy, 4) || !aligned_to(d_status, 4))
        return K3HUF_E_ARG;
    if (n == 0) return K3HUF_OK;
    if (!d_logits || !d_dlogits || !d_tokens || !d_lse || !d_g_logprob) return K3HUF_E_ARG;
    if (d_logits == d_dlogits && stride != out_stride) return K3HUF_E_ARG;
    GradParams P{d_logits, d_dlogits, d_tokens, d_lse, d_entropy, d_g_logprob, d_g_entropy, d_status, stride, out_stride, uint32_t(n), vocab, id_bytes, scale};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (type == K3HUF_BF16) logprob_grad_kernel<__nv_bfloat16><<<uint32_t(n), kThreads, 0, st>>>(P);
    else logprob_grad_kernel<float><<<uint32_t(n), kThreads, 0, st>>>(P);
    return cuda_rc(cudaGetLastError());
}
