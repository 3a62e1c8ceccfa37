// Low-rank adapters of many requests beside a shared projection, and their
// gradients.  With i = ids[t] the adapter of token t, A_i (rank x cols),
// B_i (rank x rows) and s_i its factors and scale:
//   y[t]  = base[t] + s_i (x[t] A_i^T) B_i
//   dh[t] = s_i dy[t] B_i^T         dx[t] = dx_base[t] + dh[t] A_i
//   dA_i  = sum_t dh[t]^T x[t]      dB_i  = sum_t (s_i x[t] A_i^T)^T dy[t]
// Both factors are stored rank-major, so forward and backward are the same
// three products: "shrink" (a dot product with every row of a factor),
// "expand" (a sum of a factor's rows) and "outer" (a sum over tokens).
// The rank-wide intermediates stay in fp32.
#include "k3huf_ops.h"

namespace k3huf {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ bool adapter_of(const int32_t *ids, uint64_t t, uint32_t n_adapters, int32_t &i) {
    i = ids[t];
    return i >= 0 && uint32_t(i) < n_adapters;
}

// h[t, r] = s_i v[t] . w[i, r]; zero without an adapter.  One CTA per token, one warp per row of the factor.
__global__ void __launch_bounds__(kThreads)
shrink_kernel(const __nv_bfloat16 *v, uint64_t stride, const __nv_bfloat16 *w, const float *scales, const int32_t *ids, uint32_t n_adapters, uint32_t rank, uint64_t len, float *h, uint32_t *status) {
    const uint64_t t = blockIdx.x;
    int32_t i;
    const bool any = adapter_of(ids, t, n_adapters, i);
    if (!any && i >= 0 && threadIdx.x == 0) atomicOr(status, K3HUF_ST_TOKEN);
    for (uint32_t r = threadIdx.x / 32; r < rank; r += kThreads / 32) {
        float acc = 0.f;
        if (any)
            for (uint64_t c = threadIdx.x % 32; c < len; c += 32)
                acc = fmaf(ld_f32(v + t * stride + c), ld_f32(w + (uint64_t(i) * rank + r) * len + c), acc);
        acc = warp_sum(acc);
        if (threadIdx.x % 32 == 0) h[t * rank + r] = any ? scales[i] * acc : 0.f;
    }
}

// y[t] = base[t] + sum_r h[t, r] w[i, r]
template <typename T>
__global__ void __launch_bounds__(kThreads)
expand_kernel(const float *h, const __nv_bfloat16 *w, const int32_t *ids, uint32_t n_adapters, uint32_t rank, uint64_t len, const T *base, uint64_t base_stride, T *y, uint64_t y_stride) {
    const uint64_t t = blockIdx.x;
    int32_t i;
    const bool any = adapter_of(ids, t, n_adapters, i);
    for (uint64_t c = threadIdx.x; c < len; c += kThreads) {
        float acc = 0.f;
        if (any)
            for (uint32_t r = 0; r < rank; ++r) acc = fmaf(h[t * rank + r], ld_f32(w + (uint64_t(i) * rank + r) * len + c), acc);
        st_f32(y + t * y_stride + c, base ? ld_f32(base + t * base_stride + c) + acc : acc);
    }
}

// g[i, r] (+)= sum over tokens of adapter i of h[t, r] v[t].  One CTA per adapter, row and column block.
__global__ void __launch_bounds__(kThreads)
outer_kernel(const float *h, const __nv_bfloat16 *v, uint64_t stride, const int32_t *ids, uint64_t n, uint32_t rank, uint64_t len, float *g, bool add) {
    const uint32_t i = blockIdx.y / rank, r = blockIdx.y % rank;
    const uint64_t c = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (c >= len) return;
    float acc = 0.f;
    for (uint64_t t = 0; t < n; ++t)
        if (ids[t] == int32_t(i)) acc = fmaf(h[t * rank + r], ld_f32(v + t * stride + c), acc);
    float *out = g + uint64_t(blockIdx.y) * len + c;
    *out = add ? *out + acc : acc;
}

bool adapters_ok(const k3huf_adapters_t *ad, uint64_t n) {
    return ad && ad->a && ad->b && ad->scales && ad->n_adapters && ad->n_adapters < (1u << 24) && ad->rank && ad->rank <= K3HUF_MAX_RANK &&
           ad->cols && ad->rows && ad->cols < (1ull << 31) && ad->rows < (1ull << 31) && n < (1ull << 31) && aligned_to(ad->a, 2) &&
           aligned_to(ad->b, 2) && aligned_to(ad->scales, 4);
}

}  // namespace
}  // namespace k3huf

using namespace k3huf;

extern "C" int k3huf_adapter_scratch_bytes(uint64_t n_tokens, uint32_t n_adapters, uint32_t rank, uint64_t cols, uint64_t rows, int grad, size_t *scratch_bytes) {
    if (!scratch_bytes || n_adapters == 0 || rank == 0 || rank > K3HUF_MAX_RANK || cols == 0 || rows == 0 || n_tokens >= (1ull << 31)) return K3HUF_E_ARG;
    const uint64_t h = align_up(n_tokens * rank * 4, 256);
    *scratch_bytes = 256 + h * (grad ? 2 : 1);
    return K3HUF_OK;
}

extern "C" int k3huf_adapter_apply(const k3huf_adapters_t *ad, const void *d_x, uint64_t x_stride, const int32_t *d_ids, uint64_t n_tokens,
                                   const void *d_base, uint64_t base_stride, void *d_y, uint64_t y_stride, uint32_t y_type,
                                   void *d_scratch, size_t scratch_bytes, uint32_t *d_status, void *stream) {
    size_t need = 0;
    if (!adapters_ok(ad, n_tokens) || !elem_ok(y_type) || !d_status || x_stride < ad->cols || y_stride < ad->rows || (d_base && base_stride < ad->rows) ||
        k3huf_adapter_scratch_bytes(n_tokens, ad->n_adapters, ad->rank, ad->cols, ad->rows, 0, &need) || !d_scratch || scratch_bytes < need)
        return K3HUF_E_ARG;
    if (!aligned_to(d_x, 2) || !aligned_to(d_ids, 4) || !aligned_to(d_base, elem_bytes(y_type)) || !aligned_to(d_y, elem_bytes(y_type)) ||
        !aligned_to(d_scratch, 256) || !aligned_to(d_status, 4) || (d_base == d_y && d_base && base_stride != y_stride))
        return K3HUF_E_ARG;
    if (n_tokens == 0) return K3HUF_OK;
    if (!d_x || !d_ids || !d_y) return K3HUF_E_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *h = static_cast<float *>(d_scratch);
    const uint32_t n = uint32_t(n_tokens);
    const auto *a = static_cast<const __nv_bfloat16 *>(ad->a), *b = static_cast<const __nv_bfloat16 *>(ad->b), *x = static_cast<const __nv_bfloat16 *>(d_x);
    shrink_kernel<<<n, kThreads, 0, st>>>(x, x_stride, a, ad->scales, d_ids, ad->n_adapters, ad->rank, ad->cols, h, d_status);
    if (y_type == K3HUF_BF16)
        expand_kernel<<<n, kThreads, 0, st>>>(h, b, d_ids, ad->n_adapters, ad->rank, ad->rows, static_cast<const __nv_bfloat16 *>(d_base), base_stride, static_cast<__nv_bfloat16 *>(d_y), y_stride);
    else
        expand_kernel<<<n, kThreads, 0, st>>>(h, b, d_ids, ad->n_adapters, ad->rank, ad->rows, static_cast<const float *>(d_base), base_stride, static_cast<float *>(d_y), y_stride);
    return cuda_rc(cudaGetLastError());
}

extern "C" int k3huf_adapter_grad(const k3huf_adapters_t *ad, const void *d_x, uint64_t x_stride, const int32_t *d_ids, uint64_t n_tokens,
                                  const void *d_dy, uint64_t dy_stride, const void *d_dx_base, uint64_t dx_base_stride, void *d_dx, uint64_t dx_stride,
                                  uint32_t dx_type, float *d_da, float *d_db, void *d_scratch, size_t scratch_bytes, uint32_t *d_status, uint32_t flags, void *stream) {
    size_t need = 0;
    if (!adapters_ok(ad, n_tokens) || !elem_ok(dx_type) || !d_status || !d_da || !d_db || x_stride < ad->cols || dy_stride < ad->rows ||
        (d_dx && dx_stride < ad->cols) || (d_dx_base && (!d_dx || dx_base_stride < ad->cols)) || (flags & ~uint32_t(K3HUF_ACCUMULATE)) ||
        k3huf_adapter_scratch_bytes(n_tokens, ad->n_adapters, ad->rank, ad->cols, ad->rows, 1, &need) || !d_scratch || scratch_bytes < need)
        return K3HUF_E_ARG;
    if (!aligned_to(d_x, 2) || !aligned_to(d_dy, 2) || !aligned_to(d_ids, 4) || !aligned_to(d_dx_base, elem_bytes(dx_type)) || !aligned_to(d_dx, elem_bytes(dx_type)) ||
        !aligned_to(d_da, 4) || !aligned_to(d_db, 4) || !aligned_to(d_scratch, 256) || !aligned_to(d_status, 4) || (d_dx_base == d_dx && d_dx && dx_base_stride != dx_stride))
        return K3HUF_E_ARG;
    if (n_tokens && (!d_x || !d_ids || !d_dy)) return K3HUF_E_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *h = static_cast<float *>(d_scratch), *dh = h + align_up(n_tokens * ad->rank * 4, 256) / 4;
    const uint32_t n = uint32_t(n_tokens), S = ad->n_adapters, r = ad->rank;
    if (uint64_t(S) * r > 65535) return K3HUF_E_ARG;
    const auto *a = static_cast<const __nv_bfloat16 *>(ad->a), *b = static_cast<const __nv_bfloat16 *>(ad->b);
    const auto *x = static_cast<const __nv_bfloat16 *>(d_x), *dy = static_cast<const __nv_bfloat16 *>(d_dy);
    if (n) {
        shrink_kernel<<<n, kThreads, 0, st>>>(x, x_stride, a, ad->scales, d_ids, S, r, ad->cols, h, d_status);
        shrink_kernel<<<n, kThreads, 0, st>>>(dy, dy_stride, b, ad->scales, d_ids, S, r, ad->rows, dh, d_status);
        if (d_dx && dx_type == K3HUF_BF16)
            expand_kernel<<<n, kThreads, 0, st>>>(dh, a, d_ids, S, r, ad->cols, static_cast<const __nv_bfloat16 *>(d_dx_base), dx_base_stride, static_cast<__nv_bfloat16 *>(d_dx), dx_stride);
        else if (d_dx)
            expand_kernel<<<n, kThreads, 0, st>>>(dh, a, d_ids, S, r, ad->cols, static_cast<const float *>(d_dx_base), dx_base_stride, static_cast<float *>(d_dx), dx_stride);
    }
    const bool add = (flags & K3HUF_ACCUMULATE) != 0;
    outer_kernel<<<dim3(uint32_t((ad->cols + kThreads - 1) / kThreads), S * r), kThreads, 0, st>>>(dh, x, x_stride, d_ids, n, r, ad->cols, d_da, add);
    outer_kernel<<<dim3(uint32_t((ad->rows + kThreads - 1) / kThreads), S * r), kThreads, 0, st>>>(h, dy, dy_stride, d_ids, n, r, ad->rows, d_db, add);
    return cuda_rc(cudaGetLastError());
}
