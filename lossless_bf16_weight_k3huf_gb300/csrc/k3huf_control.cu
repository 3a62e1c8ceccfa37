// Control of logits before a token is chosen: penalties for tokens that a request has seen, biases, a grammar's mask.
//
// For token j of a row, with `seen` whether the request's prompt or output holds it and c how often its output does:
//   v = x_j;  if seen: v = v > 0 ? v / repetition : v repetition;  v -= frequency c;  if c > 0: v -= presence
//   v += bias_j;  v = -infinity where the mask's bit j is 0
//
// A CTA takes a slice of a row.  Few of its tokens are touched by a history or a bias, so what it knows of them lies
// in shared memory by token (a count and a place in the list of biases), cleared only where it is used, beside one
// bit per token that says whether to look.  Counts are whole numbers: their order does not matter.  What is not
// touched and not banned is copied, or, where the logits are changed in place, not even read; what is banned is
// written without being read.
#include <algorithm>
#include <cmath>

#include "k3huf_rows.h"

namespace k3huf {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kUnit = 8;                             // values handled at once: one byte of bits
constexpr uint32_t kSlice = 8192;                         // values per CTA
constexpr int kUnits = int(kSlice / kUnit) / kThreads;    // units per thread
constexpr uint32_t kSeen = 1u << 31;

struct ControlParams {
    const void *x;
    void *y;
    k3huf_control_t c;
    uint32_t *status;
    uint64_t x_stride, y_stride, row0;
    uint32_t vocab, slices;
};

template <typename T> __device__ __forceinline__ void load_unit(const T *p, float (&f)[kUnit]) {
#pragma unroll
    for (int h = 0; h < int(kUnit) / kPer<T>; ++h) {
        float g[kPer<T>];
        unpack<T>(__ldcs(reinterpret_cast<const uint4 *>(p) + h), g);
#pragma unroll
        for (int k = 0; k < kPer<T>; ++k) f[h * kPer<T> + k] = g[k];
    }
}
__device__ __forceinline__ void store_unit(float *p, const float (&f)[kUnit]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}
__device__ __forceinline__ void store_unit(__nv_bfloat16 *p, const float (&f)[kUnit]) {
    uint4 o;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
    __stcs(reinterpret_cast<uint4 *>(p), o);
}

// A row's span [from, to) of a list, or nothing (and the status bit) where it is none.
__device__ __forceinline__ bool span_ok(int64_t from, int64_t to, uint64_t n, uint32_t *status) {
    if (from >= 0 && from <= to && uint64_t(to) <= n) return true;
    if (threadIdx.x == 0) atomicOr(status, K3HUF_ST_INDEX);
    return false;
}

template <typename T, typename U>
__global__ void __launch_bounds__(kThreads) control_kernel(const __grid_constant__ ControlParams P) {
    extern __shared__ uint32_t s_mem[];
    uint32_t *s_count = s_mem, *s_place = s_mem + kSlice, *s_touched = s_mem + 2 * kSlice;
    const uint64_t row = P.row0 + blockIdx.x / P.slices;
    const uint32_t slice = blockIdx.x % P.slices, tid = threadIdx.x;
    const T *x = static_cast<const T *>(P.x) + row * P.x_stride;
    U *y = static_cast<U *>(P.y) + row * P.y_stride;
    // unit u of the row: values [8 u - shift, 8 u - shift + 8); both rows' units on 16 bytes, or neither taken as such
    const uint32_t sx = uint32_t(reinterpret_cast<uintptr_t>(x) / sizeof(T) % kUnit), sy = uint32_t(reinterpret_cast<uintptr_t>(y) / sizeof(U) % kUnit);
    const bool vec = sx == sy;
    const uint32_t shift = vec ? sx : 0u;
    const bool in_place = static_cast<const void *>(x) == static_cast<const void *>(y);
    const int64_t j0 = int64_t(slice) * kSlice - shift;    // the slice's first value
    const k3huf_control_t &c = P.c;
    for (uint32_t i = tid; i < kSlice / 32; i += kThreads) s_touched[i] = 0;
    __syncthreads();

    // the lists twice: places cleared and marked, then counted
    const uint32_t *mask = nullptr;
    if (c.mask) {
        const int64_t m = c.mask_rows ? c.mask_rows[row] : int64_t(row);
        if (m >= int64_t(c.n_masks)) {
            if (slice == 0 && tid == 0) atomicOr(P.status, K3HUF_ST_INDEX);
        } else if (m >= 0) {
            mask = c.mask + uint64_t(m) * c.mask_stride;
        }
    }
    int64_t h0 = 0, hs = 0, h1 = 0, b0 = 0, b1 = 0;
    if (c.history) {
        h0 = c.spans[3 * row], hs = c.spans[3 * row + 1], h1 = c.spans[3 * row + 2];
        if (!span_ok(h0, h1, c.n_history, P.status) || !span_ok(h0, hs, uint64_t(h1), P.status)) h0 = hs = h1 = 0;
    }
    if (c.bias_ids) {
        b0 = c.bias_spans[2 * row], b1 = c.bias_spans[2 * row + 1];
        if (!span_ok(b0, b1, c.n_bias, P.status)) b0 = b1 = 0;
    }
    auto place_of = [&](const void *ids, uint32_t id_bytes, int64_t i) {           // in the slice, or kSlice
        const int64_t id = ld_id(ids, id_bytes, uint64_t(i));
        if (id >= int64_t(P.vocab) && slice == 0) atomicOr(P.status, K3HUF_ST_TOKEN);
        const int64_t at = id - j0;
        return id >= 0 && id < int64_t(P.vocab) && at >= 0 && at < int64_t(kSlice) ? uint32_t(at) : kSlice;
    };
    auto clear = [&](uint32_t at) {
        if (at == kSlice) return;
        s_count[at] = 0;
        s_place[at] = 0;
        atomicOr(&s_touched[at / 32], 1u << (at % 32));
    };
    for (int64_t i = h0 + tid; i < h1; i += kThreads) clear(place_of(c.history, c.history_id_bytes, i));
    for (int64_t i = b0 + tid; i < b1; i += kThreads) clear(place_of(c.bias_ids, c.bias_id_bytes, i));
    __syncthreads();
    for (int64_t i = h0 + tid; i < h1; i += kThreads) {
        const uint32_t at = place_of(c.history, c.history_id_bytes, i);
        if (at == kSlice) continue;
        if (i < hs) atomicOr(&s_count[at], kSeen);
        else atomicAdd(&s_count[at], 1u);
    }
    // (a token that is listed twice takes its last bias)
    for (int64_t i = b0 + tid; i < b1; i += kThreads) {
        const uint32_t at = place_of(c.bias_ids, c.bias_id_bytes, i);
        if (at < kSlice) atomicMax(&s_place[at], uint32_t(i - b0) + 1);
    }
    __syncthreads();

    const float repetition = c.repetition ? c.repetition[row] : 1.f, frequency = c.frequency ? c.frequency[row] : 0.f, presence = c.presence ? c.presence[row] : 0.f;
    auto change = [&](float v, uint32_t at) {
        const uint32_t n = s_count[at], place = s_place[at];
        if (n && c.repetition) v = v > 0.f ? v / repetition : v * repetition;
        const uint32_t times = n & ~kSeen;
        if (times) {
            v -= frequency * float(times);
            v -= presence;
        }
        return place ? v + c.bias_values[b0 + place - 1] : v;
    };
    // the mask's bits of the unit from value j on
    auto allowed = [&](int64_t j) {
        if (!mask) return 0xFFu;
        const int64_t from = j < 0 ? 0 : j;
        const uint32_t w = uint32_t(from / 32), last = (P.vocab - 1) / 32;
        const uint64_t two = mask[w] | (w < last ? uint64_t(mask[w + 1]) << 32 : 0ull);
        const uint32_t bits = uint32_t(two >> (from % 32));
        return (j < 0 ? bits << uint32_t(-j) : bits) & 0xFFu;
    };
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = i * kThreads + tid;            // of the slice
        const int64_t j = j0 + int64_t(u) * kUnit;
        if (j >= int64_t(P.vocab)) break;
        const uint32_t touched = s_touched[u / 4] >> (u % 4 * 8) & 0xFFu, ok = allowed(j);
        if (in_place && !touched && ok == 0xFFu) continue;
        float f[kUnit];
        const bool whole = vec && j >= 0 && j + kUnit <= int64_t(P.vocab);
        if (whole) {
            if (ok) load_unit(x + j, f);
        } else {
#pragma unroll
            for (int k = 0; k < int(kUnit); ++k) f[k] = j + k >= 0 && j + k < int64_t(P.vocab) ? ld_f32(x + j + k) : 0.f;
        }
        if (touched & ok) {
#pragma unroll 1
            for (uint32_t k = 0; k < kUnit; ++k)
                if (touched & ok & (1u << k)) {
                    float v = 0.f;
#pragma unroll
                    for (uint32_t q = 0; q < kUnit; ++q) v = q == k ? f[q] : v;
                    v = change(v, u * kUnit + k);
#pragma unroll
                    for (uint32_t q = 0; q < kUnit; ++q) f[q] = q == k ? v : f[q];
                }
        }
#pragma unroll
        for (uint32_t k = 0; k < kUnit; ++k)
            if (!(ok >> k & 1)) f[k] = -INFINITY;
        if (whole) {
            store_unit(y + j, f);
        } else {
#pragma unroll
            for (int k = 0; k < int(kUnit); ++k)
                if (j + k >= 0 && j + k < int64_t(P.vocab)) st_f32(y + j + k, f[k]);
        }
    }
}

constexpr size_t kSmem = (2 * kSlice + kSlice / 32) * 4;

template <typename T, typename U>
int launch(const ControlParams &P, uint64_t n, cudaStream_t stream) {
    static std::atomic<uint64_t> once{0};
    const int rc = once_per_device(once, [] { return cudaFuncSetAttribute(control_kernel<T, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem)); });
    if (rc) return rc;
    const uint64_t most = 0x7FFFFFFFull / P.slices;
    for (uint64_t r0 = 0; r0 < n; r0 += most) {
        ControlParams Q = P;
        Q.row0 = r0;
        control_kernel<T, U><<<uint32_t(std::min(most, n - r0) * P.slices), kThreads, kSmem, stream>>>(Q);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_rc(e);
    }
    return K3HUF_OK;
}

}  // namespace
}  // namespace k3huf

using namespace k3huf;

extern "C" int k3huf_logits_control(const k3huf_control_t *control, const void *d_logits, uint32_t type, uint64_t stride, uint64_t n, uint32_t vocab, void *d_out, uint32_t out_type,
                                    uint64_t out_stride, uint32_t *d_status, void *stream) {
    if (!control || !elem_ok(type) || !elem_ok(out_type) || vocab == 0 || vocab > 0x7FFFFFFFu || stride < vocab || out_stride < vocab || !d_status || n > 0x7FFFFFFFull) return K3HUF_E_ARG;
    const k3huf_control_t &c = *control;
    auto id_ok = [](uint32_t b) { return b == 4 || b == 8; };
    if (!aligned_to(d_logits, elem_bytes(type)) || !aligned_to(d_out, elem_bytes(out_type)) || !aligned_to(d_status, 4) || !aligned_to(c.spans, 8) || !aligned_to(c.bias_spans, 8) ||
        !aligned_to(c.repetition, 4) || !aligned_to(c.frequency, 4) || !aligned_to(c.presence, 4) || !aligned_to(c.bias_values, 4) || !aligned_to(c.mask, 4) || !aligned_to(c.mask_rows, 4))
        return K3HUF_E_ARG;
    if (c.history && (!id_ok(c.history_id_bytes) || !aligned_to(c.history, c.history_id_bytes) || !c.spans || c.n_history > 0x7FFFFFFFull)) return K3HUF_E_ARG;
    if (c.bias_ids && (!id_ok(c.bias_id_bytes) || !aligned_to(c.bias_ids, c.bias_id_bytes) || !c.bias_values || !c.bias_spans || c.n_bias > 0x7FFFFFFFull)) return K3HUF_E_ARG;
    if (c.mask && (c.mask_stride < (uint64_t(vocab) + 31) / 32 || (!c.mask_rows && c.n_masks < n))) return K3HUF_E_ARG;
    if (n == 0) return K3HUF_OK;
    if (!d_logits || !d_out || (d_logits == d_out && (type != out_type || stride != out_stride))) return K3HUF_E_ARG;
    const ControlParams P{d_logits, d_out, c, d_status, stride, out_stride, 0, vocab, uint32_t((uint64_t(vocab) + kUnit - 1 + kSlice - 1) / kSlice)};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (type == K3HUF_BF16) return out_type == K3HUF_BF16 ? launch<__nv_bfloat16, __nv_bfloat16>(P, n, st) : launch<__nv_bfloat16, float>(P, n, st);
    return out_type == K3HUF_BF16 ? launch<float, __nv_bfloat16>(P, n, st) : launch<float, float>(P, n, st);
}
