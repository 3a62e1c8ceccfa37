// Control of logits before a token is chosen: penalties for tokens that a request has seen, biases, a grammar's mask.
//
// For token j of a row, with `seen` whether the request's prompt or output holds it and c how often its output does:
//   v = x_j;  if seen: v = v > 0 ? v / repetition : v repetition;  v -= frequency c;  if c > 0: v -= presence
//   v += bias_j;  v = -infinity where the mask's bit j is 0
//
// Two jobs.  The stream: logits that the mask allows are copied (or, where the logits are changed in place, not even
// read), the others written as -infinity without being read; bound by that traffic.  The lists: what the history and
// the biases touch, a few of a row's tokens, is changed after the stream has passed; bound by the latencies of its
// chain (a row's spans, its entries, the touched logits).  One bit per token says what is touched, and a token's place
// among the touched ones (those of the words before its own, and its word's bits below it) is where its count and its
// bias's place in the list are kept.  Counts are whole numbers: their order does not matter.  Parts with more touched
// tokens than places are worked through in windows.  1024 rows of 131072 bf16 with histories of 1500 tokens, 100 biases
// and masks: the stream 85 us (a copy 83), the lists 31 (39 on a cold cache); 8 rows of fp32 in place 6.9 us, 60 rows of
// 50021 9.1 us.  Rows of logits and results that do not sit alike go one value at a time: 1024 x 131072 bf16 618 us.
// (Counters of the vocabulary's size, cleared per row, cost 409 us instead of 123.)
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "k3huf_rows.h"
#include "k3huf_tc.h"

namespace k3huf {
namespace {

constexpr uint32_t kMaxThreads = 1024;
constexpr uint32_t kUnit = 8;                             // values handled at once
template <typename T> constexpr int kUnits = 8 / int(sizeof(T));         // units in flight per thread
constexpr uint32_t kPart = 1u << 17;                      // values per CTA at most
constexpr uint32_t kPlaces = 2048, kMostPlaces = 12288;   // touched tokens that are looked after at once, by default and at most
constexpr uint32_t kSeen = 1u << 31;

struct ControlParams {
    const void *x;
    void *y;
    k3huf_control_t c;
    uint32_t *status;
    uint64_t x_stride, y_stride, row0;
    uint32_t vocab, parts, part, streaming;   // CTAs per row; values of each; threads that stream (the others see to the lists)
    uint32_t places;                          // touched tokens that a CTA looks after at once
    bool after;                               // the stream is the launch before this one
};

// 16 bytes that nobody reads again (and that push nothing out of L1)
__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// a unit as loaded
template <typename T> struct Raw {
    uint4 v[kUnit / kPer<T>];
};
template <typename T> __device__ __forceinline__ void load_unit(const T *p, Raw<T> &r) {
#pragma unroll
    for (int h = 0; h < int(kUnit) / kPer<T>; ++h) r.v[h] = ld_stream(reinterpret_cast<const uint4 *>(p) + h);
}
template <typename T> __device__ __forceinline__ void unpack_unit(const Raw<T> &r, float (&f)[kUnit]) {
#pragma unroll
    for (int h = 0; h < int(kUnit) / kPer<T>; ++h) {
        float g[kPer<T>];
        unpack<T>(r.v[h], g);
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

// ... a unit of bf16 as it is, -infinity where the mask's bit is 0 (by way of fp32 every NaN would become the same one)
__device__ __forceinline__ void store_allowed(__nv_bfloat16 *p, const Raw<__nv_bfloat16> &r, uint32_t ok) {
    uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t keep = (ok >> (2 * k) & 1 ? 0xFFFFu : 0u) | (ok >> (2 * k + 1) & 1 ? 0xFFFF0000u : 0u);
        w[k] = (w[k] & keep) | (0xFF80FF80u & ~keep);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
// ... and one value
template <typename T, typename U> __device__ __forceinline__ void copy_to(U *to, const T *from) {
    if constexpr (std::is_same_v<T, U>) *to = *from;
    else st_f32(to, ld_f32(from));
}

// A row's span [from, to) of a list, or nothing (and the status bit) where it is none.
__device__ __forceinline__ bool span_ok(int64_t from, int64_t to, uint64_t n, uint32_t *status) {
    if (from >= 0 && from <= to && uint64_t(to) <= n) return true;
    atomicOr(status, K3HUF_ST_INDEX);
    return false;
}

template <typename T, typename U>
__global__ void __launch_bounds__(kMaxThreads) control_kernel(const __grid_constant__ ControlParams P) {
    extern __shared__ uint32_t s_touched[];   // a bit per token of the part
    uint32_t *s_before = s_touched + P.part / 32;             // touched tokens before the word
    uint32_t *s_count = s_before + P.part / 32, *s_bias = s_count + P.places, *s_token = s_bias + P.places;
    __shared__ uint32_t s_warp[kMaxThreads / 32];
    const uint64_t row = P.row0 + blockIdx.x / P.parts;
    const uint32_t part = blockIdx.x % P.parts;
    const T *x = static_cast<const T *>(P.x) + row * P.x_stride;
    U *y = static_cast<U *>(P.y) + row * P.y_stride;
    const bool in_place = static_cast<const void *>(x) == static_cast<const void *>(y);
    // the part's values: [j0, j1)
    const uint32_t j0 = part * P.part, j1 = min(P.vocab - j0, P.part) + j0;
    const k3huf_control_t &c = P.c;
    const uint32_t *mask = nullptr;
    if (c.mask) {
        const int64_t m = c.mask_rows ? c.mask_rows[row] : int64_t(row);
        if (m >= int64_t(c.n_masks)) {
            if (part == 0 && threadIdx.x == 0) atomicOr(P.status, K3HUF_ST_INDEX);
        } else if (m >= 0) {
            mask = c.mask + uint64_t(m) * c.mask_stride;
        }
    }
    auto banned = [&](uint32_t j) { return mask && !(__ldg(mask + j / 32) >> (j % 32) & 1); };
    if (threadIdx.x < P.streaming) {
        if (P.streaming == blockDim.x) grid_dep_launch();     // (the lists' launch, if there is one, may begin)
        const uint32_t tid = threadIdx.x, step = kUnits<T> * P.streaming * kUnit;
        // whole units: 16-byte blocks of both rows, [first, last) in values; what is around them, or all where the two do
        // not sit alike, one value at a time
        const uint32_t sx = uint32_t(reinterpret_cast<uintptr_t>(x + j0) / sizeof(T) % kUnit), sy = uint32_t(reinterpret_cast<uintptr_t>(y + j0) / sizeof(U) % kUnit);
        const uint32_t first = sx == sy ? min(j0 + (kUnit - sx) % kUnit, j1) : j1, last = first + (j1 - first) / kUnit * kUnit;
        // a step's units are on their way while the one before is written, and the mask's bits a step ahead of them
        uint32_t ok[kUnits<T>], ahead[kUnits<T>];
        Raw<T> raw[kUnits<T>], next[kUnits<T>];
        auto bits = [&](uint32_t u0, uint32_t (&to)[kUnits<T>]) {
#pragma unroll
            for (int i = 0; i < kUnits<T>; ++i) {
                const uint32_t j = u0 + (i * P.streaming + tid) * kUnit;
                to[i] = 0xFFu;
                if (mask && j < last) {
                    // (the words of a unit's bits, both within the vocabulary's)
                    const uint32_t w = j / 32, v = (j + kUnit - 1) / 32;
                    const uint32_t lo = __ldg(mask + w), hi = v == w ? 0u : __ldg(mask + v);
                    to[i] = __funnelshift_r(lo, hi, j % 32) & 0xFFu;
                }
            }
        };
        auto load = [&](uint32_t u0, const uint32_t (&of)[kUnits<T>], Raw<T> (&to)[kUnits<T>]) {
#pragma unroll
            for (int i = 0; i < kUnits<T>; ++i) {
                const uint32_t j = u0 + (i * P.streaming + tid) * kUnit;
                if (j < last && of[i] && !(in_place && of[i] == 0xFFu)) load_unit(x + j, to[i]);
            }
        };
        bits(first, ok);
        load(first, ok, raw);
        bits(first + step, ahead);
        for (uint32_t u0 = first; u0 < last; u0 += step) {
            load(u0 + step, ahead, next);
#pragma unroll
            for (int i = 0; i < kUnits<T>; ++i) {
                const uint32_t j = u0 + (i * P.streaming + tid) * kUnit;
                if (j >= last || (in_place && ok[i] == 0xFFu)) continue;
                if constexpr (std::is_same_v<T, U> && sizeof(T) == 2) {
                    store_allowed(y + j, raw[i], ok[i]);
                } else {
                    float f[kUnit];
                    unpack_unit(raw[i], f);
#pragma unroll
                    for (uint32_t k = 0; k < kUnit; ++k) f[k] = ok[i] >> k & 1 ? f[k] : -INFINITY;
                    store_unit(y + j, f);
                }
            }
#pragma unroll
            for (int i = 0; i < kUnits<T>; ++i) raw[i] = next[i], ok[i] = ahead[i];
            bits(u0 + 2 * step, ahead);
        }
        const uint32_t rest = j1 - j0 - (last - first);
#pragma unroll 1
        for (uint32_t i = tid; i < rest; i += P.streaming) {
            const uint32_t j = j0 + i < first ? j0 + i : j0 + i + (last - first);
            if (banned(j)) st_f32(y + j, -INFINITY);
            else if (!in_place) copy_to(y + j, x + j);
        }
        if (P.streaming < blockDim.x) __syncthreads();
        return;
    }
    const bool streams = P.streaming > 0;
    const uint32_t n = blockDim.x - P.streaming, tid = threadIdx.x - P.streaming, lane = tid % 32, warp = tid / 32;
    auto sync = [&]() {                       // (of these threads; a warp's come to it together, wherever they parted before)
        __syncwarp();
        asm volatile("bar.sync 1, %0;" ::"r"(n) : "memory");
    };
    // the two lists, numbered as one: tokens of the history, then of the biases
    const void *ids[2] = {c.history, c.bias_ids};
    uint32_t n_history = 0, n_prompt = 0, entries = 0;
    const float *bias_values = c.bias_values;
    const float repetition = c.repetition ? c.repetition[row] : 1.f, frequency = c.frequency ? c.frequency[row] : 0.f, presence = c.presence ? c.presence[row] : 0.f;
    const uint32_t wide0 = c.history_id_bytes / 4, wide1 = c.bias_id_bytes / 4;
    if (c.history) {
        const int64_t a = c.spans[3 * row], b = c.spans[3 * row + 1], e = c.spans[3 * row + 2];
        if (span_ok(a, e, c.n_history, P.status) && span_ok(a, b, uint64_t(e), P.status)) {
            n_history = entries = uint32_t(e - a), n_prompt = uint32_t(b - a);
            ids[0] = static_cast<const uint32_t *>(c.history) + a * wide0;
        }
    }
    if (c.bias_ids) {
        const int64_t a = c.bias_spans[2 * row], e = c.bias_spans[2 * row + 1];
        if (span_ok(a, e, c.n_bias, P.status)) {
            entries += uint32_t(e - a);
            ids[1] = static_cast<const uint32_t *>(c.bias_ids) + a * wide1;
            bias_values += a;
        }
    }
    if (entries == 0) {
        if (streams) __syncthreads();
        if (P.after) grid_dep_wait();
        return;
    }
    constexpr uint32_t kAhead = 8;            // loads at once
    const uint32_t size = j1 - j0, words = (size + 31) / 32;
    // places in the part of the entries i0, i0 + n, ... (2^32 - 1: none, or a token of another part)
    auto load = [&](uint32_t i0, bool check, uint32_t (&at)[kAhead]) {
        // (nothing but loads in the first loops: the use of one before the next is issued would wait for it)
        int32_t lo[kAhead], hi[kAhead];
        bool past = false;
        // (where all threads' are of the history, a third of the instructions does: 8 rows of 30000 tokens 25 us, 33 without)
        const bool whole = i0 - tid + kAhead * n <= n_history;
        if (whole && wide0 == 1) {
            const int32_t *q = static_cast<const int32_t *>(ids[0]) + i0;
#pragma unroll
            for (uint32_t k = 0; k < kAhead; ++k) lo[k] = __ldg(q + k * n);
#pragma unroll
            for (uint32_t k = 0; k < kAhead; ++k) {
                past = past || lo[k] >= int32_t(P.vocab);
                at[k] = uint32_t(lo[k]) - j0 < size ? uint32_t(lo[k]) - j0 : 0xFFFFFFFFu;
            }
            if (past && check) atomicOr(P.status, K3HUF_ST_TOKEN);
            return;
        }
        if (whole) {
            const int2 *q = static_cast<const int2 *>(ids[0]) + i0;
#pragma unroll
            for (uint32_t k = 0; k < kAhead; ++k) {
                const int2 v = __ldg(q + k * n);
                lo[k] = v.x, hi[k] = v.y;
            }
#pragma unroll
            for (uint32_t k = 0; k < kAhead; ++k) {
                past = past || (hi[k] >= 0 && (hi[k] > 0 || uint32_t(lo[k]) >= P.vocab));
                at[k] = hi[k] == 0 && uint32_t(lo[k]) - j0 < size ? uint32_t(lo[k]) - j0 : 0xFFFFFFFFu;
            }
            if (past && check) atomicOr(P.status, K3HUF_ST_TOKEN);
            return;
        }
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint32_t i = i0 + k * n;
            lo[k] = hi[k] = -1;
            if (i >= entries) continue;
            const bool bias = i >= n_history;
            const uint32_t wide = bias ? wide1 : wide0;
            const int32_t *q = static_cast<const int32_t *>(bias ? ids[1] : ids[0]) + uint64_t(bias ? i - n_history : i) * wide;
            lo[k] = __ldg(q);
            if (wide == 2) hi[k] = __ldg(q + 1);
        }
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            if ((i0 + k * n >= n_history ? wide1 : wide0) != 2) hi[k] = lo[k] >> 31;
            past = past || (hi[k] >= 0 && (hi[k] > 0 || uint32_t(lo[k]) >= P.vocab));
            at[k] = hi[k] == 0 && uint32_t(lo[k]) - j0 < size ? uint32_t(lo[k]) - j0 : 0xFFFFFFFFu;
        }
        if (past && check) atomicOr(P.status, K3HUF_ST_TOKEN);
    };
    // f(entry, its place) for the entries in the part; the first kAhead of every thread stay in registers
    uint32_t held[kAhead];
    auto each = [&](bool first_time, auto f) {
#pragma unroll 1
        for (uint32_t i0 = tid; i0 < entries; i0 += kAhead * n) {
            uint32_t at[kAhead];
            if (i0 == tid) {
#pragma unroll
                for (uint32_t k = 0; k < kAhead; ++k) at[k] = held[k];
            } else {
                load(i0, first_time && part == 0, at);
            }
#pragma unroll
            for (uint32_t k = 0; k < kAhead; ++k)
                if (at[k] != 0xFFFFFFFFu) f(i0 + k * n, at[k]);
        }
    };
    load(tid, part == 0, held);
    for (uint32_t w = tid; w < words; w += n) s_touched[w] = 0;
    sync();
    // (text has few tokens of many occurrences: most find their bit set.  A touched token's logit is wanted soon)
    each(true, [&](uint32_t, uint32_t at) {
        if (*const_cast<volatile uint32_t *>(&s_touched[at / 32]) >> (at % 32) & 1) return;
        asm volatile("prefetch.global.L1 [%0];" ::"l"(x + j0 + at));
        atomicOr(&s_touched[at / 32], 1u << (at % 32));
    });
    sync();
    // (a thread's words are n apart: their places count on in the order of the threads)
    uint32_t mine = 0;
#pragma unroll 4
    for (uint32_t w = tid; w < words; w += n) mine += __popc(s_touched[w]);
    uint32_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= uint32_t(d)) upto += v;
    }
    if (lane == 31) s_warp[warp] = upto;
    sync();
    const uint32_t of_warp = lane < n / 32 ? s_warp[lane] : 0u, all = __reduce_add_sync(0xffffffffu, of_warp);
    uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0u) + upto - mine;
#pragma unroll 4
    for (uint32_t w = tid; w < words; w += n) {
        s_before[w] = before;
        before += __popc(s_touched[w]);
    }
    bool streamed = !streams;
    // windows of so many places (nearly always one)
    for (uint32_t first = 0; first < all; first += P.places) {
        const uint32_t count = min(all - first, P.places);
        for (uint32_t i = tid; i < count; i += n) s_count[i] = s_bias[i] = 0;
        sync();
        each(false, [&](uint32_t i, uint32_t at) {
            const uint32_t p = s_before[at / 32] + __popc(s_touched[at / 32] & ((1u << (at % 32)) - 1u)) - first;
            if (p >= P.places) return;
            s_token[p] = at;
            if (i >= n_history) atomicMax(&s_bias[p], i - n_history + 1);      // (a token that is listed twice takes its last bias)
            else if (i < n_prompt) atomicOr(&s_count[p], kSeen);
            else atomicAdd(&s_count[p], 1u);
        });
        sync();
        // the touched tokens' new values (in place, the stream may write a token that it does not ban: the value it has)
        constexpr uint32_t kFew = 4;
#pragma unroll 1
        for (uint32_t p0 = tid; p0 < count; p0 += kFew * n) {
            float v[kFew], add[kFew];
            bool ban[kFew];
#pragma unroll
            for (uint32_t k = 0; k < kFew; ++k) {
                const uint32_t p = p0 + k * n;
                v[k] = add[k] = 0.f;
                ban[k] = true;
                if (p >= count) continue;
                const uint32_t j = j0 + s_token[p], bias = s_bias[p];
                v[k] = ld_f32(x + j);
                if (bias) add[k] = __ldg(bias_values + (bias - 1));
                ban[k] = banned(j);
            }
#pragma unroll
            for (uint32_t k = 0; k < kFew; ++k) {
                const uint32_t p = p0 + k * n;
                if (p >= count) continue;
                const uint32_t seen = s_count[p], times = seen & ~kSeen;
                float r = v[k];
                if (seen && c.repetition) r = r > 0.f ? r / repetition : r * repetition;
                if (times) {
                    r -= frequency * float(times);
                    r -= presence;
                }
                s_count[p] = __float_as_uint(s_bias[p] ? r + add[k] : r);
                if (ban[k]) s_token[p] = 0xFFFFFFFFu;
            }
        }
        if (!streamed) __syncthreads();       // (else each thread has its own)
        if (P.after) grid_dep_wait();
        streamed = true;
        for (uint32_t p = tid; p < count; p += n)
            if (s_token[p] != 0xFFFFFFFFu) st_f32(y + j0 + s_token[p], __uint_as_float(s_count[p]));
        if (all - first > P.places) sync();    // (the next window's counts)
    }
    if (!streamed) __syncthreads();
    if (P.after) grid_dep_wait();             // (a part without touched tokens too: this launch ends after the stream)
}

template <typename T, typename U>
int launch(ControlParams P, uint64_t n, cudaStream_t stream) {
    uint64_t sms = 0;
    const int rc = sm_count(&sms);
    if (rc) return rc;
    const bool streams = P.x != P.y || P.c.mask, lists = P.c.history || P.c.bias_ids;
    if (!streams && !lists) return K3HUF_OK;
    static std::atomic<uint64_t> once{0};
    const int attr_rc = once_per_device(once, [] { return cudaFuncSetAttribute(control_kernel<T, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kPart / 4 + 12 * kMostPlaces)); });
    if (attr_rc) return attr_rc;
    const uint64_t least = (uint64_t(P.vocab) + kPart - 1) / kPart, most = std::max<uint64_t>(least, P.vocab / 4096);
    auto run = [&](uint64_t parts, uint32_t threads, uint32_t streaming, bool after) {
        P.part = uint32_t(((P.vocab + parts - 1) / parts + 63) / 64 * 64);
        P.parts = (P.vocab + P.part - 1) / P.part;
        P.streaming = streaming;
        P.after = after;
        const uint64_t rows = 0x7FFFFFFFull / P.parts;
        for (uint64_t r0 = 0; r0 < n; r0 += rows) {
            P.row0 = r0;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(uint32_t(std::min(rows, n - r0) * P.parts));
            cfg.blockDim = dim3(threads);
            cfg.dynamicSmemBytes = streaming == threads ? 0 : P.part / 4 + 12 * P.places;
            cfg.stream = stream;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = after && r0 == 0;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            const cudaError_t e = cudaLaunchKernelEx(&cfg, control_kernel<T, U>, P);
            if (e != cudaSuccess) return cuda_rc(e);
        }
        return int(K3HUF_OK);
    };
    // Few rows: one launch, as many parts as there are SMs, a CTA of 1024 threads each, half of which see to the lists
    // (they take a thread's time per entry).  More, as long as the GPU holds two CTAs of 512 per SM for all: the same with
    // those (100 rows of 131072 10.7 us, 19 with two launches; 300 rows of 50021 20 and 26).  Many: a launch for the stream,
    // then one for the lists, which begins while the first one ends (400 rows of 50021 31 us, 33 with one launch; 1024 of
    // 131072 118 and 127).  Long lists touch more tokens than kPlaces, and each window reads them all again: such rows get
    // more places (432 rows of 14338 different tokens 92 us, 128 with 2048 places; 8 rows of 30000 33 us, 48).
    const uint64_t total = (P.c.history ? P.c.n_history : 0) + (P.c.bias_ids ? P.c.n_bias : 0);
    auto places = [&](uint64_t list, uint32_t limit) { return uint32_t(std::clamp<uint64_t>((list + kPlaces - 1) / kPlaces * kPlaces, kPlaces, limit)); };
    if (n <= sms / 2) {
        P.places = places(total, kMostPlaces);
        return run(std::max(least, std::min(most, sms / n)), kMaxThreads, !streams ? 0 : lists ? kMaxThreads / 2 : kMaxThreads, false);
    }
    P.places = places(total / n, kMostPlaces / 2);
    if (streams && lists && n <= 2 * sms) return run(std::max(least, std::min(most, sms * 2 / n)), 512, 256, false);
    if (streams) {
        const int stream_rc = run(std::max(least, std::min(most, sms * 24 / n)), 256, 256, false);
        if (stream_rc || !lists) return stream_rc;
    }
    // (of the lists, as many threads per row as the GPU has for it: 93 rows of 8000 entries 30 us with 256)
    return run(least, n <= sms ? 1024 : n <= 2 * sms || P.places > kPlaces ? 512 : 256, 0, streams);
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
    if (c.history && (!id_ok(c.history_id_bytes) || !aligned_to(c.history, c.history_id_bytes) || !c.spans || c.n_history > 0x40000000ull)) return K3HUF_E_ARG;
    if (c.bias_ids && (!id_ok(c.bias_id_bytes) || !aligned_to(c.bias_ids, c.bias_id_bytes) || !c.bias_values || !c.bias_spans || c.n_bias > 0x40000000ull)) return K3HUF_E_ARG;
    if (c.mask && (c.mask_stride < (uint64_t(vocab) + 31) / 32 || (!c.mask_rows && c.n_masks < n))) return K3HUF_E_ARG;
    if (n == 0) return K3HUF_OK;
    if (!d_logits || !d_out || (d_logits == d_out && (type != out_type || stride != out_stride))) return K3HUF_E_ARG;
    const ControlParams P{d_logits, d_out, c, d_status, stride, out_stride, 0, vocab, 1, 0, 0, kPlaces, false};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (type == K3HUF_BF16) return out_type == K3HUF_BF16 ? launch<__nv_bfloat16, __nv_bfloat16>(P, n, st) : launch<__nv_bfloat16, float>(P, n, st);
    return out_type == K3HUF_BF16 ? launch<float, __nv_bfloat16>(P, n, st) : launch<float, float>(P, n, st);
}
