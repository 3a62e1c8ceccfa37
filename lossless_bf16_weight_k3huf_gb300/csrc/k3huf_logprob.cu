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
// Logits of -infinity take no part (p_j = 0).
//
// Forward, one read of the logits: a CTA (128 threads, 256 for the largest
// vocabularies) streams a row (or, when there are fewer rows than the GPU holds CTAs, the CTAs of a cluster take a
// slice each and their results meet in the first one's shared memory).  Every
// thread keeps a running maximum with sum and dot rescaled to it (in base 2);
// 4 x 16 bytes per thread and step, the next step's loads issued before this
// one's arithmetic.  What bounds it: the read of the logits from HBM; per
// value one exponential and about six more instructions, half of them paired:
// 4095 rows of 131072 bf16 170 us, 6.3 TB/s;
// 270 us with 20 alternatives (2047 rows of fp32 189 us).
//
// Top alternatives in the same pass: a value can only be among the `top`
// largest if it is not below the top-th largest of any set of values.  The
// first step takes the top-th largest of 64 or 128 groups' largest values as the
// threshold (bit by bit within a warp); from then on a thread notes the vectors
// whose largest value reaches the threshold, without a barrier, and after steps
// 1, 4, 16, ... the CTA reads the noted vectors again, one value per thread, lists
// the keys that reach the threshold and cuts the list to its `top` largest, the
// last of which is the new threshold.  Rows that keep growing can fill the notes (ascending values): such a row's
// alternatives are taken again in a second read that counts and raises the
// threshold at every step.  A value's order as a whole number with its index
// below it is one key, so ties need no more.
//
// Backward: elementwise, 16 bytes per thread and load, one read and one write,
// at the rate of a copy: 2047 rows of 131072 bf16 157 us, 6.8 TB/s.
#include <cooperative_groups.h>

#include <cmath>

#include "k3huf_rows.h"

namespace cg = cooperative_groups;

namespace k3huf {
namespace {

constexpr int kGradThreads = 256;
constexpr int kVecs = 4;                      // 16-byte vectors per thread and step
constexpr int kMaxCluster = 16;
constexpr uint32_t kList = 2432;              // keys listed in shared memory
template <int kThreads> constexpr uint32_t kNotes = kVecs * kThreads;     // vectors noted: a step's
static_assert(K3HUF_MAX_TOP + (K3HUF_MAX_TOP + 8) * kVecs * 8 <= int(kList), "a counted step's notes and keys");

// (value, index) order of the top alternatives: larger values first, ties to
// the lower index.  +0 and -0 are equal and a NaN ranks as -infinity; never 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x == x ? x + 0.f : -INFINITY);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t j) { return (uint64_t(order_of(x)) << 32) | (0xFFFFFFFFu - j); }

// A running softmax state: e_j = 2^((x_j - m) c), sum of e_j, sum of e_j (x_j - m) c.
struct State {
    float m, sum, dot;
};
__device__ __forceinline__ void rescale(State &s, float m, float c) {
    const float d = max_nan((s.m - m) * c, kFloor), f = exp2_fast(d);
    s.dot = f * fmaf(d, s.sum, s.dot);
    s.sum *= f;
    s.m = m;
}
__device__ __forceinline__ State join(State a, State b, float c) {
    const float m = fmaxf(a.m, b.m);
    rescale(a, m, c);
    rescale(b, m, c);
    return {m, a.sum + b.sum, a.dot + b.dot};
}

// The `k`-th largest key of the CTA's threads (mine: each thread's own), down
// to bit `to`, given that its bits above `from` are those of `t`: the largest
// t' with k or more keys at or above it (0 if there are fewer than k keys).
__device__ uint64_t kth_largest(uint64_t mine, uint32_t k, uint64_t t, int from, int to) {
    for (int b = from; b >= to; --b) {
        const uint64_t tryit = t | (1ull << b);
        if (uint32_t(__syncthreads_count(mine >= tryit)) >= k) t = tryit;
    }
    return t;
}

struct LogprobParams {
    const void *x;
    const void *tokens;
    float *logprob, *entropy, *lse, *top_logprobs;
    int32_t *top_ids;
    uint32_t *status;
    uint64_t stride;
    uint32_t vocab, id_bytes, top;
    float scale, c;                           // c: scale log2 e, finite for every scale (infinity times a difference of 0 is NaN)
};

// Cuts the list to its `top` largest keys, the smallest of them last, and
// notes whether keys were lost because it was full.
template <int kThreads>
__device__ void cut_list(uint64_t *list, uint32_t *count, uint32_t *lost, uint32_t top) {
    constexpr int kMine = (kList + kThreads - 1) / kThreads;
    __shared__ uint32_t s_above[2];
    __syncthreads();
    const uint32_t n = min(*count, kList);
    if (n < *count && threadIdx.x == 0) *lost = 1;
    if (n < top) return;
    if (n <= 2 * kThreads) {
        // few: every key's rank is its place
        const uint64_t a = threadIdx.x < n ? list[threadIdx.x] : 0, b = threadIdx.x + kThreads < n ? list[threadIdx.x + kThreads] : 0;
        uint32_t above_a = 0, above_b = 0;
        if (n <= kThreads) {
            if (a)
                for (uint32_t i = 0; i < n; ++i) above_a += list[i] > a;
        } else {
            for (uint32_t i = 0; i < n; ++i) {
                const uint64_t k = list[i];
                above_a += k > a;
                above_b += k > b;
            }
        }
        __syncthreads();
        if (a && above_a < top) list[above_a] = a;
        if (b && above_b < top) list[above_b] = b;
        if (threadIdx.x == 0) *count = top;
        __syncthreads();
        return;
    }
    uint64_t mine[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) mine[i] = threadIdx.x + i * kThreads < n ? list[threadIdx.x + i * kThreads] : 0;
    if (threadIdx.x < 2) s_above[threadIdx.x] = 0;
    uint64_t t = 0;
    for (int b = 63; b >= 0; --b) {
        const uint64_t tryit = t | (1ull << b);
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) c += mine[i] >= tryit;
        c = __reduce_add_sync(0xffffffffu, c);
        __syncthreads();
        if (threadIdx.x % 32 == 0 && c) atomicAdd(&s_above[b & 1], c);
        if (threadIdx.x == 0) s_above[(b + 1) & 1] = 0;
        __syncthreads();
        if (s_above[b & 1] >= top) t = tryit;
    }
    if (threadIdx.x == 0) *count = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        if (mine[i] > t) list[atomicAdd(count, 1u)] = mine[i];        // (keys differ: t is one, and the last)
    __syncthreads();
    if (threadIdx.x == 0) list[(*count)++] = t;
    __syncthreads();
}

// kTop: 0 without alternatives, 1 for up to kNarrow (the first threshold is taken
// from 64 groups of threads), 2 for more (from 128; the 64th largest of 64 would be
// the smallest, and let 300 of a step's values through instead of 90: 1000 rows
// of 131072 with 64 alternatives 168 and 115 us, of 32000 124 and 60).
constexpr uint32_t kNarrow = 24;
template <typename T, int kTop, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logprob_kernel(const LogprobParams P) {
    constexpr int E = kPer<T>, kWarps = kThreads / 32;
    constexpr uint32_t kMaxNotes = kNotes<kThreads>;
    __shared__ State s_part[kWarps], s_all[kMaxCluster];
    __shared__ uint32_t s_count, s_noted, s_lost, s_counts[kMaxCluster], s_notes[kTop ? kMaxNotes : 1], s_group[kTop ? 64 * kTop : 1];
    __shared__ uint64_t s_list[kTop ? kList : 1];
    extern __shared__ uint64_t s_sent[];                   // (of the other CTAs of a cluster)
    const cg::cluster_group cluster = cg::this_cluster();
    const uint32_t C = cluster.num_blocks(), rank = cluster.block_rank(), row = blockIdx.x / C;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const T *x = static_cast<const T *>(P.x) + uint64_t(row) * P.stride;
    const float c = P.c;
    const uint32_t shift = uint32_t(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
    const uint32_t vecs = (P.vocab + shift + E - 1) / E;
    // this CTA's vectors: whole steps, as even as they come
    const uint32_t steps = (vecs + kThreads * kVecs - 1) / (kThreads * kVecs);
    const uint32_t step0 = uint32_t(uint64_t(steps) * rank / C), step1 = uint32_t(uint64_t(steps) * (rank + 1) / C);
    if (C > 1) cluster_arrive();                           // (waited for before the first remote store)
    if (kTop && tid == 0) s_count = s_noted = s_lost = 0;
    if (kTop) __syncthreads();

    uint4 v[kVecs], next[kVecs];
    auto load = [&](uint4 (&to)[kVecs], uint32_t step) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const uint32_t at = (step * kVecs + i) * kThreads + tid;
            to[i] = step < step1 && at < vecs ? load_vec(x, shift, P.vocab, at)
                                              : (sizeof(T) == 4 ? make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u)
                                                                : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u));
        }
    };
    // (-FLT_MAX, not -infinity: then -infinity minus it is -infinity)
    State s{-3.402823466e38f, 0.f, 0.f};
    uint64_t threshold = 0;
    // Notes this step's vectors that reach the threshold; `first`: sets it first; `count`: raises
    // it first where many do, so that at most top + 8 threads note any.
    auto note = [&](uint32_t step, const float (&top_of)[kVecs], float big, bool first, bool count) {
        const uint32_t few = P.top + 8, v0 = step * (kVecs * kThreads) + tid;
        const uint32_t mine = v0 < vecs ? order_of(big) : 0u;
        // (no value of this thread's step has a lower index than its first vector's first)
        const uint32_t low = 0xFFFFFFFFu - (v0 ? v0 * E - shift : 0u);
        auto reaches = [&](uint64_t t) { return mine && ((uint64_t(mine) << 32) | low) >= t; };
        bool raised = false;
        uint64_t t = 0;
        if (first) {
            // the top-th largest of the largest values of 64 or 128 groups of threads
            constexpr int kSets = kTop ? 2 * kTop : 1, kGroup = kThreads / (32 * kSets);
            uint32_t most = mine;
#pragma unroll
            for (int d = 1; d < kGroup; d <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
            if (tid % kGroup == 0) s_group[tid / kGroup] = most;
            __syncthreads();
            uint32_t g[kSets], hi = 0;
#pragma unroll
            for (int i = 0; i < kSets; ++i) g[i] = s_group[lane + 32 * i];
            for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit >>= 1) {
                uint32_t above = 0;
#pragma unroll
                for (int i = 0; i < kSets; ++i) above += __popc(__ballot_sync(0xffffffffu, g[i] >= (hi | bit)));
                if (above >= P.top) hi |= bit;
            }
            t = uint64_t(hi) << 32;
            raised = true;
        } else if (count && uint32_t(__syncthreads_count(reaches(threshold))) > few) {
            // (the 16 high bits are a bf16 value; for fp32 a little lower a threshold)
            t = kth_largest(uint64_t(mine) << 32, P.top, 0, 63, 48);
            raised = true;
        }
        if (raised) {
            // (0: fewer than `top` groups or threads have values at all)
            if (t && uint32_t(__syncthreads_count((uint64_t(mine) << 32) >= t)) > (count ? few : 4 * few)) {
                // many equal ones: the whole key of each thread's first largest value decides
                uint64_t key = 0;
#pragma unroll 1
                for (int i = 0; i < kVecs; ++i)
                    for (int k = 0; k < E; ++k) {
                        const int64_t j = int64_t(v0 + i * kThreads) * E + k - shift;
                        if (j >= 0 && j < int64_t(P.vocab)) key = max(key, key_of(ld_f32(x + j), uint32_t(j)));
                    }
                t = kth_largest(key, P.top, 0, 63, 0);
            }
            threshold = max(threshold, t);
        }
        if (reaches(threshold)) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                if (v0 + i * kThreads < vecs && order_of(top_of[i]) >= uint32_t(threshold >> 32)) {
                    const uint32_t at = atomicAdd(&s_noted, 1u);
                    if (at < kMaxNotes) s_notes[at] = v0 + i * kThreads;
                }
        }
    };
    // Lists the noted vectors' keys and raises the threshold to the top-th largest so far.
    auto raise = [&]() {
        __syncthreads();
        const uint32_t noted = min(s_noted, kMaxNotes);
        if (tid == 0 && s_noted > kMaxNotes) s_lost = 1;
        for (uint32_t i = tid; i < noted * E; i += kThreads) {
            const int64_t j = int64_t(s_notes[i / E]) * E + i % E - shift;
            if (j < 0 || j >= int64_t(P.vocab)) continue;
            const uint64_t key = key_of(ld_f32(x + j), uint32_t(j));
            if (key < threshold) continue;
            const uint32_t at = atomicAdd(&s_count, 1u);
            if (at < kList) s_list[at] = key;
        }
        cut_list<kThreads>(s_list, &s_count, &s_lost, P.top);
        if (s_count >= P.top) threshold = max(threshold, s_list[P.top - 1]);
        if (tid == 0) s_noted = 0;
        __syncthreads();
    };
    load(next, step0);
    for (uint32_t step = step0; step < step1; ++step) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = next[i];
        load(next, step + 1);
        float top_of[kVecs], big = -INFINITY;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) big = fmaxf(big, top_of[i] = vec_max<T>(v[i]));
        rescale(s, fmaxf(s.m, big), c);
        const float2 minus_m = make_float2(-s.m, -s.m), cc = make_float2(c, c);
        float2 sum = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float f[E];
            unpack<T>(v[i], f);
#pragma unroll
            for (int k = 0; k < E; k += 2) {
                float2 t = __fmul2_rn(__fadd2_rn(make_float2(f[k], f[k + 1]), minus_m), cc);
                t.x = max_nan(t.x, kFloor);
                t.y = max_nan(t.y, kFloor);
                const float2 e = make_float2(exp2_fast(t.x), exp2_fast(t.y));
                sum = __fadd2_rn(sum, e);
                dot = __ffma2_rn(e, t, dot);
            }
        }
        s.sum += sum.x + sum.y;
        s.dot += dot.x + dot.y;
        if constexpr (kTop) {
            note(step, top_of, big, step == step0, false);
            const uint32_t done = step - step0;
            if (step + 1 < step1 && done && (done & (done - 1)) == 0 && (done & 0x55555555u)) raise();
        }
    }
    if constexpr (kTop) {
        raise();
        if (s_lost) {
            threshold = 0;
            if (tid == 0) s_count = 0;
#pragma unroll 1
            for (uint32_t step = step0; step < step1; ++step) {
                load(v, step);
                float top_of[kVecs], big = -INFINITY;
#pragma unroll
                for (int i = 0; i < kVecs; ++i) big = fmaxf(big, top_of[i] = vec_max<T>(v[i]));
                note(step, top_of, big, false, true);
                raise();
            }
        }
    }
    // the CTA's state, and its candidates
#pragma unroll
    for (int d = 16; d; d >>= 1) s = join(s, State{__shfl_xor_sync(0xffffffffu, s.m, d), __shfl_xor_sync(0xffffffffu, s.sum, d), __shfl_xor_sync(0xffffffffu, s.dot, d)}, c);
    if (lane == 0) s_part[warp] = s;
    __syncthreads();
    s = s_part[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s = join(s, s_part[w], c);
    uint32_t count = kTop ? s_count : 0;
    if (C > 1) {
        // to the first CTA of the cluster: the state, and at most `top` candidates
        cluster_wait();
        if (tid == 0) {
            cluster.map_shared_rank(s_all, 0)[rank] = s;
            if (kTop) cluster.map_shared_rank(s_counts, 0)[rank] = count;
        }
        if (kTop && rank > 0)
            for (uint32_t i = tid; i < count; i += kThreads) cluster.map_shared_rank(s_sent, 0)[(rank - 1) * K3HUF_MAX_TOP + i] = s_list[i];
        cluster_arrive();
        cluster_wait();
        if (rank > 0) return;
        for (uint32_t r = 1; r < C; ++r) s = join(s, s_all[r], c);
        if (kTop) {
            for (uint32_t r = 1; r < C; ++r) {
                for (uint32_t i = tid; i < s_counts[r]; i += kThreads) s_list[count + i] = s_sent[(r - 1) * K3HUF_MAX_TOP + i];
                count += s_counts[r];
            }
            if (tid == 0) s_count = count;
            __syncthreads();
        }
    }
    // a row with no finite logit: sum is 0, lse -infinity
    const bool none = s.sum == 0.f;
    const float log2sum = log2f(s.sum), logsum = log2sum * kLn2;
    // (a logit of -infinity where the sum is 0, whose log is -infinity too; a NaN sum goes on)
    auto log_prob = [&](float z) { return z == -INFINITY && s.sum == s.sum ? z : fmaf(z - s.m, P.scale, -logsum); };
    if (tid == 0) {
        const int64_t t = ld_id(P.tokens, P.id_bytes, row);
        float lp = 0.f;
        if (t >= int64_t(P.vocab)) atomicOr(P.status, K3HUF_ST_TOKEN);
        else if (t >= 0) lp = log_prob(ld_f32(x + t));
        P.logprob[row] = lp;
        if (P.entropy) P.entropy[row] = none ? 0.f : logsum - s.dot / s.sum * kLn2;
        if (P.lse) P.lse[row] = none ? -INFINITY : fmaf(s.m, P.scale, logsum);
    }
    if constexpr (kTop) {
        if (count > 2 * kThreads) {
            cut_list<kThreads>(s_list, &s_count, &s_lost, P.top);
            count = s_count;
        }
        for (uint32_t i = tid; i < count; i += kThreads) {
            const uint64_t key = s_list[i];
            uint32_t above = 0;
            for (uint32_t k = 0; k < count; ++k) above += s_list[k] > key;
            if (above >= P.top) continue;
            const uint32_t j = 0xFFFFFFFFu - uint32_t(key);
            P.top_ids[uint64_t(row) * P.top + above] = int32_t(j);
            P.top_logprobs[uint64_t(row) * P.top + above] = log_prob(ld_f32(x + j));
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
    uint32_t vocab, id_bytes;
    float scale;
};

constexpr int kGradVecs = 4;

// kVec: logits and gradients sit alike in their 16-byte blocks
template <typename T, bool kVec>
__global__ void __launch_bounds__(kGradThreads) logprob_grad_kernel(const GradParams P) {
    constexpr int E = kVec ? kPer<T> : 1;
    const uint32_t row = blockIdx.y;
    const T *x = static_cast<const T *>(P.x) + uint64_t(row) * P.stride;
    T *dx = static_cast<T *>(P.dx) + uint64_t(row) * P.dx_stride;
    const uint32_t shift = kVec ? uint32_t(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T)) : 0u;
    const int64_t t = ld_id(P.tokens, P.id_bytes, row);
    const bool scored = t >= 0 && t < int64_t(P.vocab);
    if (!scored && t >= 0 && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.status, K3HUF_ST_TOKEN);
    const float g = scored ? P.g_logprob[row] : 0.f;
    const float h = P.g_entropy ? P.g_entropy[row] : 0.f, ent = P.g_entropy ? P.entropy[row] : 0.f, lse = P.lse[row];
    // dx_j = p_j (hs lp_j + gs), and scale g more at the token; two values at a time.  A logit of
    // -infinity, and one so low that p_j is 0, stop at kFloor: 0 times infinity is not 0.  p_j is 1 at
    // most: where logits are so large (masks of the type's lowest value in a whole row) that lse is
    // off by more than 1, a log of p_j above 0 would give infinities.
    const float hs = -h * P.scale, gs = -P.scale * fmaf(h, ent, g), base = lse == -INFINITY ? 0.f : -lse;
    auto grad = [&](float2 v) {
        float2 lp = __ffma2_rn(v, make_float2(P.scale, P.scale), make_float2(base, base));
        lp.x = min_nan(max_nan(lp.x, kFloor), 0.f);
        lp.y = min_nan(max_nan(lp.y, kFloor), 0.f);
        const float2 a = __fmul2_rn(lp, make_float2(kLog2e, kLog2e));
        return __fmul2_rn(make_float2(exp2_fast(a.x), exp2_fast(a.y)), __ffma2_rn(make_float2(hs, hs), lp, make_float2(gs, gs)));
    };
    const uint32_t token = scored ? uint32_t(t) : 0xFFFFFFFFu;
    const uint32_t vecs = (P.vocab + shift + E - 1) / E;
    const uint32_t v0 = blockIdx.x * (kGradThreads * kGradVecs) + threadIdx.x;
    if constexpr (kVec) {
        uint4 v[kGradVecs];
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i)
            if (v0 + i * kGradThreads < vecs) v[i] = load_vec(x, shift, P.vocab, v0 + i * kGradThreads);
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            if (v0 + i * kGradThreads >= vecs) break;
            const int64_t j = int64_t(v0 + i * kGradThreads) * E - shift;
            float f[E];
            unpack<T>(v[i], f);
#pragma unroll
            for (int k = 0; k < E; k += 2) {
                const float2 d = grad(make_float2(f[k], f[k + 1]));
                f[k] = d.x;
                f[k + 1] = d.y;
            }
            if (token - uint32_t(j) < uint32_t(E)) {
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (token == uint32_t(j) + k) f[k] = fmaf(P.scale, g, f[k]);
            }
            if (j >= 0 && j + E <= int64_t(P.vocab)) {
                uint4 o;
                if constexpr (sizeof(T) == 4) {
                    o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
                } else {
                    __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
                    for (int k = 0; k < 4; ++k) q[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
                }
                __stcs(reinterpret_cast<uint4 *>(dx + j), o);
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (j + k >= 0 && j + k < int64_t(P.vocab)) st_f32(dx + j + k, f[k]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            const uint32_t j = v0 + i * kGradThreads;
            if (j >= vecs) break;
            const float d = grad(make_float2(ld_f32(x + j), 0.f)).x;
            st_f32(dx + j, j == token ? fmaf(P.scale, g, d) : d);
        }
    }
}

template <typename T, int kTop, int kThreads>
int launch_forward(const LogprobParams &P, uint32_t n, cudaStream_t stream) {
    // one CTA per row, or a cluster per row while the GPU has room for more CTAs (two or
    // more per SM) and every CTA still has a step to do
    constexpr uint32_t kStep = kThreads * kVecs * kPer<T>;
    static std::atomic<uint64_t> wide{0};
    const int rc = once_per_device(wide, [] { return cudaFuncSetAttribute(logprob_kernel<T, kTop, kThreads>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
    if (rc) return rc;
    uint64_t sms = 0;
    const int sm_rc = sm_count(&sms);
    if (sm_rc) return sm_rc;
    uint32_t C = 1;
    while (C < uint32_t(kMaxCluster) && n * C < sms * 512 / kThreads && P.vocab / kStep >= 2 * C) C *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n * C);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.dynamicSmemBytes = kTop && C > 1 ? (kMaxCluster - 1) * K3HUF_MAX_TOP * sizeof(uint64_t) : 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_rc(cudaLaunchKernelEx(&cfg, logprob_kernel<T, kTop, kThreads>, P));
}

// CTAs of 128 threads, twice as many rows at once, up to this vocabulary, of 256
// above it.  4000 rows of bf16 logits with 20 alternatives, 128 and 256 threads:
// 35 and 52 us at 4096, 115 and 117 at 32768, 177 both at 65536, 289 and 279 at
// 131072; without alternatives 19 and 29, 54 and 60, 93 and 98, 177 and 175.
constexpr uint32_t kSmallVocab = 65536;
template <typename T, int kTop>
int launch_forward(const LogprobParams &P, uint32_t n, cudaStream_t stream) {
    return P.vocab <= kSmallVocab ? launch_forward<T, kTop, 128>(P, n, stream) : launch_forward<T, kTop, 256>(P, n, stream);
}

template <typename T>
int launch_forward(const LogprobParams &P, uint32_t n, cudaStream_t stream) {
    return P.top == 0 ? launch_forward<T, 0>(P, n, stream) : P.top <= kNarrow ? launch_forward<T, 1>(P, n, stream) : launch_forward<T, 2>(P, n, stream);
}

template <typename T>
int launch_backward(const GradParams &P, uint32_t n, cudaStream_t stream) {
    const bool vec = (reinterpret_cast<uintptr_t>(P.x) - reinterpret_cast<uintptr_t>(P.dx)) % 16 == 0 &&
                     (P.stride - P.dx_stride) * sizeof(T) % 16 == 0;
    const uint32_t per = kGradThreads * kGradVecs * (vec ? kPer<T> : 1);
    // (a row that starts inside a 16-byte block may need one vector more)
    const uint32_t bx = uint32_t((uint64_t(P.vocab) + (vec ? kPer<T> - 1 : 0) + per - 1) / per);
    for (uint32_t r0 = 0; r0 < n; r0 += 65535) {
        GradParams Q = P;
        Q.x = static_cast<const T *>(P.x) + uint64_t(r0) * P.stride;
        Q.dx = static_cast<T *>(P.dx) + uint64_t(r0) * P.dx_stride;
        Q.tokens = static_cast<const uint8_t *>(P.tokens) + uint64_t(r0) * P.id_bytes;
        Q.lse += r0;
        Q.g_logprob += r0;
        if (Q.entropy) Q.entropy += r0;
        if (Q.g_entropy) Q.g_entropy += r0;
        const dim3 grid(bx, min(65535u, n - r0));
        if (vec) logprob_grad_kernel<T, true><<<grid, kGradThreads, 0, stream>>>(Q);
        else logprob_grad_kernel<T, false><<<grid, kGradThreads, 0, stream>>>(Q);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_rc(e);
    }
    return K3HUF_OK;
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
    const LogprobParams P{d_logits, d_tokens, d_logprob, d_entropy, d_lse, d_top_logprobs, d_top_ids, d_status, stride, vocab, id_bytes, top, scale, fminf(scale * kLog2e, 3.402823466e38f)};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (type == K3HUF_BF16)
        return launch_forward<__nv_bfloat16>(P, uint32_t(n), st);
    return launch_forward<float>(P, uint32_t(n), st);
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
    const GradParams P{d_logits, d_dlogits, d_tokens, d_lse, d_entropy, d_g_logprob, d_g_entropy, d_status, stride, out_stride, vocab, id_bytes, scale};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return type == K3HUF_BF16 ? launch_backward<__nv_bfloat16>(P, uint32_t(n), st) : launch_backward<float>(P, uint32_t(n), st);
}
