// Distillation of a row of logits from a teacher's top alternatives, and its gradient.
//
// With z = s x the student's scaled logits, p = softmax(z), and q_i = exp(t_i) the teacher's probabilities of its
// alternatives i (t_i as given, or less their log-sum-exp where the alternatives are taken as the whole):
//   loss = sum_i q_i (t_i - log p_i)  [ + q_r (log q_r - log p_r) ]
// where the bracket is the rest's share if it is wanted: q_r = 1 - sum_i q_i, p_r = 1 - sum_i p_i, the sum of the
// other tokens' p.  With Q = sum_i q_i (+ q_r), g the upstream gradient:
//   dx_j = s g (Q p_j - q_j) for an alternative,   s g (Q - q_r / p_r) p_j for another token.
//
// A loss is what is left of terms far larger than itself, so what there are few of (the alternatives' terms, the
// rest's mass, the logarithms) is computed in 64 bits or pairs of floats; the sum over the vocabulary in 32.  p_r is summed over the
// other tokens alone, never taken as a difference, beside their own maximum: a small rest keeps its digits, and its logarithm
// reaches as far down as the logits do.
//
// Forward, one read of the logits: a CTA streams a row, or the CTAs of a cluster when there are fewer rows than the
// GPU holds CTAs.  To leave the alternatives out of the rest's sum, every thread has a bit for each of its
// vectors (modulo 64); it passes over those that may hold one, and the warp beside the stream adds what else they
// hold.  What bounds it: the read of the logits, 4095 rows of 131072 bf16 164 us (6.5 TB/s), 188 with the rest, whose
// rows cannot start before their alternatives are known.
//
// Backward: elementwise; every other token's gradient is s g (Q p_r - q_r) exp(z_j - lse - log p_r), the
// alternatives' are written over it behind a barrier.  The CTAs stay, and a warp beside the stream prepares the next
// piece's factors: 2047 rows of 131072 bf16 165 us, 6.5 TB/s (412 with the factors computed where they are used).
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

#include "k3huf_rows.h"

namespace cg = cooperative_groups;

namespace k3huf {
namespace {

constexpr int kThreads = 256;                 // that stream; one warp more sees to the alternatives
constexpr int kAll = kThreads + 32;
constexpr int kVecs = 4;                      // 16-byte vectors per thread and step
constexpr int kMaxCluster = 16;
static_assert(64 % kVecs == 0, "a step's bits lie side by side in a mask of 64");

struct Sum {
    float m, sum;                             // sum of 2^((x - m) c)
};
__device__ __forceinline__ void rescale(Sum &s, float m, float c) {
    s.sum *= exp2_fast(max_nan((s.m - m) * c, kFloor));
    s.m = m;
}
// 64-bit arithmetic runs at a sixtieth of the 32-bit rate here: 4992 rows of 1744 logits took 52 us with it throughout, 5 of
// them for their bytes.  So exponentials, logarithms and sums are taken in pairs of floats, a value and what its rounding left
// (Dekker's double-length numbers): 45 bits and more.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {               // a + b, without loss
    const float s = a + b, other = s - a;
    return {s, (a - (s - other)) + (b - other)};
}
__device__ __forceinline__ Two two_fast(float a, float b) {              // ... of |a| >= |b|
    const float s = a + b;
    return {s, b - (s - a)};
}
__device__ __forceinline__ Two two_mul(Two a, Two b) {
    const float p = __fmul_rn(a.hi, b.hi);
    return {p, fmaf(a.hi, b.hi, -p) + fmaf(a.hi, b.lo, a.lo * b.hi)};
}
__device__ __forceinline__ double wide(Two a) { return double(a.hi) + double(a.lo); }
__device__ __forceinline__ Two narrow(double a) {                         // (an infinity's rest would be NaN)
    const float hi = float(a);
    return {hi, isfinite(hi) ? float(a - double(hi)) : 0.f};
}

// e^a for |a| <= 80: a = n ln 2 + 16 u with ln 2 in three parts, whose first two give exact products with n (Cody and Waite's
// reduction); w = e^u - 1 by its series, whose terms from the third on need but 32 bits (|u| < 0.022: 2e-13 of 1); then four
// times e^2u - 1 = 2 w + w^2.  In all 4e-12 of the result at most.
constexpr float kExpMost = 80.f;
__device__ __forceinline__ Two two_exp(Two a) {
    constexpr double ln2 = 0.693147180559945309417;
    constexpr float l1 = float(int(ln2 * 131072)) / 131072.f, l2 = float(int((ln2 - l1) * 17179869184.)) / 17179869184.f, l3 = float(ln2 - l1 - l2);
    const float n = rintf(a.hi * kLog2e);
    Two u = two_sum(fmaf(-n, l1, a.hi), -n * l2);
    u = two_sum(u.hi, u.lo + fmaf(-n, l3, a.lo));
    const float h = u.hi * 0.0625f, l = u.lo * 0.0625f;
    const float square = __fmul_rn(h, h), left = fmaf(h, h, -square);
    const float tail = square * h * fmaf(h, fmaf(h, fmaf(h, 1.f / 720, 1.f / 120), 1.f / 24), 1.f / 6);
    Two w = two_fast(h, 0.5f * square);
    w = two_fast(w.hi, w.lo + (tail + (l + fmaf(h, l, 0.5f * left))));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float p = __fmul_rn(w.hi, w.hi), e = fmaf(w.hi, w.hi, -p);
        const Two s = two_fast(2.f * w.hi, p);
        w = two_fast(s.hi, s.lo + fmaf(2.f, w.lo, fmaf(2.f * w.hi, w.lo, e)));
    }
    const Two one = two_fast(1.f, w.hi);
    const float power = __int_as_float((int(n) + 127) << 23);
    return {one.hi * power, (one.lo + w.lo) * power};
}
// log v, by a whole warp: y = logf(v) and, as v e^-y is 1 but for 2e-6 at most, what that is off (its square's half beside it)
__device__ __forceinline__ double log_of(double v) {
    const float f = float(v);
    if (__any_sync(0xffffffffu, !(f >= 1e-30f && f <= 1e30f))) return log(v);
    const float y = logf(f);
    const double d = fma(v, wide(two_exp({-y, 0.f})), -1.);
    const float low = float(d);
    return double(y) + (d - double(0.5f * low * low));
}
__device__ __forceinline__ Two warp_sum(Two v) {                          // (of finite values)
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float b = __shfl_xor_sync(0xffffffffu, v.hi, d);
        const Two s = two_sum(v.hi, b);
        v = {s.hi, v.lo + __shfl_xor_sync(0xffffffffu, v.lo, d) + s.lo};
    }
    return v;
}

// A warp's sums as one, its largest value and the sum: every lane's is brought to that value once, by an exponent
// whose rounding is made good, and they are added up without loss (each addition's rounding error in a sum of its own).
// Sums joined pair by pair, 32 bits each, were 5e-8 off: as much as a loss between near distributions shows.
struct Part {
    float m;
    Two sum;
};
__device__ __forceinline__ Part warp_part(Sum s, float c) {
    float m = s.m;
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    // (far below the largest there is nothing to make good, and infinities of the difference would give NaN)
    const float d = s.m - m, t = max_nan(d * c, kFloor), low = t > kFloor ? fmaf(d, c, -t) : 0.f;
    return {m, warp_sum(Two{s.sum * exp2_fast(t) * fmaf(low, kLn2, 1.f), 0.f})};
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
// (x - m) scale
__device__ __forceinline__ Two below(float x, float m, Two scale) {
    const Two a = two_mul(two_sum(0.5f * x, -0.5f * m), scale);           // (halves: a difference of 6e38 has its place too)
    return {2.f * a.hi, 2.f * a.lo};
}
// e^a for a <= 0; nothing below e^-80, which no sum with a term of 1 shows
__device__ __forceinline__ Two weight(Two a) { return a.hi < -kExpMost ? Two{0.f, 0.f} : two_exp(a); }
// ... to 32 bits, for what is 1 for the largest part (the rounding of a alone would cost |a| 2^-24 of it)
__device__ __forceinline__ float weight32(Two a) {
    const float e = a.hi < -kExpMost ? 0.f : expf(a.hi);
    return e == 0.f ? 0.f : fmaf(e, a.lo, e);
}

// Of a warp's list (entry `lane`, and lane + 32 where it has more than 32; below 0: none) the entries that are like another
// one, a bit each.  There are few, and what depends on an entry's likes looks at those alone.
__device__ __forceinline__ uint64_t alike(int32_t a, int32_t b, bool more, uint32_t lane) {
    bool a_like = false, b_like = false;
#pragma unroll
    for (uint32_t k = 0; k < 32; ++k) {
        const int32_t one = __shfl_sync(0xffffffffu, a, k);
        a_like |= one == a && k != lane;
        b_like |= one == b;
    }
    if (more) {
#pragma unroll
        for (uint32_t k = 0; k < 32; ++k) {
            const int32_t one = __shfl_sync(0xffffffffu, b, k);
            a_like |= one == a;
            b_like |= one == b && k != lane;
        }
    }
    return __ballot_sync(0xffffffffu, a_like && a >= 0) | uint64_t(__ballot_sync(0xffffffffu, b_like && b >= 0)) << 32;
}

struct Teacher {
    const int32_t *ids;
    const float *top;
    uint32_t count, mode;                     // alternatives per row
};

// A row's alternatives, by one warp: entry `lane`, and, of more than 32, entry lane + 32 (id -1: none, q 0).  Nothing is
// computed for a second entry that is not there.
struct Alternatives {
    int32_t id[2];
    double t[2], q[2];                        // log q + log `whole` (-infinity for none), q
    double mass, rest;                        // sum of q; what is left of 1, where that is wanted
    double whole;                             // what the q were divided by
    bool any;
};
__device__ __forceinline__ Alternatives alternatives(const Teacher &T, uint64_t row, uint32_t vocab, uint32_t lane, uint32_t *status) {
    Alternatives A;
    const int entries = T.count > 32 ? 2 : 1;
    A.whole = 1.;
    float top[2];                             // (fetched beside the ids, not after them)
#pragma unroll
    for (int e = 0; e < 2; ++e) top[e] = lane + 32 * e < T.count ? T.top[row * T.count + lane + 32 * e] : 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t i = lane + 32 * e;
        A.id[e] = i < T.count ? T.ids[row * T.count + i] : -1;
        if (A.id[e] >= 0 && uint32_t(A.id[e]) >= vocab) {
            if (status) atomicOr(status, K3HUF_ST_TOKEN);
            A.id[e] = -1;
        }
        if (A.id[e] < 0) top[e] = -INFINITY;
    }
    A.any = __any_sync(0xffffffffu, A.id[0] >= 0 || A.id[1] >= 0);
    float m = 0.f;
    if (T.mode == K3HUF_DISTILL_NORMALISED) {
        // (the largest; where it is -infinity every q is 0; NaN, and +infinity, make the row NaN)
        float most = fmaxf(top[0], top[1]);
#pragma unroll
        for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        m = most == -INFINITY ? 0.f : most;
    }
    auto within = [&](float t) { return t == -INFINITY || fabsf(t - m) <= kExpMost; };
    if (__all_sync(0xffffffffu, within(top[0]) && within(top[1]))) {
        Two mass{0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            A.t[e] = -INFINITY, A.q[e] = 0.;
            if (e >= entries) break;
            if (top[e] == -INFINITY) continue;
            const Two t = two_sum(top[e], -m), q = two_exp(t), sum = two_sum(mass.hi, q.hi);
            A.t[e] = wide(t), A.q[e] = wide(q);
            mass = {sum.hi, sum.lo + mass.lo + q.lo};
        }
        A.mass = wide(warp_sum(mass));
    } else {
        double mass = 0.;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            A.t[e] = double(top[e]) - double(m);
            A.q[e] = top[e] == -INFINITY ? 0. : exp(A.t[e]);
            mass += A.q[e];
        }
        A.mass = warp_sum(mass);
    }
    if (T.mode == K3HUF_DISTILL_NORMALISED && !(A.mass == 0.)) {
        // (the largest q is 1, and of 64 none is larger: a reciprocal, once refined, has 45 bits)
        const double first = 1.f / float(A.mass), one = fma(first, fma(-A.mass, first, 1.), first);
        A.whole = A.mass;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (e < entries) A.q[e] *= one;
        A.mass = A.mass == A.mass ? 1. : A.mass;
    }
    A.rest = T.mode != K3HUF_DISTILL_REST ? 0. : A.mass > 1. ? 0. : 1. - A.mass;
    return A;
}

struct DistillParams {
    const void *x;
    Teacher teacher;
    float *loss, *lse, *log_rest;
    uint32_t *status;
    uint64_t stride;
    uint32_t vocab;
    float c;                                  // scale log2 e, finite for every scale
    double scale;                             // c ln 2: what the sum is taken with, so that c's rounding meets both sides of a loss
    Two scale2;                               // ... in floats
};

// What the alternatives give to the loss, by the warp that does not stream, while the others do.
struct Terms {
    double sum, mass, rest, whole;            // sum of q (t + log whole - s (x - from)); of q; the rest's q
    float from, top;                          // the largest of their logits, and, where it is not finite, 0
    Two top_sum;                              // sum of exp(s (x - top)), each token once
    uint32_t any;
};
template <typename T, bool kRest>
__device__ Terms terms(const DistillParams &P, const T *x, uint64_t row, uint32_t lane) {
    const Alternatives A = alternatives(P.teacher, row, P.vocab, lane, P.status);
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) f[e] = A.id[e] >= 0 ? ld_f32(x + A.id[e]) : -INFINITY;
    float top = fmaxf(f[0], f[1]);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    // (logits of 1e38 would leave nothing of t beside them)
    Terms R{0., A.mass, A.rest, A.whole, isfinite(top) ? top : 0.f, top, {0.f, 0.f}, A.any};
    const int entries = P.teacher.count > 32 ? 2 : 1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (e >= entries) break;
        if (A.id[e] >= 0 && !(A.q[e] == 0.)) R.sum += A.q[e] * (A.t[e] - (double(f[e]) - double(R.from)) * P.scale);
    }
    R.sum = warp_sum(R.sum);
    if constexpr (kRest) {
        // (a token that is listed twice counts at its first place)
        bool first[2] = {A.id[0] >= 0, A.id[1] >= 0};
        for (uint64_t left = alike(A.id[0], A.id[1], entries > 1, lane); left; left &= left - 1) {
            const uint32_t k = __ffsll(left) - 1;
            const int32_t id = __shfl_sync(0xffffffffu, k < 32 ? A.id[0] : A.id[1], k % 32);
            if (k < lane && id == A.id[0]) first[0] = false;
            if (k < lane + 32 && id == A.id[1]) first[1] = false;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (e >= entries) break;
            if (!first[e] || f[e] == -INFINITY) continue;
            const Two p = weight(below(f[e], top, P.scale2)), sum = two_sum(R.top_sum.hi, p.hi);
            R.top_sum = {sum.hi, sum.lo + R.top_sum.lo + p.lo};
        }
        R.top_sum = warp_sum(R.top_sum);
    }
    return R;
}

// Adds vectors of logits to a running sum.
template <typename T, int N>
__device__ __forceinline__ void add_vectors(Sum &s, const uint4 (&v)[N], float c) {
    constexpr int E = kPer<T>;
    float big = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) big = fmaxf(big, vec_max<T>(v[i]));
    rescale(s, fmaxf(s.m, big), c);
    const float2 minus_m = make_float2(-s.m, -s.m), cc = make_float2(c, c);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float f[E];
        unpack<T>(v[i], f);
#pragma unroll
        for (int k = 0; k < E; k += 2) {
            float2 t = __fmul2_rn(__fadd2_rn(make_float2(f[k], f[k + 1]), minus_m), cc);
            t.x = max_nan(t.x, kFloor);
            t.y = max_nan(t.y, kFloor);
            sum = __fadd2_rn(sum, make_float2(exp2_fast(t.x), exp2_fast(t.y)));
        }
    }
    s.sum += sum.x + sum.y;
}
template <typename T> __device__ __forceinline__ uint4 nothing() {       // a vector of -infinity
    constexpr uint32_t w = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
    return make_uint4(w, w, w, w);
}

// The sum of what the vectors that the stream passes over hold beside the alternatives, of the CTA's steps: those that share
// a bit with an alternative's (`places`: vector and element of each), one per lane of the warp that does not stream.  (Apart
// from the kernel, whose registers it would take.)
template <typename T, int kThreads>
__device__ __noinline__ Sum passed_over(const T *x, uint32_t shift, uint32_t vocab, uint32_t vecs, uint32_t step0, uint32_t step1, const uint2 *places, uint32_t count, float c) {
    Sum s{-3.402823466e38f, 0.f};
    const uint32_t turns = (vecs + kThreads * 64 - 1) / (kThreads * 64), lane = threadIdx.x % 32;                 // vectors per bit
    auto bit_of = [&](uint32_t k) { return k >= count || places[k].x == 0xFFFFFFFFu ? -1 : int32_t(places[k].x % (kThreads * 64)); };
    const uint64_t sharing = alike(bit_of(lane), bit_of(lane + 32), count > 32, lane);
    for (uint32_t e = lane; e < count * turns; e += 32) {
        const uint32_t k = e % count, of = places[k].x, home = of % (kThreads * 64), at = home + e / count * (kThreads * 64);
        if (of == 0xFFFFFFFFu || at >= vecs || at / (kThreads * kVecs) < step0 || at / (kThreads * kVecs) >= step1) continue;
        uint4 one[1] = {load_vec(x, shift, vocab, at)};
        // (its bit is another's, earlier in the list: that one's thread adds it)
        uint32_t out = of == at ? 1u << places[k].y : 0u;
        bool mine = true;
        for (uint64_t left = sharing; left; left &= left - 1) {
            const uint32_t q = __ffsll(left) - 1;
            const uint2 p = places[q];
            mine = mine && !(q < k && p.x % (kThreads * 64) == home);
            out |= p.x == at ? 1u << p.y : 0u;
        }
        if (!mine) continue;
        uint32_t w[4] = {one[0].x, one[0].y, one[0].z, one[0].w};
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u) {
            if constexpr (sizeof(T) == 4) {
                if (out >> u & 1) w[u] = 0xFF800000u;
            } else {
                if (out >> (2 * u) & 1) w[u] = (w[u] & 0xFFFF0000u) | 0xFF80u;
                if (out >> (2 * u + 1) & 1) w[u] = (w[u] & 0xFFFFu) | 0xFF800000u;
            }
        }
        one[0] = make_uint4(w[0], w[1], w[2], w[3]);
        add_vectors<T>(s, one, c);
    }
    return s;
}

template <typename T, bool kRest, int kThreads>
__global__ void __launch_bounds__(kThreads + 32, kThreads == 256 ? 4 : kRest ? 6 : 7) distill_kernel(const DistillParams P) {
    constexpr int E = kPer<T>, kWarps = kThreads / 32;
    constexpr uint32_t kSteps = 64 / kVecs;                // of a mask
    constexpr uint32_t kParts = kRest ? kWarps + 1 : kWarps;
    __shared__ Part s_part[kParts], s_all[kMaxCluster];
    __shared__ Terms s_terms;
    __shared__ unsigned long long s_mask[kRest ? kThreads : 1];
    __shared__ uint2 s_places[kRest ? K3HUF_MAX_TOP : 1];
    const cg::cluster_group cluster = cg::this_cluster();
    const uint32_t C = cluster.num_blocks(), rank = cluster.block_rank(), row = blockIdx.x / C;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const T *x = static_cast<const T *>(P.x) + uint64_t(row) * P.stride;
    const float c = P.c;
    const uint32_t shift = uint32_t(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
    const uint32_t vecs = (P.vocab + shift + E - 1) / E, K = P.teacher.count;
    const uint32_t steps = (vecs + kThreads * kVecs - 1) / (kThreads * kVecs);
    const uint32_t step0 = uint32_t(uint64_t(steps) * rank / C), step1 = uint32_t(uint64_t(steps) * (rank + 1) / C);
    if (C > 1) cluster_arrive();              // (waited for before the first remote store)
    uint4 v[kVecs], next[kVecs];
    auto load = [&](uint4 (&to)[kVecs], uint32_t step) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const uint32_t at = (step * kVecs + i) * kThreads + tid;
            to[i] = step < step1 && at < vecs ? load_vec(x, shift, P.vocab, at) : nothing<T>();
        }
    };
    if (warp < kWarps) load(next, step0);
    // which of a thread's vectors (modulo 64) may hold an alternative: a bit each, kVecs of a step.  The stream passes these
    // over
    uint64_t mask = 0;
    Sum s{-3.402823466e38f, 0.f};             // (not -infinity: then -infinity minus it is -infinity)
    if constexpr (kRest) {
        const int32_t id = uint32_t(tid) < K ? P.teacher.ids[uint64_t(row) * K + tid] : -1;
        if (tid < kThreads) s_mask[tid] = 0;
        __syncthreads();
        const bool in = id >= 0 && uint32_t(id) < P.vocab;
        const uint32_t place = (uint32_t(id) + shift) / E;
        if (uint32_t(tid) < K) s_places[tid] = in ? make_uint2(place, (uint32_t(id) + shift) % E) : make_uint2(0xFFFFFFFFu, 0);
        if (in) atomicOr(&s_mask[place % kThreads], 1ull << (place / kThreads % 64));
        __syncthreads();
        if (tid < kThreads) mask = s_mask[tid];
    }
    if (warp == kWarps) {
        if constexpr (kRest) {
            s = passed_over<T, kThreads>(x, shift, P.vocab, vecs, step0, step1, s_places, K, c);
            const Part part = warp_part(s, c);
            if (lane == 0) s_part[kWarps] = part;
        }
        if (rank == 0) {
            const Terms R = terms<T, kRest>(P, x, row, lane);
            if (lane == 0) s_terms = R;
        }
    } else {
        for (uint32_t step = step0; step < step1; ++step) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = next[i];
            load(next, step + 1);
            if constexpr (kRest) {
                const uint32_t some = uint32_t(mask >> (step % kSteps * kVecs)) & ((1u << kVecs) - 1);
                if (some) {
#pragma unroll
                    for (int i = 0; i < kVecs; ++i)
                        if (some >> i & 1) v[i] = nothing<T>();
                }
            }
            add_vectors<T>(s, v, c);
        }
        const Part part = warp_part(s, c);
        if (lane == 0) s_part[warp] = part;
    }
    __syncthreads();
    if (C == 1 && warp > 0) return;
    // one warp: the warps' sums, then the CTAs'
    float m;                                  // the largest of what was streamed (without the alternatives, where there is a rest)
    double rest;                              // its sum, beside that
    auto add = [&](const Part *parts, uint32_t count) {
        const Part p = uint32_t(lane) < count ? parts[lane] : Part{-3.402823466e38f, {0.f, 0.f}};
        m = p.m;
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        rest = warp_sum(p.sum.hi == 0.f ? 0. : wide(two_mul(p.sum, {weight32(below(p.m, m, P.scale2)), 0.f})));
    };
    add(s_part, kParts);
    if (C > 1) {
        cluster_wait();
        if (tid == 0) cluster.map_shared_rank(s_all, 0)[rank] = Part{m, narrow(rest)};
        cluster_arrive();
        cluster_wait();
        if (rank > 0 || warp > 0) return;
        add(s_all, C);
    }
    const Terms R = s_terms;
    // With the alternatives' sum (a lane for each of the two), beside the larger maximum.  The rest keeps its own: p_r may lie
    // as far below the alternatives as the logits do, and its logarithm is wanted, not what it adds to them.
    float big = m;
    double total = rest;
    if constexpr (kRest) {
        big = fmaxf(m, R.top);
        const double one = lane == 0 ? rest : wide(R.top_sum), v = one == 0. ? 0. : one * wide(weight(below(lane == 0 ? m : R.top, big, P.scale2)));
        total = __shfl_sync(0xffffffffu, v, 0) + __shfl_sync(0xffffffffu, v, 1);
    }
    // (a lane each; of what is 0, or not there, no logarithm is used)
    const double of = lane == 0 ? total : lane == 1 && kRest ? rest : lane == 2 ? R.rest : lane == 3 ? R.whole : 1., logs = log_of(of == 0. ? 1. : of);
    const double log_total = __shfl_sync(0xffffffffu, logs, 0), log_q = __shfl_sync(0xffffffffu, logs, 2), log_whole = __shfl_sync(0xffffffffu, logs, 3);
    const double log_sum = __shfl_sync(0xffffffffu, logs, 1);
    if (lane) return;
    const double lse = total == 0. ? -INFINITY : double(big) * P.scale + log_total;
    // (a row of -infinity alone: every log p is -infinity)
    double loss = total != 0. ? R.sum + R.mass * ((double(big) - double(R.from)) * P.scale + log_total - log_whole) : R.mass == 0. ? 0. : R.mass * INFINITY;
    if constexpr (kRest) {
        const double log_rest = (rest == 0. ? -INFINITY : (double(m) - double(big)) * P.scale + log_sum) - log_total;
        if (P.log_rest) P.log_rest[row] = float(log_rest);
        if (R.rest > 0.) loss += R.rest * (log_q - log_rest);
    }
    P.loss[row] = R.any ? float(loss) : 0.f;
    if (P.lse) P.lse[row] = float(lse);
}

struct GradParams {
    const void *x;
    void *dx;
    Teacher teacher;
    const float *lse, *log_rest, *g;
    uint32_t *status;
    uint64_t stride, dx_stride, n;
    uint32_t vocab, steps, parts;             // steps of a row, in so many pieces
    float scale;
};

constexpr int kGradVecs = 4, kGradPerSm = 3;

// One piece of work: some steps of a row.
struct Piece {
    uint64_t row;
    uint32_t step, steps;                     // the first, and the one behind the last
};

// kVec: logits and gradients sit alike in their 16-byte blocks
template <typename T, bool kVec>
__global__ void __launch_bounds__(kAll, kGradPerSm) distill_grad_kernel(const GradParams P) {
    constexpr int E = kVec ? kPer<T> : 1;
    constexpr uint32_t kStep = kThreads * kGradVecs;          // vectors of a step
    // of every other token: what exp(z - the first) is multiplied by; whether there is a teacher.  (This piece's and the next one's)
    __shared__ float s_of[2][3];
    const uint32_t tid = threadIdx.x, lane = tid % 32;
    auto row_of = [&](uint64_t row) { return static_cast<const T *>(P.x) + row * P.stride; };
    auto out_of = [&](uint64_t row) { return static_cast<T *>(P.dx) + row * P.dx_stride; };
    auto shift_of = [&](const T *x) { return kVec ? uint32_t(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T)) : 0u; };
    const uint64_t pieces = P.n * P.parts;
    auto piece_of = [&](uint64_t i) {
        const uint32_t part = uint32_t(i % P.parts);
        return Piece{i / P.parts, uint32_t(uint64_t(P.steps) * part / P.parts), uint32_t(uint64_t(P.steps) * (part + 1) / P.parts)};
    };
    if (tid >= kThreads) {
        // this warp: a piece's factors, and the gradients of the alternatives in it, a piece ahead of the others;
        // those of the alternatives are written when the others are done with the piece
        float d_top[2], d_next[2];
        int32_t at_top[2] = {-1, -1}, at_next[2];
        uint64_t row = 0;
        auto prepare = [&](uint64_t i) {
            at_next[0] = at_next[1] = -1;
            if (i >= pieces) return;
            const Piece p = piece_of(i);
            const T *x = row_of(p.row);
            const Alternatives A = alternatives(P.teacher, p.row, P.vocab, lane, p.step == 0 ? P.status : nullptr);
            const bool rest = P.teacher.mode == K3HUF_DISTILL_REST;
            const double lse = P.lse[p.row], log_rest = rest ? double(P.log_rest[p.row]) : 0., sg = A.any ? double(P.scale) * P.g[p.row] : 0., Q = A.mass + A.rest;
            if (lane == 0) {
                // (no other token: every p of the rest is 0)
                const bool some = lse != -INFINITY && log_rest != -INFINITY;
                float *of = s_of[i / gridDim.x & 1];
                of[0] = some ? float(lse + log_rest) : 0.f;
                of[1] = !some ? 0.f : float(rest ? sg * (Q * exp(log_rest) - A.rest) : sg * Q);
                of[2] = A.any ? 1.f : 0.f;
            }
            const int64_t shift = shift_of(x), j0 = int64_t(p.step) * kStep * E - shift, j1 = int64_t(p.steps) * kStep * E - shift;
            double q[2] = {A.q[0], A.q[1]};
            bool mine[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) mine[e] = A.id[e] >= 0 && A.id[e] >= j0 && A.id[e] < j1;
            // a token that is listed more than once: its first place takes all of its q, in their order
            for (uint64_t left = alike(A.id[0], A.id[1], P.teacher.count > 32, lane); left; left &= left - 1) {
                const uint32_t k = __ffsll(left) - 1;
                const int32_t id = __shfl_sync(0xffffffffu, k < 32 ? A.id[0] : A.id[1], k % 32);
                const double other = __shfl_sync(0xffffffffu, k < 32 ? A.q[0] : A.q[1], k % 32);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (id != A.id[e] || k == lane + 32 * e) continue;
                    if (k < lane + 32 * e) mine[e] = false;
                    else q[e] += other;
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (mine[e]) {
                    const float f = ld_f32(x + A.id[e]);
                    const float lp = float(double(f) * P.scale - lse), prob = f == -INFINITY ? 0.f : lp > 0.f ? 1.f : expf(lp);
                    at_next[e] = A.id[e];
                    d_next[e] = float(sg * (Q * prob - q[e]));
                }
        };
        auto write = [&]() {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (at_top[e] >= 0) st_f32(out_of(row) + at_top[e], d_top[e]);
        };
        prepare(blockIdx.x);
        for (uint64_t i = blockIdx.x; i < pieces; i += gridDim.x) {
            __syncthreads();
            write();                          // (of the piece before)
#pragma unroll
            for (int e = 0; e < 2; ++e) at_top[e] = at_next[e], d_top[e] = d_next[e];
            row = i / P.parts;
            prepare(i + gridDim.x);
        }
        __syncthreads();
        write();
        return;
    }
    uint4 v[kGradVecs], next[kGradVecs];
    auto load = [&](uint4 (&to)[kGradVecs], uint64_t row, uint32_t step) {
        const T *x = row_of(row);
        const uint32_t shift = shift_of(x), vecs = (P.vocab + shift + E - 1) / E;
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            const uint32_t at = step * kStep + i * kThreads + tid;
            if (at >= vecs) continue;
            if constexpr (kVec) to[i] = load_vec(x, shift, P.vocab, at);
            else to[i].x = __float_as_uint(ld_f32(x + at));
        }
    };
    if (blockIdx.x < pieces) {
        const Piece p = piece_of(blockIdx.x);
        load(next, p.row, p.step);
    }
    for (uint64_t i = blockIdx.x; i < pieces; i += gridDim.x) {
        const Piece p = piece_of(i);
        const T *x = row_of(p.row);
        T *dx = out_of(p.row);
        const uint32_t shift = shift_of(x), vecs = (P.vocab + shift + E - 1) / E;
        __syncthreads();
        const float *of = s_of[i / gridDim.x & 1];
        const float base = -of[0], coef = of[1];
        const bool any = of[2] != 0.f;
        // exp(z - the sum's logarithm) is 1 at most, as a probability is (see the log probabilities' gradient)
        auto grad = [&](float2 f) {
            float2 lp = __ffma2_rn(f, make_float2(P.scale, P.scale), make_float2(base, base));
            lp.x = min_nan(max_nan(lp.x, kFloor), 0.f);
            lp.y = min_nan(max_nan(lp.y, kFloor), 0.f);
            const float2 a = __fmul2_rn(lp, make_float2(kLog2e, kLog2e));
            return any ? __fmul2_rn(make_float2(exp2_fast(a.x), exp2_fast(a.y)), make_float2(coef, coef)) : make_float2(0.f, 0.f);
        };
        for (uint32_t step = p.step; step < p.steps; ++step) {
#pragma unroll
            for (int k = 0; k < kGradVecs; ++k) v[k] = next[k];
            if (step + 1 < p.steps) {
                load(next, p.row, step + 1);
            } else if (i + gridDim.x < pieces) {
                const Piece q = piece_of(i + gridDim.x);
                load(next, q.row, q.step);
            }
#pragma unroll
            for (int m = 0; m < kGradVecs; ++m) {
                const uint32_t at = step * kStep + m * kThreads + tid;
                if (at >= vecs) break;
                if constexpr (kVec) {
                    const int64_t j = int64_t(at) * E - shift;
                    float f[E];
                    unpack<T>(v[m], f);
#pragma unroll
                    for (int k = 0; k < E; k += 2) {
                        const float2 d = grad(make_float2(f[k], f[k + 1]));
                        f[k] = d.x;
                        f[k + 1] = d.y;
                    }
                    if (j >= 0 && j + E <= int64_t(P.vocab)) {
                        uint4 o;
                        if constexpr (sizeof(T) == 4) {
                            o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
                        } else {
                            __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
                            for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
                        }
                        __stcs(reinterpret_cast<uint4 *>(dx + j), o);
                    } else {
#pragma unroll
                        for (int k = 0; k < E; ++k)
                            if (j + k >= 0 && j + k < int64_t(P.vocab)) st_f32(dx + j + k, f[k]);
                    }
                } else {
                    st_f32(dx + at, grad(make_float2(__uint_as_float(v[m].x), 0.f)).x);
                }
            }
        }
    }
    __syncthreads();
}

template <typename T, bool kRest, int kThreads>
int launch_forward(const DistillParams &P, uint32_t n, cudaStream_t stream) {
    constexpr uint32_t kStep = kThreads * kVecs * kPer<T>;
    static std::atomic<uint64_t> wide{0};
    uint64_t sms = 0;
    int rc = once_per_device(wide, [] { return cudaFuncSetAttribute(distill_kernel<T, kRest, kThreads>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
    if (!rc) rc = sm_count(&sms);
    if (rc) return rc;
    // one CTA per row, or a cluster per row while the GPU has room for more CTAs and every CTA still has a step to do
    uint32_t C = 1;
    while (C < uint32_t(kMaxCluster) && uint64_t(n) * C * 2 <= sms * (kThreads == 256 ? 4 : kRest ? 6 : 7) && P.vocab / kStep >= 2 * C) C *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n * C);
    cfg.blockDim = dim3(kThreads + 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_rc(cudaLaunchKernelEx(&cfg, distill_kernel<T, kRest, kThreads>, P));
}

// Short rows take CTAs of 128 threads, more of them at once.
constexpr uint32_t kSmallVocab = 65536;
template <typename T, bool kRest>
int launch_forward(const DistillParams &P, uint32_t n, cudaStream_t stream) {
    return P.vocab <= kSmallVocab ? launch_forward<T, kRest, 128>(P, n, stream) : launch_forward<T, kRest, 256>(P, n, stream);
}

template <typename T>
int launch_backward(GradParams P, cudaStream_t stream) {
    const bool vec = (reinterpret_cast<uintptr_t>(P.x) - reinterpret_cast<uintptr_t>(P.dx)) % 16 == 0 && (P.stride - P.dx_stride) * sizeof(T) % 16 == 0;
    uint64_t sms = 0;
    const int rc = sm_count(&sms);
    if (rc) return rc;
    const uint64_t per = uint64_t(kThreads) * kGradVecs * (vec ? kPer<T> : 1);
    // (a row that starts inside a 16-byte block may need one vector more)
    P.steps = uint32_t((uint64_t(P.vocab) + (vec ? kPer<T> - 1 : 0) + per - 1) / per);
    // whole rows, or pieces of three steps or more (one, while the GPU's CTAs would not all have a piece) where the CTAs'
    // last round of them is fuller: every piece costs its row's factors again (4095 rows of 131072 bf16 whole 332 us, in
    // halves 341, in quarters 349; 515 of 50021 fp32 47, 43, 42)
    const uint64_t slots = sms * kGradPerSm;
    auto rounds = [&](uint32_t parts) { return double((P.n * parts + slots - 1) / slots) / parts; };      // (in rows)
    P.parts = 1;
    for (uint32_t parts = 2; parts <= P.steps && (3 * parts <= P.steps || P.n * (parts - 1) < slots) && P.n * parts < 64 * slots; ++parts)
        if (rounds(parts) < 0.98 * rounds(P.parts)) P.parts = parts;
    const uint32_t grid = uint32_t(std::min<uint64_t>(P.n * P.parts, sms * kGradPerSm));
    if (vec) distill_grad_kernel<T, true><<<grid, kAll, 0, stream>>>(P);
    else distill_grad_kernel<T, false><<<grid, kAll, 0, stream>>>(P);
    return cuda_rc(cudaGetLastError());
}

bool common_ok(const void *d_logits, uint32_t type, uint64_t stride, uint64_t n, uint32_t vocab, float scale, const int32_t *d_top_ids, const float *d_top, uint32_t top,
               uint32_t mode, const uint32_t *d_status) {
    return elem_ok(type) && vocab && vocab <= 0x7FFFFFFFu && stride >= vocab && d_status && scale > 0.f && std::isfinite(scale) && top && top <= K3HUF_MAX_TOP &&
           n <= 0x7FFFFFFFull / kMaxCluster && mode <= K3HUF_DISTILL_REST && aligned_to(d_logits, elem_bytes(type)) && aligned_to(d_top_ids, 4) && aligned_to(d_top, 4) &&
           aligned_to(d_status, 4);
}

}  // namespace
}  // namespace k3huf

using namespace k3huf;

extern "C" int k3huf_distill(const void *d_logits, uint32_t type, uint64_t stride, uint64_t n, uint32_t vocab, float scale, const int32_t *d_top_ids,
                             const float *d_top_logprobs, uint32_t top, uint32_t mode, float *d_loss, float *d_lse, float *d_log_rest, uint32_t *d_status, void *stream) {
    if (!common_ok(d_logits, type, stride, n, vocab, scale, d_top_ids, d_top_logprobs, top, mode, d_status) || !aligned_to(d_loss, 4) || !aligned_to(d_lse, 4) ||
        !aligned_to(d_log_rest, 4) || (d_log_rest && mode != K3HUF_DISTILL_REST))
        return K3HUF_E_ARG;
    if (n == 0) return K3HUF_OK;
    if (!d_logits || !d_top_ids || !d_top_logprobs || !d_loss) return K3HUF_E_ARG;
    const float c = float(fmin(double(scale) * 1.4426950408889634074, 3.402823466e38));
    const double scale_of = double(c) * 0.69314718055994530942;
    const DistillParams P{d_logits, {d_top_ids, d_top_logprobs, top, mode}, d_loss, d_lse, d_log_rest, d_status, stride, vocab, c, scale_of, {float(scale_of), float(scale_of - double(float(scale_of)))}};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool rest = mode == K3HUF_DISTILL_REST;
    if (type == K3HUF_BF16) return rest ? launch_forward<__nv_bfloat16, true>(P, uint32_t(n), st) : launch_forward<__nv_bfloat16, false>(P, uint32_t(n), st);
    return rest ? launch_forward<float, true>(P, uint32_t(n), st) : launch_forward<float, false>(P, uint32_t(n), st);
}

extern "C" int k3huf_distill_grad(const void *d_logits, uint32_t type, uint64_t stride, uint64_t n, uint32_t vocab, float scale, const int32_t *d_top_ids,
                                  const float *d_top_logprobs, uint32_t top, uint32_t mode, const float *d_lse, const float *d_log_rest, const float *d_g_loss, void *d_dlogits,
                                  uint64_t out_stride, uint32_t *d_status, void *stream) {
    if (!common_ok(d_logits, type, stride, n, vocab, scale, d_top_ids, d_top_logprobs, top, mode, d_status) || out_stride < vocab || !aligned_to(d_dlogits, elem_bytes(type)) ||
        !aligned_to(d_lse, 4) || !aligned_to(d_log_rest, 4) || !aligned_to(d_g_loss, 4) || (d_log_rest != nullptr) != (mode == K3HUF_DISTILL_REST))
        return K3HUF_E_ARG;
    if (n == 0) return K3HUF_OK;
    if (!d_logits || !d_dlogits || !d_top_ids || !d_top_logprobs || !d_lse || !d_g_loss || (d_logits == d_dlogits && stride != out_stride)) return K3HUF_E_ARG;
    const GradParams P{d_logits, d_dlogits, {d_top_ids, d_top_logprobs, top, mode}, d_lse, d_log_rest, d_g_loss, d_status, stride, out_stride, n, vocab, 0, 0, scale};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return type == K3HUF_BF16 ? launch_backward<__nv_bfloat16>(P, st) : launch_backward<float>(P, st);
}
