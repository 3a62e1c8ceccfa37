// The matrix product with bias, activation and residual in its epilogue, and its gradients:
//   z = x W^T + bias          y = act(z) + residual
//   dz = dy act'(z)           dbias = sum over tokens of dz
//   dx = dz W                 dW = dz^T x
// The three products are one kernel on tcgen05.mma,
//   out[j][i] = sum_k A[i][k] B[j][k]         (i runs along a row of the result),
// with A = W, B = x for y; A = W^T, B = dz for dx; A = x^T, B = dz^T for dW.  An operand that lies
// contraction-last is read K-major, one that lies contraction-first (W for dx; x and dz for dW) MN-major from
// the same 128-byte swizzled tiles, so nothing is transposed in memory.  i is the tile's 128 lanes of TMEM: a
// warp's store of one j is 32 neighbouring elements of the result, and the results need no shared memory (a residual
// comes through it, see Ahead).
//
// Bound by the tensor cores where there are many tokens (4096 x 8192 x 8192 bf16 285 to 296 us, 1.9 PFLOP/s, the tensor
// pipe busy in 97% of the cycles; 8192 x 24576 x 8192 1.70 to 1.97 ms, as the power limit allows), by the read of the
// weight where there are few (3 x 8192 x 8192 26 to 29 us, 4.6 to 5.2 TB/s with the launch), by the epilogue where the
// contraction is short (8192 x 8192 x 576 62 to 70 us).
#include <algorithm>
#include <cmath>

#include "k3huf_tc.h"

namespace k3huf {
namespace {

constexpr uint32_t kTileI = 128;              // lanes of TMEM: elements of a result row per tile
constexpr uint32_t kStep = 64;                // contraction per staged step: one 128-byte row
constexpr uint32_t kEpilogue = 256;           // threads that read TMEM: the first eight warps
constexpr uint32_t kThreads = kEpilogue + 64; // ... one warp for the copies, one for the products
constexpr uint32_t kMaxSplits = 8;
// Additions in the tensor core before a sum that ends as fp32 moves to registers: one of them errs by about 1.3e-8
// of the sum, always to the same side.
constexpr uint32_t kChain = 32;
// Steps of a sum that ends as bf16: 65536 values, 5e-5 of the sum, and a wait for them that stays far from its limit.
constexpr uint32_t kLongRun = 1024;

// Place in a ring of stages: the stage, and the parity of the phase that its barrier is in this time round.
template <uint32_t kStages> struct Ring {
    uint32_t stage = 0, parity = 0, used = 0;
    __device__ __forceinline__ void next() {
        used = min(used + 1, kStages);
        if (++stage == kStages) stage = 0, parity ^= 1;
    }
    // Back by one stage, of those that were used last; false when all have been gone through.
    __device__ __forceinline__ bool back() {
        if (used == 0) return false;
        --used;
        if (stage == 0) stage = kStages, parity ^= 1;
        --stage;
        return true;
    }
};
// The same thread of a converged warp, each time.
__device__ __forceinline__ bool one_thread() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

template <uint32_t kTileJ> struct Shape {
    static constexpr uint32_t a_bytes = kTileI * 128, b_bytes = kTileJ * 128, stage = a_bytes + b_bytes;
    static constexpr uint32_t per_sm = kTileJ <= 64 ? 2 : 1;                 // CTAs
    static constexpr uint32_t stages = kTileJ == 128 ? 6 : kTileJ == 64 ? 4 : kTileJ == 32 ? 5 : 6;
    static constexpr uint32_t part = kTileJ >= 32 ? kTileJ / 2 : kTileJ;     // columns of TMEM per epilogue thread
    static constexpr size_t smem = stages * stage + 1024;
    static_assert(smem * per_sm <= 220 * 1024, "shared memory of an SM");
    static_assert(stages * stage >= kTileI * kTileJ * 4, "a split's partial sums");
};

struct Epilogue {
    const void *bias, *residual;
    void *out, *z;
    uint64_t out_stride, residual_stride, z_stride;
    uint32_t out_type, bias_type, z_type, act;
};

struct ProductParams {
    CUtensorMap a, b;
    Epilogue e;
    uint32_t *status;
    uint32_t tiles, size_i, size_j, steps, tiles_i, tiles_j, splits, run;     // run: steps added up in TMEM
};

__device__ __forceinline__ float bias_at(const Epilogue &e, uint32_t i) {
    return !e.bias ? 0.f : e.bias_type == K3HUF_F32 ? static_cast<const float *>(e.bias)[i] : ld_f32(static_cast<const __nv_bfloat16 *>(e.bias) + i);
}

__device__ __forceinline__ bool aligned_to_device(const void *p, uint32_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// kCount neighbouring columns j of the thread's i, stored.
template <int kCount, typename T>
__device__ __forceinline__ void store_as(T *o, uint64_t stride, uint32_t left, const float (&v)[kCount]) {       // left: columns to the matrix's end
    if (left >= kCount) {
#pragma unroll
        for (int c = 0; c < kCount; ++c, o += stride) st_f32(o, v[c]);
    } else {
#pragma unroll
        for (int c = 0; c < kCount; ++c, o += stride)
            if (c < left) st_f32(o, v[c]);
    }
}
template <int kCount>
__device__ __forceinline__ void store_to(void *matrix, uint32_t type, uint64_t stride, uint32_t i, uint32_t j, uint32_t size_j, const float (&v)[kCount]) {
    const uint64_t at = uint64_t(j) * stride + i;
    const uint32_t left = j < size_j ? size_j - j : 0u;
    if (type == K3HUF_F32) store_as(static_cast<float *>(matrix) + at, stride, left, v);
    else store_as(static_cast<__nv_bfloat16 *>(matrix) + at, stride, left, v);
}
template <int kCount>
__device__ __forceinline__ void store(const Epilogue &e, uint32_t i, uint32_t j, uint32_t size_j, const float (&v)[kCount]) {
    store_to(e.out, e.out_type, e.out_stride, i, j, size_j, v);
}

// The residual's values there.
template <int kCount>
__device__ __forceinline__ void residual_at(const Epilogue &e, uint32_t i, uint32_t j, uint32_t size_j, float (&res)[kCount]) {
    const uint64_t at = uint64_t(j) * e.residual_stride + i;
    if (e.out_type == K3HUF_F32) {
        const float *r = static_cast<const float *>(e.residual) + at;
#pragma unroll
        for (int c = 0; c < kCount; ++c, r += e.residual_stride) res[c] = j + c < size_j ? *r : 0.f;
    } else {
        const __nv_bfloat16 *r = static_cast<const __nv_bfloat16 *>(e.residual) + at;
#pragma unroll
        for (int c = 0; c < kCount; ++c, r += e.residual_stride) res[c] = j + c < size_j ? ld_f32(r) : 0.f;
    }
}

// Sums to values of the result.  (With the hardware's exponential and quotient, for fp32 results too: they err by some units
// of the last place more than expf and a division, with which the slopes of 4095 x 24576 took 299 us instead of 100.  A
// quotient by more than 2^126 is 0.)
template <int kCount>
__device__ __forceinline__ void apply(const Epilogue &e, uint32_t i, uint32_t j, uint32_t size_j, float (&v)[kCount], float bias, const float (&res)[kCount]) {
    if (e.bias) {
#pragma unroll
        for (int c = 0; c < kCount; ++c) v[c] += bias;
    }
    if (e.z) store_to(e.z, e.z_type, e.z_stride, i, j, size_j, v);
    if (e.act == K3HUF_ACT_RELU) {
#pragma unroll
        for (int c = 0; c < kCount; ++c) v[c] = v[c] < 0.f ? 0.f : v[c];
    } else if (e.act == K3HUF_ACT_SILU) {
#pragma unroll
        for (int c = 0; c < kCount; ++c) v[c] = __fdividef(v[c], 1.f + __expf(-v[c]));
    } else if (e.act == K3HUF_ACT_GELU) {
        // (1 + tanh u) / 2 is the logistic function of 2 u
#pragma unroll
        for (int c = 0; c < kCount; ++c) v[c] = __fdividef(v[c], 1.f + __expf(-1.5957691216057308f * fmaf(0.044715f * v[c] * v[c], v[c], v[c])));
    }
    if (e.residual) {
#pragma unroll
        for (int c = 0; c < kCount; ++c) v[c] += res[c];
    }
}

// Four neighbouring i of one column: sums to results.
__device__ __forceinline__ void finish_four(const Epilogue &e, uint32_t i, uint32_t size_i, uint32_t j, const float (&v)[4], const float (&bias)[4]) {
    Epilogue at = e;                          // (as a row of columns: i and j change places)
    at.out_stride = at.residual_stride = at.z_stride = 1;
    const uint32_t w = e.out_type == K3HUF_F32 ? 4 : 2;
    at.out = static_cast<uint8_t *>(e.out) + (uint64_t(j) * e.out_stride + i) * w;
    if (e.residual) at.residual = static_cast<const uint8_t *>(e.residual) + (uint64_t(j) * e.residual_stride + i) * w;
    if (e.z) at.z = static_cast<uint8_t *>(e.z) + (uint64_t(j) * e.z_stride + i) * (e.z_type == K3HUF_F32 ? 4 : 2);
    at.bias = nullptr;
    float u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = e.bias ? v[k] + bias[k] : v[k];
    const uint32_t count = i < size_i ? min(size_i - i, 4u) : 0u;
    if (count == 0) return;
    float res[4];
    if (e.residual) residual_at(at, 0, 0, count, res);
    apply(at, 0, 0, count, u, 0.f, res);
    if (count == 4 && e.out_type == K3HUF_F32 && aligned_to_device(at.out, 16)) *static_cast<float4 *>(at.out) = make_float4(u[0], u[1], u[2], u[3]);
    else if (count == 4 && e.out_type == K3HUF_BF16 && aligned_to_device(at.out, 8)) {
        uint2 o;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&o);
        h[0] = __floats2bfloat162_rn(u[0], u[1]);
        h[1] = __floats2bfloat162_rn(u[2], u[3]);
        *static_cast<uint2 *>(at.out) = o;
    } else {
        store(at, 0, 0, count, u);
    }
}

// A tile's sums of several runs are added up in registers, and go back to TMEM, to where the last run's were.
template <uint32_t kPart>
__device__ __forceinline__ void add_run(uint32_t from, float (&sum)[kPart], bool first, bool last) {
#pragma unroll
    for (uint32_t c = 0; c < kPart; c += 16) {
        float v[16];
        tmem_load16(from + c, v);
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[c + k] = first ? v[k] : sum[c + k] + v[k];
        if (last) tmem_store16(from + c, &sum[c]);
    }
    if (last) asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// ... and from there, 16 columns at a time, to the result; the next columns, and their residual, are on
// their way meanwhile (`res`: the first columns').
template <uint32_t kPart>
__device__ __forceinline__ void finish_tile(const Epilogue &e, uint32_t from, uint32_t i, uint32_t size_i, uint32_t j, uint32_t size_j, float bias, float (&res)[16]) {
    uint32_t next[16];
    tmem_start16(from, next);
#pragma unroll 1
    for (uint32_t c = 0; c < kPart; c += 16) {
        float v[16], mine[16];
        tmem_wait16(next);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(next[k]), mine[k] = res[k];
        if (c + 16 < kPart) tmem_start16(from + c + 16, next);
        if (i < size_i) {
            if (e.residual && c + 16 < kPart) residual_at(e, i, j + c + 16, size_j, res);
            apply(e, i, j + c, size_j, v, bias, mine);
            store(e, i, j + c, size_j, v);
        }
        __syncwarp();
    }
}

// The same for a warp whose 32 elements of every column lie in the matrix, with a residual whose rows start on 16 bytes: it
// comes through a buffer in shared memory, kSlots x 16 columns ahead.  (16 columns of loads at a time, in registers, are
// 8 KB in flight per SM: 3012 x 8192 x 192 with a residual 108 us, and 40 us so.)
constexpr uint32_t kAheadBytes = 4096;                    // of a warp
template <typename T> struct Ahead {
    static constexpr uint32_t slot = 16 * 32 * sizeof(T), slots = kAheadBytes / slot, parts = 32 * sizeof(T) / 16;      // parts: of a column, 16 bytes each
    // columns j to j + 15, elements i0 to i0 + 31, on their way to the slot
    __device__ static __forceinline__ void start(const Epilogue &e, uint32_t to, uint32_t i0, uint32_t j, uint32_t size_j, uint32_t lane) {
        const T *r = static_cast<const T *>(e.residual);
#pragma unroll
        for (uint32_t q = 0; q < slot / 512; ++q) {
            const uint32_t p = lane + 32 * q, col = p / parts, off = p % parts * (16 / sizeof(T));
            const bool in = j + col < size_j;
            cp_async16z(to + p * 16, in ? r + uint64_t(j + col) * e.residual_stride + i0 + off : r, in ? 16 : 0);
        }
    }
    // ... the first of a tile's
    template <uint32_t kPart> __device__ static __forceinline__ void start_tile(const Epilogue &e, uint32_t buffer, uint32_t i0, uint32_t j, uint32_t size_j, uint32_t lane) {
#pragma unroll
        for (uint32_t q = 0; q < slots; ++q) {
            if (q * 16 < kPart) start(e, buffer + q * slot, i0, j + q * 16, size_j, lane);
            cp_async_commit();
        }
    }
    template <uint32_t kPart>
    __device__ static __forceinline__ void finish(const Epilogue &e, uint8_t *buffer, uint32_t from, uint32_t i0, uint32_t lane, uint32_t j, uint32_t size_j, float bias) {
        uint32_t next[16];
        tmem_start16(from, next);
#pragma unroll 1
        for (uint32_t c = 0; c < kPart; c += 16) {
            float v[16], res[16];
            const uint32_t at = c / 16 % slots * slot;
            cp_async_wait<slots - 1>();
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 16; ++k) res[k] = ld_f32(reinterpret_cast<const T *>(buffer + at) + k * 32 + lane);
            __syncwarp();
            if (c + 16 * slots < kPart) start(e, smem_addr(buffer + at), i0, j + c + 16 * slots, size_j, lane);
            cp_async_commit();
            tmem_wait16(next);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(next[k]);
            if (c + 16 < kPart) tmem_start16(from + c + 16, next);
            apply(e, i0 + lane, j + c, size_j, v, bias, res);
            store(e, i0 + lane, j + c, size_j, v);
        }
        cp_async_wait<0>();
        __syncwarp();
    }
};

// Order of the tiles: kGroup rows of tiles at a time, so that the CTAs at work at once share operands.
constexpr uint32_t kGroup = 16;
__device__ __forceinline__ void tile_place(const ProductParams &P, uint32_t t, uint32_t &ti, uint32_t &tj) {
    const uint32_t whole = kGroup * P.tiles_j, g = t / whole, rest = t % whole, rows = min(kGroup, P.tiles_i - g * kGroup);
    ti = g * kGroup + rest % rows;
    tj = rest / rows;
}

// Sums of the splits' partial sums, in their order, to results: columns c, c + 8, ... below c1 of the tile that begins at
// column j, four neighbouring i of each; the loads of kBatch columns from kMost (or fewer) CTAs are in flight at once.
template <uint32_t kBatch, uint32_t kMost>
__device__ __forceinline__ void join(const ProductParams &P, const float *mine, uint32_t i, uint32_t j, uint32_t c, uint32_t c1) {
    constexpr uint32_t kWarps = kEpilogue / 32;
    float bias[4];
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u) bias[u] = i + u < P.size_i ? bias_at(P.e, i + u) : 0.f;
    for (; c < c1; c += kBatch * kWarps) {
        float4 part[kBatch][kMost];
#pragma unroll
        for (uint32_t k = 0; k < kBatch; ++k)
#pragma unroll
            for (uint32_t q = 0; q < kMost; ++q)
                if (q < P.splits && c + k * kWarps < c1) part[k][q] = cluster_load4(smem_addr(mine + (c + k * kWarps) * kTileI), q);
#pragma unroll
        for (uint32_t k = 0; k < kBatch; ++k) {
            const uint32_t col = c + k * kWarps;
            if (col >= c1) break;
            float v[4] = {part[k][0].x, part[k][0].y, part[k][0].z, part[k][0].w};
#pragma unroll
            for (uint32_t q = 1; q < kMost; ++q)
                if (q < P.splits) v[0] += part[k][q].x, v[1] += part[k][q].y, v[2] += part[k][q].z, v[3] += part[k][q].w;
            finish_four(P.e, i, P.size_i, j + col, v, bias);
        }
    }
}

template <uint32_t kTileJ, bool kMnA, bool kMnB>
__global__ void __launch_bounds__(kThreads, Shape<kTileJ>::per_sm) product_kernel(const __grid_constant__ ProductParams P) {
    using S = Shape<kTileJ>;
    constexpr uint32_t NS = S::stages;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_full[NS], s_free[NS], s_sum[2], s_read[2];
    __shared__ uint32_t s_tmem;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32, base = smem_addr(smem);
    const uint32_t split = blockIdx.x % P.splits;
    const uint32_t t_first = blockIdx.x / P.splits, t_step = gridDim.x / P.splits;
    const uint32_t k0 = uint32_t(uint64_t(P.steps) * split / P.splits), n_steps = uint32_t(uint64_t(P.steps) * (split + 1) / P.splits) - k0;
    const uint32_t runs = (n_steps + P.run - 1) / P.run;
    // (the warp that copies makes the barriers and starts; the others meet behind its back)
    if (warp == 0) tmem_alloc(smem_addr(&s_tmem), 2 * kTileJ);
    if (warp == kEpilogue / 32) {
        if (lane == 0) {
            for (uint32_t i = 0; i < NS; ++i) {
                mbar_init(smem_addr(&s_full[i]), 1);
                mbar_init(smem_addr(&s_free[i]), 1);
            }
            for (uint32_t i = 0; i < 2; ++i) {
                mbar_init(smem_addr(&s_sum[i]), 1);
                mbar_init(smem_addr(&s_read[i]), kEpilogue / 32);
            }
            fence_async_shared();
        }
        __syncwarp();
        asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
    } else {
        tc_fence_before();
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
        tc_fence_after();
    }
    const uint32_t tmem = warp == kEpilogue / 32 ? 0u : s_tmem;
    bool ok = true;
    float sum[S::part];
    const uint32_t quarter = warp % 4, c_first = warp / 4 * S::part;         // (epilogue warps)
    const bool reads = warp < kEpilogue / 32 && c_first < kTileJ;

    if (warp == kEpilogue / 32) {
        // (the whole warp goes through the loop, one thread issues: addresses stay in uniform registers)
        const bool issues = one_thread();
        Ring<NS> ring;
        const uint32_t full = smem_addr(&s_full[0]), free = smem_addr(&s_free[0]);
        for (uint32_t t = t_first; t < P.tiles && ok; t += t_step) {
            uint32_t ti, tj;
            tile_place(P, t, ti, tj);
            const int32_t i0 = int32_t(ti * kTileI), j0 = int32_t(tj * kTileJ);
            int32_t k = int32_t(k0 * kStep);
            for (uint32_t s = 0; s < n_steps; ++s, k += int32_t(kStep)) {
                ok = mbar_wait(free + ring.stage * 8, ring.parity ^ 1);       // (the first round's stages are free)
                if (!ok) break;
                if (issues) {
                    const uint32_t at = base + ring.stage * S::stage, bar = full + ring.stage * 8;
                    mbar_expect(bar, S::stage);
                    if constexpr (kMnA) {
                        tma_load(at, &P.a, i0, k, bar);
                        tma_load(at + kStep * 128, &P.a, i0 + 64, k, bar);
                    } else {
                        tma_load(at, &P.a, k, i0, bar);
                    }
                    if constexpr (kMnB) {
#pragma unroll
                        for (uint32_t b = 0; b < kTileJ / 64; ++b) tma_load(at + S::a_bytes + b * (kStep * 128), &P.b, j0 + int32_t(b * 64), k, bar);
                    } else {
                        tma_load(at + S::a_bytes, &P.b, k, j0, bar);
                    }
                }
                ring.next();
            }
        }
        // the last copies land before the CTA ends, whichever thread's wait may have given up
        while (ring.back()) mbar_wait(full + ring.stage * 8, ring.parity);
    } else if (warp == kEpilogue / 32 + 1) {
        const bool issues = one_thread();
        constexpr uint32_t desc = mma_desc(kTileI, kTileJ, kMnA, kMnB);
        const uint64_t a0 = tile_desc(base, kMnA ? kStep * 128 : 16, 1024), b0 = tile_desc(base + S::a_bytes, kMnB ? kStep * 128 : 16, 1024);
        const uint32_t full = smem_addr(&s_full[0]), free = smem_addr(&s_free[0]);
        Ring<NS> ring;
        Ring<2> run;
        for (uint32_t t = t_first; t < P.tiles && ok; t += t_step)
            for (uint32_t s0 = 0; s0 < n_steps && ok; s0 += P.run) {
                ok = mbar_wait(smem_addr(&s_read[run.stage]), run.parity ^ 1);
                const uint32_t d = tmem + run.stage * kTileJ, s1 = min(s0 + P.run, n_steps);
                for (uint32_t s = s0; s < s1 && ok; ++s) {
                    ok = mbar_wait(full + ring.stage * 8, ring.parity);
                    if (!ok) break;
                    tc_fence_after();
                    if (issues) {
                        const uint64_t a = a0 + ring.stage * (S::stage >> 4), b = b0 + ring.stage * (S::stage >> 4);
#pragma unroll
                        for (uint32_t q = 0; q < kStep / 16; ++q) mma(d, a + q * (kMnA ? 128 : 2), b + q * (kMnB ? 128 : 2), desc, s > s0 || q);
                        mma_commit(free + ring.stage * 8);
                    }
                    ring.next();
                }
                if (issues) mma_commit(smem_addr(&s_sum[run.stage]));
                run.next();
            }
        // (products whose end nobody waited for, if a wait gave up, end before the CTA does)
        while (ring.back()) mbar_wait(free + ring.stage * 8, ring.parity);
    } else {
        uint32_t r = 0;
        auto bias_of = [&](uint32_t t) {
            uint32_t ti, tj;
            if (t >= P.tiles || !P.e.bias) return 0.f;
            tile_place(P, t, ti, tj);
            const uint32_t i = ti * kTileI + quarter * 32 + lane;
            return i < P.size_i ? bias_at(P.e, i) : 0.f;
        };
        float next_bias = bias_of(t_first);
        for (uint32_t t = t_first; t < P.tiles; t += t_step) {
            uint32_t ti, tj;
            tile_place(P, t, ti, tj);
            const uint32_t i = ti * kTileI + quarter * 32 + lane;
            const float bias = next_bias;
            next_bias = bias_of(t + t_step);  // (on its way while this tile is finished)
            float res[16];
            if (P.e.residual && i < P.size_i && reads && P.splits == 1) residual_at(P.e, i, tj * kTileJ + c_first, P.size_j, res);
            for (uint32_t q = 0; q < runs; ++q, ++r) {
                if (ok) ok = mbar_wait(smem_addr(&s_sum[r & 1]), r / 2 & 1);
                tc_fence_after();
                const bool last = q + 1 == runs && P.splits == 1;
                const uint32_t from = tmem + (quarter << 21) + (r & 1) * kTileJ + c_first;
                if (reads && (runs > 1 || !last)) add_run<S::part>(from, sum, q == 0, last);
                if (reads && last) finish_tile<S::part>(P.e, from, i, P.size_i, tj * kTileJ + c_first, P.size_j, bias, res);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&s_read[r & 1]));
            }
        }
    }
    if (P.splits > 1) {
        // (one tile per cluster) the CTAs' partial sums lie in their stages, whose copies and products are all
        // done; every CTA adds up and finishes a share of the columns, in the order of the splits
        float *parts = reinterpret_cast<float *>(smem);
        if (reads) {
#pragma unroll
            for (uint32_t c = 0; c < S::part; ++c) parts[(c_first + c) * kTileI + quarter * 32 + lane] = sum[c];
        }
        cluster_arrive();
        cluster_wait();
        uint32_t ti, tj;
        tile_place(P, t_first, ti, tj);
        if (warp < kEpilogue / 32) {
            const uint32_t c0 = kTileJ * split / P.splits, c1 = min(kTileJ * (split + 1) / P.splits, P.size_j - tj * kTileJ);
            const float *mine = parts + lane * 4;             // four neighbouring i of a column per thread, a column per warp
            if (P.splits <= 2) join<8, 2>(P, mine, ti * kTileI + lane * 4, tj * kTileJ, c0 + warp, c1);
            else if (P.splits <= 4) join<4, 4>(P, mine, ti * kTileI + lane * 4, tj * kTileJ, c0 + warp, c1);
            else join<2, 8>(P, mine, ti * kTileI + lane * 4, tj * kTileJ, c0 + warp, c1);
        }
        __syncwarp();
        cluster_arrive_relaxed();             // (nobody reads another CTA's sums any more)
        cluster_wait();
    }
    if (!ok) atomicOr(P.status, K3HUF_ST_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free(tmem, 2 * kTileJ);
}

// The same for large results (single CTAs of 128 x 256 reached 790 TFLOP/s): the two CTAs of a pair work on one tile of 256 x kTileJ.  Each holds 128 of its rows (and
// their sums, in its own TMEM) and half of its columns' operand, which both use: per product a CTA's shared memory is
// filled with and read for half as much of B.  The first CTA's threads issue the products of both; the copies of both
// complete on its barriers, the products' ends on barriers of both.
constexpr uint32_t kPairThreads = kEpilogue + 128;       // (whole warpgroups: registers move from the last one to the others)
constexpr uint32_t kPairMoreRegs = 232, kPairFewRegs = 40;
static_assert(kPairMoreRegs * kEpilogue + kPairFewRegs * 128 <= 168 * kPairThreads, "registers that the CTA is launched with");
template <uint32_t kTileJ> struct Pair {
    static constexpr uint32_t a_bytes = kTileI * 128, b_bytes = kTileJ / 2 * 128, stage = a_bytes + b_bytes;
    static constexpr uint32_t stages = kTileJ == 256 ? 6 : 8;
    static constexpr uint32_t part = kTileJ / 2;
    static constexpr size_t smem = stages * stage + 1024, ahead = kEpilogue / 32 * kAheadBytes;
    static_assert(smem + ahead <= 226 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ uint32_t in_cta(uint32_t at, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, uint32_t cluster_bar) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y),
                 "r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(desc),
                 "r"(uint32_t(add)) : "memory");
}
// the barrier at this address of both CTAs completes when all products issued before have
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"(uint16_t(3)) : "memory");
}
// (nothing but the sums in TMEM is handed back, and their loads are complete: a release would wait for every store of the
// results, 110 us instead of 88 for 8192 x 8192 x 576 fp32)
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) { asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory"); }
// a wait for arrivals of the other CTA's threads
__device__ __forceinline__ bool mbar_wait_pair(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < kTcPolls; ++i) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
    }
    return false;
}

// (kAhead: a residual whose rows start on 16 bytes; an instantiation of its own, whose code would slow the others' epilogue,
// 8192 x 8192 x 576 from 69 to 83 us)
template <uint32_t kTileJ, bool kMnA, bool kMnB, bool kAhead>
__global__ void __cluster_dims__(2) __launch_bounds__(kPairThreads, 1) pair_kernel(const __grid_constant__ ProductParams P) {
    using S = Pair<kTileJ>;
    constexpr uint32_t NS = S::stages;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_full[NS], s_free[NS], s_sum[2], s_read[2];
    __shared__ uint32_t s_tmem;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32, base = smem_addr(smem), rank = blockIdx.x % 2;
    const uint32_t t_first = blockIdx.x / 2, t_step = gridDim.x / 2;
    const uint32_t runs = (P.steps + P.run - 1) / P.run;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)), "r"(2 * kTileJ) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    if (tid == 0) {
        for (uint32_t i = 0; i < NS; ++i) {
            mbar_init(smem_addr(&s_full[i]), 1);
            mbar_init(smem_addr(&s_free[i]), 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&s_sum[i]), 1);
            mbar_init(smem_addr(&s_read[i]), 2 * kEpilogue / 32);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_shared();
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    if (warp >= kEpilogue / 32) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairFewRegs));
        if (warp == kEpilogue / 32) {
            const bool issues = one_thread();
            Ring<NS> ring;
            const uint32_t full = smem_addr(&s_full[0]), first_full = in_cta(full, 0), free = smem_addr(&s_free[0]);
            for (uint32_t t = t_first; t < P.tiles && ok; t += t_step) {
                uint32_t ti, tj;
                tile_place(P, t, ti, tj);
                const int32_t i0 = int32_t((ti * 2 + rank) * kTileI), j0 = int32_t(tj * kTileJ + rank * (kTileJ / 2));
                int32_t k = 0;
                for (uint32_t s = 0; s < P.steps; ++s, k += int32_t(kStep)) {
                    ok = mbar_wait(free + ring.stage * 8, ring.parity ^ 1);       // (the first round's stages are free)
                    if (!ok) break;
                    if (issues) {
                        const uint32_t at = base + ring.stage * S::stage, bar = first_full + ring.stage * 8;
                        if (rank == 0) mbar_expect(full + ring.stage * 8, 2 * S::stage);
                        if constexpr (kMnA) {
                            pair_load(at, &P.a, i0, k, bar);
                            pair_load(at + kStep * 128, &P.a, i0 + 64, k, bar);
                        } else {
                            pair_load(at, &P.a, k, i0, bar);
                        }
                        if constexpr (kMnB) {
#pragma unroll
                            for (uint32_t b = 0; b < kTileJ / 128; ++b) pair_load(at + S::a_bytes + b * (kStep * 128), &P.b, j0 + int32_t(b * 64), k, bar);
                        } else {
                            pair_load(at + S::a_bytes, &P.b, k, j0, bar);
                        }
                    }
                    ring.next();
                }
            }
            // the last copies of both CTAs land before either ends (the barrier below), whichever thread's wait may have
            // given up; if one has, the second CTA, whose own barriers nothing completes, waits until its limit
            if (rank == 0) {
                while (ring.back()) mbar_wait_pair(full + ring.stage * 8, ring.parity);
            } else if (!ok) {
                mbar_wait(full, 0);
            }
        } else if (warp == kEpilogue / 32 + 1 && rank == 0) {
            const bool issues = one_thread();
            constexpr uint32_t desc = mma_desc(2 * kTileI, kTileJ, kMnA, kMnB);
            const uint64_t a0 = tile_desc(base, kMnA ? kStep * 128 : 16, 1024), b0 = tile_desc(base + S::a_bytes, kMnB ? kStep * 128 : 16, 1024);
            const uint32_t full = smem_addr(&s_full[0]), free = smem_addr(&s_free[0]);
            Ring<NS> ring;
            Ring<2> run;
            for (uint32_t t = t_first; t < P.tiles && ok; t += t_step)
                for (uint32_t s0 = 0; s0 < P.steps && ok; s0 += P.run) {
                    ok = mbar_wait_pair(smem_addr(&s_read[run.stage]), run.parity ^ 1);
                    const uint32_t d = tmem + run.stage * kTileJ, s1 = min(s0 + P.run, P.steps);
                    for (uint32_t s = s0; s < s1 && ok; ++s) {
                        ok = mbar_wait(full + ring.stage * 8, ring.parity);
                        if (!ok) break;
                        tc_fence_after();
                        if (issues) {
                            const uint64_t a = a0 + ring.stage * (S::stage >> 4), b = b0 + ring.stage * (S::stage >> 4);
#pragma unroll
                            for (uint32_t q = 0; q < kStep / 16; ++q) pair_mma(d, a + q * (kMnA ? 128 : 2), b + q * (kMnB ? 128 : 2), desc, s > s0 || q);
                            pair_commit(free + ring.stage * 8);
                        }
                        ring.next();
                    }
                    if (issues) pair_commit(smem_addr(&s_sum[run.stage]));
                    run.next();
                }
            // (products whose end nobody waited for, if a wait gave up, end before the CTAs do)
            while (ring.back()) mbar_wait(free + ring.stage * 8, ring.parity);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairMoreRegs));
        const uint32_t quarter = warp % 4, c_first = warp / 4 * S::part;
        uint32_t r = 0;
        auto bias_of = [&](uint32_t t) {
            uint32_t ti, tj;
            if (t >= P.tiles || !P.e.bias) return 0.f;
            tile_place(P, t, ti, tj);
            const uint32_t i = (ti * 2 + rank) * kTileI + quarter * 32 + lane;
            return i < P.size_i ? bias_at(P.e, i) : 0.f;
        };
        float next_bias = bias_of(t_first);
        for (uint32_t t = t_first; t < P.tiles; t += t_step) {
            uint32_t ti, tj;
            tile_place(P, t, ti, tj);
            const uint32_t i = (ti * 2 + rank) * kTileI + quarter * 32 + lane;
            const float bias = next_bias;
            next_bias = bias_of(t + t_step);  // (on its way while this tile is finished)
            float res[16];
            const bool f32 = P.e.out_type == K3HUF_F32, ahead = kAhead && i - lane + 32 <= P.size_i;
            uint8_t *buffer = smem + NS * S::stage + warp * kAheadBytes;
            if (!ahead && P.e.residual && i < P.size_i) residual_at(P.e, i, tj * kTileJ + c_first, P.size_j, res);
            if constexpr (kAhead) {
                if (ahead && f32) Ahead<float>::template start_tile<S::part>(P.e, smem_addr(buffer), i - lane, tj * kTileJ + c_first, P.size_j, lane);
                if (ahead && !f32) Ahead<__nv_bfloat16>::template start_tile<S::part>(P.e, smem_addr(buffer), i - lane, tj * kTileJ + c_first, P.size_j, lane);
            }
            float sum[S::part];
            for (uint32_t q = 0; q < runs; ++q, ++r) {
                if (ok) ok = mbar_wait(smem_addr(&s_sum[r & 1]), r / 2 & 1);
                tc_fence_after();
                const uint32_t from = tmem + (quarter << 21) + (r & 1) * kTileJ + c_first;
                if (runs > 1) add_run<S::part>(from, sum, q == 0, q + 1 == runs);
                if (q + 1 == runs) {
                    const uint32_t j = tj * kTileJ + c_first;
                    if constexpr (kAhead) {
                        if (ahead && f32) Ahead<float>::template finish<S::part>(P.e, buffer, from, i - lane, lane, j, P.size_j, bias);
                        else if (ahead) Ahead<__nv_bfloat16>::template finish<S::part>(P.e, buffer, from, i - lane, lane, j, P.size_j, bias);
                    }
                    if (!ahead) finish_tile<S::part>(P.e, from, i, P.size_i, j, P.size_j, bias, res);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(in_cta(smem_addr(&s_read[r & 1]), 0));
            }
        }
    }
    __syncwarp();
    if (!ok) atomicOr(P.status, K3HUF_ST_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    cluster_arrive_relaxed();
    cluster_wait();
    tc_fence_after();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kTileJ) : "memory");
}

// Rows that do not start on 16 bytes, copied to rows that do (TMA reads no others): 8 values per thread.
constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads) align_rows_kernel(const uint16_t *from, uint64_t stride, uint64_t rows, uint32_t cols, uint32_t pitch, uint16_t *to) {
    const uint32_t per_row = pitch / 8;
    for (uint64_t at = uint64_t(blockIdx.x) * kCopyThreads + threadIdx.x; at < rows * per_row; at += uint64_t(gridDim.x) * kCopyThreads) {
        const uint64_t r = at / per_row;
        const uint32_t c = uint32_t(at % per_row) * 8;
        const uint16_t *src = from + r * stride + c;
        const uint32_t past = uint32_t(reinterpret_cast<uintptr_t>(src) % 16 / 2);
        uint32_t w[8];
        if (c >= past && c + 16 - past <= cols) {
            // (two whole 16-byte blocks of the row's own hold them)
            const uint4 *q = reinterpret_cast<const uint4 *>(src - past), one = __ldg(q), two = __ldg(q + 1);
            w[0] = one.x, w[1] = one.y, w[2] = one.z, w[3] = one.w, w[4] = two.x, w[5] = two.y, w[6] = two.z, w[7] = two.w;
#pragma unroll
            for (uint32_t k = 0; k < 6; ++k) w[k] = past & 4 ? w[k + 2] : w[k];
#pragma unroll
            for (uint32_t k = 0; k < 5; ++k) w[k] = past & 2 ? w[k + 1] : w[k];
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) w[k] = past & 1 ? __funnelshift_r(w[k], w[k + 1], 16) : w[k];
        } else {
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) w[k] = (c + 2 * k < cols ? src[2 * k] : 0u) | (c + 2 * k + 1 < cols ? uint32_t(src[2 * k + 1]) << 16 : 0u);
        }
        reinterpret_cast<uint4 *>(to)[at] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// act'(z).  Far out, where it no longer changes in 32 bits, z stops: infinities give the limit.
template <uint32_t kAct> __device__ __forceinline__ float slope(float z) {
    if constexpr (kAct == K3HUF_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if constexpr (kAct == K3HUF_ACT_SILU) {
        z = z > 80.f ? 80.f : z < -80.f ? -80.f : z;
        const float x = __expf(-z), q = __fdividef(1.f, 1.f + x);
        return fmaf(z * q, x * q, q);
    }
    if constexpr (kAct == K3HUF_ACT_GELU) {
        z = z > 10.f ? 10.f : z < -10.f ? -10.f : z;
        const float x = __expf(-1.5957691216057308f * fmaf(0.044715f * z * z, z, z)), q = __fdividef(1.f, 1.f + x);
        return fmaf(z * q, x * q * 1.5957691216057308f * fmaf(3.f * 0.044715f * z, z, 1.f), q);
    }
    return 1.f;
}

struct SlopeParams {
    const void *z, *dy;
    __nv_bfloat16 *dz;
    float *dbias;
    uint64_t n, z_stride, dy_stride, dz_stride;
    uint32_t rows, act;
    bool add;
};

// dz and the columns' sums in one read of z and dy.  A CTA takes kSlopeLanes x kPer columns (kPer neighbouring ones per
// thread) and its share of the tokens; the CTAs of a cluster, which share the columns, add up in the order of their tokens.
// Bound by HBM: 4095 x 24576 bf16 102 to 104 us, 5.9 TB/s.  Narrow rows leave SMs idle (8192 tokens x 64 35 us, x 576 38,
// x 1024 41), and rows of no multiple of 8 go one value at a time (4095 x 24571 186 us).
constexpr int kSlopeThreads = 256, kSlopeLanes = 16, kSlopePerSm = 4;        // threads along the columns
template <typename T, int kPer> struct Few {              // neighbouring values as loaded
    T v[kPer];
};
template <typename T> struct Few<T, 8> {
    uint4 v[8 * sizeof(T) / 16];
};
template <typename T, int kPer> __device__ __forceinline__ void load_few(const T *p, Few<T, kPer> &f) {
    if constexpr (kPer == 1) {
        f.v[0] = *p;
    } else {
#pragma unroll
        for (int h = 0; h < int(8 * sizeof(T) / 16); ++h) f.v[h] = __ldcs(reinterpret_cast<const uint4 *>(p) + h);
    }
}
template <typename T, int kPer> __device__ __forceinline__ void unpack_few(const Few<T, kPer> &f, float (&o)[kPer]) {
    if constexpr (kPer == 1) {
        o[0] = ld_f32(&f.v[0]);
    } else {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(f.v);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = sizeof(T) == 4 ? __uint_as_float(w[k]) : __uint_as_float(k % 2 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
    }
}

// dz of a thread's columns for the tokens t0 + down, + kDown, ... and their sums
template <uint32_t kAct, typename Z, typename D, int kPer>
__device__ __forceinline__ void slope_rows(const SlopeParams &P, uint64_t c, uint64_t t0, uint64_t t1, float (&sum)[kPer]) {
    constexpr int kDown = kSlopeThreads / kSlopeLanes, kDepth = kPer == 1 || sizeof(Z) + sizeof(D) == 4 ? 4 : 2;      // tokens in flight
    for (uint64_t t = t0; t < t1; t += uint64_t(kDown) * kDepth) {
        Few<Z, kPer> z[kDepth];
        Few<D, kPer> g[kDepth];
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            const uint64_t at = t + uint64_t(d) * kDown;
            if (at >= t1) break;
            load_few(static_cast<const Z *>(P.z) + at * P.z_stride + c, z[d]);
            load_few(static_cast<const D *>(P.dy) + at * P.dy_stride + c, g[d]);
        }
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            const uint64_t at = t + uint64_t(d) * kDown;
            if (at >= t1) break;
            float a[kPer], b[kPer];
            unpack_few(z[d], a);
            unpack_few(g[d], b);
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                b[k] *= slope<kAct>(a[k]);
                sum[k] += b[k];
            }
            __nv_bfloat16 *o = P.dz + at * P.dz_stride + c;
            if constexpr (kPer == 8) {
                uint4 v;
                __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
                for (int k = 0; k < 4; ++k) q[k] = __floats2bfloat162_rn(b[2 * k], b[2 * k + 1]);
                __stcs(reinterpret_cast<uint4 *>(o), v);
            } else {
                st_f32(o, b[0]);
            }
        }
    }
}

template <typename Z, typename D, int kPer>
__global__ void __launch_bounds__(kSlopeThreads, kSlopePerSm) slope_kernel(const SlopeParams P, uint32_t splits) {
    constexpr int kCols = kSlopeLanes * kPer, kDown = kSlopeThreads / kSlopeLanes;
    __shared__ float s_sum[kDown][kCols + 1], s_cta[kCols];
    const uint32_t split = blockIdx.x % splits, lane = threadIdx.x % kSlopeLanes, down = threadIdx.x / kSlopeLanes;
    const uint64_t c0 = uint64_t(blockIdx.x / splits) * kCols, c = c0 + lane * kPer;
    const uint64_t t0 = P.n * split / splits + down, t1 = P.n * (split + 1) / splits;
    float sum[kPer] = {};
    if (c < P.rows) {
        if (P.act == K3HUF_ACT_NONE) slope_rows<K3HUF_ACT_NONE, Z, D, kPer>(P, c, t0, t1, sum);
        else if (P.act == K3HUF_ACT_RELU) slope_rows<K3HUF_ACT_RELU, Z, D, kPer>(P, c, t0, t1, sum);
        else if (P.act == K3HUF_ACT_SILU) slope_rows<K3HUF_ACT_SILU, Z, D, kPer>(P, c, t0, t1, sum);
        else slope_rows<K3HUF_ACT_GELU, Z, D, kPer>(P, c, t0, t1, sum);
    }
    if (!P.dbias) return;                     // (the whole grid)
#pragma unroll
    for (int k = 0; k < kPer; ++k) s_sum[down][lane * kPer + k] = sum[k];
    __syncthreads();
    if (threadIdx.x < kCols) {
        float v = 0.f;
#pragma unroll
        for (int d = 0; d < kDown; ++d) v += s_sum[d][threadIdx.x];
        s_cta[threadIdx.x] = v;
    }
    if (splits > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (split == 0 && threadIdx.x < kCols && c0 + threadIdx.x < P.rows) {
        float v = 0.f;
        for (uint32_t q = 0; q < splits; ++q) v += splits > 1 ? cluster_load(smem_addr(&s_cta[threadIdx.x]), q) : s_cta[threadIdx.x];
        float *o = P.dbias + c0 + threadIdx.x;
        *o = P.add ? *o + v : v;
    }
    __syncwarp();
    if (splits > 1) {
        cluster_arrive_relaxed();
        cluster_wait();
    }
}

// --- host -----------------------------------------------------------------------

// One operand: `rows` rows of `cols` bf16.
struct Operand {
    const void *p;
    uint64_t stride, rows;
    uint32_t cols;
};
uint32_t pitch_of(uint64_t cols) { return uint32_t((cols + 7) / 8 * 8); }
uint64_t copy_bytes(uint64_t rows, uint64_t cols) { return align_up(rows * pitch_of(cols) * 2, 256); }
// (a single row has no stride)
bool rows16(const Operand &o) { return aligned_to(o.p, 16) && (o.rows == 1 || o.stride % 8 == 0); }
uint64_t need_of(const Operand &o) { return rows16(o) ? 0 : copy_bytes(o.rows, o.cols); }

// The operand with its rows on 16 bytes: itself, or a copy in the scratch.
int aligned_rows(Operand &o, uint8_t *&scratch, uint64_t sms, cudaStream_t stream) {
    if (rows16(o)) {
        if (o.rows == 1) o.stride = pitch_of(o.cols);
        return K3HUF_OK;
    }
    const uint32_t pitch = pitch_of(o.cols);
    const uint64_t blocks = (o.rows * (pitch / 8) + kCopyThreads - 1) / kCopyThreads;
    align_rows_kernel<<<uint32_t(std::min<uint64_t>(blocks, sms * 16)), kCopyThreads, 0, stream>>>(static_cast<const uint16_t *>(o.p), o.stride, o.rows, o.cols, pitch,
                                                                                                   reinterpret_cast<uint16_t *>(scratch));
    o.p = scratch;
    o.stride = pitch;
    scratch += copy_bytes(o.rows, o.cols);
    return cuda_rc(cudaGetLastError());
}

// How a result is cut: tiles of `pair` CTAs, 128 pair x tile_j, the contraction in `splits`.
struct Cut {
    uint32_t tile_j, pair, splits;
    uint64_t tiles;
};
// Clusters of so many CTAs, each with an SM of its own, that the GPU holds at once: fewer than its SMs would make room for, as
// a cluster lies within one of its parts (50 clusters of three do not fit: 186 x 3176 x 9960 57 us with them, 45 in twos).
uint64_t clusters_of(uint32_t splits, uint64_t sms) {
    static std::atomic<int> known[64][kMaxSplits + 1];        // (by device: a cut decides the order of a result's sums)
    int dev = 0, n = 0;
    const bool kept = cudaGetDevice(&dev) == cudaSuccess && dev < 64;
    if (kept) n = known[dev][splits].load(std::memory_order_relaxed);
    if (n > 0) return uint64_t(n);
    constexpr auto kernel = product_kernel<128, false, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<128>::smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Shape<128>::smem)) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
        (void)cudaGetLastError();             // (only the choice depends on it, and the next call asks again)
        return sms / splits;
    }
    if (kept) known[dev][splits].store(n, std::memory_order_relaxed);
    return uint64_t(n);
}

// The cut of the lowest cost by this count of cycles.  A step of 64 of the contraction takes the tensor core 128 x tile_j x
// 64 / 4096 cycles per CTA, a tenth more where it is kept busiest, and the copies their bytes at kLoadRate; CTAs that share
// an SM share both.  The epilogue's time (of all the SM's CTAs; fitted to 8192 x 8192 x 64) passes beside the next tile's
// steps, and after the last tile; partial sums that meet cost kJoinCost; and the operands come from memory at kMemoryRate.
// (Times of the cuts it chooses between, us: 777 x 8192 x 576 in pairs of 128 columns 12, of 256 15, single CTAs of 128 15;
// 256 x 8192 x 8192 32, 43, 36; 8192 x 8192 x 576 62, 61, 87; 8192 x 576 x 8192 70, 78, 90; 4096 x 4096 x 4096 83, 80,
// 105; 100 x 1000 x 1000 in CTAs of 32 columns 6.7 with four splits, 7.7 without.)
constexpr uint64_t kLoadRate = 64, kJoinCost = 4500, kMemoryRate = 3344;
template <bool kMnB>
Cut choose(uint64_t size_i, uint64_t size_j, uint64_t steps, uint64_t sms) {
    Cut best{};
    uint64_t least = ~0ull;
    auto consider = [&](uint32_t tile_j, uint32_t pair, uint64_t per_sm, uint64_t epilogue) {
        Cut c{tile_j, pair, 1, (size_i + kTileI * pair - 1) / (kTileI * pair) * ((size_j + tile_j - 1) / tile_j)};
        const uint64_t busy = tile_j == 256 ? 580 : 2 * tile_j;
        const uint64_t slots = sms * per_sm / pair, step = per_sm * std::max<uint64_t>(busy, (kTileI + tile_j / pair) * 128 / kLoadRate);
        // (an operand that several tiles read comes from L2 after the first)
        const uint64_t memory = (size_i * (3 + (size_j + tile_j - 1) / tile_j) / 4 + size_j) * steps * kStep * 2 / kMemoryRate;
        const uint64_t most = pair == 2 ? 1 : std::max<uint64_t>(1, std::min<uint64_t>({kMaxSplits, slots / c.tiles, steps / 2}));
        for (c.splits = 1; c.splits <= most; ++c.splits) {
            const uint64_t at_once = c.splits > 1 ? clusters_of(c.splits, sms) * per_sm : slots;
            const uint64_t waves = (c.tiles + at_once - 1) / at_once;
            const uint64_t cost = std::max(memory, waves * std::max((steps + c.splits - 1) / c.splits * step, epilogue)) + epilogue + (c.splits > 1 ? kJoinCost : 0);
            if (cost < least || (cost == least && c.tile_j == best.tile_j)) least = cost, best = c;
        }
    };
    consider(256, 2, 1, 6600);
    consider(128, 2, 1, 3600);
    consider(128, 1, Shape<128>::per_sm, 5400);
    consider(64, 1, Shape<64>::per_sm, 4500);
    if constexpr (!kMnB) {
        consider(32, 1, Shape<32>::per_sm, 2300);
        consider(16, 1, Shape<16>::per_sm, 1900);
    }
    return best;
}

template <typename Kernel>
int launch_product(Kernel kernel, std::atomic<uint64_t> &once, uint32_t threads, size_t smem, uint64_t slots, const Cut &cut, ProductParams &P, cudaStream_t stream) {
    const int rc = once_per_device(once, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)); });
    if (rc) return rc;
    if (cut.tiles > 0x3FFFFFFFu) return K3HUF_E_ARG;           // (results of more than 2 x 10^12 elements)
    P.tiles = uint32_t(cut.tiles);
    P.tiles_i = (P.size_i + kTileI * cut.pair - 1) / (kTileI * cut.pair);
    P.tiles_j = (P.size_j + cut.tile_j - 1) / cut.tile_j;
    P.splits = cut.splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(uint32_t(std::min(cut.tiles * cut.splits, slots) * cut.pair));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cut.pair * cut.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cut.pair == 1 ? 1 : 0;     // (a pair's kernel has its cluster in its declaration)
    return cuda_rc(cudaLaunchKernelEx(&cfg, kernel, P));
}

template <uint32_t kTileJ, bool kMnA, bool kMnB>
int launch_one(const Cut &cut, ProductParams &P, uint64_t sms, cudaStream_t stream) {
    static std::atomic<uint64_t> once{0};
    return launch_product(product_kernel<kTileJ, kMnA, kMnB>, once, kThreads, Shape<kTileJ>::smem, sms * Shape<kTileJ>::per_sm, cut, P, stream);
}
template <uint32_t kTileJ, bool kMnA, bool kMnB, bool kAhead>
int launch_pair(const Cut &cut, ProductParams &P, uint64_t sms, cudaStream_t stream) {
    static std::atomic<uint64_t> once{0};
    return launch_product(pair_kernel<kTileJ, kMnA, kMnB, kAhead>, once, kPairThreads, Pair<kTileJ>::smem + (kAhead ? Pair<kTileJ>::ahead : 0), sms / 2, cut, P, stream);
}

// out[j][i] = sum_k A[i][k] B[j][k]
template <bool kMnA, bool kMnB>
int product(const Operand &a, const Operand &b, uint64_t size_i, uint64_t size_j, uint64_t size_k, const Epilogue &e, uint32_t *status, uint64_t sms, cudaStream_t stream) {
    ProductParams P{};
    P.e = e;
    P.status = status;
    P.size_i = uint32_t(size_i), P.size_j = uint32_t(size_j), P.steps = uint32_t((size_k + kStep - 1) / kStep);
    const uint32_t width = uint32_t(elem_bytes(e.out_type));
    const bool ahead = e.residual && aligned_to(e.residual, 16) && e.residual_stride * width % 16 == 0;
    const bool f32 = e.out_type == K3HUF_F32 || (e.z && e.z_type == K3HUF_F32);
    P.run = f32 ? kChain / (kStep / 16) : std::min(P.steps, kLongRun);
    const Cut cut = choose<kMnB>(size_i, size_j, P.steps, sms);
    int rc = tensor_map(&P.a, a.p, K3HUF_BF16, a.rows, a.cols, a.stride, kMnA ? kStep : kTileI, kStep, true);
    if (!rc) rc = tensor_map(&P.b, b.p, K3HUF_BF16, b.rows, b.cols, b.stride, kMnB ? kStep : cut.tile_j / cut.pair, kStep, true);
    if (rc) return rc;
    if constexpr (kMnA == kMnB) {             // (dx has no residual)
        if (cut.pair == 2 && ahead) return cut.tile_j == 256 ? launch_pair<256, kMnA, kMnB, true>(cut, P, sms, stream) : launch_pair<128, kMnA, kMnB, true>(cut, P, sms, stream);
    }
    if (cut.pair == 2) return cut.tile_j == 256 ? launch_pair<256, kMnA, kMnB, false>(cut, P, sms, stream) : launch_pair<128, kMnA, kMnB, false>(cut, P, sms, stream);
    if constexpr (!kMnB) {
        if (cut.tile_j == 16) return launch_one<16, kMnA, kMnB>(cut, P, sms, stream);
        if (cut.tile_j == 32) return launch_one<32, kMnA, kMnB>(cut, P, sms, stream);
    }
    return cut.tile_j == 64 ? launch_one<64, kMnA, kMnB>(cut, P, sms, stream) : launch_one<128, kMnA, kMnB>(cut, P, sms, stream);
}

bool sizes_ok(uint64_t n, uint64_t rows, uint64_t cols) { return rows && cols && n < (1ull << 31) && rows < (1ull << 31) && cols < (1ull << 31); }
bool act_ok(uint32_t act) { return act <= K3HUF_ACT_GELU; }

}  // namespace
}  // namespace k3huf

using namespace k3huf;

extern "C" int k3huf_linear_scratch_bytes(uint64_t n_tokens, uint64_t rows, uint64_t cols, int grad, int any, size_t *scratch_bytes) {
    if (!scratch_bytes || !sizes_ok(n_tokens, rows, cols)) return K3HUF_E_ARG;
    const bool odd_cols = any || cols % 8, odd_rows = any || rows % 8;
    *scratch_bytes = (odd_cols ? copy_bytes(n_tokens, cols) + copy_bytes(rows, cols) : 0) + (grad && odd_rows ? copy_bytes(n_tokens, rows) : 0);
    return K3HUF_OK;
}

extern "C" int k3huf_linear(const void *d_x, uint64_t x_stride, uint64_t n_tokens, const void *d_w, uint64_t w_stride, uint64_t rows, uint64_t cols,
                            const void *d_bias, uint32_t bias_type, uint32_t act, const void *d_residual, uint64_t residual_stride, void *d_y, uint64_t y_stride,
                            uint32_t y_type, void *d_z, uint64_t z_stride, uint32_t z_type, void *d_scratch, size_t scratch_bytes, uint32_t *d_status, void *stream) {
    if (!sizes_ok(n_tokens, rows, cols) || !act_ok(act) || !elem_ok(y_type) || (d_bias && !elem_ok(bias_type)) || (d_z && !elem_ok(z_type)) || !d_status || x_stride < cols ||
        w_stride < cols || y_stride < rows || (d_residual && residual_stride < rows) || (d_z && z_stride < rows))
        return K3HUF_E_ARG;
    if (!aligned_to(d_x, 2) || !aligned_to(d_w, 2) || (d_bias && !aligned_to(d_bias, elem_bytes(bias_type))) || !aligned_to(d_residual, elem_bytes(y_type)) ||
        !aligned_to(d_y, elem_bytes(y_type)) || (d_z && !aligned_to(d_z, elem_bytes(z_type))) || !aligned_to(d_scratch, 256) || !aligned_to(d_status, 4) ||
        (d_residual && d_residual == d_y && residual_stride != y_stride) || (d_z && d_z == d_y))
        return K3HUF_E_ARG;
    if (n_tokens == 0) return K3HUF_OK;
    if (!d_x || !d_w || !d_y) return K3HUF_E_ARG;
    // (other CTAs read x and w, and the bias, while a result is written)
    for (const void *out : {d_y, d_z})
        if (out && (out == d_x || out == d_w || out == d_bias)) return K3HUF_E_ARG;
    if (d_z && d_z == d_residual && (z_type != y_type || z_stride != residual_stride)) return K3HUF_E_ARG;
    Operand w{d_w, w_stride, rows, uint32_t(cols)}, x{d_x, x_stride, n_tokens, uint32_t(cols)};
    const uint64_t need = need_of(w) + need_of(x);
    if (need && (!d_scratch || scratch_bytes < need)) return K3HUF_E_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *scratch = static_cast<uint8_t *>(d_scratch);
    uint64_t sms = 0;
    int rc = sm_count(&sms);
    if (!rc) rc = aligned_rows(w, scratch, sms, st);
    if (!rc) rc = aligned_rows(x, scratch, sms, st);
    if (rc) return rc;
    const Epilogue e{d_bias, d_residual, d_y, d_z, y_stride, residual_stride, z_stride, y_type, bias_type, z_type, act};
    return product<false, false>(w, x, rows, n_tokens, cols, e, d_status, sms, st);
}

extern "C" int k3huf_linear_dz(const void *d_z, uint32_t z_type, uint64_t z_stride, const void *d_dy, uint32_t dy_type, uint64_t dy_stride, uint64_t n_tokens,
                               uint64_t rows, uint32_t act, void *d_dz, uint64_t dz_stride, float *d_dbias, uint32_t flags, void *stream) {
    if (!sizes_ok(n_tokens, rows, 1) || !act_ok(act) || !elem_ok(z_type) || !elem_ok(dy_type) || z_stride < rows || dy_stride < rows || dz_stride < rows ||
        (flags & ~uint32_t(K3HUF_ACCUMULATE)))
        return K3HUF_E_ARG;
    if (!aligned_to(d_z, elem_bytes(z_type)) || !aligned_to(d_dy, elem_bytes(dy_type)) || !aligned_to(d_dz, 2) || !aligned_to(d_dbias, 4)) return K3HUF_E_ARG;
    if (n_tokens && (!d_z || !d_dy || !d_dz)) return K3HUF_E_ARG;
    // (in place where the elements are as wide, so that no thread meets another's)
    if ((d_dz && d_dz == d_dy && (dy_type != K3HUF_BF16 || dy_stride != dz_stride)) || (d_dz && d_dz == d_z && (z_type != K3HUF_BF16 || z_stride != dz_stride))) return K3HUF_E_ARG;
    const bool add = (flags & K3HUF_ACCUMULATE) != 0;
    if (n_tokens == 0 && (!d_dbias || add)) return K3HUF_OK;
    if (n_tokens && d_dbias && (d_dbias == d_z || d_dbias == d_dy || d_dbias == d_dz)) return K3HUF_E_ARG;
    uint64_t sms = 0;
    const int rc = sm_count(&sms);
    if (rc) return rc;
    const SlopeParams P{d_z, d_dy, static_cast<__nv_bfloat16 *>(d_dz), d_dbias, n_tokens, z_stride, dy_stride, dz_stride, uint32_t(rows), act, add};
    auto on16 = [](const void *p, uint64_t stride, uint32_t type) { return aligned_to(p, 16) && stride * elem_bytes(type) % 16 == 0; };
    const bool vec = rows % 8 == 0 && on16(d_z, z_stride, z_type) && on16(d_dy, dy_stride, dy_type) && on16(d_dz, dz_stride, K3HUF_BF16);
    const uint32_t cols = kSlopeLanes * (vec ? 8 : 1);
    const uint64_t blocks = (rows + cols - 1) / cols;
    // the tokens split over a cluster of up to eight CTAs, so that the GPU's places (four per SM) are filled best
    const uint64_t slots = sms * kSlopePerSm;
    uint32_t splits = 1;
    auto idle = [&](uint64_t k) { return double((blocks * k + slots - 1) / slots) * double(slots) / double(blocks * k); };      // places taken per CTA
    for (uint32_t k = 2; k <= 8 && n_tokens / k >= 64; ++k)
        if (idle(k) < idle(splits) - 0.02) splits = k;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(uint32_t(blocks * splits));
    cfg.blockDim = dim3(kSlopeThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    using BF = __nv_bfloat16;
    auto run = [&](auto vec8, auto one) { return cuda_rc(vec ? cudaLaunchKernelEx(&cfg, vec8, P, splits) : cudaLaunchKernelEx(&cfg, one, P, splits)); };
    if (z_type == K3HUF_BF16) return dy_type == K3HUF_BF16 ? run(slope_kernel<BF, BF, 8>, slope_kernel<BF, BF, 1>) : run(slope_kernel<BF, float, 8>, slope_kernel<BF, float, 1>);
    return dy_type == K3HUF_BF16 ? run(slope_kernel<float, BF, 8>, slope_kernel<float, BF, 1>) : run(slope_kernel<float, float, 8>, slope_kernel<float, float, 1>);
}

extern "C" int k3huf_linear_grad(const void *d_x, uint64_t x_stride, uint64_t n_tokens, const void *d_w, uint64_t w_stride, uint64_t rows, uint64_t cols,
                                 const void *d_dz, uint64_t dz_stride, void *d_dx, uint64_t dx_stride, uint32_t dx_type, float *d_dw, void *d_scratch,
                                 size_t scratch_bytes, uint32_t *d_status, uint32_t flags, void *stream) {
    if (!sizes_ok(n_tokens, rows, cols) || !d_status || dz_stride < rows || (d_dx && (!elem_ok(dx_type) || dx_stride < cols || w_stride < cols)) || (d_dw && x_stride < cols) ||
        (flags & ~uint32_t(K3HUF_ACCUMULATE)))
        return K3HUF_E_ARG;
    if (!aligned_to(d_x, 2) || !aligned_to(d_w, 2) || !aligned_to(d_dz, 2) || (d_dx && !aligned_to(d_dx, elem_bytes(dx_type))) || !aligned_to(d_dw, 4) ||
        !aligned_to(d_scratch, 256) || !aligned_to(d_status, 4))
        return K3HUF_E_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool add = (flags & K3HUF_ACCUMULATE) != 0;
    if (n_tokens == 0) return d_dw && !add ? cuda_rc(cudaMemsetAsync(d_dw, 0, rows * cols * 4, st)) : K3HUF_OK;
    if ((!d_dx && !d_dw) || !d_dz || (d_dx && !d_w) || (d_dw && !d_x)) return K3HUF_E_ARG;
    // (dx is written before dW's sums read x and dz; and other CTAs read what a result is made from while it is written)
    if (d_dx && (d_dx == d_dz || d_dx == d_w || d_dx == d_dw || (d_dw && d_dx == d_x))) return K3HUF_E_ARG;
    if (d_dw && (d_dw == d_dz || d_dw == d_x || (d_dx && d_dw == d_w))) return K3HUF_E_ARG;
    Operand dz{d_dz, dz_stride, n_tokens, uint32_t(rows)}, w{d_w, w_stride, rows, uint32_t(cols)}, x{d_x, x_stride, n_tokens, uint32_t(cols)};
    const uint64_t need = need_of(dz) + (d_dx ? need_of(w) : 0) + (d_dw ? need_of(x) : 0);
    if (need && (!d_scratch || scratch_bytes < need)) return K3HUF_E_ARG;
    uint8_t *scratch = static_cast<uint8_t *>(d_scratch);
    uint64_t sms = 0;
    int rc = sm_count(&sms);
    if (!rc) rc = aligned_rows(dz, scratch, sms, st);
    if (!rc && d_dx) rc = aligned_rows(w, scratch, sms, st);
    if (!rc && d_dx) rc = product<true, false>(w, dz, cols, n_tokens, rows, Epilogue{nullptr, nullptr, d_dx, nullptr, dx_stride, 0, 0, dx_type, 0, 0, K3HUF_ACT_NONE}, d_status, sms, st);
    if (!rc && d_dw) rc = aligned_rows(x, scratch, sms, st);
    if (!rc && d_dw)
        rc = product<true, true>(x, dz, cols, rows, n_tokens, Epilogue{nullptr, add ? d_dw : nullptr, d_dw, nullptr, cols, cols, 0, K3HUF_F32, 0, 0, K3HUF_ACT_NONE}, d_status, sms, st);
    return rc;
}
