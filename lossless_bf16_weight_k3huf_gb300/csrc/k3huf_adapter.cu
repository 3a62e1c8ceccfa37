// Low-rank adapters of many requests beside a shared projection, and their
// gradients.  With i = ids[t] the adapter of token t, A_i (rank x cols),
// B_i (rank x rows) and s_i its factors and scale:
//   y[t]  = base[t] + s_i (x[t] A_i^T) B_i
//   dh[t] = s_i dy[t] B_i^T         dx[t] = dx_base[t] + dh[t] A_i
//   dA_i  = sum_t dh[t]^T x[t]      dB_i  = sum_t (s_i x[t] A_i^T)^T dy[t]
// Both factors are stored rank-major, so forward and backward are the same
// three products: "shrink" (a dot product with every row of a factor),
// "expand" (a sum of a factor's rows) and "outer" (a sum over tokens).
//
// Three forms, by a rule on sizes and alignment (run_form):
//  - few tokens (their factor rows up to kFewBytes): fp32 arithmetic, a CTA per
//    token and part of the factor; every factor row is read once per token,
//    mostly from L2;
//  - many: tcgen05.mma on tiles of 128 tokens, described at each kernel;
//  - rows that do not start on 16 bytes: one CTA per token, element by element.
// The rank-wide intermediates are fp32 sums.  The tensor cores take them as a
// sum of bf16 parts: three parts (24 bits) where the result is fp32, two (to
// 2^-17 of themselves) where it is rounded to bf16, to 2^-9.  Three there too
// cost 8192 tokens x 64 x (8192 + 24576) 202 us instead of 194, 4000 tokens of
// 64 adapters in any order, rank 16, 139 instead of 125.
#include <algorithm>
#include <cmath>

#include "k3huf_tc.h"

namespace k3huf {
namespace {

constexpr int kThreads = 256;
constexpr uint64_t kFewBytes = 300'000'000;    // of factor rows, read once per token

__device__ __forceinline__ bool adapter_of(const int32_t *ids, uint64_t t, uint32_t n_adapters, int32_t &i) {
    i = ids[t];
    return i >= 0 && uint32_t(i) < n_adapters;
}

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load4(const float *p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&f)[4]) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u), f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float *p, const float (&f)[4]) { *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]); }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&f)[4]) {
    uint2 o;
    __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(&o);
    q[0] = __floats2bfloat162_rn(f[0], f[1]);
    q[1] = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2 *>(p) = o;
}

// --- rows of any alignment --------------------------------------------------------
//
// Bound by their loads of one element each: 192 tokens x 16 x (8192 + 8192) 133 us (15
// with rows on 16 bytes); gradients of 515 tokens x 32 1044 us (43), most of it the
// outer product's search through the ids for every element.

// h[t, r] = s_i v[t] . w[i, r]; zero without an adapter.  One CTA per token, one warp per row of the factor.
__global__ void __launch_bounds__(kThreads)
shrink_any_kernel(const __nv_bfloat16 *v, uint64_t stride, const __nv_bfloat16 *w, const float *scales, const int32_t *ids, uint32_t n_adapters, uint32_t rank, uint64_t len, float *h, uint32_t *status) {
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
expand_any_kernel(const float *h, const __nv_bfloat16 *w, const int32_t *ids, uint32_t n_adapters, uint32_t rank, uint64_t len, const T *base, uint64_t base_stride, T *y, uint64_t y_stride) {
    const uint64_t t = blockIdx.x;
    int32_t i;
    const bool any = adapter_of(ids, t, n_adapters, i);
    for (uint64_t c = threadIdx.x; c < len; c += kThreads) {
        float acc = 0.f;
        if (any)
            for (uint32_t r = 0; r < rank; ++r) acc = fmaf(h[t * rank + r], ld_f32(w + (uint64_t(i) * rank + r) * len + c), acc);
        // (without an adapter the base as it is: -0 + 0 would be +0)
        const float b = base ? ld_f32(base + t * base_stride + c) : 0.f;
        st_f32(y + t * y_stride + c, any ? b + acc : b);
    }
}

// g[i, r] (+)= sum over tokens of adapter i of h[t, r] v[t].  One CTA per column block and row of a factor.
__global__ void __launch_bounds__(kThreads)
outer_any_kernel(const float *h, const __nv_bfloat16 *v, uint64_t stride, const int32_t *ids, uint64_t n, uint32_t n_adapters, uint32_t rank, uint64_t len, float *g, bool add) {
    const uint64_t c = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (c >= len) return;
    for (uint64_t row = blockIdx.y; row < uint64_t(n_adapters) * rank; row += gridDim.y) {
        const uint32_t i = uint32_t(row / rank), r = uint32_t(row % rank);
        float acc = 0.f;
        bool used = false;
        for (uint64_t t = 0; t < n; ++t)
            if (ids[t] == int32_t(i)) {
                acc = fmaf(h[t * rank + r], ld_f32(v + t * stride + c), acc);
                used = true;
            }
        float *out = g + row * len + c;
        // (adapters without a token are left alone: another call may be adding to them)
        if (used || !add) *out = add ? *out + acc : acc;
    }
}

// --- few tokens ---------------------------------------------------------------

constexpr int kRows = 4;                      // factor rows per CTA
constexpr uint32_t kFewCols = 512;            // columns of y per CTA

// h[t, r] = s_i v[t] . w[i, r], zero without an adapter, for kRows rows r: one
// CTA per token and group of rows, 16-byte loads.  At 4 tokens x 16 x 8192 it
// takes the latency of two dependent loads and a block sum.
__global__ void __launch_bounds__(kThreads)
shrink_few_kernel(const __nv_bfloat16 *v, uint64_t stride, const __nv_bfloat16 *w, const float *scales, const int32_t *ids, uint32_t n_adapters, uint32_t rank, uint32_t len, float *h, uint32_t *status) {
    __shared__ float s_sum[kThreads / 32][kRows];
    grid_dep_launch();
    const uint64_t t = blockIdx.x;
    const uint32_t r0 = blockIdx.y * kRows, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int32_t i;
    const bool any = adapter_of(ids, t, n_adapters, i);
    if (!any) {
        if (i >= 0 && r0 == 0 && threadIdx.x == 0) atomicOr(status, K3HUF_ST_TOKEN);
        if (threadIdx.x < kRows && r0 + threadIdx.x < rank) h[t * rank + r0 + threadIdx.x] = 0.f;
        return;
    }
    const uint4 *x = reinterpret_cast<const uint4 *>(v + t * stride);
    const uint4 *a = reinterpret_cast<const uint4 *>(w + (uint64_t(i) * rank + r0) * len);
    float acc[kRows] = {};
#pragma unroll 4
    for (uint32_t c = threadIdx.x; c < len / 8; c += kThreads) {
        float f[8], g[8];
        unpack8(__ldg(x + c), f);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r0 + r >= rank) break;
            unpack8(__ldg(a + uint64_t(r) * (len / 8) + c), g);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[r] = fmaf(f[k], g[k], acc[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        acc[r] = warp_sum(acc[r]);
        if (lane == 0) s_sum[warp][r] = acc[r];
    }
    __syncthreads();
    if (threadIdx.x < kRows && r0 + threadIdx.x < rank) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) sum += s_sum[k][threadIdx.x];
        h[t * rank + r0 + threadIdx.x] = scales[i] * sum;
    }
}

// y[t] = base[t] + sum_r h[t, r] w[i, r]: one CTA per token and kFewCols columns,
// four per thread.
template <typename T>
__global__ void __launch_bounds__(kFewCols / 4)
expand_few_kernel(const float *h, const __nv_bfloat16 *w, const int32_t *ids, uint32_t n_adapters, uint32_t rank, uint32_t len, const T *base, uint64_t base_stride, T *y, uint64_t y_stride) {
    __shared__ float s_h[K3HUF_MAX_RANK];
    const uint64_t t = blockIdx.x;
    const uint32_t c = blockIdx.y * kFewCols + threadIdx.x * 4;
    grid_dep_wait();
    int32_t i;
    const bool any = adapter_of(ids, t, n_adapters, i);
    if (any && threadIdx.x < rank) s_h[threadIdx.x] = h[t * rank + threadIdx.x];
    __syncthreads();
    if (c >= len) return;
    float acc[4] = {};
    if (base) load4(base + t * base_stride + c, acc);
    float sum[4] = {};
    if (any) {
        const uint2 *b = reinterpret_cast<const uint2 *>(w + uint64_t(i) * rank * len + c);
#pragma unroll 16
        for (uint32_t r = 0; r < rank; ++r) {
            const uint2 v = __ldg(b + uint64_t(r) * (len / 4));
            const float f = s_h[r];
            sum[0] = fmaf(f, __uint_as_float(v.x << 16), sum[0]);
            sum[1] = fmaf(f, __uint_as_float(v.x & 0xFFFF0000u), sum[1]);
            sum[2] = fmaf(f, __uint_as_float(v.y << 16), sum[2]);
            sum[3] = fmaf(f, __uint_as_float(v.y & 0xFFFF0000u), sum[3]);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = any ? acc[k] + sum[k] : acc[k];       // (the base as it is: -0 + 0 would be +0)
    store4(y + t * y_stride + c, acc);
}

// --- many tokens: tensor cores --------------------------------------------------

constexpr uint32_t kTile = 128;               // tokens per tile
constexpr uint32_t kMaxParts = 3;             // bf16 parts of a rank-wide intermediate
constexpr uint32_t kStep = 64;                // contraction per staged step: one 128-byte row
constexpr uint32_t kTileBytes = kTile * 128;  // one staged tile of 128 rows
// Additions in the tensor core before a sum moves to registers.  One of them
// errs by about 1.3e-8 of the sum, always to the same side (measured: 2e-5 after
// 1536), while fp32 additions in registers round to nearest.
constexpr uint32_t kChain = 32;

// The adapters of a tile's tokens, each once, in the order of their first
// token: of[t] the place of token t's adapter (-1: none), list the adapters.
// All threads of the CTA (at least 128); returns their number.
struct TileAdapters {
    int32_t id[kTile], list[kTile];
    int16_t of[kTile];
    uint32_t count[4];
};
__device__ uint32_t tile_adapters(TileAdapters &s, const int32_t *ids, uint64_t t0, uint64_t n, uint32_t n_adapters, uint32_t *status) {
    const uint32_t t = threadIdx.x, lane = t % 32, warp = t / 32;
    int32_t id = -1;
    bool first = false;
    uint32_t below = 0;
    if (t < kTile) {
        if (t0 + t < n) id = ids[t0 + t];
        if (id >= 0 && uint32_t(id) >= n_adapters) {
            if (status) atomicOr(status, K3HUF_ST_TOKEN);
            id = -1;
        }
        s.id[t] = id;
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        first = id >= 0 && uint32_t(__ffs(same)) - 1 == lane;
    }
    __syncthreads();
    if (t < kTile) {
        if (first)
            for (uint32_t u = 0; u < warp * 32; ++u) first = first && s.id[u] != id;
        const uint32_t firsts = __ballot_sync(0xffffffffu, first);
        below = __popc(firsts & ((1u << lane) - 1u));
        if (lane == 0) s.count[warp] = __popc(firsts);
    }
    __syncthreads();
    if (first) {
        for (uint32_t w = 0; w < warp; ++w) below += s.count[w];
        s.list[below] = id;
    }
    __syncthreads();
    const uint32_t count = s.count[0] + s.count[1] + s.count[2] + s.count[3];
    if (t < kTile) {
        int32_t k = -1;
        if (id >= 0)
            for (uint32_t u = 0; u < count && k < 0; ++u)
                if (s.list[u] == id) k = int32_t(u);
        s.of[t] = int16_t(k);
    }
    __syncthreads();
    return count;
}

// x as a sum of bf16 parts.  A finite one that would round to an infinity starts with the largest
// bf16 instead, whose rest the other parts hold; an infinity is the first part and zeros.
__device__ __forceinline__ void parts_of(float x, __nv_bfloat16 (&p)[3]) {
    p[0] = __float2bfloat16_rn(x);
    float a = x - __bfloat162float(p[0]);
    const float most = __uint_as_float(0x7F7F0000u);          // the largest bf16
    if (fabsf(x) > most) {
        const bool infinite = fabsf(x) == INFINITY;
        p[0] = __float2bfloat16_rn(infinite ? x : copysignf(most, x));
        a = infinite ? 0.f : x - copysignf(most, x);
    }
    p[1] = __float2bfloat16_rn(a);
    p[2] = __float2bfloat16_rn(a - __bfloat162float(p[1]));
}

struct ShrinkJob {
    CUtensorMap v, w;                         // tokens x len, boxes of 64 x kTile; rank rows x len, boxes of 64 x rank
    uint32_t len;
    __nv_bfloat16 *h;                         // parts x tokens x pitch
};
struct ShrinkParams {
    ShrinkJob job[2];
    const float *scales;
    const int32_t *ids;
    uint32_t *status;
    uint64_t n;
    uint32_t n_adapters, rank, rank_pad, pitch, parts, splits;
};

// The shrink.  D[128 tokens, rank rows of the tile's adapters] = V W^T, both
// operands K-major tiles brought by TMA, kStep of the contraction per stage;
// every token keeps the columns of its own adapter.  CTAs: a tile of tokens x some
// of its groups of adapters, whose rank rows fill 128 columns (a tile whose tokens
// share adapters has one or two groups), x a split of the contraction; the splits
// are a cluster, whose partial sums meet through shared memory in the order of
// the splits.  One thread keeps the products and one the
// copies going for a run of kRun steps while the CTA moves the run before it from
// the other half of TMEM to registers.  Bound by the read of V (and of the factors
// when every token has its own): 36 us for 8192 tokens x 8192 to rank 64, 3.7 TB/s.
constexpr uint32_t kShrinkStages = 3, kShrinkStage = 2 * kTileBytes;
constexpr size_t kShrinkSmem = kShrinkStages * kShrinkStage + 1024;
constexpr uint32_t kMaxSplits = 8;

__global__ void __launch_bounds__(kThreads) shrink_kernel(const __grid_constant__ ShrinkParams P) {
    extern __shared__ uint8_t raw[];
    __shared__ TileAdapters tile;
    __shared__ __align__(8) uint64_t s_full[kShrinkStages], s_free[kShrinkStages], s_run[2];
    __shared__ uint32_t s_tmem, s_gave_up;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32, base = smem_addr(smem);
    const ShrinkJob &J = P.job[blockIdx.z];
    const uint32_t split = blockIdx.x % P.splits, rp = P.rank_pad;
    const uint64_t t0 = uint64_t(blockIdx.x / P.splits) * kTile;
    grid_dep_launch();
    const uint32_t per = kTile / rp, count = tile_adapters(tile, P.ids, t0, P.n, P.n_adapters, split + blockIdx.y + blockIdx.z == 0 ? P.status : nullptr);
    if (blockIdx.y * per >= count) return;    // (the whole cluster)
    if (warp == 0) tmem_alloc(smem_addr(&s_tmem), 256);
    if (tid == 0) {
        for (uint32_t i = 0; i < kShrinkStages; ++i) {
            mbar_init(smem_addr(&s_full[i]), 1);
            mbar_init(smem_addr(&s_free[i]), 1);
        }
        s_gave_up = 0;
        mbar_init(smem_addr(&s_run[0]), 1);
        mbar_init(smem_addr(&s_run[1]), 1);
        fence_async_shared();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t steps = (J.len + kStep - 1) / kStep;
    const uint32_t k0 = steps * split / P.splits, n_steps = steps * (split + 1) / P.splits - k0;
    constexpr uint32_t kRun = kChain / (kStep / 16);
    const uint32_t runs = (n_steps + kRun - 1) / kRun;
    bool ok = true;
    // the tile's groups of adapters that fall to this cluster; steps and runs count on (step0, run0)
    for (uint32_t a0 = blockIdx.y * per, step0 = 0, run0 = 0; a0 < count; a0 += gridDim.y * per, step0 += n_steps, run0 += runs) {
        const uint32_t na = min(per, count - a0), cols = na * rp;          // (<= 128, a multiple of 16)
        auto load = [&](uint32_t i) {             // by one thread
            const uint32_t stage = (step0 + i) % kShrinkStages, at = base + stage * kShrinkStage, bar = smem_addr(&s_full[stage]);
            mbar_expect(bar, kTileBytes + na * P.rank * 128);
            tma_load(at, &J.v, int32_t((k0 + i) * kStep), int32_t(t0), bar);
            for (uint32_t a = 0; a < na; ++a) tma_load(at + kTileBytes + a * rp * 128, &J.w, int32_t((k0 + i) * kStep), tile.list[a0 + a] * int32_t(P.rank), bar);
        };
        const uint32_t desc = mma_desc(kTile, cols, 0, 0);
        const uint64_t d0 = tile_desc(base, 16, 1024);
        uint32_t loaded = 0;
        if (tid == 32)
            for (; loaded < min(kShrinkStages - 1, n_steps); ++loaded) load(loaded);
        // this thread's sums: token (lane) warp % 4 * 32 + lane, columns warp / 4 * 64 on
        float sum[64] = {};
        for (uint32_t run = 0; run <= runs; ++run) {
            const uint32_t last = min((run + 1) * kRun, n_steps);
            if (tid == 0 && run < runs) {
                for (uint32_t i = run * kRun; i < last && ok; ++i) {
                    const uint32_t stage = (step0 + i) % kShrinkStages;
                    ok = mbar_wait(smem_addr(&s_full[stage]), (step0 + i) / kShrinkStages & 1);
                    tc_fence_after();
                    const uint64_t a = d0 + stage * (kShrinkStage >> 4), b = a + (kTileBytes >> 4);
#pragma unroll
                    for (uint32_t s = 0; s < kStep / 16; ++s) mma(tmem + ((run0 + run) & 1) * 128, a + 2 * s, b + 2 * s, desc, i % kRun || s);
                    mma_commit(smem_addr(&s_free[stage]));
                }
                mma_commit(smem_addr(&s_run[(run0 + run) & 1]));
            }
            if (tid == 32 && run < runs)
                // a stage is free once the products of the step before are done
                for (uint32_t i = run * kRun; i < last && loaded < n_steps && ok; ++i) {
                    if (i > 0) ok = mbar_wait(smem_addr(&s_free[(step0 + i - 1) % kShrinkStages]), (step0 + i - 1) / kShrinkStages & 1);
                    if (ok) load(loaded++);
                }
            __syncwarp();
            if (run > 0) {
                const uint32_t r = run0 + run - 1;
                if (!mbar_wait(smem_addr(&s_run[r & 1]), r / 2 & 1)) ok = false;
                tc_fence_after();
#pragma unroll
                for (uint32_t c = 0; c < 64; c += 16)
                    if (warp / 4 * 64 + c < cols) {
                        float v[16];
                        tmem_load16(tmem + ((warp % 4) << 21) + (r & 1) * 128 + warp / 4 * 64 + c, v);
#pragma unroll
                        for (int k = 0; k < 16; ++k) sum[c + k] += v[k];
                    }
                tc_fence_before();
            }
            __syncthreads();                      // (the run after the next writes this half)
        }
        if (!ok) {
            atomicOr(P.status, K3HUF_ST_TIMEOUT);
            s_gave_up = 1;
        }
        __syncthreads();
        // a wait gave up, in any thread: copies still in flight, if any, land before the CTA ends
        if (tid == 32 && s_gave_up)
            for (uint32_t i = loaded > kShrinkStages ? loaded - kShrinkStages : 0; i < loaded; ++i) mbar_wait(smem_addr(&s_full[(step0 + i) % kShrinkStages]), (step0 + i) / kShrinkStages & 1);

        // each token's own columns, to shared memory (odd stride: one bank per lane)
        float *part = reinterpret_cast<float *>(smem);
        const uint32_t stride = rp + 1;
        {
            const uint32_t t = warp % 4 * 32 + lane;
            const int32_t of = tile.of[t];
#pragma unroll
            for (uint32_t c = 0; c < 64; c += 16) {
                const uint32_t q = warp / 4 * 64 + c;
                if (q < cols && of == int32_t(a0 + q / rp))
#pragma unroll
                    for (uint32_t k = 0; k < 16; ++k) part[t * stride + q % rp + k] = sum[c + k];
            }
        }
        if (P.splits > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        // a share of the tile's tokens per split: sum over the splits, scale, parts; zeros for the
        // rank's padding (whose columns of D hold the next adapter's)
        const uint32_t r0 = kTile * split / P.splits, r1 = kTile * (split + 1) / P.splits;
        for (uint32_t i = r0 * rp + tid; i < r1 * rp; i += kThreads) {
            const uint32_t t = i / rp, j = i % rp;
            const int32_t of = tile.of[t];
            if (of < int32_t(a0) || of >= int32_t(a0 + na)) continue;
            float total = 0.f;
            if (j < P.rank)
                for (uint32_t q = 0; q < P.splits; ++q) total += P.splits > 1 ? cluster_load(smem_addr(part + t * stride + j), q) : part[t * stride + j];
            __nv_bfloat16 p[3];
            parts_of(j < P.rank ? P.scales[tile.list[of]] * total : 0.f, p);
            for (uint32_t q = 0; q < P.parts; ++q) J.h[(q * P.n + t0 + t) * P.pitch + j] = p[q];
        }
        fence_async_shared();                     // (the next group's copies overwrite what was read here)
        if (P.splits > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
    }
    if (warp == 0) tmem_free(tmem, 256);
}

struct ExpandParams {
    CUtensorMap h, w, base, y;                // parts x tokens rows of 64-value blocks; rank rows x len, boxes of 64 x rank; boxes of 128 bytes x 128 tokens
    const int32_t *ids;
    uint32_t *status;
    uint64_t n;
    uint32_t n_adapters, rank, rank_pad, len, groups;
    bool has_base;
};

// The expand.  D[128 tokens, columns] = H W_a for one adapter a of the tile after
// another, each added only where a token has that adapter: no token meets
// another adapter's values, not even as zero times infinity.  H (the same for
// all of them) is read K-major, in parts, W MN-major as it lies in memory.  A
// thread holds a token's neighbouring columns, so it adds 16 bytes of the base
// at a time, in tiles of 128-byte rows that TMA brings and takes away swizzled.
// CTAs: a tile of tokens x a range of column tiles; a step is one adapter of
// one column tile.  Warps 0 to 7 add; a thread of warp 8 issues the products, two
// steps ahead of the additions; one of warp 9 brings the base and takes y away;
// one of warp 10 brings W.  Bound by the read of the base and the write of y: 142 us for
// 8192 tokens x 24576 bf16 columns, 5.7 TB/s.  (With columns as the lanes, 2 bytes
// at a time, the additions took five times the instructions, 184 us.)
constexpr uint32_t kExpandThreads = kThreads + 96;
template <typename T, uint32_t kBlocks> struct Expand {       // kBlocks: blocks of 64 rank rows
    static constexpr uint32_t row = 128 / sizeof(T), cols = 2 * row;      // columns of a 128-byte row; of a tile of two of them
    static constexpr uint32_t parts = sizeof(T) == 4 ? 3 : 2;
    static constexpr uint32_t h_bytes = parts * kBlocks * kTileBytes, w_block = kBlocks * kStep * 128, w_bytes = cols / 64 * w_block, w_stages = kBlocks == 1 ? 3 : 2;
    static constexpr uint32_t io_bytes = 2 * kTileBytes, io_stages = kBlocks == 1 ? 4 : 2;
    static constexpr size_t smem = h_bytes + w_stages * w_bytes + io_stages * io_bytes + 1024;
    static_assert(smem <= 220 * 1024, "shared memory of one CTA");
};

__device__ __forceinline__ void add_chunk(uint4 &v, const uint32_t *r, __nv_bfloat16) {
    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __fadd2_rn(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
}
__device__ __forceinline__ void add_chunk(uint4 &v, const uint32_t *r, float) {
    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) + __uint_as_float(r[i]));
}

template <typename T, uint32_t kBlocks>
__global__ void __launch_bounds__(kExpandThreads) expand_kernel(const __grid_constant__ ExpandParams P) {
    using E = Expand<T, kBlocks>;
    constexpr uint32_t WS = E::w_stages, IS = E::io_stages;
    extern __shared__ uint8_t raw[];
    __shared__ TileAdapters tile;
    __shared__ __align__(8) uint64_t s_h, s_w[WS], s_wfree[WS], s_d[2], s_dfree[2], s_io[IS], s_iodone[IS];
    __shared__ uint32_t s_tmem;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t h_at = smem_addr(smem), w_at = h_at + E::h_bytes, io_at = w_at + WS * E::w_bytes;
    uint8_t *io = smem + E::h_bytes + WS * E::w_bytes;
    const uint32_t rp = P.rank_pad;
    const uint64_t t0 = uint64_t(blockIdx.x / P.groups) * kTile;
    const uint32_t group = blockIdx.x % P.groups, col_tiles = (P.len + E::cols - 1) / E::cols;
    const uint32_t c0 = uint32_t(uint64_t(col_tiles) * group / P.groups), tiles = uint32_t(uint64_t(col_tiles) * (group + 1) / P.groups) - c0;
    if (warp == 0) tmem_alloc(smem_addr(&s_tmem), 256);
    if (tid == 0) {
        mbar_init(smem_addr(&s_h), 1);
        for (uint32_t i = 0; i < WS; ++i) {
            mbar_init(smem_addr(&s_w[i]), 1);
            mbar_init(smem_addr(&s_wfree[i]), 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&s_d[i]), 1);
            mbar_init(smem_addr(&s_dfree[i]), kThreads / 32);
        }
        for (uint32_t i = 0; i < IS; ++i) {
            mbar_init(smem_addr(&s_io[i]), 1);
            mbar_init(smem_addr(&s_iodone[i]), kThreads / 32);
        }
    }
    // the rank's padding in the stages of W, which no copy writes
    for (uint32_t i = tid; i < WS * (E::cols / 64) * (rp - P.rank) * 8; i += kExpandThreads) {
        const uint32_t c = i % 8, j = P.rank + i / 8 % (rp - P.rank), block = i / 8 / (rp - P.rank);
        *reinterpret_cast<uint4 *>(smem + E::h_bytes + block * E::w_block + j * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async_shared();
    grid_dep_wait();
    grid_dep_launch();                        // (the outer products need the shrink only, which is done)
    const uint32_t count = tile_adapters(tile, P.ids, t0, P.n, P.n_adapters, nullptr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem, steps = tiles * count;
    bool ok = true;
    if (warp == kThreads / 32) {
        if (lane == 0 && steps) {
            mbar_expect(smem_addr(&s_h), E::h_bytes);
            for (uint32_t q = 0; q < E::parts; ++q)
                for (uint32_t b = 0; b < kBlocks; ++b) tma_load(h_at + (q * kBlocks + b) * kTileBytes, &P.h, int32_t(b * 64), int32_t(q * P.n + t0), smem_addr(&s_h));
            // (descriptors and places kept up to date, not worked out: one thread issues for all)
            constexpr uint32_t desc = mma_desc(kTile, E::cols, 0, 1);
            const uint64_t h0 = tile_desc(h_at, 16, 1024), w0 = tile_desc(w_at, E::w_block, 1024);
            const uint32_t subs = rp / 16;
            uint32_t stage = 0, round = 0;    // of W: s % WS and s / WS & 1
            ok = mbar_wait(smem_addr(&s_h), 0);
            for (uint32_t s = 0; s < steps && ok; ++s) {
                ok = mbar_wait(smem_addr(&s_w[stage]), round);
                if (s >= 2 && ok) ok = mbar_wait(smem_addr(&s_dfree[s & 1]), (s / 2 - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t w = w0 + stage * (E::w_bytes >> 4);
                const uint32_t d = tmem + (s & 1) * 128;
#pragma unroll
                for (uint32_t q = 0; q < E::parts; ++q)
#pragma unroll
                    for (uint32_t k = 0; k < 4 * kBlocks; ++k)
                        if (k < subs) mma(d, h0 + (((q * kBlocks + k / 4) * kTileBytes) >> 4) + 2 * (k % 4), w + k * 128, desc, q || k);
                mma_commit(smem_addr(&s_wfree[stage]));
                mma_commit(smem_addr(&s_d[s & 1]));
                if (++stage == WS) stage = 0, round ^= 1u;
            }
            if (!ok) mbar_wait(smem_addr(&s_h), 0);   // (a copy in flight lands before the CTA ends)
        }
    } else if (warp == kThreads / 32 + 2) {
        if (lane == 0) {
            // W of a step: blocks of 64 columns, each the adapter's rank rows
            uint32_t stage = 0, round = 1, s = 0;      // (the first round's stages are free)
            for (uint32_t i = 0; i < tiles && ok; ++i)
                for (uint32_t a = 0; a < count && ok; ++a, ++s) {
                    const uint32_t bar = smem_addr(&s_w[stage]), at = w_at + stage * E::w_bytes;
                    if (s >= WS) ok = mbar_wait(smem_addr(&s_wfree[stage]), round);
                    if (!ok) break;
                    mbar_expect(bar, E::cols / 64 * P.rank * 128);
#pragma unroll
                    for (uint32_t b = 0; b < E::cols / 64; ++b) tma_load(at + b * E::w_block, &P.w, int32_t((c0 + i) * E::cols + b * 64), tile.list[a] * int32_t(P.rank), bar);
                    if (++stage == WS) stage = 0, round ^= 1u;
                }
            // the last copies land before the CTA ends, whichever thread's wait may have given up
            for (uint32_t k = 0; k < min(s, WS); ++k) {
                stage = stage ? stage - 1 : WS - 1;
                mbar_wait(smem_addr(&s_w[stage]), (s - 1 - k) / WS & 1);
            }
        }
    } else if (warp == kThreads / 32 + 1) {
        if (lane == 0) {
            auto load = [&](uint32_t i) {
                const uint32_t bar = smem_addr(&s_io[i % IS]);
                mbar_expect(bar, P.has_base ? E::io_bytes : 0);
                if (P.has_base)
                    for (uint32_t b = 0; b < 2; ++b) tma_load(io_at + i % IS * E::io_bytes + b * kTileBytes, &P.base, int32_t((c0 + i) * E::cols + b * E::row), int32_t(t0), bar);
            };
            uint32_t loaded = min(IS, tiles);
            for (uint32_t i = 0; i < loaded; ++i) load(i);
            for (uint32_t i = 0; i < tiles && ok; ++i) {
                ok = mbar_wait(smem_addr(&s_iodone[i % IS]), i / IS & 1);
                if (!ok) break;
                for (uint32_t b = 0; b < 2; ++b)
                    if ((c0 + i) * E::cols + b * E::row < P.len) tma_store(&P.y, int32_t((c0 + i) * E::cols + b * E::row), int32_t(t0), io_at + i % IS * E::io_bytes + b * kTileBytes);
                bulk_commit();
                if (i + IS < tiles) {
                    bulk_wait_read<0>();
                    load(loaded++);
                }
            }
            bulk_wait_all();
            for (uint32_t i = loaded > IS ? loaded - IS : 0; i < loaded; ++i) mbar_wait(smem_addr(&s_io[i % IS]), i / IS & 1);
        }
    } else {
        // this thread: token warp % 4 * 32 + lane, the tile's columns of row block warp / 4
        const uint32_t t = warp % 4 * 32 + lane;
        const int32_t mine = tile.of[t];
        constexpr uint32_t kPer = 16 / sizeof(T);              // columns of a 16-byte chunk
        for (uint32_t i = 0; i < tiles; ++i) {
            if (ok) ok = mbar_wait(smem_addr(&s_io[i % IS]), i / IS & 1);
            uint8_t *rows = io + i % IS * E::io_bytes + warp / 4 * kTileBytes;
            if (!P.has_base && mine < 0)
#pragma unroll
                for (uint32_t c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(rows + tile_at(t, c)) = make_uint4(0, 0, 0, 0);
            for (uint32_t a = 0; a < count; ++a) {
                const uint32_t s = i * count + a;
                if (ok) ok = mbar_wait(smem_addr(&s_d[s & 1]), s / 2 & 1);
                tc_fence_after();
                if (__any_sync(0xffffffffu, mine == int32_t(a))) {
#pragma unroll
                    for (uint32_t piece = 0; piece < E::row / 32; ++piece) {
                        // (the base's chunks are fetched while the product comes from TMEM)
                        uint32_t r[32];
                        tmem_load32(tmem + ((warp % 4) << 21) + (s & 1) * 128 + warp / 4 * E::row + piece * 32, r);
                        uint4 b[32 / kPer];
#pragma unroll
                        for (uint32_t c = 0; c < 32 / kPer; ++c)
                            b[c] = P.has_base ? *reinterpret_cast<const uint4 *>(rows + tile_at(t, piece * (32 / kPer) + c)) : make_uint4(0, 0, 0, 0);
                        tmem_wait32(r);
                        if (mine == int32_t(a))
#pragma unroll
                            for (uint32_t c = 0; c < 32 / kPer; ++c) {
                                add_chunk(b[c], r + c * kPer, T());
                                *reinterpret_cast<uint4 *>(rows + tile_at(t, piece * (32 / kPer) + c)) = b[c];
                            }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&s_dfree[s & 1]));
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&s_iodone[i % IS]));
        }
    }
    if (!ok) atomicOr(P.status, K3HUF_ST_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free(tmem, 256);
}

struct OuterJob {
    const __nv_bfloat16 *h, *v;               // parts x tokens x pitch; the rows that it multiplies
    float *g;
    uint64_t stride;
    uint32_t len;
};
struct OuterParams {
    OuterJob job[2];
    const int32_t *ids;
    uint32_t *status;
    uint64_t n;
    uint32_t n_adapters, rank, rank_pad, pitch, col_tiles0;        // column tiles of job 0
    bool add, beside;                         // add to g; launched beside an expand (see the kernel's first wait)
};

// The outer product.  D[128 columns, rank] = V^T H over the tokens of one
// adapter, 64 of them per step, gathered by their indexes: both operands lie
// token by token, so both are read MN-major.  CTAs: a tile of columns (of
// either gradient) x an adapter; the tokens' indexes come from the ids,
// kWindow at a time, in order.  Bound by the read of V, in pieces of 256 bytes:
// 46 us for 4096 tokens x 32 x (8192 + 8192) of 4 adapters, 2.9 TB/s.
//
// Ranks up to 32 (kBlocks 0) stage the parts side by side and multiply them at
// once into columns of their own, which takes a third of the products and
// leaves room for a third stage; above, a part is kBlocks blocks of 64 rank rows
// and the parts add up in the same columns.
constexpr uint32_t kWindow = 2048;
template <uint32_t kBlocks> struct Outer {
    static constexpr uint32_t stages = kBlocks == 0 ? 3 : 2, h_bytes = (kBlocks == 0 ? 2 : kMaxParts * kBlocks) * kStep * 128;
    static constexpr uint32_t stage = kStep * 256 + h_bytes, half = kBlocks == 0 ? 128 : kBlocks * 64;      // (half: columns of TMEM)
    static constexpr uint32_t run = kChain / (kBlocks == 0 ? kStep / 16 : kMaxParts * kStep / 16);
    static constexpr uint32_t pieces = kBlocks == 0 ? 1 : 2 * kBlocks;      // of 16 columns per thread
    static constexpr size_t smem = stages * stage + 1024;
};

template <uint32_t kBlocks>
__global__ void __launch_bounds__(kThreads) outer_kernel(const __grid_constant__ OuterParams P) {
    using O = Outer<kBlocks>;
    constexpr uint32_t kStage = O::stage, kOuterStages = O::stages;
    extern __shared__ uint8_t raw[];
    __shared__ uint32_t s_token[kWindow], s_count[kThreads / 32 + 1], s_tmem;
    __shared__ __align__(8) uint64_t s_bar[kOuterStages];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32, base = smem_addr(smem), rp = P.rank_pad;
    const bool second = blockIdx.x >= P.col_tiles0;
    const OuterJob &J = P.job[second];
    const uint32_t col = (blockIdx.x - (second ? P.col_tiles0 : 0)) * 128;
    if (warp == 0) tmem_alloc(smem_addr(&s_tmem), 2 * O::half);
    if (tid == 0)
        for (uint32_t i = 0; i < kOuterStages; ++i) mbar_init(smem_addr(&s_bar[i]), 1);
    if (tid == 0) fence_async_shared();
    // Behind an expand this kernel's CTAs start once all of that one's have seen the shrink end, so
    // nothing that they read is still being written; they wait for the expand at their end
    if (!P.beside) grid_dep_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem, desc = mma_desc(128, kBlocks == 0 ? kMaxParts * rp : rp, 1, 1);
    bool ok = true;
    uint32_t step = 0;                        // steps of this CTA so far: their stages and phases follow
    for (uint32_t a = blockIdx.y; a < P.n_adapters; a += gridDim.y) {
        const uint32_t first = step;
        // this thread's sums: column (lane) warp % 4 * 32 + lane, rank rows warp / 4 * 16 + 32 b on
        constexpr uint32_t kRun = O::run;
        float sum[O::pieces][16] = {};
        auto drain = [&](uint32_t run) {
            tc_fence_after();
#pragma unroll
            for (uint32_t b = 0; b < O::pieces; ++b)
#pragma unroll
                for (uint32_t q = 0; q < (kBlocks == 0 ? kMaxParts : 1); ++q)
                    if (warp / 4 * 16 + b * 32 < rp) {
                        float v[16];
                        tmem_load16(tmem + ((warp % 4) << 21) + (run & 1) * O::half + q * rp + warp / 4 * 16 + b * 32, v);
#pragma unroll
                        for (int k = 0; k < 16; ++k) sum[b][k] += v[k];
                    }
            tc_fence_before();
        };
        for (uint64_t w0 = 0; w0 < P.n; w0 += kWindow) {
            // the window's tokens of this adapter, in order
            const uint32_t size = uint32_t(min(uint64_t(kWindow), P.n - w0));
            constexpr uint32_t kMine = kWindow / kThreads;
            uint32_t mine = 0;
#pragma unroll
            for (uint32_t k = 0; k < kMine; ++k) {
                const uint32_t t = tid * kMine + k;
                if (t < size && P.ids[w0 + t] == int32_t(a)) mine |= 1u << k;
            }
            uint32_t at = __popc(mine);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, at, d);
                if (lane >= uint32_t(d)) at += v;
            }
            __syncthreads();                  // (the last window's list has been read)
            if (lane == 31) s_count[warp] = at;
            __syncthreads();
            uint32_t total = 0;
            at -= __popc(mine);
            for (uint32_t w = 0; w < kThreads / 32; ++w) {
                if (w < warp) at += s_count[w];
                total += s_count[w];
            }
            for (uint32_t k = 0; k < kMine; ++k)
                if (mine >> k & 1) s_token[at++] = tid * kMine + k;
            __syncthreads();
            const uint32_t steps = (total + kStep - 1) / kStep;
            auto load = [&](uint32_t s) {
                // chunk tid % 16 of rows tid / 16 + 16 m: of the rows' 128 columns, and, where
                // there is one, of each part's rank rows
                const uint32_t to = base + (step + s) % kOuterStages * kStage, c = tid % 16;
                const bool v_in = col + c * 8 < J.len, h_in = c * 8 < rp;
#pragma unroll
                for (uint32_t m = 0; m < 4; ++m) {
                    const uint32_t r = tid / 16 + 16 * m, k = s * kStep + r, at = c / 8 * (kStep * 128) + tile_at(r, c % 8);
                    const uint64_t t = w0 + (k < total ? s_token[k] : 0u);
                    const bool in = k < total;
                    cp_async16z(to + at, in && v_in ? J.v + t * J.stride + col + c * 8 : J.v, in && v_in ? 16 : 0);
                    if (h_in) {
                        const __nv_bfloat16 *src = J.h + t * P.pitch + c * 8;
#pragma unroll
                        for (uint32_t q = 0; q < kMaxParts; ++q) {
                            const uint32_t hc = kBlocks == 0 ? q * (rp / 8) + c : c;
                            cp_async16z(to + kStep * 256 + q * (kBlocks * kStep * 128) + hc / 8 * (kStep * 128) + tile_at(r, hc % 8), src + q * P.n * P.pitch, in ? 16 : 0);
                        }
                    }
                }
            };
            for (uint32_t s = 0; s < kOuterStages - 1; ++s) {
                if (s < steps) load(s);
                cp_async_commit();
            }
            for (uint32_t s = 0; s < steps; ++s) {
                const uint32_t g = step + s;
                // the stage before this one is free once its products are done
                if (s > 0 && ok) ok = mbar_wait(smem_addr(&s_bar[(g - 1) % kOuterStages]), (g - 1) / kOuterStages & 1);
                if (s + kOuterStages - 1 < steps && ok) load(s + kOuterStages - 1);
                cp_async_commit();
                cp_async_wait<kOuterStages - 1>();
                fence_async_shared();
                __syncthreads();
                if (tid == 0 && ok) {
                    tc_fence_after();
                    const uint32_t at = base + g % kOuterStages * kStage, d = tmem + ((g - first) / kRun & 1) * O::half;
                    const uint64_t va = tile_desc(at, kStep * 128, 1024);
#pragma unroll
                    for (uint32_t q = 0; q < (kBlocks == 0 ? 1 : kMaxParts); ++q) {
                        const uint64_t hb = tile_desc(at + kStep * 256 + q * kBlocks * (kStep * 128), kStep * 128, 1024);
#pragma unroll
                        for (uint32_t k = 0; k < kStep / 16; ++k) mma(d, va + k * 128, hb + k * 128, desc, (g - first) % kRun || q || k);
                    }
                    mma_commit(smem_addr(&s_bar[g % kOuterStages]));
                }
                // the run before is done: its last step was waited for above, or with its window
                if (g != first && (g - first) % kRun == 0) drain((g - first) / kRun - 1);
            }
            if (steps && ok) ok = mbar_wait(smem_addr(&s_bar[(step + steps - 1) % kOuterStages]), (step + steps - 1) / kOuterStages & 1);
            cp_async_wait<0>();
            step += steps;
        }
        if (step != first) drain((step - first - 1) / kRun);
        // lane: column; a warp's stores of one rank row are 128 adjacent bytes.  (Added to: adapters
        // without a token are left alone, another call may be adding to them)
        const uint32_t c = col + warp % 4 * 32 + lane;
        const bool alone = P.add && step == first;
        if (c < J.len && !alone)
#pragma unroll
            for (uint32_t b = 0; b < O::pieces; ++b)
#pragma unroll
                for (uint32_t k = 0; k < 16; ++k) {
                    const uint32_t j = warp / 4 * 16 + b * 32 + k;
                    if (j >= P.rank) break;
                    float *o = J.g + (uint64_t(a) * P.rank + j) * J.len + c;
                    *o = P.add ? *o + sum[b][k] : sum[b][k];
                }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (!ok) atomicOr(P.status, K3HUF_ST_TIMEOUT);
    if (P.beside) grid_dep_wait();
    if (warp == 0) tmem_free(tmem, 2 * O::half);
}

// --- host -----------------------------------------------------------------------

bool adapters_ok(const k3huf_adapters_t *ad, uint64_t n) {
    return ad && ad->a && ad->b && ad->scales && ad->n_adapters && uint64_t(ad->n_adapters) * ad->rank < (1ull << 31) && ad->rank && ad->rank <= K3HUF_MAX_RANK &&
           ad->cols && ad->rows && ad->cols < (1ull << 31) && ad->rows < (1ull << 31) && n < (1ull << 29) && aligned_to(ad->a, 2) &&
           aligned_to(ad->b, 2) && aligned_to(ad->scales, 4);
}

uint32_t padded(uint32_t rank) { return (rank + 15) / 16 * 16; }
// A rank-wide intermediate: fp32, or three bf16 parts in blocks of 64 values.
uint32_t h_pitch(uint32_t rank) { return (rank + 63) / 64 * 64; }
uint64_t h_bytes(uint64_t n, uint32_t rank) { return align_up(n * 2 * kMaxParts * h_pitch(rank), 256); }

enum class Form { any, few, many };
bool rows16(const void *p, uint64_t stride, uint32_t type) { return aligned_to(p, 16) && stride * elem_bytes(type) % 16 == 0; }
// Few tokens: each reads its factor rows on its own, at about 10 TB/s from L2.
// Per call, few and many, fp32 or bf16 results: 128 tokens x 32 x (8192 + 8192)
// of 32 adapters, 134 MB, 19 us and 50 or 48; 256 x 64 x (4096 + 4096) of 8, 268
// MB, 27 us both; 250 x 32 x (8192 + 8192) of 64, 262 MB, 42 or 39 and 115 or 72;
// 1000 x 32 x (4096 + 4096) of 32, 524 MB, 48 and 48 or 34; 2000 x 16 x (8192 +
// 8192) of 8, 1 GB, 118 or 113 and 60 or 39.
// (A grid's second dimension takes 65535 blocks: more rows than that many blocks of
// kFewCols run as many tokens.)
Form run_form(uint64_t n, const k3huf_adapters_t *ad, bool rows_ok) {
    const bool few = n <= 65535 && n * ad->rank * (ad->cols + ad->rows) * 2 <= kFewBytes && (ad->rows + kFewCols - 1) / kFewCols <= 65535;
    return !rows_ok ? Form::any : few ? Form::few : Form::many;
}

// A launch that may begin while the kernel before it ends (its blocks wait for that one themselves).
template <typename... Args, typename... Given>
int launch_after(void (*kernel)(Args...), dim3 grid, uint32_t threads, size_t smem, cudaStream_t stream, Given... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_rc(cudaLaunchKernelEx(&cfg, kernel, Args(args)...));
}

int shrink_job(ShrinkParams &P, uint32_t j, const void *v, uint64_t stride, const void *w, uint64_t len, __nv_bfloat16 *h) {
    P.job[j].len = uint32_t(len);
    P.job[j].h = h;
    const int rc = tensor_map(&P.job[j].v, v, K3HUF_BF16, P.n, len, stride, kTile, kStep, true);
    return rc ? rc : tensor_map(&P.job[j].w, w, K3HUF_BF16, uint64_t(P.n_adapters) * P.rank, len, len, P.rank, kStep, true);
}

int launch_shrink(ShrinkParams &P, uint32_t jobs, uint64_t sms, cudaStream_t stream) {
    static std::atomic<uint64_t> once{0};
    const int rc = once_per_device(once, [] { return cudaFuncSetAttribute(shrink_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kShrinkSmem)); });
    if (rc) return rc;
    const uint64_t tiles = (P.n + kTile - 1) / kTile;
    const uint32_t per = kTile / P.rank_pad, most = std::min<uint32_t>(P.n_adapters, uint32_t(std::min<uint64_t>(kTile, P.n)));
    const uint32_t groups = (most + per - 1) / per;
    // splits of the contraction: two CTAs per SM, counting one group per tile (the usual case),
    // and four steps or more for each
    const uint32_t steps = (std::max(P.job[0].len, jobs > 1 ? P.job[1].len : 0u) + kStep - 1) / kStep;
    P.splits = 1;
    while (P.splits < kMaxSplits && tiles * jobs * P.splits * 2 <= 2 * sms && steps >= 8 * P.splits) P.splits *= 2;
    cudaLaunchConfig_t cfg = {};
    // clusters per tile: as many as its groups may be, but no more than fill the GPU
    const uint64_t clusters = tiles * P.splits * jobs;
    cfg.gridDim = dim3(uint32_t(tiles * P.splits), std::min<uint32_t>(groups, uint32_t((2 * sms + clusters - 1) / clusters)), jobs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kShrinkSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = P.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_rc(cudaLaunchKernelEx(&cfg, shrink_kernel, P));
}

template <typename T, uint32_t kBlocks>
int launch_expand(ExpandParams &P, const void *h, const void *w, const void *base, uint64_t base_stride, void *y, uint64_t y_stride, uint64_t sms, cudaStream_t stream) {
    using E = Expand<T, kBlocks>;
    static std::atomic<uint64_t> once{0};
    int rc = once_per_device(once, [] { return cudaFuncSetAttribute(expand_kernel<T, kBlocks>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(E::smem)); });
    if (rc) return rc;
    constexpr uint32_t type = sizeof(T) == 4 ? K3HUF_F32 : K3HUF_BF16;
    rc = tensor_map(&P.h, h, K3HUF_BF16, E::parts * P.n, kBlocks * 64, kBlocks * 64, kTile, 64, true);
    if (!rc) rc = tensor_map(&P.w, w, K3HUF_BF16, uint64_t(P.n_adapters) * P.rank, P.len, P.len, P.rank, 64, true);
    if (!rc) rc = tensor_map(&P.y, y, type, P.n, P.len, y_stride, kTile, E::row, true);
    if (!rc) rc = base ? tensor_map(&P.base, base, type, P.n, P.len, base_stride, kTile, E::row, true) : K3HUF_OK;
    if (rc) return rc;
    P.has_base = base != nullptr;
    const uint64_t tiles = (P.n + kTile - 1) / kTile, cols = (P.len + E::cols - 1) / E::cols;
    // column ranges per token tile: the count whose last wave of CTAs (one per SM) is fullest,
    // among those that give an SM up to three waves
    uint64_t best = 1;
    double waste = 1e30;
    for (uint64_t g = 1; g <= cols && g <= std::max<uint64_t>(1, 3 * sms / tiles); ++g) {
        const uint64_t waves = (tiles * g + sms - 1) / sms, per = (cols + g - 1) / g;
        const double cost = double(waves * (per + 2));     // (a CTA's start costs about two column tiles)
        if (cost < waste) waste = cost, best = g;
    }
    P.groups = uint32_t(best);
    return launch_after(expand_kernel<T, kBlocks>, dim3(uint32_t(tiles * best)), kExpandThreads, E::smem, stream, P);
}
int launch_expand(ExpandParams &P, const void *h, const void *w, const void *base, uint64_t base_stride, void *y, uint64_t y_stride, uint32_t type, uint64_t sms, cudaStream_t stream) {
    if (P.rank_pad <= kStep)
        return type == K3HUF_BF16 ? launch_expand<__nv_bfloat16, 1>(P, h, w, base, base_stride, y, y_stride, sms, stream)
                                  : launch_expand<float, 1>(P, h, w, base, base_stride, y, y_stride, sms, stream);
    return type == K3HUF_BF16 ? launch_expand<__nv_bfloat16, 2>(P, h, w, base, base_stride, y, y_stride, sms, stream)
                              : launch_expand<float, 2>(P, h, w, base, base_stride, y, y_stride, sms, stream);
}

int launch_outer(const OuterParams &P, uint32_t col_tiles, cudaStream_t stream) {
    static std::atomic<uint64_t> once{0};
    const int rc = once_per_device(once, [] {
        cudaError_t e = cudaFuncSetAttribute(outer_kernel<0>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Outer<0>::smem));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(outer_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Outer<1>::smem));
        return e != cudaSuccess ? e : cudaFuncSetAttribute(outer_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Outer<2>::smem));
    });
    if (rc) return rc;
    const dim3 grid(col_tiles, std::min(P.n_adapters, 65535u));
    if (P.rank_pad <= 32) return launch_after(outer_kernel<0>, grid, kThreads, Outer<0>::smem, stream, P);
    return P.rank_pad <= kStep ? launch_after(outer_kernel<1>, grid, kThreads, Outer<1>::smem, stream, P)
                               : launch_after(outer_kernel<2>, grid, kThreads, Outer<2>::smem, stream, P);
}

}  // namespace
}  // namespace k3huf

using namespace k3huf;

extern "C" int k3huf_adapter_scratch_bytes(uint64_t n_tokens, uint32_t n_adapters, uint32_t rank, uint64_t cols, uint64_t rows, int grad, size_t *scratch_bytes) {
    if (!scratch_bytes || n_adapters == 0 || rank == 0 || rank > K3HUF_MAX_RANK || cols == 0 || rows == 0 || n_tokens >= (1ull << 29)) return K3HUF_E_ARG;
    *scratch_bytes = 256 + h_bytes(n_tokens, rank) * (grad ? 2 : 1);
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
    const uint32_t n = uint32_t(n_tokens), S = ad->n_adapters, r = ad->rank;
    const auto *a = static_cast<const __nv_bfloat16 *>(ad->a), *b = static_cast<const __nv_bfloat16 *>(ad->b), *x = static_cast<const __nv_bfloat16 *>(d_x);
    const bool rows_ok = rows16(a, ad->cols, K3HUF_BF16) && rows16(b, ad->rows, K3HUF_BF16) && rows16(x, x_stride, K3HUF_BF16) &&
                         rows16(d_y, y_stride, y_type) && (!d_base || rows16(d_base, base_stride, y_type));
    switch (run_form(n, ad, rows_ok)) {
        case Form::any: {
            float *h = static_cast<float *>(d_scratch);
            shrink_any_kernel<<<n, kThreads, 0, st>>>(x, x_stride, a, ad->scales, d_ids, S, r, ad->cols, h, d_status);
            if (y_type == K3HUF_BF16)
                expand_any_kernel<<<n, kThreads, 0, st>>>(h, b, d_ids, S, r, ad->rows, static_cast<const __nv_bfloat16 *>(d_base), base_stride, static_cast<__nv_bfloat16 *>(d_y), y_stride);
            else
                expand_any_kernel<<<n, kThreads, 0, st>>>(h, b, d_ids, S, r, ad->rows, static_cast<const float *>(d_base), base_stride, static_cast<float *>(d_y), y_stride);
            return cuda_rc(cudaGetLastError());
        }
        case Form::few: {
            float *h = static_cast<float *>(d_scratch);
            shrink_few_kernel<<<dim3(n, (r + kRows - 1) / kRows), kThreads, 0, st>>>(x, x_stride, a, ad->scales, d_ids, S, r, uint32_t(ad->cols), h, d_status);
            const int rc = cuda_rc(cudaGetLastError());
            if (rc) return rc;
            const dim3 grid(n, uint32_t((ad->rows + kFewCols - 1) / kFewCols));
            if (y_type == K3HUF_BF16)
                return launch_after(expand_few_kernel<__nv_bfloat16>, grid, kFewCols / 4, 0, st, h, b, d_ids, S, r, uint32_t(ad->rows), static_cast<const __nv_bfloat16 *>(d_base), base_stride, static_cast<__nv_bfloat16 *>(d_y), y_stride);
            return launch_after(expand_few_kernel<float>, grid, kFewCols / 4, 0, st, h, b, d_ids, S, r, uint32_t(ad->rows), static_cast<const float *>(d_base), base_stride, static_cast<float *>(d_y), y_stride);
        }
        case Form::many: break;
    }
    uint64_t sms = 0;
    int rc = sm_count(&sms);
    if (rc) return rc;
    auto *h = static_cast<__nv_bfloat16 *>(d_scratch);
    ShrinkParams sp{};
    sp.scales = ad->scales, sp.ids = d_ids, sp.status = d_status, sp.n = n;
    sp.n_adapters = S, sp.rank = r, sp.rank_pad = padded(r), sp.pitch = h_pitch(r), sp.parts = y_type == K3HUF_F32 ? 3 : 2;
    rc = shrink_job(sp, 0, x, x_stride, a, ad->cols, h);
    if (!rc) rc = launch_shrink(sp, 1, sms, st);
    if (rc) return rc;
    ExpandParams ep{};
    ep.ids = d_ids, ep.status = d_status, ep.n = n, ep.n_adapters = S, ep.rank = r, ep.rank_pad = padded(r), ep.len = uint32_t(ad->rows);
    return launch_expand(ep, h, b, d_base, base_stride, d_y, y_stride, y_type, sms, st);
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
    const uint32_t n = uint32_t(n_tokens), S = ad->n_adapters, r = ad->rank;
    const auto *a = static_cast<const __nv_bfloat16 *>(ad->a), *b = static_cast<const __nv_bfloat16 *>(ad->b);
    const auto *x = static_cast<const __nv_bfloat16 *>(d_x), *dy = static_cast<const __nv_bfloat16 *>(d_dy);
    uint8_t *h0 = static_cast<uint8_t *>(d_scratch), *h1 = h0 + h_bytes(n, r);
    const bool add = (flags & K3HUF_ACCUMULATE) != 0;
    const bool rows_ok = rows16(a, ad->cols, K3HUF_BF16) && rows16(b, ad->rows, K3HUF_BF16) && rows16(x, x_stride, K3HUF_BF16) && rows16(dy, dy_stride, K3HUF_BF16) &&
                         (!d_dx || rows16(d_dx, dx_stride, dx_type)) && (!d_dx_base || rows16(d_dx_base, dx_base_stride, dx_type));
    if (!rows_ok || n == 0) {
        float *h = reinterpret_cast<float *>(h0), *dh = reinterpret_cast<float *>(h1);
        if (n) {
            shrink_any_kernel<<<n, kThreads, 0, st>>>(x, x_stride, a, ad->scales, d_ids, S, r, ad->cols, h, d_status);
            shrink_any_kernel<<<n, kThreads, 0, st>>>(dy, dy_stride, b, ad->scales, d_ids, S, r, ad->rows, dh, d_status);
            if (d_dx && dx_type == K3HUF_BF16)
                expand_any_kernel<<<n, kThreads, 0, st>>>(dh, a, d_ids, S, r, ad->cols, static_cast<const __nv_bfloat16 *>(d_dx_base), dx_base_stride, static_cast<__nv_bfloat16 *>(d_dx), dx_stride);
            else if (d_dx)
                expand_any_kernel<<<n, kThreads, 0, st>>>(dh, a, d_ids, S, r, ad->cols, static_cast<const float *>(d_dx_base), dx_base_stride, static_cast<float *>(d_dx), dx_stride);
        }
        outer_any_kernel<<<dim3(uint32_t((ad->cols + kThreads - 1) / kThreads), std::min(S * r, 65535u)), kThreads, 0, st>>>(dh, x, x_stride, d_ids, n, S, r, ad->cols, d_da, add);
        outer_any_kernel<<<dim3(uint32_t((ad->rows + kThreads - 1) / kThreads), std::min(S * r, 65535u)), kThreads, 0, st>>>(h, dy, dy_stride, d_ids, n, S, r, ad->rows, d_db, add);
        return cuda_rc(cudaGetLastError());
    }
    uint64_t sms = 0;
    int rc = sm_count(&sms);
    if (rc) return rc;
    auto *h = reinterpret_cast<__nv_bfloat16 *>(h0), *dh = reinterpret_cast<__nv_bfloat16 *>(h1);
    ShrinkParams sp{};
    sp.scales = ad->scales, sp.ids = d_ids, sp.status = d_status, sp.n = n;
    sp.n_adapters = S, sp.rank = r, sp.rank_pad = padded(r), sp.pitch = h_pitch(r), sp.parts = kMaxParts;
    rc = shrink_job(sp, 0, x, x_stride, a, ad->cols, h);
    if (!rc) rc = shrink_job(sp, 1, dy, dy_stride, b, ad->rows, dh);
    if (!rc) rc = launch_shrink(sp, 2, sms, st);
    if (rc) return rc;
    if (d_dx) {
        ExpandParams ep{};
        ep.ids = d_ids, ep.status = d_status, ep.n = n, ep.n_adapters = S, ep.rank = r, ep.rank_pad = padded(r), ep.len = uint32_t(ad->cols);
        rc = launch_expand(ep, dh, a, d_dx_base, dx_base_stride, d_dx, dx_stride, dx_type, sms, st);
        if (rc) return rc;
    }
    const uint32_t tiles_a = uint32_t((ad->cols + 127) / 128), tiles_b = uint32_t((ad->rows + 127) / 128);
    const OuterParams op{{{dh, x, d_da, x_stride, uint32_t(ad->cols)}, {h, dy, d_db, dy_stride, uint32_t(ad->rows)}}, d_ids, d_status, n, S, r, padded(r), h_pitch(r), tiles_a, add, d_dx != nullptr};
    return launch_outer(op, tiles_a + tiles_b, st);
}
