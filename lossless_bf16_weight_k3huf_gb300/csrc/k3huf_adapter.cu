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
//  - few tokens (tokens x rank up to kFewWork): fp32 arithmetic, a CTA per
//    token and part of the factor; every factor row is read once per token,
//    mostly from L2;
//  - many: tcgen05.mma on tiles of 128 tokens, described at each kernel;
//  - rows that do not start on 16 bytes: one CTA per token, element by element.
// The rank-wide intermediates are fp32 sums.  The tensor cores take them as a
// sum of bf16 parts: three parts (24 bits) where the result is fp32, two (16
// bits) where it is rounded to bf16.
#include <algorithm>

#include "k3huf_tc.h"

namespace k3huf {
namespace {

constexpr int kThreads = 256;
constexpr uint64_t kFewWork = 4096;           // tokens x rank

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
        st_f32(y + t * y_stride + c, base ? ld_f32(base + t * base_stride + c) + acc : acc);
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
        for (uint64_t t = 0; t < n; ++t)
            if (ids[t] == int32_t(i)) acc = fmaf(h[t * rank + r], ld_f32(v + t * stride + c), acc);
        float *out = g + row * len + c;
        *out = add ? *out + acc : acc;
    }
}

// --- few tokens ---------------------------------------------------------------

constexpr int kRows = 4;                      // factor rows per CTA

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

// y[t] = base[t] + sum_r h[t, r] w[i, r]: one CTA per token and 512 columns,
// four per thread.
template <typename T>
__global__ void __launch_bounds__(128)
expand_few_kernel(const float *h, const __nv_bfloat16 *w, const int32_t *ids, uint32_t n_adapters, uint32_t rank, uint32_t len, const T *base, uint64_t base_stride, T *y, uint64_t y_stride) {
    __shared__ float s_h[K3HUF_MAX_RANK];
    const uint64_t t = blockIdx.x;
    const uint32_t c = blockIdx.y * 512 + threadIdx.x * 4;
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
    for (int k = 0; k < 4; ++k) acc[k] += sum[k];
    store4(y + t * y_stride + c, acc);
}

// --- many tokens: tensor cores --------------------------------------------------

constexpr uint32_t kTile = 128;               // tokens per tile
constexpr uint32_t kStep = 64;                // contraction per staged step: one 128-byte row
constexpr uint32_t kTileBytes = kTile * 128;  // one staged tile of 128 rows
// Additions in the tensor core before a sum moves to registers.  One of them
// errs by about 1.3e-8 of the sum, always to the same side (measured: 2e-5 after
// 1536), while fp32 additions in registers round to nearest.
constexpr uint32_t kChain = 32;

// The adapters of a tile's tokens, each once, in the order of their first
// token: of[t] the place of token t's adapter (-1: none), list the adapters.
// All threads of the CTA (at least 128) for `size` tokens; returns their number.
struct TileAdapters {
    int32_t id[kTile], list[kTile];
    int16_t of[kTile];
    uint32_t count[4];
};
__device__ uint32_t tile_adapters(TileAdapters &s, const int32_t *ids, uint64_t t0, uint64_t n, uint32_t size, uint32_t n_adapters, uint32_t *status) {
    const uint32_t t = threadIdx.x, lane = t % 32, warp = t / 32;
    int32_t id = -1;
    bool first = false;
    uint32_t below = 0;
    if (t < kTile) {
        if (t < size && t0 + t < n) id = ids[t0 + t];
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

// x as a sum of bf16 parts
__device__ __forceinline__ void parts_of(float x, __nv_bfloat16 (&p)[3]) {
    p[0] = __float2bfloat16_rn(x);
    const float a = x - __bfloat162float(p[0]);
    p[1] = __float2bfloat16_rn(a);
    p[2] = __float2bfloat16_rn(a - __bfloat162float(p[1]));
}

struct ShrinkJob {
    const __nv_bfloat16 *v, *w;
    uint64_t stride;
    uint32_t len;
    __nv_bfloat16 *h;                         // parts x tokens x rank_pad
};
struct ShrinkParams {
    ShrinkJob job[2];
    const float *scales;
    const int32_t *ids;
    uint32_t *status;
    uint64_t n;
    uint32_t n_adapters, rank, rank_pad, parts, splits;
};

// The shrink.  D[128 tokens, rank rows of the tile's adapters] = V W^T, both
// operands K-major, kStep of the contraction per stage; every token keeps the
// columns of its own adapter.  CTAs: a tile of tokens x a group of adapters
// whose rank rows fill 128 columns (all but the first few groups of a tile
// whose tokens share adapters end at once) x a split of the contraction; the
// splits are a cluster, whose partial sums meet through shared memory in the
// order of the splits.  Bound by the read of V (and of the factors when every
// token has its own).
constexpr uint32_t kShrinkStages = 3, kShrinkStage = 2 * kTileBytes;
constexpr size_t kShrinkSmem = kShrinkStages * kShrinkStage + 1024;
constexpr uint32_t kMaxSplits = 8;

__global__ void __launch_bounds__(kThreads) shrink_kernel(const __grid_constant__ ShrinkParams P) {
    extern __shared__ uint8_t raw[];
    __shared__ TileAdapters tile;
    __shared__ __align__(8) uint64_t s_bar[kShrinkStages];
    __shared__ uint32_t s_tmem;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32, base = smem_addr(smem);
    const ShrinkJob &J = P.job[blockIdx.z];
    const uint32_t split = blockIdx.x % P.splits, rp = P.rank_pad;
    const uint64_t t0 = uint64_t(blockIdx.x / P.splits) * kTile;
    grid_dep_launch();
    const uint32_t per = kTile / rp, count = tile_adapters(tile, P.ids, t0, P.n, kTile, P.n_adapters, split + blockIdx.y + blockIdx.z == 0 ? P.status : nullptr);
    const uint32_t a0 = blockIdx.y * per, na = a0 < count ? min(per, count - a0) : 0u;
    if (na == 0) return;                      // (the whole cluster)
    const uint32_t cols = na * rp;            // <= 128, a multiple of 16
    if (warp == 0) tmem_alloc(smem_addr(&s_tmem), 256);
    if (tid == 0)
        for (uint32_t i = 0; i < kShrinkStages; ++i) mbar_init(smem_addr(&s_bar[i]), 1);
    if (tid == 0) fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t steps = (J.len + kStep - 1) / kStep;
    const uint32_t k0 = steps * split / P.splits, k1 = steps * (split + 1) / P.splits;

    // this thread's part of a step: chunk tid % 8 of rows tid / 8 + 32 m of both operands, their
    // addresses worked out once (null: zeros)
    const uint32_t chunk = tid % 8;
    const __nv_bfloat16 *v_row[4], *w_row[4];
    uint32_t to[4];
#pragma unroll
    for (uint32_t m = 0; m < 4; ++m) {
        const uint32_t r = tid / 8 + 32 * m, j = r % rp;
        to[m] = tile_at(r, chunk);
        v_row[m] = t0 + r < P.n && tile.of[r] >= 0 ? J.v + (t0 + r) * J.stride + chunk * 8 : nullptr;
        w_row[m] = r < cols && j < P.rank ? J.w + (uint64_t(tile.list[a0 + r / rp]) * P.rank + j) * J.len + chunk * 8 : nullptr;
    }
    auto load = [&](uint32_t k) {
        const uint32_t at = base + (k - k0) % kShrinkStages * kShrinkStage, col = k * kStep;
        const bool in = col + chunk * 8 < J.len;
#pragma unroll
        for (uint32_t m = 0; m < 4; ++m) {
            const bool some = in && v_row[m];
            cp_async16z(at + to[m], some ? v_row[m] + col : J.v, some ? 16 : 0);
        }
#pragma unroll
        for (uint32_t m = 0; m < 4; ++m) {
            if (tid / 8 + 32 * m >= cols) break;
            const bool some = in && w_row[m];
            cp_async16z(at + kTileBytes + to[m], some ? w_row[m] + col : J.w, some ? 16 : 0);
        }
    };
    const uint32_t desc = mma_desc(kTile, cols, 0, 0);
    bool ok = true;
    // this thread's sums: token (lane) warp % 4 * 32 + lane, columns warp / 4 * 64 on.  Runs of
    // kRun steps take turns in the two halves of TMEM
    constexpr uint32_t kRun = kChain / (kStep / 16);
    float sum[64] = {};
    auto drain = [&](uint32_t run) {
        tc_fence_after();
#pragma unroll
        for (uint32_t c = 0; c < 64; c += 16)
            if (warp / 4 * 64 + c < cols) {
                float v[16];
                tmem_load16(tmem + ((warp % 4) << 21) + (run & 1) * 128 + warp / 4 * 64 + c, v);
#pragma unroll
                for (int k = 0; k < 16; ++k) sum[c + k] += v[k];
            }
        tc_fence_before();
    };
    for (uint32_t k = k0; k < k0 + kShrinkStages - 1; ++k) {
        if (k < k1) load(k);
        cp_async_commit();
    }
    for (uint32_t k = k0; k < k1; ++k) {
        const uint32_t i = k - k0, stage = i % kShrinkStages;
        cp_async_wait<kShrinkStages - 2>();
        fence_async_shared();
        __syncthreads();
        if (tid == 0 && ok) {
            tc_fence_after();
            const uint64_t a = tile_desc(base + stage * kShrinkStage, 16, 1024), b = tile_desc(base + stage * kShrinkStage + kTileBytes, 16, 1024);
#pragma unroll
            for (uint32_t s = 0; s < kStep / 16; ++s) mma(tmem + (i / kRun & 1) * 128, a + 2 * s, b + 2 * s, desc, i % kRun || s);
            mma_commit(smem_addr(&s_bar[stage]));
        }
        // the stage before this one is free once its products are done
        if (i > 0 && ok) ok = mbar_wait(smem_addr(&s_bar[(i - 1) % kShrinkStages]), (i - 1) / kShrinkStages & 1);
        if (k + kShrinkStages - 1 < k1 && ok) load(k + kShrinkStages - 1);
        cp_async_commit();
        if (i > 0 && i % kRun == 0) drain(i / kRun - 1);
    }
    if (k1 > k0 && ok) ok = mbar_wait(smem_addr(&s_bar[(k1 - k0 - 1) % kShrinkStages]), (k1 - k0 - 1) / kShrinkStages & 1);
    cp_async_wait<0>();
    if (!ok) atomicOr(P.status, K3HUF_ST_TIMEOUT);
    if (k1 > k0) drain((k1 - k0 - 1) / kRun);
    __syncthreads();
    tc_fence_after();

    // each token's own columns, to shared memory (odd stride: one bank per lane)
    float *part = reinterpret_cast<float *>(smem);
    const uint32_t pitch = rp + 1;
    {
        const uint32_t t = warp % 4 * 32 + lane;
        const int32_t of = tile.of[t];
#pragma unroll
        for (uint32_t c = 0; c < 64; c += 16) {
            const uint32_t q = warp / 4 * 64 + c;
            if (q < cols && of == int32_t(a0 + q / rp))
#pragma unroll
                for (uint32_t k = 0; k < 16; ++k) part[t * pitch + q % rp + k] = sum[c + k];
        }
    }
    if (P.splits > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // a share of the tile's tokens per split: sum over the splits, scale, parts
    const uint32_t r0 = kTile * split / P.splits, r1 = kTile * (split + 1) / P.splits;
    for (uint32_t i = r0 * rp + tid; i < r1 * rp; i += kThreads) {
        const uint32_t t = i / rp, j = i % rp;
        const int32_t of = tile.of[t];
        if (of < int32_t(a0) || of >= int32_t(a0 + na)) continue;
        float sum = 0.f;
        for (uint32_t q = 0; q < P.splits; ++q) sum += P.splits > 1 ? cluster_load(smem_addr(part + t * pitch + j), q) : part[t * pitch + j];
        __nv_bfloat16 p[3];
        parts_of(P.scales[tile.list[of]] * sum, p);
        for (uint32_t q = 0; q < P.parts; ++q) J.h[(q * P.n + t0 + t) * rp + j] = p[q];
    }
    if (P.splits > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 0) tmem_free(tmem, 256);
}

struct ExpandParams {
    const __nv_bfloat16 *h, *w;
    const void *base;
    void *y;
    const int32_t *ids;
    uint32_t *status;
    uint64_t n, base_stride, y_stride;
    uint32_t n_adapters, rank, rank_pad, len, groups;
};

// The expand.  D[128 columns, 128 tokens] = W^T H^T with the adapters of the
// tile one after another along the contraction and H zero where a token has
// another one: W is read MN-major as it lies in memory, H K-major, in kParts
// parts.  With columns as the operand's rows a warp holds 32 neighbouring
// columns of a token, so the additions to the base run along shared memory rows
// that bulk copies bring and take away.  CTAs: a tile of tokens x a range of
// column tiles.  While one column tile is added, the next one's product runs
// and the one after is loaded.  Bound by the read of the base and the write of y.
constexpr uint32_t kMaxParts = 3;
template <typename T> struct Expand {
    static constexpr uint32_t tokens = sizeof(T) == 4 ? 64 : 128;         // (two tiles of the base in 64 KB)
    static constexpr uint32_t parts = sizeof(T) == 4 ? 3 : 2, part_bytes = tokens * 128;
    static constexpr uint32_t h_bytes = parts * part_bytes, w_bytes = kTileBytes;
    static constexpr uint32_t io_bytes = tokens * 128 * sizeof(T);
    static constexpr size_t smem = 2 * (h_bytes + w_bytes + io_bytes) + 1024;
    static_assert(smem <= 220 * 1024, "shared memory of one CTA");
};

template <typename T>
__global__ void __launch_bounds__(kThreads) expand_kernel(const __grid_constant__ ExpandParams P) {
    using E = Expand<T>;
    constexpr uint32_t NT = E::tokens;
    extern __shared__ uint8_t raw[];
    __shared__ TileAdapters tile;
    __shared__ __align__(8) uint64_t s_mma[2], s_io[2];
    __shared__ uint32_t s_tmem;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t h_at = smem_addr(smem), w_at = h_at + 2 * E::h_bytes, io_at = w_at + 2 * E::w_bytes;
    uint8_t *io = smem + 2 * (E::h_bytes + E::w_bytes);
    const uint32_t rp = P.rank_pad;
    const uint64_t t0 = uint64_t(blockIdx.x / P.groups) * NT;
    const uint32_t group = blockIdx.x % P.groups, col_tiles = (P.len + 127) / 128;
    const uint32_t c0 = uint32_t(uint64_t(col_tiles) * group / P.groups), c1 = uint32_t(uint64_t(col_tiles) * (group + 1) / P.groups);
    if (warp == 0) tmem_alloc(smem_addr(&s_tmem), 256);
    if (tid == 0)
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&s_mma[i]), 1);
            mbar_init(smem_addr(&s_io[i]), NT);
        }
    if (tid == 0) fence_async_shared();
    grid_dep_wait();
    const uint32_t count = tile_adapters(tile, P.ids, t0, P.n, NT, P.n_adapters, nullptr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // the contraction in chunks of 64 rank rows: whole adapters, or 64 rows of one
    const uint32_t per = rp <= kStep ? kStep / rp : 1, blocks = rp <= kStep ? 1 : (rp + kStep - 1) / kStep;
    const uint32_t chunks = rp <= kStep ? (count + per - 1) / per : count * blocks;
    const uint32_t tiles = c1 - c0, steps = tiles * max(chunks, 1u);
    const bool resident = chunks <= 2;        // H of both chunks stays in its two places
    // place of a chunk's row: adapter (in the tile's list), rank row
    auto row_of = [&](uint32_t chunk, uint32_t r, uint32_t &a, uint32_t &j) {
        if (rp <= kStep) {
            a = chunk * per + r / rp;
            j = r % rp;
            return r < per * rp && a < count;
        }
        a = chunk / blocks;
        j = chunk % blocks * kStep + r;
        return j < rp;
    };
    auto load_h = [&](uint32_t chunk, uint32_t place) {
        for (uint32_t i = tid; i < NT * 8; i += kThreads) {
            const uint32_t t = i / 8, c = i % 8;
            uint32_t a, j;
            const bool in = row_of(chunk, c * 8, a, j) && t0 + t < P.n && tile.of[t] == int32_t(a);
            const __nv_bfloat16 *src = in ? P.h + (t0 + t) * rp + j : P.h;
#pragma unroll
            for (uint32_t q = 0; q < E::parts; ++q)
                cp_async16z(h_at + place * E::h_bytes + q * E::part_bytes + tile_at(t, c), in ? src + q * P.n * rp : src, in ? 16 : 0);
        }
    };
    // this thread's part of a step: chunk tid % 16 of rows tid / 16 + 16 m
    const uint32_t w_chunk = tid % 16;
    uint32_t w_a[4], w_j[4], w_to[4];
#pragma unroll
    for (uint32_t m = 0; m < 4; ++m) {
        const uint32_t r = tid / 16 + 16 * m;
        w_a[m] = rp <= kStep ? r / rp : 0;
        w_j[m] = rp <= kStep ? r % rp : 0;
        w_to[m] = w_chunk / 8 * (kStep * 128) + tile_at(r, w_chunk % 8);
    }
    // step s: column tile c0 + s / chunks, chunk s % chunks
    auto load_step = [&](uint32_t s) {
        const uint32_t chunk = s % chunks, col = (c0 + s / chunks) * 128 + w_chunk * 8;
#pragma unroll
        for (uint32_t m = 0; m < 4; ++m) {
            const uint32_t a = rp <= kStep ? chunk * per + w_a[m] : chunk / blocks, j = rp <= kStep ? w_j[m] : chunk % blocks * kStep + tid / 16 + 16 * m;
            const bool in = w_a[m] < per && a < count && j < P.rank && col < P.len;
            cp_async16z(w_at + (s & 1) * E::w_bytes + w_to[m], in ? P.w + (uint64_t(tile.list[a]) * P.rank + j) * P.len + col : P.w, in ? 16 : 0);
        }
        if (!resident) load_h(chunk, s & 1);
    };
    const uint32_t desc = mma_desc(128, NT, 1, 0);
    auto multiply = [&](uint32_t s) {         // by one thread
        const uint32_t chunk = s % chunks, d = tmem + (s / chunks & 1) * 128;
        const uint64_t a = tile_desc(w_at + (s & 1) * E::w_bytes, kStep * 128, 1024);
        const uint32_t h = h_at + (resident ? chunk : s & 1) * E::h_bytes;
        tc_fence_after();
#pragma unroll
        for (uint32_t q = 0; q < E::parts; ++q) {
            const uint64_t b = tile_desc(h + q * E::part_bytes, 16, 1024);
#pragma unroll
            for (uint32_t k = 0; k < kStep / 16; ++k) mma(d, a + k * 128, b + 2 * k, desc, chunk || q || k);
        }
        mma_commit(smem_addr(&s_mma[s & 1]));
    };
    // the base's rows of a column tile: thread t brings and takes away row t
    const uint32_t rows = uint32_t(min(uint64_t(NT), P.n - t0));
    auto row_bytes = [&](uint32_t i) { return min(128u, P.len - (c0 + i) * 128) * uint32_t(sizeof(T)); };
    auto load_io = [&](uint32_t i) {
        const uint32_t bar = smem_addr(&s_io[i & 1]);
        if (tid < NT) {
            const bool in = P.base && tid < rows;
            mbar_expect(bar, in ? row_bytes(i) : 0);
            if (in)
                bulk_load(io_at + (i & 1) * E::io_bytes + tid * (128 * sizeof(T)), static_cast<const T *>(P.base) + (t0 + tid) * P.base_stride + (c0 + i) * 128, row_bytes(i), bar);
        }
    };
    bool ok = true;
    load_io(0);
    if (chunks) {
        if (resident)
            for (uint32_t c = 0; c < chunks; ++c) load_h(c, c);
        load_step(0);
        cp_async_commit();
        if (steps > 1) load_step(1);
        cp_async_commit();
        cp_async_wait<1>();
        fence_async_shared();
        __syncthreads();
        if (tid == 0) multiply(0);
    }
    for (uint32_t s = 0; s < steps; ++s) {
        const uint32_t i = chunks ? s / chunks : s;
        if (chunks) {
            if (s + 1 < steps) {
                cp_async_wait<0>();
                fence_async_shared();
                tc_fence_before();
                __syncthreads();
                if (tid == 0 && ok) multiply(s + 1);
            }
            if (ok) ok = mbar_wait(smem_addr(&s_mma[s & 1]), s / 2 & 1);
            if (s + 2 < steps && ok) load_step(s + 2);
            cp_async_commit();
            if (s % chunks + 1 < chunks) continue;
        }
        // column tile i: the product is in its half of TMEM
        if (i + 1 < tiles) {
            if (tid < NT) bulk_wait_read<0>();          // (tile i - 1 has left the other buffer)
            load_io(i + 1);
        }
        if (ok) ok = mbar_wait(smem_addr(&s_io[i & 1]), i / 2 & 1);
        tc_fence_after();
        T *mine = reinterpret_cast<T *>(io + (i & 1) * E::io_bytes) + warp % 4 * 32 + lane;
        const uint32_t t_end = min((warp / 4 + 1) * (NT / 2), rows);
        for (uint32_t t = warp / 4 * (NT / 2); t < t_end; t += 32) {
            // (the base's values are fetched while the product comes from TMEM)
            uint32_t r[32];
            float b[32];
            if (chunks) tmem_load32(tmem + ((warp % 4) << 21) + (i & 1) * 128 + t, r);
            T *q = mine + t * 128;
            if (P.base) {
#pragma unroll
                for (uint32_t k = 0; k < 32; ++k) b[k] = ld_f32(q + k * 128);
            } else {
#pragma unroll
                for (uint32_t k = 0; k < 32; ++k) b[k] = 0.f;
            }
            if (chunks) {
                tmem_wait32(r);
#pragma unroll
                for (uint32_t k = 0; k < 32; ++k) b[k] += __uint_as_float(r[k]);
            }
#pragma unroll
            for (uint32_t k = 0; k < 32; ++k) st_f32(q + k * 128, b[k]);
        }
        tc_fence_before();
        fence_async_shared();
        __syncthreads();
        if (tid < rows) bulk_store(static_cast<T *>(P.y) + (t0 + tid) * P.y_stride + (c0 + i) * 128, io_at + (i & 1) * E::io_bytes + tid * (128 * sizeof(T)), row_bytes(i));
        if (tid < NT) bulk_commit();
    }
    if (tid < NT) bulk_wait_all();
    cp_async_wait<0>();
    if (!ok) atomicOr(P.status, K3HUF_ST_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free(tmem, 256);
}

struct OuterJob {
    const __nv_bfloat16 *h, *v;               // parts x tokens x rank_pad; the rows that it multiplies
    float *g;
    uint64_t stride;
    uint32_t len;
};
struct OuterParams {
    OuterJob job[2];
    const int32_t *ids;
    uint32_t *status;
    uint64_t n;
    uint32_t n_adapters, rank, rank_pad, col_tiles0;       // column tiles of job 0
    bool add;
};

// The outer product.  D[128 columns, rank] = V^T H over the tokens of one
// adapter, 64 of them per step, gathered by their indexes: both operands lie
// token by token, so both are read MN-major.  CTAs: a tile of columns (of
// either gradient) x an adapter; the tokens' indexes come from the ids,
// kWindow at a time, in order.  Bound by the read of V.
constexpr uint32_t kWindow = 4096;
constexpr uint32_t kOuterStages = 2;

template <uint32_t kBlocks>                   // blocks of 64 rank rows
constexpr uint32_t kOuterStage = kStep * 256 + kMaxParts * kBlocks * kStep * 128;
template <uint32_t kBlocks>
constexpr size_t kOuterSmem = kOuterStages * kOuterStage<kBlocks> + 1024;

template <uint32_t kBlocks>
__global__ void __launch_bounds__(kThreads) outer_kernel(const __grid_constant__ OuterParams P) {
    constexpr uint32_t kStage = kOuterStage<kBlocks>;
    extern __shared__ uint8_t raw[];
    __shared__ uint32_t s_token[kWindow], s_count[kThreads / 32 + 1], s_tmem;
    __shared__ __align__(8) uint64_t s_bar[kOuterStages];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32, base = smem_addr(smem), rp = P.rank_pad;
    const bool second = blockIdx.x >= P.col_tiles0;
    const OuterJob &J = P.job[second];
    const uint32_t col = (blockIdx.x - (second ? P.col_tiles0 : 0)) * 128;
    if (warp == 0) tmem_alloc(smem_addr(&s_tmem), kBlocks * 128);
    if (tid == 0)
        for (uint32_t i = 0; i < kOuterStages; ++i) mbar_init(smem_addr(&s_bar[i]), 1);
    if (tid == 0) fence_async_shared();
    grid_dep_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem, desc = mma_desc(128, rp, 1, 1);
    bool ok = true;
    uint32_t step = 0;                        // steps of this CTA so far: stage step % 2, phase step / 2 % 2
    for (uint32_t a = blockIdx.y; a < P.n_adapters; a += gridDim.y) {
        const uint32_t first = step;
        // this thread's sums: column (lane) warp % 4 * 32 + lane, rank rows warp / 4 * 16 + 32 b on
        constexpr uint32_t kRun = kChain / (kMaxParts * kStep / 16);
        float sum[2 * kBlocks][16] = {};
        auto drain = [&](uint32_t run) {
            tc_fence_after();
#pragma unroll
            for (uint32_t b = 0; b < 2 * kBlocks; ++b)
                if (warp / 4 * 16 + b * 32 < rp) {
                    float v[16];
                    tmem_load16(tmem + ((warp % 4) << 21) + (run & 1) * (kBlocks * 64) + warp / 4 * 16 + b * 32, v);
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
                        const __nv_bfloat16 *src = J.h + t * rp + c * 8;
#pragma unroll
                        for (uint32_t q = 0; q < kMaxParts; ++q) cp_async16z(to + kStep * 256 + q * (kBlocks * kStep * 128) + at, src + q * P.n * rp, in ? 16 : 0);
                    }
                }
            };
            if (steps) load(0);
            cp_async_commit();
            for (uint32_t s = 0; s < steps; ++s) {
                const uint32_t g = step + s;
                // the other stage is free once the step before is done
                if (s > 0 && ok) ok = mbar_wait(smem_addr(&s_bar[(g - 1) % kOuterStages]), (g - 1) / kOuterStages & 1);
                if (s + 1 < steps && ok) load(s + 1);
                cp_async_commit();
                cp_async_wait<1>();
                fence_async_shared();
                __syncthreads();
                if (tid == 0 && ok) {
                    tc_fence_after();
                    const uint32_t at = base + g % kOuterStages * kStage;
                    const uint64_t va = tile_desc(at, kStep * 128, 1024);
#pragma unroll
                    for (uint32_t q = 0; q < kMaxParts; ++q) {
                        const uint64_t hb = tile_desc(at + kStep * 256 + q * kBlocks * (kStep * 128), kStep * 128, 1024);
#pragma unroll
                        for (uint32_t k = 0; k < kStep / 16; ++k) mma(tmem + ((g - first) / kRun & 1) * (kBlocks * 64), va + k * 128, hb + k * 128, desc, (g - first) % kRun || q || k);
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
        // lane: column; a warp's stores of one rank row are 128 adjacent bytes
        const uint32_t c = col + warp % 4 * 32 + lane;
        if (c < J.len)
#pragma unroll
            for (uint32_t b = 0; b < 2 * kBlocks; ++b)
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
    if (warp == 0) tmem_free(tmem, kBlocks * 128);
}

// --- host -----------------------------------------------------------------------

bool adapters_ok(const k3huf_adapters_t *ad, uint64_t n) {
    return ad && ad->a && ad->b && ad->scales && ad->n_adapters && ad->n_adapters < (1u << 24) && ad->rank && ad->rank <= K3HUF_MAX_RANK &&
           ad->cols && ad->rows && ad->cols < (1ull << 31) && ad->rows < (1ull << 31) && n < (1ull << 31) && aligned_to(ad->a, 2) &&
           aligned_to(ad->b, 2) && aligned_to(ad->scales, 4);
}

uint32_t padded(uint32_t rank) { return (rank + 15) / 16 * 16; }
// Bytes of one rank-wide intermediate: fp32, or three bf16 parts of the padded rank.
uint64_t h_bytes(uint64_t n, uint32_t rank) { return align_up(n * std::max<uint64_t>(4 * rank, 2 * kMaxParts * padded(rank)), 256); }

enum class Form { any, few, many };
bool rows16(const void *p, uint64_t stride, uint32_t type) { return aligned_to(p, 16) && stride * elem_bytes(type) % 16 == 0; }
// Tokens x rank up to kFewWork: each token's factor rows are read on their own,
// about 100 MB from L2 at 4096 x (8192 + 8192) in 14 us; the tiles take about 20 us
// for 192 tokens of as many adapters.
Form run_form(uint64_t n, uint32_t rank, bool rows_ok) { return !rows_ok ? Form::any : n * rank <= kFewWork ? Form::few : Form::many; }

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
    cfg.gridDim = dim3(uint32_t(tiles * P.splits), groups, jobs);
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

template <typename T>
int launch_expand(ExpandParams &P, uint64_t sms, cudaStream_t stream) {
    static std::atomic<uint64_t> once{0};
    const int rc = once_per_device(once, [] { return cudaFuncSetAttribute(expand_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Expand<T>::smem)); });
    if (rc) return rc;
    const uint64_t tiles = (P.n + Expand<T>::tokens - 1) / Expand<T>::tokens, cols = (P.len + 127) / 128;
    // column ranges per token tile: the count whose last wave of CTAs (one per SM) is fullest,
    // among those that give an SM up to three waves
    uint64_t best = 1;
    double waste = 1e30;
    for (uint64_t g = 1; g <= cols && g <= std::max<uint64_t>(1, 3 * sms / tiles); ++g) {
        const uint64_t waves = (tiles * g + sms - 1) / sms, per = (cols + g - 1) / g;
        const double w = double(waves * (per + 1));        // (a CTA's start costs about one column tile)
        if (w < waste) waste = w, best = g;
    }
    P.groups = uint32_t(best);
    return launch_after(expand_kernel<T>, dim3(uint32_t(tiles * best)), kThreads, Expand<T>::smem, stream, P);
}

int launch_outer(const OuterParams &P, uint32_t col_tiles, cudaStream_t stream) {
    static std::atomic<uint64_t> once{0};
    const int rc = once_per_device(once, [] {
        const cudaError_t e = cudaFuncSetAttribute(outer_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kOuterSmem<1>));
        return e != cudaSuccess ? e : cudaFuncSetAttribute(outer_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kOuterSmem<2>));
    });
    if (rc) return rc;
    const dim3 grid(col_tiles, std::min(P.n_adapters, 65535u));
    return P.rank_pad <= kStep ? launch_after(outer_kernel<1>, grid, kThreads, kOuterSmem<1>, stream, P)
                               : launch_after(outer_kernel<2>, grid, kThreads, kOuterSmem<2>, stream, P);
}

}  // namespace
}  // namespace k3huf

using namespace k3huf;

extern "C" int k3huf_adapter_scratch_bytes(uint64_t n_tokens, uint32_t n_adapters, uint32_t rank, uint64_t cols, uint64_t rows, int grad, size_t *scratch_bytes) {
    if (!scratch_bytes || n_adapters == 0 || rank == 0 || rank > K3HUF_MAX_RANK || cols == 0 || rows == 0 || n_tokens >= (1ull << 31)) return K3HUF_E_ARG;
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
    switch (run_form(n, r, rows_ok)) {
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
            const dim3 grid(n, uint32_t((ad->rows + 511) / 512));
            if (y_type == K3HUF_BF16)
                return launch_after(expand_few_kernel<__nv_bfloat16>, grid, 128, 0, st, h, b, d_ids, S, r, uint32_t(ad->rows), static_cast<const __nv_bfloat16 *>(d_base), base_stride, static_cast<__nv_bfloat16 *>(d_y), y_stride);
            return launch_after(expand_few_kernel<float>, grid, 128, 0, st, h, b, d_ids, S, r, uint32_t(ad->rows), static_cast<const float *>(d_base), base_stride, static_cast<float *>(d_y), y_stride);
        }
        case Form::many: break;
    }
    uint64_t sms = 0;
    int rc = sm_count(&sms);
    if (rc) return rc;
    auto *h = static_cast<__nv_bfloat16 *>(d_scratch);
    ShrinkParams sp{{{x, a, x_stride, uint32_t(ad->cols), h}}, ad->scales, d_ids, d_status, n, S, r, padded(r), y_type == K3HUF_F32 ? 3u : 2u, 1};
    rc = launch_shrink(sp, 1, sms, st);
    if (rc) return rc;
    ExpandParams ep{h, b, d_base, d_y, d_ids, d_status, n, base_stride, y_stride, S, r, padded(r), uint32_t(ad->rows), 1};
    return y_type == K3HUF_BF16 ? launch_expand<__nv_bfloat16>(ep, sms, st) : launch_expand<float>(ep, sms, st);
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
    ShrinkParams sp{{{x, a, x_stride, uint32_t(ad->cols), h}, {dy, b, dy_stride, uint32_t(ad->rows), dh}}, ad->scales, d_ids, d_status, n, S, r, padded(r), kMaxParts, 1};
    rc = launch_shrink(sp, 2, sms, st);
    if (rc) return rc;
    if (d_dx) {
        ExpandParams ep{dh, a, d_dx_base, d_dx, d_ids, d_status, n, dx_base_stride, dx_stride, S, r, padded(r), uint32_t(ad->cols), 1};
        rc = dx_type == K3HUF_BF16 ? launch_expand<__nv_bfloat16>(ep, sms, st) : launch_expand<float>(ep, sms, st);
        if (rc) return rc;
    }
    const uint32_t tiles_a = uint32_t((ad->cols + 127) / 128), tiles_b = uint32_t((ad->rows + 127) / 128);
    const OuterParams op{{{dh, x, d_da, x_stride, uint32_t(ad->cols)}, {h, dy, d_db, dy_stride, uint32_t(ad->rows)}}, d_ids, d_status, n, S, r, padded(r), tiles_a, add};
    return launch_outer(op, tiles_a + tiles_b, st);
}
