// The matrix product with bias, activation and residual in its epilogue, and its gradients:
//   z = x W^T + bias          y = act(z) + residual
//   dz = dy act'(z)           dbias = sum over tokens of dz
//   dx = dz W                 dW = dz^T x
// The three products are one kernel on tcgen05.mma,
//   out[j][i] = sum_k A[i][k] B[j][k]         (i runs along a row of the result),
// with A = W, B = x for y; A = W^T, B = dz for dx; A = x^T, B = dz^T for dW.  An operand that lies
// contraction-last is read K-major, one that lies contraction-first (W for dx; x and dz for dW) MN-major from
// the same 128-byte swizzled tiles, so nothing is transposed in memory.  i is the tile's 128 lanes of TMEM: a
// warp's store of one j is 32 neighbouring elements of the result, and the epilogue needs no shared memory.
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

template <uint32_t kTileJ> struct Shape {
    static constexpr uint32_t a_bytes = kTileI * 128, b_bytes = kTileJ * 128, stage = a_bytes + b_bytes;
    static constexpr uint32_t per_sm = kTileJ <= 64 ? 2 : 1;                 // CTAs
    static constexpr uint32_t stages = kTileJ == 256 ? 4 : kTileJ == 128 ? 6 : kTileJ == 64 ? 4 : kTileJ == 32 ? 5 : 6;
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
    uint64_t tiles;
    uint32_t size_i, size_j, steps, tiles_i, tiles_j, splits, run;     // run: steps added up in TMEM
};

__device__ __forceinline__ float activate(float z, uint32_t act) {
    if (act == K3HUF_ACT_RELU) return z < 0.f ? 0.f : z;
    if (act == K3HUF_ACT_SILU) return z / (1.f + expf(-z));
    // (1 + tanh u) / 2 is the logistic function of 2 u
    if (act == K3HUF_ACT_GELU) return z / (1.f + expf(-1.5957691216057308f * fmaf(0.044715f * z * z, z, z)));
    return z;
}

// Order of the tiles: kGroup rows of tiles at a time, so that the CTAs at work at once share operands.
constexpr uint32_t kGroup = 16;
__device__ __forceinline__ void tile_place(const ProductParams &P, uint64_t t, uint32_t &ti, uint32_t &tj) {
    const uint64_t whole = uint64_t(kGroup) * P.tiles_j;
    const uint32_t g = uint32_t(t / whole), rest = uint32_t(t % whole), rows = min(kGroup, P.tiles_i - g * kGroup);
    ti = g * kGroup + rest % rows;
    tj = rest / rows;
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
    const uint64_t t_first = blockIdx.x / P.splits, t_step = gridDim.x / P.splits;
    const uint32_t k0 = uint32_t(uint64_t(P.steps) * split / P.splits), n_steps = uint32_t(uint64_t(P.steps) * (split + 1) / P.splits) - k0;
    const uint32_t runs = (n_steps + P.run - 1) / P.run;
    if (warp == 0) tmem_alloc(smem_addr(&s_tmem), 2 * kTileJ);
    if (tid == 0) {
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    float sum[S::part];
    const uint32_t quarter = warp % 4, c_first = warp / 4 * S::part;         // (epilogue warps)
    const bool reads = warp < kEpilogue / 32 && c_first < kTileJ;

    // (out, z: the column j, a row of the result, at the thread's i)
    const Epilogue &e = P.e;
    auto finish = [&](uint32_t i, uint32_t j, const float *v, int count, float bias) {       // count (<= 16) neighbouring j
        float res[16];
        if (e.residual) {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                if (c >= count) break;
                const uint64_t at = uint64_t(j + c) * e.residual_stride + i;
                res[c] = j + c >= P.size_j ? 0.f : e.out_type == K3HUF_F32 ? static_cast<const float *>(e.residual)[at] : ld_f32(static_cast<const __nv_bfloat16 *>(e.residual) + at);
            }
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            if (c >= count || j + c >= P.size_j) break;
            const float z = e.bias ? v[c] + bias : v[c];
            if (e.z) {
                const uint64_t at = uint64_t(j + c) * e.z_stride + i;
                if (e.z_type == K3HUF_F32) static_cast<float *>(e.z)[at] = z;
                else st_f32(static_cast<__nv_bfloat16 *>(e.z) + at, z);
            }
            float y = activate(z, e.act);
            if (e.residual) y += res[c];
            const uint64_t at = uint64_t(j + c) * e.out_stride + i;
            if (e.out_type == K3HUF_F32) static_cast<float *>(e.out)[at] = y;
            else st_f32(static_cast<__nv_bfloat16 *>(e.out) + at, y);
        }
    };
    auto bias_at = [&](uint32_t i) {
        return !e.bias ? 0.f : e.bias_type == K3HUF_F32 ? static_cast<const float *>(e.bias)[i] : ld_f32(static_cast<const __nv_bfloat16 *>(e.bias) + i);
    };

    if (warp == kEpilogue / 32) {
        if (lane == 0) {
            uint32_t stage = 0, round = 0;    // copies so far: round * NS + stage
            for (uint64_t t = t_first; t < P.tiles && ok; t += t_step) {
                uint32_t ti, tj;
                tile_place(P, t, ti, tj);
                const int32_t i0 = int32_t(ti * kTileI), j0 = int32_t(tj * kTileJ);
                for (uint32_t s = 0; s < n_steps; ++s) {
                    if (round) ok = mbar_wait(smem_addr(&s_free[stage]), (round - 1) & 1);
                    if (!ok) break;
                    const uint32_t at = base + stage * S::stage, bar = smem_addr(&s_full[stage]);
                    const int32_t k = int32_t((k0 + s) * kStep);
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
                    if (++stage == NS) stage = 0, ++round;
                }
            }
            // the last copies land before the CTA ends, whichever thread's wait may have given up
            for (uint32_t q = 0; q < NS && (round || stage); ++q) {
                if (stage == 0) stage = NS, --round;
                --stage;
                mbar_wait(smem_addr(&s_full[stage]), round & 1);
            }
        }
        __syncwarp();
    } else if (warp == kEpilogue / 32 + 1) {
        if (lane == 0) {
            constexpr uint32_t desc = mma_desc(kTileI, kTileJ, kMnA, kMnB);
            const uint64_t a0 = tile_desc(base, kMnA ? kStep * 128 : 16, 1024), b0 = tile_desc(base + S::a_bytes, kMnB ? kStep * 128 : 16, 1024);
            uint32_t stage = 0, round = 0, r = 0;      // r: runs so far
            for (uint64_t t = t_first; t < P.tiles && ok; t += t_step)
                for (uint32_t s = 0, in_run = 0; s < n_steps; ++s) {
                    if (in_run == 0 && r >= 2) ok = mbar_wait(smem_addr(&s_read[r & 1]), (r / 2 - 1) & 1);
                    if (ok) ok = mbar_wait(smem_addr(&s_full[stage]), round & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a = a0 + stage * (S::stage >> 4), b = b0 + stage * (S::stage >> 4);
                    const uint32_t d = tmem + (r & 1) * kTileJ;
#pragma unroll
                    for (uint32_t q = 0; q < kStep / 16; ++q) mma(d, a + q * (kMnA ? 128 : 2), b + q * (kMnB ? 128 : 2), desc, in_run || q);
                    mma_commit(smem_addr(&s_free[stage]));
                    if (++stage == NS) stage = 0, ++round;
                    if (++in_run == P.run || s + 1 == n_steps) {
                        mma_commit(smem_addr(&s_sum[r & 1]));
                        in_run = 0;
                        ++r;
                    }
                }
            // (products whose end nobody waited for, if a wait gave up, end before the CTA does)
            for (uint32_t q = 0; q < NS && (round || stage); ++q) {
                if (stage == 0) stage = NS, --round;
                --stage;
                mbar_wait(smem_addr(&s_free[stage]), round & 1);
            }
        }
        __syncwarp();
    } else {
        uint32_t r = 0;
        for (uint64_t t = t_first; t < P.tiles; t += t_step) {
            uint32_t ti, tj;
            tile_place(P, t, ti, tj);
            const uint32_t i = ti * kTileI + quarter * 32 + lane;
            const float bias = i < P.size_i ? bias_at(i) : 0.f;
            for (uint32_t q = 0; q < runs; ++q, ++r) {
                if (ok) ok = mbar_wait(smem_addr(&s_sum[r & 1]), r / 2 & 1);
                tc_fence_after();
                if (reads) {
                    const uint32_t from = tmem + (quarter << 21) + (r & 1) * kTileJ + c_first;
#pragma unroll
                    for (uint32_t c = 0; c < S::part; c += 16) {
                        float v[16];
                        tmem_load16(from + c, v);
#pragma unroll
                        for (int k = 0; k < 16; ++k) sum[c + k] = q ? sum[c + k] + v[k] : v[k];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&s_read[r & 1]));
            }
            if (P.splits == 1 && reads && i < P.size_i) {
#pragma unroll
                for (uint32_t c = 0; c < S::part; c += 16) finish(i, tj * kTileJ + c_first + c, sum + c, 16, bias);
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
        const uint32_t i = ti * kTileI + quarter * 32 + lane;
        if (warp < kEpilogue / 32 && i < P.size_i) {
            const float bias = bias_at(i);
            const uint32_t c0 = kTileJ * split / P.splits, c1 = kTileJ * (split + 1) / P.splits;
            for (uint32_t c = c0 + warp / 4; c < c1 && tj * kTileJ + c < P.size_j; c += 2) {
                float part[kMaxSplits], v = 0.f;
#pragma unroll
                for (uint32_t q = 0; q < kMaxSplits; ++q)
                    if (q < P.splits) part[q] = cluster_load(smem_addr(parts + c * kTileI + quarter * 32 + lane), q);
#pragma unroll
                for (uint32_t q = 0; q < kMaxSplits; ++q)
                    if (q < P.splits) v += part[q];
                finish(i, tj * kTileJ + c, &v, 1, bias);
            }
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
    if (!ok) atomicOr(P.status, K3HUF_ST_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free(tmem, 2 * kTileJ);
}

// Rows that do not start on 16 bytes, copied to rows that do (TMA reads no others): 8 values per thread.
constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads) align_rows_kernel(const uint16_t *from, uint64_t stride, uint64_t rows, uint32_t cols, uint32_t pitch, uint16_t *to) {
    const uint32_t per_row = pitch / 8;
    for (uint64_t at = uint64_t(blockIdx.x) * kCopyThreads + threadIdx.x; at < rows * per_row; at += uint64_t(gridDim.x) * kCopyThreads) {
        const uint64_t r = at / per_row;
        const uint32_t c = uint32_t(at % per_row) * 8;
        const uint16_t *src = from + r * stride + c;
        uint32_t w[4];
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) w[k] = (c + 2 * k < cols ? src[2 * k] : 0u) | (c + 2 * k + 1 < cols ? uint32_t(src[2 * k + 1]) << 16 : 0u);
        reinterpret_cast<uint4 *>(to)[at] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// act'(z).  Far out, where it no longer changes in 32 bits, z stops: infinities give the limit.
__device__ __forceinline__ float slope(float z, uint32_t act) {
    if (act == K3HUF_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (act == K3HUF_ACT_SILU) {
        z = z > 80.f ? 80.f : z < -80.f ? -80.f : z;
        const float x = expf(-z), q = 1.f / (1.f + x);
        return fmaf(z * q, x * q, q);
    }
    if (act == K3HUF_ACT_GELU) {
        z = z > 10.f ? 10.f : z < -10.f ? -10.f : z;
        const float x = expf(-1.5957691216057308f * fmaf(0.044715f * z * z, z, z)), q = 1.f / (1.f + x);
        return fmaf(z * q, x * q * 1.5957691216057308f * fmaf(3.f * 0.044715f * z, z, 1.f), q);
    }
    return 1.f;
}

struct SlopeParams {
    const void *z, *dy;
    __nv_bfloat16 *dz;
    float *dbias;
    uint64_t n, z_stride, dy_stride, dz_stride;
    uint32_t rows, z_type, dy_type, act;
    bool add;
};

// dz and the columns' sums in one read of z and dy.  A CTA takes kSlopeCols columns (kPer neighbouring ones per thread)
// and its share of the tokens; the CTAs of a cluster, which share the columns, add up in the order of their tokens.
constexpr int kSlopeThreads = 256, kSlopeLanes = 16, kSlopeDepth = 4;        // threads along the columns; tokens in flight per thread
template <int kPer> __device__ __forceinline__ void load_row(const void *p, uint32_t type, uint64_t at, float (&f)[kPer]) {
    if constexpr (kPer == 8) {
        if (type == K3HUF_F32) {
            const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
            const float4 a = __ldcs(q), b = __ldcs(q + 1);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        } else {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + at));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) f[2 * k] = __uint_as_float(w[k] << 16), f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    } else {
        f[0] = type == K3HUF_F32 ? static_cast<const float *>(p)[at] : ld_f32(static_cast<const __nv_bfloat16 *>(p) + at);
    }
}

template <int kPer>
__global__ void __launch_bounds__(kSlopeThreads) slope_kernel(const SlopeParams P, uint32_t splits) {
    constexpr int kCols = kSlopeLanes * kPer, kDown = kSlopeThreads / kSlopeLanes;
    __shared__ float s_sum[kDown][kCols + 1], s_cta[kCols];
    const uint32_t split = blockIdx.x % splits, lane = threadIdx.x % kSlopeLanes, down = threadIdx.x / kSlopeLanes;
    const uint64_t c0 = uint64_t(blockIdx.x / splits) * kCols, c = c0 + lane * kPer;
    const uint64_t t0 = P.n * split / splits, t1 = P.n * (split + 1) / splits;
    float sum[kPer] = {};
    if (c < P.rows) {
        for (uint64_t t = t0 + down; t < t1; t += uint64_t(kDown) * kSlopeDepth) {
            float z[kSlopeDepth][kPer], g[kSlopeDepth][kPer];
#pragma unroll
            for (int d = 0; d < kSlopeDepth; ++d) {
                const uint64_t at = t + uint64_t(d) * kDown;
                if (at >= t1) break;
                load_row<kPer>(P.z, P.z_type, at * P.z_stride + c, z[d]);
                load_row<kPer>(P.dy, P.dy_type, at * P.dy_stride + c, g[d]);
            }
#pragma unroll
            for (int d = 0; d < kSlopeDepth; ++d) {
                const uint64_t at = t + uint64_t(d) * kDown;
                if (at >= t1) break;
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    g[d][k] *= slope(z[d][k], P.act);
                    sum[k] += g[d][k];
                }
                __nv_bfloat16 *o = P.dz + at * P.dz_stride + c;
                if constexpr (kPer == 8) {
                    uint4 v;
                    __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) q[k] = __floats2bfloat162_rn(g[d][2 * k], g[d][2 * k + 1]);
                    *reinterpret_cast<uint4 *>(o) = v;
                } else {
                    st_f32(o, g[d][0]);
                }
            }
        }
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
        cluster_arrive();
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

template <uint32_t kTileJ, bool kMnA, bool kMnB>
int launch_product(ProductParams &P, const Operand &a, const Operand &b, uint64_t sms, cudaStream_t stream) {
    using S = Shape<kTileJ>;
    static std::atomic<uint64_t> once{0};
    int rc = once_per_device(once, [] { return cudaFuncSetAttribute(product_kernel<kTileJ, kMnA, kMnB>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::smem)); });
    if (!rc) rc = tensor_map(&P.a, a.p, K3HUF_BF16, a.rows, a.cols, a.stride, kMnA ? kStep : kTileI, kStep, true);
    if (!rc) rc = tensor_map(&P.b, b.p, K3HUF_BF16, b.rows, b.cols, b.stride, kMnB ? kStep : kTileJ, kStep, true);
    if (rc) return rc;
    P.tiles_i = (P.size_i + kTileI - 1) / kTileI;
    P.tiles_j = (P.size_j + kTileJ - 1) / kTileJ;
    P.tiles = uint64_t(P.tiles_i) * P.tiles_j;
    const bool e_f32 = P.e.out_type == K3HUF_F32 || (P.e.z && P.e.z_type == K3HUF_F32);
    // fewer tiles than the GPU holds CTAs: the CTAs of a cluster share a tile's contraction
    const uint64_t slots = sms * S::per_sm;
    P.splits = uint32_t(std::max<uint64_t>(1, std::min<uint64_t>({kMaxSplits, slots / P.tiles, P.steps / 4})));
    P.run = e_f32 ? kChain / (kStep / 16) : P.steps;
    const uint64_t ctas = P.splits > 1 ? P.tiles * P.splits : std::min(P.tiles, slots);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(uint32_t(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = P.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_rc(cudaLaunchKernelEx(&cfg, product_kernel<kTileJ, kMnA, kMnB>, P));
}

// out[j][i] = sum_k A[i][k] B[j][k]
template <bool kMnA, bool kMnB>
int product(const Operand &a, const Operand &b, uint64_t size_i, uint64_t size_j, uint64_t size_k, const Epilogue &e, uint32_t *status, uint64_t sms, cudaStream_t stream) {
    ProductParams P{};
    P.e = e;
    P.status = status;
    P.size_i = uint32_t(size_i), P.size_j = uint32_t(size_j), P.steps = uint32_t((size_k + kStep - 1) / kStep);
    if constexpr (!kMnB) {
        if (size_j <= 16) return launch_product<16, kMnA, kMnB>(P, a, b, sms, stream);
        if (size_j <= 32) return launch_product<32, kMnA, kMnB>(P, a, b, sms, stream);
    }
    if (size_j <= 64) return launch_product<64, kMnA, kMnB>(P, a, b, sms, stream);
    if (size_j <= 128) return launch_product<128, kMnA, kMnB>(P, a, b, sms, stream);
    return launch_product<256, kMnA, kMnB>(P, a, b, sms, stream);
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
        (d_residual && d_residual == d_y && residual_stride != y_stride))
        return K3HUF_E_ARG;
    if (n_tokens == 0) return K3HUF_OK;
    if (!d_x || !d_w || !d_y) return K3HUF_E_ARG;
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
    uint64_t sms = 0;
    const int rc = sm_count(&sms);
    if (rc) return rc;
    const SlopeParams P{d_z, d_dy, static_cast<__nv_bfloat16 *>(d_dz), d_dbias, n_tokens, z_stride, dy_stride, dz_stride, uint32_t(rows), z_type, dy_type, act, add};
    auto on16 = [](const void *p, uint64_t stride, uint32_t type) { return aligned_to(p, 16) && stride * elem_bytes(type) % 16 == 0; };
    const bool vec = rows % 8 == 0 && on16(d_z, z_stride, z_type) && on16(d_dy, dy_stride, dy_type) && on16(d_dz, dz_stride, K3HUF_BF16);
    const uint32_t cols = kSlopeLanes * (vec ? 8 : 1);
    const uint64_t blocks = (rows + cols - 1) / cols;
    // tokens split over a cluster until the GPU is full (four CTAs per SM)
    uint32_t splits = 1;
    while (splits < 8 && blocks * splits < sms * 4 && n_tokens / splits > kSlopeThreads / kSlopeLanes * kSlopeDepth) splits *= 2;
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
    return cuda_rc(vec ? cudaLaunchKernelEx(&cfg, slope_kernel<8>, P, splits) : cudaLaunchKernelEx(&cfg, slope_kernel<1>, P, splits));
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
