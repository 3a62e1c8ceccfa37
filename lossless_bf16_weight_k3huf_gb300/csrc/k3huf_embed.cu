// Rows of a coded embedding table, scaled, and the gradient of such a lookup
// with respect to the table.
//
//   out[t, c] = s * W[ids[t], c]
//   G[v, c]   = s * sum over t with ids[t] = v of dY[t, c]
//
// Lookup: the container's chunk and sub-stream indexes give the first bit of
// every run of sub_syms values, so the sub-streams that a row meets are
// decoded and no others.  A unit is one sub-stream of one row; a warp takes up
// to 32 of them (one per lane; fewer when a call has few, so that they spread
// over the SMs), copies their bits to shared memory with 16-byte asynchronous
// copies, and decodes 64 values of each at a time.  A lookup of the next 12
// bits gives up to four whole codes (their mean length is under 3 bits), so a
// sub-stream of 256 values takes about 70 dependent lookups instead of 256.
// The warp then joins the 64 high bytes of each unit with the raw low bytes
// (loaded before the decode), scales in fp32 and stores 16 bytes per lane.
// What bounds it: a few units, the chain of lookups (about 55 cycles each)
// after the table's build (14 us for 32 rows of 8192); many, the lookups'
// wavefronts and the instructions of both halves (66 to 76 us for 8192 such
// rows, by their ids; 78 us in fp32).
#include <algorithm>

#include "k3huf_tc.h"

namespace k3huf {
namespace {

constexpr int kMaxStripes = 256;              // stripes of the tensor (kernel parameter space)
constexpr int kThreads = 128;                 // (one-symbol lookup kernel)
// Warps per CTA and the 16-byte pieces of bits that each stages; more warps leave
// each too few pieces, and rows of long codes take two passes (8192 rows of 8192
// values: 24 warps with 256 pieces 92 us, 18 with 464 70 us).
constexpr int kWarps = 18, kEmbedThreads = 32 * kWarps;
constexpr uint32_t kPieces = 464;
constexpr int kRound = 64;                    // values per unit between joins
constexpr int kRowWords = kRound / 4 + 1;     // a unit's high bytes of one round; the odd stride spreads the banks
constexpr uint32_t kMaxStagedSub = 1024;      // longest sub-stream whose bits surely fit a warp's pieces

struct EmbedParams {
    const uint8_t *blob;
    const void *ids;
    void *out;
    uint32_t *status;
    uint64_t n_tokens, n_values, rows, cols, out_stride;
    uint64_t units;                           // work units per row: an upper bound of the sub-streams it meets
    uint32_t chunk_syms, sub_syms, id_bytes, n_stripes, table;
    uint32_t lanes;                           // units per warp and item
    uint64_t total, items;                    // units and items of the call
    float scale;
    // canonical code of the tensor's table: codes of length l take the 12-bit
    // windows [lo[l], hi[l]), in the order of sorted[adj[l] + (window >> (12 - l))];
    // longer codes take the lower windows
    uint16_t lo[K3HUF_MAXLEN + 1], hi[K3HUF_MAXLEN + 1];
    int16_t adj[K3HUF_MAXLEN + 1];
    alignas(4) uint8_t sorted[256];
    uint64_t stripe[kMaxStripes];             // offset of each stripe in the container
    uint64_t last_bytes;                      // container bytes from the last stripe on
};

__device__ __forceinline__ uint32_t bswap32(uint32_t x) { return __byte_perm(x, 0, 0x0123); }

// The canonical code in shared memory (its lookups differ from lane to lane,
// which parameter space would serialise).
struct Code {
    uint32_t lo[K3HUF_MAXLEN + 1], hi[K3HUF_MAXLEN + 1];
    int32_t adj[K3HUF_MAXLEN + 1];
    uint8_t sorted[256];
};

// Barrier 1 of the threads that build tables.
__device__ __forceinline__ void build_sync(uint32_t threads) { asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); }

// Place of entry e in the tables that a build reads.  Neighbouring entries
// mostly start with the same code, of l bits say, so a warp looks entries up
// that lie 2^l apart: straight tables would put up to 32 of them in one bank.
__device__ __forceinline__ uint32_t spread(uint32_t e) { return e ^ (e >> 5 & 31u) ^ (e >> 10); }

// The 12-bit table, entry (symbol << 4) | length; 0 where no code is; also
// spread out, for the builds.  By threads 0 .. n - 1 (n a multiple of 32, at
// least 64); t < n is this one.  The builds take a few entries per thread:
// their dependent lookups are what they cost, so each table is built from the
// one before in one step.
__device__ void build_lut(const EmbedParams &P, Code &code, uint16_t *lut, uint32_t *lut1, uint32_t t, uint32_t n) {
    if (t <= K3HUF_MAXLEN) {
        code.lo[t] = P.lo[t];
        code.hi[t] = P.hi[t];
        code.adj[t] = P.adj[t];
    }
    if (t < 64) reinterpret_cast<uint32_t *>(code.sorted)[t] = reinterpret_cast<const uint32_t *>(P.sorted)[t];
    uint32_t lo[K3HUF_MAXLEN];
#pragma unroll
    for (int k = 1; k < K3HUF_MAXLEN; ++k) lo[k] = P.lo[k];
    build_sync(n);
#pragma unroll 1
    for (uint32_t e = t; e < K3HUF_TABLE_ENTRIES; e += n) {
        uint32_t l = K3HUF_MAXLEN;
#pragma unroll
        for (int k = 1; k < K3HUF_MAXLEN; ++k) l -= e >= lo[k];
        const uint32_t s = (uint32_t(code.sorted[(code.adj[l] + int(e >> (K3HUF_MAXLEN - l))) & 255]) << 4) | l;
        const uint32_t v = e >= code.lo[l] && e < code.hi[l] ? s : 0u;
        lut[e] = uint16_t(v);
        if (lut1) lut1[spread(e)] = v;
    }
    build_sync(n);
}

// The table of up to two codes, spread out: symbols [7:0] and [15:8], the first
// code's bits [19:16], all bits [24:20], bit 25 for two codes; 0 where no code is.
constexpr uint32_t kTwo = 1u << 25;
__device__ void build_lut2(const uint32_t *lut1, uint32_t *lut2, uint32_t t, uint32_t n) {
#pragma unroll 1
    for (uint32_t e = t; e < K3HUF_TABLE_ENTRIES; e += n) {
        const uint32_t a = lut1[spread(e)], l = a & 15u, b = lut1[spread((e << l) & (K3HUF_TABLE_ENTRIES - 1))], m = b & 15u;
        const uint32_t one = (a >> 4) | (l << 16) | (l << 20);
        lut2[spread(e)] = !l ? 0u : m && l + m <= K3HUF_MAXLEN ? (one + (m << 20)) | (b >> 4) << 8 | kTwo : one;
    }
    build_sync(n);
}

// The table of up to four codes, two by two: .x their symbols, .y their bits
// [4:0], eight times their number [15:8], and kBad where no code starts (which
// counts as one symbol 0 of one bit).
constexpr uint32_t kBad = 1u << 31;
__device__ void build_lut4(const uint32_t *lut2, uint2 *lut4, uint32_t t, uint32_t n) {
#pragma unroll 1
    for (uint32_t e = t; e < K3HUF_TABLE_ENTRIES; e += n) {
        const uint32_t a = lut2[spread(e)], l = a >> 20 & 31u, b = lut2[spread((e << l) & (K3HUF_TABLE_ENTRIES - 1))], m1 = b >> 16 & 15u, m = b >> 20 & 31u;
        uint2 f = make_uint2(a & 0xFFFFu, l | (a & kTwo ? 0x1000u : 0x800u));
        if ((a & kTwo) && b) {
            if (l + m <= K3HUF_MAXLEN) f = make_uint2(f.x | (b & 0xFFFFu) << 16, f.y + m + (b & kTwo ? 0x1000u : 0x800u));
            else if (l + m1 <= K3HUF_MAXLEN) f = make_uint2(f.x | (b & 0xFFu) << 16, f.y + m1 + 0x800u);
        }
        lut4[e] = a ? f : make_uint2(0u, kBad | 0x801u);
    }
}

// One sub-stream of one row.
struct Unit {
    const uint8_t *bits, *even;               // the stripe's stream and low bytes
    uint32_t a, len;                          // first value in the stripe, values
    uint32_t off, end;                        // first bit, and the one after the last
    uint32_t huff_bits;
    int64_t col;                              // column of its first value (negative: the row starts inside)
    uint64_t token;
    bool any, none;                           // there is one; its row is zeros
};

// Unit k of token t.  Sets status bits for what it finds wrong.
template <bool kFixed>
__device__ Unit unit_of(const EmbedParams &P, uint64_t t, uint32_t k) {
    Unit q{};
    int64_t id = ld_id(P.ids, P.id_bytes, t);
    q.token = t;
    if (id < 0 || uint64_t(id) >= P.rows) {
        if (id >= 0 && k == 0) atomicOr(P.status, K3HUF_ST_TOKEN);
        q.none = true;                        // (the columns are dealt out as the first row's)
        id = 0;
    }
    const uint32_t cs = kFixed ? 4096u : P.chunk_syms, ss = kFixed ? 256u : P.sub_syms, S = cs / ss;
    const uint32_t full = (K3HUF_STRIPE_VALUES + cs - 1) / cs * S;       // sub-streams of a full stripe
    const uint64_t v0 = uint64_t(id) * P.cols;
    const uint32_t l0 = uint32_t(v0 % K3HUF_STRIPE_VALUES);
    const uint64_t u = v0 / K3HUF_STRIPE_VALUES * full + uint64_t(l0 / cs) * S + l0 % cs / ss + k;
    const uint32_t si = uint32_t(u / full), g = uint32_t(u % full);
    if (si >= P.n_stripes) return q;
    const uint64_t base = uint64_t(si) * K3HUF_STRIPE_VALUES;
    const uint32_t n = uint32_t(min(uint64_t(K3HUF_STRIPE_VALUES), P.n_values - base));
    const uint32_t c = g / S, j = g % S, nch = (n + cs - 1) / cs;
    // this sub-stream's values in the stripe, [a, b), and those of the row
    const uint64_t a = uint64_t(c) * cs + uint64_t(j) * ss;
    uint64_t b = min(min(a + ss, uint64_t(c) * cs + cs), uint64_t(n));
    if (a >= b || base + a >= v0 + P.cols || base + b <= v0) return q;
    q.any = true;
    q.a = uint32_t(a);
    q.len = uint32_t(b - a);
    q.col = int64_t(base + a) - int64_t(v0);
    if (q.none) return q;
    const uint8_t *stripe = P.blob + P.stripe[si];
    const uint4 *hv = reinterpret_cast<const uint4 *>(stripe);
    const uint4 h0 = __ldg(hv), h1 = __ldg(hv + 1);
    // (the index is read along with the header that says whether it is there: it
    // lies inside the stripe by the host's check of the layer header)
    const uint32_t *chunk_off = reinterpret_cast<const uint32_t *>(stripe + K3HUF_STRIPE_HDR_BYTES);
    const uint16_t *sub_off = reinterpret_cast<const uint16_t *>(chunk_off + nch);
    const uint32_t cb = __ldg(chunk_off + c), ce = c + 1 < nch ? __ldg(chunk_off + c + 1) : h1.x;
    const uint32_t sb = j ? uint32_t(__ldg(sub_off + size_t(c) * (S - 1) + j - 1)) : 0u;
    const uint32_t se = j + 1 < S ? uint32_t(__ldg(sub_off + size_t(c) * (S - 1) + j)) : 0u;
    const uint64_t region = si + 1 < P.n_stripes ? P.stripe[si + 1] - P.stripe[si] : P.last_bytes;
    const uint64_t bits_need = ((uint64_t(h1.x) + 7) / 8 + 15) / 16 * 16 + kBitsSlack;
    const uint64_t index = 4ull * nch + 2ull * nch * (S - 1);
    if (h0.x != kStripeMagic || h0.y != P.table || h0.z != n || h0.w != nch || h1.y != 0 ||
        h1.z != (K3HUF_STRIPE_HDR_BYTES + index + 15) / 16 * 16 || h1.w < h1.z + bits_need || h1.w % 16 != 0 || uint64_t(h1.w) + n > region) {
        atomicOr(P.status, K3HUF_ST_HEADER);
        q.none = true;                        // (zeros are written)
        return q;
    }
    q.huff_bits = h1.x;
    q.bits = stripe + h1.z;
    q.even = stripe + h1.w;
    q.off = cb + sb;
    q.end = j + 1 < S ? cb + se : ce;
    return q;
}

// What the join needs of a unit, in shared memory.
struct Join {
    const uint8_t *even;                      // low byte of its first value (null: zeros)
    uint8_t *out;                             // where its first value goes (before the row if it starts inside)
    uint32_t skip, len;                       // its values [skip, len) are the row's
};
static_assert(sizeof(Join) == 24, "");

constexpr size_t kWarpBytes = kPieces * 16 + 32 * kRowWords * 4 + 32 * sizeof(Join);
constexpr size_t kEmbedSmem = K3HUF_TABLE_ENTRIES * (8 + 2) + kWarps * kWarpBytes;
static_assert(kEmbedSmem + sizeof(Code) + 1024 + 64 <= 227 * 1024, "shared memory of one CTA");
static_assert(kWarpBytes % 16 == 0, "16-byte pieces");

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
}

// Eight values: their high bytes (two words) and low bytes, scaled.
__device__ __forceinline__ void scaled8(uint32_t h0, uint32_t h1, uint2 even, float scale, float (&f)[8]) {
    const uint32_t w[4] = {__byte_perm(even.x, h0, 0x5140), __byte_perm(even.x, h0, 0x7362), __byte_perm(even.y, h1, 0x5140), __byte_perm(even.y, h1, 0x7362)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __fmul2_rn(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), make_float2(scale, scale));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
    uint4 o;
    __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    __stcs(reinterpret_cast<uint4 *>(p), o);
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}

// kVec: whole 8-value pieces (rows, sub-streams and output rows all start on them)
template <typename T, bool kFixed, bool kVec>
__global__ void __launch_bounds__(kEmbedThreads, 1) embed_kernel(const __grid_constant__ EmbedParams P) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint2 *lut4 = reinterpret_cast<uint2 *>(smem);
    uint16_t *lut = reinterpret_cast<uint16_t *>(smem + K3HUF_TABLE_ENTRIES * 8);
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint8_t *slot = smem + K3HUF_TABLE_ENTRIES * 10 + warp * kWarpBytes;
    uint32_t *row = reinterpret_cast<uint32_t *>(slot + kPieces * 16);
    Join *join = reinterpret_cast<Join *>(slot + kPieces * 16 + 32 * kRowWords * 4);
    __shared__ Code code;
    __shared__ uint32_t s_next;
    const uint64_t total = P.total, items = P.items;
    auto fetch = [&](uint64_t i) {
        const uint64_t w = i * P.lanes + lane;
        if (i >= items || lane >= P.lanes || w >= total) return Unit{};
        const uint64_t t = total <= 0xFFFFFFFFull ? uint32_t(w) / uint32_t(P.units) : w / P.units;
        return unit_of<kFixed>(P, t, uint32_t(w - t * P.units));
    };
    // the CTA's items are every gridDim.x-th, handed out to its warps one by one
    uint64_t item = blockIdx.x + uint64_t(gridDim.x) * warp;
    if (threadIdx.x == 0) s_next = kWarps;
    // the tables; where only one warp has an item, it looks that up meanwhile
    const bool few = items <= gridDim.x;
    Unit q;
    if (few && warp == 0) {
        q = fetch(item);
    } else {
        const uint32_t n = few ? kEmbedThreads - 32 : kEmbedThreads, t = threadIdx.x - (kEmbedThreads - n);
        if (!few) q = fetch(item);
        // (two more tables lie in the warps' slots, which are not in use yet)
        uint32_t *lut1 = reinterpret_cast<uint32_t *>(smem + K3HUF_TABLE_ENTRIES * 10), *lut2 = lut1 + K3HUF_TABLE_ENTRIES;
        build_lut(P, code, lut, lut1, t, n);
        build_lut2(lut1, lut2, t, n);
        build_lut4(lut2, lut4, t, n);
    }
    __syncthreads();
    if (few && warp > 0) return;
    uint32_t bad = 0;
    while (item < items) {
        // what of the unit is wanted: decoding stops there
        const uint32_t want = q.any ? uint32_t(min(int64_t(q.len), int64_t(P.cols) - q.col)) : 0u;
        const uint32_t skip = q.col < 0 ? uint32_t(-q.col) : 0u;
        join[lane] = Join{q.none ? nullptr : q.even + q.a, static_cast<uint8_t *>(P.out) + (int64_t(q.token * P.out_stride) + q.col) * int64_t(sizeof(T)), skip, want};
        // nothing to check in the join: whole units of rows that are there; and nothing to look up where
        // they follow one another in one row (row_even, row_out: this lane's place in the first of four)
        constexpr uint32_t kSub = 256;
        const bool there = q.any && !q.none && q.col >= 0 && want == (kFixed ? kSub : P.sub_syms);
        // (whole rounds of them: a shorter sub-stream's last round holds less than the 64 values that the join takes)
        const bool plain = __all_sync(0xffffffffu, there) && (kFixed || P.sub_syms % kRound == 0);
        const uint8_t *row_even = nullptr;
        T *row_out = nullptr;
        if (kFixed && kVec) {
            const uint8_t *e = q.even + q.a;
            T *o = static_cast<T *>(P.out) + q.token * P.out_stride + q.col;
            const uint64_t e0 = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(e), 0), o0 = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(o), 0);
            if (__all_sync(0xffffffffu, lane >= P.lanes || (there && reinterpret_cast<uint64_t>(e) == e0 + lane * kSub && reinterpret_cast<uint64_t>(o) == o0 + lane * kSub * sizeof(T)))) {
                row_even = reinterpret_cast<const uint8_t *>(e0) + lane / 8 * kSub + lane % 8 * 8;
                row_out = reinterpret_cast<T *>(o0) + lane / 8 * kSub + lane % 8 * 8;
            }
        }
        const uint32_t live = q.none ? 0u : want;
        // clamped, so that a corrupt index cannot move a read outside the stream
        const uint32_t off = min(q.off, q.huff_bits), end = min(max(q.end, off), q.huff_bits);
        // its 16-byte pieces of the stream, [p0, p1) (a window may reach past the last one, but no code
        // that is taken does; no more than the longest codes would take, and one at least: the
        // stream has 32 bytes past its end)
        const uint32_t p0 = off >> 7, p1 = min(max((end + 127) >> 7, p0 + 1), p0 + (q.len * K3HUF_MAXLEN + 127) / 128 + 1);
        // a unit that goes on where the lane before ends shares that one's last piece
        const uint32_t last_p1 = __shfl_up_sync(0xffffffffu, p1, 1), last_end = __shfl_up_sync(0xffffffffu, end, 1);
        const uint64_t last_bits = __shfl_up_sync(0xffffffffu, live ? reinterpret_cast<uint64_t>(q.bits) : 0ull, 1);
        bool on = live && lane > 0 && last_bits == reinterpret_cast<uint64_t>(q.bits) && last_end == off && last_p1 - p0 <= 1 && p1 >= last_p1;
        uint32_t pieces = 0, before = 0;      // of this lane; of the lanes up to this one
        auto count_pieces = [&]() {
            before = pieces = live ? p1 - (on ? last_p1 : p0) : 0u;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, before, d);
                if (lane >= uint32_t(d)) before += v;
            }
        };
        count_pieces();
        if (__shfl_sync(0xffffffffu, before, 31) > kPieces) {  // several passes: every lane for itself
            on = false;
            count_pieces();
        }
        __syncwarp();
        const uint32_t longest = __reduce_max_sync(0xffffffffu, want);
        uint32_t done = 0, first = 0;         // pieces and lanes of the passes so far
        while (first < 32) {                  // one pass, unless the codes are long
            const uint32_t over = __ballot_sync(0xffffffffu, lane >= first && before - done > kPieces);
            const uint32_t last = over ? uint32_t(__ffs(over)) - 1 : 32u;
            const bool in = lane >= first && lane < last;
            const uint32_t mine = in ? live : 0u;
            const uint32_t at = before - done - pieces;            // where its own pieces start
            // the pass's runs of pieces, each copied by the whole warp
            for (uint32_t heads = __ballot_sync(0xffffffffu, in && live && !on); heads; ) {
                const uint32_t h = __ffs(heads) - 1;
                heads &= heads - 1;
                const uint32_t from = __shfl_sync(0xffffffffu, at, h), to = heads ? __shfl_sync(0xffffffffu, at, (__ffs(heads) - 1) & 31) : __shfl_sync(0xffffffffu, before, last - 1) - done;
                const uint8_t *src = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(q.bits) + uint64_t(p0) * 16, h));
                for (uint32_t p = from + lane; p < to; p += 32) cp_async16(slot + p * 16, src + (p - from) * 16);
            }
            const uint8_t *buf = slot + (in && live ? at - (on ? last_p1 - p0 : 0u) : 0u) * 16;
            const uint32_t most = in && live ? p1 - p0 : 0u;
            asm volatile("cp.async.commit_group;" ::: "memory");
            const bool whole = plain && first == 0 && last == 32;
            if (first > 0 || last < 32) row_even = nullptr;
            // low bytes of a round's pieces: unit 4 i + lane / 8, values 8 (lane % 8) ..
            uint2 even[8];
            auto load_even = [&](uint32_t v0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (4u * i >= P.lanes) break;
                    const uint32_t u = 4 * i + lane / 8, v = v0 + lane % 8 * 8;
                    if (row_even) {
                        even[i] = __ldg(reinterpret_cast<const uint2 *>(row_even + i * (4 * kSub) + v0));
                        continue;
                    }
                    const Join &J = join[u];
                    even[i] = whole || (u >= first && u < last && v < J.len && J.even) ? __ldg(reinterpret_cast<const uint2 *>(J.even + v)) : make_uint2(0, 0);
                }
            };
            if (kVec) load_even(0);
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();                     // (copies by other lanes)

            const uint32_t *words = reinterpret_cast<const uint32_t *>(buf);
            const uint32_t max_word = most ? most * 4 - 1 : 0u;       // (a window's words past it hold no bit that is taken)
            uint32_t cur = off - p0 * 128;    // the next bit, from the buffer's first
            const uint32_t cur0 = cur;
            uint32_t last_window = 0, last_entry = 0;
            // the 64 bits from `cur` on
            auto window = [&](uint32_t &hi, uint32_t &lo) {
                const uint32_t i = cur / 32;
                const uint32_t w0 = bswap32(words[min(i, max_word)]), w1 = bswap32(words[min(i + 1, max_word)]), w2 = bswap32(words[min(i + 2, max_word)]);
                hi = __funnelshift_l(w1, w0, cur);
                lo = __funnelshift_l(w2, w1, cur);
            };
            // high bytes that wait for a whole word: fill bits of them (0, 8, 16 or 24)
            uint32_t acc = 0, fill = 0;
            uint32_t *const my_row = row + lane * kRowWords;
            // (selects, not branches: in most steps some lane fills a word)
            auto take = [&](uint2 e, uint32_t *&to) {
                bad |= e.y;
                const uint32_t more = __funnelshift_l(e.x, 0u, fill);     // what does not fit in the word
                acc |= e.x << fill;
                fill += __byte_perm(e.y, 0u, 0x4441);
                const bool full = fill >= 32;
                if (full) *to = acc;
                to += full;
                acc = full ? more : acc;
                fill &= 31u;
            };
            for (uint32_t r = 0; r < longest; r += kRound) {
                if (r < mine) {
                    // Until 64 values, or the unit's last, are there.  n lookups give 4 n values at most,
                    // so the first ones need no test for the end.  A window holds the bits of four
                    // lookups (48 at most); an entry's low five bits are the shift, and its low byte
                    // adds up.  The last lookup may give up to three values too many, the next round's
                    // first or, past the unit, nobody's
                    uint32_t *to = my_row;
                    const uint32_t stop = min(uint32_t(kRound), mine - r);
                    uint32_t hi = 0, lo = 0;
                    auto look = [&]() {
                        const uint2 e = lut4[hi >> 20];
                        last_window = hi;
                        last_entry = e.y;
                        hi = __funnelshift_l(lo, hi, e.y);
                        lo <<= e.y & 31u;
                        take(e, to);
                        return e.y;
                    };
                    for (uint32_t k = 0; k < stop / 16; ++k) {
                        window(hi, lo);
                        uint32_t sum = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum += look();
                        cur += sum & 255u;
                    }
                    auto more = [&]() { return uint32_t(to - my_row) * 4 + fill / 8 < stop; };
                    while (more()) {
                        window(hi, lo);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (i && !more()) break;
                            cur += look() & 31u;
                        }
                    }
                    if (r + kRound >= mine) {
                        if (to < my_row + kRowWords) *to = acc;            // a partial word
                        // the bits of the values too many do not count
                        uint32_t codes = (last_entry >> 11 & 31u) - (uint32_t(to - my_row) * 4 + fill / 8 - stop);
                        cur -= last_entry & 31u;
                        for (; codes; --codes) {
                            const uint32_t l = max(lut[last_window >> 20] & 15u, 1u);
                            last_window <<= l;
                            cur += l;
                        }
                    }
                }
                __syncwarp();
                // the join
                if constexpr (kVec) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (4u * i >= P.lanes) break;
                        const uint32_t u = 4 * i + lane / 8, s8 = lane % 8, v = r + s8 * 8;
                        const uint32_t *h = row + u * kRowWords + 2 * s8;
                        float f[8];
                        if (row_even) {
                            scaled8(h[0], h[1], even[i], P.scale, f);
                            store8(row_out + i * (4 * kSub) + r, f);
                            continue;
                        }
                        const Join &J = join[u];
                        if (whole || (u >= first && u < last && v >= J.skip && v < J.len)) {
                            if (whole || J.even) scaled8(h[0], h[1], even[i], P.scale, f);
                            else
#pragma unroll
                                for (int k = 0; k < 8; ++k) f[k] = 0.f;
                            store8(reinterpret_cast<T *>(J.out) + v, f);
                        }
                    }
                    if (r + kRound < longest) load_even(r + kRound);
                } else {
                    for (uint32_t u = first; u < min(last, P.lanes); ++u) {
                        const Join J = join[u];
#pragma unroll
                        for (int i = 0; i < kRound / 32; ++i) {
                            const uint32_t s = i * 32 + lane, v = r + s;
                            if (v >= J.skip && v < J.len) {
                                float f = 0.f;
                                if (J.even) f = P.scale * __uint_as_float((uint32_t(reinterpret_cast<const uint8_t *>(row + u * kRowWords)[s]) << 24) | (uint32_t(__ldg(J.even + v)) << 16));
                                st_f32(reinterpret_cast<T *>(J.out) + v, f);
                            }
                        }
                    }
                }
                __syncwarp();
            }
            // a whole sub-stream ends where the next one begins
            const uint32_t past = off + (cur - cur0);
            if (mine && mine == q.len && past != q.end) bad |= past > q.huff_bits ? kBad >> 1 : kBad >> 2;
            first = last;
            done = __shfl_sync(0xffffffffu, before, last - 1);
        }
        __syncwarp();
        uint32_t k = lane == 0 ? atomicAdd(&s_next, 1u) : 0u;
        item = blockIdx.x + uint64_t(gridDim.x) * __shfl_sync(0xffffffffu, k, 0);
        q = fetch(item);
    }
    const uint32_t found = (bad & kBad ? K3HUF_ST_BADCODE : 0u) | (bad & kBad >> 1 ? K3HUF_ST_OVERRUN : 0u) | (bad & kBad >> 2 ? K3HUF_ST_INDEX : 0u);
    if (found) atomicOr(P.status, found);
}

// Containers with sub-streams longer than kMaxStagedSub: one thread decodes
// one of them straight from global memory, a symbol per lookup.
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_long_kernel(const __grid_constant__ EmbedParams P) {
    __shared__ uint16_t lut[K3HUF_TABLE_ENTRIES];
    __shared__ Code code;
    build_lut(P, code, lut, nullptr, threadIdx.x, kThreads);
    const uint64_t w = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (w >= P.n_tokens * P.units) return;
    const uint64_t t = w / P.units;
    const Unit q = unit_of<false>(P, t, uint32_t(w - t * P.units));
    if (!q.any) return;
    T *out = static_cast<T *>(P.out) + q.token * P.out_stride;
    const uint32_t want = uint32_t(min(int64_t(q.len), int64_t(P.cols) - q.col));
    const uint32_t *words = reinterpret_cast<const uint32_t *>(q.bits);
    uint32_t pos = q.off, bad = 0;
    for (uint32_t v = 0; v < want; ++v) {
        float f = 0.f;
        if (!q.none) {
            // (the stream is followed by 32 zero bytes, so word huff_bits / 32 + 1 is inside)
            const uint32_t p = min(pos, q.huff_bits);
            const uint32_t e = lut[__funnelshift_l(bswap32(words[p / 32 + 1]), bswap32(words[p / 32]), p) >> 20];
            if (!(e & 15u)) bad = K3HUF_ST_BADCODE;
            pos += max(e & 15u, 1u);
            f = P.scale * __uint_as_float(((e >> 4) << 24) | (uint32_t(q.even[q.a + v]) << 16));
        }
        if (q.col + int64_t(v) >= 0) st_f32(out + q.col + int64_t(v), f);
    }
    if (!q.none && want == q.len && pos != q.end) bad |= pos > q.huff_bits ? K3HUF_ST_OVERRUN : K3HUF_ST_INDEX;
    if (bad) atomicOr(P.status, bad);
}

template <typename T, bool kFixed, bool kVec>
int launch_embed(const EmbedParams &P, uint32_t grid, cudaStream_t stream) {
    static std::atomic<uint64_t> once{0};
    const int rc = once_per_device(once, [] { return cudaFuncSetAttribute(embed_kernel<T, kFixed, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kEmbedSmem)); });
    if (rc) return rc;
    embed_kernel<T, kFixed, kVec><<<grid, kEmbedThreads, kEmbedSmem, stream>>>(P);
    return cuda_rc(cudaGetLastError());
}

template <typename T>
int launch_rows(EmbedParams &P, cudaStream_t stream) {
    const uint64_t total = P.total = P.n_tokens * P.units;
    if (P.sub_syms > kMaxStagedSub) {
        const uint64_t blocks = (total + kThreads - 1) / kThreads;
        if (blocks > 0x7FFFFFFFull) return K3HUF_E_ARG;
        embed_long_kernel<T><<<uint32_t(blocks), kThreads, 0, stream>>>(P);
        return cuda_rc(cudaGetLastError());
    }
    // units per item: 32, fewer while every warp of the GPU still gets one item at most (a warp's
    // latency then counts, not its instructions: 4000 rows of 577 values 30 us, 54 with 32 units
    // per item; 2000 and 8000 rows of 8192 values are the same 27 and 63 us, since they keep 32)
    uint64_t sms = 0;
    const int rc = sm_count(&sms);
    if (rc) return rc;
    P.lanes = 32;
    while (P.lanes > 4 && total <= P.lanes / 2 * sms * kWarps) P.lanes /= 2;
    P.items = (total + P.lanes - 1) / P.lanes;
    const uint32_t grid = uint32_t(std::min<uint64_t>(sms, P.items));
    const bool fixed = P.chunk_syms == 4096 && P.sub_syms == 256;
    const bool vec = P.cols % 8 == 0 && P.sub_syms % 8 == 0 && aligned_to(P.out, 16) && P.out_stride * sizeof(T) % 16 == 0;
    if (fixed) return vec ? launch_embed<T, true, true>(P, grid, stream) : launch_embed<T, true, false>(P, grid, stream);
    return vec ? launch_embed<T, false, true>(P, grid, stream) : launch_embed<T, false, false>(P, grid, stream);
}

// --- the gradient ---------------------------------------------------------------
//
// Blocks of up to kBlock tokens.  A CTA sorts a block's tokens by id in shared
// memory (stable, so equal ids keep the tokens' order), while the other CTAs of
// the launch write the zeros of a gradient that is not accumulated.  The second
// launch adds up each id's rows: a warp per id and 1024 columns (256 of narrow
// tables), 16 bytes per lane and load, eight of them in flight, or, for an id
// with more than kHeavy tokens, a CTA per 256 columns whose warps take a share of
// the tokens each and meet in shared memory.
// One such launch per block, in order, so that every sum has one order.  Bound
// by the write of the gradient, or by the read of dY and the rows that it meets:
// 8192 tokens x 8192 bf16 into 32768 rows, zeros 157 us (6.8 TB/s), sums 67 us.
constexpr uint32_t kBlock = 16384, kSortThreads = 1024, kHeavy = 32, kDigit = 9;
constexpr uint32_t kItems = kBlock / kSortThreads;
constexpr uint32_t kSumThreads = 256, kHeavyCols = 256;
constexpr size_t kSortSmem = kBlock * (4 + 2) + (kSortThreads / 32) * (1u << kDigit) * 2;

// A block's outcome in the scratch.
struct Sorted {
    uint32_t ids, heavy, pad[62];             // numbers of distinct ids and of those with many tokens
    uint32_t order[kBlock];                   // tokens by id
    uint32_t id[kBlock], start[kBlock + 1];   // each id and its first place in `order`; start[ids] is the end
    uint32_t many[kBlock / kHeavy];           // places in `id` of those with many tokens
    uint32_t pad1[63];
};
static_assert(sizeof(Sorted) % 256 == 0, "");

struct GradSortParams {
    const void *ids;
    Sorted *out;
    float4 *zero;                             // gradient to zero, or null
    uint64_t zero_vecs, n, rows;
    uint32_t *status;
    uint32_t id_bytes, blocks, bits;          // bits of a key: the id, or `rows` for none
};

__global__ void __launch_bounds__(kSortThreads) grad_sort_kernel(const GradSortParams P) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t s_base[1u << kDigit], s_warp[kSortThreads / 32 + 1], s_heavy;
    grid_dep_launch();
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (blockIdx.x >= P.blocks) {
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
        // (four vectors per thread and step)
        for (uint64_t i = uint64_t(blockIdx.x - P.blocks) * (4 * kSortThreads) + tid; i < P.zero_vecs; i += uint64_t(gridDim.x - P.blocks) * (4 * kSortThreads))
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
                if (i + k * kSortThreads < P.zero_vecs) __stcs(P.zero + i + k * kSortThreads, none);
        return;
    }
    uint32_t *keys = reinterpret_cast<uint32_t *>(smem);
    uint16_t *places = reinterpret_cast<uint16_t *>(smem + kBlock * 4);
    uint16_t(*hist)[1u << kDigit] = reinterpret_cast<uint16_t(*)[1u << kDigit]>(smem + kBlock * 6);
    const uint64_t t0 = uint64_t(blockIdx.x) * kBlock;
    const uint32_t n = uint32_t(min(uint64_t(kBlock), P.n - t0));
    Sorted &out = P.out[blockIdx.x];
    // item k of a thread is number (warp * items + k) * 32 + lane: warps hold runs
    const uint32_t items = (n + kSortThreads - 1) / kSortThreads;
    uint32_t key[kItems], place[kItems];
#pragma unroll
    for (uint32_t k = 0; k < kItems; ++k) {
        const uint32_t i = (warp * items + k) * 32 + lane;
        key[k] = 0xFFFFFFFFu;                 // (past the block: after everything)
        place[k] = i;
        if (k < items && i < n) {
            const int64_t id = ld_id(P.ids, P.id_bytes, t0 + i);
            key[k] = id >= 0 && uint64_t(id) < P.rows ? uint32_t(id) : uint32_t(P.rows);
            if (id >= 0 && uint64_t(id) >= P.rows) atomicOr(P.status, K3HUF_ST_TOKEN);
        }
    }
    // sums over the CTA's threads before this one
    auto before = [&](uint32_t v, uint32_t &total) {
        uint32_t incl = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= uint32_t(d)) incl += o;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            const uint32_t w = s_warp[lane];
            uint32_t all = w;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, all, d);
                if (lane >= uint32_t(d)) all += o;
            }
            s_warp[lane] = all - w;
            if (lane == 31) s_warp[32] = all;
        }
        __syncthreads();
        total = s_warp[32];
        return s_warp[warp] + incl - v;
    };
    const uint32_t passes = (P.bits + kDigit - 1) / kDigit, width = (P.bits + passes - 1) / passes, bins = 1u << width;
    for (uint32_t pass = 0; pass < passes; ++pass) {
        // places within the warp's items of equal digit, in order
        uint32_t rank[kItems];
        for (uint32_t d = lane; d < bins; d += 32) hist[warp][d] = 0;
        __syncwarp();
#pragma unroll
        for (uint32_t k = 0; k < kItems; ++k) {
            if (k >= items) break;
            const uint32_t d = key[k] >> (pass * width) & (bins - 1);
            // lanes of the same digit, bit by bit
            uint32_t same = 0xffffffffu;
            for (uint32_t b = 0; b < width; ++b) {
                const uint32_t ones = __ballot_sync(0xffffffffu, d >> b & 1u);
                same &= d >> b & 1u ? ones : ~ones;
            }
            const uint32_t below = __popc(same & ((1u << lane) - 1u)), had = hist[warp][d];
            __syncwarp();
            if (below == 0) hist[warp][d] = uint16_t(had + __popc(same));
            __syncwarp();
            rank[k] = had + below;
        }
        __syncthreads();
        // counts to first places: by digit, then by warp
        uint32_t mine = 0;
        if (tid < bins)
            for (uint32_t w0 = 0; w0 < kSortThreads / 32; w0 += 16) {
                uint16_t c[16];               // (all loads before the stores, which could be to the same place for all the compiler knows)
#pragma unroll
                for (uint32_t w = 0; w < 16; ++w) c[w] = hist[w0 + w][tid];
#pragma unroll
                for (uint32_t w = 0; w < 16; ++w) {
                    hist[w0 + w][tid] = uint16_t(mine);
                    mine += c[w];
                }
            }
        uint32_t total;
        const uint32_t first = before(mine, total);
        if (tid < bins) s_base[tid] = first;
        __syncthreads();
#pragma unroll
        for (uint32_t k = 0; k < kItems; ++k) {
            if (k >= items) break;
            const uint32_t d = key[k] >> (pass * width) & (bins - 1), to = s_base[d] + hist[warp][d] + rank[k];
            keys[to] = key[k];
            places[to] = uint16_t(place[k]);
        }
        __syncthreads();
#pragma unroll
        for (uint32_t k = 0; k < kItems; ++k) {
            if (k >= items) break;
            const uint32_t i = (warp * items + k) * 32 + lane;
            key[k] = keys[i];
            place[k] = places[i];
        }
    }
    // the distinct ids, in order: each warp looks at its items' places, 32 at a time
    if (tid == 0) s_heavy = 0;
    uint32_t heads = 0;
    for (uint32_t k = 0; k < items; ++k) {
        const uint32_t i = (warp * items + k) * 32 + lane;
        heads += __popc(__ballot_sync(0xffffffffu, i < n && keys[i] < P.rows && (i == 0 || keys[i - 1] != keys[i])));
    }
    uint32_t total;
    uint32_t at = before(lane == 0 ? heads : 0u, total);       // (lane 0's: the warps before)
    at = __shfl_sync(0xffffffffu, at, 0);
    for (uint32_t k = 0; k < items; ++k) {
        const uint32_t i = (warp * items + k) * 32 + lane;
        const bool valid = i < n && keys[i] < P.rows, head = valid && (i == 0 || keys[i - 1] != keys[i]);
        const uint32_t all = __ballot_sync(0xffffffffu, head);
        if (i < n) out.order[i] = places[i];
        if (head) {
            const uint32_t u = at + __popc(all & ((1u << lane) - 1u));
            out.id[u] = keys[i];
            out.start[u] = i;
            // (equal keys are adjacent: more than kHeavy of them reach kHeavy places on)
            if (i + kHeavy < n && keys[i + kHeavy] == keys[i]) out.many[atomicAdd(&s_heavy, 1u)] = u;
        }
        if (valid && (i + 1 == n || keys[i + 1] >= P.rows)) out.start[total] = i + 1;
        at += __popc(all);
    }
    __syncthreads();
    if (tid == 0) {
        out.ids = total;
        out.heavy = s_heavy;
    }
}

struct GradSumParams {
    const Sorted *block;
    const void *dy;                           // the block's first token's row
    float *grad;
    uint64_t dy_stride, cols;
    uint32_t slabs, heavy_slabs, heavy_blocks;             // of a warp's columns; of kHeavyCols; CTAs for ids with many tokens
    float scale;
    bool add;
};

// Eight adjacent columns of a row as they were loaded: 16-byte loads (kVec), or fp32 values one by one.
template <typename T, bool kVec> struct Row8 {
    static constexpr int words = kVec && sizeof(T) == 2 ? 4 : 8;
    uint32_t w[words];
    __device__ __forceinline__ void load(const T *p, uint64_t left) {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < words / 4; ++i) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = uint64_t(i) < left ? __float_as_uint(ld_f32(p + i)) : 0u;
        }
    }
    __device__ __forceinline__ void add_to(float (&acc)[8]) const {
#pragma unroll
        for (int i = 0; i < words; ++i) {
            if constexpr (words == 4) {
                acc[2 * i] += __uint_as_float(w[i] << 16);
                acc[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                acc[i] += __uint_as_float(w[i]);
            }
        }
    }
};
template <bool kVec>
__device__ __forceinline__ void put8(float *g, uint64_t left, const float (&v)[8], float scale, bool add) {
    if constexpr (kVec) {
        float4 *q = reinterpret_cast<float4 *>(g);
        float4 a = make_float4(scale * v[0], scale * v[1], scale * v[2], scale * v[3]), b = make_float4(scale * v[4], scale * v[5], scale * v[6], scale * v[7]);
        if (add) {
            const float4 x = q[0], y = q[1];
            a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w, b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
        }
        q[0] = a;
        q[1] = b;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (uint64_t(i) < left) g[i] = add ? g[i] + scale * v[i] : scale * v[i];
    }
}

// Adds up rows `token(j)` of dy for j in [j0, j1), in order, kVecs vectors of eight
// columns per lane: 32 tokens' numbers are fetched at once, and 8 / kVecs rows are
// in flight together.
template <typename T, bool kVec, int kVecs, typename F>
__device__ __forceinline__ void add_rows(const T *dy, uint64_t stride, uint64_t c0, uint64_t cols, uint32_t j0, uint32_t j1, F token, float (&acc)[kVecs][8]) {
    constexpr uint32_t kRows = 8 / kVecs;
    const uint32_t lane = threadIdx.x % 32;
    for (uint32_t j = j0; j < j1; j += 32) {
        const uint32_t mine = j + lane < j1 ? token(j + lane) : 0u, n = min(32u, j1 - j);
        for (uint32_t k = 0; k < n; k += kRows) {
            Row8<T, kVec> rows[kRows][kVecs] = {};
#pragma unroll
            for (uint32_t r = 0; r < kRows; ++r) {
                const uint32_t t = __shfl_sync(0xffffffffu, mine, (k + r) & 31u);
#pragma unroll
                for (int v = 0; v < kVecs; ++v) {
                    const uint64_t c = c0 + v * 256;
                    if (k + r < n && c < cols) rows[r][v].load(dy + t * stride + c, cols - c);
                }
            }
#pragma unroll
            for (uint32_t r = 0; r < kRows; ++r)
#pragma unroll
                for (int v = 0; v < kVecs; ++v) rows[r][v].add_to(acc[v]);
        }
    }
}

// kVecs: vectors of eight columns per lane and id
template <typename T, bool kVec, int kVecs>
__global__ void __launch_bounds__(kSumThreads) grad_sum_kernel(const GradSumParams P) {
    __shared__ float s_part[kSumThreads / 32][kHeavyCols];
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Sorted &S = *P.block;
    const T *dy = static_cast<const T *>(P.dy);
    grid_dep_launch();
    grid_dep_wait();
    if (blockIdx.x < P.heavy_blocks) {
        const uint32_t h = blockIdx.x / P.heavy_slabs;
        if (h >= S.heavy) return;
        const uint32_t u = S.many[h], begin = S.start[u], count = S.start[u + 1] - begin;
        const uint64_t c = uint64_t(blockIdx.x % P.heavy_slabs) * kHeavyCols + lane * 8;
        const uint64_t left = c < P.cols ? P.cols - c : 0;
        float sum[1][8] = {};
        add_rows<T, kVec, 1>(dy, P.dy_stride, c, P.cols, begin + uint32_t(uint64_t(count) * warp / 8), begin + uint32_t(uint64_t(count) * (warp + 1) / 8), [&](uint32_t j) { return S.order[j]; }, sum);
        float(&acc)[8] = sum[0];
#pragma unroll
        for (int i = 0; i < 8; ++i) s_part[warp][i * 32 + lane] = acc[i];
        __syncthreads();
        if (warp == 0 && left) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float sum = 0.f;
                for (uint32_t w = 0; w < kSumThreads / 32; ++w) sum += s_part[w][i * 32 + lane];
                acc[i] = sum;
            }
            put8<kVec>(P.grad + uint64_t(S.id[u]) * P.cols + c, left, acc, P.scale, P.add);
        }
        return;
    }
    const uint64_t unit = uint64_t(blockIdx.x - P.heavy_blocks) * (kSumThreads / 32) + warp;
    const uint64_t u = unit / P.slabs;
    if (u >= S.ids) return;
    const uint32_t begin = S.start[u], end = S.start[u + 1];
    if (end - begin > kHeavy) return;
    const uint64_t c0 = unit % P.slabs * (256 * kVecs) + lane * 8;
    float *g = P.grad + uint64_t(S.id[u]) * P.cols;
    float acc[kVecs][8] = {};
    add_rows<T, kVec, kVecs>(dy, P.dy_stride, c0, P.cols, begin, end, [&](uint32_t j) { return S.order[j]; }, acc);
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
        if (c0 + k * 256 < P.cols) put8<kVec>(g + c0 + k * 256, P.cols - (c0 + k * 256), acc[k], P.scale, P.add);
}

// Up to kFewTokens tokens, without a sort: a CTA per token and 2048 columns
// compares its id with all others; the id's first token's CTA adds up all of
// them, a warp per 256 columns, eight tokens' loads in flight.
constexpr uint32_t kFewTokens = 1024;
struct GradFewParams {
    const void *ids, *dy;
    float *grad;
    uint32_t *status;
    uint64_t dy_stride, rows, cols;
    uint32_t n, id_bytes;
    float scale;
    bool add;
};
template <typename T, bool kVec>
__global__ void __launch_bounds__(kSumThreads) grad_few_kernel(const GradFewParams P) {
    __shared__ uint32_t s_same[kFewTokens / 32];
    __shared__ uint16_t s_token[kFewTokens];
    const uint32_t t = blockIdx.x, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t id = ld_id(P.ids, P.id_bytes, t);
    if (id < 0 || uint64_t(id) >= P.rows) {
        if (id >= 0 && tid == 0 && blockIdx.y == 0) atomicOr(P.status, K3HUF_ST_TOKEN);
        return;
    }
    int earlier = 0;
#pragma unroll
    for (uint32_t k = 0; k < kFewTokens / kSumThreads; ++k) {
        const uint32_t u = k * kSumThreads + tid;
        const bool same = u < P.n && ld_id(P.ids, P.id_bytes, u) == id;
        earlier |= same && u < t;
        const uint32_t m = __ballot_sync(0xffffffffu, same);
        if (lane == 0) s_same[k * (kSumThreads / 32) + warp] = m;
    }
    if (__syncthreads_or(earlier)) return;
    // the tokens in order: word `lane` of the matches goes behind the words before it
    const uint32_t mine = s_same[lane];
    uint32_t at = __popc(mine);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, at, d);
        if (lane >= uint32_t(d)) at += v;
    }
    const uint32_t count = __shfl_sync(0xffffffffu, at, 31);
    if (warp == 0) {
        at -= __popc(mine);
        for (uint32_t m = mine; m; m &= m - 1) s_token[at++] = uint16_t(lane * 32 + __ffs(m) - 1);
    }
    __syncthreads();
    const uint64_t c = uint64_t(blockIdx.y) * 2048 + warp * 256 + lane * 8;
    float acc[1][8] = {};
    add_rows<T, kVec, 1>(static_cast<const T *>(P.dy), P.dy_stride, c, P.cols, 0, count, [&](uint32_t j) { return uint32_t(s_token[j]); }, acc);
    if (c < P.cols) put8<kVec>(P.grad + uint64_t(id) * P.cols + c, P.cols - c, acc[0], P.scale, P.add);
}

// Fewer than four gradient elements, or an address that is not 16-byte aligned: the zeros that
// whole vectors leave out.
__global__ void zero_kernel(float *g, uint64_t n) {
    for (uint64_t i = uint64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += uint64_t(gridDim.x) * blockDim.x) g[i] = 0.f;
}

template <typename T>
int launch_grad(const void *d_ids, uint32_t id_bytes, uint64_t n, const T *dy, uint64_t dy_stride, uint64_t rows, uint64_t cols, float scale, float *grad, Sorted *sorted,
                uint32_t *status, bool add, cudaStream_t stream) {
    static std::atomic<uint64_t> once{0};
    int rc = once_per_device(once, [] { return cudaFuncSetAttribute(grad_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSortSmem)); });
    if (rc) return rc;
    uint64_t sms = 0;
    rc = sm_count(&sms);
    if (rc) return rc;
    const bool vec = cols % 8 == 0 && aligned_to(dy, 16) && dy_stride * sizeof(T) % 16 == 0 && aligned_to(grad, 16);
    const bool few = n <= kFewTokens;
    GradSortParams Q{};
    Q.ids = d_ids, Q.out = sorted, Q.n = n, Q.rows = rows, Q.status = status, Q.id_bytes = id_bytes;
    Q.blocks = few ? 0 : uint32_t((n + kBlock - 1) / kBlock);
    for (Q.bits = 1; (rows >> Q.bits) != 0; ++Q.bits) {}
    uint32_t zero_blocks = 0;
    if (!add) {
        const uint64_t all = rows * cols, vecs = aligned_to(grad, 16) ? all / 4 : 0;
        Q.zero = reinterpret_cast<float4 *>(grad);
        Q.zero_vecs = vecs;
        zero_blocks = uint32_t(std::min<uint64_t>(sms, (vecs + kSortThreads - 1) / kSortThreads));
        if (vecs * 4 < all) {
            zero_kernel<<<uint32_t(std::min<uint64_t>(8 * sms, (all - vecs * 4 + 255) / 256)), 256, 0, stream>>>(grad + vecs * 4, all - vecs * 4);
            rc = cuda_rc(cudaGetLastError());
            if (rc) return rc;
        }
    }
    if (Q.blocks + zero_blocks) {
        grad_sort_kernel<<<Q.blocks + zero_blocks, kSortThreads, kSortSmem, stream>>>(Q);
        rc = cuda_rc(cudaGetLastError());
    }
    if (few && n && !rc) {
        const GradFewParams F{d_ids, dy, grad, status, dy_stride, rows, cols, uint32_t(n), id_bytes, scale, add};
        const dim3 grid(uint32_t(n), uint32_t((cols + 2047) / 2048));
        if (vec) grad_few_kernel<T, true><<<grid, kSumThreads, 0, stream>>>(F);
        else grad_few_kernel<T, false><<<grid, kSumThreads, 0, stream>>>(F);
        rc = cuda_rc(cudaGetLastError());
    }
    for (uint32_t b = 0; b < Q.blocks && !rc; ++b) {
        const uint64_t size = std::min<uint64_t>(kBlock, n - uint64_t(b) * kBlock);
        GradSumParams P{};
        P.block = sorted + b;
        P.dy = dy + uint64_t(b) * kBlock * dy_stride;
        P.grad = grad, P.dy_stride = dy_stride, P.cols = cols, P.scale = scale, P.add = add || b > 0;
        const bool wide = cols > 1024;
        P.slabs = uint32_t((cols + (wide ? 1023 : 255)) / (wide ? 1024 : 256));
        P.heavy_slabs = uint32_t((cols + kHeavyCols - 1) / kHeavyCols);
        const uint64_t heavy = size / (kHeavy + 1) * P.heavy_slabs, light = (std::min(size, rows) * P.slabs + kSumThreads / 32 - 1) / (kSumThreads / 32);
        P.heavy_blocks = uint32_t(heavy);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(uint32_t(heavy + light));
        cfg.blockDim = dim3(kSumThreads);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        rc = cuda_rc(vec ? cudaLaunchKernelEx(&cfg, wide ? grad_sum_kernel<T, true, 4> : grad_sum_kernel<T, true, 1>, P)
                         : cudaLaunchKernelEx(&cfg, wide ? grad_sum_kernel<T, false, 4> : grad_sum_kernel<T, false, 1>, P));
    }
    return rc;
}

}  // namespace
}  // namespace k3huf

using namespace k3huf;

extern "C" int k3huf_embed_layer(const void *h_layer_hdr, size_t hdr_bytes, const void *d_layer, size_t layer_bytes,
                                 uint32_t tensor, uint64_t cols, const void *d_ids, uint32_t id_bytes, uint64_t n_tokens,
                                 float scale, void *d_out, uint32_t out_type, uint64_t out_stride, uint32_t *d_status,
                                 void *stream) {
    if (!h_layer_hdr || !d_layer || !d_status || cols == 0 || (id_bytes != 4 && id_bytes != 8) || !elem_ok(out_type))
        return K3HUF_E_ARG;
    if (!aligned_to(d_layer, 16) || !aligned_to(d_status, 4) || !aligned_to(d_ids, id_bytes) || !aligned_to(d_out, elem_bytes(out_type)))
        return K3HUF_E_ARG;
    Layer L;
    try {
        const int rc = parse_layer(h_layer_hdr, hdr_bytes, &L);
        if (rc) return rc;
    } catch (...) {
        return K3HUF_E_NOMEM;
    }
    if (layer_bytes < L.info.blob_bytes || tensor >= L.tensors.size()) return K3HUF_E_ARG;
    const TensorEntry &te = L.tensors[tensor];
    if (te.n_values % cols != 0 || te.n_stripes > uint32_t(kMaxStripes) || out_stride < cols || cols >= (1ull << 31)) return K3HUF_E_ARG;
    if (n_tokens == 0) return K3HUF_OK;
    if (!d_ids || !d_out || n_tokens > (1ull << 31)) return K3HUF_E_ARG;
    EmbedParams P{};
    P.blob = static_cast<const uint8_t *>(d_layer);
    P.ids = d_ids;
    P.out = d_out;
    P.status = d_status;
    P.n_tokens = n_tokens;
    P.n_values = te.n_values;
    P.rows = te.n_values / cols;
    P.cols = cols;
    P.out_stride = out_stride;
    // (a chunk is no longer than its stripe: the same layout, and sums with it stay in 32 bits; such chunks
    // are one sub-stream each)
    P.chunk_syms = std::min(L.info.chunk_syms, K3HUF_STRIPE_VALUES);
    P.sub_syms = std::min(L.info.sub_syms, P.chunk_syms);
    P.id_bytes = id_bytes;
    P.n_stripes = te.n_stripes;
    P.table = te.table;
    P.scale = scale;
    const uint32_t cs = P.chunk_syms, ss = P.sub_syms, S = cs / ss;
    // sub-streams that a row can meet: whole ones where rows start on them;
    // a stripe whose last chunk is short counts that chunk's S in full
    P.units = cols % ss == 0 && K3HUF_STRIPE_VALUES % cs == 0 ? cols / ss : (cols - 1) / ss + 2;
    if (K3HUF_STRIPE_VALUES % cs != 0) P.units += (cols / K3HUF_STRIPE_VALUES + 1) * (S + 1);
    uint32_t code[256], first[K3HUF_MAXLEN + 1], count[K3HUF_MAXLEN + 1];
    const uint8_t *len = L.tables + 256ull * te.table;
    canonical_codes(len, code, first, count);
    int at[K3HUF_MAXLEN + 1], off = 0;
    for (int l = 1; l <= K3HUF_MAXLEN; ++l) {
        P.lo[l] = uint16_t(first[l] << (K3HUF_MAXLEN - l));
        P.hi[l] = uint16_t((first[l] + count[l]) << (K3HUF_MAXLEN - l));
        P.adj[l] = int16_t(off - int(first[l]));
        at[l] = off;
        off += int(count[l]);
    }
    for (int s = 0; s < 256; ++s)
        if (len[s]) P.sorted[at[len[s]]++] = uint8_t(s);
    for (uint32_t s = 0; s < te.n_stripes; ++s) P.stripe[s] = L.stripes[te.first_stripe + s].blob_offset;
    P.last_bytes = L.info.blob_bytes - P.stripe[te.n_stripes - 1];
    if (P.units > 0xFFFFFFFFull || n_tokens > (1ull << 62) / P.units) return K3HUF_E_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return out_type == K3HUF_BF16 ? launch_rows<__nv_bfloat16>(P, st) : launch_rows<float>(P, st);
}

extern "C" int k3huf_embed_grad_scratch_bytes(uint64_t n_tokens, uint64_t rows, uint64_t cols, size_t *scratch_bytes) {
    if (!scratch_bytes || rows == 0 || rows >= (1ull << 31) || cols == 0 || cols > (1ull << 26) || n_tokens > 0x7FFFFFFFull) return K3HUF_E_ARG;
    *scratch_bytes = std::max<uint64_t>(1, (n_tokens + kBlock - 1) / kBlock) * sizeof(Sorted);
    return K3HUF_OK;
}

extern "C" int k3huf_embed_grad(const void *d_ids, uint32_t id_bytes, uint64_t n_tokens, const void *d_dy, uint32_t dy_type,
                                uint64_t dy_stride, uint64_t rows, uint64_t cols, float scale, float *d_grad, void *d_scratch,
                                size_t scratch_bytes, uint32_t *d_status, uint32_t flags, void *stream) {
    size_t need = 0;
    if (k3huf_embed_grad_scratch_bytes(n_tokens, rows, cols, &need) || (id_bytes != 4 && id_bytes != 8) || !elem_ok(dy_type) ||
        !d_grad || !d_status || !d_scratch || scratch_bytes < need || dy_stride < cols || (flags & ~uint32_t(K3HUF_ACCUMULATE)))
        return K3HUF_E_ARG;
    if (!aligned_to(d_grad, 4) || !aligned_to(d_status, 4) || !aligned_to(d_scratch, 256) || !aligned_to(d_ids, id_bytes) ||
        !aligned_to(d_dy, elem_bytes(dy_type)) || n_tokens > 0x7FFFFFFFull || (n_tokens && (!d_ids || !d_dy)))
        return K3HUF_E_ARG;
    if (n_tokens == 0 && (flags & K3HUF_ACCUMULATE)) return K3HUF_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool add = (flags & K3HUF_ACCUMULATE) != 0;
    Sorted *sorted = static_cast<Sorted *>(d_scratch);
    if (dy_type == K3HUF_BF16)
        return launch_grad(d_ids, id_bytes, n_tokens, static_cast<const __nv_bfloat16 *>(d_dy), dy_stride, rows, cols, scale, d_grad, sorted, d_status, add, st);
    return launch_grad(d_ids, id_bytes, n_tokens, static_cast<const float *>(d_dy), dy_stride, rows, cols, scale, d_grad, sorted, d_status, add, st);
}
