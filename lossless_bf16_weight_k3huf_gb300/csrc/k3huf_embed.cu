// Rows of a coded embedding table, scaled, and the gradient of such a lookup
// with respect to the table.
//
//   out[t, c] = s * W[ids[t], c]
//   G[v, c]   = s * sum over t with ids[t] = v of dY[t, c]
//
// Lookup: the container's chunk and sub-stream indexes give the first bit of
// every run of sub_syms values, so the sub-streams that a row meets are
// decoded and no others.  One thread decodes one sub-stream of one row, from
// its recorded offset, a symbol per table lookup.
#include <algorithm>

#include "k3huf_ops.h"

namespace k3huf {
namespace {

constexpr int kMaxStripes = 256;              // stripes of the tensor (kernel parameter space)
constexpr int kThreads = 128;

struct EmbedParams {
    const uint8_t *blob;
    const void *ids;
    void *out;
    uint32_t *status;
    uint64_t n_tokens, n_values, rows, cols, out_stride;
    uint64_t units;                           // work units per row: an upper bound of the sub-streams it meets
    uint32_t chunk_syms, sub_syms, id_bytes, n_stripes, table;
    float scale;
    // canonical code of the tensor's table: codes of length l take the 12-bit
    // windows [lo[l], hi[l]), in the order of sorted[adj[l] + (window >> (12 - l))]
    uint16_t lo[K3HUF_MAXLEN + 1], hi[K3HUF_MAXLEN + 1];
    int16_t adj[K3HUF_MAXLEN + 1];
    uint8_t sorted[256];
    uint64_t stripe[kMaxStripes];             // offset of each stripe in the container
    uint64_t last_bytes;                      // container bytes from the last stripe on
};

__device__ __forceinline__ uint32_t bswap32(uint32_t x) { return __byte_perm(x, 0, 0x0123); }

// The 12-bit table, entry (symbol << 4) | length; 0 where no code is.
__device__ void build_lut(const EmbedParams &P, uint16_t *lut) {
    for (uint32_t e = threadIdx.x; e < K3HUF_TABLE_ENTRIES; e += blockDim.x) {
        uint32_t v = 0;
        for (int l = 1; l <= K3HUF_MAXLEN && !v; ++l)
            if (e >= P.lo[l] && e < P.hi[l]) v = (uint32_t(P.sorted[P.adj[l] + int(e >> (K3HUF_MAXLEN - l))]) << 4) | uint32_t(l);
        lut[e] = uint16_t(v);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) embed_kernel(const __grid_constant__ EmbedParams P) {
    __shared__ uint16_t lut[K3HUF_TABLE_ENTRIES];
    build_lut(P, lut);
    __syncthreads();
    const uint64_t w = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (w >= P.n_tokens * P.units) return;
    const uint64_t t = w / P.units, k = w - t * P.units;
    const int64_t id = ld_id(P.ids, P.id_bytes, t);
    T *out = static_cast<T *>(P.out) + t * P.out_stride;
    if (id < 0 || uint64_t(id) >= P.rows) {
        // no row: zeros, and the status bit for an id past the table
        if (id >= 0 && k == 0) atomicOr(P.status, K3HUF_ST_TOKEN);
        for (uint64_t c = k; c < P.cols; c += P.units) st_f32(out + c, 0.f);
        return;
    }
    const uint32_t cs = P.chunk_syms, ss = P.sub_syms, S = cs / ss;
    const uint32_t full = (K3HUF_STRIPE_VALUES + cs - 1) / cs * S;       // sub-streams of a full stripe
    const uint64_t v0 = uint64_t(id) * P.cols;
    const uint32_t l0 = uint32_t(v0 % K3HUF_STRIPE_VALUES);
    const uint64_t u = v0 / K3HUF_STRIPE_VALUES * full + uint64_t(l0 / cs) * S + l0 % cs / ss + k;
    const uint32_t si = uint32_t(u / full), g = uint32_t(u % full);
    if (si >= P.n_stripes) return;
    const uint64_t base = uint64_t(si) * K3HUF_STRIPE_VALUES;
    const uint32_t n = uint32_t(min(uint64_t(K3HUF_STRIPE_VALUES), P.n_values - base));
    const uint32_t c = g / S, j = g % S, nch = (n + cs - 1) / cs;
    // this sub-stream's values in the stripe, [a, b), and those of the row
    const uint64_t a = uint64_t(c) * cs + uint64_t(j) * ss, b = min(a + ss, uint64_t(n));
    if (a >= b || base + a >= v0 + P.cols || base + b <= v0) return;
    const uint8_t *stripe = P.blob + P.stripe[si];
    const uint32_t *h = reinterpret_cast<const uint32_t *>(stripe);
    const uint64_t region = si + 1 < P.n_stripes ? P.stripe[si + 1] - P.stripe[si] : P.last_bytes;
    const uint64_t bits_need = ((uint64_t(h[4]) + 7) / 8 + 15) / 16 * 16 + kBitsSlack;
    const uint64_t index = 4ull * nch + 2ull * nch * (S - 1);
    if (h[0] != kStripeMagic || h[1] != P.table || h[2] != n || h[3] != nch || h[5] != 0 ||
        h[6] != (K3HUF_STRIPE_HDR_BYTES + index + 15) / 16 * 16 || h[7] < h[6] + bits_need || uint64_t(h[7]) + n > region) {
        atomicOr(P.status, K3HUF_ST_HEADER);
        return;
    }
    const uint32_t huff_bits = h[4];
    const uint32_t *chunk_off = h + K3HUF_STRIPE_HDR_BYTES / 4;
    const uint16_t *sub_off = reinterpret_cast<const uint16_t *>(chunk_off + nch);
    const uint32_t *words = reinterpret_cast<const uint32_t *>(stripe + h[6]);
    const uint8_t *even = stripe + h[7];
    const uint32_t cb = chunk_off[c];
    uint32_t pos = cb + (j ? uint32_t(sub_off[size_t(c) * (S - 1) + j - 1]) : 0u);
    const uint32_t end = j + 1 < S ? cb + sub_off[size_t(c) * (S - 1) + j] : c + 1 < nch ? chunk_off[c + 1] : huff_bits;
    uint32_t bad = 0;
    for (uint64_t v = a; v < b; ++v) {
        // (the stream is followed by 32 zero bytes, so word huff_bits / 32 + 1 is inside)
        const uint32_t p = min(pos, huff_bits);
        const uint32_t e = lut[__funnelshift_l(bswap32(words[p / 32 + 1]), bswap32(words[p / 32]), p) >> 20];
        if (!(e & 15u)) bad = K3HUF_ST_BADCODE;
        pos += max(e & 15u, 1u);
        if (base + v >= v0 && base + v < v0 + P.cols)
            st_f32(out + (base + v - v0), P.scale * __uint_as_float(((e >> 4) << 24) | (uint32_t(even[v]) << 16)));
    }
    if (pos != end) bad |= pos > huff_bits ? K3HUF_ST_OVERRUN : K3HUF_ST_INDEX;
    if (bad) atomicOr(P.status, bad);
}

// One CTA per token; the first token of each id adds up all of that id, in
// the order of the tokens.
template <typename T>
__global__ void __launch_bounds__(kThreads)
embed_grad_kernel(const void *ids, uint32_t id_bytes, uint64_t n, const T *dy, uint64_t dy_stride, uint64_t rows, uint64_t cols, float scale, float *grad, uint32_t *status) {
    const uint64_t t = blockIdx.x;
    const int64_t id = ld_id(ids, id_bytes, t);
    if (id < 0 || uint64_t(id) >= rows) {
        if (id >= 0 && threadIdx.x == 0) atomicOr(status, K3HUF_ST_TOKEN);
        return;
    }
    int seen = 0;
    for (uint64_t u = threadIdx.x; u < t; u += kThreads) seen |= ld_id(ids, id_bytes, u) == id;
    if (__syncthreads_or(seen)) return;
    for (uint64_t c = threadIdx.x; c < cols; c += kThreads) {
        float sum = 0.f;
        for (uint64_t u = t; u < n; ++u)
            if (ld_id(ids, id_bytes, u) == id) sum += ld_f32(dy + u * dy_stride + c);
        grad[uint64_t(id) * cols + c] += scale * sum;
    }
}

__global__ void zero_kernel(float *g, uint64_t n) {
    for (uint64_t i = uint64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += uint64_t(gridDim.x) * blockDim.x) g[i] = 0.f;
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
    if (te.n_values % cols != 0 || te.n_stripes > uint32_t(kMaxStripes) || out_stride < cols) return K3HUF_E_ARG;
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
    P.chunk_syms = L.info.chunk_syms;
    P.sub_syms = L.info.sub_syms;
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
    int off = 0;
    for (int l = 1; l <= K3HUF_MAXLEN; ++l) {
        P.lo[l] = uint16_t(first[l] << (K3HUF_MAXLEN - l));
        P.hi[l] = uint16_t((first[l] + count[l]) << (K3HUF_MAXLEN - l));
        P.adj[l] = int16_t(off - int(first[l]));
        for (int s = 0; s < 256; ++s)
            if (len[s] == l) P.sorted[off++] = uint8_t(s);
    }
    for (uint32_t s = 0; s < te.n_stripes; ++s) P.stripe[s] = L.stripes[te.first_stripe + s].blob_offset;
    P.last_bytes = L.info.blob_bytes - P.stripe[te.n_stripes - 1];
    const uint64_t blocks = (n_tokens * P.units + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFFull) return K3HUF_E_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (out_type == K3HUF_BF16) embed_kernel<__nv_bfloat16><<<uint32_t(blocks), kThreads, 0, st>>>(P);
    else embed_kernel<float><<<uint32_t(blocks), kThreads, 0, st>>>(P);
    return cuda_rc(cudaGetLastError());
}

extern "C" int k3huf_embed_grad_scratch_bytes(uint64_t n_tokens, uint64_t rows, uint64_t cols, size_t *scratch_bytes) {
    if (!scratch_bytes || rows == 0 || cols == 0) return K3HUF_E_ARG;
    *scratch_bytes = 256;
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
    if (!(flags & K3HUF_ACCUMULATE)) {
        const uint64_t n = rows * cols;
        zero_kernel<<<uint32_t(std::min<uint64_t>(1216, (n + 255) / 256)), 256, 0, st>>>(d_grad, n);
    }
    if (n_tokens && dy_type == K3HUF_BF16)
        embed_grad_kernel<<<uint32_t(n_tokens), kThreads, 0, st>>>(d_ids, id_bytes, n_tokens, static_cast<const __nv_bfloat16 *>(d_dy), dy_stride, rows, cols, scale, d_grad, d_status);
    else if (n_tokens)
        embed_grad_kernel<<<uint32_t(n_tokens), kThreads, 0, st>>>(d_ids, id_bytes, n_tokens, static_cast<const float *>(d_dy), dy_stride, rows, cols, scale, d_grad, d_status);
    return cuda_rc(cudaGetLastError());
}
