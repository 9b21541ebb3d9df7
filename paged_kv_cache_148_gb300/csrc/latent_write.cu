// pa_write_latent and pa_copy_latent_blocks: the two writes of a latent pool.
//
// A latent pool keeps one row a token, [latent | rotary key], shared by every
// query head.  pa_write_latent copies the latent part, turns the rotary key and
// each query head's rotary part by the token's angles (rope.cuh), and scatters
// the row to its slot; the turned query part goes behind the absorbed part of
// q.  Each byte is read once and written once.  8192 tokens of 32 heads (86 MB): 16.6 us,
// 5.2 TB/s, 76 % of the copy bandwidth: the transfer is short, and a CTA's chain of
// loads (position, then rows) is not hidden at its start and end.  1211 blocks of 64
// tokens (179 MB): 31 us as a loop of calls.
#include "host_common.h"
#include "rope.cuh"

namespace pa {

pa_status check_rope(const pa_rope* r);

struct LatentWriteParams {
    const uint16_t *latent, *k_rope, *q_rope;
    int64_t latent_stride, k_stride, q_stride, q_head_stride;  // elements
    int32_t latent_dim, rope_dim, heads;
    uint32_t per_units, per_turning;  // 2^32 / units and / turning, rounded up; 0: divide
    const uint64_t* turns;
    int32_t interleaved;
    float magnitude;
    const int64_t *positions, *slots;
    int32_t tokens;
    int64_t num_slots;
    uint16_t* q;     // [tokens][heads][latent_dim + rope_dim]
    uint16_t* rows;  // the pool
    int32_t* d_err;
};

constexpr int kLatentWriteThreads = 256;

// kTokens tokens a CTA, their cosines and sines in shared memory first.  A unit
// is two 16-byte vectors: latent_dim / 16 units of plain copy, then
// rope_dim / 16 turned units for the key and for each query head.
__global__ void __launch_bounds__(kLatentWriteThreads) latent_write_kernel(const LatentWriteParams p,
                                                                           const int kTokens) {
    using V = Vec16<uint16_t>;
    extern __shared__ float2 cs[];  // [kTokens][rope_dim / 2]
    griddep_wait();
    griddep_launch();
    const int pairs = p.rope_dim >> 1;
    const int t0 = blockIdx.x * kTokens;
    const int tokens = min(kTokens, p.tokens - t0);
    const int width = p.latent_dim + p.rope_dim;
    const int copies = p.latent_dim >> 4, turning = p.rope_dim >> 4;
    const int units = copies + turning * (1 + p.heads);
    const int all = tokens * units;
    struct Unit {
        uint4 a, b;
        uint4* dst;       // null: nothing to store
        int va, vb, first;  // first pair, -1: plain copy
    };
    auto load = [&](int i) {
        Unit x;
        x.dst = nullptr;
        if (i >= all) return x;
        const int t = p.per_units ? (int)__umulhi(i, p.per_units) : i / units, w = i - t * units;
        const int64_t tok = t0 + t;
        // -1: the pool's row
        const int head = w < copies ? -1 : (turning == 1 ? w - copies : (int)__umulhi(w - copies, p.per_turning)) - 1;
        const uint4* src;
        if (w < copies) {
            src = (const uint4*)(p.latent + tok * p.latent_stride);
            x.va = 2 * w;
            x.vb = x.va + 1;
            x.first = -1;
        } else {
            const int u = (w - copies) - (head + 1) * turning;
            src = head < 0 ? (const uint4*)(p.k_rope + tok * p.k_stride)
                           : (const uint4*)(p.q_rope + tok * p.q_stride + head * p.q_head_stride);
            x.va = p.interleaved ? 2 * u : u;
            x.vb = p.interleaved ? x.va + 1 : u + turning;
            x.first = t * pairs + u * V::N;
        }
        x.a = src[x.va];
        x.b = src[x.vb];
        if (head < 0) {
            const int64_t slot = __ldg(p.slots + tok);
            if (slot >= 0 && slot < p.num_slots)
                x.dst = (uint4*)(p.rows + slot * width + (w < copies ? 0 : p.latent_dim));
            else if (w == 0)
                set_error(p.d_err, PA_ERR_OUT_OF_RANGE);
        } else {
            x.dst = (uint4*)(p.q + (tok * p.heads + head) * (int64_t)width + p.latent_dim);
        }
        return x;
    };
    // the first units are on their way while the angles are computed
    Unit x = load(threadIdx.x);
    for (int i = threadIdx.x; i < tokens * pairs; i += blockDim.x) {
        const int t = i / pairs, j = i - t * pairs;
        cs[i] = rope_angle(__ldg(p.turns + j), __ldg(p.positions + t0 + t), p.magnitude);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < all; i += blockDim.x) {
        if (i >= blockDim.x) x = load(i);
        if (x.dst == nullptr) continue;
        if (x.first >= 0) {
            float fa[V::N], fb[V::N];
            V::open(x.a, fa);
            V::open(x.b, fb);
            rope_turn_vectors<uint16_t>(p.interleaved, cs + x.first, fa, fb);
            x.a = V::close(fa);
            x.b = V::close(fb);
        }
        x.dst[x.va] = x.a;
        x.dst[x.vb] = x.b;
    }
}

// One pool's pages: grid (pair, slice of the page), four vectors a thread and
// round, loads before stores.
constexpr int kLatentCopyU = 4;

__global__ void __launch_bounds__(256) latent_copy_kernel(uint4* rows, const int32_t* src,
                                                          const int32_t* dst, int64_t page_vecs,
                                                          int32_t num_blocks, int32_t* d_err) {
    const int32_t s = __ldg(src + blockIdx.x), d = __ldg(dst + blockIdx.x);
    if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks) {
        if (blockIdx.y == 0 && threadIdx.x == 0) set_error(d_err, PA_ERR_OUT_OF_RANGE);
        return;
    }
    const uint4* from = rows + (int64_t)s * page_vecs;
    uint4* to = rows + (int64_t)d * page_vecs;
    const int64_t step = (int64_t)gridDim.y * blockDim.x;
    for (int64_t v = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; v < page_vecs;
         v += kLatentCopyU * step) {
        uint4 a[kLatentCopyU];
#pragma unroll
        for (int u = 0; u < kLatentCopyU; ++u)
            if (v + u * step < page_vecs) a[u] = from[v + u * step];
#pragma unroll
        for (int u = 0; u < kLatentCopyU; ++u)
            if (v + u * step < page_vecs) to[v + u * step] = a[u];
    }
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_write_latent(const pa_latent_pool* pool, const pa_rope* rope,
                                     const void* latent, int64_t latent_stride, const void* k_rope,
                                     int64_t k_rope_stride, const int64_t* positions,
                                     const int64_t* slot_mapping, int32_t num_tokens,
                                     const void* q_rope, int64_t q_rope_stride,
                                     int64_t q_rope_head_stride, int32_t num_q_heads, void* q,
                                     int32_t* d_err, pa_stream_t stream) {
    pa_status st = check_latent_pool(pool);
    if (st != PA_OK) return st;
    st = check_rope(rope);
    if (st != PA_OK) return st;
    if (num_tokens < 0 || num_q_heads < 0) return PA_ERR_INVALID_ARG;
    if (rope->rot_dim != pool->rope_dim) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!latent || !k_rope || !positions || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!q_rope || !q)) return PA_ERR_INVALID_ARG;
    if (latent_stride < pool->latent_dim || k_rope_stride < pool->rope_dim) return PA_ERR_INVALID_ARG;
    if (latent_stride % 8 || k_rope_stride % 8 || !aligned16(latent) || !aligned16(k_rope) ||
        !aligned16(pool->rows))
        return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0) {
        if (q_rope_head_stride < pool->rope_dim ||
            q_rope_stride < (num_q_heads - 1) * q_rope_head_stride + pool->rope_dim)
            return PA_ERR_INVALID_ARG;
        if (q_rope_stride % 8 || q_rope_head_stride % 8 || !aligned16(q_rope) || !aligned16(q))
            return PA_ERR_INVALID_ARG;
        if (num_q_heads > 1 << 16) return PA_ERR_UNSUPPORTED;
    }
    LatentWriteParams p;
    p.latent = (const uint16_t*)latent;
    p.k_rope = (const uint16_t*)k_rope;
    p.q_rope = (const uint16_t*)q_rope;
    p.latent_stride = latent_stride;
    p.k_stride = k_rope_stride;
    p.q_stride = q_rope_stride;
    p.q_head_stride = q_rope_head_stride;
    p.latent_dim = pool->latent_dim;
    p.rope_dim = pool->rope_dim;
    p.heads = num_q_heads;
    // exact for products under 2^32: a unit's index times the divisor
    const int64_t turning = pool->rope_dim / 16, units = pool->latent_dim / 16 + turning * (1 + num_q_heads);
    p.per_units = units < 32768 ? (uint32_t)(((1ull << 32) + units - 1) / units) : 0;
    p.per_turning = (uint32_t)(((1ull << 32) + turning - 1) / turning);
    p.turns = rope->turns;
    p.interleaved = rope->layout == PA_ROPE_INTERLEAVED;
    p.magnitude = rope->magnitude;
    p.positions = positions;
    p.slots = slot_mapping;
    p.tokens = num_tokens;
    p.num_slots = (int64_t)pool->num_blocks * pool->block_size;
    p.q = (uint16_t*)q;
    p.rows = (uint16_t*)pool->rows;
    p.d_err = d_err;
    // tokens a CTA (8192 tokens of 32 heads: 21.2, 18.7, 16.6, 17.9, 16.9, 18.6 us with 1, 2,
    // 3, 4, 6, 8); small batches need the CTAs
    const int per = num_tokens >= 4 * device_sm_count() ? 3 : 1;
    cudaError_t e = launch_pdl(latent_write_kernel, dim3((unsigned)((num_tokens + per - 1) / per)),
                               dim3(kLatentWriteThreads),
                               (size_t)per * (pool->rope_dim / 2) * sizeof(float2),
                               (cudaStream_t)stream, p, per);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return PA_ERR_CUDA;
    }
    return launch_status();
}

extern "C" pa_status pa_copy_latent_blocks(const pa_latent_pool* pool, const int32_t* src,
                                           const int32_t* dst, int32_t n, int32_t* d_err,
                                           pa_stream_t stream) {
    pa_status st = check_latent_pool(pool);
    if (st != PA_OK) return st;
    if (n < 0) return PA_ERR_INVALID_ARG;
    if (n == 0) return PA_OK;
    if (!src || !dst || !aligned16(pool->rows)) return PA_ERR_INVALID_ARG;
    const int64_t page_vecs =
        (int64_t)pool->block_size * (pool->latent_dim + pool->rope_dim) * 2 / 16;
    int64_t slices = (page_vecs + 256 * kLatentCopyU - 1) / (256 * kLatentCopyU);
    if (slices > 65535) slices = 65535;
    latent_copy_kernel<<<dim3((unsigned)n, (unsigned)slices), 256, 0, (cudaStream_t)stream>>>(
        (uint4*)pool->rows, src, dst, page_vecs, pool->num_blocks, d_err);
    return launch_status();
}
