// pa_decode_latent and pa_prefill_latent: attention over a latent pool in the
// absorbed form.  A token's row is [latent | rotary key]; every query head
// carries [absorbed query | rotated query] of the same width, so
//   s_j = scale * q . row_j,   out = sum_j softmax(s)_j latent_j.
#include "host_common.h"
#include "rope.cuh"

namespace pa {

struct LatentParams {
    const uint16_t* rows;
    int32_t num_blocks, block_size, latent_dim, rope_dim;
    const uint16_t* q;
    int32_t heads;
    const int32_t *starts, *lens, *tables;  // starts: null for one query a sequence
    int32_t max_blocks, seqs, max_q, total_q, max_context, causal;
    float scale_log2;
    uint16_t* out;
    int32_t* d_err;
};

// One warp a (query, head) row, online softmax over the tokens one by one; lane
// l holds elements 2l + 64i, 2l + 64i + 1.
constexpr int kLatentPairs = 9;  // up to 576 elements a row

__global__ void __launch_bounds__(128) latent_rows_kernel(const LatentParams p) {
    const int s = blockIdx.y, lane = threadIdx.x & 31;
    const int start = p.starts ? p.starts[s] : s;
    const int new_q = p.starts ? p.starts[s + 1] - start : 1;
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int n = p.lens[s];
    if (p.starts && (start < 0 || new_q < 0 || new_q > p.total_q - start)) {
        set_error(p.d_err, PA_ERR_OUT_OF_RANGE);
        return;
    }
    if (new_q == 0 || (!p.starts && n <= 0)) return;
    if (n < new_q) {
        set_error(p.d_err, PA_ERR_INVALID_ARG);
        return;
    }
    if (n > p.max_context || new_q > p.max_q) set_error(p.d_err, PA_ERR_OUT_OF_RANGE);
    if (r >= (int64_t)min(new_q, p.max_q) * p.heads) return;
    const int i = (int)(r / p.heads);
    const int seen = min(p.causal ? n - new_q + i + 1 : n, p.max_context);
    const int width = p.latent_dim + p.rope_dim;
    const int64_t row = (int64_t)start * p.heads + r;
    const uint32_t* q = (const uint32_t*)(p.q + row * width);
    float2 qf[kLatentPairs], acc[kLatentPairs];
#pragma unroll
    for (int c = 0; c < kLatentPairs; ++c) {
        const int e = 2 * lane + 64 * c;
        const uint32_t w = e < width ? q[e >> 1] : 0;
        qf[c] = make_float2(bf16_lo(w), bf16_hi(w));
        acc[c] = make_float2(0.f, 0.f);
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < seen; ++j) {
        const int e = j / p.block_size;
        const int blk = e < p.max_blocks ? p.tables[(int64_t)s * p.max_blocks + e] : -1;
        if (blk < 0 || blk >= p.num_blocks) {
            set_error(p.d_err, blk < 0 ? PA_ERR_NEGATIVE_BLOCK : PA_ERR_OUT_OF_RANGE);
            continue;
        }
        const uint32_t* kr = (const uint32_t*)(
            p.rows + ((int64_t)blk * p.block_size + j % p.block_size) * width);
        float2 kf[kLatentPairs];
        float d = 0.f;
#pragma unroll
        for (int c = 0; c < kLatentPairs; ++c) {
            const int x = 2 * lane + 64 * c;
            const uint32_t w = x < width ? kr[x >> 1] : 0;
            kf[c] = make_float2(bf16_lo(w), bf16_hi(w));
            d += qf[c].x * kf[c].x + qf[c].y * kf[c].y;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        d *= p.scale_log2;
        const float up = fmaxf(m, d);
        const float f = m == -INFINITY ? 0.f : exp2f(m - up), w = exp2f(d - up);
        m = up;
        l = l * f + w;
#pragma unroll
        for (int c = 0; c < kLatentPairs; ++c) {
            acc[c].x = acc[c].x * f + w * kf[c].x;
            acc[c].y = acc[c].y * f + w * kf[c].y;
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint32_t* out = (uint32_t*)(p.out + row * p.latent_dim);
#pragma unroll
    for (int c = 0; c < kLatentPairs; ++c) {
        const int x = 2 * lane + 64 * c;
        if (x < p.latent_dim) out[x >> 1] = pack_bf16(acc[c].x * inv, acc[c].y * inv);
    }
}

static pa_status latent_attention(const pa_latent_pool* pool, const void* q, int32_t heads,
                                  const int32_t* starts, const int32_t* tables,
                                  int32_t max_blocks, const int32_t* lens, int32_t seqs,
                                  int32_t max_q, int32_t total_q, int32_t max_context, float scale,
                                  int causal,
                                  void* out, int32_t* d_err, cudaStream_t stream) {
    LatentParams p;
    p.rows = (const uint16_t*)pool->rows;
    p.num_blocks = pool->num_blocks;
    p.block_size = pool->block_size;
    p.latent_dim = pool->latent_dim;
    p.rope_dim = pool->rope_dim;
    p.q = (const uint16_t*)q;
    p.heads = heads;
    p.starts = starts;
    p.lens = lens;
    p.tables = tables;
    p.max_blocks = max_blocks;
    p.seqs = seqs;
    p.max_q = max_q;
    p.total_q = total_q;
    p.max_context = max_context;
    p.causal = causal;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = (uint16_t*)out;
    p.d_err = d_err;
    const int64_t blocks = ((int64_t)max_q * heads + 3) / 4;
    latent_rows_kernel<<<dim3((unsigned)blocks, (unsigned)seqs), 128, 0, stream>>>(p);
    return launch_status();
}

static pa_status check_latent_attention(const pa_latent_pool* pool, int32_t heads, int32_t seqs,
                                        int32_t max_context) {
    pa_status st = check_latent_pool(pool);
    if (st != PA_OK) return st;
    if (heads <= 0 || seqs < 0 || max_context < 0) return PA_ERR_INVALID_ARG;
    if (pool->latent_dim % 128 != 0 || pool->latent_dim > 512 || pool->rope_dim > 64 ||
        !is_pow2(pool->block_size) || pool->block_size < 8 || pool->block_size > 128 ||
        heads > 128 || seqs > 65535)
        return PA_ERR_UNSUPPORTED;
    if ((int64_t)pool->num_blocks * pool->block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_decode_latent_workspace_bytes(const pa_latent_pool* pool, int32_t num_seqs,
                                                      int32_t num_q_heads, int32_t max_context,
                                                      size_t* bytes) {
    if (bytes == nullptr) return PA_ERR_INVALID_ARG;
    pa_status st = check_latent_attention(pool, num_q_heads, num_seqs, max_context);
    if (st != PA_OK) return st;
    *bytes = 0;
    return PA_OK;
}

extern "C" pa_status pa_decode_latent(const pa_latent_pool* pool, const void* q, int32_t num_q_heads,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* context_lens, int32_t num_seqs,
                                      int32_t max_context, float scale, void* out, void* workspace,
                                      size_t workspace_bytes, int32_t* d_err, pa_stream_t stream) {
    (void)workspace;
    (void)workspace_bytes;
    pa_status st = check_latent_attention(pool, num_q_heads, num_seqs, max_context);
    if (st != PA_OK) return st;
    if (max_blocks_per_seq < 0 || !(scale == scale)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || max_context == 0) return PA_OK;
    if (!q || !block_tables || !context_lens || !out) return PA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(pool->rows)) return PA_ERR_INVALID_ARG;
    return latent_attention(pool, q, num_q_heads, nullptr, block_tables, max_blocks_per_seq,
                            context_lens, num_seqs, 1, num_seqs, max_context, scale, 0, out, d_err,
                            (cudaStream_t)stream);
}

extern "C" pa_status pa_prefill_latent_workspace_bytes(const pa_latent_pool* pool, int32_t num_seqs,
                                                       int32_t num_q_heads, int32_t total_q,
                                                       int32_t max_q_len, int32_t max_context,
                                                       size_t* bytes) {
    if (bytes == nullptr || total_q < 0 || max_q_len < 0) return PA_ERR_INVALID_ARG;
    pa_status st = check_latent_attention(pool, num_q_heads, num_seqs, max_context);
    if (st != PA_OK) return st;
    *bytes = 0;
    return PA_OK;
}

extern "C" pa_status pa_prefill_latent(const pa_latent_pool* pool, const void* q, int32_t total_q,
                                       int32_t num_q_heads, const int32_t* cu_seqlens_q,
                                       const int32_t* context_lens, const int32_t* block_tables,
                                       int32_t max_blocks_per_seq, int32_t num_seqs,
                                       int32_t max_q_len, int32_t max_context, float scale,
                                       int32_t causal, void* out, void* workspace,
                                       size_t workspace_bytes, int32_t* d_err, pa_stream_t stream) {
    (void)workspace;
    (void)workspace_bytes;
    pa_status st = check_latent_attention(pool, num_q_heads, num_seqs, max_context);
    if (st != PA_OK) return st;
    if (total_q < 0 || max_q_len < 0 || max_blocks_per_seq < 0 || !(scale == scale))
        return PA_ERR_INVALID_ARG;
    if ((int64_t)total_q * num_q_heads > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0 || max_context == 0) return PA_OK;
    if (!q || !cu_seqlens_q || !context_lens || !block_tables || !out) return PA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(pool->rows)) return PA_ERR_INVALID_ARG;
    return latent_attention(pool, q, num_q_heads, cu_seqlens_q, block_tables, max_blocks_per_seq,
                            context_lens, num_seqs, max_q_len, total_q, max_context, scale,
                            causal ? 1 : 0, out, d_err, (cudaStream_t)stream);
}
