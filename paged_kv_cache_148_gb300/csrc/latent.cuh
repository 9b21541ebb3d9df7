// What the kernels of latent attention share: the arguments, the line of tiles
// that a call's units form, and how a CTA finds its stretch of it.
#pragma once

#include <cuda.h>

#include "host_common.h"
#include "rope.cuh"
#include "tcgen05.cuh"

namespace pa {
namespace lat {

constexpr int kTok = 64;             // tokens of a tile
constexpr int kBlock = kTok * 128;   // bytes of 64 tokens x 64 elements
constexpr float kRescale = 16.0f;
constexpr int kSmemLimit = 232448;   // 227 KB

// Rings of what the producer tells the softmax about a tile: it is at most kSlots + 2
// tiles ahead of its slowest reader.
constexpr int kInfo = 8;

struct Params {
    int32_t num_blocks, log2_bp, latent_dim, rope_dim;
    int32_t heads;
    const int32_t *starts, *lens, *tables;  // starts: null for one query a sequence
    int32_t max_blocks, seqs, max_q, total_q, max_context, causal;
    float scale_log2;
    int32_t unit_rows;               // rows of a unit
    int32_t R;                       // unit_rows rounded up to 16
    int32_t step, more;              // causal: tiles that the line adds from unit to unit
    int32_t groups;                  // stretches
    int32_t min_tiles;               // least tiles a stretch
    uint16_t* out;
    int4* meta;                      // [groups]: parts of the unit cut behind this stretch
    float2* stats;                   // [2 * groups][R]: (max, sum) of a part's rows
    float* parts;                    // [2 * groups][R][latent_dim]
    int32_t* d_err;
};

// A warp's bounded wait.  Once one has run out the CTA winds down: every later
// wait that would block returns at once.
template <typename B>
PA_DEVICE bool wait_warp(uint64_t* bar, uint32_t parity, B* b, int32_t* d_err) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
        while (!(ok = mbar_try_wait(bar, parity))) {
            if (*(volatile int32_t*)&b->abort) break;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                set_error(d_err, PA_ERR_TIMEOUT);
                *(volatile int32_t*)&b->abort = 1;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

PA_DEVICE void named_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }
PA_DEVICE bool named_any(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(id), "r"((uint32_t)x) : "memory");
    return r != 0;
}

// ---------------------------------------------------------------- the line of tiles
// A sequence's units and the tiles that the line holds for each.  With a causal
// mask unit u needs ceil(seen / 64) tiles, and seen grows by unit_rows / heads
// tokens a unit; the line gives it first + more * (u / step) (host: step and more
// from unit_rows and heads), at least as many and with a sum in closed form, so
// that a stretch finds its place without walking the units.
struct Seq {
    int32_t start, fresh, n;   // first query token; query tokens; context
    int32_t units, first, step, more;  // tiles of unit u: first + more * (u / step); step 0: first

    PA_DEVICE int64_t before(int u) const {
        if (step == 0) return (int64_t)u * first;
        const int64_t k = u / step;
        return (int64_t)u * first + more * (step * (k * (k - 1) / 2) + k * (u - k * step));
    }
};



PA_DEVICE Seq read_seq(const Params& p, int s, bool report) {
    Seq q;
    q.units = q.first = q.step = q.more = 0;
    q.start = p.starts ? __ldg(p.starts + s) : s;
    q.fresh = p.starts ? __ldg(p.starts + s + 1) - q.start : 1;
    q.n = __ldg(p.lens + s);
    if (p.starts && (q.start < 0 || q.fresh < 0 || q.fresh > p.total_q - q.start)) {
        if (report) set_error(p.d_err, PA_ERR_OUT_OF_RANGE);
        return q;
    }
    if (q.fresh == 0 || (!p.starts && q.n <= 0)) return q;
    if (q.n < q.fresh) {
        if (report) set_error(p.d_err, PA_ERR_INVALID_ARG);
        return q;
    }
    if (report && (q.n > p.max_context || q.fresh > p.max_q)) set_error(p.d_err, PA_ERR_OUT_OF_RANGE);
    const int64_t rows = (int64_t)min(q.fresh, p.max_q) * p.heads;
    q.units = (int)((rows + p.unit_rows - 1) / p.unit_rows);
    if (p.causal) {
        const int64_t base = q.n - q.fresh;
        q.first = (int)((base + 2 + (p.unit_rows - 1) / p.heads + kTok - 1) / kTok) + 1;
        q.step = p.step;
        q.more = p.more;
    } else {
        q.first = (min(q.n, p.max_context) + kTok - 1) / kTok;
    }
    return q;
}

// A stretch's share of one unit.
struct Part {
    int32_t seq;
    int32_t row;          // first query row of the unit, over the whole call
    int32_t rows;         // its rows
    int32_t token;        // first row's index within the sequence's rows
    int32_t limit;        // tokens that the unit's last row sees
    int32_t t0, t1;       // tiles
    int32_t tiles;        // of the whole unit
    int64_t unit_at;      // the unit's place on the line
    Seq q;
};

struct Line {
    int64_t at, end;      // what is left of the stretch
    int64_t seq_at;       // place of sequence s on the line
    int32_t s;
};

// The next share of the stretch, skipping places that the line holds too many.
PA_DEVICE bool next_part(const Params& p, Line& l, Part& w) {
    while (l.at < l.end && l.s < p.seqs) {
        const Seq q = read_seq(p, l.s, false);
        const int64_t all = q.before(q.units);
        if (l.at >= l.seq_at + all) {
            l.seq_at += all;
            ++l.s;
            continue;
        }
        int u = 0, hi = q.units - 1;       // last unit that begins at or before `at`
        const int64_t off = l.at - l.seq_at;
        while (u < hi) {
            const int mid = (int)(((unsigned)u + hi + 1) >> 1);
            if (q.before(mid) <= off) u = mid; else hi = mid - 1;
        }
        const int64_t begin = l.seq_at + q.before(u), stop = l.seq_at + q.before(u + 1);
        const int r0 = u * p.unit_rows;
        const int all_rows = min(q.fresh, p.max_q) * p.heads;
        const int rows = min(p.unit_rows, all_rows - r0);
        int seen = q.n;
        if (p.causal) seen = q.n - q.fresh + (r0 + rows - 1) / p.heads + 1;
        seen = min(seen, p.max_context);
        const int tiles = (seen + kTok - 1) / kTok;
        const int t0 = (int)(l.at - begin);
        const int t1 = (int)min((int64_t)tiles, l.end - begin);
        l.at = min(stop, l.end);
        if (t0 >= t1) continue;
        w.seq = l.s;
        w.row = q.start * p.heads + r0;
        w.rows = rows;
        w.token = r0;
        w.limit = seen;
        w.t0 = t0;
        w.t1 = t1;
        w.tiles = tiles;
        w.unit_at = begin;
        w.q = q;
        return true;
    }
    return false;
}

// A block finds its stretch and the first share of it.  Every thread calls it;
// scratch is shared memory.
struct Scan {
    int64_t sums[8];
    Line line;
    Part part;
    int32_t some;
};

template <int THREADS>
PA_DEVICE bool find_stretch(const Params& p, int group, bool report, Scan& sc, Line& line, Part& part,
                            int64_t& per) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the line's length, then the sequence in which this stretch begins: each
    // thread adds up an equal run of sequences, and the one whose run holds the
    // stretch's first tile walks it
    if (threadIdx.x == 0) sc.some = 0;
    const int run = (p.seqs + THREADS - 1) / THREADS;
    const int s0 = min(p.seqs, (int)threadIdx.x * run), s1 = min(p.seqs, s0 + run);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) {
        const Seq q = read_seq(p, s, report);
        mine += q.before(q.units);
    }
    int64_t upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += x;
    }
    if (lane == 31) sc.sums[warp] = upto;
    __syncthreads();
    int64_t total = 0, ahead = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) ahead += sc.sums[w];
        total += sc.sums[w];
    }
    const int64_t sum = total + p.groups - 1;
    per = sum <= INT32_MAX ? (int64_t)((uint32_t)sum / (uint32_t)p.groups) : sum / p.groups;
    per = max(per, (int64_t)p.min_tiles);
    line.at = min(total, group * per);
    line.end = min(total, line.at + per);
    ahead += upto - mine;
    if (line.at < line.end && ahead <= line.at && line.at < ahead + mine) {
        line.s = s0;
        line.seq_at = ahead;
        sc.some = next_part(p, line, part);
        sc.line = line;
        sc.part = part;
    }
    __syncthreads();
    line = sc.line;
    part = sc.part;
    return sc.some != 0;
}

// Tiles of the pair kernel (latent_pair.cu): units of up to 128 rows, a CTA pair each.
cudaError_t launch_pair(const Params& p, const void* q, const pa_latent_pool* pool, int64_t q_rows,
                        cudaStream_t stream);

}  // namespace lat
}  // namespace pa
