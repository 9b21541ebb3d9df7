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
// And what it tells the issuers about a unit: its tiles, 0 behind the last.  The issuers
// know no more of units: with the search for them in their loops the compiler loses
// track of what is uniform in the warp, and an MMA with descriptors from general
// registers takes 40 to 100 cycles to issue, against 24 to 64 to run.  The producer is
// at most two units ahead of them (Q has one buffer).
constexpr int kUnits = 4;

struct Params {
    const char* q;
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
    int32_t ahead;        // tokens before the sequence's first new one
    int32_t context;      // tokens of the sequence that may be seen
    int32_t t0, t1;       // tiles
    int32_t tiles;        // of the whole unit
    int64_t unit_at;      // the unit's place on the line

    // tokens that row r of the unit sees
    PA_DEVICE int32_t seen(const Params& p, int r) const {
        if (r >= rows) return 0;
        return p.causal ? min(ahead + (token + r) / p.heads + 1, context) : context;
    }
};

struct Line {
    int64_t at, end;      // what is left of the stretch
    int64_t unit_at;      // place of unit u of sequence s on the line
    int32_t s, u;
    Seq q;
};

// The next share of the stretch, skipping places that the line holds too many.
PA_DEVICE bool next_part(const Params& p, Line& l, Part& w) {
    while (l.at < l.end) {
        if (l.u >= l.q.units) {
            if (++l.s >= p.seqs) return false;
            l.q = read_seq(p, l.s, false);
            l.u = 0;
            continue;
        }
        const int u = l.u++;
        const int64_t begin = l.unit_at;
        l.unit_at = begin + l.q.first + (l.q.step == 0 ? 0 : l.q.more * (u / l.q.step));
        if (l.at >= l.unit_at) continue;
        const int r0 = u * p.unit_rows;
        w.seq = l.s;
        w.row = l.q.start * p.heads + r0;
        w.rows = min(p.unit_rows, min(l.q.fresh, p.max_q) * p.heads - r0);
        w.token = r0;
        w.ahead = l.q.n - l.q.fresh;
        w.context = min(l.q.n, p.max_context);
        w.tiles = (w.seen(p, w.rows - 1) + kTok - 1) / kTok;
        w.t0 = (int)(l.at - begin);
        w.t1 = (int)min((int64_t)w.tiles, l.end - begin);
        w.unit_at = begin;
        l.at = min(l.unit_at, l.end);
        if (w.t0 < w.t1) return true;
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
        line.unit_at = ahead;
        line.q = read_seq(p, s0, false);
        for (int64_t all; line.at >= line.unit_at + (all = line.q.before(line.q.units));) {
            line.unit_at += all;
            line.q = read_seq(p, ++line.s, false);
        }
        const int64_t off = line.at - line.unit_at;
        int u = 0, hi = line.q.units - 1;  // last unit that begins at or before `at`
        while (u < hi) {
            const int mid = (int)(((unsigned)u + hi + 1) >> 1);
            if (line.q.before(mid) <= off) u = mid; else hi = mid - 1;
        }
        line.u = u;
        line.unit_at += line.q.before(u);
        sc.some = next_part(p, line, part);
        sc.line = line;
        sc.part = part;
    }
    __syncthreads();
    line = sc.line;
    part = sc.part;
    return sc.some != 0;
}

// Asks for the rows behind this unit's, the next unit's queries, in L2: the stretch goes
// on with them, and HBM's latency would stand between the two units.
PA_DEVICE void ask_next_q(const Params& p, const Line& l, const Part& w, int rows, int row_bytes) {
    const int64_t first = (int64_t)w.row + w.rows, left = (int64_t)p.total_q * p.heads - first;
    if (l.at < l.end && left > 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                     ::"l"(p.q + first * row_bytes), "r"((uint32_t)min((int64_t)rows, left) * row_bytes) : "memory");
}

// Tiles of the pair kernel (latent_pair.cu): units of up to 128 rows, a CTA pair each.
cudaError_t launch_pair(const Params& p, const void* q, const pa_latent_pool* pool, int64_t q_rows,
                        cudaStream_t stream);

}  // namespace lat
}  // namespace pa
