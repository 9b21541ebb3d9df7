// What the kernels of latent attention share: the arguments, the line of tiles
// that a call's units form, and how a CTA finds its stretch of it.
#pragma once

#include <cuda.h>

#include "host_common.h"
#include "rope.cuh"
#include "tcgen05_pair.cuh"

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
// two units ahead of S's issuer at most (Q has one buffer), S two tiles ahead of the
// softmax, which ends a unit when its O is done: four units at the most in all.
constexpr int kUnits = 8;

struct Params {
    const char *q, *rows;
    int32_t num_blocks, log2_bp, latent_dim, rope_dim;
    int32_t heads;
    const int32_t *starts, *lens, *tables;  // starts: null for one query a sequence
    int32_t max_blocks, seqs, max_q, total_q, max_context, causal;
    float scale_log2;
    int32_t unit_rows;               // rows of a unit
    int32_t unit_shift;              // its logarithm where a sequence may have more than two units
    int32_t R;                       // unit_rows rounded up to 16
    int32_t step, more;              // causal: tiles that the line adds from unit to unit
    int32_t slack;                   // causal: tokens, (unit_rows - 1) / heads
    int32_t unit_tokens, unit_rest;  // unit_rows / heads and its remainder
    uint32_t per_head;               // 65536 / heads, rounded up: x / heads for x < 256
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
//
// All of this runs once a launch with a cold instruction cache, some ten cycles an
// instruction, so it is kept short: no division but in the search for a stretch's
// first unit, steps from unit to unit by counters.
struct Seq {
    int32_t start, fresh, n;   // first query token; query tokens; context
    int32_t units, first;      // tiles of unit u: first, with a mask + more * (u / step)

    PA_DEVICE int64_t before(const Params& p, int u) const {
        const int64_t flat = (int64_t)u * first;
        if (!p.causal || u <= p.step) return flat;
        const int64_t k = u / p.step;
        return flat + p.more * (p.step * (k * (k - 1) / 2) + k * (u - k * p.step));
    }
};

PA_DEVICE Seq read_seq(const Params& p, int s, bool report) {
    Seq q;
    q.units = q.first = 0;
    q.start = s;
    q.fresh = 1;
    q.n = __ldg(p.lens + s);
    if (p.starts) {
        q.start = __ldg(p.starts + s);
        q.fresh = __ldg(p.starts + s + 1) - q.start;
        if (q.start < 0 || q.fresh < 0 || q.fresh > p.total_q - q.start) {
            if (report) set_error(p.d_err, PA_ERR_OUT_OF_RANGE);
            return q;
        }
        if (q.fresh > 0 && q.n < q.fresh) {
            if (report) set_error(p.d_err, PA_ERR_INVALID_ARG);
            return q;
        }
    }
    if (q.fresh == 0 || q.n <= 0) return q;
    if (report && (q.n > p.max_context || q.fresh > p.max_q)) set_error(p.d_err, PA_ERR_OUT_OF_RANGE);
    const int rows = min(q.fresh, p.max_q) * p.heads;
    q.units = rows <= p.unit_rows ? 1 : p.unit_shift == 0 ? 2 : ((rows - 1) >> p.unit_shift) + 1;
    q.first = p.causal ? (int)((q.n - q.fresh + 2ll + p.slack + kTok - 1) >> 6) + 1
                       : (min(q.n, p.max_context) + kTok - 1) >> 6;
    return q;
}

// A stretch's share of one unit.
struct Part {
    int32_t seq;
    int32_t row;          // first query row of the unit, over the whole call
    int32_t rows;         // its rows
    int32_t ahead, rest;  // first row: context before its token; its head
    int32_t context;      // tokens of the sequence that may be seen
    int32_t t0, t1;       // tiles
    int32_t tiles;        // of the whole unit
    int64_t unit_at;      // the unit's place on the line

    // tokens that row r of the unit sees
    PA_DEVICE int32_t seen(const Params& p, int r) const {
        if (r >= rows) return 0;
        return p.causal ? min(ahead + (int)(((rest + r) * p.per_head) >> 16) + 1, context) : context;
    }
};

struct Line {
    int64_t at, end;      // what is left of the stretch
    int64_t unit_at;      // place of unit u of sequence s on the line
    int32_t s, u;
    int32_t extra, left;  // tiles of unit u past `first`, units until there are more
    int32_t token, rest;  // of unit u's first row
    Seq q;

    // to the first unit of sequence q
    PA_DEVICE void begin(const Params& p, const Seq& seq) {
        q = seq;
        u = extra = token = rest = 0;
        left = p.step;
    }
};

// The next share of the stretch, skipping places that the line holds too many.
PA_DEVICE bool next_part(const Params& p, Line& l, Part& w) {
    while (l.at < l.end) {
        if (l.u >= l.q.units) {
            if (++l.s >= p.seqs) return false;
            l.begin(p, read_seq(p, l.s, false));
            continue;
        }
        const int64_t begin = l.unit_at;
        l.unit_at = begin + l.q.first + l.extra;
        const int r0 = l.u * p.unit_rows;
        w.ahead = l.q.n - l.q.fresh + l.token;
        w.rest = l.rest;
        ++l.u;
        l.token += p.unit_tokens;
        l.rest += p.unit_rest;
        if (l.rest >= p.heads) {
            l.rest -= p.heads;
            ++l.token;
        }
        if (p.causal && --l.left == 0) {
            l.extra += p.more;
            l.left = p.step;
        }
        if (l.at >= l.unit_at) continue;
        w.seq = l.s;
        w.row = l.q.start * p.heads + r0;
        w.rows = min(p.unit_rows, min(l.q.fresh, p.max_q) * p.heads - r0);
        w.context = min(l.q.n, p.max_context);
        w.tiles = (w.seen(p, w.rows - 1) + kTok - 1) >> 6;
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
    int64_t per;          // tiles of a stretch
    Line line;
    Part part;
    int32_t some;
};

template <int THREADS>
PA_DEVICE void find_stretch(const Params& p, int group, bool report, Scan& sc) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the line's length, then the sequence in which this stretch begins: each
    // thread adds up an equal run of sequences, and the one whose run holds the
    // stretch's first tile walks it
    if (threadIdx.x == 0) sc.some = 0;
    const int run = (p.seqs + THREADS - 1) / THREADS;
    const int s0 = min(p.seqs, (int)threadIdx.x * run), s1 = min(p.seqs, s0 + run);
    Seq q;
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) {
        q = read_seq(p, s, report);
        mine += q.before(p, q.units);
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
    int64_t per = sum <= INT32_MAX ? (int64_t)((uint32_t)sum / (uint32_t)p.groups) : sum / p.groups;
    per = max(per, (int64_t)p.min_tiles);
    const int64_t at = min(total, group * per), end = min(total, at + per);
    ahead += upto - mine;
    if (at < end && ahead <= at && at < ahead + mine) {
        Line line;
        line.at = at;
        line.end = end;
        line.s = s0;
        line.unit_at = ahead;
        if (run > 1) {
            q = read_seq(p, s0, false);
            for (int64_t all; at >= line.unit_at + (all = q.before(p, q.units));) {
                line.unit_at += all;
                q = read_seq(p, ++line.s, false);
            }
        }
        line.begin(p, q);
        if (q.units > 1) {
            const int64_t off = at - line.unit_at;
            int u = 0, hi = q.units - 1;   // last unit that begins at or before `at`
            while (u < hi) {
                const int mid = (int)(((unsigned)u + hi + 1) >> 1);
                if (q.before(p, mid) <= off) u = mid; else hi = mid - 1;
            }
            const int r0 = u * p.unit_rows;
            line.unit_at += q.before(p, u);
            line.u = u;
            line.token = r0 / p.heads;
            line.rest = r0 - line.token * p.heads;
            if (p.causal) {
                line.extra = p.more * (u / p.step);
                line.left = p.step - u % p.step;
            }
        }
        sc.per = per;
        sc.some = next_part(p, line, sc.part);
        sc.line = line;
    }
    __syncthreads();
}

// Asks for rows of a tile ahead in L2.  The rings hold two tiles, too few to cover the
// latency of HBM.  The requests go through the TMA unit, a page an instruction (by the
// prefetches of a warp's own loads the issuing warps lost a third of their pace), and
// tiles too far ahead cost more than they save.  Eight contexts of 100K tokens:
// the one-CTA kernel on 64 heads 172.8 us without, 161.6, 160.6, 169.3, 182.7 one to
// four tiles ahead (on 16 heads 155.7; 149.4, 149.9, 158.1, 170.3); the pair kernel on
// 128 heads 204 us, 187, 184, 185, 190, 203 with 2, 3, 4, 6, 8 (64 contexts of 128 to 4096
// 60.0 us, 58.0, 57.1, 58.8, 60.0, 61.8).
PA_DEVICE void ask_rows(const Params& p, int row, int rows, int row_bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                 ::"l"(p.rows + (int64_t)row * row_bytes), "r"(rows * row_bytes) : "memory");
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
