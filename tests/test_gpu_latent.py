"""GPU parity of latent attention in the absorbed form (pa_decode_latent,
pa_prefill_latent) with the float64 oracle, elementwise within the bound that
the roundings set (oracle/latent.py)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_148_gb300 as pkv
from oracle import latent as orc
from paged_kv_cache_148_gb300.cache import PagedLatentCache

pytestmark = pytest.mark.gpu

REL_L2 = 2.0 ** -8  # two independent roundings of half a bf16 step at most, 2^-8 each at their worst


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.build()
    pkv.lib()
    yield
    torch.cuda.synchronize()


def _f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """A poisoned latent pool with the rows of some sequences, and their tables."""

    def __init__(self, lens, heads, latent=512, rope=64, bp=16, new=None, seed=0, spread=1.0,
                 slack=3, mean=0.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.latent, self.bp = list(lens), heads, latent, bp
        self.new = [1] * len(lens) if new is None else list(new)
        pages = [-(-n // bp) for n in lens]
        blocks = sum(pages) + slack
        order = rng.permutation(blocks)
        width = max(1, max(pages, default=1))
        self.pool = pkv.LatentPool(blocks, bp, latent, rope).poison()
        table = np.full((len(lens), width), -1, np.int32)
        at = 0
        self.slots = []
        for s, n in enumerate(lens):
            table[s, :pages[s]] = order[at:at + pages[s]]
            at += pages[s]
            j = np.arange(n)
            self.slots.append(table[s][j // bp].astype(np.int64) * bp + j % bp)
        slots = torch.from_numpy(np.concatenate(self.slots + [np.zeros(0, np.int64)]))
        rows = (torch.randn(len(slots), latent + rope, generator=g) * spread + mean).to(torch.bfloat16)
        self.pool.rows.view(-1, latent + rope)[slots.cuda()] = rows.cuda()
        self.table_host = table
        self.tables = torch.from_numpy(table).cuda()
        self.context = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.starts_host = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.starts = torch.from_numpy(self.starts_host).cuda()
        self.q = torch.randn(int(self.starts_host[-1]), heads, latent + rope, generator=g).to(torch.bfloat16).cuda()
        self.longest = max(self.lens, default=0)
        self.scale = (128 + rope) ** -0.5
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def decode(self, **kw):
        return pkv.decode_latent(self.pool, self.q, self.tables, self.context,
                                 kw.pop("max_context", self.longest), kw.pop("scale", self.scale),
                                 d_err=self.err, **kw)

    def prefill(self, causal=True, **kw):
        return pkv.prefill_latent(self.pool, self.q, self.starts, self.context, self.tables,
                                  kw.pop("max_q_len", max(self.new)), kw.pop("max_context", self.longest),
                                  kw.pop("scale", self.scale), causal=causal, d_err=self.err, **kw)

    def code(self):
        torch.cuda.synchronize()
        return int(self.err.item())

    def reference(self, causal=True, decode=False, scale=None, only=None, tokens=None):
        """out and bound of sequence s's queries, for s in only."""
        rows = _f64(self.pool.rows.view(-1, self.pool.width))
        q = _f64(self.q)
        out, bound = {}, {}
        for s in range(len(self.lens)) if only is None else only:
            keys = rows[self.slots[s]]
            a, b = self.starts_host[s], self.starts_host[s + 1]
            n, new = self.lens[s], b - a
            for i in range(new):
                if tokens is not None and i not in tokens:
                    continue
                seen = n - new + i + 1 if causal and not decode else n
                out[s, i], bound[s, i] = orc.attend(q[a + i], keys, self.scale if scale is None else scale,
                                                    self.latent, [seen] * self.heads)
        return out, bound

    def check(self, got, ref, bound, what=""):
        got = _f64(got)
        num = den = 0.0
        for (s, i), o in ref.items():
            x = got[self.starts_host[s] + i]
            assert np.isfinite(x).all(), "%s: sequence %d token %d is not finite" % (what, s, i)
            over = np.abs(x - o) - bound[s, i]
            assert (over <= 0).all(), "%s: sequence %d token %d: %.3g over the bound (out %.3g)" % (
                what, s, i, over.max(), np.abs(o).max())
            num += ((x - o) ** 2).sum()
            den += (o ** 2).sum()
        assert num <= REL_L2 ** 2 * den or den == 0, "%s: rel L2 %.3g" % (what, (num / den) ** 0.5)


EDGES = [1, 2, 7, 8, 9, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 200, 513]


@pytest.mark.parametrize("bp", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("heads,latent,rope", [(1, 512, 64), (16, 512, 64), (128, 512, 64),
                                               (20, 256, 32), (65, 128, 16), (7, 384, 48)])
def test_decode_edge_lengths(bp, heads, latent, rope):
    b = Batch(EDGES, heads, latent, rope, bp, seed=bp + heads)
    out = b.decode()
    assert b.code() == 0
    b.check(out, *b.reference(decode=True), "bp %d" % bp)


@pytest.mark.parametrize("heads", [1, 8, 16, 24, 33, 48, 64, 65, 96, 127, 128])
def test_decode_head_counts(heads):
    b = Batch([300, 1, 77], heads, bp=16, seed=heads)
    out = b.decode()
    assert b.code() == 0
    b.check(out, *b.reference(decode=True))


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_decode_one_long_context(heads):
    """A lone context, split over the whole machine."""
    b = Batch([20011], heads, bp=64, seed=heads)
    out = b.decode()
    assert b.code() == 0
    b.check(out, *b.reference(decode=True))


def test_decode_many_sequences():
    lens = [1 + (37 * i) % 400 for i in range(500)]
    b = Batch(lens, 8, 256, 64, bp=32, seed=3)
    out = b.decode()
    assert b.code() == 0
    b.check(out, *b.reference(decode=True, only=range(0, 500, 17)))


def test_decode_scores_far_apart():
    """Scores of several hundred: the running maximum grows again and again, and most weights vanish."""
    b = Batch([700, 90, 64], 16, bp=16, seed=5, spread=6.0)
    # contexts whose rows grow along the positions: every tile beats the one before
    flat = b.pool.rows.view(-1, b.pool.width)
    for s, sl in enumerate(b.slots):
        g = torch.linspace(0.1, 3.0, len(sl)).cuda()[:, None]
        flat[torch.from_numpy(sl).cuda()] = (flat[torch.from_numpy(sl).cuda()].float() * g).to(torch.bfloat16)
    out = b.decode()
    assert b.code() == 0
    b.check(out, *b.reference(decode=True))


def test_decode_all_scores_very_low():
    """Equal rows and a large negative score: the weights are still one over n."""
    b = Batch([130], 4, bp=16, seed=6)
    b.pool.rows.view(-1, b.pool.width)[torch.from_numpy(b.slots[0]).cuda()] = 8.0
    b.q.fill_(-8.0)
    out = b.decode(scale=1.0)
    assert b.code() == 0
    assert torch.equal(out, torch.full_like(out, 8.0))


def test_decode_empty_context_leaves_out():
    b = Batch([40, 0, 3], 16, bp=16, seed=7)
    out = torch.full((3, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    b.decode(out=out)
    assert b.code() == 0
    assert bool((out[1] == 7).all())
    b.check(out, *b.reference(decode=True, only=[0, 2]))
    z = Batch([0, 0], 8, bp=8, seed=8)
    out = torch.full((2, 8, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    z.decode(out=out, max_context=64)
    assert z.code() == 0 and bool((out == 7).all())


def test_decode_context_longer_than_stated():
    b = Batch([300, 50], 16, bp=16, seed=9)
    out = b.decode(max_context=100)
    assert b.code() == pkv.PA_ERR_OUT_OF_RANGE
    b.lens = [100, 50]
    b.slots[0] = b.slots[0][:100]
    b.check(out, *b.reference(decode=True))


@pytest.mark.parametrize("heads", [8, 128])
@pytest.mark.parametrize("bp", [8, 64])
def test_decode_bad_pages_are_skipped(heads, bp):
    b = Batch([400, 3 * bp, 130], heads, bp=bp, seed=10)
    t = b.table_host.copy()
    gone = {0: [1, 3], 1: [0, 1, 2]}          # sequence 1 loses every page
    for s, pages in gone.items():
        for i in pages:
            t[s, i] = -7 if i % 2 else b.pool.num_blocks + 5
    b.tables.copy_(torch.from_numpy(t))
    out = b.decode()
    assert b.code() in (pkv.PA_ERR_OUT_OF_RANGE, pkv.PA_ERR_NEGATIVE_BLOCK)
    assert bool((out[1] == 0).all())
    j = np.arange(400)
    b.slots[0] = b.slots[0][~np.isin(j // bp, gone[0])]
    b.lens[0] = len(b.slots[0])
    b.check(out, *b.reference(decode=True, only=[0, 2]))


def test_decode_narrow_table():
    """A table with fewer entries than the context needs: the missing pages are flagged and skipped."""
    b = Batch([100], 16, bp=16, seed=11)
    b.tables = b.tables[:, :4].contiguous()
    out = b.decode()
    assert b.code() != 0
    b.lens, b.slots = [64], [b.slots[0][:64]]
    b.check(out, *b.reference(decode=True))


PREFILL = [
    # context lengths with the new tokens, new tokens, heads, latent, rope, bp
    ([1], [1], 1, 512, 64, 8), ([5, 5], [5, 5], 16, 512, 64, 16),
    ([70, 64, 65, 130], [1, 64, 3, 130], 16, 512, 64, 16),
    ([300, 9, 64], [17, 9, 2], 20, 256, 32, 32), ([200, 77], [33, 77], 128, 512, 64, 64),
    ([90, 20], [5, 20], 65, 128, 16, 8), ([500, 33], [100, 33], 7, 384, 48, 128),
    ([66], [66], 1, 512, 64, 16),
]


@pytest.mark.parametrize("lens,new,heads,latent,rope,bp", PREFILL)
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_matches_oracle(lens, new, heads, latent, rope, bp, causal):
    b = Batch(lens, heads, latent, rope, bp, new=new, seed=len(lens) * heads)
    out = b.prefill(causal=causal)
    assert b.code() == 0
    b.check(out, *b.reference(causal=causal))


@pytest.mark.parametrize("heads", [16, 128])
def test_prefill_few_rows_on_long_contexts(heads):
    b = Batch([9001, 4097], heads, bp=64, new=[3, 1], seed=heads)
    out = b.prefill()
    assert b.code() == 0
    b.check(out, *b.reference())


def test_prefill_of_single_tokens_is_decode():
    lens = [1, 63, 64, 65, 1000, 129]
    b = Batch(lens, 32, bp=16, seed=12)
    a, d = b.prefill(), b.decode()
    assert b.code() == 0
    ref = b.reference(decode=True)
    b.check(a, *ref)
    b.check(d, *ref)


def test_prefill_skips_and_keeps_rows():
    """Sequences with no new token, and rows behind the last sequence, are left as they were."""
    b = Batch([40, 30, 50], 16, bp=16, new=[3, 0, 2], seed=13)
    q = torch.cat([b.q, torch.full_like(b.q[:4], float("nan"))])
    out = torch.full((9, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.prefill_latent(b.pool, q, b.starts, b.context, b.tables, 3, 50, b.scale, out=out, d_err=b.err)
    assert b.code() == 0
    assert bool((out[5:] == 7).all())
    b.check(out, *b.reference())


def test_prefill_bad_lengths_are_flagged():
    def flagged(starts, lens, max_q=5, max_context=64):
        b = Batch([40, 30], 16, bp=16, new=[3, 2], seed=14)
        b.err.zero_()
        out = torch.full((5, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        pkv.prefill_latent(b.pool, b.q, torch.tensor(starts, dtype=torch.int32).cuda(),
                           torch.tensor(lens, dtype=torch.int32).cuda(), b.tables, max_q, max_context,
                           b.scale, out=out, d_err=b.err)
        return b, out, b.code()
    b, out, code = flagged([0, 3, 9], [40, 30])          # leaves q's rows
    assert code == pkv.PA_ERR_OUT_OF_RANGE and bool((out[3:] == 7).all())
    b.check(out, *b.reference(only=[0]))
    b, out, code = flagged([0, 3, 1], [40, 30])          # descends
    assert code == pkv.PA_ERR_OUT_OF_RANGE and bool((out[3:] == 7).all())
    b, out, code = flagged([0, 3, 5], [40, 1])           # more new tokens than context
    assert code == pkv.PA_ERR_INVALID_ARG and bool((out[3:] == 7).all())
    b.check(out, *b.reference(only=[0]))
    b, out, code = flagged([0, 3, 5], [40, 30], max_q=2)  # more than stated: the first two are done
    assert code == pkv.PA_ERR_OUT_OF_RANGE and bool((out[2] == 7).all())
    b.check(out, *b.reference(tokens=[0, 1]))


def test_calls_on_another_stream_and_in_graphs():
    b = Batch([700, 90, 1300], 16, bp=16, seed=15)
    ref = b.reference(decode=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = b.decode(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b.check(out, *ref, "side stream")
    ws = pkv.decode_latent_workspace(b.pool, 3, 16, b.longest)
    with torch.cuda.stream(side):
        b.decode(workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.decode(workspace=ws)
        again = b.prefill()
    for _ in range(3):
        out.zero_()
        again.zero_()
        graph.replay()
        assert b.code() == 0
        b.check(out, *ref, "graph")
        b.check(again, *ref, "graph")
    # lengths change between replays, as they do from step to step
    b.context.copy_(torch.tensor([650, 1, 1300], dtype=torch.int32))
    b.lens, b.slots = [650, 1, 1300], [b.slots[0][:650], b.slots[1][:1], b.slots[2]]
    graph.replay()
    assert b.code() == 0
    b.check(out, *b.reference(decode=True), "graph, other lengths")


def test_same_call_twice_gives_the_same_bits():
    b = Batch([5000, 33, 700], 64, bp=64, seed=16)
    a, c = b.decode(), b.decode()
    p, r = b.prefill(), b.prefill()
    assert b.code() == 0 and torch.equal(a, c) and torch.equal(p, r)


def test_decoding_through_the_cache():
    """Write, fork, copy on write, decode and a chunk behind the cached part, as a server runs them."""
    L, R, H, bp = 256, 64, 16, 16
    cache = PagedLatentCache(64, bp, L, R)
    rope = pkv.Rope(R, layout="interleaved")
    g = torch.Generator().manual_seed(17)

    def draw(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()
    f, m = orc.frequencies(R)
    keys, lat, pos = {}, {}, {}

    def add(sid, n, q_heads=0):
        first = cache.lengths[sid]
        p = torch.arange(first, first + n, device="cuda")
        c, kr = draw(n, L), draw(n, R)
        q = qr = None
        if q_heads:
            q, qr = draw(n, q_heads, L + R), draw(n, q_heads, R)
        cache.append(sid, c, kr, p, rope, q_rope=qr, q=q)
        rot, _ = orc.rotate(_f64(kr)[:, None], _f64(p), f, "interleaved", m)
        rows = np.concatenate([_f64(c), _f64(torch.from_numpy(rot[:, 0]).to(torch.bfloat16))], 1)
        keys[sid] = np.concatenate([keys.get(sid, np.zeros((0, L + R))), rows])
        return q
    a = cache.add_sequence()
    add(a, 37)
    b = cache.fork(a)
    keys[b] = keys[a]
    for sid in (a, b):
        add(sid, 1)
    qa, qb = add(a, 5, H), add(b, 2, H)
    q = torch.cat([qa, qb])
    starts = torch.tensor([0, 5, 7], dtype=torch.int32).cuda()
    tables, lens = cache.block_tables([a, b]), cache.context_lens([a, b])
    out = pkv.prefill_latent(cache.pool, q, starts, lens, tables, 5, 64, 0.1)
    torch.cuda.synchronize()
    got = _f64(out)
    at = 0
    for sid, n in ((a, 5), (b, 2)):
        total = len(keys[sid])
        assert total == cache.lengths[sid]
        for i in range(n):
            ref, bound = orc.attend(_f64(q[at]), keys[sid], 0.1, L, [total - n + i + 1] * H)
            # the rotated key may round to the other neighbour: half a bf16 step of an element, in the score
            extra = 2.0 ** -7 * 0.1 * (np.abs(_f64(q[at])[:, L:]) @ np.abs(keys[sid][:, L:]).T).max()
            assert (np.abs(got[at] - ref) <= bound + 2 * np.expm1(extra) * np.abs(keys[sid][:, :L]).max()).all()
            at += 1
    d = pkv.decode_latent(cache.pool, q[[4, 6]].contiguous(), tables, lens, 64, 0.1)
    torch.cuda.synchronize()
    assert np.abs(_f64(d) - got[[4, 6]]).max() <= 2.0 ** -6 * np.abs(got).max()


@pytest.mark.parametrize("heads", [16, 128])
def test_pages_past_four_gigabytes(heads):
    """Pages whose bytes lie past 2^32: every page at the end of a pool of 5.3 GB."""
    pool = pkv.LatentPool(72000, 64, 512, 64)
    assert pool.rows.numel() * 2 > 1 << 32
    n, rope = 500, pkv.Rope(64)
    ids = torch.arange(pool.num_blocks - 8, pool.num_blocks, dtype=torch.int32, device="cuda").flip(0)
    j = torch.arange(n, device="cuda")
    slots = ids.long()[j // 64] * 64 + j % 64
    g = torch.Generator().manual_seed(heads)
    draw = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    lat, kr, q = draw(n, 512), draw(n, 64), draw(1, heads, 576)
    pos = torch.zeros(n, dtype=torch.int64, device="cuda")
    pkv.write_latent(pool, lat, kr, pos, slots, rope)
    # the last page moves to the front of the pool and back
    src, dst = ids[7:].contiguous(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.copy_latent_blocks(pool, src, dst)
    pool.rows[ids[7].item()] = float("nan")
    pkv.copy_latent_blocks(pool, dst, src)
    out = pkv.decode_latent(pool, q, ids[None].contiguous(), torch.tensor([n], dtype=torch.int32).cuda(), n, 0.07)
    torch.cuda.synchronize()
    ref, bound = orc.attend(_f64(q[0]), np.concatenate([_f64(lat), _f64(kr)], 1), 0.07, 512, [n] * heads)
    assert (np.abs(_f64(out[0]) - ref) <= bound).all()


@pytest.mark.parametrize("heads", [16, 128])
def test_two_calls_at_once(heads):
    """Two streams, a workspace each, many times over: the calls do not meet."""
    a, b = Batch([2000, 77, 900], heads, bp=16, seed=20), Batch([64, 1500], heads, bp=64, seed=21)
    want_a, want_b = a.decode(), b.decode()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append((a.decode(stream=sa), b.decode(stream=sb)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want_a) and torch.equal(y, want_b)
    a.check(want_a, *a.reference(decode=True))


@pytest.mark.parametrize("heads", [64, 128])
def test_graphs_of_both_kernels(heads):
    """A captured chunk and a captured step share one workspace, replayed in turn."""
    b = Batch([700, 90, 1300], heads, bp=16, new=[40, 1, 65], seed=22)
    d = Batch([700, 90, 1300], heads, bp=16, seed=22)
    need = max(pkv.prefill_latent_workspace_bytes(b.pool, 3, heads, 106, 65, 1300),
               pkv.decode_latent_workspace_bytes(d.pool, 3, heads, 1300))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want_p, want_d = b.prefill(workspace=ws), d.decode(workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: b.prefill(workspace=ws), lambda: d.decode(workspace=ws)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want_p) and torch.equal(graphs[1][1], want_d)
    b.check(want_p, *b.reference(tokens=[0, 39, 64]))


def test_the_same_page_twice():
    """A table may name a page twice, and two sequences the same pages."""
    b = Batch([128, 128], 16, bp=64, seed=23)
    b.tables.copy_(torch.tensor([[b.table_host[0, 0]] * 2, [b.table_host[0, 0]] * 2], dtype=torch.int32))
    out = b.decode()
    assert b.code() == 0
    twice = np.concatenate([b.slots[0][:64]] * 2)
    b.slots = [twice, twice]
    b.check(out, *b.reference(decode=True))


def test_later_rows_that_are_not_finite_stay_out():
    """Rows behind a unit's last query, written or not, do not reach it."""
    b = Batch([300], 128, bp=16, new=[2], seed=24)
    flat = b.pool.rows.view(-1, b.pool.width)
    flat[int(b.slots[0][299])] = float("inf")
    out = b.prefill()            # 128 rows a unit: the first token alone
    assert b.code() == 0
    b.check(out, *b.reference(tokens=[0]))
    assert not torch.isfinite(out[1]).all()


def test_negative_scale():
    b = Batch([300, 9], 16, bp=16, seed=25)
    out = b.decode(scale=-0.05)
    assert b.code() == 0
    b.check(out, *b.reference(decode=True, scale=-0.05))


def test_rotated_append_through_the_cache():
    """Positions, copy on write and attention of an ordinary cache, as a server runs them."""
    from paged_kv_cache_148_gb300.cache import PagedCache
    cache = PagedCache(64, 16, 2, 128)
    plain = PagedCache(64, 16, 2, 128)
    rope = pkv.Rope(128)
    g = torch.Generator().manual_seed(26)
    draw = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    a, pa = cache.add_sequence(), plain.add_sequence()
    f, m = orc.frequencies(128)
    tails = []
    side = torch.cuda.Stream()
    for step, n in enumerate((21, 1, 5)):
        if step == 1:
            a, pa = cache.fork(a), plain.fork(pa)
        first = cache.lengths[a]
        q, k, v = draw(n, 8, 128), draw(n, 2, 128), draw(n, 2, 128)
        side.wait_stream(torch.cuda.current_stream())
        out = cache.append_rotated(a, q, k, v, rope, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        pos = np.arange(first, first + n)
        rk, _ = orc.rotate(_f64(k), pos, f, "half", m)
        plain.append(pa, torch.from_numpy(rk).to(torch.bfloat16), v)
        ref, off = orc.rotate(_f64(q), pos, f, "half", m)
        assert (np.abs(_f64(out) - ref) <= off + orc.BF16 * (np.abs(ref) + off)).all()
        tails.append(out[-1:])
    o = [pkv.decode(c.pool, tails[-1], c.block_tables([s]), c.context_lens([s]), 64, 0.09)
         for c, s in ((cache, a), (plain, pa))]
    torch.cuda.synchronize()
    # keys differ by the last bit of bf16 at most where the two roundings disagree
    assert (o[0] - o[1]).abs().max().item() <= 2.0 ** -7 * o[1].abs().max().item()
