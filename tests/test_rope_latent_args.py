"""Host side of the rotating writes and the latent cache (no GPU needed): the
frequency rules, the 64-bit turns, and what the binding and the C ABI refuse
before anything is enqueued."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_148_gb300 as pkv
from oracle import latent as orc

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def L():
    pkv.build()
    return pkv.lib()


@pytest.mark.parametrize("scaling", [dict(), dict(scaling="linear", factor=4.0),
                                     dict(scaling="ntk", factor=8.0),
                                     dict(scaling="by_parts", factor=16.0, original_context=4096),
                                     dict(scaling="by_parts", factor=2.0, original_context=100,
                                          fast=8.0, slow=0.5)])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_frequencies_follow_their_rules(rot, scaling):
    r = pkv.Rope(rot, base=5000.0, device="cpu", **scaling)
    f, m = orc.frequencies(rot, base=5000.0, **scaling)
    assert np.allclose(r.frequencies, f, rtol=1e-14, atol=0) and math.isclose(r.magnitude, m, rel_tol=1e-15)


def test_turns_are_the_fraction_of_a_turn():
    """turns = f / 2 pi modulo one, off by the double's own precision at most."""
    f = np.array([0.0, 1.0, 1e-4, 2 * math.pi * 0.75, 7.0, -1.0, 2 * math.pi, -1e-30, 1e9])
    r = pkv.Rope(18, frequencies=f, device="cpu")
    got = r.turns.numpy().view(np.uint64)
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    for x, t in zip(f, got):
        want = Fraction(float(x)) / two_pi % 1
        d = abs(Fraction(int(t), 2 ** 64) - want)
        d = min(d, 1 - d)                       # around the circle
        assert d <= Fraction(abs(float(x))) * Fraction(1, 2 ** 51) + Fraction(1, 2 ** 52), (x, t)


@pytest.mark.parametrize("bad", [
    dict(rot_dim=0), dict(rot_dim=7), dict(layout="pairs"), dict(scaling="other"), dict(base=0.0),
    dict(factor=0.5), dict(scaling="by_parts", factor=2.0), dict(scaling="ntk", rot_dim=2, factor=2.0),
    dict(scaling="by_parts", factor=2.0, original_context=64, fast=1.0, slow=1.0),
    dict(frequencies=[1.0]), dict(frequencies=[1.0] * 31 + [math.inf]), dict(magnitude=math.nan),
    dict(frequencies=[1.0] * 32, scaling="linear", factor=2.0),
])
def test_rope_refuses(bad):
    with pytest.raises(ValueError):
        pkv.Rope(**{**dict(rot_dim=64, device="cpu"), **bad})


def _kv(**kw):
    pool = pkv.KVPool(4, 16, 2, 128, device="cpu")
    a = dict(q=torch.zeros(3, 8, 128, dtype=BF), k_new=torch.zeros(3, 2, 128, dtype=BF),
             v_new=torch.zeros(3, 2, 128, dtype=BF), positions=torch.zeros(3, dtype=torch.int64),
             slot_mapping=torch.zeros(3, dtype=torch.int64), rope=pkv.Rope(128, device="cpu"))
    a.update(kw)
    return pkv.rope_write_kv(pool, a["q"], a["k_new"], a["v_new"], a["positions"], a["slot_mapping"],
                             a["rope"], q_out=a.get("q_out"), d_err=a.get("d_err"))


@pytest.mark.parametrize("bad,exc", [
    (dict(q=torch.zeros(3, 8, 64, dtype=BF)), ValueError),
    (dict(q=torch.zeros(3, 8, 128)), TypeError),
    (dict(q=torch.zeros(3, 1024, dtype=BF)), ValueError),
    (dict(k_new=torch.zeros(2, 2, 128, dtype=BF)), ValueError),
    (dict(v_new=torch.zeros(3, 2, 256, dtype=BF)[..., ::2]), ValueError),     # elements apart
    (dict(k_new=torch.zeros(3, 4, 128, dtype=BF)[:, ::2]), ValueError),       # heads apart
    (dict(positions=torch.zeros(3, dtype=torch.int32)), TypeError),
    (dict(positions=torch.zeros(2, dtype=torch.int64)), ValueError),
    (dict(slot_mapping=torch.zeros(3, dtype=torch.int32)), TypeError),
    (dict(rope=None), TypeError),
    (dict(q=None, q_out=torch.zeros(3, 8, 128, dtype=BF)), ValueError),
    (dict(q_out=torch.zeros(3, 4, 128, dtype=BF)), ValueError),
    (dict(d_err=torch.zeros(0, dtype=torch.int32)), ValueError),
])
def test_rope_write_refuses(bad, exc):
    with pytest.raises(exc):
        _kv(**bad)


def _latent(**kw):
    pool = pkv.LatentPool(4, 16, 128, 64, device="cpu")
    a = dict(latent=torch.zeros(3, 128, dtype=BF), k_rope=torch.zeros(3, 64, dtype=BF),
             positions=torch.zeros(3, dtype=torch.int64), slot_mapping=torch.zeros(3, dtype=torch.int64),
             rope=pkv.Rope(64, device="cpu"), q_rope=torch.zeros(3, 5, 64, dtype=BF),
             q=torch.zeros(3, 5, 192, dtype=BF))
    a.update(kw)
    return pkv.write_latent(pool, a["latent"], a["k_rope"], a["positions"], a["slot_mapping"], a["rope"],
                            q_rope=a["q_rope"], q=a["q"], d_err=a.get("d_err"))


@pytest.mark.parametrize("bad,exc", [
    (dict(latent=torch.zeros(3, 64, dtype=BF)), ValueError), (dict(latent=torch.zeros(3, 128)), TypeError),
    (dict(k_rope=torch.zeros(3, 1, 64, dtype=BF)), ValueError), (dict(q=None), ValueError),
    (dict(q_rope=None), ValueError), (dict(q=torch.zeros(3, 5, 128, dtype=BF)), ValueError),
    (dict(q_rope=torch.zeros(3, 4, 64, dtype=BF)), ValueError),
    (dict(q_rope=torch.zeros(3, 5, 128, dtype=BF)[..., ::2]), ValueError),
    (dict(rope=3), TypeError), (dict(positions=torch.zeros(3)), TypeError),
])
def test_write_latent_refuses(bad, exc):
    with pytest.raises(exc):
        _latent(**bad)


def _attend(prefill=False, **kw):
    pool = pkv.LatentPool(4, 16, 128, 64, device="cpu")
    a = dict(q=torch.zeros(2, 5, 192, dtype=BF), tables=torch.zeros(2, 3, dtype=torch.int32),
             lens=torch.ones(2, dtype=torch.int32), starts=torch.tensor([0, 1, 2], dtype=torch.int32))
    a.update(kw)
    more = {k: a[k] for k in ("out", "d_err", "workspace") if k in a}
    if prefill:
        return pkv.prefill_latent(pool, a["q"], a["starts"], a["lens"], a["tables"], 1, 48, 0.1, **more)
    return pkv.decode_latent(pool, a["q"], a["tables"], a["lens"], 48, 0.1, **more)


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("bad,exc", [
    (dict(q=torch.zeros(2, 5, 128, dtype=BF)), ValueError), (dict(q=torch.zeros(2, 5, 192)), TypeError),
    (dict(tables=torch.zeros(3, 3, dtype=torch.int32)), ValueError),
    (dict(tables=torch.zeros(2, 3, dtype=torch.int64)), TypeError),
    (dict(lens=torch.ones(2, 1, dtype=torch.int32)), ValueError),
    (dict(out=torch.zeros(2, 5, 192, dtype=BF)), ValueError), (dict(out=torch.zeros(2, 5, 128)), TypeError),
    (dict(d_err=torch.zeros(1)), TypeError), (dict(workspace=torch.zeros(8, 8)[:, ::2]), ValueError),
])
def test_latent_attention_refuses(prefill, bad, exc):
    with pytest.raises(exc):
        _attend(prefill, **bad)


def test_latent_attention_refuses_other_counts():
    with pytest.raises(ValueError):
        _attend(q=torch.zeros(3, 5, 192, dtype=BF))
    with pytest.raises(ValueError):
        _attend(True, starts=torch.tensor([0, 2], dtype=torch.int32))
    with pytest.raises(TypeError):
        pkv.LatentPool(4, 16, 128, 64, torch.float32, device="cpu")
    with pytest.raises(ValueError):
        pkv.copy_latent_blocks(pkv.LatentPool(4, 16, 128, 64, device="cpu"),
                               torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))


# ---------------------------------------------------------------- the C ABI, host errors only
def _pool(**kw):
    p = dict(rows=4096, num_blocks=8, block_size=16, latent_dim=512, rope_dim=64, dtype=pkv.DTYPE_BF16)
    p.update(kw)
    return ctypes.byref(pkv.pa_latent_pool(*[p[k] for k in ("rows", "num_blocks", "block_size",
                                                            "latent_dim", "rope_dim", "dtype")]))


def _dec(L, pool, heads=16, q=16, tables=16, width=4, lens=16, seqs=2, longest=64, scale=0.1, out=16,
         ws=None, have=0):
    return L.pa_decode_latent(pool, q, heads, tables, width, lens, seqs, longest, scale, out, ws, have, None, None)


@pytest.mark.parametrize("pool,status", [
    (dict(rows=None), 1), (dict(num_blocks=0), 1), (dict(latent_dim=-512), 1), (dict(dtype=9), 1),
    (dict(dtype=pkv.DTYPE_F32), 6), (dict(dtype=pkv.DTYPE_FP8_E4M3), 6), (dict(latent_dim=520), 6),
    (dict(latent_dim=64), 6), (dict(latent_dim=640), 6), (dict(rope_dim=80), 6), (dict(rope_dim=8), 6),
    (dict(block_size=4), 6), (dict(block_size=24), 6), (dict(block_size=256), 6),
    (dict(num_blocks=1 << 27), 6),
])
def test_decode_latent_pool_errors(L, pool, status):
    assert _dec(L, _pool(**pool)) == status
    n = ctypes.c_size_t(0)
    assert L.pa_decode_latent_workspace_bytes(_pool(**pool), 2, 16, 64, ctypes.byref(n)) == status
    assert L.pa_prefill_latent_workspace_bytes(_pool(**pool), 2, 16, 8, 4, 64, ctypes.byref(n)) == status


def test_latent_argument_errors(L):
    bad, odd = pkv.PA_ERR_INVALID_ARG, pkv.PA_ERR_UNSUPPORTED
    p = _pool()
    assert _dec(L, p, heads=0) == bad and _dec(L, p, heads=129) == odd
    assert _dec(L, p, seqs=-1) == bad and _dec(L, p, seqs=65536) == odd and _dec(L, p, longest=-1) == bad
    assert _dec(L, p, scale=math.nan) == bad and _dec(L, p, width=-1) == bad
    for name in ("q", "tables", "lens", "out"):
        assert _dec(L, p, **{name: None}) == bad
    assert _dec(L, p, q=8) == bad and _dec(L, p, out=24) == bad and _dec(L, _pool(rows=4104)) == bad
    assert _dec(L, p, seqs=0, q=None) == 0 and _dec(L, p, longest=0, q=None) == 0
    pre = lambda total=4, most=2, seqs=2, starts=16, longest=64: L.pa_prefill_latent(  # noqa: E731
        p, 16, total, 16, starts, 16, 16, 4, seqs, most, longest, 0.1, 1, 16, None, 0, None, None)
    assert pre(total=-1) == bad and pre(most=-1) == bad and pre(starts=None) == bad
    assert pre(total=0) == 0 and pre(seqs=0) == 0 and pre(most=0) == 0 and pre(longest=0) == 0
    assert pre(total=1 << 30) == odd                 # rows past 31 bits
    n = ctypes.c_size_t(0)
    assert L.pa_decode_latent_workspace_bytes(p, 2, 16, 64, None) == bad


def test_writes_argument_errors(L):
    bad, odd = pkv.PA_ERR_INVALID_ARG, pkv.PA_ERR_UNSUPPORTED

    def kv(dtype=pkv.DTYPE_BF16, dim=128, rot=128, layout=0, magnitude=1.0, turns=16, q=16, qs=1024, hq=8,
           k=16, ks=256, n=3, q_out=16, scale=16):
        pool = pkv.pa_kv_pool(4096, 4096, 8, 16, 2, dim, dtype, scale, scale)
        rope = pkv.pa_rope(turns, rot, layout, magnitude)
        return L.pa_rope_write_kv(ctypes.byref(pool), ctypes.byref(rope), q, qs, hq, k, ks, k, ks, 16, 16, n,
                                  q_out, None, None)
    assert kv(n=0) == 0 and kv(n=-1) == bad and kv(turns=None) == bad and kv(turns=12) == bad
    assert kv(rot=0) == bad and kv(rot=129) == bad and kv(rot=130) == bad and kv(layout=2) == bad
    assert kv(magnitude=math.inf) == bad and kv(rot=24) == odd and kv(dim=24, rot=16) == odd
    assert kv(dim=2048, rot=16, ks=4096, qs=16384) == odd
    assert kv(dtype=pkv.DTYPE_FP8_E4M3, dim=64, rot=64) == odd
    assert kv(q=None) == bad and kv(q_out=None) == bad and kv(q=8) == bad and kv(q_out=8) == bad
    assert kv(qs=1016) == bad and kv(qs=1028) == bad and kv(ks=255) == bad and kv(ks=260) == bad
    assert kv(k=None) == bad and kv(k=18) == bad

    def lat(rot=64, latent=16, ls=512, ks=64, n=3, q_rope=16, qs=320, qh=64, h=5, q=16, **pool):
        rope = pkv.pa_rope(16, rot, 0, 1.0)
        return L.pa_write_latent(_pool(**pool), ctypes.byref(rope), latent, ls, 16, ks, 16, 16, n, q_rope, qs,
                                 qh, h, q, None, None)
    assert lat(n=0) == 0 and lat(n=-1) == bad and lat(rot=32) == bad and lat(latent=None) == bad
    assert lat(ls=504) == bad and lat(ls=516) == bad and lat(ks=32) == bad and lat(q=None) == bad
    assert lat(q_rope=None) == bad and lat(q_rope=8) == bad and lat(qh=60) == bad and lat(qs=312) == bad
    assert lat(rope_dim=24, rot=24) == odd and lat(dtype=pkv.DTYPE_F32) == odd
    cp = lambda n=1, src=16, **pool: L.pa_copy_latent_blocks(_pool(**pool), src, 16, n, None, None)  # noqa: E731
    assert cp(0, None) == 0 and cp(-1) == bad and cp(1, None) == bad and cp(rows=4104) == bad
