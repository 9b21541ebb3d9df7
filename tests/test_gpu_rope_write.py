"""GPU parity of the rotating writes: pa_rope_write_kv (q rotated, rotated K and
plain V scattered to float32, bf16 and FP8 pages) and pa_write_latent, against
the float64 oracle with bounds from the roundings (oracle/latent.py)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_148_gb300 as pkv
from oracle import latent as orc

pytestmark = pytest.mark.gpu

F32, BF16 = orc.F32, orc.BF16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.build()
    pkv.lib()
    yield
    torch.cuda.synchronize()


def _randn(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float32).to(dtype).cuda()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _within(got, ref, bound, what):
    got = _f64(got) if isinstance(got, torch.Tensor) else got
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), "%s: %.3g over the bound of %.3g" % (
        what, over.max(), bound.reshape(-1)[over.argmax()])


def _slots(seed, T, blocks, bp):
    return torch.from_numpy(np.random.default_rng(seed).permutation(blocks * bp)[:T].astype(np.int64)).cuda()


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="by_parts", factor=16.0, original_context=4096)]

CASES = [
    # T, Hq, Hkv, D, bp, pool dtype, rot, layout, scaling
    (1, 1, 1, 64, 4, "f32", 64, "half", 0),
    (4, 4, 2, 64, 4, "f32", 64, "interleaved", 0),
    (37, 8, 8, 128, 16, "f32", 72, "half", 1),
    (3, 3, 1, 16, 8, "f32", 8, "interleaved", 2),
    (1, 32, 8, 128, 16, "bf16", 128, "half", 0),
    (65, 7, 1, 128, 16, "bf16", 128, "interleaved", 3),
    (19, 6, 2, 96, 8, "bf16", 96, "half", 2),
    (129, 5, 5, 80, 16, "bf16", 16, "half", 1),
    (700, 4, 2, 128, 3, "bf16", 64, "interleaved", 3),
    (613, 2, 1, 256, 32, "bf16", 48, "half", 0),
    (33, 8, 1, 128, 16, "fp8", 128, "half", 3),
    (609, 3, 2, 128, 4, "fp8", 64, "interleaved", 0),
    (5, 1, 3, 128, 64, "fp8", 16, "half", 1),
]


def _pages(pool_tensor, slots, bp):
    """Rows [T][H][...] that the slots hold."""
    blk, off = slots // bp, slots % bp
    return pool_tensor[blk, :, off]


@pytest.mark.parametrize("T,Hq,Hkv,D,bp,dtype,rot,layout,sc", CASES)
@pytest.mark.parametrize("fused_input", [False, True])
def test_rope_write_matches_oracle(T, Hq, Hkv, D, bp, dtype, rot, layout, sc, fused_input):
    io = torch.float32 if dtype == "f32" else torch.bfloat16
    store = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}[dtype]
    blocks = T // bp + 3
    pool = pkv.KVPool(blocks, bp, Hkv, D, store).poison()
    if fused_input:
        qkv = _randn(T, T, (Hq + 2 * Hkv) * D, dtype=io)
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        q, k, v = (_randn(T + i, T, h, D, dtype=io) for i, h in enumerate((Hq, Hkv, Hkv)))
    rng = np.random.default_rng(T * 31 + rot)
    pos = rng.integers(0, 1 << 20, T)
    pos[0] = 0
    pos[-1] = -5 if T > 2 else pos[-1]
    slots = _slots(T, T, blocks, bp)
    scaling = SCALINGS[sc]
    rope = pkv.Rope(rot, layout=layout, **scaling)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = [None if x is None else x.clone() for x in (pool.k, pool.v, pool.k_scale, pool.v_scale)]
    out = pkv.rope_write_kv(pool, q, k, v, torch.from_numpy(pos).cuda(), slots, rope, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    f, m = orc.frequencies(rot, **scaling)
    unit = F32 if dtype == "f32" else BF16
    ref, off = orc.rotate(_f64(q), pos, f, layout, m)
    # one rounding to the output's type on top of the float32 error
    _within(out, ref, off + unit * (np.abs(ref) + off), "q")
    kref, koff = orc.rotate(_f64(k), pos, f, layout, m)
    if dtype != "fp8":
        _within(_pages(pool.k, slots, bp), kref, koff + unit * (np.abs(kref) + koff), "k")
        assert torch.equal(_pages(pool.v, slots, bp), v), "v is copied bit for bit"
    else:
        codes = _f64(_pages(pool.k, slots, bp).view(torch.float8_e4m3fn))
        scale = _f64(_pages(pool.k_scale, slots, bp))[..., None]
        top = np.abs(kref).max(-1, keepdims=True)
        toff = koff.max(-1, keepdims=True)
        _within(scale, top / 448, (toff + top * F32) / 448 + top / 448 * F32, "k scale")
        # a code is off by half a step: 2^-4 of its value, or 2^-10 below the normal range
        _within(codes * scale, kref,
                2.0 ** -4 * np.abs(kref) * 1.001 + 2.0 ** -10 * scale + 2 * (koff + toff), "k codes")
        vb = _f64(v)
        got = _f64(_pages(pool.v, slots, bp).view(torch.float8_e4m3fn)) * \
            _f64(_pages(pool.v_scale, slots, bp))[..., None]
        plain = pkv.KVPool(blocks, bp, Hkv, D, store).poison()
        pkv.write_kv(plain, k.contiguous(), v.contiguous(), slots)
        assert torch.equal(plain.v, pool.v) and torch.equal(
            plain.v_scale.view(torch.int32), pool.v_scale.view(torch.int32)), "v as pa_write_kv"
        assert np.abs(got - vb).max() <= 0.07 * np.abs(vb).max()
    # every other slot is left as it was
    free = torch.ones(blocks * bp, dtype=torch.bool, device="cuda")
    free[slots] = False
    rest = free.nonzero()[:, 0]
    for now, was in zip((pool.k, pool.v, pool.k_scale, pool.v_scale), before):
        if now is not None:
            a, b = (_pages(x, rest, bp).contiguous().view(torch.uint8) for x in (now, was))
            assert torch.equal(a, b)


def test_rope_equals_write_kv_at_position_zero():
    pool, plain = (pkv.KVPool(9, 16, 2, 128).poison() for _ in range(2))
    q, k, v = (_randn(i, 100, h, 128) for i, h in enumerate((4, 2, 2)))
    pos, slots = torch.zeros(100, dtype=torch.int64, device="cuda"), _slots(1, 100, 9, 16)
    out = pkv.rope_write_kv(pool, q, k, v, pos, slots, pkv.Rope(128))
    pkv.write_kv(plain, k, v, slots)
    torch.cuda.synchronize()
    assert torch.equal(out, q)
    for a, b in ((pool.k, plain.k), (pool.v, plain.v)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_in_place_and_without_queries(layout):
    pool, other = (pkv.KVPool(9, 16, 2, 128).poison() for _ in range(2))
    q, k, v = (_randn(i, 77, h, 128) for i, h in enumerate((4, 2, 2)))
    pos, slots = torch.arange(77, device="cuda"), _slots(1, 77, 9, 16)
    rope = pkv.Rope(96, layout=layout)
    out = pkv.rope_write_kv(pool, q, k, v, pos, slots, rope)
    same = pkv.rope_write_kv(other, None, k, v, pos, slots, rope)
    own = q.clone()
    assert pkv.rope_write_kv(other, own, k, v, pos, slots, rope, q_out=own) is own and same is None
    torch.cuda.synchronize()
    assert torch.equal(out, own)
    assert torch.equal(pool.k.view(torch.int16), other.k.view(torch.int16))


def test_rope_far_positions_keep_their_angles():
    """A position near 2^40 turns as exactly as one near zero."""
    pos = np.array([0, 1, 131071, 2 ** 31 + 7, 2 ** 40 + 12345, -(2 ** 33) - 1])
    T, rot = len(pos), 64
    # frequencies that are exact fractions of a turn: p * f modulo one turn is exact too
    turns = np.arange(1, rot // 2 + 1) * 2.0 ** -20
    pool = pkv.KVPool(2, 16, 1, 64, torch.float32)
    q = _randn(3, T, 2, 64, dtype=torch.float32)
    k = _randn(4, T, 1, 64, dtype=torch.float32)
    rope = pkv.Rope(rot, frequencies=turns * 2 * np.pi)
    out = pkv.rope_write_kv(pool, q, k, k, torch.from_numpy(pos).cuda(), torch.arange(T, device="cuda"), rope)
    torch.cuda.synchronize()
    left = np.array([[(int(p) * int(t * 2 ** 20)) % 2 ** 20 / 2 ** 20 for t in turns] for p in pos])
    c, s = np.cos(2 * np.pi * left)[:, None], np.sin(2 * np.pi * left)[:, None]
    x, y = np.split(_f64(q), 2, -1)
    ref = np.concatenate([x * c - y * s, x * s + y * c], -1)
    both = np.tile(np.abs(x) + np.abs(y), 2)
    # the frequency, at most 2^-15 turn, went through two roundings of a double (2^-52 of it) and
    # one of 2^-64 turn: times 2^40 positions, 2^-27 and 2^-24 turn
    assert (np.abs(_f64(out) - ref) <= both * (2.0 ** -20 + 2 * np.pi * (2.0 ** -27 + 2.0 ** -24))).all()


def test_bad_slots_are_flagged_and_skipped():
    for dtype in (torch.bfloat16, torch.float8_e4m3fn):
        pool = pkv.KVPool(4, 16, 2, 128, dtype).poison()
        was = pool.k.clone()
        k, q = _randn(1, 3, 2, 128), _randn(2, 3, 4, 128)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        slots = torch.tensor([-1, 64, 5], device="cuda")
        pos = torch.zeros(3, dtype=torch.int64, device="cuda")
        out = pkv.rope_write_kv(pool, q, k, k, pos, slots, pkv.Rope(128), d_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == pkv.PA_ERR_OUT_OF_RANGE and torch.equal(out, q)
        now, was = pool.k.view(torch.uint8), was.view(torch.uint8)
        same = (now == was).flatten(-1).all(-1)                     # [block][head][offset]
        assert bool(same[1:].all()) and not bool(same[0, :, 5].any()) and int((~same).sum()) == 2
    lp = pkv.LatentPool(4, 16, 128, 64).poison()
    was = lp.rows.clone()
    err.zero_()
    pkv.write_latent(lp, _randn(1, 3, 128), _randn(2, 3, 64), pos, slots, pkv.Rope(64), d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pkv.PA_ERR_OUT_OF_RANGE
    same = (lp.rows.view(torch.int16) == was.view(torch.int16)).all(-1)
    assert not bool(same[0, 5]) and int((~same).sum()) == 1


LATENT_CASES = [
    # T, H, latent, rope, bp, layout
    (1, 1, 128, 16, 8, "half"), (1, 128, 512, 64, 64, "interleaved"), (7, 3, 256, 48, 16, "half"),
    (66, 16, 512, 64, 5, "interleaved"), (613, 5, 512, 32, 16, "half"), (3, 0, 48, 16, 4, "half"),
]


@pytest.mark.parametrize("T,H,L,R,bp,layout", LATENT_CASES)
@pytest.mark.parametrize("sliced", [False, True])
def test_write_latent_matches_oracle(T, H, L, R, bp, layout, sliced):
    blocks = T // bp + 2
    pool = pkv.LatentPool(blocks, bp, L, R).poison()
    if sliced:
        kv = _randn(T, T, L + R + 8)
        lat, kr = kv[:, :L], kv[:, L:L + R]
        qr = _randn(T + 1, T, H, 40 + R)[..., 40:] if H else None
    else:
        lat, kr = _randn(T, T, L), _randn(T + 5, T, R)
        qr = _randn(T + 1, T, H, R) if H else None
    q = _randn(T + 2, T, H, L + R) if H else None
    absorbed = None if q is None else q[..., :L].clone()
    pos = np.random.default_rng(T).integers(0, 1 << 20, T)
    slots = _slots(T, T, blocks, bp)
    scaling = SCALINGS[3]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    was = pool.rows.clone()
    got = pkv.write_latent(pool, lat, kr, torch.from_numpy(pos).cuda(), slots,
                           pkv.Rope(R, layout=layout, **scaling), q_rope=qr, q=q, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and got is q
    f, m = orc.frequencies(R, **scaling)
    flat = pool.rows.view(-1, L + R)
    assert torch.equal(flat[slots, :L], lat)
    ref, off = orc.rotate(_f64(kr)[:, None], pos, f, layout, m)
    _within(flat[slots, L:], ref[:, 0], (off + BF16 * (np.abs(ref) + off))[:, 0], "rotary key")
    if H:
        assert torch.equal(q[..., :L], absorbed)
        ref, off = orc.rotate(_f64(qr), pos, f, layout, m)
        _within(q[..., L:], ref, off + BF16 * (np.abs(ref) + off), "rotary query")
    free = torch.ones(blocks * bp, dtype=torch.bool, device="cuda")
    free[slots] = False
    assert torch.equal(flat[free].view(torch.int16), was.view(-1, L + R)[free].view(torch.int16))


def test_copy_latent_blocks():
    for n, bp, L in ((1, 16, 512), (37, 8, 256), (64, 128, 512)):
        pool = pkv.LatentPool(2 * n + 3, bp, L, 64)
        pool.rows.copy_(_randn(n, *pool.rows.shape))
        order = torch.from_numpy(np.random.default_rng(n).permutation(2 * n + 3).astype(np.int32)).cuda()
        src, dst = order[:n].contiguous(), order[n:2 * n].contiguous()
        want = pool.rows.clone()
        want[dst.long()] = want[src.long()]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.copy_latent_blocks(pool, src, dst, d_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and torch.equal(pool.rows, want)
        bad = torch.tensor([0, 2 * n + 3, -1], dtype=torch.int32, device="cuda")
        pkv.copy_latent_blocks(pool, bad, bad.flip(0).contiguous(), d_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == pkv.PA_ERR_OUT_OF_RANGE and torch.equal(pool.rows, want)
