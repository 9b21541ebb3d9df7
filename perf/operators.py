"""Cases of the position and latent-cache operators: rotary positions fused with
the paged write, and the latent cache (write, block copy, decode and chunked
prefill in the absorbed form).

With ``own`` false ``run`` computes an operator from elementary torch
operations in 32 bits (64 for angles), rounded once at the end; with ``own``
true it makes the calls of ``paged_kv_cache_148_gb300`` that a serving program
makes.  ``exact`` restates every operator in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "fp8": 1}
LATENT, ROPE = 512, 64


def listed():
    return [
        # one decode step of the smallest float32 batch: four sequences, interleaved pairs
        dict(name="rope_write_step_f32", op="rope_write", tokens=4, hq=4, hkv=2, dim=64, block=4,
             dtype="f32", rot=64, layout="interleaved", scaling="none", far=64),
        # the new tokens of a prefill batch (16 x 512), split halves over the whole head
        dict(name="rope_write_prefill", op="rope_write", tokens=8192, hq=32, hkv=8, dim=128, block=16,
             dtype="bf16", rot=128, layout="half", scaling="none", far=2560),
        # a ragged chunk into FP8 pages: half of each head rotated, frequencies scaled by parts for
        # a long context
        dict(name="rope_write_fp8_long", op="rope_write", tokens=1999, hq=64, hkv=8, dim=128, block=16,
             dtype="fp8", rot=64, layout="half", scaling="by_parts", far=131072),
        # one decode step of 64 sequences: latent rows and the queries' rotary part, 16 heads
        dict(name="latent_write_step", op="latent_write", tokens=64, heads=16, latent=512, block=64,
             layout="interleaved", scaling="by_parts", far=131072),
        # the new tokens of a prefill batch, 32 heads
        dict(name="latent_write_prefill", op="latent_write", tokens=8192, heads=32, latent=512, block=16,
             layout="interleaved", scaling="none", far=2560),
        # copy on write of one forked tail page
        dict(name="latent_copy_one", op="latent_copy", blocks=1, pool=512, latent=512, block=16),
        # a tenth of a pool moved at once
        dict(name="latent_copy_many", op="latent_copy", blocks=1211, pool=12112, latent=512, block=64),
        # one short sequence on 16 heads: latency
        dict(name="latent_decode_one", op="latent_decode", seqs=1, heads=16, latent=512, block=64,
             shortest=700, longest=700),
        # a ragged batch on 128 heads
        dict(name="latent_decode_ragged", op="latent_decode", seqs=64, heads=128, latent=512, block=16,
             shortest=128, longest=4096),
        # a few long contexts on 64 heads
        dict(name="latent_decode_long", op="latent_decode", seqs=8, heads=64, latent=512, block=64,
             shortest=32768, longest=131072),
        # drafted tokens checked against their contexts: one to eight queries a sequence
        dict(name="latent_prefill_drafts", op="latent_prefill", seqs=32, heads=16, latent=512, block=64,
             shortest=128, longest=4096, fewest=1, most=8),
        # chunked prefill: 512 new tokens behind 2048 cached ones
        dict(name="latent_prefill_chunk", op="latent_prefill", seqs=16, heads=32, latent=512, block=16,
             shortest=2048, longest=2048, fewest=512, most=512),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope_write", "latent_write", "latent_copy", "latent_decode", "latent_decode",
                     "latent_prefill"])
    if op == "rope_write":
        dtype = rng.choice(["f32", "bf16", "bf16", "fp8"])
        dim = 128 if dtype == "fp8" else rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 8192), hq=hkv * rng.choice([1, 2, 3, 4, 8]), hkv=hkv,
                    dim=dim, block=rng.choice([4, 16, 64]), dtype=dtype,
                    rot=rng.choice([r for r in (32, 64, 96, 128) if r <= dim]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "by_parts"]),
                    far=_log(rng, 64, 1 << 20))
    if op == "latent_write":
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=rng.choice([1, 8, 12, 16, 32]),
                    latent=rng.choice([256, 512]), block=rng.choice([8, 16, 64]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "by_parts"]), far=_log(rng, 64, 1 << 20))
    if op == "latent_copy":
        n = _log(rng, 1, 1200)
        return dict(op=op, blocks=n, pool=2 * n + rng.randrange(1, 500), latent=rng.choice([256, 512]),
                    block=rng.choice([8, 16, 64]))
    heads = rng.choice([1, 8, 16, 20, 32, 64, 96, 128])
    block = rng.choice([8, 16, 32, 64, 128])
    latent = rng.choice([256, 512, 512])
    if op == "latent_decode":
        longest = _log(rng, 1, 100000)
        seqs = min(_log(rng, 1, 128), max(1, 400000 // longest))
        return dict(op=op, seqs=seqs, heads=heads, latent=latent, block=block,
                    shortest=max(1, longest // rng.randrange(1, 20)), longest=longest)
    longest = _log(rng, 1, 8192)
    most = _log(rng, 1, 300)
    rows = 1 << 27                      # scores of one pass stay well under those of the chunk above
    seqs = max(1, min(_log(rng, 1, 16), rows // ((longest + most) * most * heads)))
    return dict(op=op, seqs=seqs, heads=heads, latent=latent, block=block,
                shortest=longest // rng.randrange(1, 20), longest=longest, fewest=1, most=most)


# ---------------------------------------------------------------- positions
BASE, FACTOR, ORIGINAL = 10000.0, 8.0, 16384


def _frequencies(rot, scaling):
    """Radians a position of each pair, and the factor on the rotated values, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    f = BASE ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / FACTOR, 1.0
    if scaling == "ntk":
        return (BASE * FACTOR ** (rot / (rot - 2))) ** (-2.0 * i / rot), 1.0
    if scaling == "by_parts":
        turns = ORIGINAL * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f * (keep + (1 - keep) / FACTOR), 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _handle(pkv, rot, case):
    scaling = case["scaling"]
    more = {} if scaling == "none" else {"factor": FACTOR}
    if scaling == "by_parts":
        more["original_context"] = ORIGINAL
    return pkv.Rope(rot, base=BASE, layout=case["layout"], scaling=scaling, device=DEV, **more)


def _angles(s):
    """Cosine and sine of every token's pairs, from angles in 64 bits."""
    f, factor = s["turning"]
    a = s["positions"].double()[:, None] * f
    return (a.cos() * factor).float()[:, None], (a.sin() * factor).float()[:, None]


def _rotate(x, c, s, rot, case):
    """x [T][H][D] float32 with the first `rot` of each head rotated."""
    y = x.clone()
    if case["layout"] == "half":
        u, w = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        u, w = slice(0, rot, 2), slice(1, rot, 2)
    y[..., u] = x[..., u] * c - x[..., w] * s
    y[..., w] = x[..., u] * s + x[..., w] * c
    return y


def _rotate64(x, positions, rot, case):
    """The same as products of complex numbers in 64 bits."""
    f, factor = _frequencies(rot, case["scaling"])
    turn = torch.polar(torch.full_like(f, factor).expand(len(positions), -1), torch.outer(positions.double(), f))
    head, tail = x[..., :rot].double(), x[..., rot:].double()
    pairs = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half" else head.unflatten(-1, (rot // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    z = z.transpose(-1, -2) if case["layout"] == "half" else z
    return torch.cat([z.flatten(-2), tail], -1)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _even(n, low, high):
    """n lengths spread evenly from low to high; one alone is high."""
    return [high - (high - low) * i // max(1, n - 1) for i in range(n)]


def _spread(g, n, low, high):
    """The same in an order that the seed gives."""
    return torch.tensor(_even(n, low, high), device=DEV)[torch.randperm(n, generator=g, device=DEV)]


def _inputs(case, seed):
    """What both sides share, made from the case and the seed alone."""
    g, op = _gen(seed), case["op"]
    if op == "rope_write":
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["dim"]
        io = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        qkv = _randn(g, t, (hq + 2 * hkv) * d, dtype=io)        # one projection's output, read in place
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
        blocks = (3 * t) // (2 * case["block"]) + 2
        slots = torch.randperm(blocks * case["block"], generator=g, device=DEV)[:t]
        return dict(q=q, k=k, v=v, blocks=blocks, slots=slots,
                    positions=torch.randint(0, case["far"], (t,), generator=g, device=DEV))
    if op == "latent_write":
        t, h = case["tokens"], case["heads"]
        kv = _randn(g, t, case["latent"] + ROPE)                # latent and rotary key side by side
        heads = _randn(g, t, h, 128 + ROPE)                     # each query head's plain and rotary part
        q = torch.zeros(t, h, case["latent"] + ROPE, dtype=torch.bfloat16, device=DEV)
        q[..., :case["latent"]] = 1                             # the absorbed part, already in place
        blocks = (3 * t) // (2 * case["block"]) + 2
        slots = torch.randperm(blocks * case["block"], generator=g, device=DEV)[:t]
        return dict(latent=kv[:, :case["latent"]], k_rope=kv[:, case["latent"]:], q_rope=heads[..., 128:],
                    q=q, blocks=blocks, slots=slots,
                    positions=torch.randint(0, case["far"], (t,), generator=g, device=DEV))
    if op == "latent_copy":
        order = torch.randperm(case["pool"], generator=g, device=DEV, dtype=torch.int32)
        n = case["blocks"]
        return dict(blocks=case["pool"], src=order[:n].contiguous(), dst=order[n:2 * n].contiguous(),
                    rows=_randn(g, case["pool"] * case["block"], case["latent"] + ROPE))
    n, bp = case["seqs"], case["block"]
    if op == "latent_decode":
        new = torch.ones(n, dtype=torch.int64, device=DEV)
        lens = _spread(g, n, case["shortest"], case["longest"])
    else:
        new = _spread(g, n, case["fewest"], case["most"])
        lens = _spread(g, n, case["shortest"], case["longest"]) + new
    pages = (lens + bp - 1) // bp
    width, total = int(pages.max()), int(pages.sum())
    blocks = total + total // 8 + 1
    order = torch.randperm(blocks, generator=g, device=DEV, dtype=torch.int32)
    held = torch.arange(width, device=DEV)[None] < pages[:, None]
    tables = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    tables[held] = order[:total]
    rows = torch.empty(blocks * bp, case["latent"] + ROPE, dtype=torch.bfloat16, device=DEV)
    rows.normal_(generator=g)
    starts = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    starts[1:] = new.cumsum(0)
    return dict(blocks=blocks, rows=rows, tables=tables, lens=lens.int(), starts=starts,
                q=_randn(g, int(new.sum()), case["heads"], case["latent"] + ROPE),
                longest=int(lens.max()), most=int(new.max()), scale=(128 + ROPE) ** -0.5)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"], op = case, case["op"]
    if "positions" in s:
        s["turning"] = _frequencies(case.get("rot", ROPE), case["scaling"])
    if own:
        import paged_kv_cache_148_gb300 as pkv
        s["pkv"] = pkv
    if op == "rope_write":
        store = torch.uint8 if case["dtype"] == "fp8" else TORCH[case["dtype"]]
        if own:
            s["pool"] = pkv.KVPool(s["blocks"], case["block"], case["hkv"], case["dim"], TORCH[case["dtype"]], DEV)
            s["rope"] = _handle(pkv, case["rot"], case)
            pages, scales = (s["pool"].k, s["pool"].v), (s["pool"].k_scale, s["pool"].v_scale)
        else:
            shape = (s["blocks"], case["hkv"], case["block"], case["dim"])
            pages = tuple(torch.empty(shape, dtype=store, device=DEV) for _ in "kv")
            scales = tuple(torch.empty(shape[:3], device=DEV) for _ in "kv")
        s["pages"], s["scales"] = pages, scales if case["dtype"] == "fp8" else ()
        for x in s["pages"] + s["scales"]:
            x.zero_()
        return s
    shape = (s["blocks"], case["block"], case["latent"] + ROPE)
    if op == "latent_write":
        s["rows"] = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
    s["rows"] = s["rows"].view(shape)
    if own:
        s["pool"] = pkv.LatentPool(s["blocks"], case["block"], case["latent"], ROPE, device=DEV, rows=s["rows"])
        if op == "latent_write":
            s["rope"] = _handle(pkv, ROPE, case)
        if op == "latent_decode":
            s["workspace"] = pkv.decode_latent_workspace(s["pool"], case["seqs"], case["heads"], s["longest"])
        if op == "latent_prefill":
            s["workspace"] = pkv.prefill_latent_workspace(s["pool"], case["seqs"], case["heads"], len(s["q"]),
                                                          s["most"], s["longest"])
    return s


# ---------------------------------------------------------------- one pass
def _pool_answer(s):
    pages = s["pages"]
    if s["scales"]:
        pages = tuple(x.view(torch.float8_e4m3fn) for x in pages)
    return pages + tuple(s["scales"])


def _run_own(s):
    case, pkv = s["case"], s["pkv"]
    op = case["op"]
    if op == "rope_write":
        q = pkv.rope_write_kv(s["pool"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"])
        return (q,) + _pool_answer(s)
    if op == "latent_write":
        pkv.write_latent(s["pool"], s["latent"], s["k_rope"], s["positions"], s["slots"], s["rope"],
                         q_rope=s["q_rope"], q=s["q"])
        return s["q"], s["rows"]
    if op == "latent_copy":
        pkv.copy_latent_blocks(s["pool"], s["src"], s["dst"])
        return s["rows"]
    if op == "latent_decode":
        return pkv.decode_latent(s["pool"], s["q"], s["tables"], s["lens"], s["longest"], s["scale"],
                                 workspace=s["workspace"])
    return pkv.prefill_latent(s["pool"], s["q"], s["starts"], s["lens"], s["tables"], s["most"], s["longest"],
                              s["scale"], causal=True, workspace=s["workspace"])


def _attend(q, rows, tables, seen, scale, latent):
    """q [B][R][W] against each sequence's rows; row r of a sequence sees its first seen[b][r] tokens."""
    b, width = tables.shape
    k = rows[tables.long().clamp(min=0)].flatten(1, 2).float()           # [B][L][W]
    at = torch.arange(k.shape[1], device=k.device)
    k.masked_fill_((at >= seen.amax(1, keepdim=True))[..., None], 0)     # rows nobody has written
    s = torch.matmul(q.float() * scale, k.transpose(1, 2))
    s.masked_fill_(at >= seen[..., None], -math.inf)
    s -= s.amax(-1, keepdim=True)
    p = s.exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, k[..., :latent]) / total


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op == "rope_write":
        cos, sin = _angles(s)
        q = _rotate(s["q"].float(), cos, sin, case["rot"], case)
        k = _rotate(s["k"].float(), cos, sin, case["rot"], case)
        v = s["v"].float()
        blk, off = s["slots"] // case["block"], s["slots"] % case["block"]
        if case["dtype"] != "fp8":
            s["pages"][0][blk, :, off] = k.to(s["pages"][0].dtype)
            s["pages"][1][blk, :, off] = v.to(s["pages"][1].dtype)
        else:
            ka, va = k.abs().amax(-1), v.abs().amax(-1)
            s["scales"][0][blk, :, off] = ka / 448
            s["scales"][1][blk, :, off] = va / 448
            kc = (k * (448 / ka)[..., None]).to(torch.float8_e4m3fn)
            vc = (v * (448 / va)[..., None]).to(torch.float8_e4m3fn)
            s["pages"][0][blk, :, off] = kc.view(torch.uint8)
            s["pages"][1][blk, :, off] = vc.view(torch.uint8)
        return (q.to(s["q"].dtype),) + _pool_answer(s)
    if op == "latent_write":
        cos, sin = _angles(s)
        kr = _rotate(s["k_rope"].float()[:, None], cos, sin, ROPE, case)[:, 0]
        flat = s["rows"].view(-1, s["rows"].shape[-1])
        flat[s["slots"], :case["latent"]] = s["latent"]
        flat[s["slots"], case["latent"]:] = kr.to(torch.bfloat16)
        s["q"][..., case["latent"]:] = _rotate(s["q_rope"].float(), cos, sin, ROPE, case).to(torch.bfloat16)
        return s["q"], s["rows"]
    if op == "latent_copy":
        s["rows"][s["dst"].long()] = s["rows"][s["src"].long()]
        return s["rows"]
    h = case["heads"]
    if op == "latent_decode":
        seen = s["lens"][:, None].expand(-1, h)
        return _attend(s["q"], s["rows"], s["tables"], seen, s["scale"], case["latent"]).to(torch.bfloat16)
    # queries padded to the longest chunk, then the real ones picked again
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(s["most"], device=new.device)
    real = i < new[:, None]
    q = torch.zeros((len(new), s["most"], h, s["q"].shape[-1]), dtype=s["q"].dtype, device=new.device)
    q[real] = s["q"]
    seen = (s["lens"].long() - new)[:, None] + i + 1
    seen = torch.minimum(seen, s["lens"][:, None].long()).repeat_interleave(h, 1)
    o = _attend(q.flatten(1, 2), s["rows"], s["tables"], seen, s["scale"], case["latent"])
    return o.unflatten(1, (s["most"], h))[real].to(torch.bfloat16)


# ---------------------------------------------------------------- floors
def work(case):
    op = case["op"]
    if op == "rope_write":
        t, io = case["tokens"], 4 if case["dtype"] == "f32" else 2
        wide = case["dim"] * BYTES[case["dtype"]] + (4 if case["dtype"] == "fp8" else 0)
        return {"bytes": t * (2 * case["hq"] * case["dim"] * io + 2 * case["hkv"] * (case["dim"] * io + wide) + 16),
                "flops": 3 * t * (case["hq"] + case["hkv"]) * case["rot"]}
    if op == "latent_write":
        t = case["tokens"]
        return {"bytes": t * (4 * (case["latent"] + ROPE) + 4 * case["heads"] * ROPE + 16),
                "flops": 3 * t * (case["heads"] + 1) * ROPE}
    if op == "latent_copy":
        return {"bytes": case["blocks"] * (4 * case["block"] * (case["latent"] + ROPE) + 8), "flops": 0}
    wide, h, n = case["latent"] + ROPE, case["heads"], case["seqs"]
    before = sum(_even(n, case["shortest"], case["longest"]))
    new = _even(n, case["fewest"], case["most"]) if op == "latent_prefill" else [1] * n
    held, pairs = before, before                            # tokens read; tokens seen, over all queries
    if op == "latent_prefill":                              # chunks and contexts are paired by chance
        held, pairs = before + sum(new), sum(new) * before / n + sum(x * (x + 1) / 2 for x in new)
    return {"bytes": 2 * held * wide + 4 * held / case["block"] + 2 * sum(new) * h * (wide + case["latent"]),
            "flops": 2 * pairs * h * (wide + case["latent"])}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op == "rope_write":
        q = _rotate64(s["q"], s["positions"], case["rot"], case)
        both = _rotate64(s["k"], s["positions"], case["rot"], case), s["v"].double()
        shape = (s["blocks"] * case["block"], case["hkv"], case["dim"])
        pages, scales = [], []
        for x in both:
            flat = torch.zeros(shape, dtype=torch.float64, device=DEV)
            if case["dtype"] == "fp8":
                top = x.abs().amax(-1, keepdim=True)
                sc = torch.zeros(shape[:2], dtype=torch.float64, device=DEV)
                sc[s["slots"]] = (top / 448)[..., 0]
                scales.append(sc.unflatten(0, (s["blocks"], -1)).transpose(1, 2).contiguous())
                x = x / top * 448
            flat[s["slots"]] = x
            pages.append(flat.unflatten(0, (s["blocks"], -1)).transpose(1, 2).contiguous())
        return (q, *pages, *scales)
    if op == "latent_write":
        rows = torch.zeros(s["blocks"] * case["block"], case["latent"] + ROPE, dtype=torch.float64, device=DEV)
        kr = _rotate64(s["k_rope"][:, None], s["positions"], ROPE, case)[:, 0]
        rows[s["slots"]] = torch.cat([s["latent"].double(), kr], 1)
        q = torch.cat([s["q"][..., :case["latent"]].double(), _rotate64(s["q_rope"], s["positions"], ROPE, case)], -1)
        return q, rows.unflatten(0, (s["blocks"], -1))
    if op == "latent_copy":
        rows = s["rows"].view(s["blocks"], case["block"], -1).double()
        came = torch.arange(s["blocks"], device=DEV)
        came[s["dst"].long()] = s["src"].long()
        return rows[came]
    out = torch.zeros(len(s["q"]), case["heads"], case["latent"], dtype=torch.float64, device=DEV)
    bp, starts, lens = case["block"], s["starts"].tolist(), s["lens"].tolist()
    for b, n in enumerate(lens):
        at = torch.arange(n, device=DEV)
        k = s["rows"][s["tables"][b].long()[at // bp] * bp + at % bp].double()
        first, new = starts[b], starts[b + 1] - starts[b]
        for i in range(0, new, 64):                     # 64 queries at a time
            j = min(i + 64, new)
            q = s["q"][first + i:first + j].double()
            w = torch.einsum("thw,lw->thl", q, k) * s["scale"]
            hidden = at > torch.arange(n - new + i, n - new + j, device=DEV)[:, None]
            w = torch.softmax(w.masked_fill(hidden[:, None], -math.inf), -1)
            out[first + i:first + j] = torch.einsum("thl,lw->thw", w, k[:, :case["latent"]])
    return out
