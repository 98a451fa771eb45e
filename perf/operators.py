"""The attention-side operators of a hybrid (GDN + softmax attention) serving step, as cases to measure.

Four operators, in the order an engine step calls them:

* ``tables``     block tables, slot map and page pieces of the step, from the request lengths;
* ``rotary``     rotary positions on q and k (half or interleaved pairs, part of the head, scaled
                 frequencies; ``inverse`` is the gradient's direction);
* ``append``     rotary on q and k, with k and v written to the 8-bit paged cache (one power-of-two
                 scale for each block and head);
* ``attention``  causal attention of the step's tokens over that cache (decode, prefill, mixed).

A case is a dict of plain values. Lengths are drawn from the case's own ``lens_seed``, so that the
work of a case is fixed; tensors are made from ``prepare``'s seed.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -100          # smallest exponent of a block's scale
NO_POSITION = float("-inf")


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # Plan of a decode step: 32 concurrent requests, one token each.
        dict(name="tables decode 32", op="tables", n=32, new_lo=1, new_hi=1, ctx_lo=512, ctx_hi=1143,
             decode=1.0, block=64, lens_seed=1),
        # Plan of a large mixed step: 4,000 requests, one in ten a prompt of up to 600 tokens.
        dict(name="tables mixed 4000", op="tables", n=4000, new_lo=9, new_hi=600, ctx_lo=0, ctx_hi=5000,
             decode=0.9, block=16, lens_seed=2),
        # Rotary of a 2,048-token prefill step: a quarter of 256-wide heads, half layout.
        dict(name="rotary half 64 of 256", op="rotary", n=4, new_lo=512, new_hi=512, ctx_lo=0, ctx_hi=1000,
             decode=0.0, hq=16, hk=2, d=256, rot=64, interleaved=False, scaling="none", inverse=False,
             lens_seed=3),
        # Gradient's direction over a long scaled context: whole heads, interleaved pairs.
        dict(name="rotary interleaved 16k", op="rotary", n=3, new_lo=5001, new_hi=5600, ctx_lo=90000,
             ctx_hi=125000, decode=0.0, hq=32, hk=8, d=128, rot=128, interleaved=True,
             scaling="by_parts", inverse=True, lens_seed=4),
        # Append of a decode step.
        dict(name="append decode 32", op="append", n=32, new_lo=1, new_hi=1, ctx_lo=512, ctx_hi=1143,
             decode=1.0, hq=16, hk=2, d=256, rot=64, interleaved=False, scaling="none", block=64,
             lens_seed=5),
        # Append of a 2,048-token prefill step of four segments that start inside a block.
        dict(name="append prefill 2k", op="append", n=4, new_lo=400, new_hi=620, ctx_lo=0, ctx_hi=700,
             decode=0.0, hq=16, hk=2, d=256, rot=64, interleaved=False, scaling="none", block=64,
             lens_seed=6),
        # Append of long prompts with a scaled rotary.
        dict(name="append prefill 16k", op="append", n=2, new_lo=7800, new_hi=8500, ctx_lo=0,
             ctx_hi=40000, decode=0.0, hq=32, hk=8, d=128, rot=128, interleaved=False,
             scaling="by_parts", block=32, lens_seed=7),
        # One request's token: latency.
        dict(name="attend decode 1", op="attention", n=1, new_lo=1, new_hi=1, ctx_lo=999, ctx_hi=999,
             decode=1.0, hq=16, hk=2, d=256, block=64, lens_seed=8),
        # The decode step of the serving mix: 32 requests of 512 to 1,143 tokens.
        dict(name="attend decode 32", op="attention", n=32, new_lo=1, new_hi=1, ctx_lo=512, ctx_hi=1143,
             decode=1.0, hq=16, hk=2, d=256, block=64, lens_seed=9),
        # Long ragged contexts.
        dict(name="attend decode 48 long", op="attention", n=48, new_lo=1, new_hi=1, ctx_lo=3000,
             ctx_hi=30001, decode=1.0, hq=32, hk=8, d=128, block=32, lens_seed=10),
        # A 2,048-token prefill step of four segments, some of them continuing a prompt.
        dict(name="attend prefill 2k", op="attention", n=4, new_lo=400, new_hi=620, ctx_lo=0, ctx_hi=700,
             decode=0.0, hq=16, hk=2, d=256, block=64, lens_seed=11),
        # The last 4,096-token chunk of a 16,384-token prompt.
        dict(name="attend prefill 4k of 16k", op="attention", n=1, new_lo=4096, new_hi=4096, ctx_lo=12288,
             ctx_hi=12288, decode=0.0, hq=32, hk=8, d=128, block=64, lens_seed=12),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rotary", "append", "append", "attention", "attention", "attention"])
    seed = rng.randrange(1 << 30)
    block = rng.choice([16, 32, 64, 128])
    if op == "tables":
        n = _spread(rng, 1, 4000)
        hi = _spread(rng, 1, 600)
        return dict(op=op, n=n, new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=0,
                    ctx_hi=_spread(rng, 1, 5000), decode=rng.choice([0.0, 0.5, 0.9, 1.0]), block=block,
                    lens_seed=seed)
    hq, hk, d = rng.choice([(16, 2, 256), (32, 8, 128), (32, 4, 128), (16, 16, 64), (8, 1, 128),
                            (12, 4, 64), (24, 2, 128), (6, 2, 256)])
    if op in ("rotary", "append"):
        n = _spread(rng, 1, 64)
        hi = max(1, _spread(rng, 1, 15000) // n)
        rot = rng.choice([d, d // 2, d // 4])
        c = dict(op=op, n=n, new_lo=rng.randint(max(1, hi // 2), hi), new_hi=hi, ctx_lo=0,
                 ctx_hi=_spread(rng, 1, 40000 if op == "rotary" else max(2, 120000 // n)),
                 decode=rng.choice([0.0, 0.5]), hq=hq, hk=hk, d=d, rot=rot,
                 interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "by_parts"]),
                 lens_seed=seed)
        c.update(dict(inverse=rng.random() < 0.5) if op == "rotary" else dict(block=block))
        return c
    kind = rng.choice(["decode", "decode", "prefill", "mixed"])
    if kind == "decode":
        n = _spread(rng, 1, 300)
        room = 1.2e9 / (2 * hk * d) / n                 # tokens of context, by bytes
        hi = _spread(rng, 17, max(18, min(60000, room)))
        # A few tokens for each request where a draft is verified.
        return dict(op=op, n=n, new_lo=1, new_hi=rng.choice([1, 1, 1, 3]), ctx_lo=rng.randint(0, hi // 2), ctx_hi=hi,
                    decode=rng.choice([1.0, 0.5]), hq=hq, hk=hk, d=d, block=block, lens_seed=seed)
    n = rng.randint(1, 6) if kind == "prefill" else rng.randint(4, 24)
    hi = max(2, _spread(rng, 30, 3000) // (n if kind == "prefill" else 4))
    room = max(1.0, 2.0e9 / (n * hq * hi) - hi)         # the score matrix of the plain form
    return dict(op=op, n=n, new_lo=max(1, hi // 2), new_hi=hi, ctx_lo=0,
                ctx_hi=_spread(rng, 1, min(12000.0, room)), decode=0.0 if kind == "prefill" else 0.8,
                hq=hq, hk=hk, d=d, block=block, lens_seed=seed)


def _lengths(case):
    """Cached tokens and new tokens of each request."""
    r = np.random.RandomState(case["lens_seed"])
    n = case["n"]
    ctx = r.randint(case["ctx_lo"], case["ctx_hi"] + 1, n)
    new = r.randint(case["new_lo"], case["new_hi"] + 1, n)
    new = np.where(r.random_sample(n) < case["decode"], 1, new)
    return ctx.astype(np.int64), new.astype(np.int64)


def _pairs(ctx, new):
    """Visible (query, key) pairs of causal attention."""
    return int((new * ctx + new * (new + 1) // 2).sum())


def work(case):
    ctx, new = _lengths(case)
    n, t = len(ctx), int(new.sum())
    if case["op"] == "tables":
        b = case["block"]
        have, want = -(-ctx // b), -(-(ctx + new) // b)
        taken, touched = int((want - have).sum()), int((want - ctx // b).sum())
        part = touched - taken
        return {"bytes": 4 * (2 * n + 1) + 8 * taken + 4 * part + 12 * t + 4 * n + 16 * touched,
                "flops": 0}
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "rotary":
        return {"bytes": 4 * t * (hq + hk) * d + 4 * t, "flops": 3 * t * (hq + hk) * case["rot"]}
    if case["op"] == "append":
        return {"bytes": t * (4 * hq * d + 4 * hk * d + 2 * hk * d + 4),
                "flops": 3 * t * (hq + hk) * case["rot"] + 4 * t * hk * d}
    return {"bytes": int((ctx + new).sum()) * hk * d * 2 + 4 * t * hq * d,
            "flops": 4 * d * hq * _pairs(ctx, new)}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

# Frequencies f_i = base^(-2i/r); "linear" divides them by a factor; "by_parts" divides those whose
# wavelength is long against the original context and keeps the short ones, with a linear ramp
# between, and scales the rotated values by 0.1 ln(factor) + 1.
ROPE_BASE = 1000000.0
ROPE_FACTOR = 4.0
ROPE_LENGTH = 32768
RAMP = (32.0, 1.0)


def _rope_scale(case):
    return 0.1 * math.log(ROPE_FACTOR) + 1.0 if case["scaling"] == "by_parts" else 1.0


def _phases(case):
    """Turns per token of each pair as 64-bit fixed point (int64 bit patterns)."""
    r = case["rot"]
    i = np.arange(r // 2, dtype=np.float64)
    f = ROPE_BASE ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        f = f / ROPE_FACTOR
    if case["scaling"] == "by_parts":
        at = [r * math.log(ROPE_LENGTH / (2 * math.pi * b)) / (2 * math.log(ROPE_BASE)) for b in RAMP]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        keep = 1.0 - np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        f = f * keep + f / ROPE_FACTOR * (1.0 - keep)
    turns = f / (2 * math.pi)
    return (turns * 2.0 ** 64).astype(np.uint64).view(np.int64)


def _step(case, dev, gen):
    """The step's maps, as index arithmetic on the host: what the tables operator computes."""
    ctx, new = _lengths(case)
    n, t, b = len(ctx), int(new.sum()), case.get("block", 64)
    cu = np.concatenate([[0], np.cumsum(new)])
    have, want = -(-ctx // b), -(-(ctx + new) // b)
    width = int(want.max()) + 1
    blocks = int(want.sum()) + 3
    ids = torch.randperm(blocks, generator=gen, device=dev).cpu().numpy()
    r = np.random.RandomState(case["lens_seed"] + 1)
    col = np.arange(width)[None, :]
    first = np.concatenate([[0], np.cumsum(want)])[:-1, None]
    table = np.where(col < want[:, None], ids[np.minimum(first + col, blocks - 1)], 0)
    seq = np.repeat(np.arange(n), new)
    pos = ctx[seq] + np.arange(t) - cu[seq]
    slot = table[seq, pos // b] * b + pos % b
    lead = np.flatnonzero((pos % b == 0) | (np.arange(t) == cu[seq]))
    last = np.append(lead[1:], t)
    pieces = np.stack([slot[lead] // b, lead, last - lead, pos[lead] % b], 1)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(dev)  # noqa: E731
    i64 = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int64)).to(dev)  # noqa: E731
    held = np.where(col < have[:, None], table, r.randint(0, blocks, table.shape))
    fresh = table[(col >= have[:, None]) & (col < want[:, None])]
    return dict(case=case, dev=dev, n=n, t=t, block=b, blocks=blocks, cu=i32(cu), ctx=i32(ctx),
                kv=i32(ctx + new), table=i32(table), held=i32(held),
                free=i32(np.concatenate([fresh, r.randint(0, blocks, 5)])), positions=i32(pos),
                slots=i64(slot), pages=i32(pieces), num_pages=i32([len(pieces)]),
                piece_count=len(pieces), taken=len(fresh), longest=int(new.max()),
                width=width, kv_max=int((ctx + new).max()))


def _cache(s, gen, held):
    """K and V codes and scales; what lies past a request's end is stale bytes, NaN codes among them."""
    c, dev = s["case"], s["dev"]
    shape = (s["blocks"], c["hk"], s["block"], c["d"])
    make = lambda f: (torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16) * f).clamp(  # noqa: E731
        -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    s["k_cache"], s["v_cache"] = make(96.0), make(96.0)
    exps = lambda: torch.randint(-8, -5, (s["blocks"], c["hk"]), generator=gen, device=dev)  # noqa: E731
    s["k_scale"], s["v_scale"] = torch.exp2(exps().float()), torch.exp2(exps().float())
    # Stale tail of each request's last block.
    kv = s["ctx"] if held else s["kv"]
    b = s["block"]
    at = torch.clamp((kv.long() - 1) // b, min=0)
    last = s["table"].long()[torch.arange(s["n"], device=dev), at]
    tail = torch.arange(b, device=dev)[None, :] >= ((kv.long() - 1) % b + 1)[:, None]
    rows, offs = torch.nonzero(tail, as_tuple=True)
    s["k_cache"].view(torch.uint8)[last[rows], :, offs] = 0x7F
    s["v_cache"].view(torch.uint8)[last[rows], :, offs] = 0x7F


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = _step(case, dev, gen)
    t, n = s["t"], s["n"]
    if case["op"] == "tables":
        s.update(kv_out=torch.empty(n, dtype=torch.int32, device=dev),
                 positions_out=torch.empty(t, dtype=torch.int32, device=dev),
                 slots_out=torch.empty(t, dtype=torch.int64, device=dev),
                 # The caller sizes the piece list by its bound; entries past the count stay zero.
                 pages_out=torch.zeros((t // s["block"] + 2 * n, 4), dtype=torch.int32, device=dev),
                 count_out=torch.empty(2, dtype=torch.int32, device=dev))
        return s
    hq, hk, d = case["hq"], case["hk"], case["d"]
    # q | k | v of a step lie in one projection output, read in place.
    qkv = torch.randn((t, (hq + 2 * hk) * d), generator=gen, device=dev, dtype=torch.bfloat16)
    qkv *= torch.exp2(torch.randn((t, 1), generator=gen, device=dev) * 0.5).bfloat16()
    s["q"] = qkv[:, :hq * d].view(t, hq, d)
    s["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
    s["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
    if case["op"] in ("rotary", "append"):
        s["phases"] = torch.from_numpy(_phases(case)).to(dev)
        s["rope_scale"] = _rope_scale(case)
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.empty((t, hk, d), dtype=torch.bfloat16, device=dev)
    if case["op"] == "append":
        _cache(s, gen, held=True)
    if case["op"] == "attention":
        _cache(s, gen, held=False)
        s["softmax_scale"] = 1.0 / math.sqrt(d)
        s["o"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
        s["workspace"] = None
    return s


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------

def _plain_tables(s):
    b, n, t = s["block"], s["n"], s["t"]
    dev = s["dev"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    new = cu[1:] - cu[:-1]
    have, want = (ctx + b - 1) // b, (ctx + new + b - 1) // b
    need = want - have
    end = torch.cumsum(need, 0)
    col = torch.arange(s["width"], device=dev)[None, :]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = ((end - need)[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"].long()[at], s["held"].long())
    tok = torch.arange(t, device=dev)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    pos = ctx[seq] + tok - cu[seq]
    slot = table[seq, pos // b] * b + pos % b
    lead = (pos % b == 0) | (tok == cu[seq])
    piece = torch.cumsum(lead, 0) - 1
    cap = s["pages_out"].shape[0]
    size = torch.zeros(cap, dtype=torch.int64, device=dev).scatter_add_(0, piece, torch.ones_like(piece))
    start = torch.cumsum(size, 0) - size
    real = size > 0
    start = torch.where(real, start, 0)
    pages = torch.stack([slot[start] // b, start, size, pos[start] % b], 1) * real[:, None]
    count = torch.stack([lead.sum(), end[-1]])
    return dict(table=table.int(), kv=(ctx + new).int(), positions=pos.int(), slots=slot,
                pages=pages.int(), count=count.int())


def _angles(s):
    """cos and sin [T, 1, r/2]: the 64-bit product wraps, which is the reduction to one turn."""
    turn = (s["positions"].long()[:, None] * s["phases"][None, :]) >> 32
    a = turn.float() * (2.0 * math.pi / 2.0 ** 32)
    if s["case"].get("inverse"):
        a = -a
    return torch.cos(a)[:, None, :], torch.sin(a)[:, None, :]


def _rotate(x, cos, sin, case, scale):
    r = case["rot"]
    x = x.float()
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
    u, w = (a * cos - b * sin) * scale, (a * sin + b * cos) * scale
    y = torch.stack([u, w], -1).flatten(-2) if case["interleaved"] else torch.cat([u, w], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_rotary(s):
    cos, sin = _angles(s)
    rot = lambda x: _rotate(x, cos, sin, s["case"], s["rope_scale"]).bfloat16()  # noqa: E731
    return dict(q=rot(s["q"]), k=rot(s["k"]))


def _headroom(case):
    """Powers of two by which a rotation may grow the largest magnitude."""
    return 1 + math.ceil(math.log2(_rope_scale(case)))


def _plain_write(s, x, raw, grow, cache, scale):
    """x [T, Hk, d] into the cache: scales from the largest magnitude of `raw` for each block and head."""
    b = s["block"]
    pages = s["pages"].long()
    block, first, off = pages[:, 0], pages[:, 1], pages[:, 3]
    piece = torch.searchsorted(first, torch.arange(s["t"], device=s["dev"]), right=True) - 1
    at = s["slots"] % b
    big = torch.where(torch.isfinite(raw), raw, 0.0).abs().float().amax(-1)            # [T, Hk]
    top = torch.zeros((len(pages), big.shape[1]), device=s["dev"]).scatter_reduce_(
        0, piece[:, None].expand_as(big), big, "amax")
    mant, ex = torch.frexp(top)
    e = torch.where(top > 0, ex - 9 + (mant > 0.875).int() + grow, MIN_EXP).clamp(min=MIN_EXP)
    old = scale[block]
    new = torch.exp2(e.float())
    new = torch.where((off == 0)[:, None], new, torch.maximum(new, old))
    # Tokens that the block held before the call keep their values under a grown scale.
    codes = cache.view(torch.uint8)[block].view(cache.dtype).float()
    held = torch.arange(b, device=s["dev"])[None, :] < off[:, None]
    kept = held[:, None, :] & (new != old)[:, :, None]
    codes = torch.where(kept[..., None], codes * (old / new)[:, :, None, None], codes)
    codes[piece, :, at] = (x / new[piece][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    cache.view(torch.uint8)[block] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    scale[block] = new


def _plain_append(s):
    cos, sin = _angles(s)
    case, f = s["case"], s["rope_scale"]
    _plain_write(s, _rotate(s["k"], cos, sin, case, f), s["k"], _headroom(case), s["k_cache"], s["k_scale"])
    _plain_write(s, s["v"].float(), s["v"], 0, s["v_cache"], s["v_scale"])
    return dict(q=_rotate(s["q"], cos, sin, case, f).bfloat16(), k_codes=s["k_cache"], v_codes=s["v_cache"],
                k_scale=s["k_scale"], v_scale=s["v_scale"])


def _plain_attention(s):
    c, dev = s["case"], s["dev"]
    n, hk, d, b = s["n"], c["hk"], c["d"], s["block"]
    g = c["hq"] // hk
    span = -(-s["kv_max"] // b) * b
    table = s["table"].long()[:, :span // b]

    def values(codes, scale):
        rows = codes.view(torch.uint8)[table].view(codes.dtype).float() * scale[table][..., None, None]
        return rows.transpose(1, 2).reshape(n, hk, span, d)

    cu, kv = s["cu"].long(), s["kv"].long()
    new = cu[1:] - cu[:-1]
    i, j = torch.arange(s["longest"], device=dev), torch.arange(span, device=dev)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=s["t"] - 1)
    q = s["q"].float()[rows].view(n, -1, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    x = (q @ values(s["k_cache"], s["k_scale"]).transpose(2, 3)).mul_(s["softmax_scale"])
    seen = j[None, None, :] <= (kv - new)[:, None, None] + i[None, :, None]
    seen &= j[None, None, :] < kv[:, None, None]
    x = x.view(n, hk, g, -1, span).masked_fill_(~seen[:, None, None], NO_POSITION)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top == NO_POSITION, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = values(s["v_cache"], s["v_scale"])
    v = torch.where((j[None, :] < kv[:, None])[:, None, :, None], v, 0.0)
    o = (p.view(n, hk, -1, span) @ v).view(n, hk, g, -1, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, -1, c["hq"], d)
    return o[i[None, :] < new[:, None]].bfloat16()


# ---------------------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------------------

def _own_tables(s):
    from gated_deltanet_linear_build_gb300 import gdn
    gdn.build_block_tables(s["cu"], s["ctx"], s["free"], s["held"], s["kv_out"], s["positions_out"],
                           s["slots_out"], s["pages_out"], s["count_out"], block_tokens=s["block"])
    return dict(table=s["held"], kv=s["kv_out"], positions=s["positions_out"], slots=s["slots_out"],
                pages=s["pages_out"], count=s["count_out"])


def _own_rotary(s):
    from gated_deltanet_linear_build_gb300 import gdn
    c = s["case"]
    gdn.rotary(s["q"], s["k"], s["positions"], s["phases"], s["q_out"], s["k_out"],
               interleaved=c["interleaved"], scale=s["rope_scale"], inverse=c["inverse"])
    return dict(q=s["q_out"], k=s["k_out"])


def _own_append(s):
    from gated_deltanet_linear_build_gb300 import gdn
    gdn.rotary_kv_append(s["q"], s["k"], s["v"], s["positions"], s["phases"], s["pages"], s["num_pages"],
                         s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                         interleaved=s["case"]["interleaved"], scale=s["rope_scale"])
    return dict(q=s["q_out"], k_codes=s["k_cache"], v_codes=s["v_cache"], k_scale=s["k_scale"],
                v_scale=s["v_scale"])


def _own_attention(s):
    from gated_deltanet_linear_build_gb300 import gdn
    c = s["case"]
    if s["workspace"] is None:      # kept by a serving program for its whole life
        size = gdn.paged_attention_workspace_size(s["t"], s["n"], c["hq"], c["hk"], c["d"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["dev"])
    gdn.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["cu"],
                        s["kv"], s["o"], s["workspace"], softmax_scale=s["softmax_scale"],
                        max_new_tokens=s["longest"])
    return s["o"]


_PLAIN = dict(tables=_plain_tables, rotary=_plain_rotary, append=_plain_append, attention=_plain_attention)
_OWN = dict(tables=_own_tables, rotary=_own_rotary, append=_own_append, attention=_own_attention)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# 64-bit definitions
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    def exact_rotation(s, x):
        """Each pair turned by position x frequency, in float64, frequency by frequency."""
        c = s["case"]
        r = c["rot"]
        y = x.double().clone()
        pos = s["positions"].double()
        at = [r * math.log(ROPE_LENGTH / (b * 2 * math.pi)) / (2 * math.log(ROPE_BASE)) for b in RAMP]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        for i in range(r // 2):
            f = math.exp(-2.0 * i / r * math.log(ROPE_BASE))
            if c["scaling"] == "linear":
                f /= ROPE_FACTOR
            elif c["scaling"] == "by_parts":
                ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
                f = f * (1.0 - ramp) + f * ramp / ROPE_FACTOR
            a = pos * (-f if c.get("inverse") else f)
            u, w = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
            co, si = torch.cos(a)[:, None], torch.sin(a)[:, None]
            xu, xw = x[..., u].double(), x[..., w].double()
            y[..., u] = (xu * co - xw * si) * _rope_scale(c)
            y[..., w] = (xu * si + xw * co) * _rope_scale(c)
        return y

    def nearest_code(x):
        """x (float64) to the nearest value of 4 exponent and 3 fraction bits, ties to even, at most 448."""
        _, e = torch.frexp(x)
        step = torch.exp2((e - 4).clamp(min=-9).double())
        return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)

    def exact_write(s, x, raw, grow, cache, scale):
        codes, scales = cache.double().cpu(), scale.double().cpu()
        x, raw = x.cpu(), raw.double().abs().cpu()
        for block, first, count, off in s["pages"].cpu().tolist():
            top = raw[first:first + count].amax((0, 2))
            for h in range(top.numel()):
                v, e = float(top[h]), MIN_EXP
                if v > 0:
                    e = max(MIN_EXP, math.ceil(math.log2(v / E4M3_MAX)) + grow)
                new, old = 2.0 ** e, float(scales[block, h])
                if off:
                    new = max(new, old)
                    if new != old:
                        codes[block, h, :off] = nearest_code(codes[block, h, :off] * (old / new))
                scales[block, h] = new
                codes[block, h, off:off + count] = nearest_code(x[first:first + count, h] / new)
        return codes, scales

    def exact_attention(s):
        c = s["case"]
        hk, b = c["hk"], s["block"]
        g = c["hq"] // hk
        cu, kv, table = s["cu"].tolist(), s["kv"].tolist(), s["table"].long()
        out = torch.zeros((s["t"], c["hq"], c["d"]), dtype=torch.float64, device=s["dev"])
        for n in range(s["n"]):
            blocks = table[n, :-(-kv[n] // b)]
            for h in range(hk):
                k, v = ((s[x + "_cache"].view(torch.uint8)[blocks, h].view(torch.float8_e4m3fn).double()
                         * s[x + "_scale"][blocks, h].double()[:, None, None]).flatten(0, 1)[:kv[n]] for x in "kv")
                last = torch.arange(kv[n] - (cu[n + 1] - cu[n]), kv[n], device=s["dev"])
                hide = torch.arange(kv[n], device=s["dev"])[None, :] > last[:, None]
                for m in range(h * g, (h + 1) * g):
                    x = s["q"][cu[n]:cu[n + 1], m].double() @ k.t() * s["softmax_scale"]
                    out[cu[n]:cu[n + 1], m] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ v
        return out

    s = prepare(case, seed)
    if case["op"] == "tables":
        return None                     # whole numbers: the two sides are equal or one is wrong
    if case["op"] == "attention":
        return exact_attention(s)
    q = exact_rotation(s, s["q"])
    if case["op"] == "rotary":
        return dict(q=q, k=exact_rotation(s, s["k"]))
    if s["piece_count"] * case["hk"] > 12000:
        return dict(q=q, k_codes=None, v_codes=None, k_scale=None, v_scale=None)
    k, ks = exact_write(s, exact_rotation(s, s["k"]), s["k"], _headroom(case), s["k_cache"], s["k_scale"])
    v, vs = exact_write(s, s["v"].double(), s["v"], 0, s["v_cache"], s["v_scale"])
    return dict(q=q, k_codes=k, v_codes=v, k_scale=ks, v_scale=vs)
