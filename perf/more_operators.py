"""The answer side of a serving step, as cases to measure: an output head (or any projection) whose weights
are held in 4 bits, and what a request wants to know about the logits that it gives.

Three operators, in the order a program uses them:

* ``pack``      weights [N, K] to 4-bit codes (1 sign, 2 exponent, 1 fraction bit), one 8-bit scale (4 exponent and
                3 fraction bits) for every 16 values of a row and one power of two for each row; and read back;
* ``linear``    y = x W^T over such weights, from one token (a matrix-vector product) to the prompts of a step;
* ``logprobs``  from logits, for each row: the log probability and the rank of a given token, the entropy, and the
                best tokens with theirs.

A case is a dict of plain values; tensors are made from ``prepare``'s seed.
"""
import math

import torch

own = False

GROUP = 16              # values that share a scale
CODE_MAX = 6.0          # the codes' magnitudes: 0, 0.5, 1, 1.5, 2, 3, 4, 6
SCALE_MAX = 448.0
SCALE_MIN = 2.0 ** -9   # of a group that is not all zeros
MIN_EXP, MAX_EXP = -100, 110   # of a row's power of two


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # A small projection, odd in both sizes (the last group of a row is not full).
        dict(name="pack 1001 x 1111", op="pack", n=1001, k=1111, pad=1),
        # The serving stack's output head.
        dict(name="pack 4096 x 8192", op="pack", n=4096, k=8192, pad=0),
        # One request's token through the head: latency.
        dict(name="linear 1, 4096 x 8192", op="linear", t=1, n=4096, k=8192, out="float32", pad=0),
        # The decode step of the serving mix: 32 requests.
        dict(name="linear 32, 4096 x 8192", op="linear", t=32, n=4096, k=8192, out="float32", pad=0),
        # A few drafted tokens, odd sizes, rows of x inside wider ones.
        dict(name="linear 7, 5003 x 1111", op="linear", t=7, n=5003, k=1111, out="bfloat16", pad=3),
        # The same decode step with a vocabulary of 128k.
        dict(name="linear 32, 131072 x 4096", op="linear", t=32, n=131072, k=4096, out="float32", pad=0),
        # A layer's input projection (q | k | v) in a decode step of 48 requests.
        dict(name="linear 48, 12288 x 4096", op="linear", t=48, n=12288, k=4096, out="bfloat16", pad=0),
        # Every position of a 2,048-token prefill step: prompt scoring.
        dict(name="linear 2048, 4096 x 8192", op="linear", t=2048, n=4096, k=8192, out="float32", pad=0),
        # One request, a large odd vocabulary, the twenty best.
        dict(name="logprobs 1 of 200003", op="logprobs", t=1, v=200003, dtype="bfloat16", top=20, mask=0.0,
             temperature=1.0, pad=0),
        # The decode step of the serving mix.
        dict(name="logprobs 32 of 4096", op="logprobs", t=32, v=4096, dtype="float32", top=5, mask=0.0,
             temperature=1.0, pad=0),
        # Sampling under a grammar: most tokens are masked, some rows wholly.
        dict(name="logprobs 333 of 50001, masked", op="logprobs", t=333, v=50001, dtype="bfloat16", top=0,
             mask=0.95, temperature=0.7, pad=5),
        # Prompt scoring over a vocabulary of 128k.
        dict(name="logprobs 2048 of 131072", op="logprobs", t=2048, v=131072, dtype="float32", top=8, mask=0.0,
             temperature=1.0, pad=0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _maybe_round(rng, size):
    """Half of the sizes as models have them, half as they fall."""
    if rng.random() < 0.5:
        return size
    step = 256 if size >= 1024 else 16
    return max(step, size // step * step)


def draw(rng):
    op = rng.choice(["pack", "linear", "linear", "linear", "logprobs", "logprobs"])
    if op == "pack":
        k = _maybe_round(rng, _spread(rng, 1, 16384))
        n = _maybe_round(rng, _spread(rng, 1, min(131072, 2 ** 26 // k)))
        return dict(op=op, n=n, k=k, pad=rng.choice([0, 0, 1, 4]))
    if op == "linear":
        kind = rng.choice(["decode", "decode", "prompt"])
        t = _spread(rng, 1, 96) if kind == "decode" else _spread(rng, 65, 2048)
        k = _maybe_round(rng, _spread(rng, 48, 16384))
        n = _maybe_round(rng, _spread(rng, 16, max(17, min(131072, 2 ** 28 // k, 2 ** 36 // (t * k)))))
        return dict(op=op, t=t, n=n, k=k, out=rng.choice(["float32", "bfloat16"]), pad=rng.choice([0, 0, 1, 7]))
    v = _maybe_round(rng, _spread(rng, 33, 262144))
    t = _spread(rng, 1, max(2, min(4096, 2 ** 27 // v)))
    return dict(op=op, t=t, v=v, dtype=rng.choice(["float32", "bfloat16"]), top=rng.choice([0, 1, 5, 20, 32]),
                mask=rng.choice([0.0, 0.0, 0.5, 0.99]), temperature=rng.choice([1.0, 1.0, 0.6, 1.7]),
                pad=rng.choice([0, 0, 3]))


def _held_bytes(n, k):
    """4-bit codes, a scale for every group and one for every row."""
    return n * (k * 0.5 + -(-k // GROUP)) + 4 * n


def work(case):
    if case["op"] == "pack":
        n, k = case["n"], case["k"]
        return {"bytes": int(4 * n * k + 2 * _held_bytes(n, k)), "flops": 0}
    if case["op"] == "linear":
        t, n, k = case["t"], case["n"], case["k"]
        size = 4 if case["out"] == "float32" else 2
        return {"bytes": int(_held_bytes(n, k) + 2 * t * k + size * t * n), "flops": 2 * t * n * k}
    t, v = case["t"], case["v"]
    size = 4 if case["dtype"] == "float32" else 2
    return {"bytes": t * v * size + t * (16 + 8 * case["top"]), "flops": 4 * t * v}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _weights(case, gen, dev):
    """Rows of unlike size, with some columns that stick out, as trained projections have."""
    n, k = case["n"], case["k"]
    w = torch.randn((n, k), generator=gen, device=dev)
    w *= torch.exp2(torch.randn((n, 1), generator=gen, device=dev)) / math.sqrt(k)
    w *= torch.where(torch.rand((1, k), generator=gen, device=dev) < 0.01, 8.0, 1.0)
    return w.bfloat16()


def _in_wider_rows(x, pad):
    """x as a view of rows that are 8 * pad elements wider (a multiple of 8 in any case)."""
    t, k = x.shape
    wide = torch.zeros((t, -(-k // 8) * 8 + 8 * pad), dtype=x.dtype, device=x.device)
    wide[:, :k] = x
    return wide[:, :k]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case=case, dev=dev)
    if case["op"] == "pack":
        s["w"] = _in_wider_rows(_weights(case, gen, dev), case["pad"])
        s["packed"] = None
        s["back"] = _in_wider_rows(torch.empty_like(s["w"]), 0)
    elif case["op"] == "linear":
        t, n, k = case["t"], case["n"], case["k"]
        # Normalised activations, a few channels of them large.
        x = torch.randn((t, k), generator=gen, device=dev)
        x *= torch.where(torch.rand((1, k), generator=gen, device=dev) < 0.005, 20.0, 1.0)
        s["x"] = _in_wider_rows(x.bfloat16(), case["pad"])
        s["y"] = torch.empty((t, n), dtype=getattr(torch, case["out"]), device=dev)
        w = _weights(case, gen, dev)
        s["workspace"] = s["packed"] = s["held"] = None
        if own:                         # the weights are laid out once, when a model is loaded
            _own_weights(s, w)
        else:
            s["held"] = _quantise(w)
    else:
        t, v = case["t"], case["v"]
        x = torch.randn((t, v), generator=gen, device=dev)
        x *= 1.0 + 2.0 * torch.rand((t, 1), generator=gen, device=dev)
        # A row has a favourite, from hardly noticed to next to certain, and so has the given token.
        best = torch.randint(0, v, (t, 1), generator=gen, device=dev)
        x.scatter_add_(1, best, 25.0 * torch.rand((t, 1), generator=gen, device=dev))
        given = torch.randint(0, v, (t, 1), generator=gen, device=dev)
        s["tokens"] = torch.where(torch.rand((t, 1), generator=gen, device=dev) < 0.6, best, given)[:, 0].int()
        if case["mask"] > 0:
            x.masked_fill_(torch.rand((t, v), generator=gen, device=dev) < case["mask"], float("-inf"))
            x[1::7] = float("-inf")
        s["logits"] = _in_wider_rows(x.to(getattr(torch, case["dtype"])), case["pad"]) if case["pad"] else \
            x.to(getattr(torch, case["dtype"]))
        f = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)  # noqa: E731
        i = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)  # noqa: E731
        s.update(logprobs=f(t), entropy=f(t), ranks=i(t), top_ids=i(t, case["top"]), top_logprobs=f(t, case["top"]))
        s["workspace"] = None
    return s


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------

def _power_of_two(e):
    """2^e in 32 bits, from its bits (exponentials need not be exact), e from -126 to 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(w):
    """Signed values of the codes (int8, in halves), scales [N, groups] and powers of two [N]."""
    n, k = w.shape
    groups = -(-k // GROUP)
    x = torch.zeros((n, groups * GROUP), device=w.device)
    x[:, :k] = w.float()
    x = x.view(n, groups, GROUP)
    top = x.abs().amax(-1)
    row = top.amax(-1)
    # Smallest power of two under which the row's largest value fits: 6 * 448 = 0.65625 * 2^12.
    mant, ex = torch.frexp(row)
    e = torch.where(row > 0, ex - 12 + (mant > 0.65625).int(), MIN_EXP).clamp(MIN_EXP, MAX_EXP)
    power, down = _power_of_two(e), _power_of_two(-e)
    x = x * down[:, None, None]
    top = top * down[:, None]
    # (Tensor by tensor: a division by a number may become a product with its reciprocal.)
    scale = (top / torch.full_like(top, CODE_MAX)).clamp(max=SCALE_MAX).to(torch.float8_e4m3fn).float()
    scale = torch.where(top > 0, scale.clamp(min=SCALE_MIN), 0.0)
    # To the nearest code, ties to the even one. (A border times a scale is exact in 32 bits.)
    a, s = x.abs(), scale[..., None]
    halves = torch.zeros(x.shape, dtype=torch.int8, device=w.device)
    for border, up, step in ((0.25, False, 1), (0.75, True, 1), (1.25, False, 1), (1.75, True, 1),
                             (2.5, False, 2), (3.5, True, 2), (5.0, False, 4)):
        halves += ((a >= border * s) if up else (a > border * s)).to(torch.int8) * step
    halves = torch.where(s > 0, torch.where(x < 0, -halves, halves), 0)
    return halves, scale, power, k


def _values(held):
    halves, scale, power, k = held
    v = halves.float() * 0.5 * scale[..., None] * power[:, None, None]
    return v.flatten(1)[:, :k]


def _plain_pack(s):
    return _values(_quantise(s["w"])).bfloat16()


def _plain_linear(s):
    return (s["x"].float() @ _values(s["held"]).t()).to(s["y"].dtype)


def _order(x):
    """Whole numbers in the order of the values: -0 is 0."""
    bits = (x.float() + 0.0).view(torch.int32).long()
    return torch.where(bits >= 0, bits, -2 ** 31 - bits)


def _plain_logprobs(s):
    c, x = s["case"], s["logits"]
    t, v = x.shape
    z = x.float() / c["temperature"]
    top = z.amax(-1, keepdim=True)
    none = top == float("-inf")                         # no token is left
    d = torch.where(none, float("-inf"), z - top)
    e = d.exp()
    total = e.double().sum(-1, keepdim=True)
    lse = total.log()
    p = e.double() / torch.where(none, 1.0, total)
    entropy = (p * torch.where(e > 0, lse - d.double(), 0.0)).sum(-1)
    logprobs = torch.where(none, float("-inf"), d.double() - lse)
    at = s["tokens"].long()[:, None]
    key = (_order(x) << 31) + (2 ** 31 - 1 - torch.arange(v, device=x.device))   # ties: the lowest index first
    ranks = (key > key.gather(1, at)).sum(-1)
    ids = key.topk(c["top"], -1).indices if c["top"] else torch.empty((t, 0), dtype=torch.int64, device=x.device)
    return dict(logprobs=logprobs.gather(1, at)[:, 0].float(), entropy=entropy.float(), ranks=ranks.int(),
                top_ids=ids.int(), top_logprobs=logprobs.gather(1, ids).float())


# ---------------------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------------------

def _own_weights(s, w):
    from gated_deltanet_linear_build_gb300 import gdn
    n, k = w.shape
    s["packed"] = torch.empty(gdn.w4_packed_size(n, k), dtype=torch.uint8, device=s["dev"])
    gdn.w4_pack(w if w.stride(0) % 8 == 0 else _in_wider_rows(w, 0), s["packed"])
    s["workspace"] = torch.empty(gdn.w4_linear_workspace_size(s["case"]["t"], n, k), dtype=torch.uint8,
                                 device=s["dev"])


def _own_pack(s):
    from gated_deltanet_linear_build_gb300 import gdn
    if s["packed"] is None:
        s["packed"] = torch.empty(gdn.w4_packed_size(*s["w"].shape), dtype=torch.uint8, device=s["dev"])
    gdn.w4_pack(s["w"], s["packed"])
    gdn.w4_unpack(s["packed"], s["back"])
    return s["back"]


def _own_linear(s):
    from gated_deltanet_linear_build_gb300 import gdn
    gdn.w4_linear(s["x"], s["packed"], s["y"], s["workspace"])
    return s["y"]


def _own_logprobs(s):
    from gated_deltanet_linear_build_gb300 import gdn
    c = s["case"]
    if s["workspace"] is None:          # kept by a serving program for its whole life
        size = gdn.token_logprobs_workspace_size(c["t"], c["v"], c["top"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["dev"])
    gdn.token_logprobs(s["logits"], s["tokens"], s["logprobs"], s["entropy"], s["ranks"], s["top_ids"],
                       s["top_logprobs"], s["workspace"], temperature=c["temperature"])
    return {name: s[name] for name in ("logprobs", "entropy", "ranks", "top_ids", "top_logprobs")}


_PLAIN = dict(pack=_plain_pack, linear=_plain_linear, logprobs=_plain_logprobs)
_OWN = dict(pack=_own_pack, linear=_own_linear, logprobs=_own_logprobs)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# 64-bit definitions
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    def nearest(x, step):
        """x to the nearest multiple of `step` (elementwise), ties to the even multiple."""
        return torch.round(x / step) * step

    def power_of_two(e):
        return ((e.long() + 1023) << 52).view(torch.float64)

    def held_values(w):
        """What the 4-bit form of w [N, K] stands for, some rows at a time."""
        out = torch.empty(w.shape, dtype=torch.float64, device=w.device)
        for r in range(0, w.shape[0], 8192):
            x = w[r:r + 8192].double()
            n, k = x.shape
            row = x.abs().amax(1)
            # Smallest e with row / 2^e <= 6 * 448, found by trying.
            e = torch.full_like(row, -100.0)
            for bit in (128, 64, 32, 16, 8, 4, 2, 1):
                e = torch.where(row > 6.0 * 448.0 * power_of_two(e + bit - 1), e + bit, e)
            power = power_of_two(e.clamp(max=110))[:, None]
            for g in range(0, k, 16):
                v = x[:, g:g + 16] / power
                q = v.abs().amax(1, keepdim=True)
                q = q / torch.full_like(q, 6.0)
                # 8-bit scale: four significant bits, no step below 2^-9, at most 448.
                step = power_of_two(torch.frexp(q).exponent - 4).clamp(min=2.0 ** -9)
                sc = nearest(q, step).clamp(max=448.0)
                sc = torch.where((q > 0) & (sc < 2.0 ** -9), 2.0 ** -9, sc)
                u = torch.where(sc > 0, v / torch.where(sc > 0, sc, 1.0), 0.0)
                a = u.abs().clamp(max=6.0)
                # 4-bit code: two significant bits, no step below 0.5, at most 6.
                st = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
                out[r:r + 8192, g:g + 16] = torch.copysign(nearest(a, st), u) * sc * power
        return out

    gen_state = prepare(dict(case), seed)
    if case["op"] == "pack":
        if case["n"] * case["k"] > 2 ** 27:
            return None
        return held_values(gen_state["w"])
    if case["op"] == "linear":
        dev = gen_state["dev"]
        # The weights again, from the seed alone: prepare draws x and its channels before them.
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)
        torch.randn((case["t"], case["k"]), generator=gen, device=dev)
        torch.rand((1, case["k"]), generator=gen, device=dev)
        w = _weights(case, gen, dev)
        x = gen_state["x"].double()
        out = torch.empty((case["t"], case["n"]), dtype=torch.float64, device=dev)
        for r in range(0, case["n"], 16384):
            out[:, r:r + 16384] = x @ held_values(w[r:r + 16384]).t()
        return out
    x, tokens, k = gen_state["logits"], gen_state["tokens"].tolist(), case["top"]
    t, v = x.shape
    res = dict(logprobs=[], entropy=[], ranks=[], top_ids=[], top_logprobs=[])
    index = torch.arange(v, device=x.device)
    for r in range(t):
        raw = x[r].double()
        z = raw / case["temperature"]
        lp = z - torch.logsumexp(z, 0)
        lp = torch.where(torch.isnan(lp), float("-inf"), lp)
        res["logprobs"].append(lp[tokens[r]])
        res["entropy"].append(-torch.special.xlogy(lp.exp(), lp.exp()).sum())
        mine = raw[tokens[r]]
        res["ranks"].append((raw > mine).sum() + ((raw == mine) & (index < tokens[r])).sum())
        left, ids = raw.clone(), []
        if k:
            ids = torch.sort(raw, descending=True, stable=True).indices[:k]
            res["top_ids"].append(ids)
            res["top_logprobs"].append(lp[ids])
    stack = lambda a, shape: torch.stack(a) if a else torch.empty(shape, device=x.device)  # noqa: E731
    return dict(logprobs=stack(res["logprobs"], (t,)), entropy=stack(res["entropy"], (t,)),
                ranks=stack(res["ranks"], (t,)).int(), top_ids=stack(res["top_ids"], (t, 0)).int(),
                top_logprobs=stack(res["top_logprobs"], (t, 0)).double())
