"""Plain 64-bit forms of the attention-side operators, on the CPU, for their tests."""
import math

import numpy as np
import torch

MIN_EXP = -100


def e4m3_values(codes):
    """float8_e4m3fn (or uint8) codes -> float64 values."""
    return codes.detach().cpu().view(torch.uint8).view(torch.float8_e4m3fn).double()


def nearest_e4m3(x):
    """float64 -> nearest e4m3 value (3 fraction bits, exponents from -6, ties to even), at most 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def tables(new, ctx, free, table, B):
    """Sequential form: (table, kv, positions, slots, pieces, taken) of a step."""
    table = [list(map(int, row)) for row in table]
    taken, tok = 0, 0
    positions, slots, pieces, kv = [], [], [], []
    for n, (l, c) in enumerate(zip(new, ctx)):
        for j in range(-(-c // B), -(-(c + l) // B)):
            table[n][j] = int(free[taken])
            taken += 1
        for i in range(l):
            p = c + i
            block = table[n][p // B]
            positions.append(p)
            slots.append(block * B + p % B)
            if i == 0 or p % B == 0:
                pieces.append([block, tok, 0, p % B])
            pieces[-1][2] += 1
            tok += 1
        kv.append(c + l)
    return table, kv, positions, slots, pieces, taken


def frequencies(rot, base, scaling="plain", factor=1.0, length=0.0, fast=32.0, slow=1.0):
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "by_parts":
            pair = lambda b: rot * math.log(length / (2 * math.pi * b)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f * (1 - ramp) + f / factor * ramp
        out.append(f)
    return out


def rotate(x, positions, freqs, interleaved, scale=1.0, inverse=False):
    """x [T, H, d] float64, positions (ints), freqs in radians per token."""
    r = 2 * len(freqs)
    y = x.clone()
    pos = torch.tensor([float(p) for p in positions], dtype=torch.float64)[:, None]
    for i, f in enumerate(freqs):
        a = pos * (-f if inverse else f)
        u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        co, si = torch.cos(a), torch.sin(a)
        y[..., u] = (x[..., u] * co - x[..., w] * si) * scale
        y[..., w] = (x[..., u] * si + x[..., w] * co) * scale
    return y


def append(values, raw, pieces, codes, scales, headroom):
    """values, raw [T, Hk, d] float64 into codes [blocks, Hk, B, d] (values) and scales [blocks, Hk]."""
    codes, scales = codes.clone(), scales.clone()
    for block, first, count, off in pieces:
        for h in range(values.shape[1]):
            a = raw[first:first + count, h].abs()
            a = a[torch.isfinite(a)]
            top = float(a.max()) if a.numel() else 0.0
            e = MIN_EXP if top == 0 else max(MIN_EXP, math.ceil(math.log2(top / 448.0)) + headroom)
            s, old = 2.0 ** e, float(scales[block, h])
            if off:
                s = max(s, old)
                if s != old:
                    codes[block, h, :off] = nearest_e4m3(codes[block, h, :off] * (old / s))
            scales[block, h] = s
            codes[block, h, off:off + count] = nearest_e4m3(values[first:first + count, h] / s)
    return codes, scales


def attention(q, k_cache, v_cache, k_scale, v_scale, table, new, kv, softmax_scale):
    """(o, a) float64 [T, Hq, d]: the result and sum_j p_j |v_j| (the scale of its error)."""
    q = q.detach().cpu().double()
    T, Hq, d = q.shape
    Hk, B = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hk
    K = e4m3_values(k_cache) * k_scale.cpu().double()[:, :, None, None]
    V = e4m3_values(v_cache) * v_scale.cpu().double()[:, :, None, None]
    table = table.cpu().long()
    o = torch.zeros((T, Hq, d), dtype=torch.float64)
    a = torch.zeros_like(o)
    t = 0
    for n, (l, c) in enumerate(zip(new, kv)):
        blocks = table[n, :-(-c // B)]
        for h in range(Hk):
            k, v = K[blocks, h].reshape(-1, d)[:c], V[blocks, h].reshape(-1, d)[:c]
            for i in range(l):
                see = max(0, c - l + i + 1)
                if see == 0:
                    continue
                x = q[t + i, h * G:(h + 1) * G] @ k[:see].t() * softmax_scale
                p = torch.softmax(x, -1)
                o[t + i, h * G:(h + 1) * G] = p @ v[:see]
                a[t + i, h * G:(h + 1) * G] = p @ v[:see].abs()
        t += l
    return o, a


def fill_cache(rng, blocks, Hk, B, d, dev, scale_exps=(-8, -5), odd_scales=False):
    """Codes of normal values and scales 2^e (times a factor in [1, 2) with odd_scales)."""
    def codes():
        x = torch.from_numpy(rng.standard_normal((blocks, Hk, B, d)).astype(np.float32) * 96.0)
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).to(dev)

    def scales():
        e = rng.integers(scale_exps[0], scale_exps[1], (blocks, Hk)).astype(np.float64)
        s = 2.0 ** e * (rng.uniform(1.0, 2.0, e.shape) if odd_scales else 1.0)
        return torch.from_numpy(s.astype(np.float32)).to(dev)
    return codes(), codes(), scales(), scales()
