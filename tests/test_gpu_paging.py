"""Block tables, rotary positions and the append to the 8-bit cache against plain 64-bit forms.

Tolerances. Tables: equal. Rotary: angles are exact to 2^-31 turns and the hardware sine and cosine are
within 2^-21, so a result is off by at most 2^-20 of its pair's length before its one rounding to BF16
(2^-9 of its magnitude, with a little room where the two roundings meet): 2^-8 |y| + 2^-19 |pair| * scale.
Append: scales are equal; a code is the nearest one except where the value, off by 2^-20 of its pair's
length, lies that close to the middle of two codes: one step of the grid there, and at most 0.1% of codes.
"""
import math

import numpy as np
import pytest
import torch

import attnref as R

pytestmark = pytest.mark.gpu


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


# ---------------------------------------------------------------------------------------------------
# Tables
# ---------------------------------------------------------------------------------------------------

def call_tables(new, ctx, table, free, B, cap=None, max_status=None):
    from gated_deltanet_linear_build_gb300 import gdn
    N, T = len(new), int(sum(new))
    cap = T // B + 2 * N if cap is None else cap
    out = dict(table=dev(table), kv=dev([-7] * N), pos=dev([-7] * T), slots=dev([-7] * T, torch.int64),
               pieces=dev(np.full((cap, 4), -7)), counts=dev([-7, -7]), status=dev([-7]))
    gdn.build_block_tables(dev(np.concatenate([[0], np.cumsum(new)])), dev(ctx), dev(free), out["table"],
                           out["kv"], out["pos"], out["slots"], out["pieces"], out["counts"],
                           block_tokens=B, device_status=out["status"])
    return {k: v.cpu().tolist() for k, v in out.items()}


@pytest.mark.parametrize("B", [16, 32, 64, 128])
@pytest.mark.parametrize("kind", ["one", "decode", "ragged", "long", "many", "empties"])
def test_tables(B, kind):
    rng = np.random.default_rng(B)
    new, ctx = {
        "one": ([1], [0]),
        "decode": ([1] * 32, rng.integers(0, 300, 32)),
        "ragged": (rng.integers(0, 200, 40), rng.integers(0, 300, 40)),
        "long": ([30000, 1, 20011], [B - 1, 5 * B, 77]),
        "many": (rng.integers(0, 4, 3001), rng.integers(0, 3 * B, 3001)),
        "empties": ([0] * 1500 + [5, 0, 0, 2 * B] + [0] * 700, [3] * 2204),
    }[kind]
    new, ctx = [int(x) for x in new], [int(x) for x in ctx]
    width = max(-(-(c + l) // B) for l, c in zip(new, ctx)) + 1
    taken = sum(-(-(c + l) // B) - -(-c // B) for l, c in zip(new, ctx))
    table = rng.integers(0, 10000, (len(new), width))
    free = rng.permutation(50000)[:taken + 3]
    ref = R.tables(new, ctx, free, table, B)
    got = call_tables(new, ctx, table, free, B)
    assert got["status"] == [0]
    assert got["table"] == ref[0]
    assert got["kv"] == ref[1]
    assert got["pos"] == ref[2]
    assert got["slots"] == ref[3]
    assert got["counts"] == [len(ref[4]), ref[5]]
    assert got["pieces"][:len(ref[4])] == ref[4]
    assert all(p == [-7] * 4 for p in got["pieces"][len(ref[4]):])


def test_tables_report_what_does_not_fit():
    from gated_deltanet_linear_build_gb300 import gdn
    table = [[9, 9, 9], [8, 8, 8]]

    def untouched(got):
        assert got["counts"] == [0, 0] and got["table"] == table
        assert set(got["slots"]) == {-1} and set(got["pos"]) == {-7} and set(got["kv"]) == {-7}

    got = call_tables([20, 20], [0, 0], table, [1, 2, 3], 16)           # 4 blocks wanted
    assert got["status"] == [gdn.GDN_ERR_WORKSPACE]
    untouched(got)
    got = call_tables([20, 20], [0, 30], table, [1, 2, 3, 4], 16)        # 4 blocks in a row of 3
    assert got["status"] == [gdn.GDN_ERR_WORKSPACE]
    untouched(got)
    got = call_tables([20, 20], [0, 0], table, [1, 2, 3, 4], 16, cap=3)  # 4 pieces
    assert got["status"] == [gdn.GDN_ERR_WORKSPACE]
    untouched(got)
    got = call_tables([20, 20], [0, -1], table, [1, 2, 3, 4], 16)
    assert got["status"] == [gdn.GDN_ERR_INVALID_ARG]
    untouched(got)


@pytest.mark.parametrize("cu", [[0, 30, 20], [0, 5, 39], [1, 5, 40], [0, 50, 40], [0, -3, 40]])
def test_tables_refuse_malformed_offsets(cu):
    from gated_deltanet_linear_build_gb300 import gdn
    o = dict(table=dev([[1] * 9] * 2), kv=dev([-7] * 2), pos=dev([-7] * 40), slots=dev([-7] * 40, torch.int64),
             pieces=dev(np.full((9, 4), -7)), counts=dev([-7, -7]), status=dev([-7]))
    gdn.build_block_tables(dev(cu), dev([0, 0]), dev(range(9)), o["table"], o["kv"], o["pos"], o["slots"],
                           o["pieces"], o["counts"], block_tokens=16, device_status=o["status"])
    assert o["status"].tolist() == [gdn.GDN_ERR_INVALID_ARG] and o["counts"].tolist() == [0, 0]
    assert set(o["slots"].tolist()) == {-1} and set(o["pos"].tolist()) == {-7}


def test_tables_without_tokens():
    got = call_tables([0, 0], [5, 0], [[1], [2]], [3], 16, cap=4)
    assert got["kv"] == [5, 0] and got["counts"] == [0, 0] and got["status"] == [0]


# ---------------------------------------------------------------------------------------------------
# Rotary
# ---------------------------------------------------------------------------------------------------

def make_qkv(rng, T, Hq, Hk, d, pad=8):
    """q, k, v as strided views of one projection output."""
    x = torch.from_numpy(rng.standard_normal((T, (Hq + 2 * Hk) * d + pad)).astype(np.float32))
    x = x.bfloat16().cuda()
    return (x[:, :Hq * d].view(T, Hq, d), x[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d),
            x[:, (Hq + Hk) * d:(Hq + 2 * Hk) * d].view(T, Hk, d))


def assert_rotated(y, x, positions, freqs, interleaved, scale, inverse):
    x = x.cpu().double()
    ref = R.rotate(x, positions, freqs, interleaved, scale, inverse)
    r = 2 * len(freqs)
    lim = 2.0 ** -8 * ref.abs()
    u, w = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    pair = torch.sqrt(u * u + w * w) * scale
    both = torch.stack([pair, pair], -1).flatten(-2) if interleaved else torch.cat([pair, pair], -1)
    lim[..., :r] += 2.0 ** -19 * both
    y = y.cpu().double()
    assert torch.equal(y[..., r:], x[..., r:])
    assert ((y - ref).abs() <= lim).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hk,d,rot", [(16, 2, 256, 64), (32, 8, 128, 128), (5, 3, 64, 32), (1, 1, 16, 16),
                                         (7, 0, 32, 16), (2, 1, 256, 256), (9, 4, 128, 112)])
@pytest.mark.parametrize("T", [1, 33])
def test_rotary(interleaved, Hq, Hk, d, rot, T):
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(T + d)
    q, k, _ = make_qkv(rng, T, Hq, max(Hk, 1), d)
    positions = rng.integers(0, 1 << 20, T)
    positions[0] = (1 << 31) - 1
    ph = gdn.rotary_phases(rot, 10000.0)
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    for inverse in (False, True):
        gdn.rotary(q, k if Hk else None, dev(positions), ph, qo, ko if Hk else None, interleaved=interleaved,
                   inverse=inverse, scale=1.25)
        f = R.frequencies(rot, 10000.0)
        # At 2^31 positions the float64 product pos * f itself is good to 2^-22 turns.
        assert_rotated(qo, q, positions, f, interleaved, 1.25, inverse)
        if Hk:
            assert_rotated(ko, k, positions, f, interleaved, 1.25, inverse)


@pytest.mark.parametrize("scaling", ["plain", "linear", "by_parts"])
@pytest.mark.parametrize("rot,base", [(64, 1e6), (128, 500000.0), (16, 100.0)])
def test_scaled_frequencies(scaling, rot, base):
    from gated_deltanet_linear_build_gb300 import gdn
    kw = dict(scaling=scaling, factor=8.0, original_length=4096.0)
    ph = gdn.rotary_phases(rot, base, device="cpu", **kw).numpy().view(np.uint64).astype(np.float64)
    f = np.array(R.frequencies(rot, base, scaling, 8.0, 4096.0)) / (2 * math.pi)
    assert np.abs(ph / 2.0 ** 64 - f).max() <= 2.0 ** -50


def test_rotary_in_place_and_back():
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(3)
    q, k, _ = make_qkv(rng, 50, 4, 2, 128)
    x, y = q.clone(), k.clone()
    ph = gdn.rotary_phases(64, 10000.0)
    pos = dev(rng.integers(0, 5000, 50))
    qo, ko = torch.empty_like(x), torch.empty_like(y)
    gdn.rotary(q, k, pos, ph, qo, ko)
    gdn.rotary(q, k, pos, ph, q, k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    gdn.rotary(q, k, pos, ph, q, k, inverse=True)
    assert (q.float() - x.float()).abs().max() <= 2.0 ** -6 * x.abs().max()


def test_rotary_gradient_against_differences():
    # loss = sum(w * y); dloss/dx by the inverse rotation of w against central differences of the 64-bit form.
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(4)
    T, H, d, rot = 3, 2, 32, 32
    x, w = (torch.from_numpy(rng.standard_normal((T, H, d)).astype(np.float32)).bfloat16().cuda() for _ in range(2))
    pos, f = [3, 1000, 65535], R.frequencies(rot, 10000.0)
    g = torch.empty_like(w)
    gdn.rotary(w, None, dev(pos), gdn.rotary_phases(rot, 10000.0), g, None, interleaved=True, inverse=True,
               scale=1.5)
    xd, wd = x.cpu().double(), w.cpu().double()
    h = 2.0 ** -10
    for t in range(T):
        for i in range(d):
            up, dn = xd.clone(), xd.clone()
            up[t, 1, i] += h
            dn[t, 1, i] -= h
            num = float((wd * (R.rotate(up, pos, f, True, 1.5) - R.rotate(dn, pos, f, True, 1.5))).sum() / (2 * h))
            pair = float(wd[t, 1, i - i % 2:i - i % 2 + 2].norm()) * 1.5
            assert abs(float(g[t, 1, i]) - num) <= 2.0 ** -8 * abs(num) + 2.0 ** -19 * pair + 1e-9


# ---------------------------------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------------------------------

def make_step(rng, new, ctx, B, spare=2):
    want = [-(-(c + l) // B) for l, c in zip(new, ctx)]
    blocks = sum(want) + spare
    ids = list(rng.permutation(blocks))
    table = [[0] * max(want) for _ in new]
    free = []
    for n, (l, c) in enumerate(zip(new, ctx)):
        for j in range(want[n]):
            b = int(ids.pop())
            if j < -(-c // B):
                table[n][j] = b
            else:
                free.append(b)
    table, kv, pos, slots, pieces, _ = R.tables(new, ctx, free, table, B)
    return blocks, pos, pieces


def assert_codes(got, ref, scale, values, pieces, rot_len):
    """Codes equal, or neighbours where the value lies within its error of the middle of two."""
    g, r = R.e4m3_values(got), ref
    same = (g == r) | (torch.isnan(g) & torch.isnan(r))
    off = torch.nonzero(~same)
    assert len(off) <= 1e-3 * g.numel()
    at = {}
    for block, first, count, offset in pieces:
        for i in range(count):
            at[block, offset + i] = first + i
    for block, h, o, i in off.tolist():
        x = float(values[at[block, o], h, i]) / float(scale[block, h])
        err = 2.0 ** -19 * float(rot_len[at[block, o], h, i]) / float(scale[block, h])
        mid = (float(g[block, h, o, i]) + float(r[block, h, o, i])) / 2
        assert abs(x - mid) <= err, (block, h, o, i, x, mid, err)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hk,d,rot", [(16, 2, 256, 64), (32, 8, 128, 128), (3, 1, 64, 32), (4, 4, 64, 64), (2, 1, 256, 256)])
@pytest.mark.parametrize("B", [16, 32, 64, 128])
def test_append(interleaved, Hq, Hk, d, rot, B):
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(d + B)
    new, ctx = [1, 3, B, 2 * B + 5, 1, 0, 17], [0, B - 1, 5, 7, 2 * B, 9, B - 17 if B > 16 else 3]
    blocks, pos, pieces = make_step(rng, new, ctx, B)
    T = sum(new)
    q, k, v = make_qkv(rng, T, Hq, Hk, d)
    # Magnitudes that grow and shrink from token to token, so that scales of old blocks grow or stay.
    f = torch.from_numpy(2.0 ** rng.integers(-6, 7, (T, 1, 1))).bfloat16().cuda()
    k *= f
    v *= f
    kc, vc, ks, vs = R.fill_cache(rng, blocks, Hk, B, d, "cuda")
    ref_k0, ref_v0, ks0, vs0 = R.e4m3_values(kc), R.e4m3_values(vc), ks.cpu().double(), vs.cpu().double()
    qo = torch.empty((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    cap = dev(pieces + [[blocks + 5, 0, 1, 0]] * 3)              # entries past the count are not read
    freqs = R.frequencies(rot, 10000.0)
    gdn.rotary_kv_append(q, k, v, dev(pos), gdn.rotary_phases(rot, 10000.0), cap, dev([len(pieces), 0]), qo,
                         kc, vc, ks, vs, interleaved=interleaved, scale=1.1)
    assert_rotated(qo, q, pos, freqs, interleaved, float(np.float32(1.1)), False)
    kd, vd = k.cpu().double(), v.cpu().double()
    kr = R.rotate(kd, pos, freqs, interleaved, float(np.float32(1.1)))
    rk, rks = R.append(kr, kd, pieces, ref_k0, ks0, 2)          # 1 + ceil(log2 1.1)
    rv, rvs = R.append(vd, vd, pieces, ref_v0, vs0, 0)
    assert torch.equal(ks.cpu().double(), rks) and torch.equal(vs.cpu().double(), rvs)
    u, w = (kd[..., 0:rot:2], kd[..., 1:rot:2]) if interleaved else (kd[..., :rot // 2], kd[..., rot // 2:rot])
    pair = torch.sqrt(u * u + w * w) * 1.1
    both = torch.stack([pair, pair], -1).flatten(-2) if interleaved else torch.cat([pair, pair], -1)
    length = torch.zeros_like(kd)
    length[..., :rot] = both
    assert_codes(kc, rk, rks, kr, pieces, length)
    assert torch.equal(R.e4m3_values(vc), rv)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_angles_hold_float32(interleaved):
    # Codes differ from those of the 64-bit values only where a value lies on the middle of two but for
    # float32's rounding: the sine and cosine (2 * 2^-24), their products with scale and value and the sum
    # (1 + 2 * 1 of 2^-24 of the pair's length, at most sqrt 2 times in one component): below 2^-21.
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(21)
    B, Hk, d = 64, 2, 64
    T = 1500
    blocks, pos, pieces = make_step(rng, [T], [100000 // B * B], B)
    _, k, v = make_qkv(rng, T, 1, Hk, d)
    kc, vc, ks, vs = R.fill_cache(rng, blocks, Hk, B, d, "cuda")
    old, ks0 = R.e4m3_values(kc), ks.cpu().double()
    ph = gdn.rotary_phases(d, 10000.0)
    qo = torch.empty((T, 1, d), dtype=torch.bfloat16, device="cuda")
    gdn.rotary_kv_append(k[:, :1], k, v, dev(pos), ph, dev(pieces), dev([len(pieces)]), qo, kc, vc, ks, vs,
                         interleaved=interleaved)
    kd = k.cpu().double()
    turns = ph.cpu().numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    kr = R.rotate(kd, pos, list(turns * 2 * math.pi), interleaved, 1.0)
    ref, scales = R.append(kr, kd, pieces, old, ks0, 1)
    assert torch.equal(ks.cpu().double(), scales)
    u, w = (kd[..., 0::2], kd[..., 1::2]) if interleaved else (kd[..., :d // 2], kd[..., d // 2:])
    pair = torch.sqrt(u * u + w * w)
    length = torch.stack([pair, pair], -1).flatten(-2) if interleaved else torch.cat([pair, pair], -1)
    got = R.e4m3_values(kc)
    for block, first, count, off in pieces:
        for h in range(Hk):
            g, r = got[block, h, off:off + count], ref[block, h, off:off + count]
            x = kr[first:first + count, h] / scales[block, h]
            err = 2.0 ** -21 * length[first:first + count, h] / scales[block, h]
            assert (((x - (g + r) / 2).abs() <= err) | (g == r)).all()


def test_append_without_rotation_and_special_values():
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(8)
    B, Hk, d = 16, 2, 64
    blocks, pos, pieces = make_step(rng, [5, 3, 2], [0, 20, 31], B)
    T = 10
    _, k, v = make_qkv(rng, T, 1, Hk, d)
    k[0, 0, 0], k[1, 0, 1], k[2, 0, 2] = float("inf"), float("-inf"), float("nan")
    v[:5, 1] = 0.0                                               # a block of zeros
    v[9, 0, 0] = 3.0e38
    kc, vc, ks, vs = R.fill_cache(rng, blocks, Hk, B, d, "cuda")
    rk, rks = R.append(k.cpu().double(), k.cpu().double(), pieces, R.e4m3_values(kc), ks.cpu().double(), 0)
    rv, rvs = R.append(v.cpu().double(), v.cpu().double(), pieces, R.e4m3_values(vc), vs.cpu().double(), 0)
    gdn.rotary_kv_append(None, k, v, None, None, dev(pieces), dev([len(pieces)]), None, kc, vc, ks, vs)
    assert torch.equal(ks.cpu().double(), rks) and torch.equal(vs.cpu().double(), rvs)
    g = R.e4m3_values(kc)
    assert torch.equal(torch.isnan(g), torch.isnan(rk)) and torch.equal(torch.nan_to_num(g), torch.nan_to_num(rk))
    assert torch.equal(R.e4m3_values(vc), rv)


def test_append_skips_pieces_outside_the_cache_or_the_step():
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(9)
    _, k, v = make_qkv(rng, 4, 1, 1, 64)
    kc, vc, ks, vs = R.fill_cache(rng, 3, 1, 16, 64, "cuda")
    before = [x.clone() for x in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
    bad = [[3, 0, 1, 0], [-1, 0, 1, 0], [0, 3, 2, 0], [0, -1, 2, 0], [0, 0, 4, 13], [0, 0, 1, -1], [0, 0, 0, 0]]
    gdn.rotary_kv_append(None, k, v, None, None, dev(bad), dev([len(bad)]), None, kc, vc, ks, vs)
    for x, y in zip(before, (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)):
        assert torch.equal(x, y)


def test_whole_step_through_the_calls():
    """Tables -> append -> attention of a prefill and two decode steps equals attention on the values."""
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(10)
    N, Hq, Hk, d, B, rot = 3, 8, 2, 128, 16, 64
    pool, width = 40, 12
    kc = torch.full((pool, Hk, B, d), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vc = kc.clone()
    ks, vs = torch.zeros((pool, Hk), device="cuda"), torch.zeros((pool, Hk), device="cuda")
    table = torch.full((N, width), -1, dtype=torch.int32, device="cuda")
    free = list(rng.permutation(pool))
    ph = gdn.rotary_phases(rot, 10000.0)
    ctx = [0, 0, 0]
    for new in ([40, 1, 23], [1, 1, 1], [1, 0, 9]):
        T = sum(new)
        q, k, v = make_qkv(rng, T, Hq, Hk, d)
        cu = dev(np.concatenate([[0], np.cumsum(new)]))
        kv, pos = dev([0] * N), dev([0] * T)
        slots, pieces, counts = dev([0] * T, torch.int64), dev(np.zeros((T // B + 2 * N, 4))), dev([0, 0])
        gdn.build_block_tables(cu, dev(ctx), dev(free), table, kv, pos, slots, pieces, counts, block_tokens=B)
        qo = torch.empty((T, Hq, d), dtype=torch.bfloat16, device="cuda")
        gdn.rotary_kv_append(q, k, v, pos, ph, pieces, counts, qo, kc, vc, ks, vs)
        ws = torch.empty(gdn.paged_attention_workspace_size(T, N, Hq, Hk, d), dtype=torch.uint8, device="cuda")
        o = torch.empty_like(qo)
        gdn.paged_attention(qo, kc, vc, ks, vs, table, cu, kv, o, ws, softmax_scale=d ** -0.5,
                            max_new_tokens=max(new))
        free = free[int(counts[1]):]
        ctx = kv.tolist()
        ref, a = R.attention(qo, kc, vc, ks, vs, table, new, ctx, d ** -0.5)
        assert ((o.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -8 * a + 1e-6 * a.max()).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 16), (128, 64), (256, 64), (256, 48), (64, 64), (128, 128)])
@pytest.mark.parametrize("scale", [0.5, 0.25, 0.1, 2.0 ** -10])
def test_append_with_a_small_scale_saturates_nothing(interleaved, d, rot, scale):
    # Against the values, not the codes of another form: a code of 3 fraction bits is within 2^-4 of its
    # value, or within 2^-10 of the block's scale where it is subnormal; the rotation adds 2^-21 of the
    # pair's length (see the test of the angles). Values from rot on are not scaled and must not be clamped.
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(d + rot)
    B, Hk = 32, 3
    new, ctx = [1, 40, 64, 5], [0, 7, 64, 31]
    blocks, pos, pieces = make_step(rng, new, ctx, B)
    T = sum(new)
    _, k, v = make_qkv(rng, T, 1, Hk, d)
    kc, vc, ks, vs = R.fill_cache(rng, blocks, Hk, B, d, "cuda", scale_exps=(-60, -50))
    qo = torch.empty((T, 1, d), dtype=torch.bfloat16, device="cuda")
    gdn.rotary_kv_append(k[:, :1], k, v, dev(pos), gdn.rotary_phases(rot, 10000.0), dev(pieces),
                         dev([len(pieces)]), qo, kc, vc, ks, vs, interleaved=interleaved, scale=scale)
    kd, f = k.cpu().double(), float(np.float32(scale))
    kr = R.rotate(kd, pos, R.frequencies(rot, 10000.0), interleaved, f)
    u, w = (kd[..., 0:rot:2], kd[..., 1:rot:2]) if interleaved else (kd[..., :rot // 2], kd[..., rot // 2:rot])
    pair = torch.sqrt(u * u + w * w) * f
    length = torch.zeros_like(kd)
    length[..., :rot] = torch.stack([pair, pair], -1).flatten(-2) if interleaved else torch.cat([pair, pair], -1)
    for values, got, s, room in ((kr, kc, ks, length), (v.cpu().double(), vc, vs, torch.zeros_like(kd))):
        got, s = R.e4m3_values(got), s.cpu().double()
        for block, first, count, off in pieces:
            x = values[first:first + count].transpose(0, 1)
            sc = s[block][:, None, None]
            err = (got[block, :, off:off + count] * sc - x).abs()
            lim = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * sc) + \
                2.0 ** -20 * room[first:first + count].transpose(0, 1)
            assert (err <= lim).all()
    # And no coarser than the rule: the largest magnitude times what may multiply it.
    grow = 1 + math.ceil(math.log2(f))
    grow = max(grow, 0) if rot < d else grow
    ref = R.append(kr, kd, pieces, R.e4m3_values(kc), torch.full_like(ks.cpu().double(), 2.0 ** -60), grow)[1]
    for block, first, count, off in pieces:
        if off == 0:
            assert torch.equal(ks.cpu().double()[block], ref[block])


def test_append_skips_pieces_whose_sums_pass_32_bits():
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(11)
    _, k, v = make_qkv(rng, 4, 1, 1, 64)
    kc, vc, ks, vs = R.fill_cache(rng, 3, 1, 16, 64, "cuda")
    before = [x.clone() for x in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
    top = 2 ** 31 - 1
    bad = [[0, top, 1, 0], [0, top - 15, 16, 0], [0, 5, top, 1], [0, 1, top, 15], [0, 0, 1, top], [1, 0, 4, top - 1],
           [top, 0, 1, 0], [-top - 1, 0, 1, 0], [0, -top - 1, 4, 0], [0, 0, -top - 1, 0], [0, 0, 4, -top - 1]]
    gdn.rotary_kv_append(None, k, v, None, None, dev(bad), dev([len(bad)]), None, kc, vc, ks, vs)
    for x, y in zip(before, (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)):
        assert torch.equal(x, y)


def test_options_without_a_truth_value_raise_their_own_error():
    from gated_deltanet_linear_build_gb300 import gdn
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    pos, ph, neither = dev([0, 1]), gdn.rotary_phases(16, 10000.0), np.array([True, False])
    for kw in (dict(interleaved=neither), dict(inverse=neither)):
        with pytest.raises(ValueError, match="truth value"):
            gdn.rotary(x, None, pos, ph, x, None, **kw)
    kc, vc, ks, vs = R.fill_cache(np.random.default_rng(1), 3, 1, 16, 64, "cuda")
    with pytest.raises(ValueError, match="truth value"):
        gdn.rotary_kv_append(x, x, x, pos, ph, dev([[0, 0, 2, 0]]), dev([1]), x, kc, vc, ks, vs, interleaved=neither)
    with pytest.raises(ValueError, match="truth value"):
        gdn.paged_attention(x, kc, vc, ks, vs, dev([[0]]), dev([0, 2]), dev([2]), x, x, softmax_scale=1.0,
                            max_new_tokens=2, planned=neither)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="one device")
def test_tensors_of_another_device_are_refused():
    from gated_deltanet_linear_build_gb300 import gdn
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda:0")
    pos, ph = dev([0, 1]), gdn.rotary_phases(16, 10000.0)
    for bad in ((x.to("cuda:1"), pos, ph, x), (x, pos.to("cuda:1"), ph, x), (x, pos, ph.to("cuda:1"), x),
                (x, pos, ph, x.to("cuda:1"))):
        with pytest.raises(ValueError):
            gdn.rotary(bad[0], None, bad[1], bad[2], bad[3], None)
    with torch.cuda.device(1), pytest.raises(ValueError):
        gdn.rotary(x, None, pos, ph, x, None)
