"""Causal attention over the paged 8-bit cache against a 64-bit form.

Tolerance. The output is rounded to BF16 once: 2^-9 of its magnitude. The weights carry a relative
error: their rounding to 16-bit floats for the tensor cores (2^-11 with BF16-free f16 operands) and
the error of the scores (q is represented to 2^-17 of its row's largest magnitude, products are exact,
float32 accumulation of scores of at most about 16: together below 2^-10). A weight's error e moves the
output by at most e * sum_j p_j |v_j| =: e * a twice over (numerator and normalisation). So
    |o - ref| <= 2^-8 |ref| + 2^-8 a + 1e-6 max(a).
"""
import numpy as np
import pytest
import torch

import attnref as R

pytestmark = pytest.mark.gpu


def make(seed, new, kv, Hq, Hk, d, B, *, stale=True, spare=3, extra_cols=2, **cache):
    """Tensors of a step: sequence n has kv[n] keys in the cache, its last new[n] tokens are queries."""
    rng = np.random.default_rng(seed)
    dev = "cuda"
    N, T = len(new), sum(new)
    want = [-(-c // B) for c in kv]
    blocks = sum(want) + spare
    ids = rng.permutation(blocks)
    width = max(want + [1]) + extra_cols
    table = np.full((N, width), blocks - 1, np.int32)
    at = 0
    for n, m in enumerate(want):
        table[n, :m] = ids[at:at + m]
        at += m
    kc, vc, ks, vs = R.fill_cache(rng, blocks, Hk, B, d, dev, **cache)
    if stale:
        for n, c in enumerate(kv):
            if c % B:
                kc.view(torch.uint8)[int(table[n, c // B]), :, c % B:] = 0x7F
                vc.view(torch.uint8)[int(table[n, c // B]), :, c % B:] = 0xFF
    qkv = torch.from_numpy(rng.standard_normal((max(T, 1), (Hq + 2 * Hk) * d)).astype(np.float32)).bfloat16().to(dev)
    q = qkv[:T, Hk * d:(Hk + Hq) * d].view(T, Hq, d)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev)
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=torch.from_numpy(table).to(dev), cu=cu,
                kv=torch.tensor(kv, dtype=torch.int32, device=dev), new=new, kvl=kv, scale=d ** -0.5)


def run(s, planned=False, workspace=None, **kw):
    from gated_deltanet_linear_build_gb300 import gdn
    T, Hq, d = s["q"].shape
    N, Hk = len(s["new"]), s["kc"].shape[1]
    o = torch.full((T, Hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    if workspace is None:
        workspace = torch.empty(gdn.paged_attention_workspace_size(T, N, Hq, Hk, d), dtype=torch.uint8,
                                device="cuda")
        workspace.fill_(0xA5)
    gdn.paged_attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["kv"], o,
                        workspace, softmax_scale=s["scale"], max_new_tokens=max(s["new"] + [0]),
                        planned=planned, **kw)
    return o


def check(s, o):
    ref, a = R.attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["new"], s["kvl"], s["scale"])
    o = o.cpu().double()
    assert torch.isfinite(o).all()
    bad = (o - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -8 * a + 1e-6 * a.max())
    assert bad.max() <= 0, (float(bad.max()), np.unravel_index(int(bad.argmax()), bad.shape))


HEADS = [(16, 2, 256), (32, 8, 128), (8, 8, 64), (12, 1, 128), (16, 1, 256), (6, 2, 64), (3, 1, 256), (32, 2, 64)]


@pytest.mark.parametrize("Hq,Hk,d", HEADS)
@pytest.mark.parametrize("B", [16, 64])
def test_decode_lengths(Hq, Hk, d, B):
    kv = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 256, 257, 700]
    s = make(1, [1] * len(kv), kv, Hq, Hk, d, B)
    check(s, run(s))


@pytest.mark.parametrize("B", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hk,d", [(16, 2, 256), (32, 8, 128), (10, 2, 64)])
def test_long_contexts_split_over_ctas(Hq, Hk, d, B):
    s = make(2, [1, 1, 1], [9001, 5, 4096], Hq, Hk, d, B)
    check(s, run(s))


@pytest.mark.parametrize("Hq,Hk,d", HEADS)
def test_several_tokens_per_sequence(Hq, Hk, d):
    new = [1, 2, 3, 4, 5, 7, 1, 20]
    kv = [40, 2, 300, 4, 77, 500, 1, 90]
    s = make(3, new, kv, Hq, Hk, d, 32)
    check(s, run(s))


@pytest.mark.parametrize("Hq,Hk,d", [(16, 2, 256), (32, 8, 128), (4, 4, 64), (24, 2, 128)])
@pytest.mark.parametrize("B", [16, 128])
def test_prefill_and_mixed(Hq, Hk, d, B):
    new = [129, 1, 64, 1, 200, 33]
    kv = [129, 300, 500, 1, 201, 33 + 256]
    s = make(4, new, kv, Hq, Hk, d, B)
    check(s, run(s))


@pytest.mark.parametrize("Hq,Hk,d", [(16, 2, 256), (32, 8, 128), (4, 4, 64), (24, 2, 128), (3, 1, 256)])
@pytest.mark.parametrize("new,kv", [([127], [127]), ([300], [5000]), ([65, 700, 90], [65, 1400, 4000])])
def test_chunks_of_prompts(Hq, Hk, d, new, kv):
    s = make(17, new, kv, Hq, Hk, d, 64)
    check(s, run(s))


def test_rows_that_see_no_key_are_zero():
    # More new tokens than keys: the first ones see nothing; and sequences without tokens or keys.
    new, kv = [4, 0, 3, 2, 0], [2, 7, 0, 50, 0]
    s = make(5, new, kv, 8, 2, 128, 16)
    o = run(s)
    check(s, o)
    assert (o[:2] == 0).all() and (o[4:7] == 0).all()


@pytest.mark.parametrize("new,kv", [([1, 1], [777, 60]), ([150], [400])])
def test_scales_of_any_size(new, kv):
    # Blocks whose scales differ by 2^30, and scales that are no powers of two.
    s = make(6, new, kv, 8, 2, 128, 16, scale_exps=(-40, -10))
    s["ks"].copy_(torch.full_like(s["ks"], 2.0 ** -7))
    check(s, run(s))
    s = make(7, new, kv, 8, 2, 64, 32, odd_scales=True)
    check(s, run(s))


def test_a_flat_tail_behind_a_peak_keeps_its_weight():
    # One key takes almost all of the softmax; thousands of others share 2^-14 each.
    s = make(8, [1], [6000], 4, 1, 128, 64)
    s["kc"].view(torch.uint8)[:] = 0
    s["q"].fill_(0.0)
    s["q"][..., 0] = 8.0
    first = int(s["table"][0, 0])
    s["ks"].fill_(2.0 ** -6)
    s["kc"][first, 0, 0, 0] = torch.tensor(448.0, device="cuda").to(torch.float8_e4m3fn)
    s["scale"] = 14.0 / (8.0 * 448.0 / 64.0) * 0.6931471805599453
    check(s, run(s))


def test_planned_calls_and_reuse_of_a_workspace_give_the_same_bits():
    from gated_deltanet_linear_build_gb300 import gdn
    s = make(9, [1] * 9 + [70], [3000, 64, 1, 500, 501, 1000, 31, 9000, 2, 800], 16, 2, 256, 64)
    T, N = sum(s["new"]), len(s["new"])
    ws = torch.empty(gdn.paged_attention_workspace_size(T, N, 16, 2, 256), dtype=torch.uint8, device="cuda")
    a = run(s, workspace=ws)
    gdn.paged_attention_plan(s["cu"], s["kv"], ws, T=T, Hq=16, Hk=2, d=256, block_tokens=64,
                             max_blocks=s["table"].shape[1], max_new_tokens=70)
    for _ in range(5):
        b = run(s, workspace=ws, planned=True)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_an_unplanned_call_leaves_a_plan_in_the_workspace_alone():
    from gated_deltanet_linear_build_gb300 import gdn
    s = make(18, [1] * 5, [3000, 64, 1, 500, 31], 16, 2, 256, 64)
    ws = torch.empty(gdn.paged_attention_workspace_size(5, 5, 16, 2, 256), dtype=torch.uint8, device="cuda")
    gdn.paged_attention_plan(s["cu"], s["kv"], ws, T=5, Hq=16, Hk=2, d=256, block_tokens=64,
                             max_blocks=s["table"].shape[1], max_new_tokens=1)
    a = run(s, workspace=ws, planned=True)
    other = make(19, [1] * 3, [700, 2, 90], 16, 2, 256, 64)
    check(other, run(other, workspace=ws))
    assert torch.equal(a, run(s, workspace=ws, planned=True))
    check(s, a)


def test_on_another_stream():
    s = make(10, [1] * 4, [1000, 70, 3, 400], 8, 2, 128, 32)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        o = run(s)
    st.synchronize()
    check(s, o)
    o2 = run(s, stream=st)
    st.synchronize()
    check(s, o2)


@pytest.mark.parametrize("new,kv", [([1, 1], [90, 200]), ([40], [90])])
def test_non_finite_values_stay_where_they_belong(new, kv):
    # A NaN query row gives NaN rows of its own head and token, nothing else.
    s = make(11, new, kv, 8, 2, 128, 16)
    clean = run(s)
    s["q"][0, 1, 5] = float("inf")
    s["q"][sum(new) - 1, 6, 0] = float("nan")
    o = run(s)
    assert torch.isnan(o[0, 1]).all() and torch.isnan(o[sum(new) - 1, 6]).all()
    keep = torch.ones(o.shape[:2], dtype=torch.bool, device="cuda")
    keep[0, 1] = keep[sum(new) - 1, 6] = False
    assert torch.equal(o[keep], clean[keep])


@pytest.mark.parametrize("Hq,Hk,d", [(4, 2, 64), (4, 2, 128), (8, 1, 256), (12, 1, 64)])
@pytest.mark.parametrize("new,kv", [([3], [100]), ([140], [300]), ([1, 40, 1], [64, 64, 3])])
def test_non_finite_keys_and_values_reach_only_rows_that_see_them(Hq, Hk, d, new, kv):
    s = make(12, new, kv, Hq, Hk, d, 16)
    n = int(np.argmax(new))
    clean = run(s)
    first = sum(new[:n])
    for which, cache in (("k", "kc"), ("v", "vc")):
        for pos in (kv[n] - 1, kv[n] - new[n] // 2):
            block, off = int(s["table"][n, pos // 16]), pos % 16
            saved = s[cache].view(torch.uint8)[block, :, off].clone()
            s[cache].view(torch.uint8)[block, 0, off, 3] = 0x7F
            o = run(s)
            s[cache].view(torch.uint8)[block, :, off] = saved
            seen = first + pos - (kv[n] - new[n])     # the first token that sees the key
            keep = torch.ones(sum(new), dtype=torch.bool, device="cuda")
            keep[seen:first + new[n]] = False
            assert torch.equal(o[keep], clean[keep]), (which, pos)
            G = Hq // Hk
            hit = o[seen:first + new[n], :G]
            assert torch.isnan(hit).all() if which == "k" else torch.isnan(hit[..., 3]).all(), (which, pos)
            if which == "v":                          # other values of the head are not touched
                other = [i for i in range(d) if i != 3]
                assert torch.equal(hit[..., other], clean[seen:first + new[n], :G][..., other])
            assert torch.equal(o[:, G:], clean[:, G:])


def test_a_block_outside_the_cache_is_reported_and_reads_as_zeros():
    from gated_deltanet_linear_build_gb300 import gdn
    st = torch.empty(1, dtype=torch.int32, device="cuda")
    gdn.device_status(st, clear=True)
    s = make(13, [1, 1], [40, 40], 4, 1, 64, 16)
    run(s)
    gdn.device_status(st)
    assert int(st) == gdn.GDN_OK
    s["table"][1, 1] = s["kc"].shape[0]
    s["table"][0, 0] = -1
    o = run(s)
    gdn.device_status(st, clear=True)
    assert int(st) == gdn.GDN_ERR_INVALID_ARG
    assert torch.isfinite(o).all()
    gdn.device_status(st)
    assert int(st) == gdn.GDN_OK


def test_lengths_beyond_the_table_are_cut_off():
    s = make(14, [1], [64], 4, 1, 64, 16, extra_cols=0)
    a = run(s)
    s["kv"].fill_(1 << 30)
    assert torch.equal(a, run(s))


def test_offsets_past_32_bits():
    # Blocks whose bytes lie beyond 2^32 in the pool.
    Hk, B, d = 8, 128, 256
    blocks = (1 << 32) // (Hk * B * d) + 4
    dev = "cuda"
    kc = torch.zeros((blocks, Hk, B, d), dtype=torch.uint8, device=dev)
    vc = torch.zeros_like(kc)
    s = make(15, [1, 1], [130, 5], 8, Hk, d, B, spare=0, extra_cols=0)
    small = s["kc"].shape[0]
    o = run(s)
    kc[blocks - small:] = s["kc"].view(torch.uint8)
    vc[blocks - small:] = s["vc"].view(torch.uint8)
    ks = torch.ones((blocks, Hk), device=dev)
    vs = torch.ones((blocks, Hk), device=dev)
    ks[blocks - small:], vs[blocks - small:] = s["ks"], s["vs"]
    s.update(kc=kc, vc=vc, ks=ks, vs=vs, table=s["table"] + (blocks - small))
    assert torch.equal(o, run(s))


def test_refusals():
    from gated_deltanet_linear_build_gb300 import gdn
    s = make(16, [1, 1], [20, 30], 4, 2, 64, 16)
    with pytest.raises(gdn.GdnError) as e:
        run(s, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == gdn.GDN_ERR_WORKSPACE
    for key, bad in (("q", s["q"].float()), ("kc", s["kc"][:, :, ::2]), ("ks", s["ks"].double()),
                     ("table", s["table"].long()), ("kv", s["kv"].long()), ("cu", s["cu"].long())):
        with pytest.raises(ValueError):
            run(dict(s, **{key: bad}))


@pytest.mark.parametrize("planned", [False, True])
def test_mixed_steps_back_to_back_see_their_own_inputs(planned):
    # Both kernels of a mixed step, without a wait between calls whose q, scales and outputs change in place.
    from gated_deltanet_linear_build_gb300 import gdn
    new, kv = [1] * 20 + [130, 90, 300], list(range(50, 2050, 100)) + [700, 1200, 300]
    s = make(31, new, kv, 32, 8, 128, 64)
    T, N = sum(new), len(new)
    g = torch.Generator(device="cuda").manual_seed(7)
    qs = [torch.randn((T, 32, 128), generator=g, device="cuda").bfloat16() for _ in range(4)]
    base = s["vs"].clone()
    s["q"] = torch.empty_like(qs[0])
    ws = torch.empty(gdn.paged_attention_workspace_size(T, N, 32, 8, 128), dtype=torch.uint8, device="cuda")
    if planned:
        gdn.paged_attention_plan(s["cu"], s["kv"], ws, T=T, Hq=32, Hk=8, d=128, block_tokens=64,
                                 max_blocks=s["table"].shape[1], max_new_tokens=max(new))

    def step(i):
        s["q"].copy_(qs[i % 4])
        torch.mul(base, 2.0 ** (i % 3), out=s["vs"])
        return run(s, planned=planned, workspace=ws)
    expect = []
    for i in range(12):
        expect.append(step(i))
        torch.cuda.synchronize()
    got = [step(i) for i in range(12)]
    for i in range(12):
        assert torch.equal(got[i], expect[i]), i
    s["q"].copy_(qs[11 % 4])
    check(s, got[11])


@pytest.mark.parametrize("Hq,Hk,d", [(32, 8, 128), (16, 2, 256), (8, 8, 64)])
@pytest.mark.parametrize("decode", [0, 20])
def test_a_step_repeats_bit_by_bit(Hq, Hk, d, decode):
    # Copies that land while a step's data are still read would show in one step of thousands.
    from gated_deltanet_linear_build_gb300 import gdn
    new = [1] * decode + [130, 90, 300]
    kv = list(range(50, 50 + 100 * decode, 100)) + [700, 1200, 300]
    s = make(32, new, kv, Hq, Hk, d, 64)
    T, N = sum(new), len(new)
    ws = torch.empty(gdn.paged_attention_workspace_size(T, N, Hq, Hk, d), dtype=torch.uint8, device="cuda")
    first = run(s, workspace=ws)
    check(s, first)
    o, off = torch.empty_like(first), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(4000):
        gdn.paged_attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["kv"], o, ws,
                            softmax_scale=s["scale"], max_new_tokens=300)
        off += (o != first).any()
    assert int(off) == 0


@pytest.mark.parametrize("new,B", [([1], 16), ([3, 1], 64), ([70], 16), ([300, 5], 64)])
@pytest.mark.parametrize("Hq,Hk,d", [(8, 2, 64), (8, 2, 128), (16, 1, 128), (4, 1, 256)])
@pytest.mark.parametrize("exps", [(-100, 34), (34, -100), (-100, 100), (100, -100), (-100, 40, 100), (-100, 0, -100, 100)])
def test_value_scales_far_apart(new, B, Hq, Hk, d, exps):
    # Keys of blocks whose V scale is 2^200 smaller than another's keep their share of the softmax.
    kv = [l + 61 + 64 * 8 for l in new]
    s = make(41, new, kv, Hq, Hk, d, B)
    s["vs"].copy_(2.0 ** torch.tensor(exps, device="cuda")[torch.arange(len(s["vs"]), device="cuda") % len(exps)]
                  .float()[:, None].expand_as(s["vs"]))
    check(s, run(s))
    # In sequence order: all of one scale first.
    n = -(-kv[0] // B)
    s["vs"][s["table"][0, :n].long()] = 2.0 ** torch.tensor([exps[min(i * len(exps) // n, len(exps) - 1)] for i in range(n)],
                                                            device="cuda").float()[:, None]
    check(s, run(s))


@pytest.mark.parametrize("new,B", [([2], 16), ([70], 16), ([300], 64)])
def test_blocks_of_zeros_keep_their_share(new, B):
    # As the append leaves them: a block of zeros has the smallest scale.
    s = make(42, new, [new[0] + 500], 8, 2, 128, B)
    s["vs"].copy_(2.0 ** torch.tensor([40.0, 100.0], device="cuda")[torch.arange(len(s["vs"]), device="cuda") % 2]
                  [:, None].expand_as(s["vs"]))
    zero = s["table"][0, 0:-(-s["kvl"][0] // B):3].long()
    s["vc"].view(torch.uint8)[zero] = 0
    s["vs"][zero] = 2.0 ** -100
    check(s, run(s))


@pytest.mark.parametrize("new,N,keys", [(1, 400, 40000), (65, 160, 24000)])
def test_many_keys_of_the_smallest_scale(new, N, keys):
    # 2^-100 times every weight: sums of weights of up to 2^15 times 2^100 each. Equal sequences share blocks.
    d, B = 64, 64
    s = make(43, [new], [keys], 1, 1, d, B)
    s["kc"].view(torch.uint8)[:] = 0
    low = s["table"][0, :512 // B].long()                        # the first 512 keys are 2^-7.9 of the others
    s["kc"][..., 0] = torch.ones((), device="cuda").to(torch.float8_e4m3fn)
    s["kc"].view(torch.uint8)[low] = 0
    s["ks"].fill_(1.0)
    s["vs"].fill_(2.0 ** -100)
    s["q"].fill_(0.0)
    s["q"][..., 0] = 7.90625
    s["scale"] = 0.6931471805599453
    ref, a = R.attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["new"], s["kvl"], s["scale"])
    many = dict(s, q=s["q"].repeat(N, 1, 1), table=s["table"].repeat(N, 1), kv=s["kv"].repeat(N), new=[new] * N,
                cu=torch.arange(N + 1, dtype=torch.int32, device="cuda") * new)
    o = run(many).cpu().double().view(N, new, 1, d)
    assert ((o - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -8 * a + 1e-6 * a.max()).all()


@pytest.mark.parametrize("Hq,Hk,d", [(4, 2, 64), (8, 2, 128), (4, 1, 256)])
@pytest.mark.parametrize("new,kv", [([4], [2]), ([140], [100]), ([300], [0]), ([1, 1], [0, 5])])
def test_rows_without_keys_are_zero_whatever_q_holds(Hq, Hk, d, new, kv):
    s = make(44, new, kv, Hq, Hk, d, 16)
    empty = max(0, new[0] - kv[0])
    s["q"][:empty] = float("nan")
    s["q"][0, 0] = float("inf")
    o = run(s)
    assert (o[:empty] == 0).all()
    s["q"][:empty] = 0.0
    check(s, o)


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.int8, torch.bool])
def test_caches_of_another_8_bit_type_are_refused(dtype):
    from gated_deltanet_linear_build_gb300 import gdn
    s = make(45, [1, 1], [20, 30], 4, 2, 64, 16)
    for key in ("kc", "vc"):
        with pytest.raises(ValueError):
            run(dict(s, **{key: s[key].view(dtype)}))
    k = s["q"][:, :2].contiguous()
    pieces = torch.tensor([[0, 0, 2, 0]], dtype=torch.int32, device="cuda")
    before = s["kc"].view(torch.uint8).clone()
    with pytest.raises(ValueError):
        gdn.rotary_kv_append(None, k, k, None, None, pieces, pieces[0, 2:3], None, s["kc"].view(dtype),
                             s["vc"].view(dtype), s["ks"], s["vs"])
    assert torch.equal(before, s["kc"].view(torch.uint8))
    assert torch.equal(run(s), run(dict(s, kc=s["kc"].view(torch.uint8), vc=s["vc"].view(torch.uint8))))


def plan_records(ws, which, grid):
    """(starts, items) of one kernel's list in a workspace: dicts of int arrays."""
    starts_at = 0 if which == "split" else 2 * 320 * 64
    raw = ws.cpu().numpy()
    st = raw[starts_at:starts_at + grid * 64].view(np.int32).reshape(grid, 16)
    names = ("item", "head", "num", "units", "seq", "row0", "item_units", "cum", "first", "len", "kv", "c0")
    out = {k: st[:, i].astype(np.int64) for i, k in enumerate(names)}
    out["u"] = raw[starts_at:starts_at + grid * 64].view(np.int64).reshape(grid, 8)[:, 6]
    out["count"], out["pieces"] = st[:, 14].astype(np.int64), st[:, 15].astype(np.int64)
    return out


@pytest.mark.parametrize("N", [300, 1100, 3000])
@pytest.mark.parametrize("Hq,Hk,d,short", [(16, 2, 64, 20), (8, 8, 128, 70), (16, 1, 256, 8)])
def test_overlapping_sequences_stay_inside_the_plan(N, Hq, Hk, d, short):
    # Offsets that go back and forth: more tiles than a well-formed step of T tokens has. Every CTA's piece
    # lies inside its item, the pieces are the line, and a call ends with the rows that the sequences share.
    from gated_deltanet_linear_build_gb300 import gdn
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T, kv, B = 600, 700, 64
    s = make(48, [T], [kv], Hq, Hk, d, B)
    want = run(s)
    cu = np.where(np.arange(N + 1) % 2 == 0, 0, np.where(np.arange(N + 1) < 1024, T, short))
    bad = dict(s, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), kv=s["kv"].repeat(N),
               table=s["table"].repeat(N, 1), new=[T] + [0] * (N - 1))
    ws = torch.empty(gdn.paged_attention_workspace_size(T, N, Hq, Hk, d), dtype=torch.uint8, device="cuda")
    gdn.paged_attention_plan(bad["cu"], bad["kv"], ws, T=T, Hq=Hq, Hk=Hk, d=d, block_tokens=B,
                             max_blocks=s["table"].shape[1], max_new_tokens=T)
    p = plan_records(ws, "tile", min(sms, 160))
    work = p["count"] > 0
    assert work.any() and (p["units"] == p["units"][0]).all()
    if (p["c0"] >= 0).all():                                     # a line cut into pieces
        first = p["u"] - p["head"] * p["units"] - p["cum"]
        assert (p["head"][work] < Hk).all() and (p["item"][work] < p["num"][work]).all()
        assert (first[work] >= 0).all() and (first[work] < p["item_units"][work]).all()
        assert (p["u"][1:][work[1:]] == (p["u"] + p["count"])[:-1][work[1:]]).all()
        assert p["count"].sum() == p["units"][0] * Hk and p["u"][0] == 0
        last = p["num"] - 1 == p["item"]                          # the last item ends the line
        assert ((p["cum"] + p["item_units"])[last & work] == p["units"][last & work]).all()
    else:                                                        # whole items
        assert p["count"].sum() == p["num"][0] * Hk
    o = run(bad, workspace=ws)
    st = torch.empty(1, dtype=torch.int32, device="cuda")
    gdn.device_status(st, clear=True)
    assert int(st) == gdn.GDN_OK
    # Equal ranges end at T and, behind sequence 1024, at `short`: the rows of the former are the whole step's.
    rows = slice(short, T) if N > 1024 else slice(0, T)
    assert torch.equal(o[rows], want[rows]) or (o[rows].float() - want[rows].float()).abs().max() <= 2.0 ** -6


@pytest.mark.parametrize("new,N,d,which", [(1, 200, 128, "split"), (1, 700, 64, "split"), (256, 40, 64, "tile"), (3000, 30, 256, "tile")])
def test_a_plan_whose_units_pass_32_bits_is_reported_and_left_empty(new, N, d, which):
    # Lengths of 2^31 - 1024 keys, as shared blocks would allow; the plan reads no table.
    from gated_deltanet_linear_build_gb300 import gdn
    props = torch.cuda.get_device_properties(0).multi_processor_count
    T, Hq, Hk, B = new * N, 2, 2, 128
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda") * new
    ws = torch.empty(gdn.paged_attention_workspace_size(T, N, Hq, Hk, d), dtype=torch.uint8, device="cuda")
    st = torch.empty(1, dtype=torch.int32, device="cuda")
    gdn.device_status(st, clear=True)

    def plan(kv, blocks):
        ws.fill_(0x5A)
        gdn.paged_attention_plan(cu, torch.full((N,), kv, dtype=torch.int32, device="cuda"), ws, T=T, Hq=Hq, Hk=Hk, d=d,
                                 block_tokens=B, max_blocks=blocks, max_new_tokens=new)
        gdn.device_status(st, clear=True)
        return plan_records(ws, which, min(props, 160) if which == "tile" else props * (2 if d <= 128 else 1)), int(st)
    p, status = plan(0x7fffffff, (1 << 24) - 8)
    assert status == gdn.GDN_ERR_UNSUPPORTED and (p["count"] == 0).all() and (p["num"] == 0).all()
    # A table as wide, of sequences that are not as long, is planned as ever.
    p, status = plan(new + 5000, (1 << 24) - 8)
    q, ok = plan(new + 5000, -(-(new + 5000) // B))
    assert status == ok == gdn.GDN_OK and p["count"].sum() > 0
    assert all(np.array_equal(p[k], q[k]) for k in p)


@pytest.mark.parametrize("Hq,Hk,d", [(12, 1, 64), (32, 2, 64), (8, 2, 128), (24, 2, 128), (16, 1, 128), (16, 2, 256), (12, 1, 256),
                                     (16, 1, 256)])
def test_a_decode_step_repeats_bit_by_bit(Hq, Hk, d):
    # The split kernel alone, both of its row forms: its ring's slots are refilled while a unit is computed.
    from gated_deltanet_linear_build_gb300 import gdn
    kv = list(range(50, 2050, 100)) + [9000, 31, 4096, 700]
    s = make(33, [1] * len(kv), kv, Hq, Hk, d, 32)
    ws = torch.empty(gdn.paged_attention_workspace_size(len(kv), len(kv), Hq, Hk, d), dtype=torch.uint8, device="cuda")
    first = run(s, workspace=ws)
    check(s, first)
    o, off = torch.empty_like(first), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(4000):
        gdn.paged_attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["kv"], o, ws,
                            softmax_scale=s["scale"], max_new_tokens=1)
        off += (o != first).any()
    assert int(off) == 0


@pytest.mark.parametrize("new,kv", [([1, 1, 2], [700, 60, 9]), ([150, 40], [400, 40]), ([1, 90, 1], [900, 333, 20])])
@pytest.mark.parametrize("scale", [-0.11, 0.0, -0.0])
def test_softmax_scales_of_any_sign(new, kv, scale):
    s = make(46, new, kv, 8, 2, 128, 32)
    s["scale"] = scale
    check(s, run(s))


@pytest.mark.parametrize("new,kv", [([1, 2], [700, 60]), ([150, 90], [400, 2000]), ([300], [300])])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_outputs_off_a_32_byte_boundary_and_wide_tables(new, kv, d):
    from gated_deltanet_linear_build_gb300 import gdn
    s = make(47, new, kv, 4, 1, d, 32)
    a = run(s)
    check(s, a)
    T, N, M = sum(new), len(new), s["table"].shape[1]
    wide = torch.full((N, M + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :M] = s["table"]
    buf = torch.full((T * 4 * d + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
    o = buf[8:].view(T, 4, d)
    assert o.data_ptr() % 32 == 16
    ws = torch.empty(gdn.paged_attention_workspace_size(T, N, 4, 1, d), dtype=torch.uint8, device="cuda")
    gdn.paged_attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], wide[:, :M], s["cu"], s["kv"], o, ws,
                        softmax_scale=s["scale"], max_new_tokens=max(new))
    assert torch.equal(o, a) and torch.isnan(buf[:8]).all()


@pytest.mark.parametrize("decode,prompts,planned", [(20, 3, False), (20, 3, True), (0, 3, True), (24, 0, False)])
def test_steps_in_a_graph(decode, prompts, planned):
    # Tables, append and attention of two layers captured once; replays on other inputs in the same buffers
    # equal the calls made one by one.
    from gated_deltanet_linear_build_gb300 import gdn
    Hq, Hk, d, B = 16, 4, 128, 32
    new = [1] * decode + [130, 90, 300][:prompts]
    ctx = list(range(50, 50 + 60 * decode, 60)) + [700, 1200, 0][:prompts]
    N, T, L = len(new), sum(new), 2
    want = [-(-(c + l) // B) for c, l in zip(ctx, new)]
    blocks, width = sum(want), max(want)
    ids = np.random.default_rng(5).permutation(blocks)
    table, free, at = np.zeros((N, width), np.int32), [], 0
    for n in range(N):
        have = -(-ctx[n] // B)
        table[n, :want[n]] = ids[at:at + want[n]]
        free += list(table[n, have:want[n]])
        table[n, have:] = 0
        at += want[n]

    def ints(a):
        return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    cu, ctx_d, free_d, tab0 = ints(np.concatenate([[0], np.cumsum(new)])), ints(ctx), ints(free + [0]), ints(table)
    tab, kv, pos, counts = tab0.clone(), ints([0] * N), ints([0] * T), ints([0, 0])
    slots, pieces = torch.zeros(T, dtype=torch.int64, device="cuda"), ints(np.zeros((T // B + 2 * N, 4)))
    kc0, vc0, ks0, vs0 = R.fill_cache(np.random.default_rng(6), L * blocks, Hk, B, d, "cuda")
    cache = [x.clone().unflatten(0, (L, blocks)) for x in (kc0, vc0, ks0, vs0)]
    x = torch.zeros((L, T, (Hq + 2 * Hk) * d), dtype=torch.bfloat16, device="cuda")
    q_rot, o = torch.empty((T, Hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((L, T, Hq, d), dtype=torch.bfloat16, device="cuda")
    ph = gdn.rotary_phases(64, 10000.0)
    ws = torch.empty(gdn.paged_attention_workspace_size(T, N, Hq, Hk, d), dtype=torch.uint8, device="cuda")

    def step():
        gdn.build_block_tables(cu, ctx_d, free_d, tab, kv, pos, slots, pieces, counts, block_tokens=B)
        if planned:
            gdn.paged_attention_plan(cu, kv, ws, T=T, Hq=Hq, Hk=Hk, d=d, block_tokens=B, max_blocks=width,
                                     max_new_tokens=max(new))
        for l in range(L):
            q, k, v = (t.unflatten(1, (-1, d)) for t in x[l].split([Hq * d, Hk * d, Hk * d], 1))
            kc, vc, ks, vs = (c[l] for c in cache)
            gdn.rotary_kv_append(q, k, v, pos, ph, pieces, counts, q_rot, kc, vc, ks, vs)
            gdn.paged_attention(q_rot, kc, vc, ks, vs, tab, cu, kv, o[l], ws, softmax_scale=d ** -0.5,
                                max_new_tokens=max(new), planned=planned)

    gen = torch.Generator(device="cuda").manual_seed(3)
    inputs = [torch.randn(x.shape, generator=gen, device="cuda").bfloat16() for _ in range(3)]

    def reset(i):
        x.copy_(inputs[i])
        tab.copy_(tab0)
        for c, c0 in zip(cache, (kc0, vc0, ks0, vs0)):
            c.copy_(c0.unflatten(0, (L, blocks)))
        o.fill_(float("nan"))
    expect = []
    for i in range(3):
        reset(i)
        step()
        torch.cuda.synchronize()
        expect.append([t.clone() for t in (o, *cache)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in list(range(3)) * 20:
        reset(i)
        graph.replay()
        for got, ref in zip((o, *cache), expect[i]):
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))
    ref, a = R.attention(q_rot, *(c[1] for c in cache), tab, new, kv.tolist(), d ** -0.5)
    assert ((o[1].cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -8 * a + 1e-6 * a.max()).all()


@pytest.mark.parametrize("new,kv", [([1, 2], [700, 60]), ([150], [400])])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_key_scales_at_either_end(new, kv, d):
    s = make(49, new, kv, 4, 1, d, 16)
    every = torch.arange(len(s["ks"]), device="cuda")[:, None]
    ks = s["ks"].clone()
    s["ks"].copy_(torch.where(every % 2 == 0, 2.0 ** -100, ks))   # scores of a block of zeros: all zero
    check(s, run(s))
    s["ks"].copy_(ks * 2.0 ** 100)                               # with q as much smaller: the scores as before
    s["q"] *= 2.0 ** -100
    check(s, run(s))
