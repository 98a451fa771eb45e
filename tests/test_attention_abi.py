"""The attention-side entry points on the CPU: host-side refusals before any launch, calls with nothing
to do, and the host-only functions. Fake pointers are never dereferenced on these paths."""
import ctypes

import pytest

from gated_deltanet_linear_build_gb300 import build as B

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4
A, A8, A4, A2 = 0x10000, 0x10008, 0x10004, 0x10002


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    from gated_deltanet_linear_build_gb300 import gdn
    return gdn.load_library()


def tables(lib, **kw):
    a = dict(cu=A, ctx=A, free=A, num_free=4, N=2, T=8, B=16, table=A, stride=4, max_blocks=4, kv=A, pos=A,
             slots=A, pieces=A, cap=4, counts=A, status=None)
    a.update(kw)
    return lib.gdn_build_block_tables(*a.values(), None)


def test_tables_refusals(lib):
    for key in ("cu", "ctx", "free", "table", "kv", "pos", "slots", "pieces", "counts"):
        assert tables(lib, **{key: None}) == INVALID, key
    for key in ("num_free", "N", "T", "max_blocks", "cap"):
        assert tables(lib, **{key: -1}) == INVALID, key
    assert tables(lib, stride=3) == INVALID
    assert tables(lib, N=0) == INVALID                      # tokens without a sequence
    for b in (0, 8, 24, 256, -16):
        assert tables(lib, B=b) == UNSUPPORTED
    for key in ("cu", "ctx", "free", "table", "kv", "pos", "counts", "status"):
        assert tables(lib, **{key: A2}) == ALIGN, key
    assert tables(lib, slots=A4) == ALIGN
    assert tables(lib, pieces=A8) == ALIGN
    assert tables(lib, N=0, T=0, cu=None) == OK


def rotary(lib, **kw):
    a = dict(q=A, qs=512, k=A, ks=128, pos=A, ph=A, qo=A, qos=512, ko=A, kos=128, T=4, Hq=4, Hk=1, d=128,
             rot=64, inter=0, inv=0, scale=1.0)
    a.update(kw)
    return lib.gdn_rotary(*a.values(), None)


def test_rotary_refusals(lib):
    for key in ("q", "k", "pos", "ph", "qo", "ko"):
        assert rotary(lib, **{key: None}) == INVALID, key
    for key, v in (("T", -1), ("Hq", -1), ("Hk", -1), ("inter", 2), ("inv", -1), ("scale", 0.0),
                   ("scale", float("nan")), ("scale", 2000.0), ("qs", 504), ("ko", A + 16), ("kos", 120)):
        want = OK if key == "ko" and v == A + 16 else INVALID
        if want == INVALID:
            assert rotary(lib, **{key: v}) == INVALID, (key, v)
    for key, v in (("d", 96), ("d", 512), ("rot", 24), ("rot", 144), ("rot", -16)):
        assert rotary(lib, **{key: v}) == UNSUPPORTED, (key, v)
    for key, v in (("q", A8), ("ko", A8), ("qs", 516), ("ph", A8), ("pos", A2)):
        assert rotary(lib, **{key: v}) == ALIGN, (key, v)
    assert rotary(lib, q=A, qo=A, qs=1024) == INVALID       # in place with another stride
    assert rotary(lib, T=0, q=None) == OK
    assert rotary(lib, Hq=0, Hk=0) == OK


def append(lib, **kw):
    a = dict(q=A, qs=512, k=A, ks=128, v=A, vs=128, pos=A, ph=A, pieces=A, num=A, cap=4, qo=A, qos=512, kc=A,
             vc=A, ksc=A, vsc=A, blocks=9, B=64, T=4, Hq=4, Hk=1, d=128, rot=64, inter=0, scale=1.0)
    a.update(kw)
    return lib.gdn_rotary_kv_append(*a.values(), None)


def test_append_refusals(lib):
    for key in ("q", "k", "v", "pos", "ph", "pieces", "num", "qo", "kc", "vc", "ksc", "vsc"):
        assert append(lib, **{key: None}) == INVALID, key
    for key, v in (("T", -1), ("Hq", -1), ("Hk", 0), ("blocks", -1), ("cap", -1), ("inter", 3), ("scale", -1.0),
                   ("ks", 120), ("vs", 64), ("qos", 256)):
        assert append(lib, **{key: v}) == INVALID, (key, v)
    for key, v in (("B", 48), ("B", 256), ("d", 32), ("d", 192), ("rot", 40), ("rot", 256)):
        assert append(lib, **{key: v}) == UNSUPPORTED, (key, v)
    for key, v in (("k", A8), ("v", A2), ("vc", A8), ("ksc", A2), ("pieces", A8), ("num", A2), ("ks", 132)):
        assert append(lib, **{key: v}) == ALIGN, (key, v)
    assert append(lib, T=0, k=None) == OK


def attend(lib, **kw):
    need = lib.gdn_paged_attention_workspace_size(4, 2, 8, 2, 128)
    a = dict(q=A, qs=1024, kc=A, vc=A, ks=A, vs=A, blocks=9, B=64, table=A, stride=5, mb=5, cu=A, kv=A, N=2, T=4,
             longest=2, o=A, Hq=8, Hk=2, d=128, scale=0.1, flags=0, ws=A, bytes=need)
    a.update(kw)
    return lib.gdn_paged_attention(*a.values(), None)


def test_attention_refusals(lib):
    for key in ("q", "kc", "vc", "ks", "vs", "table", "cu", "kv", "o"):
        assert attend(lib, **{key: None}) == INVALID, key
    for key, v in (("N", -1), ("T", -1), ("longest", -1), ("blocks", -1), ("Hq", 0), ("Hk", 0), ("Hk", 3),
                   ("mb", -1), ("stride", 4), ("qs", 512), ("scale", float("inf")), ("scale", float("nan")),
                   ("flags", 1), ("flags", -1)):
        assert attend(lib, **{key: v}) == INVALID, (key, v)
    for key, v in (("B", 20), ("d", 96), ("Hq", 34)):
        assert attend(lib, **{key: v}) == UNSUPPORTED, (key, v)
    for key, v in (("q", A8), ("kc", A8), ("o", A8), ("ks", A2), ("table", A2), ("cu", A2), ("ws", A + 16),
                   ("qs", 1028)):
        assert attend(lib, **{key: v}) == ALIGN, (key, v)
    assert attend(lib, ws=None) == WORKSPACE
    assert attend(lib, bytes=lib.gdn_paged_attention_workspace_size(4, 2, 8, 2, 128) - 1) == WORKSPACE
    assert attend(lib, T=0, q=None) == OK
    assert attend(lib, N=0, cu=None) == OK


def test_plan_refusals(lib):
    need = lib.gdn_paged_attention_workspace_size(4, 2, 8, 2, 128)
    f = lib.gdn_paged_attention_plan
    assert f(None, A, 2, 4, 8, 2, 128, 64, 5, 2, A, need, None) == INVALID
    assert f(A, A, 2, 4, 8, 2, 128, 64, 5, 2, A, need - 1, None) == WORKSPACE
    assert f(A, A, 2, 4, 8, 2, 80, 64, 5, 2, A, need, None) == UNSUPPORTED
    assert f(A, A, 0, 4, 8, 2, 128, 64, 5, 2, None, 0, None) == OK


def test_workspace_size(lib):
    f = lib.gdn_paged_attention_workspace_size
    assert f(4, 2, 8, 3, 128) == 0 and f(4, 2, 34, 2, 128) == 0 and f(4, 2, 8, 2, 96) == 0 and f(-1, 2, 8, 2, 64) == 0
    assert 0 < f(32, 32, 16, 2, 256) <= f(2048, 32, 16, 2, 256)


def test_phases(lib):
    out = (ctypes.c_int64 * 128)()
    f = lib.gdn_rotary_phases
    assert f(64, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, None) == INVALID
    assert f(24, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, out) == UNSUPPORTED
    assert f(272, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, out) == UNSUPPORTED
    assert f(64, 1.0, 0, 1.0, 0.0, 0.0, 0.0, out) == INVALID
    assert f(64, 10000.0, 1, 0.5, 0.0, 0.0, 0.0, out) == INVALID
    assert f(64, 10000.0, 3, 2.0, 0.0, 0.0, 0.0, out) == INVALID
    assert f(64, 10000.0, 2, 2.0, 0.0, 32.0, 1.0, out) == INVALID
    assert f(64, 10000.0, 2, 2.0, 4096.0, 1.0, 32.0, out) == INVALID
    assert f(64, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, out) == OK
    # Pair 0 turns one radian a token: 2^64 / (2 pi).
    assert abs((out[0] % 2 ** 64) / 2.0 ** 64 - 0.15915494309189535) < 2.0 ** -50
    plain = list(out[:32])
    assert f(64, 10000.0, 1, 4.0, 0.0, 0.0, 0.0, out) == OK
    assert all(abs(a / 4 - b) <= 2 ** 11 for a, b in zip(plain, out[:32]))
    assert f(64, 10000.0, 2, 4.0, 4096.0, 32.0, 1.0, out) == OK
    assert out[0] == plain[0] and abs(plain[31] / 4 - out[31]) <= 2 ** 11


def test_tables_of_2_31_keys_a_row_are_refused(lib):
    f, big = lib.gdn_paged_attention_plan, 1 << 30
    for B in (16, 128):
        assert f(A, A, 2, 4, 8, 2, 128, B, (1 << 31) // B, 2, A, big, None) == UNSUPPORTED
        assert attend(lib, B=B, mb=(1 << 31) // B - 1, stride=1 << 40) == UNSUPPORTED
    assert attend(lib, B=128, mb=(1 << 31) // 128 - 8, stride=1 << 40, ws=None) == WORKSPACE


def test_plan_refuses_host_tensors_and_other_lengths(monkeypatch):
    import torch
    from gated_deltanet_linear_build_gb300 import gdn

    class OnDevice(torch.Tensor):
        is_cuda = True

    def on(t):
        return t.as_subclass(OnDevice)
    calls = []
    monkeypatch.setattr(gdn, "_lib", lambda: type("L", (), {"gdn_paged_attention_plan": lambda self, *a: calls.append(a) or 0})())
    monkeypatch.setattr(gdn, "_stream", lambda s=None: 0)
    kw = dict(T=4, Hq=8, Hk=2, d=128, block_tokens=64, max_blocks=5, max_new_tokens=2)
    cu, kv = torch.tensor([0, 2, 4], dtype=torch.int32), torch.tensor([5, 6], dtype=torch.int32)
    ws = torch.zeros(1024, dtype=torch.uint8)
    for a in ((cu, on(kv), on(ws)), (on(cu), kv, on(ws)), (on(cu), on(kv), ws), (on(cu), on(kv[:1]), on(ws)),
              (on(cu.long()), on(kv), on(ws)), (on(cu), on(torch.arange(4, dtype=torch.int32)[::2]), on(ws)),
              (on(cu), on(kv), on(ws[::2])), (on(cu), on(kv[:, None]), on(ws))):
        with pytest.raises(ValueError):
            gdn.paged_attention_plan(*a, **kw)
    assert not calls
    gdn.paged_attention_plan(on(cu), on(kv), on(ws), **kw)
    assert calls[0][2:4] == (2, 4) and calls[0][11] == 1024


def test_counts_at_the_end_of_32_bits_are_refused(lib):
    top = (1 << 31) - 1
    for n in (top, top - 65535 + 1):
        assert tables(lib, N=n) == UNSUPPORTED and tables(lib, T=n) == UNSUPPORTED
        assert attend(lib, N=n, Hq=1, Hk=1, bytes=1 << 60) == UNSUPPORTED
        assert lib.gdn_paged_attention_workspace_size(4, n, 1, 1, 128) == 0
    assert lib.gdn_paged_attention_workspace_size(4, top - 65535, 1, 1, 128) > 0
