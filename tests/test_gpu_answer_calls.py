"""The answer side's calls on the GPU as programs hold them, and at sizes that take each of its paths.
Tolerances as in test_gpu_answer.py."""
import math

import numpy as np
import pytest
import torch

import answerref as R
from test_gpu_answer import Linear, ask, bf16, compare, pack, rows, wide

pytestmark = pytest.mark.gpu


def test_logprobs_with_a_workspace():
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(1)
    for T, V, k in ((3, 300, 4), (2, 5000, 20)):
        x = rows(rng, T, V, torch.float32).cuda()
        tokens = torch.from_numpy(rng.integers(0, V, T)).int().cuda()
        first = ask(x, tokens, k)
        for size in (gdn.token_logprobs_workspace_size(T, V, k), 512):
            out = [torch.zeros_like(t) for t in first]
            ws = torch.empty(size, dtype=torch.uint8, device="cuda")
            gdn.token_logprobs(x, tokens, *out, ws, temperature=1.0)
            assert all(torch.equal(f, g) for f, g in zip(first, out))


class Repeated:
    """Products over weights of many rows that are copies of a few: every output is compared, at the price
    of the few. The workspace holds NaN before each call."""

    def __init__(self, N, K, seed=0):
        rng = np.random.default_rng(seed)
        self.N, self.K = N, K
        base = bf16(rng, 40, K)
        self.rows = torch.from_numpy(rng.integers(0, 40, N)).cuda()
        self.packed = pack(base.cuda()[self.rows])
        self.held = R.held(base).cuda()

    def workspace(self, T):
        from gated_deltanet_linear_build_gb300 import gdn
        return torch.full((gdn.w4_linear_workspace_size(T, self.N, self.K),), 0xFF, dtype=torch.uint8, device="cuda")

    def __call__(self, x, workspace, out=torch.float32):
        from gated_deltanet_linear_build_gb300 import gdn
        y = torch.full((x.shape[0], self.N), 77.0, dtype=out, device="cuda")
        gdn.w4_linear(x, self.packed, y, workspace)
        return y

    def check(self, x, y):
        xd = x.double()
        tol = (self.K / 16 + 16) * 2.0 ** -23 * (xd.abs() @ self.held.abs().T) + 2.0 ** -149
        tol = tol + 2.0 ** -22 * xd.abs().amax(1, True) * self.held.abs().sum(1)
        ref = xd @ self.held.T
        if y.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        off = (y.double() - ref[:, self.rows]).abs() - tol[:, self.rows]
        assert torch.isfinite(y).all() and off.max() <= 0, float(off.max())


@pytest.mark.parametrize("T,N,K", [(96, 4096, 8192), (70, 4096, 4096), (64, 4096, 16384), (33, 20000, 8192)])
def test_product_of_ctas_with_two_parts(T, N, K):
    # Tiles divided so that CTAs end one and begin the next, with an accumulator for each.
    p = Repeated(N, K, T)
    x = bf16(np.random.default_rng(T), T, K).cuda()
    ws = p.workspace(T)
    first = p(x, ws)
    assert not (ws == 0xFF).all()        # (the few-token kernel has no use for it)
    p.check(x, first)
    for _ in range(100):
        ws.fill_(0xFF)
        again = p(x, ws)
        assert torch.equal(again, first)


@pytest.mark.parametrize("T,N,K", [(1, 60000, 512), (9, 60000, 2048), (33, 40000, 640), (64, 60000, 1000),
                                   (64, 20000, 256), (1, 12000, 12000), (20, 9000, 8192), (33, 5000, 8192),
                                   (48, 8192, 6000), (64, 6000, 8192), (1, 131072, 64), (8, 3001, 16384),
                                   (9, 8192, 12000), (33, 9000, 6000), (64, 5000, 4096), (64, 3000, 8192)])
def test_product_of_few_tokens_over_several_row_tiles(T, N, K):
    # One row tile to seven for each cluster of one CTA or several: both accumulators, parts sent again and
    # again, a ring of codes that goes on from tile to tile. (Which of the cases with K of 4,096 and more go to
    # the general kernel instead depends on how many clusters a device holds.)
    p = Repeated(N, K, N + T)
    x = bf16(np.random.default_rng(N), T, K).cuda()
    x[T // 2] *= 2.0 ** -20              # (a token that has to be scaled beside others that have not)
    ws = p.workspace(T)
    for out in (torch.float32, torch.bfloat16):
        y = p(x, ws, out)
        p.check(x, y)
        for _ in range(20):
            assert torch.equal(p(x, ws, out), y)


@pytest.mark.parametrize("T,N,K,out", [
    (48, 12288, 4096, torch.bfloat16), (32, 131072, 4096, torch.float32), (32, 40000, 4096, torch.float32),
    (64, 30000, 1536, torch.bfloat16), (16, 60000, 8192, torch.float32), (20, 20000, 8192, torch.bfloat16),
    (9, 20000, 8192, torch.float32), (40, 5000, 16384, torch.bfloat16), (128, 4096, 8192, torch.float32),
    (112, 3001, 5000, torch.bfloat16), (256, 4096, 8192, torch.float32), (65, 20000, 2048, torch.float32)])
def test_product_whole_and_divided_by_the_general_kernel(T, N, K, out):
    # Up to 64 tokens, whole tiles and divided ones, and one accumulator or two behind them.
    p = Repeated(N, K, N + T)
    x = bf16(np.random.default_rng(N), T, K).cuda()
    ws = p.workspace(T)
    y = p(x, ws, out)
    p.check(x, y)
    for _ in range(20):
        ws.fill_(0xFF)
        assert torch.equal(p(x, ws, out), y)


@pytest.mark.parametrize("T,V", [(608, 1025), (16, 9000)])
def test_ranks_of_rows_of_a_round_or_two(T, V):
    # A warp may be through with its part of a row before another has begun; again and again.
    x = rows(np.random.default_rng(V), T, V, torch.float32).cuda()
    tokens = (torch.arange(T, device="cuda") * 37 % V).int()
    mine = x.gather(1, tokens.long()[:, None])
    index = torch.arange(V, device="cuda")
    ref = ((x > mine) | ((x == mine) & (index < tokens[:, None]))).sum(1).int()
    for k in (0, 3):
        for _ in range(200):
            assert torch.equal(ask(x, tokens, k)[2], ref)


def rows_without_probabilities(T, V, dtype):
    x = rows(np.random.default_rng(V), T, V, torch.float32)
    x[0, V // 3] = torch.nan
    x[1 % T, V // 2] = torch.inf
    if T > 7:
        x[2] = torch.nan
        x[3] = torch.inf
        x[4, ::2], x[4, 1::2] = torch.nan, -torch.inf
        x[5, 5:] = torch.nan                       # less than k tokens stand before the first NaN
        x[6, :] = 1.0
        x[6, V - 1] = torch.nan
        x[7] = torch.where(torch.arange(V) // 32 % 256 < 4, x[7].abs() + 9.0, x[7])     # the large in few lanes
        x[7, 0] = torch.inf
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", [(9, 1025), (9, 4099), (700, 3001), (1, 70001), (8, 150001), (400, 60001)])
def test_asked_long_rows_without_probabilities(T, V, dtype):
    # NaN and +inf in rows that a CTA or a cluster looks through, rows with probabilities between them.
    x = rows_without_probabilities(T, V, dtype)
    keep = list(range(min(T, 9)))
    for j, k in ((0, 32), (1, 5), (2, 0)):
        tokens = torch.tensor([(V // 3, V - 1, 3)[(t + j) % 3] for t in range(T)], dtype=torch.int32, device="cuda")
        got = [t[keep] for t in ask(x, tokens, k, 0.7)]
        compare(got, R.asked(x[keep], tokens[keep].cpu(), k, 0.7), V)


def test_a_nan_does_not_hold_up_a_call():
    # A row without probabilities is looked through again, but not once for each of the best.
    x = torch.randn((1, 3_000_017), device="cuda")
    tokens = torch.zeros(1, dtype=torch.int32, device="cuda")

    def time():
        ask(x, tokens, 32)
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            ask(x, tokens, 32)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    clean = time()
    x[0, 1_000_000] = torch.nan
    assert time() < 100 * clean


def test_packed_weights_of_other_sizes_are_refused():
    from gated_deltanet_linear_build_gb300 import gdn
    w = torch.randn((300, 200), device="cuda").bfloat16()
    whole = pack(w)
    x, y = w[:5], torch.empty((5, 300), device="cuda")
    ws = torch.empty(gdn.w4_linear_workspace_size(5, 300, 200), dtype=torch.uint8, device="cuda")
    gdn.w4_linear(x, whole, y, ws)
    for N, K in ((300, 128), (256, 200), (1, 200), (300, 1)):
        with pytest.raises(ValueError, match="other sizes"):
            gdn.w4_linear(x[:, :K] if K > 1 else x[:1, :1], whole, y[:, :N] if K > 1 else y[:1], ws)
        with pytest.raises(ValueError, match="other sizes"):
            gdn.w4_unpack(whole, w[:N, :K])
        with pytest.raises(ValueError, match="other sizes"):
            gdn.w4_pack(w[:N, :K], whole)
    with pytest.raises(RuntimeError):
        gdn.w4_linear(x, whole[:-1], y, ws)
    with pytest.raises(RuntimeError):
        gdn.w4_unpack(whole, torch.empty((400, 200), dtype=torch.bfloat16, device="cuda"))
    gdn.w4_linear(x[:0], whole, y[:0], ws)


@pytest.mark.parametrize("T", [1, 12])
def test_product_of_slices_that_lie_far_apart(T):
    # A token's largest value, 2^110, meets weights of zero; what is left is 2^-100 and smaller. Parts of other
    # slices than the largest value's count by 2^-149 of it at most, f16's largest times the weights a value.
    rng = np.random.default_rng(T)
    N, K = 200, 12000                    # (a cluster shares K)
    w = bf16(rng, N, K).float()
    w[:, :48] = 0.0
    lin = Linear(w.bfloat16())
    x = (bf16(rng, T, K).float() * 2.0 ** -100).bfloat16()
    x[:, 3] = 2.0 ** 110
    ref = x.double() @ lin.ref.T
    tol = K * 2.0 ** 15 * 2.0 ** -149 * 2.0 ** (110 - 14) * lin.ref.abs().amax(1)
    assert (ref.abs().amax(1) > 0).all()
    y = lin(wide(x, 0)).cpu().double()
    assert ((y - ref).abs() <= tol).all(), float(((y - ref).abs() / tol).max())
    x[T // 2, K - 1] = math.inf
    y, ref = lin(wide(x, 0)).cpu().double(), x.double() @ lin.ref.T
    row = ref[T // 2]
    assert torch.equal(torch.isnan(y[T // 2]), torch.isnan(row)) and torch.equal(y[T // 2] == math.inf, row == math.inf)
    assert torch.equal(y[T // 2] == -math.inf, row == -math.inf)


@pytest.mark.parametrize("stride", [256, 1 << 30, 1 << 39, 1 << 60])
def test_product_of_one_row_of_any_stride(stride):
    from gated_deltanet_linear_build_gb300 import gdn
    rng = np.random.default_rng(6)
    lin = Linear(bf16(rng, 70, 200))
    x = wide(bf16(rng, 1, 200), 0)
    first = lin(x)
    y = torch.zeros_like(first)
    ws = torch.empty(gdn.w4_linear_workspace_size(1, 70, 200), dtype=torch.uint8, device="cuda")
    rc = gdn.load_library().gdn_w4_linear(x.data_ptr(), stride, lin.packed.data_ptr(), lin.packed.numel(),
                                          y.data_ptr(), stride, 1, 1, 70, 200, ws.data_ptr(), ws.numel(),
                                          torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(y, first)


@pytest.mark.parametrize("T,N,K", [(1, 131072, 1024), (16, 131072, 640), (7, 60000, 1040), (12, 40000, 4160),
                                   (3, 20000, 2104), (16, 39000, 2304)])
def test_product_of_few_tokens_by_three_warpgroups(T, N, K):
    # CTAs of many steps: a third warpgroup widens; numbers of steps that three divides and does not, last
    # steps of one to four tiles.
    p = Repeated(N, K, N + T)
    x = bf16(np.random.default_rng(K), T, K).cuda()
    ws = p.workspace(T)
    y = p(x, ws)
    p.check(x, y)
    for _ in range(50):
        assert torch.equal(p(x, ws), y)
    assert torch.equal(p(x, ws, torch.bfloat16), y.bfloat16())
