"""The attention operators in use: a paged cache over several steps, and the hybrid stack.

Tolerance of the attention: as in test_gpu_attention (the cache is read back, so its rounding does not
enter): |o - ref| <= 2^-8 |ref| + 2^-8 a + 1e-6 max(a), and q is the layer's own rotated q."""
import numpy as np
import pytest
import torch

import attnref as R

pytestmark = pytest.mark.gpu


def test_steps_over_a_paged_cache():
    from gated_deltanet_linear_build_gb300 import hybrid
    rng = np.random.default_rng(3)
    N, hq, hk, d, B = 4, 8, 2, 128, 16
    at = hybrid.PagedAttentionLayers(2, N, num_blocks=48, max_seq_tokens=320, hq=hq, hk=hk, d=d, rot_dim=64,
                                     block_tokens=B, max_step_tokens=256)
    steps = [[200, 0, 31, 1], [56, 100, 1, 1], [1, 1, 1, 1], "release", [1, 17, 0, 40], [1, 1, 1, 1]]
    for new in steps:
        if new == "release":
            at.release(0)
            continue
        T = sum(new)
        at.begin_step(new)
        for l in range(2):
            x = torch.from_numpy(rng.standard_normal((T, (hq + 2 * hk) * d + 64)).astype(np.float32))
            x = x.bfloat16().cuda()
            q, k, v = (t.unflatten(1, (-1, d)) for t in x[:, :(hq + 2 * hk) * d].split([hq * d, hk * d, hk * d], 1))
            o = torch.full((T, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
            at.layer(l, q, k, v, o)
            ref, a = R.attention(at.q_rot[:T], at.k_cache[l], at.v_cache[l], at.k_scale[l], at.v_scale[l],
                                 at.table, new, at.context, at.scale)
            o = o.cpu().double()
            assert torch.isfinite(o).all()
            assert ((o - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -8 * a + 1e-6 * a.max()).all()
    table = at.table.cpu().numpy()
    for n in range(N):
        assert table[n, :len(at.blocks[n])].tolist() == at.blocks[n]
    assert at.kv_lens.tolist() == at.context


def weights(seed=5):
    from gated_deltanet_linear_build_gb300 import synth
    return synth.serving_stack(seed, layers=4, n_seqs=3, vocab=211, hk=2, hv=4, d=128, len_lo=40, len_hi=150)


def test_hybrid_stack_generates():
    from gated_deltanet_linear_build_gb300 import hybrid
    w = weights()
    stack = hybrid.HybridServingStack(w, budget=96, every=2, hq=8, hk=2, d_attn=64, rot_dim=32, block_tokens=16)
    ids, logits = stack.generate(6, keep_logits=(0, 2))
    again, same = stack.generate(6, keep_logits=(0, 2))
    assert ids.shape == (3, 7) and (ids >= 0).all() and (ids < 211).all()
    assert all(np.isfinite(x).all() for x in logits.values())
    # Equal inputs give equal bits: no sum depends on the order in which CTAs run.
    assert np.array_equal(ids, again) and all(np.array_equal(logits[s], same[s]) for s in logits)
    assert stack.attn.context == [len(p) + 6 for p in w["prompts"]]


def test_without_attention_layers_it_is_the_stack_of_before():
    from gated_deltanet_linear_build_gb300 import hybrid, serving
    w = weights(6)
    a, la = serving.SyntheticServingStack(w, budget=96).generate(4, keep_logits=(1,))
    h = hybrid.HybridServingStack(w, budget=96, every=9, hq=8, hk=2, d_attn=64, rot_dim=32, block_tokens=16)
    b, lb = h.generate(4, keep_logits=(1,))
    assert np.array_equal(a, b) and np.array_equal(la[1], lb[1])
