"""The answer side's calls on the GPU as programs hold them, and at sizes that take each of its paths.
Tolerances as in test_gpu_answer.py."""
import numpy as np
import pytest
import torch

from test_gpu_answer import ask, rows

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
