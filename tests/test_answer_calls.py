"""The answer side's calls as programs hold them, on the CPU: what was once accepted still is."""
import inspect

import pytest

from gated_deltanet_linear_build_gb300 import build as B


@pytest.fixture(scope="module")
def gdn():
    B.build_library()
    from gated_deltanet_linear_build_gb300 import gdn
    gdn.load_library()
    return gdn


def test_logprobs_with_a_workspace(gdn):
    # A program sizes a workspace and hands it in behind the outputs.
    for size in ((0, 1, 0), (1, 200003, 20), (4096, 262144, 32), (3, 7, 8), (-1, 7, 0), (1, 0, 0)):
        assert gdn.token_logprobs_workspace_size(*size) == 0
    call = inspect.signature(gdn.token_logprobs)
    outputs = ["logits", "tokens", "logprobs", "entropy", "ranks", "top_ids", "top_logprobs"]
    assert list(call.bind(*outputs, "workspace", temperature=0.5).arguments)[-2:] == ["workspace", "temperature"]
    call.bind(*outputs)
    call.bind(*outputs, workspace=None, stream=None)
