"""Host side of the paged attention layers' step executor: block accounting and refusals (no GPU)."""
import pytest

from gated_deltanet_linear_build_gb300 import gdn, hybrid


@pytest.fixture
def layers(monkeypatch):
    calls = []
    monkeypatch.setattr(gdn, "build_block_tables", lambda *a, **k: calls.append(("tables", a, k)))
    monkeypatch.setattr(gdn, "paged_attention_plan", lambda *a, **k: calls.append(("plan", a, k)))
    at = hybrid.PagedAttentionLayers(2, 3, num_blocks=6, max_seq_tokens=64, hq=4, hk=2, d=64, rot_dim=32,
                                     block_tokens=16, max_step_tokens=64, device="cpu")
    at.calls = calls
    return at


def test_blocks_are_taken_in_order_and_come_back(layers):
    layers.begin_step([17, 0, 1])
    assert layers.blocks == [[0, 1], [], [2]] and layers.free == [3, 4, 5] and layers.context == [17, 0, 1]
    _, a, k = layers.calls[0]
    assert a[0].tolist() == [0, 17, 17, 18] and a[1].tolist() == [0, 0, 0] and a[2].tolist() == [0, 1, 2]
    assert k == {"block_tokens": 16}
    assert layers.calls[1][2]["max_new_tokens"] == 17 and layers.calls[1][2]["T"] == 18
    layers.begin_step([1, 16, 1])
    assert layers.blocks == [[0, 1], [3], [2]] and layers.context == [18, 16, 2]
    layers.release(0)
    assert layers.free == [0, 1, 4, 5] and layers.context == [0, 16, 2]
    layers.begin_step([0, 1, 15])
    assert layers.blocks == [[], [3, 0], [2, 1]] and layers.free == [4, 5]


@pytest.mark.parametrize("new,error", [([1, 1], ValueError), ([1, -1, 1], ValueError), ([30, 30, 30], ValueError),
                                       ([0, 65, 0], ValueError)])
def test_steps_that_are_refused(layers, new, error):
    with pytest.raises(error):
        layers.begin_step(new)
    assert not layers.calls and layers.context == [0, 0, 0] and len(layers.free) == 6


def test_a_step_that_does_not_fit_changes_nothing(layers):
    layers.begin_step([33, 1, 1])
    n = len(layers.calls)
    with pytest.raises(RuntimeError):
        layers.begin_step([1, 16, 16])                           # 1 free block, 2 needed
    with pytest.raises(ValueError):
        layers.begin_step([32, 0, 0])                            # a row holds 64 tokens
    assert len(layers.calls) == n and layers.context == [33, 1, 1] and layers.free == [5]
