"""``block``'s binding without a GPU: host tensors, and what would be launched is recorded instead."""
import pytest
import torch

from diffusion_activation_residual_amd import block

CPU = torch.device("cpu")
BF = torch.bfloat16


@pytest.fixture
def log(monkeypatch):
    made = []
    monkeypatch.setattr(block, "_device", lambda t, what: t.device)

    def empty(device, stream, shape, dtype):
        made.append("allocated")
        return torch.zeros(shape, dtype=dtype)

    monkeypatch.setattr(block, "_empty_on", empty)
    monkeypatch.setattr(block, "_queue", lambda call, *a: made.append(call.__name__))
    return made


def rows(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("a,b", [(1, 2), (3, 2), (0, 2)])
def test_as_many_first_factors_as_second_ones(log, a, b):
    """Fewer would leave some adapter's first factor unset."""
    with pytest.raises(ValueError, match="adapters"):
        block.Adapters(rows(a, 8, 64), rows(b, 32, 8))
    assert log == []
    block.Adapters(rows(b, 8, 64), rows(b, 32, 8))
    assert log == ["allocated", "cfz_adapters_put"]
