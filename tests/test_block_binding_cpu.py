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
    monkeypatch.setattr(block, "_as_stream", lambda stream, device: None)
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


@pytest.mark.parametrize("held", [False, True])
def test_adapters_that_require_gradients_are_replaced_whole(log, held):
    """Nothing is recorded: neither for factors that are held nor for those that replace them."""
    b, scale = rows(2, 32, 8).requires_grad_(held), rows(2, dtype=torch.float32).requires_grad_(held)
    w = block.Adapters(rows(2, 8, 64), b, scale)
    new, ones = torch.ones(1, 32, 8, dtype=BF, requires_grad=True), torch.ones(1, requires_grad=True)
    w.put(1, rows(1, 8, 64), new, ones)
    assert (w.b[1] == 1).all() and w.scale[1] == 1 and not w.b[0].any() and not w.scale[0]
    assert w.b.grad_fn is None and w.b.requires_grad == held and w.scale.requires_grad == held


def test_adapters_made_in_inference_mode_are_replaced_outside_of_it(log):
    with torch.inference_mode():
        w = block.Adapters(rows(2, 8, 64), rows(2, 32, 8), rows(2, dtype=torch.float32))
    w.put(0, rows(1, 8, 64), torch.ones(1, 32, 8, dtype=BF), torch.ones(1))
    assert (w.b[0] == 1).all() and w.scale.tolist() == [1, 0]


def test_factors_that_are_known_by_their_address_stay(log):
    w = block.Adapters(rows(2, 8, 64), rows(2, 32, 8), rows(2, dtype=torch.float32))
    plain = block.Adapters(rows(2, 8, 64), rows(2, 32, 8))
    for held, name in ((w, "a"), (w, "b"), (w, "scale"), (plain, "scale")):
        t = getattr(held, name)
        with pytest.raises(ValueError, match=name):
            setattr(held, name, torch.zeros(2) if t is None else t.clone())
        assert getattr(held, name) is t
    w.scale += 1
    w.b *= 2
    assert w.scale.tolist() == [1, 1] and w.desc.scale == w.scale.data_ptr()
