"""LogitState keeps the addresses of the tensors it was made of, so it must not
come apart from them."""
import pytest

import token_sampling_logits_gb300 as gs

torch = pytest.importorskip("torch")
NAMES = ["history", "bias", "touched", "vocab", "rows", "ld", "device"]


class Device(torch.Tensor):
    """A host tensor that says it is on a device; its memory is not read."""
    is_cuda = True


def on_device(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Device)


@pytest.mark.parametrize("name", NAMES)
def test_attributes_cannot_be_assigned(name):
    """A state whose history was replaced would go on writing the old memory,
    which may be freed."""
    state = gs.LogitState(on_device(3, 64), on_device(3, 64, dtype=torch.float32),
                          on_device(3, 2), 50)
    before = getattr(state, name)
    with pytest.raises(AttributeError):
        setattr(state, name, before)
    assert getattr(state, name) is before or getattr(state, name) == before


def test_attributes_are_the_tensors_given():
    h, b, t = on_device(3, 64), on_device(3, 64, dtype=torch.float32), on_device(3, 2)
    state = gs.LogitState(h, b, t, 50)
    assert state.history is h and state.bias is b and state.touched is t
    assert (state.vocab, state.rows, state.ld, state.device) == (50, 3, 64, h.device)
    assert gs.LogitState(h, None, t, 64).bias is None
    c = state._c
    assert (c.history, c.bias, c.touched) == (h.data_ptr(), b.data_ptr(), t.data_ptr())
    assert (c.rows, c.vocab, c.ld) == (3, 50, 64)
