"""What the language-model operators' binding checks before it touches a GPU:
every refusal here comes ahead of the one for tensors that are not on a CUDA
device."""
import pytest
import torch


@pytest.fixture
def L(rcc_lib):
    return rcc_lib


TOKENS, DIM = 4, 256
NEED = TOKENS * 2 * (128 + 4)


@pytest.mark.parametrize("data", [
    torch.empty(NEED - 1, dtype=torch.uint8),                     # the last scale is cut
    torch.empty(TOKENS * 2 * 128, dtype=torch.uint8),             # no scales at all
    torch.empty(0, dtype=torch.uint8),
    torch.empty(2 * NEED, dtype=torch.uint8)[::2],                # every other byte
    torch.empty(1, dtype=torch.uint8).expand(NEED),               # one byte, NEED times
    torch.empty(NEED, dtype=torch.int8), torch.empty(NEED // 4)])
def test_a_kept_input_in_too_small_a_buffer_is_refused(L, data):
    x, weight = torch.zeros(TOKENS, DIM), torch.ones(DIM)
    kept = L.Kept(TOKENS, DIM, data=data)
    with pytest.raises(ValueError, match="kept's buffer"):
        L.rmsnorm_forward(x, weight, keep=kept)
    with pytest.raises(ValueError, match="kept's buffer"):
        L.rmsnorm_backward(x, kept, weight)


def test_a_kept_input_of_other_sizes_is_refused(L):
    x, weight = torch.zeros(TOKENS, DIM), torch.ones(DIM)
    kept = L.Kept(TOKENS, DIM, "cpu")
    for name, value in (("tokens", TOKENS + 1), ("dim", DIM + 1)):
        changed = L.Kept(TOKENS, DIM, data=kept.data)
        setattr(changed, name, value)
        with pytest.raises(ValueError, match="kept must hold"):
            L.rmsnorm_backward(x, changed, weight)
    changed.tokens, changed.dim = "4", DIM
    with pytest.raises(TypeError):
        L.rmsnorm_backward(x, changed, weight)


def test_a_kept_input_that_fits_is_not_refused(L):
    x, weight = torch.zeros(TOKENS, DIM), torch.ones(DIM)
    for n in (NEED, NEED + 100):
        kept = L.Kept(TOKENS, DIM, data=torch.empty(n, dtype=torch.uint8))
        with pytest.raises(ValueError, match="CUDA device"):   # the last check
            L.rmsnorm_backward(x, kept, weight)
        assert kept.values.shape == (TOKENS, 256) and kept.scales.shape == (TOKENS, 2)


def test_a_device_that_is_not_current_is_refused(L):
    """What every call decides between its tensors' device and the current one."""
    from gradient_sync_rcc_gb300 import _lm
    for same in (0, 1, 7):
        assert _lm.check_device(same, same) is None
    for device, current in ((1, 0), (0, 1), (3, 2)):
        with pytest.raises(ValueError, match="device %d is not the inputs' device %d"
                           % (current, device)):
            _lm.check_device(device, current)
    with pytest.raises(TypeError):
        _lm.check_device("0", 0)
