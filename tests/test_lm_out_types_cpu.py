"""An output whose type is asked for and passed: both have to be the same."""
import pytest
import torch

E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_residual_norm(rcc_lib, dtype):
    x, weight = torch.zeros(4, 256, dtype=dtype), torch.ones(256)
    scaled = rcc_lib.Scaled(torch.zeros(4, 256).to(E4M3), torch.zeros(4, 2))
    for out, out_dtype in ((scaled, dtype), (torch.zeros_like(x), E4M3)):
        with pytest.raises(ValueError, match="out_dtype"):
            rcc_lib.add_rmsnorm_forward(x, x, weight, out=out, out_dtype=out_dtype)
    for out, out_dtype in ((scaled, None), (scaled, E4M3), (torch.zeros_like(x), None),
                           (torch.zeros_like(x), dtype), (None, dtype), (None, E4M3)):
        with pytest.raises(ValueError, match="CUDA device"):   # the last check
            rcc_lib.add_rmsnorm_forward(x, x, weight, out=out, out_dtype=out_dtype)
