"""What the binding of the MXFP4 calls refuses before any CUDA work. CPU only."""
import pytest
import torch

from route_permute_grouped_gb300 import ops

U8 = torch.uint8


@pytest.mark.parametrize("q", [None, [], {}, {"w2": torch.zeros(16, dtype=U8)}, {"w13": None, "w2": None}, {"w13": 1, "w2": 2},
                               {"w13": torch.zeros(16, dtype=U8), "w2": torch.zeros(16, dtype=U8)}])
def test_weights_that_are_not_there(q):
    cfg = ops.make_config(1, 128, 2, 1, 128)
    with pytest.raises(ops.MoeError) as e:
        ops.mx4_dequantize_weights(cfg, q)
    assert e.value.status == ops.MOE_ERR_INVALID_ARG
