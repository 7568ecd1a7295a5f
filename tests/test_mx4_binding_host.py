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


@pytest.mark.parametrize("K", [1 << 31, (1 << 32) + 32])
def test_rows_longer_than_the_library_takes(K):
    # K is an int there: 2^32 + 32 would arrive as 32. (A row of one element's memory; nothing is read)
    long = lambda n, t: torch.zeros(1, dtype=t).expand(1, n)
    for call in (lambda: ops.mx4_quantize(long(K, torch.bfloat16)),
                 lambda: ops.mx4_dequantize(long(K // 2, U8), long(K // 32, U8))):
        with pytest.raises(ops.MoeError) as e:
            call()
        assert e.value.status == ops.MOE_ERR_UNSUPPORTED_SHAPE
