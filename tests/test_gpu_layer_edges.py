"""Cases of the decoder layer's other operators beyond test_gpu_layer.py's:
batches of more sequences than one pass over them takes, tiny scales, empty
tables."""
import pytest
import torch

import bit_weight_only_g128_gb300 as w4
from test_gpu_layer import BF16, FP16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_norm_of_no_rows_answers_as_of_some(dtype):
    w = torch.ones(64, dtype=dtype, device="cuda")
    for rows in (0, 2):
        x, r = (torch.ones((rows, 64), dtype=dtype, device="cuda") for _ in range(2))
        y, h = w4.rms_norm(x, w, residual=r)
        assert y.shape == h.shape == (rows, 64)
        for quant, code in (("int8", torch.int8), ("codes", dtype)):
            q, s = w4.rms_norm(x, w, quant=quant)
            assert q.shape == (rows, 64) and q.dtype == code and s.shape == (rows,)
            q, s, h = w4.rms_norm(x, w, residual=r, quant=quant)
            assert q.shape == h.shape == (rows, 64) and s.shape == (rows,)
