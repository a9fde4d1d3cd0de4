"""Adapters where a workgroup of the second launch takes one, two, three and four times
256 channels, with ends inside each (GPU)."""
import pytest
import torch

import int4_weight_quantized_amd as w4
from test_gpu_lora import close, cuda, formula, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,r,L", [
    (16, 8192, 16, 16), (16, 8448, 16, 16), (16, 8195, 13, 16), (16, 16384, 40, 16), (16, 16640, 40, 16),
    (16, 16901, 33, 16), (16, 24576, 8, 16), (16, 24832, 8, 16), (16, 26113, 7, 16), (33, 9000, 130, 16),
    (300, 3328, 16, 8), (300, 3333, 20, 8), (700, 1500, 100, 5)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_channels_of_a_workgroup(M, N, r, L, dt):
    X, A, B, scales, ids, ranks, Y = make(M, 96, N, r, L, dt, M + N, True)
    want, bound = formula(X, A, B, scales, ids, ranks, Y)
    c = cuda(X, A, B, scales, ids, ranks, Y)
    close(w4.lora_add(c[6], c[0], c[4], c[1], c[2], scales=c[3], ranks=c[5]), want, bound)
