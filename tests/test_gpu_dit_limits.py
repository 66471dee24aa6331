"""Calls at the edges of what include/nvfp4_dit.h allows: operands that share
memory, values that are not finite, other streams and contexts."""
import pytest
import torch

import nvfp4_w4a4_gemm_quantize_b200 as nv
from nvfp4_w4a4_gemm_quantize_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mx"])
@pytest.mark.parametrize("M", [2, 3, 8, 16])
@pytest.mark.parametrize("N,K", [(131, 256), (300, 4224)])
def test_gemv_of_one_row_expanded(cuda_ok, fmt, M, N, K):
    """A conditioning row shared by the samples: the bits of its copies."""
    w = synth.random_bf16((N, K), seed=N, scale=0.02).cuda()
    w = nv.mx_quantize(w) if fmt == "mx" else nv.quantize(w)
    row = synth.random_bf16((1, K), seed=M).cuda()
    for x in (row.expand(M, K), row[0].expand(M, K)):
        assert x.stride(0) == 0
        for dtype in (torch.float32, torch.bfloat16):
            y = nv.gemv_w4a16(x, w, out_dtype=dtype)
            assert torch.equal(y, nv.gemv_w4a16(x.contiguous(), w, out_dtype=dtype))
            assert bool((y == y[:1]).all())
