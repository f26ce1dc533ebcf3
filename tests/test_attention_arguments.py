"""Refusals of the cross attention's binding that come before any GPU is asked for."""
import numpy as np
import pytest
import torch

from streaming_sinkhorn_solver_gb300 import binding as fs


@pytest.mark.parametrize("q", [np.zeros((1, 2, 2, 8), np.float16), [[[[0.0]]]], None, 1.0,
                               torch.zeros(1, 2, 2, 8), torch.zeros(1, 2, 2, 8, dtype=torch.float16)])
def test_queries_of_other_kinds(q):
    with pytest.raises(TypeError, match="bfloat16 or float16 CUDA tensor"):
        fs.fs_cross_attention(q, q, q)
    with pytest.raises(TypeError, match="bfloat16 or float16 CUDA tensor"):
        fs.fs_cross_attention_grad(q, q, q, q, q, q)
