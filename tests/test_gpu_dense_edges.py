"""The dense half of a block where its calls could go wrong: kernels of CTA pairs again and again,
rows beyond whole tiles, buffers that overlap, values at the ends of the formats.

Tolerances as in test_gpu_dense_ops.py.
"""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import block_oracle as B
from test_gpu_dense_ops import _acc8, _close, _np, _rng, _rows8, _weights8, moe  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ 8-bit products
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_linear_fp8_pairs_again_and_again(moe, fmt):
    """Both CTAs of a pair hand their sums over 16 times a tile; each call gives the same bits,
    and rows of either CTA are right."""
    T, K, N = 2560, 2048, 1100
    g = _rng(T, K, N)
    x = _rows8(g, T, K)
    w, ws, wc, wsv = _weights8(g, N, K, fmt)
    q, s = moe.quantize_fp8_rows(x, fmt)
    y = moe.linear_fp8(q, w, ws, x_scale=s, out_dtype=torch.float32)
    at = torch.arange(0, T, 37)
    xc, _, xsv = O.quantize_blocks(_np(x)[at].astype(np.float32), 1, 128, fmt)
    ry, _, mag = B.linear_fp8(xc, xsv, wc, wsv)
    _close(y[at.cuda()], ry, mag, False, _acc8(K))
    for _ in range(40):
        assert torch.equal(moe.linear_fp8(q, w, ws, x_scale=s, out_dtype=torch.float32), y)
    moe.workspace_status(moe.default_workspace())
