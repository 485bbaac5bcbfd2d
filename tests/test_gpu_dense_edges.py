"""The dense feed-forward operators at the edges of what their header allows:
no rows."""
import pytest
import torch

import sparse_tree_structured_amd as fff
from test_gpu_dense import DEV, TY, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,N", [(4097, 8192), (8191, 8191), (4096, 8192), (65535, 1023), (1023, 65535)])
def test_gradients_of_no_rows_at_wide_weights(K, N):
    say("no rows", K, N)
    for ty in ("bf16", "f32"):
        W = torch.empty(K, N, dtype=TY[ty], device=DEV)
        x, dy = W.new_empty(0, K), W.new_empty(0, N)
        dW, dbias, up = (torch.full(s, 7.0, device=DEV) for s in ((K, N), (N,), (K, N)))
        o = fff.linear_backward(dy, x, W, dW=dW, dbias=dbias)
        assert o.dx.shape == (0, K) and not bool(dW.any()) and not bool(dbias.any())
        g = fff.gated_backward(dy, x, W, W, dy, dy, want_h=True, dW_gate=dW.fill_(7.0), dW_up=up)
        assert g.dx.shape == (0, K) and g.h.shape == (0, N) and not bool(dW.any()) and not bool(up.any())
