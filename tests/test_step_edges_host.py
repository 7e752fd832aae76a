"""The operators around the selection at the edges of what they accept, on the host."""

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_fp32_gb300 as tk  # noqa: E402


def test_gradients_are_refused():
    """A tensor that requires a gradient would lose it: refused by name while gradients are recorded."""
    x = torch.zeros((2, 2, 8), dtype=torch.bfloat16, requires_grad=True)
    pos, f = torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.float64)
    q = torch.zeros((1, 1, 2, 16), dtype=torch.bfloat16, requires_grad=True)
    n = torch.zeros((1, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="x requires a gradient"):
        tk.rotary(x, pos, f)
    with pytest.raises(ValueError, match="q requires a gradient"):
        tk.indexer_scores(q, torch.zeros((1, 1, 2)), q[0], n, n)
    with pytest.raises(ValueError, match="q requires a gradient"):
        tk.sparse_attention(q, q, q, n[None])
    with torch.no_grad(), pytest.raises(ValueError, match="x must be a CUDA tensor"):
        tk.rotary(x, pos, f)
