"""The operators around the selection at the edges of what they accept, on the host."""

import math

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_fp32_gb300 as tk  # noqa: E402
from sparse_attention_indexer_fp32_gb300 import _step  # noqa: E402
from test_step_host import ATTENTION, ROTARY, _status, lib  # noqa: E402, F401


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


def test_sizes_past_the_counters_are_refused(lib):  # noqa: F811
    """Products of sizes that pass 32 (or 64) bits, and heads whose count in steps would, before any CUDA call."""
    most = 2 ** 31 - 1
    for change in (dict(H=most), dict(H=2 ** 30 + 1, T=1)):
        assert _status(lib, "sparse_rotary", _step._RotaryArgs, ROTARY, **change) == tk.Status.EINVAL, change
    # 2^62, 2^64 (0 in 64 bits), 2^32 rows and heads, 2^31 tiles of heads
    for change in (dict(B=most, T=most), dict(B=2 ** 30, T=2 ** 30, Hkv=16, Hq=16), dict(B=2 ** 30, T=1, Hkv=4),
                   dict(B=2 ** 8, T=1, Hkv=1, Hq=most)):
        assert _status(lib, "sparse_attention", _step._AttentionArgs, ATTENTION, **change) == tk.Status.EINVAL, change


@pytest.mark.parametrize("base,rotated,length", [(10000.0, 64, 4096), (10000.0, 64, 131072), (10000.0, 128, 2 ** 20),
                                                 (500.0, 32, 65536), (1e6, 64, 8192), (10000.0, 16, 2 ** 27)])
def test_the_ramp_ends_where_the_pairs_turn_once(base, rotated, length):
    """Pairs that turn more than `fast` times are kept, those under `slow` times divided, and those between lie
    between, also where all pairs turn more than `slow` times and the ramp would end past the last."""
    plain = tk.rotary_frequencies(rotated, base, device="cpu")
    ramp = tk.rotary_frequencies(rotated, base, scaling="ramp", factor=8.0, original_length=length, device="cpu")
    turns, kept = plain * length / (2 * math.pi), ramp / plain
    assert torch.allclose(kept[turns > 32.0], torch.ones((), dtype=torch.float64), rtol=1e-14)
    assert torch.allclose(kept[turns < 1.0], torch.full((), 0.125, dtype=torch.float64), rtol=1e-14)
    assert (kept[turns > 1.001] > 0.1251).all()
    assert (kept[1:] <= kept[:-1] + 1e-14).all()


def test_the_ramp_needs_falling_frequencies():
    for base in (1.0, 0.5):
        with pytest.raises(ValueError, match="base above 1"):
            tk.rotary_frequencies(8, base, scaling="ramp", device="cpu")
