"""The attention's training step where a result is not finite: a NaN that a sum holds reaches out and the gradients as
one (a training loop finds a diverged run by it), and nothing else changes."""

import numpy as np
import pytest
import torch

from gated_linear_recurrence_conv1d_b200 import binding, inputs

pytestmark = pytest.mark.gpu

D = 256
B, T, H, W = 2, 200, 3, 64
NAMES = ("out", "dq", "dk", "dv")


def _inputs():
    rng = np.random.default_rng([31, B, T, H])
    bits = lambda *s: inputs.f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    return {"q": binding.to_device(bits(B, T, H, D)), "k": binding.to_device(bits(B, T, D)),
            "v": binding.to_device(bits(B, T, D)), "dout": binding.to_device(bits(B, T, H, D))}


def _step(x):
    dims = binding.make_mqa_dims(B, T, H, D, W)
    save = binding.alloc_workspace(binding.mqa_save_size(dims))
    ws = binding.alloc_workspace(binding.mqa_train_workspace_size(dims))
    r = {n: torch.zeros_like(x["q" if n in ("out", "dq") else "k"]) for n in NAMES}
    binding.mqa_forward(dims, x["q"], x["k"], x["v"], r["out"], save, ws)
    binding.mqa_backward(dims, x["v"], r["out"], x["dout"], save, r["dq"], r["dk"], r["dv"], ws)
    assert binding.read_device_status(ws) == binding.RGLRU_OK
    return r


def _prefill(x):
    dims = binding.make_mqa_dims(B, T, H, D, W)
    ws = binding.alloc_workspace(binding.mqa_workspace_size(dims))
    out = torch.zeros_like(x["q"])
    binding.mqa_prefill(dims, x["q"], x["k"], x["v"], out, ws)
    return out


def _same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_value_that_is_not_finite(bad):
    """Column 5 of token 100's value: that column of the rows that see the token, and every gradient that their delta
    enters; the other columns of out and the other batch row keep their bits."""
    clean = _step(_inputs())
    x = _inputs()
    x["v"][0, 100, 5] = bad
    r = _step(x)
    seen = slice(100, 100 + W)
    assert not torch.isfinite(r["out"][0, seen, :, 5]).any()
    assert not torch.isfinite(_prefill(x)[0, seen, :, 5]).any()
    if np.isnan(bad):
        assert torch.isnan(r["out"][0, seen, :, 5]).all()
        assert torch.isnan(r["dq"][0, seen]).all()
    rest = [c for c in range(D) if c != 5]
    assert _same_bits(r["out"][0][..., rest], clean["out"][0][..., rest])
    for n in NAMES:
        assert _same_bits(r[n][1], clean[n][1]), n


@pytest.mark.parametrize("where", ["q", "k"])
def test_a_query_or_key_that_is_nan(where):
    clean = _step(_inputs())
    x = _inputs()
    if where == "q":
        x["q"][0, 50, 1, 7] = float("nan")
        rows = (0, 50, 1)
    else:
        x["k"][0, 50, 7] = float("nan")
        rows = (0, slice(50, 50 + W))
    r = _step(x)
    assert torch.isnan(r["out"][rows]).all()
    assert torch.isnan(_prefill(x)[rows]).all()
    assert torch.isnan(r["dq"][rows]).all()
    for n in NAMES:
        assert _same_bits(r[n][1], clean[n][1]), n


def test_finite_inputs_whose_scores_overflow():
    """Query head 1 of token 50 and the key of token 50 in numbers of 1e20: their products are past fp32."""
    clean = _step(_inputs())
    x = _inputs()
    x["q"][0, 50, 1] = 1e20
    x["k"][0, 50] = 1e20
    r = _step(x)
    assert torch.isnan(r["out"][0, 50, 1]).all()
    assert torch.isnan(_prefill(x)[0, 50, 1]).all()
    assert torch.isnan(r["dq"][0, 50, 1]).all()
    for n in NAMES:
        assert _same_bits(r[n][1], clean[n][1]), n
