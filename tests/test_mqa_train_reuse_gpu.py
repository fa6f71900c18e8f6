"""Training steps one behind the other in the same save and workspace, on inputs that differ from step to step: none may read
what the step before it left there (its delta, sums of weights, documents, rotated queries and keys)."""

import numpy as np
import pytest
import torch

from gated_linear_recurrence_conv1d_b200 import binding, inputs

pytestmark = pytest.mark.gpu

D = 256
NAMES = ("out", "dq", "dk", "dv")


def _inputs(B, T, H, seed):
    rng = np.random.default_rng([seed, B, T, H])
    bits = lambda *s: inputs.f32_to_bf16_bits((2.0 ** rng.integers(-2, 3) * rng.standard_normal(s)).astype(np.float32))  # noqa: E731
    x = {n: binding.to_device(bits(B, T, H, D) if n in ("q", "dout") else bits(B, T, D)) for n in ("q", "k", "v", "dout")}
    x["reset"] = binding.to_device((rng.random((B, T)) < rng.choice([0.0, 0.02, 0.3])).astype(np.uint8))
    return x


def _step(dims, x, r, save, ws):
    binding.mqa_forward(dims, x["q"], x["k"], x["v"], r["out"], save, ws, reset=x["reset"])
    binding.mqa_backward(dims, x["v"], r["out"], x["dout"], save, r["dq"], r["dk"], r["dv"], ws)


def _results(x):
    return {n: torch.full_like(x["q" if n in ("out", "dq") else "k"], float("nan")) for n in NAMES}


@pytest.mark.parametrize("B,T,H,w,steps", [
    (1, 96, 1, 64, 200),               # dq ends long before dk / dv could
    (2, 300, 3, 128, 100),
    (3, 777, 3, 301, 60),
    (2, 2048, 10, 1024, 12),           # dk / dv starts on the SMs that dq leaves
])
def test_steps_in_the_same_buffers(B, T, H, w, steps):
    dims = binding.make_mqa_dims(B, T, H, D, w)
    xs = [_inputs(B, T, H, seed) for seed in range(3)]
    want = []
    for x in xs:                       # each in buffers of its own
        r, n = _results(x), (binding.mqa_save_size(dims), binding.mqa_train_workspace_size(dims))
        _step(dims, x, r, binding.alloc_workspace(n[0]), binding.alloc_workspace(n[1]))
        torch.cuda.synchronize()
        want.append(r)
    save = binding.alloc_workspace(binding.mqa_save_size(dims))
    ws = binding.alloc_workspace(binding.mqa_train_workspace_size(dims))
    got = [_results(xs[i % 3]) for i in range(steps)]
    torch.cuda.synchronize()
    for i in range(steps):
        _step(dims, xs[i % 3], got[i], save, ws)
    assert binding.read_device_status(ws) == binding.RGLRU_OK
    for i in range(steps):
        for n in NAMES:
            assert torch.equal(got[i][n].view(torch.int16), want[i % 3][n].view(torch.int16)), (i, n)


def test_backward_only_on_changing_gradients():
    """Of one forward, gradients of three losses in turn: only delta and the sums change in the workspace."""
    B, T, H, w = 3, 333, 4, 200
    dims = binding.make_mqa_dims(B, T, H, D, w)
    x = _inputs(B, T, H, 7)
    douts = [_inputs(B, T, H, seed)["dout"] for seed in (11, 12, 13)]
    save = binding.alloc_workspace(binding.mqa_save_size(dims))
    ws = binding.alloc_workspace(binding.mqa_train_workspace_size(dims))
    out = torch.empty_like(x["q"])
    binding.mqa_forward(dims, x["q"], x["k"], x["v"], out, save, ws, reset=x["reset"])

    def back(dout, r, work):
        binding.mqa_backward(dims, x["v"], out, dout, save, r["dq"], r["dk"], r["dv"], work)

    want = []
    for dout in douts:
        r = _results(x)
        back(dout, r, binding.alloc_workspace(binding.mqa_train_workspace_size(dims)))
        torch.cuda.synchronize()
        want.append(r)
    got = [_results(x) for _ in range(150)]
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        back(douts[i % 3], r, ws)
    assert binding.read_device_status(ws) == binding.RGLRU_OK
    for i, r in enumerate(got):
        for n in NAMES[1:]:
            assert torch.equal(r[n].view(torch.int16), want[i % 3][n].view(torch.int16)), (i, n)
