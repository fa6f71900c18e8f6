"""rglru_mqa_decode8 on rings with slots whose scales are zero.  Bars as for any decode
step: 2^-6 of sum P |v| per element, 5e-3 RMS."""

import numpy as np
import pytest
import torch

from gated_linear_recurrence_conv1d_b200 import binding, inputs
from oracle import mqa_train
from tests.gpu_util import to_np

pytestmark = pytest.mark.gpu

D = 256


def _bf16(rng, shape, s=1.0):
    return inputs.f32_to_bf16_bits((s * rng.standard_normal(shape)).astype(np.float32))


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _decode(c, s, q, k, v, pos):
    """One step on the GPU and by the oracle: out, the oracle's, sum P |v| (all [B, H, d]); c, s as the oracle left them."""
    B, H = q.shape[:2]
    dims = binding.make_mqa_dims(B, 1, H, D, c.shape[2])
    ws = binding.alloc_workspace(binding.mqa_decode8_workspace_size(dims))
    out = torch.full((B, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    codes, scales = _dev(c), _dev(s)
    binding.mqa_decode8(dims, binding.to_device(q), binding.to_device(k), binding.to_device(v), _dev(pos), codes, scales,
                        out, ws)
    assert binding.read_device_status(ws) == binding.RGLRU_OK
    r = [mqa_train.decode_step8(c[b], s[b], q[b], k[b], v[b], int(pos[b])) for b in range(B)]
    assert np.array_equal(codes.cpu().numpy(), c)
    return to_np(out), np.stack([y for y, _ in r]), np.stack([a for _, a in r])


def _close(g, ref, pav, what):
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    rms = float(np.sqrt(np.mean((g - ref) ** 2)) / np.sqrt(np.mean(ref * ref)))
    assert rms <= 5e-3, f"{what}: RMS {rms:.3e}"
    worst = float(np.max(np.abs(g - ref) / np.maximum(pav, 1e-37)))
    assert worst <= 2.0 ** -6, f"{what}: {worst:.3e} of sum P |v|"


@pytest.mark.parametrize("B", [1, 40])             # a tile to a CTA; several tiles to a CTA
@pytest.mark.parametrize("filled", ["none", "first tile", "later tiles"])
def test_slots_of_zero_codes_and_zero_scales(B, filled):
    """What a zero-initialised ring holds where nothing was written (a prompt that began at a position past 0): values
    of zero, whose weights count like any other's."""
    rng = np.random.default_rng([41, B])
    H, w = 5, 900
    c, s = np.zeros((B, 2, w, D), dtype=np.uint8), np.zeros((B, 2, w), dtype=np.float32)
    part = {"none": slice(0, 0), "first tile": slice(3, 90), "later tiles": slice(300, 555)}[filled]
    n = part.stop - part.start
    if n:
        c[:, :, part], s[:, :, part] = mqa_train.quantise(rng.standard_normal((B, 2, n, D)))
    pos = np.array([(700, 899, 1300, 130)[b % 4] for b in range(B)], dtype=np.int32)
    q, k, v = _bf16(rng, (B, H, D)), _bf16(rng, (B, D)), _bf16(rng, (B, D))
    _close(*_decode(c, s, q, k, v, pos), filled)
