"""rglru_mqa_decode8 on rings whose values' scales are zero, or lie many powers of two apart.  Bars as for any decode
step: 2^-6 of sum P |v| per element, 5e-3 RMS."""

import numpy as np
import pytest
import torch

from gated_linear_recurrence_conv1d_b200 import binding, inputs
from oracle import mqa, mqa_train
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


def _floor(c, s, q, pos):
    """[B, H]: what the weights' 8-bit parts may leave of every element beside the bar.  With n the largest s + log2 scale that
    the head's reference was set to, a weight is w = 2^12 2^(s + log2 scale - n), and the heaviest slot's is 2^12 at
    least.  A part (e5m2: 2 bits of mantissa, steps of 2^-16 below 2^-14) leaves an eighth of what it is given or half
    a step, 2^-17; it is given 8 times what the one before left.  Three leave max(2^-9 w, 2^-23) of w: the first is in the
    bar, the second is 2^-35 of the heaviest slot's weight times scale.  Codes are at most 448, and there are len slots."""
    B, H = q.shape[:2]
    r = np.zeros((B, H))
    for b in range(B):
        n = min(int(pos[b]) + 1, c.shape[2])
        keys = mqa_train.dequantise(c[b, 0, :n], s[b, 0, :n])
        x = mqa.rope(mqa._f64(q[b]), np.array(pos[b])) @ keys.T / 16.0
        p = np.exp(x - x.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        r[b] = n * 2.0 ** -35 * 448.0 * (p * s[b, 1, :n].astype(np.float64)).max(-1)
    return r


@pytest.mark.parametrize("order", ["same tile", "largest first", "largest last"])
@pytest.mark.parametrize("log2_ratio", [0, 20, 24, 30, 45, 90])
def test_the_heavy_slot_has_a_small_value(log2_ratio, order):
    """One key holds nearly all of every query's weight and its value is 2^-log2_ratio of the largest in the ring, whose key
    has next to no weight: e^-64 = 2^-92 against the heavy one's.  A query of zeros weighs all alike."""
    rng = np.random.default_rng([43, log2_ratio])
    B, H, w = 40, 4, 1000                          # 320 tiles: two or three to a CTA
    pos = (3 * w + np.arange(B) * 7).astype(np.int32)
    q, k = _bf16(rng, (B, H, D)), _bf16(rng, (B, D))
    v = _bf16(rng, (B, D), 2.0 ** -log2_ratio)
    q[:, 1:3] = q[:, :1]
    q[:, 3] = 0
    heavy, big = {"same tile": (200, 201), "largest first": (330, 140), "largest last": (140, 330)}[order]
    x = rng.standard_normal((B, 2, w, D))
    x[:, 1] *= 2.0 ** -log2_ratio
    x[:, 0] *= 0.1
    for b in range(B):
        qr = mqa.rope(mqa._f64(q[b, 0]), np.array(pos[b]))
        u = qr / np.dot(qr, qr)                    # q . u = 1: scores of +32 and -32 at a scale of 1 / 16
        x[b, 0, heavy], x[b, 0, big] = 512.0 * u, -512.0 * u
        x[b, 1, big] = rng.standard_normal(D)
    c, s = mqa_train.quantise(x)
    g, ref, pav = _decode(c, s, q, k, v, pos)
    pav += 2.0 ** 6 * _floor(c, s, q, pos)[..., None]
    for h in range(H):
        _close(g[:, h], ref[:, h], pav[:, h], f"head {h}")


@pytest.mark.parametrize("B", [2, 40])
def test_what_is_not_finite_stays_where_it_belongs(B):
    """A query with a NaN or an infinity: its head is NaN.  A slot, or a new key or value, that is not finite as a whole: its row's
    heads are NaN, in every column.  All other rows and heads keep their bits."""
    H, w = 6, 700
    pos = np.array([2 * w + 11 * b for b in range(B)], dtype=np.int32)

    def step(spoil):
        rng = np.random.default_rng([47, B])
        c, s = mqa_train.quantise(rng.standard_normal((B, 2, w, D)))
        q, k, v = _bf16(rng, (B, H, D)), _bf16(rng, (B, D)), _bf16(rng, (B, D))
        spoil(c, s, q, k, v)
        dims = binding.make_mqa_dims(B, 1, H, D, w)
        ws = binding.alloc_workspace(binding.mqa_decode8_workspace_size(dims))
        out = torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda")
        binding.mqa_decode8(dims, binding.to_device(q), binding.to_device(k), binding.to_device(v), _dev(pos), _dev(c), _dev(s),
                            out, ws)
        assert binding.read_device_status(ws) == binding.RGLRU_OK
        return out

    nan, inf = 0x7FC0, 0x7F80                      # bf16 bits
    b = B - 1
    head = lambda o: (o[b, 2:3], torch.cat([o[:b].flatten(), o[b, :2].flatten(), o[b, 3:].flatten()]))  # noqa: E731
    row = lambda o: (o[b], o[:b].flatten())  # noqa: E731

    def slot(half, scale):
        def spoil(c, s, q, k, v):
            c[b, half, 5], s[b, half, 5] = 0x7F, scale
        return spoil

    def put(name, at, bits):
        def spoil(c, s, q, k, v):
            dict(q=q, k=k, v=v)[name][at] = bits
        return spoil

    clean = step(lambda *x: None)
    for part, spoil in [(head, put("q", (b, 2, 9), nan)), (head, put("q", (b, 2, 200), inf)),
                        (row, slot(0, np.nan)), (row, slot(0, np.inf)), (row, slot(1, np.nan)), (row, slot(1, np.inf)),
                        (row, put("k", (b, 9), nan)), (row, put("v", (b, 9), inf)), (row, put("v", (b, 9), nan))]:
        (bad, rest), (_, same) = part(step(spoil)), part(clean)
        assert torch.isnan(bad).all()
        assert torch.equal(rest.view(torch.int16), same.view(torch.int16))
