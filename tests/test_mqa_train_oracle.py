"""Pins of oracle/mqa_train.py by something other than itself: the framework's attention oracle, differences
of the forward, separate documents, and torch's e4m3."""

import numpy as np
import pytest
import torch

from oracle import mqa, mqa_train


def _inputs(B, T, H, d, seed=0):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(s) for s in ((B, T, H, d), (B, T, d), (B, T, d), (B, T, H, d))]


def test_forward_equals_the_prefill_oracle():
    q, k, v, do = _inputs(2, 9, 3, 8)
    r = mqa_train.train_step(q, k, v, do, window=4, pos0=5)
    np.testing.assert_allclose(r["out"], mqa.prefill(q, k, v, window=4, pos0=5), rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("window,reset", [(3, None), (100, [0, 0, 0, 1, 0, 0, 1, 1]), (2, [1, 0, 0, 1, 0, 0, 0, 0])])
def test_gradients_equal_differences_of_the_forward(window, reset):
    q, k, v, do = _inputs(1, 8, 2, 4, seed=window)
    reset = None if reset is None else np.array([reset], dtype=np.uint8)
    r = mqa_train.train_step(q, k, v, do, window, reset, pos0=2)

    def loss(**kw):
        a = dict(q=q, k=k, v=v)
        a.update(kw)
        return (mqa_train.train_step(a["q"], a["k"], a["v"], do, window, reset, pos0=2)["out"] * do).sum()

    for name, x in (("q", q), ("k", k), ("v", v)):
        num = np.zeros(x.shape)
        for ix in np.ndindex(x.shape):
            def at(h):
                y = x.copy()
                y[ix] += h
                return loss(**{name: y})
            h = 1e-3                   # a fourth-order difference: error about h^4
            num[ix] = (8 * (at(h) - at(-h)) - (at(2 * h) - at(-2 * h))) / (12 * h)
        np.testing.assert_allclose(r["d" + name], num, rtol=1e-8, atol=1e-9)


def test_documents_equal_separate_rows():
    q, k, v, do = _inputs(1, 11, 2, 4)
    reset = np.zeros((1, 11), dtype=np.uint8)
    reset[0, [0, 4, 5]] = 1
    r = mqa_train.train_step(q, k, v, do, 6, reset)
    for lo, hi in ((0, 4), (4, 5), (5, 11)):
        p = mqa_train.train_step(*(x[:, lo:hi] for x in (q, k, v, do)), 6)   # scores depend on differences only
        for n in ("out", "dq", "dk", "dv"):
            # turning by other positions: the turned-back gradients agree all the same
            np.testing.assert_allclose(r[n][:, lo:hi], p[n], rtol=1e-9, atol=1e-12)


def test_e4m3_equals_torch():
    v = mqa_train.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(v, t)
    x = np.concatenate([np.random.default_rng(0).uniform(-448, 448, 20000), v[:127], -v[:127],
                        (v[:126] + v[1:127]) / 2, 10.0 ** np.random.default_rng(1).uniform(-5, 2.6, 20000)])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(mqa_train.e4m3_codes(x), want)


def test_quantised_values_are_within_half_a_step():
    x = np.random.default_rng(3).standard_normal((50, 256)) * 10.0 ** np.random.default_rng(4).uniform(-20, 20, (50, 1))
    x[7] = 0.0
    c, s = mqa_train.quantise(x)
    y = mqa_train.dequantise(c, s)
    # half a step: 2^-4 of a normal code, 2^-10 of the scale below them
    assert np.all(np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s[:, None].astype(float)) * (1 + 1e-6))
    assert np.all(y[7] == 0)


def test_decode8_equals_the_ring_decode_on_its_values():
    rng = np.random.default_rng(5)
    w, d, H = 5, 8, 2
    codes, scales = np.full((2, w, d), 0x7f, dtype=np.uint8), np.full((2, w), np.nan, dtype=np.float32)
    ring = mqa.RingCache(w, d)
    for p in range(13):
        q, k, v = rng.standard_normal((H, d)), rng.standard_normal(d), rng.standard_normal(d)
        y, _ = mqa_train.decode_step8(codes, scales, q, k, v, p)
        kv = mqa_train.dequantise(codes, scales)
        ring.push(kv[0, p % w], kv[1, p % w], p)
        keys, vals = ring.window_of(p)
        s = (mqa.rope(q, np.array(p)) @ keys.T) / np.sqrt(d)
        e = np.exp(s - s.max(axis=1, keepdims=True))
        np.testing.assert_allclose(y, (e / e.sum(axis=1, keepdims=True)) @ vals, rtol=1e-12)
