"""fp64 oracle of the local attention's training step and of its 8-bit ring cache -- TEST INFRASTRUCTURE.

Written from the formulas, with dense masks and numpy only; the CUDA library never imports it.

The training step of one batch row, heads h sharing keys and values (rotations as in oracle.mqa):

    s_hti = scale q~_ht . k~_i        for first(t) <= i <= t, first(t) = max(0, t - w + 1, start of t's document)
    P = softmax_i(s),  out = P v
    dP_hti = dout_ht . v_i,  delta_ht = dout_ht . out_ht,  dS = P (dP - delta)
    dq~ = scale dS k~,  dk~ = scale sum_h dS^T q~,  dv = sum_h P^T dout,   dq, dk turned back.

A ring slot in 8 bits: scale = fp32(max(amax, 448 2^-126) / 448), code = e4m3(x / scale) to the nearest,
ties to even, value = code * scale.
"""

from __future__ import annotations

from typing import Optional

import numpy as np

from oracle.mqa import _f64, rope


def first_key(T: int, window: int, reset: Optional[np.ndarray]) -> np.ndarray:
    """[T] for one row: the first token that token t attends to (reset [T] or None)."""
    first = np.zeros(T, dtype=np.int64)
    start = 0
    for t in range(T):
        if reset is not None and reset[t]:
            start = t
        first[t] = max(0, t - window + 1, start)
    return first


def train_step(q, k, v, dout, window: int, reset=None, pos0: int = 0, scale: Optional[float] = None,
               base: float = 10000.0) -> dict:
    """q, dout [B, T, H, d], k, v [B, T, d] -> out, dq, dk, dv in fp64, and for each the sum of the absolute
    values of the terms that its rounding errors are proportional to ("a_" + name)."""
    qf, kf, vf, of = _f64(q), _f64(k), _f64(v), _f64(dout)
    B, T, H, d = qf.shape
    sc = (1.0 / np.sqrt(d)) if scale is None else scale
    pos = pos0 + np.arange(T)
    qr, kr = rope(qf, pos[None, :, None], base), rope(kf, pos[None, :], base)
    r = {n: np.zeros(x.shape) for n, x in (("out", qf), ("dq", qf), ("dk", kf), ("dv", kf))}
    r.update({"a_" + n: np.zeros(r[n].shape) for n in list(r)})
    i = np.arange(T)
    half = d // 2

    def both(x):                       # a turn mixes the pair (j, j + d/2): |c|, |s| <= 1
        return np.tile(x[..., :half] + x[..., half:], 2)

    for b in range(B):
        first = first_key(T, window, None if reset is None else reset[b])
        seen = (i[None, :] <= i[:, None]) & (i[None, :] >= first[:, None])
        ak, av = np.abs(kr[b]), np.abs(vf[b])
        for h in range(H):
            s = np.where(seen, sc * (qr[b, :, h] @ kr[b].T), -np.inf)
            e = np.exp(s - s.max(axis=1, keepdims=True))
            p = e / e.sum(axis=1, keepdims=True)
            o = p @ vf[b]
            do = of[b, :, h]
            delta = (do * o).sum(axis=1, keepdims=True)
            ds = p * (do @ vf[b].T - delta)
            r["out"][b, :, h], r["a_out"][b, :, h] = o, p @ av
            r["dq"][b, :, h] = sc * (ds @ kr[b])
            r["dk"][b] += sc * (ds.T @ qr[b, :, h])
            r["dv"][b] += p.T @ do
            ads = p * (np.abs(do) @ av.T + (np.abs(do) * np.abs(o)).sum(axis=1, keepdims=True))
            r["a_dq"][b, :, h] = both(sc * (ads @ ak))
            r["a_dk"][b] += both(sc * (ads.T @ np.abs(qr[b, :, h])))
            r["a_dv"][b] += p.T @ np.abs(do)
    r["dq"] = rope(r["dq"], -pos[None, :, None], base)
    r["dk"] = rope(r["dk"], -pos[None, :], base)
    return r


# ---- e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN, no infinities ----
def e4m3_values() -> np.ndarray:
    """[256] the value of every code."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7f) == 0x7f, np.nan, v)
    return np.where(c & 0x80, -v, v)


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Nearest code of finite x, ties to even, saturating; a negative zero keeps its sign."""
    v = e4m3_values()[:127]
    a = np.abs(x)
    lo = np.clip(np.searchsorted(v, a, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    up = (a - v[lo] > v[hi] - a) | ((a - v[lo] == v[hi] - a) & (lo % 2 == 1))
    return (np.where(up, hi, lo) | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def quantise(x: np.ndarray):
    """x [..., d] fp64 -> (codes uint8, scales fp32)."""
    s = (np.maximum(np.abs(x).max(axis=-1), 448.0 * 2.0 ** -126) / 448.0).astype(np.float32)
    return e4m3_codes((x / s.astype(np.float64)[..., None]).astype(np.float32).astype(np.float64)), s


def dequantise(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return e4m3_values()[codes] * scales.astype(np.float64)[..., None]


def decode_step8(codes: np.ndarray, scales: np.ndarray, q, k, v, pos: int, scale: Optional[float] = None,
                 base: float = 10000.0):
    """One token of one row; codes [2, w, d], scales [2, w] are updated in place.  Returns (y [H, d], the same
    with |v|), zero for pos < 0."""
    qf = _f64(q)
    if pos < 0:
        return np.zeros(qf.shape), np.zeros(qf.shape)
    w, d = codes.shape[1], codes.shape[2]
    slot, n = pos % w, min(pos + 1, w)
    codes[0, slot], scales[0, slot] = quantise(rope(_f64(k), np.array(pos), base))
    codes[1, slot], scales[1, slot] = quantise(_f64(v))
    keys, vals = dequantise(codes[0, :n], scales[0, :n]), dequantise(codes[1, :n], scales[1, :n])
    s = ((1.0 / np.sqrt(d)) if scale is None else scale) * (rope(qf, np.array(pos), base) @ keys.T)
    e = np.exp(s - s.max(axis=-1, keepdims=True))
    p = e / e.sum(axis=-1, keepdims=True)
    return p @ vals, p @ np.abs(vals)
