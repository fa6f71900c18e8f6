"""rglru_mqa_forward / rglru_mqa_backward against the fp64 oracle of oracle/mqa_train.py on the same bf16 inputs.

Tolerances.  The kernels round to bf16 (half a step: 2^-8 relative) the rotated queries and keys, the softmax
weights P, the gradient of the scores dS, and the result; delta sees the output with 16 bits; sums are fp32.
  * RMS: every one of these roundings is off by 2^-8 u, u uniform in [0, 1] over a step and halved where the
    mantissa is large: 1.7e-3 RMS relative.  A gradient chains at most seven of them that are independent
    (q~, k~ in the scores, P or dS twice, the weights behind delta, the other factor, the result): sqrt(7) 1.7e-3 = 4.5e-3, so
    5e-3, the framework's bar for bf16.  2^-16 of the RMS of the terms' absolute sums is added: where the
    terms cancel exactly (a token that sees one key only), what remains is fp32 rounding of those terms.
  * Element by element: |g - r| <= 2^-5 a, a = the sum of the absolute values of the terms (rounding a factor
    of a term moves it by 2^-8 of itself; at most eight roundings enter it, the scores' two through P, where
    a change of the score by 2^-8 |s| with |s| up to a few units counts as often)."""

import numpy as np
import pytest
import torch

from gated_linear_recurrence_conv1d_b200 import binding, inputs
from oracle import mqa_train
from tests.gpu_util import to_np

pytestmark = pytest.mark.gpu

D = 256
NAMES = ("out", "dq", "dk", "dv")


def _bf16(rng, shape, s=1.0):
    return inputs.f32_to_bf16_bits((s * rng.standard_normal(shape)).astype(np.float32))


def _problem(B, T, H, seed=0, docs=None):
    rng = np.random.default_rng([seed, B, T, H])
    x = {n: _bf16(rng, (B, T, H, D) if n in ("q", "dout") else (B, T, D)) for n in ("q", "k", "v", "dout")}
    reset = None
    if docs == "every":
        reset = np.ones((B, T), dtype=np.uint8)
    elif docs:
        reset = (rng.random((B, T)) < 1.0 / docs).astype(np.uint8) * 7      # nonzero, not only one
    return x, reset


class Run:
    """The two calls on given inputs, with their own buffers."""

    def __init__(self, x, reset, w, pos0=0, scale=None, device="cuda"):
        B, T, H, _ = x["q"].shape
        self.dims = binding.make_mqa_dims(B, T, H, D, w, scale)
        self.x = {n: binding.to_device(a) for n, a in x.items()}
        self.reset = None if reset is None else binding.to_device(reset)
        self.pos0 = pos0
        self.save = torch.full((binding.mqa_save_size(self.dims),), 0xff, dtype=torch.uint8, device=device)
        ws = binding.mqa_train_workspace_size(self.dims)
        self.ws = torch.full((ws,), 0xff, dtype=torch.uint8, device=device)
        self.ws[:16] = 0                                                      # the status word
        nan = float("nan")
        self.r = {n: torch.full_like(self.x["q" if n in ("out", "dq") else "k"], nan) for n in NAMES}

    def forward(self, stream=None):
        binding.mqa_forward(self.dims, self.x["q"], self.x["k"], self.x["v"], self.r["out"], self.save, self.ws,
                            pos0=self.pos0, reset=self.reset, stream=stream)

    def backward(self, stream=None):
        binding.mqa_backward(self.dims, self.x["v"], self.r["out"], self.x["dout"], self.save, self.r["dq"],
                             self.r["dk"], self.r["dv"], self.ws, stream=stream)

    def step(self, stream=None):
        self.forward(stream)
        self.backward(stream)
        return self

    def ok(self):
        assert binding.read_device_status(self.ws) == binding.RGLRU_OK
        return self

    def bits(self):
        return {n: t.view(torch.int16).clone() for n, t in self.r.items()}


def _close(run, ref, what):
    run.ok()
    for n in NAMES:
        g, r, a = to_np(run.r[n]), ref[n], ref["a_" + n]
        assert np.all(np.isfinite(g)), f"{what}: {n} is not finite"
        rms = lambda v: float(np.sqrt(np.mean(v * v)))  # noqa: E731
        assert rms(g - r) <= 5e-3 * rms(r) + 2.0 ** -16 * rms(a), f"{what}: {n} RMS {rms(g - r):.3e} of {rms(r):.3e}"
        worst = float(np.max(np.abs(g - r) / np.maximum(a, 1e-30)))
        assert worst <= 2.0 ** -5, f"{what}: {n} {worst:.3e} of its terms"


@pytest.mark.parametrize("B,T,H,w,docs,pos0", [
    (1, 1, 1, 1, None, 0),             # one token
    (2, 2, 16, 4096, None, 7),         # two tokens, all heads, a window past the row
    (1, 70, 1, 1, None, 0),            # a window of one: no gradient through the softmax
    (3, 65, 5, 2, None, 0),
    (1, 128, 1, 128, None, 0),         # whole tiles
    (2, 129, 2, 64, None, 1000000),    # one token past them, far positions
    (1, 300, 10, 100, 40, 3),          # documents and a window that both cut
    (2, 257, 3, 4096, 9, 0),           # short documents, no window
    (2, 100, 4, 32, "every", 0),       # every token a document of its own
    (1, 1111, 7, 513, 200, 0),         # many key tiles, odd everything
    (1, 900, 16, 700, None, 5),
])
def test_training_step_matches_the_oracle(B, T, H, w, docs, pos0):
    x, reset = _problem(B, T, H, docs=docs)
    ref = mqa_train.train_step(x["q"], x["k"], x["v"], x["dout"], w, reset, pos0)
    _close(Run(x, reset, w, pos0).step(), ref, f"B{B} T{T} H{H} w{w} docs {docs}")


def test_many_rows_with_unequal_documents():
    """More (row, key tile) pairs than SMs, some rows of one document, some of many."""
    B, T, H, w = 40, 260, 2, 200
    x, reset = _problem(B, T, H, seed=3, docs=30)
    reset[::3] = 0
    ref = mqa_train.train_step(x["q"], x["k"], x["v"], x["dout"], w, reset)
    _close(Run(x, reset, w).step(), ref, "many rows")


@pytest.mark.parametrize("scale", [1e-4, 0.5])
def test_score_scales(scale):
    """Nearly uniform weights, and weights that mostly sit on one key.  A rounding of q~ or k~ moves a score by
    up to 2^-8 sum |q| |k| scale, 0.6 of it at scale 0.5 on these inputs, in the worst case; typical is
    2^-8 |s| / 1.7 with |s| ~ 16 scale: 0.02 at 0.5.  So the RMS bar grows with 16 scale."""
    x, reset = _problem(1, 200, 3, seed=5, docs=64)
    ref = mqa_train.train_step(x["q"], x["k"], x["v"], x["dout"], 128, reset, scale=scale)
    run = Run(x, reset, 128, scale=scale).step().ok()
    for n in NAMES:
        g, r = to_np(run.r[n]), ref[n]
        assert np.sqrt(np.mean((g - r) ** 2)) <= 5e-3 * max(1.0, 16 * scale) * np.sqrt(np.mean(r * r)), n


def test_short_documents():
    """Rows of one and two keys: dS_1 = -dS_2 = P_1 P_2 (dP_1 - dP_2), what is left where dP_1 and delta cancel."""
    B, T, H = 2, 64, 16
    x, _ = _problem(B, T, H, seed=21)
    reset = np.zeros((B, T), dtype=np.uint8)
    reset[:, ::2] = 1
    ref = mqa_train.train_step(x["q"], x["k"], x["v"], x["dout"], 2048, reset)
    _close(Run(x, reset, 2048).step(), ref, "documents of two")


@pytest.mark.parametrize("scale", [0.67, 0.25])
def test_gradients_where_one_key_has_nearly_all_the_weight(scale):
    """A window of two, and scores that lie several units apart without a rounding error: the queries and keys fill
    only pairs whose angle is below 1e-8, so turning them leaves their bf16 values as they are.  Then
    dS_1 = P_1 P_2 (dP_1 - dP_2) = -dS_2 and dq = scale (dS_1 k_1 + dS_2 k_2).  Relative to dS: the weights behind out
    are rounded (2^-8 each of the two), dS itself is (2^-8), a score is off by fp32 sums (256 terms, 2^-16 of 50: under
    2^-10), so 4 2^-8.  Relative to the products behind the difference: out has 16 bits in delta (2^-15), the fp32
    sums of dP and delta 256 2^-24 each: P_j 2^-15 of sum |dO| |out| and 2^-15 of sum |dO| |v|.  The result: 2^-8."""
    B, T, H = 3, 33, 5
    rng = np.random.default_rng(77)
    x, _ = _problem(B, T, H, seed=22)
    for n in ("q", "k"):
        a = rng.uniform(0.5, 1.0, x[n].shape) * rng.choice([-1.0, 1.0], x[n].shape)
        a[..., :64] = 0.0
        a[..., 128:192] = 0.0
        x[n] = inputs.f32_to_bf16_bits(a.astype(np.float32))
    ref = mqa_train.train_step(x["q"], x["k"], x["v"], x["dout"], 2, scale=scale, base=1e20)
    run = Run(x, None, 2, scale=scale)
    run.dims.rope_base = 1e20
    _close(run.step(), ref, f"scale {scale}")

    q, k, v, g = (inputs.bf16_bits_to_f32(x[n]).astype(np.float64) for n in ("q", "k", "v", "dout"))
    q, g, out = q[:, 1:], g[:, 1:], ref["out"][:, 1:]
    k1, k2, v1, v2 = (y[:, :, None] for y in (k[:, :-1], k[:, 1:], v[:, :-1], v[:, 1:]))
    dot = lambda a, b: np.sum(a * b, -1, keepdims=True)  # noqa: E731
    s = scale * (dot(q, k2) - dot(q, k1))
    p1, p2 = 1.0 / (1.0 + np.exp(s)), 1.0 / (1.0 + np.exp(-s))
    ds = np.abs(p1 * p2 * (dot(g, v1) - dot(g, v2)))
    terms = dot(np.abs(g), np.abs(out)) + np.maximum(dot(np.abs(g), np.abs(v1)), dot(np.abs(g), np.abs(v2)))
    tol = scale * (4 * 2.0 ** -8 * ds * (np.abs(k1) + np.abs(k2)) + 2.0 ** -15 * terms * (p1 * np.abs(k1) + p2 * np.abs(k2)))
    err = np.abs(to_np(run.r["dq"])[:, 1:] - ref["dq"][:, 1:])
    assert np.min(np.minimum(p1, p2)) < 1e-3
    assert np.all(err <= tol + 2.0 ** -8 * np.abs(ref["dq"][:, 1:])), float(np.max(err / np.maximum(tol, 1e-30)))


def test_gradient_against_differences():
    """<dx, e> against (L(x + h e) - L(x - h e)) / 2h along random directions, L = <dout, out> from the kernel's
    own forward: out is bf16 (2^-8 relative, 1.7e-3 RMS), so L over n values is off by 1.7e-3 |dout| |out| / sqrt(n)
    per value ~ 1.7e-3 sqrt(n) 0.2; with h = 1/4 and n = 98304 that is 0.4 in the difference over 0.5: 0.6.  The
    rounding of x +- h e to bf16 is taken out by differencing the rounded values.  Curvature (h^2) is kept small
    against <dx, e> ~ |dx| by directions along dx itself, where <dx, e> = |dx| >> 1."""
    B, T, H, w = 1, 128, 3, 64
    x, reset = _problem(B, T, H, seed=9, docs=50)
    run = Run(x, reset, w).step().ok()
    for n in ("q", "k", "v"):
        d = to_np(run.r["d" + n])
        e = d / np.linalg.norm(d)
        vals = []
        moved = []
        for sgn in (1.0, -1.0):
            y = dict(x)
            bits = inputs.f32_to_bf16_bits((inputs.bf16_bits_to_f32(x[n]) + sgn * 4.0 * e).astype(np.float32))
            y[n] = bits
            r2 = Run(y, reset, w)
            r2.forward()
            vals.append(float((to_np(r2.r["out"]) * inputs.bf16_bits_to_f32(x["dout"]).astype(np.float64)).sum()))
            moved.append(inputs.bf16_bits_to_f32(bits).astype(np.float64))
        got = float((d * (moved[0] - moved[1])).sum())
        # a step of 4 along a unit vector over >= 32768 values moves each by ~0.02: curvature terms of (0.02)^2
        # relative per value, 2 % covers them and the 0.6 / |got| of the rounding above
        assert abs((vals[0] - vals[1]) - got) <= 0.02 * abs(got) + 1.0, (n, vals, got)


def test_the_same_call_gives_the_same_bits():
    x, reset = _problem(3, 400, 5, seed=1, docs=90)
    run = Run(x, reset, 200).step()
    first = run.bits()
    for _ in range(3):
        run.ws[16:] = 0x5a
        again = run.step().bits()
        assert all(torch.equal(first[n], again[n]) for n in NAMES)
    run.ok()


def test_rows_do_not_see_each_other():
    """A row alone gives the bits that it gives in a batch next to a row of large values."""
    x, reset = _problem(2, 150, 3, seed=2, docs=40)
    big = {n: a.copy() for n, a in x.items()}
    for n in big:
        if n == "v":
            big[n][1] = inputs.f32_to_bf16_bits(1e30 * np.ones(big[n][1].shape, dtype=np.float32))
    a, b = Run(x, reset, 64).step().bits(), Run(big, reset, 64).step().bits()
    assert all(torch.equal(a[n][0], b[n][0]) for n in NAMES)


def test_the_save_outlives_the_queries_and_the_workspace():
    x, reset = _problem(2, 200, 4, seed=4, docs=60)
    a = Run(x, reset, 100).step().bits()
    run = Run(x, reset, 100)
    run.forward()
    run.x["q"].fill_(float("nan"))
    run.x["k"].fill_(float("nan"))
    run.ws[16:] = 0x7f
    run.backward()
    b = run.bits()
    assert all(torch.equal(a[n], b[n]) for n in NAMES)


def test_two_steps_on_two_streams_and_a_captured_one():
    xa, ra = _problem(2, 300, 3, seed=6, docs=50)
    xb, rb = _problem(1, 555, 2, seed=7)
    want = [Run(xa, ra, 128).step().bits(), Run(xb, rb, 300).step().bits()]
    torch.cuda.synchronize()
    runs = [Run(xa, ra, 128), Run(xb, rb, 300)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for r, s in zip(runs, streams):
            r.step(s)
    torch.cuda.synchronize()
    for r, wv in zip(runs, want):
        assert all(torch.equal(r.ok().bits()[n], wv[n]) for n in NAMES)
    g = torch.cuda.CUDAGraph()
    cap = Run(xa, ra, 128)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cap.step()
    # new inputs in the captured buffers, other documents: the work of a step is decided on the device
    cap.reset.copy_(torch.roll(cap.reset, 37, 1))
    x2 = dict(xa)
    ref = mqa_train.train_step(x2["q"], x2["k"], x2["v"], x2["dout"], 128, cap.reset.cpu().numpy())
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    _close(cap, ref, "replayed with other documents")


def test_forward_agrees_with_the_prefill():
    """Without documents the forward computes what rglru_mqa_prefill computes: the same roundings of q~, k~ and
    P, another order of the sums and another reference maximum, so one step of bf16 (2^-7) of the result at
    most beside 2^-8 of the terms."""
    x, _ = _problem(2, 333, 5, seed=8)
    run = Run(x, None, 150, pos0=21)
    run.forward()
    ws = binding.alloc_workspace(binding.mqa_workspace_size(run.dims))
    out = torch.empty_like(run.x["q"])
    binding.mqa_prefill(run.dims, run.x["q"], run.x["k"], run.x["v"], out, ws, pos0=21)
    ref = mqa_train.train_step(x["q"], x["k"], x["v"], x["dout"], 150, None, 21)
    d = np.abs(to_np(run.r["out"]) - to_np(out))
    assert np.all(d <= 2.0 ** -7 * np.abs(ref["out"]) + 2.0 ** -7 * ref["a_out"])


def test_offsets_past_32_bits():
    """600000 tokens of 16 heads are 2.4 10^9 elements: the last tokens agree with the same tokens in a row of their
    own (both within 5e-3 of the exact values; the window keeps the rest of the row out of them)."""
    T, H, w, n = 600000, 16, 64, 640
    g = torch.Generator(device="cuda").manual_seed(3)
    big = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    x = {"q": big(1, T, H, D), "k": big(1, T, D), "v": big(1, T, D), "dout": big(1, T, H, D)}

    def step(y, pos0):
        t = y["q"].shape[1]
        dims = binding.make_mqa_dims(1, t, H, D, w)
        save = torch.empty(binding.mqa_save_size(dims), dtype=torch.uint8, device="cuda")
        ws = binding.alloc_workspace(binding.mqa_train_workspace_size(dims))
        r = {m: torch.empty_like(y["q" if m in ("out", "dq") else "k"]) for m in NAMES}
        binding.mqa_forward(dims, y["q"], y["k"], y["v"], r["out"], save, ws, pos0=pos0)
        binding.mqa_backward(dims, y["v"], r["out"], y["dout"], save, r["dq"], r["dk"], r["dv"], ws)
        assert binding.read_device_status(ws) == binding.RGLRU_OK
        return {m: t_[:, -(n - w):].clone() for m, t_ in r.items()}       # whole windows in both

    a = step(x, 5)
    b = step({m: t[:, -n:].contiguous() for m, t in x.items()}, 5 + T - n)
    for m in NAMES:
        u, v = to_np(a[m]), to_np(b[m])
        assert np.sqrt(np.mean((u - v) ** 2)) <= 1e-2 * np.sqrt(np.mean(v * v)), m
