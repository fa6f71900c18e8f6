"""The 8-bit ring cache (rglru_mqa_cache8_write, rglru_mqa_decode8, rglru_mqa_cache8_read) against the fp64 oracle.

Codes and scales are compared for equality (scales to one rounding, 2^-23): both sides rotate and divide in
fp64.  At far positions p fp64 itself ends: base^(-2j/d) is off by up to 2 units of 2^-53 on the GPU and 1 on the
host, each product with p by half of one, so the two angles differ by up to p 2^-51, an element by sqrt(2) amax of
that, a scale by delta = 1.5 p 2^-51 of itself.  A code then differs where its quotient is within delta of a border:
borders are at least 1/16 of the value apart, so a share of at most 32 delta of the elements; 4 times that is
allowed, which is none below p = 10^7 on these sizes.  The decode's out: the roundings on the way are those of the rotated query (at most 2^-8 of each element),
of the softmax weight (2^-8 relative) and of the result; the ring's values are exact.  So as for the bf16
decode |O - O_ref| <= 2^-6 sum P |v|, RMS 5e-3."""

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


def _ring(rng, B, w):
    c, s = mqa_train.quantise(rng.standard_normal((B, 2, w, D)) * 10.0 ** rng.uniform(-1, 0.5, (B, 2, w, 1)))
    return c, s


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _same(codes, scales, c, s, what="", far=0):
    delta = 1.5 * far * 2.0 ** -51
    got = codes.view(torch.uint8).cpu().numpy()
    assert np.sum(got != c) <= int(4 * 32 * delta * c.size), f"{what}: {np.sum(got != c)} codes differ"
    assert np.all(np.abs(got.astype(int) - c) <= 1), what
    gs = scales.cpu().numpy()
    fin = np.isfinite(s)
    assert np.array_equal(np.isfinite(gs), fin), what
    assert np.all(np.abs(gs[fin] - s[fin]) <= (2.0 ** -23 + delta) * np.abs(s[fin])), what


def _close(g, ref, pav, what):
    assert np.all(np.isfinite(g)), what
    assert np.sqrt(np.mean((g - ref) ** 2)) <= 5e-3 * np.sqrt(np.mean(ref * ref)), what
    worst = float(np.max(np.abs(g - ref) / np.maximum(pav, 1e-30)))
    assert worst <= 2.0 ** -6, f"{what}: {worst:.3e} of sum P |v|"


@pytest.mark.parametrize("B,T,w,pos0,lengths", [
    (1, 1, 1, 0, None), (2, 5, 3, 0, None), (3, 40, 64, 10, None), (2, 300, 129, 1000003, None),
    (5, 70, 33, 5, [0, 70, 1, 33, 34]), (4, 20, 50, 0, [-3, 99, 20, 7]), (1, 700, 512, 2 ** 31 - 1 - 700, None)])
def test_write_matches_the_oracle(B, T, w, pos0, lengths):
    rng = np.random.default_rng([B, T, w])
    k, v = _bf16(rng, (B, T, D)), _bf16(rng, (B, T, D), 3.0)
    k[0, 0] = 0                                              # a zero key
    c, s = _ring(rng, B, w)
    codes, scales = _dev(c), _dev(s)
    dims = binding.make_mqa_dims(B, T, 1, D, w)
    binding.mqa_cache8_write(dims, binding.to_device(k), binding.to_device(v), codes, scales, pos0=pos0,
                             lengths=None if lengths is None else _dev(np.array(lengths, dtype=np.int32)))
    for b in range(B):
        n = T if lengths is None else min(max(lengths[b], 0), T)
        for t in range(max(0, n - w), n):
            slot = (pos0 + t) % w
            c[b, 0, slot], s[b, 0, slot] = mqa_train.quantise(mqa.rope(mqa._f64(k[b, t]), np.array(pos0 + t)))
            c[b, 1, slot], s[b, 1, slot] = mqa_train.quantise(mqa._f64(v[b, t]))
    _same(codes, scales, c, s, "write", far=pos0 + T)


def test_write_of_values_out_of_the_ordinary():
    """The smallest and largest bf16 values; a slot with an infinity or a NaN is not finite as a whole and leaves
    its neighbours alone."""
    T, w = 8, 8
    x = np.ones((1, T, D), dtype=np.float32)
    x[0, 0], x[0, 1], x[0, 2] = 1e-40, 3e38, 0.0
    x[0, 3, 5], x[0, 4, 200], x[0, 5, 0] = np.inf, np.nan, -1e30
    v = inputs.f32_to_bf16_bits(x)
    k = inputs.f32_to_bf16_bits(np.ones_like(x))
    codes, scales = torch.zeros(1, 2, w, D, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(1, 2, w, device="cuda")
    binding.mqa_cache8_write(binding.make_mqa_dims(1, T, 1, D, w), binding.to_device(k), binding.to_device(v), codes, scales)
    val = (codes.double() * scales.double()[..., None]).cpu().numpy()[0, 1]
    ref = inputs.bf16_bits_to_f32(v).astype(np.float64)[0]
    for t in (3, 4):
        assert not np.any(np.isfinite(val[t]))
    for t in (0, 1, 2, 5, 6, 7):
        s = float(scales[0, 1, t])
        assert np.all(np.abs(val[t] - ref[t]) <= np.maximum(2.0 ** -4 * np.abs(ref[t]), 2.0 ** -10 * s) * (1 + 1e-6)), t


@pytest.mark.parametrize("B,H,w,start,steps", [
    (1, 1, 1, 0, 3),                   # a ring of one slot
    (2, 3, 5, 0, 12),                  # from the first token through several turns of the ring
    (3, 16, 64, 60, 8),                # across the end of the ring
    (2, 10, 129, 120, 20),             # one slot past a tile
    (2, 7, 300, 128, 3),
    (1, 10, 2048, 100000, 2),          # a long full ring, one row
    (2, 2, 4095, 4000, 2),
])
def test_decode_steps_match_the_oracle(B, H, w, start, steps):
    """Slots that no step has reached hold NaN codes and scales: they must not leak."""
    rng = np.random.default_rng([B, H, w])
    c, s = _ring(rng, B, w)
    if start < w:
        c[:, :, start:], s[:, :, start:] = 0x7f, np.nan
    codes, scales = _dev(c).view(torch.float8_e4m3fn), _dev(s)
    dims = binding.make_mqa_dims(B, 1, H, D, w)
    ws = torch.full((binding.mqa_decode8_workspace_size(dims),), 0xff, dtype=torch.uint8, device="cuda")
    ws[:16] = 0
    for i in range(steps):
        q, k, v = _bf16(rng, (B, H, D)), _bf16(rng, (B, D)), _bf16(rng, (B, D))
        pos = np.full(B, start + i, dtype=np.int32)
        out = torch.full((B, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        binding.mqa_decode8(dims, binding.to_device(q), binding.to_device(k), binding.to_device(v), _dev(pos), codes,
                            scales, out, ws)
        r = [mqa_train.decode_step8(c[b], s[b], q[b], k[b], v[b], int(pos[b])) for b in range(B)]
        _close(to_np(out), np.stack([y for y, _ in r]), np.stack([a for _, a in r]), f"step {i}")
        _same(codes, scales, c, s, f"step {i}")
    assert binding.read_device_status(ws) == binding.RGLRU_OK


@pytest.mark.parametrize("B,H,w", [
    (80, 10, 2048), (160, 4, 700), (7, 16, 333),
    (1300, 5, 100),                    # many short rings, several to an SM
    (500, 16, 300),
])
def test_decode_of_rows_at_any_point(B, H, w):
    """Full and partly filled rings of values of many sizes, empty rows among them."""
    rng = np.random.default_rng([1, B])
    c, s = _ring(rng, B, w)
    pos = np.array([w + 997 * b if b % 3 else (b * 97) % w for b in range(B)], dtype=np.int32)
    pos[::5] = -1 - np.arange(len(pos[::5]))
    for b in range(B):
        if pos[b] + 1 < w:
            c[b, :, max(0, pos[b]):], s[b, :, max(0, pos[b]):] = 0xff, np.inf
    q, k, v = _bf16(rng, (B, H, D)), _bf16(rng, (B, D)), _bf16(rng, (B, D))
    codes, scales = _dev(c), _dev(s)
    dims = binding.make_mqa_dims(B, 1, H, D, w)
    ws = binding.alloc_workspace(binding.mqa_decode8_workspace_size(dims))
    out = torch.full((B, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    binding.mqa_decode8(dims, binding.to_device(q), binding.to_device(k), binding.to_device(v), _dev(pos), codes, scales,
                        out, ws)
    assert binding.read_device_status(ws) == binding.RGLRU_OK
    g = to_np(out)
    for b in range(B):
        y, a = mqa_train.decode_step8(c[b], s[b], q[b], k[b], v[b], int(pos[b]))
        if pos[b] < 0:
            assert np.all(g[b] == 0)
        else:
            _close(g[b], y, a, f"row {b} pos {pos[b]}")
    _same(codes, scales, c, s)


def test_decode_without_any_token():
    rng = np.random.default_rng(12)
    B, H, w = 9, 4, 50
    c, s = _ring(rng, B, w)
    codes, scales, pos = _dev(c), _dev(s), torch.full((B,), -1, dtype=torch.int32, device="cuda")
    x = [binding.to_device(_bf16(rng, sh)) for sh in ((B, H, D), (B, D), (B, D))]
    dims = binding.make_mqa_dims(B, 1, H, D, w)
    ws = torch.full((binding.mqa_decode8_workspace_size(dims),), 0xff, dtype=torch.uint8, device="cuda")
    ws[:16] = 0
    out = torch.full((B, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    binding.mqa_decode8(dims, *x, pos, codes, scales, out, ws)
    assert torch.all(out == 0)
    _same(codes, scales, c, s)
    assert binding.read_device_status(ws) == binding.RGLRU_OK


def test_decode_graphs_that_share_a_workspace():
    """Two captured decodes of unequal shapes in one workspace, replayed in turn on one stream."""
    rng = np.random.default_rng(13)
    cases = []
    for B, H, w in ((3, 16, 600), (200, 2, 130)):
        c, s = _ring(rng, B, w)
        x = [binding.to_device(_bf16(rng, sh)) for sh in ((B, H, D), (B, D), (B, D))]
        pos = torch.tensor(rng.integers(-1, 2 * w, B).astype(np.int32), device="cuda")
        cases.append(dict(dims=binding.make_mqa_dims(B, 1, H, D, w), x=x, pos=pos, ring=(_dev(c), _dev(s)), out=torch.zeros_like(x[0])))
    ws = binding.alloc_workspace(max(binding.mqa_decode8_workspace_size(m["dims"]) for m in cases))

    def step(m, stream=None):
        binding.mqa_decode8(m["dims"], *m["x"], m["pos"], *m["ring"], m["out"], ws, stream=stream)

    want = []
    for m in cases:
        step(m)
        want.append(m["out"].clone())
    torch.cuda.synchronize()
    stream, graphs = torch.cuda.Stream(), []
    for m in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step(m, stream)
        graphs.append(g)
    for _ in range(5):
        for m, g, y in zip(cases, graphs, want):
            m["out"].fill_(float("nan"))
            g.replay()
            assert torch.equal(m["out"], y)
    assert binding.read_device_status(ws) == binding.RGLRU_OK


def test_decode_of_keys_and_values_of_unequal_sizes():
    """One key dominates; values differ by 10^8 between slots; a query of zeros averages."""
    rng = np.random.default_rng(3)
    B, H, w = 2, 3, 200
    x = rng.standard_normal((B, 2, w, D))
    x[:, 0, 17] *= 6.0
    x[:, 1] *= 10.0 ** rng.uniform(-8, 0, (B, w, 1))
    c, s = mqa_train.quantise(x)
    q, k, v = _bf16(rng, (B, H, D)), _bf16(rng, (B, D)), _bf16(rng, (B, D))
    q[:, 1] = 0
    pos = np.array([1000, 1001], dtype=np.int32)
    dims = binding.make_mqa_dims(B, 1, H, D, w)
    ws = binding.alloc_workspace(binding.mqa_decode8_workspace_size(dims))
    out = torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
    binding.mqa_decode8(dims, binding.to_device(q), binding.to_device(k), binding.to_device(v), _dev(pos), _dev(c), _dev(s),
                        out, ws)
    for b in range(B):
        y, a = mqa_train.decode_step8(c[b], s[b], q[b], k[b], v[b], int(pos[b]))
        # scores up to 16 * 6 / 16 times larger than usual: a query's rounding moves them by 2^-8 of that
        assert np.all(np.abs(to_np(out)[b] - y) <= 2.0 ** -4 * a)


@pytest.mark.parametrize("B,w,fill", [(1, 1, None), (3, 33, None), (4, 100, [0, -1, 50, 1000]), (2, 2048, [2047, 12])])
def test_read_equals_code_times_scale(B, w, fill):
    rng = np.random.default_rng([B, w])
    c, s = _ring(rng, B, w)
    c[0, 0, 0] = np.arange(256)                              # every code, NaN among them
    cache = torch.full((B, 2, w, D), 3.0, dtype=torch.bfloat16, device="cuda")
    binding.mqa_cache8_read(binding.make_mqa_dims(B, 1, 1, D, w), _dev(c), _dev(s), cache,
                            pos=None if fill is None else _dev(np.array(fill, dtype=np.int32)))
    want = torch.from_numpy(mqa_train.e4m3_values()[c].astype(np.float32) * s[..., None]).to(torch.bfloat16).float().numpy()
    for b in range(B):
        n = w if fill is None else min(max(fill[b] + 1, 0), w)
        want[b, :, n:] = 3.0
    np.testing.assert_array_equal(to_np(cache).astype(np.float32), want)


def test_prompt_decode_and_hand_over_to_the_bf16_ring():
    """A serving run: a prompt through the forward, its keys and values into the 8-bit ring, decode steps, the ring
    read back, one more step against it with rglru_mqa_decode.  Every step against the oracle."""
    B, T, H, w = 2, 150, 4, 64
    rng = np.random.default_rng(21)
    q, k, v = _bf16(rng, (B, T, H, D)), _bf16(rng, (B, T, D)), _bf16(rng, (B, T, D))
    dims = binding.make_mqa_dims(B, T, H, D, w)
    ws = binding.alloc_workspace(binding.mqa_workspace_size(dims))
    out = torch.empty(B, T, H, D, dtype=torch.bfloat16, device="cuda")
    codes, scales = torch.zeros(B, 2, w, D, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(B, 2, w, device="cuda")
    binding.mqa_prefill(dims, binding.to_device(q), binding.to_device(k), binding.to_device(v), out, ws)
    binding.mqa_cache8_write(dims, binding.to_device(k), binding.to_device(v), codes, scales)
    c, s = np.zeros((B, 2, w, D), dtype=np.uint8), np.zeros((B, 2, w), dtype=np.float32)
    for b in range(B):
        for t in range(T - w, T):
            c[b, 0, t % w], s[b, 0, t % w] = mqa_train.quantise(mqa.rope(mqa._f64(k[b, t]), np.array(t)))
            c[b, 1, t % w], s[b, 1, t % w] = mqa_train.quantise(mqa._f64(v[b, t]))
    dd = binding.make_mqa_dims(B, 1, H, D, w)
    w8 = binding.alloc_workspace(binding.mqa_decode8_workspace_size(dd))
    od = torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
    for i in range(5):
        q1, k1, v1 = _bf16(rng, (B, H, D)), _bf16(rng, (B, D)), _bf16(rng, (B, D))
        pos = np.full(B, T + i, dtype=np.int32)
        binding.mqa_decode8(dd, binding.to_device(q1), binding.to_device(k1), binding.to_device(v1), _dev(pos), codes,
                            scales, od, w8)
        r = [mqa_train.decode_step8(c[b], s[b], q1[b], k1[b], v1[b], T + i) for b in range(B)]
        _close(to_np(od), np.stack([y for y, _ in r]), np.stack([a for _, a in r]), f"step {i}")
    cache = torch.empty(B, 2, w, D, dtype=torch.bfloat16, device="cuda")
    binding.mqa_cache8_read(dd, codes, scales, cache)
    rings = []
    for b in range(B):
        ring = mqa.RingCache(w, D)
        val = to_np(cache)[b].astype(np.float64)
        ring.k[:], ring.v[:] = val[0], val[1]
        rings.append(ring)
    q1, k1, v1 = _bf16(rng, (B, H, D)), _bf16(rng, (B, D)), _bf16(rng, (B, D))
    wd = binding.alloc_workspace(binding.mqa_workspace_size(dd, decode=True))
    binding.mqa_decode(dd, binding.to_device(q1), binding.to_device(k1), binding.to_device(v1),
                       _dev(np.full(B, T + 5, dtype=np.int32)), cache, od, wd)
    ref = np.stack([mqa.decode_step(rings[b], q1[b], k1[b], v1[b], T + 5) for b in range(B)])
    assert np.sqrt(np.mean((to_np(od) - ref) ** 2)) <= 5e-3 * np.sqrt(np.mean(ref * ref))


def test_decode_on_two_streams_and_replayed():
    rng = np.random.default_rng(8)
    w, H = 300, 5

    def make(B):
        c, s = _ring(rng, B, w)
        x = [binding.to_device(_bf16(rng, sh)) for sh in ((B, H, D), (B, D), (B, D))]
        dims = binding.make_mqa_dims(B, 1, H, D, w)
        return dict(c=c, s=s, x=x, dims=dims, pos=torch.full((B,), 100, dtype=torch.int32, device="cuda"),
                    ws=binding.alloc_workspace(binding.mqa_decode8_workspace_size(dims)))

    def fresh(m):
        return _dev(m["c"]), _dev(m["s"]), torch.empty_like(m["x"][0])

    def step(m, f, stream=None):
        binding.mqa_decode8(m["dims"], *m["x"], m["pos"], f[0], f[1], f[2], m["ws"], stream=stream)

    ms = [make(3), make(20)]
    want = []
    for m in ms:
        f = fresh(m)
        step(m, f)
        want.append(f[2].clone())
    bufs = [fresh(m) for m in ms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for m, f, st in zip(ms, bufs, streams):
            step(m, f, st)
    torch.cuda.synchronize()
    for f, wv in zip(bufs, want):
        assert torch.equal(f[2], wv)
    # one captured step replayed at other positions: lengths are read on the device
    m, f = ms[0], bufs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(m, f)
    for p in (100, 101, 299, 300, 5000):
        m["pos"].fill_(p)
        g.replay()
        a = f[2].clone()
        f2 = (f[0].clone(), f[1].clone(), torch.empty_like(a))
        step(m, f2)
        assert torch.equal(a, f2[2]), p


def test_rings_past_32_bits():
    """2100 rings of 4096 slots are 4.4 10^9 bytes: the last rows agree with the same rows in a batch of their own (bf16
    of sums in another order: one step of 2^-7), and their new slots are the same bytes."""
    B, H, w, n = 2100, 3, 4096, 2
    rng = np.random.default_rng(21)
    codes = torch.randint(0, 0x70, (B, 2, w, D), dtype=torch.uint8, device="cuda")
    scales = torch.rand(B, 2, w, device="cuda") * 0.01
    x = [binding.to_device(_bf16(rng, s)) for s in ((B, H, D), (B, D), (B, D))]
    pos = torch.full((B,), 3 * w + 77, dtype=torch.int32, device="cuda")

    def step(codes, scales, pos, *x):
        dims = binding.make_mqa_dims(pos.shape[0], 1, H, D, w)
        ws = binding.alloc_workspace(binding.mqa_decode8_workspace_size(dims))
        out = torch.empty_like(x[0])
        binding.mqa_decode8(dims, *x, pos, codes, scales, out, ws)
        assert binding.read_device_status(ws) == binding.RGLRU_OK
        return out

    own = (codes[-n:].clone(), scales[-n:].clone(), pos[-n:].clone(), *(t[-n:].clone() for t in x))
    y, z = to_np(step(codes, scales, pos, *x)[-n:]), to_np(step(*own))
    assert np.all(np.abs(y - z) <= 2.0 ** -7 * np.abs(z) + 2.0 ** -12 * np.max(np.abs(z)))
    assert torch.equal(codes[-n:], own[0]) and torch.equal(scales[-n:], own[1])
    cache = torch.empty(B, 2, w, D, dtype=torch.bfloat16, device="cuda")
    dims = binding.make_mqa_dims(B, 1, H, D, w)
    binding.mqa_cache8_read(dims, codes, scales, cache)
    small = torch.empty(n, 2, w, D, dtype=torch.bfloat16, device="cuda")
    binding.mqa_cache8_read(binding.make_mqa_dims(n, 1, H, D, w), own[0], own[1], small)
    assert torch.equal(cache[-n:], small)
