"""Host-side checks of the attention's training and 8-bit cache entry points (no GPU: nothing is launched)."""

import ctypes

import pytest
import torch

from gated_linear_recurrence_conv1d_b200 import binding

A = [0x10000 * (i + 1) for i in range(10)]     # aligned addresses, never dereferenced: a check fails first
V = ctypes.c_void_p
BIG = 1 << 40


def _dims(B=2, T=16, H=3, d=256, w=8, scale=None, base=10000.0):
    return binding.make_mqa_dims(B, T, H, d, w, scale, base)


def _call(name, dims, *args):
    fn = getattr(binding.load(), name)
    return fn(ctypes.byref(dims) if dims is not None else None, *args)


def forward(dims, q=A[0], k=A[1], v=A[2], reset=None, pos0=0, out=A[3], save=A[4], sb=BIG, ws=A[5], wb=BIG):
    return _call("rglru_mqa_forward", dims, V(q), V(k), V(v), V(reset), pos0, V(out), V(save), sb, V(ws), wb, None)


def backward(dims, v=A[0], out=A[1], dout=A[2], save=A[3], sb=BIG, dq=A[4], dk=A[5], dv=A[6], ws=A[7], wb=BIG):
    return _call("rglru_mqa_backward", dims, V(v), V(out), V(dout), V(save), sb, V(dq), V(dk), V(dv), V(ws), wb, None)


def write8(dims, k=A[0], v=A[1], lengths=None, pos0=0, codes=A[2], scales=A[3]):
    return _call("rglru_mqa_cache8_write", dims, V(k), V(v), V(lengths), pos0, V(codes), V(scales), None)


def decode8(dims, q=A[0], k=A[1], v=A[2], pos=A[3], codes=A[4], scales=A[5], out=A[6], ws=A[7], wb=BIG):
    return _call("rglru_mqa_decode8", dims, V(q), V(k), V(v), V(pos), V(codes), V(scales), V(out), V(ws), wb, None)


def read8(dims, codes=A[0], scales=A[1], pos=None, cache=A[2]):
    return _call("rglru_mqa_cache8_read", dims, V(codes), V(scales), V(pos), V(cache), None)


ALL = [forward, backward, write8, decode8, read8]
SIZES = ["rglru_mqa_save_size", "rglru_mqa_train_workspace_size", "rglru_mqa_decode8_workspace_size"]


@pytest.mark.parametrize("fn", ALL)
@pytest.mark.parametrize("bad,code", [(dict(B=0), 1), (dict(H=0), 1), (dict(w=0), 1), (dict(scale=0.0), 1),
                                      (dict(scale=float("nan")), 1), (dict(base=-1.0), 1), (dict(d=128), 2),
                                      (dict(H=17), 2), (dict(B=65536), 2)])
def test_bad_dims(fn, bad, code):
    assert fn(_dims(**bad)) == code
    assert fn(None) == 1


def test_bad_sizes():
    for fn in (forward, backward, write8):
        assert fn(_dims(T=0)) == 1
    for fn in (forward, backward):
        assert fn(_dims(B=1, T=(1 << 30) // 3 + 1, H=3)) == 2          # T H > 2^30
    for fn in (write8, decode8, read8):
        assert fn(_dims(B=4, w=(1 << 27) + 1)) == 2                     # B w > 2^29


@pytest.mark.parametrize("fn,names", [
    (forward, ("q", "k", "v", "out")), (backward, ("v", "out", "dout", "dq", "dk", "dv")),
    (write8, ("k", "v", "codes")), (decode8, ("q", "k", "v", "codes", "out")), (read8, ("codes", "cache"))])
def test_missing_and_misaligned_tensors(fn, names):
    for n in names:
        assert fn(_dims(), **{n: None}) == 1, n
        assert fn(_dims(), **{n: 0x99998}) == 1, n


def test_missing_and_misaligned_vectors():
    for fn in (write8, decode8, read8):
        assert fn(_dims(), scales=None) == 1
        assert fn(_dims(), scales=0x99992) == 1
    assert decode8(_dims(), pos=None) == 1
    assert decode8(_dims(), pos=0x99992) == 1
    assert read8(_dims(), pos=0x99992) == 1
    assert write8(_dims(), lengths=0x99992) == 1


def test_outputs_may_not_alias():
    for n in ("q", "k", "v"):
        assert forward(_dims(), **{n: A[3]}) == 1
    for a, b in (("dq", A[2]), ("dk", A[0]), ("dv", A[1]), ("dk", A[4]), ("dv", A[5])):
        assert backward(_dims(), **{a: b}) == 1
    assert decode8(_dims(), out=A[0]) == 1
    assert decode8(_dims(), out=A[4]) == 1
    assert read8(_dims(), cache=A[0]) == 1
    assert write8(_dims(), codes=A[1]) == 1
    assert forward(_dims(), save=A[5]) == 1                             # save and workspace
    assert backward(_dims(), ws=A[3]) == 1


def test_positions_have_to_fit():
    for fn in (forward, write8):
        assert fn(_dims(), pos0=-1) == 1
        assert fn(_dims(T=16), pos0=2 ** 31 - 16) == 1


def test_buffers_have_to_be_large_enough():
    d = _dims()
    save, ws, w8 = (binding.mqa_save_size(d), binding.mqa_train_workspace_size(d), binding.mqa_decode8_workspace_size(d))
    assert min(save, ws, w8) >= 256
    for fn in (forward, backward):
        assert fn(d, sb=save - 1) == 3
        assert fn(d, save=None) == 3
        assert fn(d, wb=ws - 1) == 3
        assert fn(d, ws=None) == 3
        assert fn(d, ws=A[9] + 16) == 1
        assert fn(d, save=A[9] + 16) == 1
    assert decode8(d, wb=w8 - 1) == 3
    assert decode8(d, ws=None) == 3
    assert decode8(d, ws=A[9] + 16) == 1


def test_sizes_of_invalid_dims_are_zero():
    for n in SIZES:
        assert _call(n, _dims()) > 0
        assert _call(n, _dims(d=64)) == 0
        assert _call(n, None) == 0


def test_save_size_passes_32_bits():
    d = _dims(B=64, T=8192, H=16)
    assert binding.mqa_save_size(d) > 64 * 8192 * 16 * 512


def test_the_binding_refuses_tensors_that_are_not_what_the_dims_say():
    d = _dims()
    cpu = torch.zeros(2, 16, 3, 256, dtype=torch.bfloat16)
    kv = torch.zeros(2, 16, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.mqa_forward(d, cpu, kv, kv, cpu, kv, kv)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.mqa_backward(d, kv, cpu, cpu, kv, cpu, kv, kv, kv)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.mqa_cache8_read(d, kv, kv, kv)
