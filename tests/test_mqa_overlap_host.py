"""What a call of the attention's training step or of its 8-bit ring writes may not overlap anything else that it is given:
refused on the host, byte by byte (no GPU: nothing is launched)."""

import ctypes

import pytest

from gated_linear_recurrence_conv1d_b200 import binding

V = ctypes.c_void_p
B, T, H, D, W = 2, 16, 3, 256, 8
DIMS = binding.make_mqa_dims(B, T, H, D, W)
STEP = 1 << 28                         # addresses 256 MB apart, never dereferenced: a check fails first


def _sizes():
    q, kv, tok = B * T * H * D * 2, B * T * D * 2, B * T
    save, train = binding.mqa_save_size(DIMS), binding.mqa_train_workspace_size(DIMS)
    codes, scales = B * 2 * W * D, B * 2 * W * 4
    return {
        "forward": (dict(q=q, k=kv, v=kv, reset=tok), dict(out=q, save=save, ws=train)),
        "backward": (dict(v=kv, out=q, dout=q, save=save), dict(dq=q, dk=kv, dv=kv, ws=train)),
        "write": (dict(k=kv, v=kv, lengths=B * 4), dict(codes=codes, scales=scales)),
        "decode": (dict(q=B * H * D * 2, k=B * D * 2, v=B * D * 2, pos=B * 4),
                   dict(codes=codes, scales=scales, out=B * H * D * 2, ws=binding.mqa_decode8_workspace_size(DIMS))),
        "read": (dict(codes=codes, scales=scales, pos=B * 4), dict(cache=codes * 2)),
    }


def _call(name, a, sizes):
    lib, d = binding.load(), ctypes.byref(DIMS)
    p = {n: V(x) for n, x in a.items()}
    if name == "forward":
        return lib.rglru_mqa_forward(d, p["q"], p["k"], p["v"], p["reset"], 0, p["out"], p["save"], sizes["save"], p["ws"],
                                     sizes["ws"], None)
    if name == "backward":
        return lib.rglru_mqa_backward(d, p["v"], p["out"], p["dout"], p["save"], sizes["save"], p["dq"], p["dk"], p["dv"],
                                      p["ws"], sizes["ws"], None)
    if name == "write":
        return lib.rglru_mqa_cache8_write(d, p["k"], p["v"], p["lengths"], 0, p["codes"], p["scales"], None)
    if name == "decode":
        return lib.rglru_mqa_decode8(d, p["q"], p["k"], p["v"], p["pos"], p["codes"], p["scales"], p["out"], p["ws"],
                                     sizes["ws"], None)
    return lib.rglru_mqa_cache8_read(d, p["codes"], p["scales"], p["pos"], p["cache"], None)


def _pairs():
    for name, (ins, outs) in _sizes().items():
        names = list(ins) + list(outs)
        for o in outs:
            for n in names:
                if n != o:
                    yield name, o, n


@pytest.mark.parametrize("name,written,other", list(_pairs()))
def test_overlap_is_refused(name, written, other):
    ins, outs = _sizes()[name]
    sizes = {**ins, **outs}
    apart = {n: STEP * (i + 1) for i, n in enumerate(sizes)}
    at = apart[other]
    small = lambda n: n in ("scales", "pos", "lengths", "reset")  # noqa: E731
    unit = lambda n: 4 if small(n) else (256 if n in ("save", "ws") else 16)  # noqa: E731
    # at the same address; the written one's last bytes in the other's first; its first in the other's last
    for where in (at, at - (sizes[written] - 1) // unit(written) * unit(written),
                  at + (sizes[other] - 1) // unit(written) * unit(written)):
        assert _call(name, {**apart, written: where}, sizes) == 1, hex(where)


@pytest.mark.parametrize("name", list(_sizes()))
def test_an_optional_argument_that_is_not_given_overlaps_nothing(name):
    """Found by what is checked last: with the optional argument away, the overlap of two others is still what is refused,
    and a missing tensor as well."""
    ins, outs = _sizes()[name]
    sizes = {**ins, **outs}
    optional = {"forward": "reset", "write": "lengths", "read": "pos"}.get(name)
    a = {n: STEP * (i + 1) for i, n in enumerate(sizes)}
    if optional:
        a[optional] = None
    first_out = next(iter(outs))
    first_in = next(iter(ins))
    assert _call(name, {**a, first_out: a[first_in]}, sizes) == 1
    assert _call(name, {**a, first_in: None}, sizes) == 1
