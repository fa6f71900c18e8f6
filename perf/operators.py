"""Local sliding-window MQA for training and its 8-bit ring cache: the cases that are measured, and their plain forms.

Four kinds of case, by ``case["op"]``:

  train   one training step of the attention: rglru_mqa_forward with documents and positions, then
          rglru_mqa_backward, returning out, dq, dk, dv
  write   rglru_mqa_cache8_write: a prompt's last keys (rotated) and values into the 8-bit ring
  decode  rglru_mqa_decode8: one token per row against the 8-bit ring, which it updates
  read    rglru_mqa_cache8_read: the 8-bit ring back as the bf16 ring

The 8-bit ring holds e4m3 codes [B, 2, w, 256] and one fp32 scale per slot and half [B, 2, w]:
scale = max(amax, 448 * 2^-126) / 448 over the 256 elements, code = e4m3(x / scale); the value is
code * scale.  Keys are stored after their rotation.
"""

import math

import numpy as np
import torch

own = False

D = 256                      # head_dim
BASE = 10000.0               # RoPE base
SCALE = 1.0 / 16.0           # 1 / sqrt(head_dim)
E4M3_MAX = 448.0
TINY = 2.0 ** -126


def listed():
    return [
        # a short prompt of one head: the step's latency
        dict(name="train_tiny", op="train", B=1, T=96, H=1, w=64, docs=0, pos0=0),
        # odd sizes, several documents a row, a window that does not divide anything
        dict(name="train_odd", op="train", B=3, T=777, H=3, w=301, docs=5, pos0=11),
        # RecurrentGemma-2B-shaped: 8 rows of 2048 tokens, 10 query heads, window 2048
        dict(name="train_rg2b", op="train", B=8, T=2048, H=10, w=2048, docs=0, pos0=0),
        # packed documents in one long row, 10 query heads, window 2048
        dict(name="train_packed", op="train", B=1, T=8192, H=10, w=2048, docs=2, pos0=0),
        # right-padded prompts of odd lengths, far positions
        dict(name="write_padded", op="write", B=5, T=515, w=300, pos0=1000003, pads=3),
        # the prompts of a RecurrentGemma-2B-shaped batch into rings of 2048
        dict(name="write_rg2b", op="write", B=8, T=2048, w=2048, pos0=0, pads=0),
        # one sequence, its ring full: the latency of a step
        dict(name="decode_one", op="decode", B=1, H=10, w=2048, fill=0),
        # a few rows at any point of short odd rings, one head count above the usual
        dict(name="decode_odd", op="decode", B=7, H=3, w=333, fill=4),
        # rows at all points of long rings, 16 heads (continuous batching)
        dict(name="decode_mixed", op="decode", B=48, H=16, w=4096, fill=9),
        # a serving batch, every ring full
        dict(name="decode_batch", op="decode", B=256, H=10, w=2048, fill=0),
        # partly filled rings of an odd size
        dict(name="read_odd", op="read", B=5, w=333, fill=6),
        # a batch's rings handed to a bf16 decode
        dict(name="read_batch", op="read", B=64, w=2048, fill=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["train", "train", "write", "decode", "decode", "read"])
    if op == "train":
        while True:
            # two tokens at least: the gradient through the softmax of a single key is zero
            B, T, H, w = _log_int(rng, 1, 8), _log_int(rng, 2, 8192), rng.randint(1, 16), _log_int(rng, 2, 4096)
            if B * H * T * T <= 10 * 8192 * 8192:
                return dict(op=op, B=B, T=T, H=H, w=w, docs=rng.choice([0, rng.randint(1, 10 ** 6)]),
                            pos0=rng.choice([0, rng.randint(1, 10 ** 6)]))
    if op == "write":
        while True:
            B, T, w = _log_int(rng, 1, 64), _log_int(rng, 1, 8192), _log_int(rng, 1, 4096)
            if B * T <= 8 * 2048 and B * w <= 64 * 2048:
                return dict(op=op, B=B, T=T, w=w, pos0=rng.choice([0, rng.randint(1, 10 ** 7)]),
                            pads=rng.choice([0, rng.randint(1, 10 ** 6)]))
    while True:
        B, w = _log_int(rng, 1, 256), _log_int(rng, 1, 4096)
        if B * w <= (256 if op == "decode" else 64) * 2048:
            break
    fill = rng.choice([0, rng.randint(1, 10 ** 6)])
    if op == "read":
        return dict(op=op, B=B, w=w, fill=fill)
    return dict(op=op, B=B, H=rng.randint(1, 16), w=w, fill=fill)


# ---- what a case fixes beside its sizes: documents, prompt lengths, positions ------------------
def _reset(case):
    """Packed documents until the row is full, lengths U{64..4096} (short rows: up to half the row);
    a nonzero byte starts a document."""
    if not case["docs"]:
        return None
    rng = np.random.RandomState(case["docs"])
    r = np.zeros((case["B"], case["T"]), dtype=np.uint8)
    for b in range(case["B"]):
        t = 0
        while t < case["T"]:
            r[b, t] = 1
            t += rng.randint(64, 4097) if case["T"] > 1024 else rng.randint(2, max(3, case["T"] // 2))
    return r


def _lengths(case):
    if not case["pads"]:
        return None
    return np.random.RandomState(case["pads"]).randint(0, case["T"] + 1, case["B"]).astype(np.int32)


def _positions(case):
    """fill 0: every ring full, at some far position; else rows anywhere from the first token to two rings."""
    rng = np.random.RandomState(case["fill"] + 1)
    if case["fill"] == 0:
        return (case["w"] + rng.randint(0, 100000, case["B"])).astype(np.int32)
    return rng.randint(0, 2 * case["w"], case["B"]).astype(np.int32)


def _first_key(case):
    """[B, T]: the first token that token t of a row attends to."""
    t = np.arange(case["T"])
    lo = np.broadcast_to(np.maximum(0, t - case["w"] + 1), (case["B"], case["T"]))
    r = _reset(case)
    if r is not None:
        lo = np.maximum(lo, np.maximum.accumulate(np.where(r != 0, t, 0), axis=1))
    return lo


def work(case):
    op, B = case["op"], case["B"]
    if op == "train":
        T, H = case["T"], case["H"]
        pairs = float((np.arange(T) + 1 - _first_key(case)).sum()) * H
        # forward: S and P V; backward: S again, dP, dV, dK, dQ
        return {"bytes": B * T * D * 2.0 * (4 * H + 4), "flops": 7 * 2.0 * D * pairs}
    if op == "write":
        T, w = case["T"], case["w"]
        n = _lengths(case)
        n = B * min(T, w) if n is None else int(np.minimum(n, w).sum())
        return {"bytes": n * 2.0 * (2 * D + D + 4), "flops": n * 6.0 * D}
    slots = float(np.minimum(_positions(case) + 1, case["w"]).sum())
    if op == "decode":
        H = case["H"]
        return {"bytes": slots * 2 * (D + 4) + B * D * 2.0 * (2 * H + 2), "flops": 4.0 * D * H * slots}
    return {"bytes": slots * 2 * (D + 4 + 2 * D), "flops": slots * 2 * D}


# ---- inputs -------------------------------------------------------------------------------------
def _quantise64(x):
    """[..., D] fp64 -> (e4m3 codes, fp32 scales)."""
    s = (x.abs().amax(-1).clamp_min(E4M3_MAX * TINY) / E4M3_MAX).float()
    return (x / s.double().unsqueeze(-1)).float().to(torch.float8_e4m3fn), s


def _ring(g, B, w):
    """A ring as earlier steps left it: rotated keys and values ~ N(0, 1), quantised."""
    codes = torch.empty(B, 2, w, D, dtype=torch.float8_e4m3fn, device="cuda")
    x = torch.randn(B, 2, w, D, generator=g, device="cuda")
    s = x.abs().amax(-1).clamp_min(E4M3_MAX * TINY) / E4M3_MAX
    codes.copy_((x / s.unsqueeze(-1)).to(torch.float8_e4m3fn))
    return codes, s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def bf(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    op, B = case["op"], case["B"]
    st = dict(case=case)
    if op == "train":
        T, H = case["T"], case["H"]
        st.update(q=bf(B, T, H, D), k=bf(B, T, D), v=bf(B, T, D), dout=bf(B, T, H, D))
        r = _reset(case)
        st["reset"] = None if r is None else torch.from_numpy(r).cuda()
        return st
    if op == "write":
        st.update(k=bf(B, case["T"], D), v=bf(B, case["T"], D))
        n = _lengths(case)
        st["lengths"] = None if n is None else torch.from_numpy(n).cuda()
        st["codes"], st["scales"] = _ring(g, B, case["w"])
        return st
    st["pos"] = torch.from_numpy(_positions(case)).cuda()
    st["codes"], st["scales"] = _ring(g, B, case["w"])
    if op == "decode":
        st.update(q=bf(B, case["H"], D), k=bf(B, D), v=bf(B, D))
    else:
        st["cache"] = torch.zeros(B, 2, case["w"], D, dtype=torch.bfloat16, device="cuda")
    return st


# ---- the plain forms ------------------------------------------------------------------------------
def _rotate(x, pos, back=False):
    """x [..., D] fp64 turned by its position (pos broadcasts over x's leading axes)."""
    inv = BASE ** (-2.0 * torch.arange(D // 2, device=x.device, dtype=torch.float64) / D)
    ang = pos.double().unsqueeze(-1) * inv
    c, s = torch.cos(ang), torch.sin(ang)
    if back:
        s = -s
    x1, x2 = x[..., : D // 2], x[..., D // 2:]
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)


def _plain_train(st):
    case = st["case"]
    B, T, H, w = case["B"], case["T"], case["H"], case["w"]
    t = torch.arange(T, device="cuda")
    pos = t + case["pos0"]
    lo = (t - w + 1).clamp_min(0).expand(B, T)
    if st["reset"] is not None:
        lo = torch.maximum(lo, torch.where(st["reset"] != 0, t, 0).cummax(1).values)
    mask = (t[None, None, :] <= t[None, :, None]) & (t[None, None, :] >= lo[:, :, None])       # [B, t, key]
    qr = _rotate(st["q"].double(), pos[:, None]).float().permute(0, 2, 1, 3)                   # [B, H, T, D]
    kr = _rotate(st["k"].double(), pos).float().unsqueeze(1)                                   # [B, 1, T, D]
    v, do = st["v"].float().unsqueeze(1), st["dout"].float().permute(0, 2, 1, 3)
    p = (qr @ kr.transpose(-1, -2)) * SCALE
    p = torch.where(mask.unsqueeze(1), p, -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = p @ v
    ds = do @ v.transpose(-1, -2)
    ds = p * (ds - (do * out).sum(-1, keepdim=True)) * SCALE
    dq = ds @ kr
    dk = (ds.transpose(-1, -2) @ qr).sum(1)
    dv = (p.transpose(-1, -2) @ do).sum(1)
    bf = torch.bfloat16
    return {"out": out.permute(0, 2, 1, 3).to(bf),
            "dq": _rotate(dq.permute(0, 2, 1, 3).double(), pos[:, None], back=True).to(bf),
            "dk": _rotate(dk.double(), pos, back=True).to(bf), "dv": dv.to(bf)}


def _plain_write(st):
    case = st["case"]
    B, T, w = case["B"], case["T"], case["w"]
    t = torch.arange(T, device="cuda")
    n = torch.full((B,), T, device="cuda") if st["lengths"] is None else st["lengths"]
    kc, ks = _quantise64(_rotate(st["k"].double(), t + case["pos0"]))
    vc, vs = _quantise64(st["v"].double())
    keep = (t < n[:, None]) & (t >= n[:, None] - w)
    b, i = keep.nonzero(as_tuple=True)
    slot = (case["pos0"] + i) % w
    codes = st["codes"].view(torch.uint8)
    codes[b, 0, slot], codes[b, 1, slot] = kc.view(torch.uint8)[b, i], vc.view(torch.uint8)[b, i]
    st["scales"][b, 0, slot], st["scales"][b, 1, slot] = ks[b, i], vs[b, i]
    return {"codes": st["codes"], "scales": st["scales"]}


def _plain_decode(st):
    case = st["case"]
    B, w = case["B"], case["w"]
    b, pos = torch.arange(B, device="cuda"), st["pos"].long()
    slot = pos % w
    kc, ks = _quantise64(_rotate(st["k"].double(), pos))
    vc, vs = _quantise64(st["v"].double())
    codes = st["codes"].view(torch.uint8)
    codes[b, 0, slot], codes[b, 1, slot] = kc.view(torch.uint8), vc.view(torch.uint8)
    st["scales"][b, 0, slot], st["scales"][b, 1, slot] = ks, vs
    kv = st["codes"].float() * st["scales"].unsqueeze(-1)                                      # [B, 2, w, D]
    qr = _rotate(st["q"].double(), pos[:, None]).float()
    s = (qr @ kv[:, 0].transpose(-1, -2)) * SCALE
    s = torch.where(torch.arange(w, device="cuda") < (pos + 1)[:, None, None], s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    out = (p @ kv[:, 1]) / p.sum(-1, keepdim=True)
    return {"out": out.to(torch.bfloat16), "codes": st["codes"], "scales": st["scales"]}


def _plain_read(st):
    w = st["case"]["w"]
    n = (st["pos"].long() + 1).clamp_max(w)
    x = (st["codes"].float() * st["scales"].unsqueeze(-1)).to(torch.bfloat16)
    have = (torch.arange(w, device="cuda") < n[:, None])[:, None, :, None]
    st["cache"] = torch.where(have, x, st["cache"])
    return {"cache": st["cache"]}


# ---- the framework's calls --------------------------------------------------------------------------
def _own_train(st):
    from gated_linear_recurrence_conv1d_b200 import binding
    case = st["case"]
    if "save" not in st:                  # a training loop keeps its workspace and its gradients' tensors
        st["dims"] = binding.make_mqa_dims(case["B"], case["T"], case["H"], D, case["w"], SCALE, BASE)
        st["save"] = binding.alloc_workspace(binding.mqa_save_size(st["dims"]))
        st["ws"] = binding.alloc_workspace(binding.mqa_train_workspace_size(st["dims"]))
        st["out"], st["dq"] = torch.empty_like(st["q"]), torch.empty_like(st["q"])
        st["dk"], st["dv"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    binding.mqa_forward(st["dims"], st["q"], st["k"], st["v"], st["out"], st["save"], st["ws"], pos0=case["pos0"],
                        reset=st["reset"])
    binding.mqa_backward(st["dims"], st["v"], st["out"], st["dout"], st["save"], st["dq"], st["dk"], st["dv"], st["ws"])
    return {"out": st["out"], "dq": st["dq"], "dk": st["dk"], "dv": st["dv"]}


def _own_write(st):
    from gated_linear_recurrence_conv1d_b200 import binding
    case = st["case"]
    dims = binding.make_mqa_dims(case["B"], case["T"], 1, D, case["w"], SCALE, BASE)
    binding.mqa_cache8_write(dims, st["k"], st["v"], st["codes"], st["scales"], pos0=case["pos0"], lengths=st["lengths"])
    return {"codes": st["codes"], "scales": st["scales"]}


def _own_decode(st):
    from gated_linear_recurrence_conv1d_b200 import binding
    case = st["case"]
    if "ws" not in st:
        st["dims"] = binding.make_mqa_dims(case["B"], 1, case["H"], D, case["w"], SCALE, BASE)
        st["ws"] = binding.alloc_workspace(binding.mqa_decode8_workspace_size(st["dims"]))
        st["out"] = torch.empty_like(st["q"])
    binding.mqa_decode8(st["dims"], st["q"], st["k"], st["v"], st["pos"], st["codes"], st["scales"], st["out"], st["ws"])
    return {"out": st["out"], "codes": st["codes"], "scales": st["scales"]}


def _own_read(st):
    from gated_linear_recurrence_conv1d_b200 import binding
    case = st["case"]
    dims = binding.make_mqa_dims(case["B"], 1, 1, D, case["w"], SCALE, BASE)
    binding.mqa_cache8_read(dims, st["codes"], st["scales"], st["cache"], pos=st["pos"])
    return {"cache": st["cache"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"train": _own_train, "write": _own_write, "decode": _own_decode, "read": _own_read}[op](state)
    return {"train": _plain_train, "write": _plain_write, "decode": _plain_decode, "read": _plain_read}[op](state)


# ---- 64 bits, from the definition ---------------------------------------------------------------------
def _turn(x, pos):
    """The rotation as a product with e^{i angle} on the pairs (j, j + D/2) taken as complex numbers."""
    z = torch.complex(x[..., : D // 2].contiguous(), x[..., D // 2:].contiguous())
    j = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    ang = pos.double().unsqueeze(-1) * torch.exp(j * (-2.0 * math.log(BASE) / D))
    z = z * torch.polar(torch.ones_like(ang), ang)
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    st = prepare(case, seed)
    op, B = case["op"], case["B"]
    if op == "train":
        T = case["T"]
        lo = torch.from_numpy(np.ascontiguousarray(_first_key(case))).cuda()
        i = torch.arange(T, device="cuda")
        bad = (i[None, None, :] > i[None, :, None]) | (i[None, None, :] < lo[:, :, None])
        q, k, v = (st[n].double().requires_grad_() for n in ("q", "k", "v"))
        qr, kr = _turn(q, i[:, None] + case["pos0"]), _turn(k, i + case["pos0"])
        # one head after another keeps the score matrices small; heads only share k and v
        for h in range(case["H"]):
            s = torch.softmax((torch.bmm(qr[:, :, h], kr.transpose(1, 2)) * SCALE).masked_fill(bad, -math.inf), -1)
            o = torch.bmm(s, v)
            st.setdefault("o", []).append(o.detach())
            o.backward(st["dout"][:, :, h].double(), retain_graph=h + 1 < case["H"])
        return {"out": torch.stack(st["o"], 2), "dq": q.grad, "dk": k.grad, "dv": v.grad}
    if op == "read":
        n = (st["pos"].long() + 1).clamp_max(case["w"])
        x = st["codes"].double() * st["scales"].double()[..., None]
        return {"cache": x * (torch.arange(case["w"], device="cuda") < n[:, None])[:, None, :, None]}
    scales = st["scales"].double()
    if op == "write":
        k, v = _turn(st["k"].double(), torch.arange(case["T"], device="cuda") + case["pos0"]), st["v"].double()
        n = _lengths(case)
        n = [case["T"]] * B if n is None else n.tolist()
        for b in range(B):
            i = torch.arange(max(0, n[b] - case["w"]), n[b], device="cuda")
            slot = (i + case["pos0"]) % case["w"]
            scales[b, 0, slot], scales[b, 1, slot] = k[b, i].abs().amax(-1) / 448, v[b, i].abs().amax(-1) / 448
        return {"codes": None, "scales": scales}
    pos = st["pos"].long()
    q, k, v = _turn(st["q"].double(), pos[:, None]), _turn(st["k"].double(), pos), st["v"].double()
    out = torch.empty(B, case["H"], D, dtype=torch.float64, device="cuda")
    for b in range(B):
        n, slot = min(int(pos[b]) + 1, case["w"]), int(pos[b]) % case["w"]
        ring = st["codes"][b].double() * scales[b].unsqueeze(-1)
        for half, x in ((0, k[b]), (1, v[b])):
            scales[b, half, slot] = x.abs().amax() / 448
            s32 = scales[b, half, slot].float().double()
            ring[half, slot] = (x / s32).float().to(torch.float8_e4m3fn).double() * s32
        out[b] = torch.softmax(q[b] @ ring[0, :n].T * SCALE, -1) @ ring[1, :n]
    return {"out": out, "codes": None, "scales": scales}
