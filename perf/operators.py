"""The operators around the distillation loss, each in a plain form and as a user calls it.

  embed        rows of the (tied) LM-head weight looked up by token id and scaled
  embed_grad   its gradient, added into the fp32 dW the loss writes, or a dW of its own
  act8         an activation checkpoint in 8 bits: written in the forward pass, read back later
  norm         RMS norm with the residual addition in the same pass and an 8-bit checkpoint of
               the sum, and its backward pass, which reads nothing of the forward but that
               checkpoint and one float per row
  weight_grad  the weight gradient dY^T X of a linear layer whose input is kept in 8 bits

An 8-bit checkpoint holds, for every 32 neighbouring columns of a row, one power-of-two
scale 2^e (a byte, e + 127; 255 for a block that held an infinity or a NaN) and 32 codes:
whole numbers up to 127 ("int8") or e4m3 values up to 448 ("e4m3"); e is the smallest
exponent, -126 at least, under which the block's largest magnitude is in range.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 64 sequences: latency
        {"name": "embed_decode_64", "op": "embed", "dtype": "bf16", "T": 64, "d": 2880, "V": 201088,
         "scale": 53.665631, "masked": False},
        # the 32K-token training step, 5% of the positions masked (packed documents)
        {"name": "embed_32k", "op": "embed", "dtype": "bf16", "T": 32768, "d": 2880, "V": 201088,
         "scale": 53.665631, "masked": True},
        # a 4K-token step of an untied model: the whole dW is written
        {"name": "embed_grad_4k", "op": "embed_grad", "dtype": "bf16", "T": 4096, "d": 2048,
         "V": 32000, "scale": 1.0, "masked": False, "accumulate": False},
        # the 32K-token step of a tied model: added into the dW that the loss wrote
        {"name": "embed_grad_32k_tied", "op": "embed_grad", "dtype": "bf16", "T": 32768, "d": 2880,
         "V": 201088, "scale": 53.665631, "masked": True, "accumulate": True},
        # a ragged fp32 activation: a last block of 8 columns, an odd number of rows
        {"name": "act8_ragged_f32", "op": "act8", "dtype": "f32", "T": 257, "d": 136, "fmt": "e4m3"},
        # the hidden states of the 32K-token step
        {"name": "act8_32k", "op": "act8", "dtype": "bf16", "T": 32768, "d": 2880, "fmt": "int8"},
        # the tiny fp32 model: forward and backward of one norm
        {"name": "norm_tiny_f32", "op": "norm", "dtype": "f32", "T": 256, "d": 128, "fmt": "int8",
         "residual": True, "backward": True},
        # one decoding step of 64 sequences: forward only, no checkpoint
        {"name": "norm_decode_64", "op": "norm", "dtype": "bf16", "T": 64, "d": 2880, "fmt": "int8",
         "residual": True, "backward": False},
        # a norm without a residual stream at the 4K-token step
        {"name": "norm_4k_e4m3", "op": "norm", "dtype": "bf16", "T": 4096, "d": 2048, "fmt": "e4m3",
         "residual": False, "backward": True},
        # a layer's norm at the 32K-token step
        {"name": "norm_32k", "op": "norm", "dtype": "bf16", "T": 32768, "d": 2880, "fmt": "int8",
         "residual": True, "backward": True},
        # a square projection at the 4K-token step
        {"name": "weight_grad_4k", "op": "weight_grad", "dtype": "bf16", "T": 4096, "n": 2048,
         "d": 2048, "fmt": "e4m3", "accumulate": False},
        # a projection at the 32K-token step, added to the gradient of earlier micro-batches
        {"name": "weight_grad_32k", "op": "weight_grad", "dtype": "bf16", "T": 32768, "n": 2880,
         "d": 2880, "fmt": "int8", "accumulate": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "act8", "norm", "weight_grad"])
    c = {"op": op, "dtype": "f32" if rng.random() < 0.2 else "bf16"}
    c["T"] = _log_int(rng, 1, 32768)
    c["d"] = 8 * _log_int(rng, 8, 360)
    if op in ("embed", "embed_grad"):
        c.update(V=_log_int(rng, 500, 201088), scale=round(rng.uniform(0.5, 60.0), 3),
                 masked=rng.random() < 0.5)
        if op == "embed_grad":
            c["accumulate"] = rng.random() < 0.5
    else:
        c["fmt"] = rng.choice(["int8", "e4m3"])
    if op == "norm":
        c.update(residual=rng.random() < 0.5, backward=rng.random() < 0.75)
    if op == "weight_grad":
        c.update(n=8 * _log_int(rng, 8, 360), accumulate=rng.random() < 0.5)
        if c["dtype"] == "f32":  # CUDA cores: the small models
            c.update(T=min(c["T"], 2048), n=min(c["n"], 1024), d=min(c["d"], 1024))
    return c


# --------------------------------------------------------------------------- inputs
def _id_weights(V):
    """Probability of a token id's rank: 80% Zipf(1.1), 20% uniform."""
    w = np.arange(1, V + 1, dtype=np.float64) ** -1.1
    return 0.8 * w / w.sum() + 0.2 / V


def _ids(T, V, g):
    p = torch.from_numpy(np.cumsum(_id_weights(V))).to("cuda")
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.searchsorted(p, u).clamp_(max=V - 1)
    return torch.randperm(V, generator=g, device="cuda")[rank].to(torch.int32)


def _mask(case, g):
    if not case.get("masked"):
        return None
    return (torch.rand(case["T"], generator=g, device="cuda") >= 0.05).to(torch.uint8)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _stream(g, T, d, dt):
    """A residual stream: rows of different size, a few channels far larger than the rest."""
    col = torch.exp(0.5 * _randn(g, d))
    col[torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")] *= 20.0
    return (_randn(g, T, d) * torch.exp(0.5 * _randn(g, T, 1)) * col).to(dt)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    T, d, op = case["T"], case["d"], case["op"]
    s = {"case": case}
    if op == "embed":
        s["W"] = (_randn(g, case["V"], d) / math.sqrt(d)).to(dt)
        s["ids"], s["mask"] = _ids(T, case["V"], g), _mask(case, g)
    elif op == "embed_grad":
        s["ids"], s["mask"] = _ids(T, case["V"], g), _mask(case, g)
        s["dX"] = (_randn(g, T, d) * 1e-3).to(dt)
        s["dW"] = _randn(g, case["V"], d) * 1e-2 if case["accumulate"] else \
            torch.empty(case["V"], d, device="cuda")
        s["like"] = torch.empty(1, d, device="cuda", dtype=dt)
    elif op == "act8":
        s["x"] = _stream(g, T, d, dt)
    elif op == "norm":
        s["x"] = _stream(g, T, d, dt)
        s["r"] = _stream(g, T, d, dt) if case["residual"] else None
        s["gain"] = (1.0 + 0.1 * _randn(g, d)).to(dt)
        s["dy"] = (_randn(g, T, d) * 1e-2).to(dt)
        s["dres"] = (_randn(g, T, d) * 1e-2).to(dt) if case["residual"] else None
    else:
        s["q"], s["e"] = _pack(_stream(g, T, d, dt), case["fmt"])
        s["dy"] = (_randn(g, T, case["n"]) * 1e-2).to(dt)
        s["dW"] = _randn(g, case["n"], d) if case["accumulate"] else \
            torch.empty(case["n"], d, device="cuda")
    return s


# --------------------------------------------------------------------------- plain forms
EPS = 1e-5


def _pack(x, fmt):
    """(codes T x d uint8, scale bytes T x ceil(d / 32)) of an activation."""
    T, d = x.shape
    nb = (d + 31) // 32
    f = torch.zeros(T, nb * 32, dtype=torch.float32, device=x.device)
    f[:, :d] = x.float()
    f = f.view(T, nb, 32)
    bits = f.abs().amax(2).view(torch.int32)  # a NaN is the amax of its block
    top, most = (6, 0x7E0000) if fmt == "int8" else (8, 0x600000)  # 127 = 1.984375 * 2^6, 448 = 1.75 * 2^8
    byte = (bits >> 23) - top + ((bits & 0x7FFFFF) > most).int()
    byte = torch.where((bits >> 23) == 255, 255, byte.clamp(min=1))
    inv = ((254 - byte.clamp(max=253)) << 23).view(torch.float32)  # 2^-e
    v = torch.where((byte == 255)[..., None], 0.0, f * inv[..., None])
    q = v.round().to(torch.int8).view(torch.uint8) if fmt == "int8" else \
        v.to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(T, nb * 32)[:, :d].contiguous(), byte.to(torch.uint8)


def _unpack(q, e, fmt):
    """The fp32 values a checkpoint stands for."""
    T, d = q.shape
    v = q.view(torch.int8).float() if fmt == "int8" else q.view(torch.float8_e4m3fn).float()
    k = e.int()
    m = torch.where(k == 255, math.nan, (k << 23).view(torch.float32))
    return v * m.repeat_interleave(32, 1)[:, :d]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "embed":
        out = s["W"][s["ids"].long()].float() * c["scale"]
        if s["mask"] is not None:
            out = torch.where(s["mask"][:, None] != 0, out, 0.0)
        return out.to(s["W"].dtype)
    if op == "embed_grad":
        g = s["dX"].float() * c["scale"]
        if s["mask"] is not None:
            g = torch.where(s["mask"][:, None] != 0, g, 0.0)
        if not c["accumulate"]:
            s["dW"].zero_()
        return s["dW"].index_add_(0, s["ids"].long(), g)
    if op == "act8":
        q, e = _pack(s["x"], c["fmt"])
        return _unpack(q, e, c["fmt"]).to(s["x"].dtype)
    if op == "norm":
        dt = s["x"].dtype
        x = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(dt)
        f, gain = x.float(), s["gain"].float()
        rstd = 1.0 / torch.sqrt(f.square().mean(1, keepdim=True) + EPS)
        y = (f * rstd * gain).to(dt)
        out = {"y": y} if s["r"] is None else {"y": y, "sum": x}
        if c["backward"]:
            h = _unpack(*_pack(x, c["fmt"]), c["fmt"]) * rstd
            dy = s["dy"].float()
            a = dy * gain
            dx = rstd * (a - h * (a * h).mean(1, keepdim=True))
            if s["dres"] is not None:
                dx = dx + s["dres"].float()
            out.update(dx=dx.to(dt), dgain=(dy * h).sum(0))
        return out
    dW = s["dy"].float().t() @ _unpack(s["q"], s["e"], c["fmt"])
    return s["dW"].add_(dW) if c["accumulate"] else dW


# --------------------------------------------------------------------------- the framework's calls
def _own(s):
    from chunked_kl_loss_logits_b200 import ckl

    c = s["case"]
    op = c["op"]
    if op == "embed":
        h = ckl.operator_handle(s["W"], V=c["V"])
        return h.embed(s["ids"], s["W"], mask=s["mask"], scale=c["scale"], sync=False)
    if op == "embed_grad":
        h = ckl.operator_handle(s["like"], V=c["V"])
        return h.embed_grad(s["ids"], s["dX"], mask=s["mask"], scale=c["scale"], dW=s["dW"],
                            accumulate=c["accumulate"], sync=False)
    if op == "act8":
        h = ckl.operator_handle(s["x"])
        return h.act8_unpack(h.act8_pack(s["x"], c["fmt"]))
    if op == "norm":
        h = ckl.operator_handle(s["x"])
        y, x, ckpt = h.norm(s["x"], s["gain"], residual=s["r"], eps=EPS,
                            checkpoint=c["fmt"] if c["backward"] else None)
        out = {"y": y} if s["r"] is None else {"y": y, "sum": x}
        if c["backward"]:
            out["dx"], out["dgain"] = h.norm_bwd(s["dy"], ckpt, s["gain"], d_residual=s["dres"])
        return out
    h = ckl.operator_handle(s["dy"])
    ckpt = ckl.Act8(s["q"], s["e"], c["fmt"])
    if c["accumulate"]:
        return h.act8_weight_grad(s["dy"], ckpt, dW=s["dW"], accumulate=True, sync=False)
    return h.act8_weight_grad(s["dy"], ckpt, sync=False)


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------- work, exact values
def _distinct(T, V):
    """Expected number of different ids among T."""
    return float(-np.expm1(T * np.log1p(-_id_weights(V))).sum()) if V > 1 else 1.0


def work(case):
    T, d, op = case["T"], case["d"], case["op"]
    es = 2 if case["dtype"] == "bf16" else 4
    act, ck = T * d * es, T * d + T * ((d + 31) // 32)
    if op == "embed":
        return {"bytes": 4 * T + _distinct(T, case["V"]) * d * es + act, "flops": T * d}
    if op == "embed_grad":
        rows = 2 * _distinct(T, case["V"]) if case["accumulate"] else case["V"]
        return {"bytes": 4 * T + act + rows * d * 4, "flops": 2 * T * d}
    if op == "act8":
        return {"bytes": 2 * act + 2 * ck, "flops": 4 * T * d}
    if op == "norm":
        n = act * (4 if case["residual"] else 2) + d * es
        if case["backward"]:
            n += 2 * (ck + 4 * T) + act * (3 if case["residual"] else 2) + d * (es + 4)
        return {"bytes": n, "flops": T * d * (16 if case["backward"] else 5)}
    n = case["n"]
    return {"bytes": T * n * es + ck + n * d * 4 * (2 if case["accumulate"] else 1),
            "flops": 2 * T * n * d}


def _levels(x, fmt):
    """The values an activation's checkpoint stands for, in 64 bits, from the definition."""
    T, d = x.shape
    x = x.double()
    out = torch.empty_like(x)
    for b in range(0, d, 32):
        v = x[:, b:b + 32]
        top = v.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(top / (127.0 if fmt == "int8" else 448.0))).clamp(min=-126)
        # the logarithm may be off by one near a power of two: move to the smallest that holds
        lim = 127.0 if fmt == "int8" else 448.0
        e = torch.where(top > lim * torch.exp2(e), e + 1, e)
        e = torch.where((e > -126) & (top <= lim * torch.exp2(e - 1)), e - 1, e)
        u = v / torch.exp2(e)
        if fmt == "int8":
            w = torch.round(u)
        else:  # 3 fraction bits, exponents from -6
            k = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
            step = torch.exp2(k - 3)
            w = torch.round(u / step) * step
        out[:, b:b + 32] = torch.where(torch.isfinite(top), w * torch.exp2(e), math.nan)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "embed":
        keep = torch.ones_like(s["ids"]) if s["mask"] is None else (s["mask"] != 0)
        rows = torch.index_select(s["W"], 0, s["ids"].long()).double()
        return rows * (keep.double() * np.float64(np.float32(case["scale"])))[:, None]
    if op == "embed_grad":
        keep = torch.ones_like(s["ids"]) if s["mask"] is None else (s["mask"] != 0)
        order = torch.argsort(s["ids"].long(), stable=True)
        ids, count = torch.unique_consecutive(s["ids"].long()[order], return_counts=True)
        end = torch.cumsum(count, 0)
        out = s["dW"].double() if case["accumulate"] else \
            torch.zeros(case["V"], d, device="cuda", dtype=torch.float64)
        for c0 in range(0, d, 256):
            v = s["dX"][order, c0:c0 + 256].double() * keep[order].double()[:, None]
            run_sum = torch.cumsum(v, 0)[end - 1]
            run_sum[1:] = run_sum[1:] - run_sum[:-1].clone()
            out[ids, c0:c0 + 256] += run_sum * np.float64(np.float32(case["scale"]))
        return out
    if op == "act8":
        return _levels(s["x"], case["fmt"])
    if op == "norm":
        x = s["x"].double() + (0.0 if s["r"] is None else s["r"].double())
        kept = x.to(s["x"].dtype).double()  # the sum as it is kept
        ms = (kept * kept).sum(1, keepdim=True) / d + EPS
        gain = s["gain"].double()
        out = {"y": kept / ms.sqrt() * gain}
        if s["r"] is not None:
            out["sum"] = x
        if case["backward"]:
            lv, dy = _levels(kept, case["fmt"]), s["dy"].double()
            dot = (dy * gain * lv).sum(1, keepdim=True)
            dx = dy * gain / ms.sqrt() - lv * dot / (d * ms * ms.sqrt())
            out["dx"] = dx if s["dres"] is None else dx + s["dres"].double()
            out["dgain"] = (dy * lv / ms.sqrt()).sum(0)
        return out
    v = s["q"].view(torch.int8).double() if case["fmt"] == "int8" else \
        s["q"].view(torch.float8_e4m3fn).double()
    block = torch.arange(d, device="cuda") // 32
    v = v * torch.exp2(s["e"].double() - 127.0)[:, block]
    dW = torch.einsum("tn,td->nd", s["dy"].double(), v)
    return dW + s["dW"].double() if case["accumulate"] else dW
