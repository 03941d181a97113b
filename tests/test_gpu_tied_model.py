"""The operators together as a training step uses them: a tied model's embedding, a norm that
keeps its input in 8 bits, and the distillation loss; and a linear layer's weight gradient from
the checkpoint of its input.
"""
import numpy as np
import pytest
import torch

import oracle
from chunked_kl_loss_logits_b200 import ckl
from chunked_kl_loss_logits_b200.workloads import small_case
from oracle import ops_oracle as O
from tests._helpers import TOL, f64, rel, upload

pytestmark = pytest.mark.gpu
SCALE, EPS = 2.0, 1e-3


def inputs(dt, T=300, d=64, V=1000, K=16):
    x = small_case(T, d, V, K, seed=5, dtype="f32" if dt == torch.float32 else "bf16",
                   teacher_var=3.0, ids="zipf", packing=True)
    _, W, idx, logit, mask = upload(x, dt)
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    gain = (1 + 0.1 * torch.randn(d, generator=g)).to(dt).cuda()
    return W, ids, gain, idx, logit, mask


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_a_tied_step_is_its_calls(dt):
    """Autograd against the calls made one by one on handles: the same bits where autograd adds
    nothing of its own, and the embedding's gradient added into the loss's dW."""
    W, ids, gain, idx, logit, mask = inputs(dt)
    V, d = W.shape
    h = ckl.ChunkedKL(V, d, idx.shape[1], dtype=dt, max_chunk=128)
    E = h.embed(ids, W, scale=SCALE)
    H, _, ckpt = h.norm(E, gain, eps=EPS)
    loss, dH, dW = h.fwd_bwd(H, W, idx, logit, mask, chunk=128)
    dE, dg = h.norm_bwd(dH, ckpt, gain)
    head = dW.clone()
    h.embed_grad(ids, dE, scale=SCALE, dW=dW, accumulate=True)
    own = h.embed_grad(ids, dE, scale=SCALE)
    assert torch.equal(dW, head + own)

    Wp, gp = W.clone().requires_grad_(), gain.clone().requires_grad_()
    out = ckl.chunked_kl_loss(ckl.rms_norm(ckl.embedding(ids, Wp, scale=SCALE), gp, eps=EPS), Wp,
                              idx, logit, mask, chunk=128, handle=h)
    out.backward()
    assert torch.equal(out.detach(), loss) and torch.equal(gp.grad, dg.to(dt))
    # autograd rounds the two shares to W's type before it adds them, and the sum: three half steps
    if dt == torch.float32:
        assert torch.equal(Wp.grad, head + own)
    else:
        err = (Wp.grad.double() - (head.double() + own.double())).abs()
        assert bool((err <= 2.0 ** -8 * 2.02 * (head.abs() + own.abs()).double()).all())
    h.close()


def test_a_tied_step_against_the_formulas():
    """fp32, against 64 bits without checkpoints. A checkpoint's element is off by delta, at most half
    a step (2^(e-1)) of its block, which moves dE by at most
        r (|delta r| mean|a h| + |h + delta r| mean(|a| |delta r|))
    and the gradient of W by the sum of that over a row's tokens; the rest is the loss's own
    fp32 tolerance (1e-4 of the norm), once for each of the two shares."""
    W, ids, gain, idx, logit, mask = inputs(torch.float32)
    W.requires_grad_()
    gain.requires_grad_()
    loss = ckl.chunked_kl_loss(ckl.rms_norm(ckl.embedding(ids, W, scale=SCALE), gain, eps=EPS), W,
                               idx, logit, mask, chunk=128)
    loss.backward()

    i, keep = ids.cpu().numpy(), mask.cpu().numpy()
    E = O.embed(i, f64(W), None, SCALE)
    H, rstd = O.norm(E, f64(gain), EPS)
    r = oracle.fwd_bwd(H, f64(W), idx.cpu().numpy(), logit.cpu().numpy(), keep)
    dE, dg, _, _ = O.norm_bwd(r["dH"], E, rstd, f64(gain))
    own, _ = O.embed_grad(i, dE, W.shape[0], None, SCALE)
    want = r["dW"] + own
    byte = O.act8_pack(E.astype(np.float32), "int8")[1]
    delta = np.repeat(2.0 ** (byte.astype(np.float64) - 128), 32, axis=1) * rstd[:, None]
    a, hh = np.abs(r["dH"] * f64(gain)), np.abs(E * rstd[:, None])
    moved = rstd[:, None] * (delta * (a * hh).mean(1, keepdims=True) +
                             (hh + delta) * (a * delta).mean(1, keepdims=True))
    room, _ = O.embed_grad(i, moved, W.shape[0], None, SCALE)
    tol = TOL["f32"]
    assert rel(loss.item(), r["loss"]) <= tol["loss"]
    err = np.linalg.norm(f64(W.grad) - want)
    assert err <= np.linalg.norm(room) + tol["grad"] * (np.linalg.norm(r["dW"]) + np.linalg.norm(own))
    g_room = np.linalg.norm((np.abs(r["dH"]) * delta).sum(0))
    assert np.linalg.norm(f64(gain.grad) - dg) <= g_room + tol["grad"] * np.linalg.norm(dg)
    print(f"W.grad off {err / np.linalg.norm(want):.1e}, room {np.linalg.norm(room) / np.linalg.norm(want):.1e}")


class Linear8(torch.autograd.Function):
    """y W^T with y kept in 8 bits for the weight gradient: what a user's layer looks like."""

    @staticmethod
    def forward(ctx, y, W):
        ctx.h = ckl.operator_handle(y)
        ctx.ckpt = ctx.h.act8_pack(y.detach(), "e4m3")
        ctx.save_for_backward(W)
        return y @ W.t()

    @staticmethod
    def backward(ctx, dZ):
        (W,) = ctx.saved_tensors
        dW = ctx.h.act8_weight_grad(dZ.contiguous(), ctx.ckpt, sync=False)
        return dZ @ W, dW.to(W.dtype)


def test_a_block_with_a_residual_stream():
    """Two residual blocks of norm and linear layer on the embedding, the final norm and the loss:
    the gradients are those of the same blocks with each layer's call made by hand."""
    W, ids, gain, idx, logit, mask = inputs(torch.bfloat16)
    T, d = ids.numel(), W.shape[1]
    g = torch.Generator().manual_seed(3)
    L = [(torch.randn(d, d, generator=g) / 8).bfloat16().cuda().requires_grad_() for _ in range(2)]
    G = [gain.clone().requires_grad_() for _ in range(3)]
    Wp = W.clone().requires_grad_()
    s = ckl.embedding(ids, Wp, scale=SCALE)
    z = torch.zeros_like(s)
    for k in range(2):
        y, s = ckl.rms_norm(z, G[k], residual=s)
        z = Linear8.apply(y, L[k])
    H, s = ckl.rms_norm(z, G[2], residual=s)
    loss = ckl.chunked_kl_loss(H, Wp, idx, logit, mask, chunk=128)
    loss.backward()

    h = ckl.operator_handle(W, V=W.shape[0])
    s0 = h.embed(ids, W, scale=SCALE)
    kept, z0 = [], torch.zeros_like(s0)
    for k in range(3):
        y0, s0, c = h.norm(z0, G[k].detach(), residual=s0)
        if k < 2:
            kept.append((c, h.act8_pack(y0, "e4m3")))
            z0 = y0 @ L[k].detach().t()
    loss0, dH, dW = ckl.handle_for(W, idx.shape[1], 128).fwd_bwd(y0, W, idx, logit, mask, chunk=128)
    ds, dg = h.norm_bwd(dH, c, G[2].detach())
    assert torch.equal(loss0, loss.detach()) and torch.equal(G[2].grad, dg.bfloat16())
    for k in (1, 0):
        assert torch.equal(L[k].grad, h.act8_weight_grad(ds, kept[k][1]).bfloat16())
        ds, dg = h.norm_bwd(ds @ L[k].detach(), kept[k][0], G[k].detach(), d_residual=ds)
        assert torch.equal(G[k].grad, dg.bfloat16())
    own = h.embed_grad(ids, ds, scale=SCALE)
    err = (Wp.grad.double() - (dW.double() + own.double())).abs()
    assert bool((err <= 2.0 ** -8 * 2.02 * (dW.abs() + own.abs()).double()).all())
    assert torch.isfinite(Wp.grad.float()).all()
