"""8-bit activation checkpoints and the RMS norm that keeps one, against the fp64 oracle.

Codes and scales are whole numbers with one right answer (scaling by a power of two is exact)
and have to be equal. Bounds of the norm, with u = 2^-24: the mean of d squares is off by at
most (d + 1) u relative (d - 1 additions in some order, a square each, a division), its
reciprocal root by half that plus 3 u (the addition of eps, the root, the reciprocal), so rstd by
(d / 2 + 4) u, and y adds two products and the rounding to its type (half a step, eps / 2). In the
backward pass the mean of a h takes d + 4 roundings and rstd's own error once more for every
factor of it: dX is off by at most (2 d + 24) u of the magnitudes that enter it, plus half a step
of the result; dgain by (T + d / 2 + 12) u of them. (1.01: the higher orders.)
"""
import numpy as np
import pytest
import torch

from chunked_kl_loss_logits_b200 import ckl
from oracle import ops_oracle as O
from tests._helpers import f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# one vector of 8 columns; ragged last blocks; every count of warps and vectors a row takes
WIDTHS = [8, 24, 40, 136, 264, 520, 1032, 2048, 2880, 4104, 8192, 12000, 24000]


def rows(T, d, dt, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + d)
    x = torch.randn(T, d, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))
    x[:, ::61] *= 30
    return x.to(DT[dt]).cuda()


def check_pack(x, ckpt, fmt):
    q, e = O.act8_pack(f64(x), fmt)
    assert np.array_equal(ckpt.scale.cpu().numpy(), e)
    assert np.array_equal(ckpt.q.cpu().numpy() & 0x7F if fmt == "e4m3" else ckpt.q.cpu().numpy(),
                          q & 0x7F if fmt == "e4m3" else q)  # e4m3: the sign of zero is free
    v = O.act8_values(ckpt.q.cpu().numpy(), e, fmt)
    assert np.array_equal(v, O.act8_values(q, e, fmt), equal_nan=True)
    return v


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("T,cols", [(1, 8), (5, 24), (33, 40), (7, 264), (9, 1032), (3, 2880),
                                    (2, 70000)])
def test_pack_and_unpack(T, cols, fmt, dt):
    x = rows(T, cols, dt)
    x[0, :8] = 0
    h = ckl.operator_handle(rows(1, 8, dt))  # its d does not matter to these
    ckpt = h.act8_pack(x, fmt)
    v = check_pack(x, ckpt, fmt)
    assert np.array_equal(f64(h.act8_unpack(ckpt)), v)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_pack_extreme_values(fmt, dt):
    """Every power of two with fractions about the largest code's, zeros, subnormals, the
    largest finite values, infinities and NaN."""
    e = torch.arange(-126, 128).float()[:, None]
    f = torch.tensor([1.0, 1.75, 1.7578125, 1.984375, 1.9921875, -1.0, -1.984375, 0.0])
    x = torch.zeros(254 + 8, 32)
    x[:254, 5:13] = torch.exp2(e) * f * torch.tensor([1, .5, .5, .25, .25, 1, 1, 1])
    x[:254, 5] = torch.exp2(e[:, 0]) * torch.tensor([1.0, 1.75, 1.7578125, 1.984375, 1.9921875])[
        torch.arange(254) % 5]
    x[254, 3], x[255, 3], x[256, 3] = 3e38, 1e-40, float("nan")
    x[257, 31], x[258, 0] = float("inf"), float("-inf")
    x[259] = 3.3895e38
    x[260] = 2.0 ** -126
    x = x.to(DT[dt]).cuda()
    h = ckl.operator_handle(x)
    ckpt = h.act8_pack(x, fmt)
    v = check_pack(x, ckpt, fmt)
    assert np.isnan(v[256:259]).all() and np.isfinite(v[:256]).all()
    got = f64(h.act8_unpack(ckpt))
    # a value below the type's smallest normal number is rounded to its subnormal step
    tiny = 2.0 ** -133 / 2 if dt == "bf16" else 2.0 ** -149 / 2
    near = np.abs(got - v) <= np.where(np.abs(v) < 2.0 ** -126, tiny, 0.0)
    assert np.all(near | (np.isnan(got) & np.isnan(v)))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_unpack_reads_every_code_and_scale(fmt):
    q = torch.arange(256, dtype=torch.uint8).repeat(255, 1).cuda()
    e = torch.arange(1, 256, dtype=torch.uint8)[:, None].repeat(1, 8).cuda()
    h = ckl.operator_handle(torch.zeros(1, 8, device="cuda"))
    got = f64(h.act8_unpack(ckl.Act8(q, e, fmt)))
    want = O.act8_values(q.cpu().numpy(), e.cpu().numpy(), fmt)
    with np.errstate(over="ignore"):
        assert np.array_equal(got, want.astype(np.float32).astype(np.float64), equal_nan=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_forward_and_backward(d, dt, residual):
    if dt == "f32" and d > 12800:
        pytest.skip("no fp32 handle has rows this wide")
    for T, fmt in ((1, "int8"), (3, "e4m3"), (37, "int8")):
        x, r = rows(T, d, dt), rows(T, d, dt, 1) if residual else None
        gain = (1 + 0.2 * torch.randn(d, device="cuda")).to(DT[dt])
        h = ckl.operator_handle(x)
        half = torch.finfo(DT[dt]).eps / 2
        eps = 1e-3
        y, s, ckpt = h.norm(x, gain, residual=r, eps=eps, checkpoint=fmt)
        if residual:
            sum64 = f64(x) + f64(r)
            assert np.all(np.abs(f64(s) - sum64) <= (half + 1.01 * U) * np.abs(sum64))
        else:
            assert s is x
        want, rstd = O.norm(f64(s), f64(gain), eps)
        assert np.all(np.abs(f64(ckpt.rstd) - rstd) <= 1.01 * (d / 2 + 4) * U * rstd)
        assert np.all(np.abs(f64(y) - want) <= (half + 1.01 * (d / 2 + 6) * U) * np.abs(want))
        kept = check_pack(s, ckpt, fmt)
        assert torch.equal(h.norm(x, gain, residual=r, eps=eps, checkpoint=None)[0], y)

        dY, dS = rows(T, d, dt, 2), rows(T, d, dt, 3) if residual else None
        base = torch.randn(d, device="cuda")
        dX, dg = h.norm_bwd(dY, ckpt, gain, d_residual=dS, dgain=base.clone(), accumulate=True)
        wX, wg, magX, magG = O.norm_bwd(f64(dY), kept, rstd, f64(gain),
                                        None if dS is None else f64(dS))
        assert np.all(np.abs(f64(dX) - wX) <= half * np.abs(wX) + 1.01 * (2 * d + 24) * U * magX)
        wg = wg + f64(base)
        magG = magG + np.abs(f64(base))
        assert np.all(np.abs(f64(dg) - wg) <= 1.01 * (T + d / 2 + 12) * U * magG)
        dX2, dg2 = h.norm_bwd(dY, ckpt, gain, d_residual=dS)
        assert torch.equal(dX2, dX)
        assert np.all(np.abs(f64(dg2) - (wg - f64(base))) <= 1.01 * (T + d / 2 + 12) * U * magG)


@pytest.mark.parametrize("T,d", [(5000, 64), (3001, 520), (1203, 2880)])
def test_norm_backward_over_many_rows(T, d):
    """Blocks walk several rows and dgain's partial sums come from all of them."""
    x, dY, dS = rows(T, d, "bf16"), rows(T, d, "bf16", 2), rows(T, d, "bf16", 3)
    gain = (1 + 0.2 * torch.randn(d, device="cuda")).to(torch.bfloat16)
    h = ckl.operator_handle(x)
    _, s, ckpt = h.norm(x, gain)
    kept = O.act8_values(ckpt.q.cpu().numpy(), ckpt.scale.cpu().numpy(), "int8")
    rstd = O.norm(f64(s), f64(gain), 1e-5)[1]
    runs = [h.norm_bwd(dY, ckpt, gain, d_residual=dS) for _ in range(2)]
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    wX, wg, magX, magG = O.norm_bwd(f64(dY), kept, rstd, f64(gain), f64(dS))
    dX, dg = runs[0]
    assert np.all(np.abs(f64(dX) - wX) <= 2.0 ** -8 * np.abs(wX) + 1.01 * (2 * d + 24) * U * magX)
    assert np.all(np.abs(f64(dg) - wg) <= 1.01 * (T + d / 2 + 12) * U * magG)


def test_norm_gradient_against_differences():
    """fp32, inputs that the checkpoint holds exactly (int8 codes times a power of two), so the
    gradient is the forward pass's own: central differences in 64 bits along a direction."""
    T, d, eps = 20, 64, 1e-2
    g = torch.Generator().manual_seed(3)
    x = (torch.randint(-127, 128, (T, d), generator=g).float() / 64).cuda()
    x[:, ::32] = 127 / 64  # every block at the same scale
    gain, dY = torch.rand(d, generator=g).cuda() + 0.5, torch.randn(T, d, generator=g).cuda()
    h = ckl.operator_handle(x)
    _, _, ckpt = h.norm(x, gain, eps=eps)
    assert torch.equal(h.act8_unpack(ckpt), x)
    dX, _ = h.norm_bwd(dY, ckpt, gain)
    u = np.random.default_rng(0).normal(size=(T, d))
    f = lambda t: (O.norm(f64(x) + t * u, f64(gain), eps)[0] * f64(dY)).sum()
    want = (f(1e-5) - f(-1e-5)) / 2e-5
    # the difference quotient: 2e-16 * |f| / 1e-5 and the third derivative times 1e-10
    assert abs((f64(dX) * u).sum() - want) <= 1e-5 * np.abs(f64(dX) * u).sum() + 1e-7


def test_norm_in_place_and_given_buffers():
    T, d = 50, 264
    x, r = rows(T, d, "bf16"), rows(T, d, "bf16", 1)
    gain = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    h = ckl.operator_handle(x)
    y, s, c = h.norm(x, gain, residual=r)
    x2, r2 = x.clone(), r.clone()
    c2 = h.act8_empty(T, d, "int8", rstd=True)
    y2, s2, c3 = h.norm(x2, gain, residual=r2, out=(x2, r2, c2))  # y over x, s over r
    assert y2 is x2 and s2 is r2 and c3 is c2
    assert torch.equal(x2, y) and torch.equal(r2, s)
    assert torch.equal(c2.q, c.q) and torch.equal(c2.scale, c.scale) and torch.equal(c2.rstd, c.rstd)
    dY, dS = rows(T, d, "bf16", 2), rows(T, d, "bf16", 3)
    dX, dg = h.norm_bwd(dY, c, gain, d_residual=dS)
    for into in (0, 1):
        a, b = dY.clone(), dS.clone()
        got, dg2 = h.norm_bwd(a, c, gain, d_residual=b, dX=(a, b)[into])
        assert torch.equal(got, dX) and torch.equal(dg2, dg)


def test_rows_with_zeros_infinities_and_nan():
    T, d = 12, 72
    x = rows(T, d, "bf16")
    x[3] = 0
    x[5, 40], x[7, 3] = float("nan"), float("inf")
    gain = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    h = ckl.operator_handle(x)
    y, _, ckpt = h.norm(x, gain)
    dX, dg = h.norm_bwd(torch.ones_like(x), ckpt, gain)
    ok = torch.ones(T, dtype=torch.bool)
    ok[[5, 7]] = False
    assert torch.all(y[3] == 0) and torch.isfinite(y[ok]).all() and torch.isfinite(dX[ok]).all()
    assert torch.isnan(y[5]).all() and torch.isnan(dX[5]).all()
    assert torch.isnan(dX[7]).all()  # the checkpoint of an infinity reads back as NaN
    clean = h.norm(x[ok.cuda()].contiguous(), gain)
    assert torch.equal(clean[0], y[ok.cuda()])


def test_no_rows():
    d = 64
    x = torch.empty(0, d, device="cuda")
    gain = torch.ones(d, device="cuda")
    h = ckl.operator_handle(x)
    y, s, ckpt = h.norm(x, gain, residual=x.clone())
    assert y.shape == (0, d) and ckpt.q.shape == (0, d)
    dX, dg = h.norm_bwd(y, ckpt, gain)
    assert dX.shape == (0, d) and torch.all(dg == 0)
    base = torch.randn(d, device="cuda")
    assert torch.equal(h.norm_bwd(y, ckpt, gain, dgain=base.clone(), accumulate=True)[1], base)
    assert h.act8_unpack(h.act8_pack(x)).shape == (0, d)


def test_many_rows_pass_32_bit_offsets():
    T, d = 760000, 2880  # 2.19e9 elements
    x = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16)
    x[-3:] = rows(3, d, "bf16")
    gain = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    h = ckl.operator_handle(x)
    y, _, ckpt = h.norm(x, gain)
    few_y, _, few = h.norm(x[-3:].contiguous(), gain)
    assert torch.equal(y[-3:], few_y) and torch.equal(ckpt.q[-3:], few.q)
    assert torch.equal(ckpt.scale[-3:], few.scale) and torch.all(y[:-3:1000] == 0)
    dX, _ = h.norm_bwd(x, ckpt, gain, dX=y)
    assert torch.equal(dX[-3:], h.norm_bwd(x[-3:].contiguous(), few, gain)[0])
    again = h.act8_pack(x, out=ckpt)
    assert torch.equal(again.q[-3:], few.q)
    assert torch.equal(h.act8_unpack(ckpt, out=y)[-3:], h.act8_unpack(few))


def test_calls_captured_in_a_graph():
    T, d = 300, 520
    x, r, dY = rows(T, d, "bf16"), rows(T, d, "bf16", 1), rows(T, d, "bf16", 2)
    gain = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    h = ckl.operator_handle(x)
    out = (torch.empty_like(x), torch.empty_like(x), h.act8_empty(T, d, "e4m3", rstd=True))
    dX, dg = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = h.norm_bwd_workspace(T)

    def call():
        h.norm(x, gain, residual=r, checkpoint="e4m3", out=out)
        h.norm_bwd(dY, out[2], gain, dX=dX, dgain=dg, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (5, 6):
        x.copy_(rows(T, d, "bf16", seed))
        g.replay()
        torch.cuda.synchronize()
        y, sm, c = h.norm(x, gain, residual=r, checkpoint="e4m3")
        assert torch.equal(out[0], y) and torch.equal(out[1], sm) and torch.equal(out[2].q, c.q)
        wX, wg = h.norm_bwd(dY, c, gain)
        assert torch.equal(dX, wX) and torch.equal(dg, wg)


def test_two_calls_in_flight_on_two_streams():
    xs = [rows(2000, 520, "bf16", k) for k in (0, 1)]
    gain = torch.ones(520, device="cuda", dtype=torch.bfloat16)
    hs = [ckl.ChunkedKL(1, 520, 1, max_chunk=1) for _ in xs]
    alone = [h.norm_bwd(x, h.norm(x, gain)[2], gain) for h, x in zip(hs, xs)]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        both = []
        for h, x, s in zip(hs, xs, ss):
            with torch.cuda.stream(s):
                both.append(h.norm_bwd(x, h.norm(x, gain)[2], gain))
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    [h.close() for h in hs]


@pytest.mark.parametrize("residual", [False, True])
def test_autograd_rms_norm(residual):
    T, d = 24, 136
    x, r = rows(T, d, "f32").requires_grad_(), rows(T, d, "f32", 1).requires_grad_()
    gain = (1 + 0.1 * torch.randn(d, device="cuda")).requires_grad_()
    dY, dS = rows(T, d, "f32", 2), rows(T, d, "f32", 3)
    h = ckl.operator_handle(x)
    shape = (4, 6, d)
    if residual:
        y, s = ckl.rms_norm(x.view(shape), gain, residual=r.view(shape), eps=1e-3)
        torch.autograd.backward((y, s), (dY.view(shape), dS.view(shape)))
    else:
        y = ckl.rms_norm(x.view(shape), gain, eps=1e-3)
        y.backward(dY.view(shape))
    y0, s0, c = h.norm(x.detach(), gain.detach(), residual=r.detach() if residual else None, eps=1e-3)
    dX, dg = h.norm_bwd(dY, c, gain.detach(), d_residual=dS if residual else None)
    assert torch.equal(y.view(T, d), y0) and torch.equal(x.grad, dX) and torch.equal(gain.grad, dg)
    if residual:
        assert torch.equal(s.view(T, d), s0) and torch.equal(r.grad, dX)
        x.grad = r.grad = gain.grad = None
        ckl.rms_norm(x, gain, residual=r)[1].sum().backward()  # only the sum is used
        assert torch.all(x.grad == 1) and torch.all(r.grad == 1) and gain.grad is None


def test_saved_tensors_may_come_back_elsewhere():
    """What autograd saved goes to the host and back to another address."""
    x = rows(40, 136, "bf16")
    gain = torch.ones(136, device="cuda", dtype=torch.bfloat16)
    dY = rows(40, 136, "bf16", 2)
    grads = []
    for hooks in (False, True):
        xp, gp = x.clone().requires_grad_(), gain.clone().requires_grad_()
        if hooks:
            with torch.autograd.graph.save_on_cpu():
                y = ckl.rms_norm(xp, gp)
        else:
            y = ckl.rms_norm(xp, gp)
        held = [torch.full((40 * 200,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
        y.backward(dY)
        del held
        grads.append((xp.grad, gp.grad))
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])


def test_calls_on_a_given_stream_and_from_threads():
    import threading
    x = rows(500, 520, "bf16")
    gain = torch.ones(520, device="cuda", dtype=torch.bfloat16)
    h = ckl.operator_handle(x)
    y, _, c = h.norm(x, gain)
    dX, dg = h.norm_bwd(x, c, gain)
    p = h.act8_unpack(h.act8_pack(x, "e4m3"))
    dW = h.act8_weight_grad(x, c)
    torch.cuda.synchronize()
    got, errs = {}, []

    def work(k):
        try:
            h = ckl.operator_handle(x)  # each thread has its own
            s = torch.cuda.Stream()
            for _ in range(20):
                y, _, c = h.norm(x, gain, stream=s)
                got[k] = (h, y, *h.norm_bwd(x, c, gain, stream=s),
                          h.act8_unpack(h.act8_pack(x, "e4m3", stream=s), stream=s),
                          h.act8_weight_grad(x, c, stream=s))
            s.synchronize()
        except Exception as e:
            errs.append(e)

    th = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    [t.start() for t in th]
    [t.join(120) for t in th]
    assert not errs, errs
    assert len({id(g[0]) for g in got.values()} | {id(h)}) == 4
    for g in got.values():
        for a, b in zip(g[1:], (y, dX, dg, p, dW)):
            assert torch.equal(a, b)


def test_a_closed_handle_is_refused():
    h = ckl.ChunkedKL(1, 64, 1, max_chunk=1)
    h.close()
    with pytest.raises(ckl.CKLError) as e:
        h.act8_pack(rows(3, 64, "bf16"))
    assert e.value.code == 1


def test_refusals():
    x = rows(10, 64, "bf16")
    gain = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    h = ckl.operator_handle(x)
    y, s, ckpt = h.norm(x, gain)
    for bad in (lambda: h.norm(x.float(), gain), lambda: h.norm(x, gain.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: h.norm(x[:, :32].contiguous(), gain), lambda: h.norm(x, gain[:32]),
                lambda: h.norm(x, gain, residual=x[:5]), lambda: h.norm(x, gain, checkpoint="fp8"),
                lambda: h.norm(x.t().contiguous().t(), gain), lambda: h.norm(x.cpu(), gain),
                lambda: h.norm_bwd(x[:5], ckpt, gain),
                lambda: h.norm_bwd(x, h.act8_pack(x), gain),  # no rstd
                lambda: h.norm_bwd(x, ckpt, gain, accumulate=True),
                lambda: h.act8_pack(x, out=ckl.Act8(ckpt.q[:5], ckpt.scale[:5])),
                lambda: h.norm(x, gain, out=(y, s, None)),
                lambda: h.norm_bwd(x, ckl.Act8(torch.zeros(10, 32, dtype=torch.uint8, device="cuda"),
                                               ckpt.scale[:, :1].contiguous(), rstd=ckpt.rstd), gain)):
        with pytest.raises(ValueError):
            bad()
    codes = []
    for bad in (lambda: h.norm(x, gain, eps=0.0), lambda: h.norm(x, gain, eps=float("nan")),
                lambda: h.norm(x, gain, residual=x, out=(y, y, ckpt)),
                lambda: h.act8_pack(torch.zeros(4, 12, device="cuda", dtype=torch.bfloat16)),
                lambda: h.norm_bwd(x, ckpt, gain, workspace=torch.empty(
                    256, dtype=torch.uint8, device="cuda")),
                lambda: h.act8_pack(torch.zeros(65, device="cuda", dtype=torch.bfloat16)[1:].view(1, 64))):
        with pytest.raises(ckl.CKLError) as e:
            bad()
        codes.append(e.value.code)
    assert codes == [1, 1, 1, 2, 3, 7]


def test_a_cached_handle_that_was_closed_is_replaced():
    x = torch.randn(4, 72, device="cuda")
    g = torch.ones(72, device="cuda")
    want = ckl.rms_norm(x, g)
    h = ckl.operator_handle(x)
    h.close()
    with pytest.raises(ckl.CKLError):
        h.norm(x, g)
    assert torch.equal(ckl.rms_norm(x, g), want)


@pytest.mark.parametrize("dt,d", [("f32", 40), ("f32", 136), ("f32", 520), ("f32", 2880), ("f32", 4104),
                                  ("f32", 8192), ("f32", 12000), ("bf16", 40), ("bf16", 1032),
                                  ("bf16", 4104), ("bf16", 8192), ("bf16", 12000), ("bf16", 24000)])
@pytest.mark.parametrize("residual", [False, True])
def test_blocks_that_walk_several_rows(dt, d, residual):
    """Every count of vectors a lane and of rows ahead, refilled several times: against the formulas
    in 64 bits, against the same rows in a call of their own (a row a block), and in place."""
    T = 8003 if d <= 136 else 4001 if d <= 1032 else 1203
    x, dY = rows(T, d, dt), rows(T, d, dt, 2)
    r, dS = (rows(T, d, dt, 1), rows(T, d, dt, 3)) if residual else (None, None)
    gain = (1 + 0.2 * torch.randn(d, device="cuda")).to(DT[dt])
    h, eps, half = ckl.operator_handle(x), 1e-3, torch.finfo(DT[dt]).eps / 2
    y, s, c = h.norm(x, gain, residual=r, eps=eps)
    dX, dg = h.norm_bwd(dY, c, gain, d_residual=dS)

    s64, g64, dY64 = s.double(), gain.double(), dY.double()
    rstd = 1 / (s64.square().mean(1, keepdim=True) + float(np.float32(eps))).sqrt()
    want = s64 * rstd * g64
    assert bool(((y.double() - want).abs() <= (half + 1.01 * (d / 2 + 6) * U) * want.abs()).all())
    kept = ckl.operator_handle(torch.empty(1, 8, device="cuda")).act8_unpack(c).double()
    hat, a = kept * rstd, dY64 * g64
    p = 0.0 if dS is None else dS.double()
    wX = rstd * (a - hat * (a * hat).mean(1, keepdim=True)) + p
    mag = rstd * (a.abs() + hat.abs() * (a * hat).abs().mean(1, keepdim=True)) + abs(p)
    assert bool(((dX.double() - wX).abs() <= half * wX.abs() + 1.01 * (2 * d + 24) * U * mag).all())
    wg, magG = (dY64 * hat).sum(0), (dY64 * hat).abs().sum(0)
    assert bool(((dg.double() - wg).abs() <= 1.01 * (T + d / 2 + 12) * U * magG).all())

    few = torch.tensor([0, 1, 700, T // 2, T - 2, T - 1], device="cuda")
    at = lambda t: None if t is None else t[few].contiguous()
    y1, s1, c1 = h.norm(at(x), gain, residual=at(r), eps=eps)
    assert torch.equal(y[few], y1) and torch.equal(s[few], s1) and torch.equal(c.rstd[few], c1.rstd)
    assert torch.equal(c.q[few], c1.q) and torch.equal(c.scale[few], c1.scale)
    assert torch.equal(dX[few], h.norm_bwd(at(dY), c1, gain, d_residual=at(dS))[0])

    x2, r2, c2 = x.clone(), None if r is None else r.clone(), h.act8_empty(T, d, rstd=True)
    h.norm(x2, gain, residual=r2, eps=eps, out=(x2, r2, c2))
    assert torch.equal(x2, y) and (r is None or torch.equal(r2, s)) and torch.equal(c2.q, c.q)
    dY2 = dY.clone()
    _, dg2 = h.norm_bwd(dY2, c2, gain, d_residual=dS, dX=dY2)
    assert torch.equal(dY2, dX) and torch.equal(dg2, dg)
