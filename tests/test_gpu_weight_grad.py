"""The weight gradient of a linear layer whose input is kept as an 8-bit checkpoint.

The products are exact (8 bits times 8 bits, or three such parts of an fp32 dY), so an element
is off only by the fp32 sums of its T terms (3 T for fp32): each addition, of whatever order and
cut or rounded, is off by at most one step, 2^-23 of the magnitudes summed so far; a few more for
the partial results of token ranges and what was there before.
"""
import ctypes

import numpy as np
import pytest
import torch

from chunked_kl_loss_logits_b200 import ckl
from oracle import ops_oracle as O
from tests._helpers import f64

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -23
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(T, n, cols, dt, fmt, seed=0):
    g = torch.Generator().manual_seed(seed + T + n + cols)
    x = (torch.randn(T, cols, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))).to(DT[dt])
    dY = torch.randn(T, n, generator=g).to(DT[dt]).cuda()
    h = ckl.operator_handle(torch.empty(1, 8, dtype=DT[dt], device="cuda"))
    return h, dY, h.act8_pack(x.cuda(), fmt)


def check(dW, dY, ckpt, base=None):
    """Against the products in 64 bits (on the GPU where they are large)."""
    kept = torch.from_numpy(O.act8_values(ckpt.q.cpu().numpy(), ckpt.scale.cpu().numpy(),
                                          ckpt.fmt)).cuda()
    y = dY.double()
    want, mag = y.t() @ kept, y.abs().t() @ kept.abs()
    if base is not None:
        want, mag = want + base.double(), mag + base.double().abs()
    terms = dY.shape[0] * (1 if dY.dtype == torch.bfloat16 else 3)
    err = (dW.double() - want).abs()
    assert bool((err <= (terms + 80) * STEP * mag).all()), float((err / mag).max())
    return float(err.norm() / want.norm())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("T,n,cols", [
    (1, 8, 8), (63, 64, 32), (64, 256, 256), (65, 264, 40), (130, 136, 264), (300, 520, 72),
    (1000, 8, 1032),
    (5000, 64, 64),       # split over token ranges
    (4097, 264, 136),
    (2049, 1032, 1544),
])
def test_weight_grad(T, n, cols, fmt, dt):
    h, dY, ckpt = inputs(T, n, cols, dt, fmt)
    base = torch.randn(n, cols, device="cuda")
    dW = h.act8_weight_grad(dY, ckpt, dW=torch.full((n, cols), float("nan"), device="cuda"))
    rel = check(dW, dY, ckpt)
    acc = h.act8_weight_grad(dY, ckpt, dW=base.clone(), accumulate=True)
    check(acc, dY, ckpt, base)
    assert torch.equal(h.act8_weight_grad(dY, ckpt), dW)
    print(T, n, cols, fmt, dt, f"{rel:.2e}")


def test_against_the_oracle_and_exact_sums():
    h, dY, ckpt = inputs(200, 72, 104, "bf16", "int8")
    want, mag = O.weight_grad(f64(dY), O.act8_values(ckpt.q.cpu().numpy(),
                                                     ckpt.scale.cpu().numpy(), "int8"))
    assert np.all(np.abs(f64(h.act8_weight_grad(dY, ckpt)) - want) <= 280 * STEP * mag)
    for T, n, cols in ((257, 264, 520), (9000, 136, 72)):  # small integers: every order is exact
        g = torch.Generator(device="cuda").manual_seed(T)
        x = torch.randint(-8, 9, (T, cols), generator=g, device="cuda").to(torch.bfloat16)
        dY = torch.randint(-4, 5, (T, n), generator=g, device="cuda").to(torch.bfloat16)
        for fmt in ("int8", "e4m3"):
            got = h.act8_weight_grad(dY, h.act8_pack(x, fmt))
            assert torch.equal(got.double(), dY.double().t() @ x.double())
            f = ckl.operator_handle(torch.empty(1, 8, device="cuda"))
            got = f.act8_weight_grad(dY.float(), f.act8_pack(x.float(), fmt))
            assert torch.equal(got.double(), dY.double().t() @ x.double())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_more_tokens_than_one_chunk(dt):
    """50001 tokens of 2880 columns are contracted in two chunks; small integers, so that every
    order of the sums is exact."""
    T, n, cols = 50001, 72, 2880
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randint(-8, 9, (T, cols), generator=g, device="cuda").to(DT[dt])
    dY = torch.randint(-4, 5, (T, n), generator=g, device="cuda").to(DT[dt])
    h = ckl.operator_handle(dY)
    ckpt = h.act8_pack(x)
    want = dY.double().t() @ x.double()
    assert torch.equal(h.act8_weight_grad(dY, ckpt).double(), want)
    base = torch.randint(-99, 99, (n, cols), generator=g, device="cuda").float()
    got = h.act8_weight_grad(dY, ckpt, dW=base.clone(), accumulate=True)
    assert torch.equal(got.double(), want + base.double())


def test_fp32_gradients_keep_all_their_bits():
    """One token: the product of a 24-bit dY and a code, rounded to fp32."""
    g = torch.Generator(device="cuda").manual_seed(1)
    dY = torch.randn(1, 512, generator=g, device="cuda") * torch.exp2(
        torch.randint(-90, 90, (1, 512), generator=g, device="cuda").float())
    x = torch.zeros(1, 32, device="cuda")
    x[0, :3] = torch.tensor([1.0, -0.5, 127.0], device="cuda")
    h = ckl.operator_handle(dY)
    ckpt = h.act8_pack(x)
    got = h.act8_weight_grad(dY, ckpt)
    want = dY.double().t() @ h.act8_unpack(ckpt).double()  # -0.5 is half a step beside 127: 0
    assert bool(((got.double() - want).abs() <= 4 * STEP * want.abs()).all())
    assert torch.equal(got[:, 0], dY[0])  # times one: the three parts add up again


def test_non_finite_values_reach_their_elements():
    h, dY, ckpt = inputs(100, 64, 64, "f32", "int8")
    x = h.act8_unpack(ckpt)
    x[7, 3] = float("nan")
    dY[9, 5] = float("inf")
    got = h.act8_weight_grad(dY, h.act8_pack(x))
    bad = ~torch.isfinite(got)
    assert bad[:, :32].all() and bad[5].all()
    keep = torch.ones(64, dtype=torch.bool, device="cuda")
    keep[5] = False
    assert not bad[keep][:, 32:].any()


def test_no_tokens():
    h, _, _ = inputs(3, 16, 40, "bf16", "int8")
    ckpt = h.act8_pack(torch.empty(0, 40, device="cuda", dtype=torch.bfloat16))
    dY = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16)
    assert torch.all(h.act8_weight_grad(dY, ckpt) == 0)
    base = torch.randn(16, 40, device="cuda")
    assert torch.equal(h.act8_weight_grad(dY, ckpt, dW=base.clone(), accumulate=True), base)


def test_long_checkpoints_pass_32_bit_offsets():
    T, n, cols = 760000, 8, 2880  # 2.19e9 codes
    q = torch.zeros(T, cols, dtype=torch.uint8, device="cuda")
    e = torch.full((T, 90), 127, dtype=torch.uint8, device="cuda")
    dY = torch.zeros(T, n, dtype=torch.bfloat16, device="cuda")
    q[-70:] = torch.randint(0, 100, (70, cols), device="cuda", dtype=torch.uint8)
    dY[-70:] = torch.randint(-9, 9, (70, n), device="cuda").to(torch.bfloat16)
    h = ckl.operator_handle(dY)
    got = h.act8_weight_grad(dY, ckl.Act8(q, e))
    assert torch.equal(got.double(), dY[-70:].double().t() @ q[-70:].double())


def test_calls_captured_in_a_graph():
    h, dY, ckpt = inputs(3000, 136, 200, "bf16", "int8")
    dW = torch.empty(136, 200, device="cuda")
    ws = h.act8_weight_grad_workspace(3000, 136, 200)
    call = lambda: h.act8_weight_grad(dY, ckpt, dW=dW, workspace=ws, sync=False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (1, 2):
        _, dY2, c2 = inputs(3000, 136, 200, "bf16", "int8", seed)
        dY.copy_(dY2)
        ckpt.q.copy_(c2.q)
        ckpt.scale.copy_(c2.scale)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dW, h.act8_weight_grad(dY2, c2))


def test_refusals():
    h, dY, ckpt = inputs(40, 64, 72, "bf16", "int8")
    with pytest.raises(ValueError):
        h.act8_weight_grad(dY[:39], ckpt)
    with pytest.raises(TypeError):
        h.act8_weight_grad(dY.float(), ckpt)
    with pytest.raises(ValueError):
        h.act8_weight_grad(dY, ckpt, accumulate=True)
    with pytest.raises(TypeError):
        h.act8_weight_grad(dY, ckpt, dW=torch.empty(64, 64, device="cuda"))
    with pytest.raises(ckl.CKLError) as e:
        h.act8_weight_grad(dY[:, :12].contiguous(), ckpt)
    assert e.value.code == 2
    h, dY, ckpt = inputs(5000, 64, 64, "bf16", "int8")
    with pytest.raises(ckl.CKLError) as e:
        h.act8_weight_grad(dY, ckpt, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 3


@pytest.mark.parametrize("T,n,cols", [(32768, 201088, 1024), (400_000, 64000, 64), (1 << 22, 2880, 64),
                                      (1 << 22, 64, 2880), (32768, 2880, 2880)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_the_workspace_is_bounded_whatever_the_tokens_and_outputs(T, n, cols, dt):
    """A copy of X' and, for fp32, three parts of dY: 256 MB or 4096 tokens of each; the partial
    results of at most 64 ranges where dW is small. (Sizes only: nothing is allocated.)"""
    h = ckl.operator_handle(torch.empty(1, 8, dtype=DT[dt], device="cuda"))
    size = ctypes.c_size_t()
    assert ckl.lib().ckl_act8_weight_grad_workspace_bytes(h._h, T, n, cols, ctypes.byref(size)) == 0
    copy = lambda width: max(256 << 20, 4096 * width * 2)
    partial = 64 * n * cols * 4 if n * cols < 1 << 24 else 0
    assert size.value <= copy(cols) + (3 * copy(n) if dt == "f32" else 0) + partial + 1024


def test_fp32_layer_of_many_outputs_in_chunks():
    """9000 tokens of 32768 outputs are contracted in three chunks, since the parts of dY take 192 KB
    a token; small integers, so that every order of the sums is exact."""
    T, n, cols = 9000, 32768, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randint(-8, 9, (T, cols), generator=g, device="cuda").float()
    dY = torch.randint(-4, 5, (T, n), generator=g, device="cuda").float()
    h = ckl.operator_handle(x)  # (n is above a handle's largest d)
    ckpt = h.act8_pack(x)
    want = dY.double().t() @ x.double()
    assert torch.equal(h.act8_weight_grad(dY, ckpt).double(), want)
    base = torch.randint(-99, 99, (n, cols), generator=g, device="cuda").float()
    got = h.act8_weight_grad(dY, ckpt, dW=base.clone(), accumulate=True)
    assert torch.equal(got.double(), want + base.double())


def test_how_far_down_fp32_gradients_keep_all_their_bits():
    """bf16 ends at 2^-133, the lowest bit of a number from 2^-110 on: from there the three parts add
    up to dY, and below they leave out less than 2^-133 of it. One token, times 2^40."""
    g = torch.Generator(device="cuda").manual_seed(3)
    frac = 1 + (2 * torch.randint(0, 1 << 22, (1, 512), generator=g, device="cuda") + 1).double() * 2.0 ** -23
    sign = 1 - 2 * torch.randint(0, 2, (1, 512), generator=g, device="cuda").double()
    x = torch.full((1, 32), 2.0 ** 40, device="cuda")
    h = ckl.operator_handle(x)
    ckpt = h.act8_pack(x)
    for low, high, left_out in ((-110, -90, 0.0), (-126, -110, 2.0 ** -133)):
        exponent = torch.randint(low, high, (1, 512), generator=g, device="cuda").double()
        exponent[0, 0] = low
        dY = (sign * frac * torch.exp2(exponent)).float()
        got = h.act8_weight_grad(dY, ckpt).double()
        assert bool(((got - dY.double().t() * 2.0 ** 40).abs() <= left_out * 2.0 ** 40).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_relative_error_over_many_tokens(dt):
    """The bound of the other cases grows with the tokens; the error must not. The tensor cores cut
    a running sum after each 16 tokens, and an accumulator runs over 1024. A cut takes on average
    0.72 2^-24 of the sum (half a step of it, which is 2^-24 to 2^-23 of the value). Terms of random
    sign make the 64 sums of a run a random walk: their own sum is 64^1.5 / 3^0.5 of a step of the walk,
    the last one 8, so the cuts take 37 * 0.72 * 2^-24 = 1.6e-6 of the result, and the 32 runs' sums in
    registers, rounded, some 2^-24. (One accumulator over all the tokens: 181 / 8 times that.) The
    layer is large enough that no range of tokens is split off."""
    T, n, cols = 32768, 2880, 2880
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, cols, generator=g, device="cuda").to(DT[dt])
    dY = torch.randn(T, n, generator=g, device="cuda").to(DT[dt])
    h = ckl.operator_handle(x)
    ckpt = h.act8_pack(x)
    want = dY.double().t() @ h.act8_unpack(ckpt).double()
    rel = float((h.act8_weight_grad(dY, ckpt).double() - want).norm() / want.norm())
    print(dt, f"{rel:.2e}")
    assert rel <= 2e-6
