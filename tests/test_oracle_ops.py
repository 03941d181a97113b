"""Pins of the oracle of the operators around the loss (CPU)."""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as O

rng = np.random.default_rng


def test_embed_and_gradient_are_adjoint():
    r = rng(1)
    ids, mask = r.integers(0, 9, 40), (r.random(40) < 0.8).astype(np.uint8)
    W, G = r.normal(size=(9, 8)), r.normal(size=(40, 8))
    out = O.embed(ids, W, mask, 1.5)
    dW, _ = O.embed_grad(ids, G, 9, mask, 1.5)
    assert abs((out * G).sum() - (W * dW).sum()) < 1e-12
    t = torch.from_numpy(W).requires_grad_()
    (torch.nn.functional.embedding(torch.from_numpy(ids), t) * 1.5 *
     torch.from_numpy(mask[:, None] * G)).sum().backward()
    assert np.allclose(t.grad.numpy(), dW, rtol=1e-13, atol=1e-13)


def test_embed_shards_add_up():
    r = rng(2)
    ids, W, G = r.integers(0, 30, 50), r.normal(size=(30, 8)), r.normal(size=(50, 8))
    parts = [O.embed(ids, W[a:b], v0=a) for a, b in ((0, 11), (11, 30))]
    assert np.array_equal(sum(parts), O.embed(ids, W))
    grads = [O.embed_grad(ids, G, b - a, v0=a)[0] for a, b in ((0, 11), (11, 30))]
    assert np.array_equal(np.concatenate(grads), O.embed_grad(ids, G, 30)[0])


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_table(), t, equal_nan=True)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("cols", [8, 32, 40, 72])
def test_act8_error_bound_and_minimal_scale(fmt, cols):
    x = (rng(cols).normal(size=(20, cols)) * np.exp(rng(3).normal(size=(20, 1)) * 8)).astype(np.float32)
    q, byte = O.act8_pack(x, fmt)
    v = O.act8_values(q, byte, fmt)
    step = np.repeat(2.0 ** (byte.astype(np.float64) - 127), 32, axis=1)[:, :cols]
    if fmt == "int8":
        assert np.all(np.abs(v - x) <= step / 2)
    else:  # 2^-4 of the value, half a subnormal step below
        assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10))
    for b in range(byte.shape[1]):  # one exponent less would not hold the block
        top = np.abs(x[:, 32 * b:32 * b + 32]).max(1)
        e = byte[:, b].astype(np.float64) - 127
        assert np.all(top <= O.LIMIT[fmt] * 2.0 ** e)
        assert np.all((top > O.LIMIT[fmt] * 2.0 ** (e - 1)) | (e == -126))


def test_act8_e4m3_rounds_as_torch_does():
    x = np.concatenate([np.linspace(-448, 448, 4096), O.e4m3_table()[:127],
                        (O.e4m3_table()[:126] + O.e4m3_table()[1:127]) / 2])[:4320].reshape(-1, 32)
    x[:, 0] = 448.0  # every block at exponent 0
    q, byte = O.act8_pack(x, "e4m3")
    assert np.all(byte == 127)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(q, want)


def test_act8_bad_blocks_and_zeros():
    x = np.zeros((3, 64), np.float32)
    x[0, 5], x[1, 40], x[2, 3] = np.nan, -np.inf, 1e-45
    for fmt in ("int8", "e4m3"):
        q, byte = O.act8_pack(x, fmt)
        assert byte.tolist() == [[255, 1], [1, 255], [1, 1]]
        v = O.act8_values(q, byte, fmt)
        assert np.isnan(v[0, :32]).all() and np.isnan(v[1, 32:]).all() and np.all(v[2] == 0)


def test_norm_gradient_is_that_of_the_formula_and_of_differences():
    r = rng(5)
    s, g, dY, dS = r.normal(size=(6, 24)), r.normal(size=24), r.normal(size=(6, 24)), r.normal(size=(6, 24))
    y, rstd = O.norm(s, g, 1e-3)
    dX, dg, *_ = O.norm_bwd(dY, s, rstd, g, dS)
    eps = float(np.float32(1e-3))
    ts, tg = torch.from_numpy(s).requires_grad_(), torch.from_numpy(g).requires_grad_()
    ty = ts * torch.rsqrt((ts * ts).mean(1, keepdim=True) + eps) * tg
    assert np.allclose(ty.detach().numpy(), y, rtol=1e-13)
    ((ty * torch.from_numpy(dY)).sum() + (ts * torch.from_numpy(dS)).sum()).backward()
    assert np.allclose(ts.grad.numpy(), dX, rtol=1e-11, atol=1e-12)
    assert np.allclose(tg.grad.numpy(), dg, rtol=1e-11, atol=1e-12)
    u = r.normal(size=s.shape)
    f = lambda h: (O.norm(s + h * u, g, 1e-3)[0] * dY).sum() + ((s + h * u) * dS).sum()
    assert abs((f(1e-6) - f(-1e-6)) / 2e-6 - (dX * u).sum()) < 1e-7
