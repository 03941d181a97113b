"""Checks of the operators around the loss that need no GPU: null handles, and what the
Python side refuses before it calls the library."""
import ctypes
import threading

import pytest
import torch

from chunked_kl_loss_logits_b200 import ckl


@pytest.fixture(scope="module")
def L():
    from chunked_kl_loss_logits_b200 import build
    build.build()
    return ckl.lib()


def test_null_handle_calls(L):
    n = ctypes.c_size_t()
    N = None
    assert L.ckl_embed(N, N, N, N, 4, 8, 0, 1.0, N, N, 0) == 1
    assert L.ckl_embed_vp_workspace_bytes(N, 4, ctypes.byref(n)) == 1
    assert L.ckl_embed_vocab_parallel(N, N, N, N, N, 4, 1.0, N, N, 0, N, 0) == 1
    assert L.ckl_embed_grad_workspace_bytes(N, 4, ctypes.byref(n)) == 1
    assert L.ckl_embed_grad(N, N, N, N, 4, 8, 0, 1.0, 0, N, N, 0, N, 0) == 1
    assert L.ckl_act8_pack(N, N, 4, 8, 0, N, N, N) == 1
    assert L.ckl_act8_unpack(N, N, N, 4, 8, 0, N, N) == 1
    assert L.ckl_act8_weight_grad_workspace_bytes(N, 4, 8, 8, ctypes.byref(n)) == 1
    assert L.ckl_act8_weight_grad(N, N, 4, 8, N, N, 8, 0, 0, N, N, 0, N, 0) == 1
    assert L.ckl_norm(N, N, N, N, 4, 1e-5, 0, N, N, N, N, N, N) == 1
    assert L.ckl_norm_bwd_workspace_bytes(N, 4, ctypes.byref(n)) == 1
    assert L.ckl_norm_bwd(N, N, N, N, N, N, N, 4, 0, 0, N, N, N, 0, N) == 1


def test_act8_refuses_inconsistent_parts():
    q, e = torch.zeros(3, 40, dtype=torch.uint8), torch.zeros(3, 2, dtype=torch.uint8)
    c = ckl.Act8(q, e, "e4m3", torch.ones(3))
    assert c.nbytes == 3 * 40 + 3 * 2 + 12
    with pytest.raises(ValueError):
        ckl.Act8(q, e, "int4")
    with pytest.raises(TypeError):
        ckl.Act8(q.to(torch.int8), e)
    with pytest.raises(ValueError):
        ckl.Act8(q, e[:, :1].contiguous())
    with pytest.raises(ValueError):
        ckl.Act8(q[:, ::2], e)
    with pytest.raises(TypeError):
        ckl.Act8(q, e, rstd=torch.ones(4))
    with pytest.raises(TypeError):
        ckl.Act8(q, e, rstd=torch.ones(3, dtype=torch.float64))


def test_the_module_refuses_before_it_calls(L):
    """The checks of the operators' module, on tensors that are not on a GPU: types and shapes
    first, then the device; a null handle would be refused by the library only after them."""
    m = ckl._ops()
    ctx = (0, 30, 16, True, 0)
    ids, W, x = torch.zeros(4, dtype=torch.int32), torch.zeros(30, 16).bfloat16(), \
        torch.zeros(4, 16).bfloat16()
    ck = ckl.Act8(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))
    T, V = TypeError, ValueError
    for err, call in (
            (T, lambda: m.embed(ctx, ids)),
            (T, lambda: m.embed(ctx, ids.long(), W, None, 1.0, None, 0, None, False)),
            (T, lambda: m.embed(ctx, [1, 2], W, None, 1.0, None, 0, None, False)),
            (V, lambda: m.embed(ctx, ids, W, None, 1.0, None, 0, None, False)),  # on the CPU
            (T, lambda: m.embed_grad(ctx, ids.float(), x, None, 1.0, None, 0, None, 0, None, 0)),
            (T, lambda: m.norm(ctx, x.float(), x[0], None, 1e-5, -1, None, None, None)),
            (V, lambda: m.norm(ctx, x[:, :8], x[0], None, 1e-5, -1, None, None, None)),
            (T, lambda: m.norm(ctx, None, x[0], None, 1e-5, -1, None, None, None)),
            (V, lambda: m.norm(ctx, x, x[0], None, 1e-5, -1, None, None, None)),
            (V, lambda: m.norm_bwd(ctx, x, ck._desc, x[0], None, None, None, 0, None)),
            (V, lambda: m.act8_unpack(ctx, ck._desc, None)),
            (V, lambda: m.act8_pack(ctx, x, 0, None))):
        with pytest.raises(err):
            call()


def test_operator_handle_refuses_cpu_tensors():
    with pytest.raises(ValueError):
        ckl.operator_handle(torch.zeros(2, 8))


def test_rms_norm_refuses_strided_inputs():
    x, g = torch.zeros(4, 16), torch.ones(8)
    with pytest.raises(ValueError):
        ckl.rms_norm(x[:, ::2], g, handle=object())
    with pytest.raises(ValueError):
        ckl.rms_norm(torch.zeros(4, 8), g, residual=torch.zeros(3, 8), handle=object())


class _OlderLibrary:
    """A build of the library from before the operators: it creates handles, and has the loss."""

    def __init__(self, path):
        for f in ckl.header_functions():
            if not any(w in f for w in ("embed", "act8", "norm")):
                setattr(self, f, lambda *a: 0)


def test_the_loss_needs_neither_the_module_nor_a_library_with_the_operators(monkeypatch):
    monkeypatch.setattr(ckl, "_ops_module", None)
    monkeypatch.setattr(ckl, "_lib", None)
    monkeypatch.setattr(ckl, "LIB_PATH", __file__)
    monkeypatch.setattr(ckl.ctypes, "CDLL", _OlderLibrary)
    x = torch.zeros(2, 8)
    h = ckl.ChunkedKL(16, 8, 4, dtype=torch.float32, max_chunk=8, device="cuda:0")
    assert h.workspace_bytes(2, 2) == 0
    with pytest.raises(RuntimeError, match="without these operators"):
        h.act8_pack(x)
    monkeypatch.setattr(ckl, "OPS_PATH", "/nowhere/_ckl_ops.so")
    h = ckl.ChunkedKL(16, 8, 4, dtype=torch.float32, max_chunk=8, device="cuda:0")
    with pytest.raises(RuntimeError, match="is missing"):
        h.act8_pack(x)
    h.close()


def test_operator_handle_replaces_a_closed_one(monkeypatch):
    class Handle:
        def __init__(self, *a, **k):
            self._h = object()

        def close(self):
            self._h = None

    class OnGpu:
        dtype, shape, device = torch.float32, (4, 8), torch.device("cuda", 0)

        def get_device(self):
            return 0

    monkeypatch.setattr(ckl, "ChunkedKL", Handle)
    monkeypatch.setattr(ckl, "_OP_HANDLES", threading.local())
    a = ckl.operator_handle(OnGpu())
    assert ckl.operator_handle(OnGpu()) is a
    a.close()
    b = ckl.operator_handle(OnGpu())
    assert b is not a and b._h and ckl.operator_handle(OnGpu()) is b


def test_rms_norm_refuses_a_handle_of_another_width():
    """16 columns are not two rows of 8."""
    class Handle:
        d = 8

        def norm(self, *a):
            raise AssertionError("called")

    with pytest.raises(ValueError):
        ckl.rms_norm(torch.zeros(4, 16), torch.ones(8), handle=Handle())
