"""Checks of the operators around the loss that need no GPU: null handles, and what the
Python side refuses before it calls the library."""
import ctypes

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


def test_operator_handle_refuses_cpu_tensors():
    with pytest.raises(ValueError):
        ckl.operator_handle(torch.zeros(2, 8))


def test_rms_norm_refuses_strided_inputs():
    x, g = torch.zeros(4, 16), torch.ones(8)
    with pytest.raises(ValueError):
        ckl.rms_norm(x[:, ::2], g, handle=object())
    with pytest.raises(ValueError):
        ckl.rms_norm(torch.zeros(4, 8), g, residual=torch.zeros(3, 8), handle=object())
