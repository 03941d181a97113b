"""The operators' calls and their backward passes captured in CUDA graphs."""
import pytest
import torch

from chunked_kl_loss_logits_b200 import ckl

pytestmark = pytest.mark.gpu
T, V, D = 300, 500, 264


def inputs():
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    W = torch.randn(V, D, generator=g).to(torch.bfloat16).cuda()
    gain = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
    return ids, W, gain


def test_a_call_that_would_wait_is_refused_in_a_capture_that_goes_on():
    ids, W, gain = inputs()
    h = ckl.operator_handle(W, V)
    x = h.embed(ids, W)
    dW = h.embed_grad(ids, x)
    c = h.act8_pack(x)
    dL = h.act8_weight_grad(x, c)
    torch.cuda.synchronize()
    before = h.launch_count()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in (lambda: h.embed(ids, W), lambda: h.embed_grad(ids, x),
                     lambda: h.act8_weight_grad(x, c)):
            with pytest.raises(ckl.CKLError) as e:
                call()
            assert e.value.code == 1
        assert h.launch_count() == before
        out = h.embed(ids, W, sync=False)
        dW2 = h.embed_grad(ids, x, sync=False)
        dL2 = h.act8_weight_grad(x, c, sync=False)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, x) and torch.equal(dW2, dW) and torch.equal(dL2, dL)
    h.sync_status()


def test_a_backward_pass_captured():
    """embedding and rms_norm with their backward passes in one graph, replayed on other ids."""
    ids, W, gain = inputs()
    W.requires_grad_()
    gain.requires_grad_()
    weight = torch.randn(T, D, device="cuda").to(torch.bfloat16)

    def step():
        x = ckl.embedding(ids, W, scale=2.0, check=False)
        y, s = ckl.rms_norm(x, gain, residual=x.detach() * 0.5)
        ((y * weight).sum() + s.sum()).backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            W.grad = gain.grad = None
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    W.grad = gain.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    static = W.grad, gain.grad
    replayed = []
    for seed in (1, 2):
        ids.copy_(torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(seed),
                                dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        replayed.append((ids.clone(), static[0].clone(), static[1].clone()))
    ckl.operator_handle(W, V).sync_status()
    for k, gW, gg in replayed:
        ids.copy_(k)
        W.grad = gain.grad = None
        step()
        assert torch.equal(W.grad, gW) and torch.equal(gain.grad, gg)


@pytest.mark.parametrize("none", ["masked", "other rows"])
@pytest.mark.parametrize("T", [1, 40, 512])
def test_a_captured_gradient_without_a_token_is_read_by_the_next_node(T, none):
    """An overwritten dW of 690 MB whose batch has no token here: the node after the call, which
    depends on the call's last kernel alone, reads the zeros."""
    rows, d = 60000, 2880
    dX = torch.full((T, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, 1000, (T,), dtype=torch.int32, device="cuda")
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda") if none == "masked" else None
    kw = {} if mask is not None else {"V_total": 1000 + rows, "v0": 1000}
    h = ckl.operator_handle(dX, V=rows)
    dW, seen = torch.empty(rows, d, device="cuda"), torch.empty(rows, d, device="cuda")
    call = lambda: (h.embed_grad(ids, dX, mask=mask, dW=dW, sync=False, **kw), seen.copy_(dW))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(5):
        dW.fill_(7.0)
        seen.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert not seen.any() and not dW.any()
    h.sync_status()


@pytest.mark.parametrize("tokens", [4097, 6000, 20000])
@pytest.mark.parametrize("rows", [400, 70000])
def test_a_captured_gradient_whose_tokens_are_sorted(tokens, rows):
    """More tokens than have their places counted, sorted by digits (one, and two): 4097 tokens leave
    CTAs of the sort without any, which are done long before those whose counts they were asked for."""
    gen = torch.Generator().manual_seed(tokens + rows)
    ids = torch.randint(0, rows, (tokens,), generator=gen, dtype=torch.int32).cuda()
    dX = torch.randint(-4, 5, (tokens, 40), generator=gen).to(torch.bfloat16).cuda()
    h = ckl.operator_handle(dX, V=rows)
    dW, ws = torch.empty(rows, 40, device="cuda"), h.embed_grad_workspace(tokens)
    call = lambda: h.embed_grad(ids, dX, dW=dW, workspace=ws, sync=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(20):
        ids.copy_(torch.randint(0, rows, (tokens,), generator=gen, dtype=torch.int32))
        ids[::3] = k
        dW.fill_(7.0)
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        want = torch.zeros(rows, 40, device="cuda").index_add_(0, ids, dX.float())
        assert torch.equal(dW, want)  # whole numbers: every order of the sums is exact
    h.sync_status()
