"""Embedding lookup and its gradient by sorted tokens, against the fp64 oracle.

Bounds, with u = 2^-24 (half a step of fp32) and n the tokens of a row: a looked-up element is
one fp32 product and one rounding to its type (half a step, eps / 2 of the value). A gradient
element is n - 1 additions in some order, one product with the scale and one addition to what
was there, so it is off by at most (n + 2) u times the sum of the magnitudes that enter it
(1.01: the higher orders).

The gradient of up to 512 tokens needs no sort, of up to 4096 each token's place is counted, and
above that a cluster sorts by digits; comments at smaller cases that speak of the sort are from
when it began there.
"""
import threading

import numpy as np
import pytest
import torch

from chunked_kl_loss_logits_b200 import ckl
from oracle import ops_oracle as O
from tests._helpers import f64
from tests.test_gpu_vocab_parallel import ThreadGroup

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def case(T, d, V, dt, seed=0, masked=False, hot=0.0):
    g = torch.Generator().manual_seed(seed + T + d + V)
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    ids[torch.rand(T, generator=g) < hot] = V // 2  # a frequent token
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8) if masked else None
    W = torch.randn(V, d, generator=g).to(DT[dt])
    dX = torch.randn(T, d, generator=g).to(DT[dt])
    return [None if t is None else t.cuda() for t in (ids, mask, W, dX)]


def check_grad(dW, ids, dX, V, mask, scale, base=None, v0=0):
    keep = None if mask is None else mask.cpu().numpy()
    want, mag = O.embed_grad(ids.cpu().numpy(), f64(dX), V, keep, scale, v0,
                             None if base is None else f64(base))
    local = ids.cpu().numpy().astype(np.int64) - v0
    sel = (local >= 0) & (local < V) & (True if keep is None else keep != 0)
    n = np.bincount(local[sel], minlength=V)[:, None]
    err = np.abs(f64(dW) - want)
    assert np.all(err <= 1.01 * (n + 2) * U * mag), float((err - 1.01 * (n + 2) * U * mag).max())
    if base is not None:  # rows without a token are left as they were
        assert torch.equal(dW[torch.from_numpy(n[:, 0] == 0).cuda()],
                           base[torch.from_numpy(n[:, 0] == 0).cuda()])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V", [(1, 8, 1), (3, 64, 5), (65, 136, 777), (257, 2880, 3001),
                                   (300, 1032, 512)])
@pytest.mark.parametrize("masked", [False, True])
def test_embed(T, d, V, dt, masked):
    ids, mask, W, _ = case(T, d, V, dt, masked=masked)
    h = ckl.operator_handle(W, V=V)
    out = h.embed(ids, W, mask=mask, scale=3.7)
    want = O.embed(ids.cpu().numpy(), f64(W), None if mask is None else mask.cpu().numpy(),
                   float(np.float32(3.7)))
    half = torch.finfo(DT[dt]).eps / 2
    assert np.all(np.abs(f64(out) - want) <= (half + 1.01 * U) * np.abs(want))
    out2 = h.embed(ids.view(1, T), W, mask=mask, scale=3.7)
    assert out2.shape == (1, T, d) and torch.equal(out2[0], out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,hot", [
    (1, 8, 1, 0), (2, 64, 1, 0), (33, 136, 777, 0), (700, 64, 5, 0.3),
    (1025, 264, 511, 0.1),     # two CTAs sort; 9-bit keys
    (5000, 72, 512, 0.5),      # 10-bit keys in two digits; a row over many tiles
    (4097, 128, 70000, 0),     # nearly all rows distinct
])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad(T, d, V, hot, dt, accumulate):
    ids, mask, W, dX = case(T, d, V, dt, masked=T % 2 == 1, hot=hot)
    if mask is not None and T > 4:
        dX[mask == 0] = float("nan")  # what a masked place holds does not matter
    h = ckl.operator_handle(W, V=V)
    base = torch.randn(V, d, device="cuda")
    runs = []
    for _ in range(2):
        dW = base.clone() if accumulate else torch.full((V, d), float("nan"), device="cuda")
        got = h.embed_grad(ids, dX, mask=mask, scale=0.37, dW=dW, accumulate=accumulate)
        assert got is dW
        runs.append(dW)
    assert torch.equal(*runs)
    clean = torch.nan_to_num(dX.float()).to(dX.dtype)
    check_grad(runs[0], ids, clean, V, mask, float(np.float32(0.37)), base if accumulate else None)


def test_embed_grad_one_row_takes_every_token():
    for T in (31, 32, 33, 64, 65, 4096, 40000):
        ids = torch.full((T,), 6, dtype=torch.int32, device="cuda")
        dX = torch.randn(T, 8, device="cuda")
        h = ckl.operator_handle(dX, V=9)
        check_grad(h.embed_grad(ids, dX), ids, dX, 9, None, 1.0)


def test_embed_grad_many_tokens_three_digits():
    """A long sequence (every CTA of the sort walks its range several times) and a vocabulary
    of 19 bits; integers, so that every order of the sums is exact."""
    T, d, V = 150001, 16, 300000
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = (torch.rand(T, generator=g, device="cuda") ** 6 * V).to(torch.int32)
    dX = torch.randint(-4, 5, (T, d), generator=g, device="cuda").to(torch.bfloat16)
    h = ckl.operator_handle(dX, V=V)
    want = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, ids.long(), dX.double())
    assert torch.equal(h.embed_grad(ids, dX).double(), want)


def test_embed_grad_largest_keys():
    """A vocabulary of 28 bits (four digits) and a shard of it that starts far up."""
    V, d = 140_000_000, 8
    ids = torch.tensor([V - 1, 0, V - 1, 77_777_777, 0, V - 1], dtype=torch.int32, device="cuda")
    dX = torch.arange(48, device="cuda", dtype=torch.float32).view(6, 8)
    h = ckl.ChunkedKL(V, d, 1, dtype=torch.float32, max_chunk=1)
    dW = h.embed_grad(ids, dX)
    assert torch.equal(dW[V - 1], dX[0] + dX[2] + dX[5]) and torch.equal(dW[0], dX[1] + dX[4])
    assert torch.equal(dW[77_777_777], dX[3])
    dW[V - 1] = dW[0] = dW[77_777_777] = 0
    assert not dW.any()
    h.close()
    s = ckl.operator_handle(dX, V=10)
    got = s.embed_grad(ids, dX, V_total=2 ** 31 - 1, v0=77_777_770)
    assert torch.equal(got[7], dX[3]) and not got[:7].any() and not got[8:].any()
    wild = torch.tensor([-2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    with pytest.raises(ckl.CKLError):
        s.embed_grad(wild, dX[:2], V_total=2 ** 31 - 1, v0=77_777_770)


def test_masks_and_lengths_that_leave_nothing():
    ids, _, W, dX = case(40, 64, 30, "bf16")
    h = ckl.operator_handle(W, V=30)
    none = torch.zeros(40, dtype=torch.uint8, device="cuda")
    wild = torch.full_like(ids, -1)  # the ids of masked tokens are not looked at
    assert torch.all(h.embed(wild, W, mask=none) == 0)
    assert torch.all(h.embed_grad(wild, dX, mask=none) == 0)
    base = torch.randn(30, 64, device="cuda")
    assert torch.equal(h.embed_grad(wild, dX, mask=none, dW=base.clone(), accumulate=True), base)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert h.embed(e, W).shape == (0, 64)
    dX0 = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    assert torch.all(h.embed_grad(e, dX0, dW=torch.ones(30, 64, device="cuda")) == 0)
    assert torch.equal(h.embed_grad(e, dX0, dW=base.clone(), accumulate=True), base)


@pytest.mark.parametrize("bad", [-1, 30, 2 ** 31 - 1])
def test_an_id_out_of_range_is_reported_and_adds_nothing(bad):
    ids, _, W, dX = case(40, 64, 30, "bf16")
    ids[7] = bad
    h = ckl.operator_handle(W, V=30)
    out = torch.empty(40, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ckl.CKLError) as e:
        h.embed(ids, W, out=out)
    assert e.value.code == 4 and torch.all(out[7] == 0)
    dW = torch.empty(30, 64, device="cuda")
    with pytest.raises(ckl.CKLError) as e:
        h.embed_grad(ids, dX, dW=dW)
    assert e.value.code == 4
    keep = torch.ones(40, dtype=torch.uint8, device="cuda")
    keep[7] = 0
    assert torch.equal(dW, h.embed_grad(ids, dX, mask=keep))  # the status was cleared


def test_shards_of_the_vocabulary():
    ids, mask, W, dX = case(300, 64, 100, "bf16", masked=True)
    whole = ckl.operator_handle(W, V=100)
    out, dW = whole.embed(ids, W, mask=mask), whole.embed_grad(ids, dX, mask=mask)
    total = torch.zeros_like(out)
    for v0, n in ((0, 37), (37, 63)):
        h = ckl.operator_handle(W, V=n)
        total += h.embed(ids, W[v0:v0 + n], mask=mask, V_total=100, v0=v0)
        assert torch.equal(h.embed_grad(ids, dX, mask=mask, V_total=100, v0=v0), dW[v0:v0 + n])
    assert torch.equal(total, out)


def test_embed_vocab_parallel():
    ids, mask, W, _ = case(130, 128, 700, "bf16", masked=True)
    want = ckl.operator_handle(W, V=700).embed(ids, W, mask=mask, scale=2.5)
    torch.cuda.synchronize()
    shards, tg, got, errs = ckl.vocab_shards(700, 2), ThreadGroup(2), [None, None], []

    def rank(r):
        try:
            v0, n = shards[r]
            h = ckl.ChunkedKL(n, 128, 4, max_chunk=64)
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[r] = h.embed_vocab_parallel(tg.member(r, 700, v0), ids, W[v0:v0 + n], mask,
                                                scale=2.5).cpu()
            h.close()
        except Exception as e:
            errs.append(e)
            tg.barrier.abort()

    th = [threading.Thread(target=rank, args=(r,)) for r in range(2)]
    [t.start() for t in th]
    [t.join(120) for t in th]
    assert not errs, errs
    assert torch.equal(got[0], want.cpu()) and torch.equal(got[1], want.cpu())
    assert tg.calls[0] == [("reduce", 130 * 128)] and tg.calls[0] == tg.calls[1]


def test_long_sequences_pass_32_bit_offsets():
    T, d, V = 760000, 2880, 64  # 2.19e9 elements
    W = torch.randn(V, d, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, V - 1, (T,), device="cuda", dtype=torch.int32)
    ids[-5:] = V - 1
    h = ckl.operator_handle(W, V=V)
    out = h.embed(ids, W)
    assert torch.equal(out[-9:], W[ids[-9:].long()])
    out.zero_()
    out[-5:] = 1.0  # as dX: the last row's gradient comes from the far end alone
    dW = h.embed_grad(ids, out)
    assert torch.all(dW[:-1] == 0) and torch.all(dW[-1] == 5.0)


def test_calls_captured_in_a_graph_and_on_a_stream():
    ids, mask, W, dX = case(3000, 264, 900, "bf16", masked=True, hot=0.2)
    h = ckl.operator_handle(W, V=900)
    out, dW = torch.empty_like(dX), torch.empty(900, 264, device="cuda")
    ws = h.embed_grad_workspace(3000)
    call = lambda: (h.embed(ids, W, mask=mask, out=out, sync=False),
                    h.embed_grad(ids, dX, mask=mask, dW=dW, workspace=ws, sync=False))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (1, 2):
        ids2, _, _, dX2 = case(3000, 264, 900, "bf16", seed=seed, hot=0.4 * seed)
        ids.copy_(ids2)
        dX.copy_(dX2)
        out.fill_(7)
        dW.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, h.embed(ids, W, mask=mask))
        assert torch.equal(dW, h.embed_grad(ids, dX, mask=mask))


def test_two_calls_in_flight_and_a_stream_of_its_own():
    cs = [case(5000, 264, 3000, "bf16", seed=k, hot=0.2) for k in (0, 1)]
    hs = [ckl.ChunkedKL(3000, 264, 1, max_chunk=1) for _ in cs]
    alone = [(h.embed(c[0], c[2]), h.embed_grad(c[0], c[3])) for h, c in zip(hs, cs)]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        both = [(h.embed(c[0], c[2], sync=False, stream=s), h.embed_grad(c[0], c[3], sync=False, stream=s))
                for h, c, s in zip(hs, cs, ss)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    [h.sync_status() for h in hs]
    [h.close() for h in hs]


def test_autograd_embedding():
    ids, mask, W, dX = case(500, 64, 90, "f32", masked=True)
    W.requires_grad_()
    out = ckl.embedding(ids.view(5, 100), W, mask=mask, scale=2.0)
    assert out.shape == (5, 100, 64)
    out.backward(dX.view(5, 100, 64))
    check_grad(W.grad, ids, dX, 90, mask, 2.0)
    W.grad = None
    ckl.embedding(ids, W).sum().backward()  # an expanded gradient
    n = torch.bincount(ids.long(), minlength=90).float()[:, None].expand(90, 64)
    assert torch.equal(W.grad, n)
    ids[3] = 90
    with pytest.raises(ckl.CKLError):
        ckl.embedding(ids, W).sum().backward()


def test_refusals():
    ids, mask, W, dX = case(40, 64, 30, "bf16")
    h = ckl.operator_handle(W, V=30)
    with pytest.raises(TypeError):
        h.embed(ids.long(), W)
    with pytest.raises(TypeError):
        h.embed(ids, W.float())
    with pytest.raises(ValueError):
        h.embed(ids, W[:29])
    with pytest.raises(TypeError):
        h.embed(ids, W, mask=torch.ones(39, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        h.embed(ids[::2], W)
    with pytest.raises(ValueError):
        h.embed(ids.cpu(), W)
    with pytest.raises(ValueError):
        h.embed_grad(ids, dX, accumulate=True)
    with pytest.raises(ValueError):
        h.embed_grad(ids, dX[:39])
    with pytest.raises(TypeError):
        h.embed_grad(ids, dX, dW=torch.empty(30, 64, device="cuda", dtype=torch.bfloat16))
    for kw in ({"scale": float("nan")}, {"scale": float("inf")}, {"v0": -1}, {"v0": 1},
               {"V_total": 29}):
        with pytest.raises(ckl.CKLError) as e:
            h.embed(ids, W, **kw)
        assert e.value.code == 1
    with pytest.raises(ckl.CKLError) as e:
        h.embed_grad(ids, dX, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 3
    shifted = torch.empty(30 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(30, 64)
    with pytest.raises(ckl.CKLError) as e:
        h.embed(ids, shifted)
    assert e.value.code == 7


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 31, 32, 33, 255, 256, 257])
@pytest.mark.parametrize("hot", [0, 0.6, 1])
def test_embed_grad_of_few_tokens(T, hot, dt):
    """Both sides of where the sort begins: rows met once, a row met by most tokens, by all; a
    last column block that is not full; overwritten, added to, and on a shard."""
    d, V = 520, 90
    ids, mask, W, dX = case(T, d, V, dt, masked=True, hot=hot)
    dX[mask == 0] = float("inf")
    ids[mask == 0] = -7
    h = ckl.operator_handle(W, V=V)
    base = torch.randn(V, d, device="cuda")
    clean = torch.where((mask != 0)[:, None], dX, torch.zeros_like(dX))
    look = torch.where(mask != 0, ids, torch.zeros_like(ids))
    got = h.embed_grad(ids, dX, mask=mask, scale=1.7)
    check_grad(got, look, clean, V, mask, float(np.float32(1.7)), None)
    assert torch.equal(got, h.embed_grad(ids, dX, mask=mask, scale=1.7))
    more = h.embed_grad(ids, dX, mask=mask, scale=1.7, dW=base.clone(), accumulate=True)
    check_grad(more, look, clean, V, mask, float(np.float32(1.7)), base)
    s = ckl.operator_handle(W, V=50)
    part = s.embed_grad(ids, dX, mask=mask, scale=1.7, V_total=V, v0=30)
    # (not the same bits as got[30:80]: how a sorted row's tokens are grouped depends on where it is)
    check_grad(part, look, clean, 50, mask, float(np.float32(1.7)), v0=30)


def test_embed_grad_of_few_tokens_behind_another_call():
    """Its inputs written by the call before it, which lets what follows start early."""
    T, d, V = 200, 2048, 300
    ids, _, _, dX = case(T, d, V, "bf16")
    x = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    gain = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    h, he = ckl.operator_handle(x), ckl.operator_handle(x, V=V)
    _, _, c = h.norm(x, gain)
    dW = torch.zeros(V, d, device="cuda")
    for k in range(20):
        dY = (dX * (k + 1)).contiguous()
        ref = he.embed_grad(ids, h.norm_bwd(dY, c, gain)[0].clone())
        out = torch.full_like(dY, float("nan"))
        dW.zero_()
        h.norm_bwd(dY, c, gain, dX=out)
        he.embed_grad(ids, out, dW=dW, accumulate=True, sync=False)
        torch.cuda.synchronize()
        assert torch.equal(dW, ref)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 264, 776, 1288, 2880])
def test_embed_grad_of_few_tokens_by_how_often_a_row_occurs(d, dt):
    """Rows of 1, 2, 3 ... tokens: the ways in which a row's work is shared out, with one slab of
    columns and with many; up to and past the most tokens that go without a sort."""
    g = torch.Generator().manual_seed(d)
    often = [1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 12, 13, 16, 17, 40, 64, 65, 150]
    for T in (sum(often), 511, 512, 513, 1025):
        ids = torch.repeat_interleave(torch.arange(len(often), dtype=torch.int32), torch.tensor(often))
        ids = torch.cat([ids, torch.full((T - len(ids),), 40, dtype=torch.int32)])
        ids = ids[torch.randperm(T, generator=g)].cuda()
        dX = torch.randn(T, d, generator=g).to(DT[dt]).cuda()
        h = ckl.operator_handle(dX, V=41)
        got = h.embed_grad(ids, dX, scale=3.0)
        check_grad(got, ids, dX, 41, None, 3.0)
        assert torch.equal(got, h.embed_grad(ids, dX, scale=3.0))
        base = torch.randn(41, d, device="cuda")
        check_grad(h.embed_grad(ids, dX, dW=base.clone(), accumulate=True), ids, dX, 41, None, 1.0, base)


@pytest.mark.parametrize("T,V,hot", [
    (1025, 3, 0), (1153, 70000, 0.3), (4000, 40, 0), (4095, 9000, 0.05),
    (4096, 300000, 0.2),                       # the most tokens whose places are counted
    (4097, 511, 0.1), (8193, 512, 0),          # sorted by digits: one of 9 bits, two of 5
    (12345, 70000, 0.5), (20000, 1, 0),
])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_embed_grad_by_both_ways_to_sort(T, V, hot, dt):
    ids, mask, W, dX = case(T, 72, V, dt, masked=True, hot=hot)
    ids[mask == 0] = 2 ** 31 - 1
    dX[mask == 0] = float("nan")
    clean = torch.where((mask != 0)[:, None], dX, torch.zeros_like(dX))
    look = torch.where(mask != 0, ids, torch.zeros_like(ids))
    h = ckl.operator_handle(W, V=V)
    got = h.embed_grad(ids, dX, mask=mask, scale=0.7, dW=torch.full((V, 72), float("nan"), device="cuda"))
    check_grad(got, look, clean, V, mask, float(np.float32(0.7)))
    assert torch.equal(got, h.embed_grad(ids, dX, mask=mask, scale=0.7))
    base = torch.randn(V, 72, device="cuda")
    check_grad(h.embed_grad(ids, dX, mask=mask, dW=base.clone(), accumulate=True), look, clean, V,
               mask, 1.0, base)


@pytest.mark.parametrize("T", [3000, 9000])
def test_an_id_out_of_range_among_many(T):
    ids, _, W, dX = case(T, 64, 300, "bf16")
    ids[T - 3] = 300
    h = ckl.operator_handle(W, V=300)
    dW = torch.empty(300, 64, device="cuda")
    with pytest.raises(ckl.CKLError) as e:
        h.embed_grad(ids, dX, dW=dW)
    assert e.value.code == 4
    keep = torch.ones(T, dtype=torch.uint8, device="cuda")
    keep[T - 3] = 0
    assert torch.equal(dW, h.embed_grad(ids, dX, mask=keep))


def test_embed_grad_four_digits_of_many_tokens():
    """A vocabulary of 28 bits and more tokens than have their places counted; whole numbers."""
    V, T = 140_000_000, 8200
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    ids[::3] = V - 1
    dX = torch.randint(-4, 5, (T, 8), generator=g, device="cuda").float()
    h = ckl.ChunkedKL(V, 8, 1, dtype=torch.float32, max_chunk=1)
    dW = h.embed_grad(ids, dX)
    rows, back = torch.unique(ids, return_inverse=True)
    want = torch.zeros(len(rows), 8, device="cuda").index_add_(0, back, dX)
    assert torch.equal(dW[rows.long()], want)
    dW[rows.long()] = 0
    assert not dW.any()
    h.close()


@pytest.mark.parametrize("frozen", [False, True])
def test_autograd_embedding_without_a_gradient_reports_ids_out_of_range(frozen):
    """No backward pass will tell: the lookup itself waits and raises, and leaves no status that a later
    call with right ids would raise."""
    ids, mask, W, _ = case(40, 64, 31, "bf16", masked=True)
    W.requires_grad_(not frozen)
    wild = ids.clone()
    wild[mask.nonzero()[0]] = 31
    with torch.set_grad_enabled(frozen):
        with pytest.raises(ckl.CKLError) as e:
            ckl.embedding(wild, W, mask=mask)
        assert e.value.code == 4
        out = ckl.embedding(ids, W, mask=mask)
        assert not out.requires_grad
        assert torch.equal(out, ckl.operator_handle(W, V=31).embed(ids, W, mask=mask))
        quiet = ckl.embedding(wild, W, mask=mask, check=False)  # nothing waits: the status stays
    assert not quiet[mask.nonzero()[0]].any()
    with pytest.raises(ckl.CKLError):
        ckl.operator_handle(W, V=31).sync_status()


def test_autograd_embedding_without_a_gradient_in_a_capture():
    """What is captured waits for nothing, whatever `check` says; the status is there to ask for."""
    ids, _, W, _ = case(40, 64, 31, "bf16")
    with torch.no_grad():
        want = ckl.embedding(ids, W)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ckl.embedding(ids, W)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    ids[3] = 31
    g.replay()
    torch.cuda.synchronize()
    assert not out[3].any()
    with pytest.raises(ckl.CKLError):
        ckl.operator_handle(W, V=31).sync_status()
