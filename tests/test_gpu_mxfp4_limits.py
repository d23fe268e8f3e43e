"""The MXFP4 layers on the longest rows they take (2^20 values), the balance statistics of
a long live batch, and workspaces that two captured graphs share.

References are in 64 bits, on the values that the codes stand for (whose encoding
test_gpu_mxfp4.py holds to the oracle bit for bit).  A product of k values adds in fp32,
where its sum is not exact, within (4 k / 128 + 16) 2^-23 of the sum of the magnitudes: four
blocks and one accumulation for every 128 values, and the joining of the waves' sums.
"""

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LONG = 1 << 20


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from block_diffusion_lm_tq4_amd import ops  # noqa: F401  (loads libtq4.so)
    return torch.device("cuda:0")


def _ops():
    from block_diffusion_lm_tq4_amd import ops
    return ops


def _randn(dev, *shape, gain=1.0, seed=0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return (gain * torch.randn(*shape, generator=g, device=dev)).to(torch.bfloat16)


def _values(rows):
    return _ops().mxfp4_values(*_ops().act_mxfp4(rows), rows.shape[1]).double()


@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_longest_rows(dev, m):
    o = _ops()
    n = 37
    x, w = _randn(dev, m, LONG, seed=m), _randn(dev, n, LONG, gain=0.02, seed=1)
    y = o.linear_mxfp4(x, o.mxfp4_cache_bf16(w), n).double()
    xv, wv = _values(x), _values(w).t().contiguous()
    want, size = torch.mm(xv, wv), torch.mm(xv.abs(), wv.abs())
    assert torch.all((y - want).abs() <= (4 * LONG / 128 + 16) * 2 * U * size)


@pytest.mark.parametrize("t", [3, 26, 200])
@pytest.mark.parametrize("k,n1", [(LONG, 32), (32, LONG)])
def test_moe_on_longest_rows(dev, t, k, n1):
    o = _ops()
    x = _randn(dev, t, k, seed=t)
    if k == LONG:  # the up sums of 2048 values, 512 apart, are exact: so are the hidden codes
        x[:, torch.arange(k, device=dev) % 512 != 511] = 0
    w1, w2 = _randn(dev, n1, k, gain=0.02, seed=1), _randn(dev, k, n1, gain=0.02, seed=2)
    ids = torch.zeros(t, 1, dtype=torch.int32, device=dev)
    gates = torch.rand(t, 1, device=dev)
    out = o.moe_grouped_mxfp4(x, ids, gates, o.mxfp4_cache_bf16(w1), o.mxfp4_cache_bf16(w2), 1,
                              n1).double()
    u = torch.mm(_values(x), _values(w1).t().contiguous()).float().clamp_min(0)
    h = O.mxfp4_values(*O.mxfp4_rows((u * u).cpu().numpy().astype(np.float64)))
    h, w = torch.from_numpy(h).to(dev), _values(w2).t().contiguous()
    want, size = gates * torch.mm(h, w), gates * torch.mm(h, w.abs())
    assert torch.all((out - want).abs() <= ((4 * n1 / 128 + 16) * 2 + 3) * U * size)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_of_a_million_tokens(dev, score):
    """A lane adds 64 scores in fp32, four lanes and then fp64: 68 roundings beside
    those of a score, 150 U for these logits."""
    o = _ops()
    t, e, topk = (1 << 20) + 3, 24, 4
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    l = torch.randn(t, e, generator=g, device=dev)
    ids = l.topk(topk, dim=1).indices.int()
    ids[::7] = -1
    loss, counts, tokens, mean = o.moe_balance(l, ids, score=score)
    live = ids[:, 0] >= 0
    p = torch.softmax(l[live].double(), 1) if score == "softmax" else torch.sigmoid(l[live].double())
    want = (p / p.sum(1, keepdim=True)).mean(0)
    count = torch.bincount(ids[live].flatten().long(), minlength=e)
    assert int(tokens) == int(live.sum()) and torch.equal(counts.long(), count)
    assert torch.all((mean.double() - want).abs() <= (150 + 68) * U * want)
    ref = float(e * (count.double() / count.sum() * want).sum())
    assert abs(float(loss) - ref) <= (150 + 68) * U * ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_weights_that_are_all_but_one(dev, score):
    """A renormalized weight is constant where a token has one slot, and nearly where one of
    its slots has nearly all of it: only what is left of the gradient may remain."""
    o = _ops()
    rng = np.random.default_rng(0)
    t, e = 60, 16
    l = rng.standard_normal((t, e)).astype(np.float32)
    lg = torch.from_numpy(l).to(dev)
    ids, _ = o.moe_router_scored(lg, 1, score=score, renormalize=True)
    loss, counts, tokens, _ = o.moe_balance(lg, ids, score=score)
    rest = dict(score=score, renormalize=True, scale=2.5, counts=counts, tokens=tokens, dloss=loss)
    one = o.moe_router_backward(lg, ids, torch.randn(t, 1, device=dev), **rest)
    assert torch.equal(one, o.moe_router_backward(lg, ids, torch.zeros(t, 1, device=dev), **rest))
    l[:, 0] = -40 if score == "sigmoid" else 0
    l[:, 1:] = l[:, :1] - 12 - np.arange(15, dtype=np.float32)
    i = np.tile(np.array([[1, 0, 2]], np.int32), (t, 1))
    d = rng.standard_normal((t, 3)).astype(np.float32)
    grad = o.moe_router_backward(torch.from_numpy(l).to(dev), torch.from_numpy(i).to(dev),
                                 torch.from_numpy(d).to(dev), score=score, renormalize=True)
    p = np.exp(l[:, :3].astype(np.float64) - l[:, :1])     # (sigmoid of -40: 1 + e^l is 1)
    u = p / p.sum(1, keepdims=True)
    by = d[:, [1, 0, 2]].astype(np.float64)
    diff = by[:, :, None] - by[:, None, :]                 # dw_j - dw_i
    want = u * (diff * u[:, None, :]).sum(2)
    size = u * (np.abs(diff) * u[:, None, :]).sum(2)
    # differences of logits up to 14: (4 * 14 + 160) roundings, as test_gpu_balance.py counts
    assert np.all(np.abs(grad[:, :3].double().cpu().numpy() - want) <= (4 * 14 + 160) * U * size)


def test_graphs_that_share_a_workspace(dev):
    """Two graphs on one stream with the same scratch memory, replayed in turn."""
    o = _ops()
    e, topk, k, n1 = 8, 2, 256, 96
    c1 = o.mxfp4_cache_bf16(_randn(dev, e * n1, k, gain=0.02, seed=1))
    c2 = o.mxfp4_cache_bf16(_randn(dev, e * k, n1, gain=0.02, seed=2))
    ts = (300, 700)
    ws = torch.empty(max(o.moe_grouped_mxfp4_workspace_size(t, topk, e, n1, k) for t in ts),
                     dtype=torch.uint8, device=dev)
    x = [_randn(dev, t, k, seed=t) for t in ts]
    l = [torch.randn(t, e, device=dev) for t in ts]

    def step(i):
        ids, gates = o.moe_router_scored(l[i], topk, renormalize=True)
        out = o.moe_grouped_mxfp4(x[i], ids, gates, c1, c2, e, n1, workspace=ws)
        loss, counts, tokens, mean = o.moe_balance(l[i], ids, workspace=ws)
        y = o.linear_mxfp4(x[i], c1, e * n1, workspace=ws)
        return out, y, loss, counts, mean, o.moe_router_backward(
            l[i], ids, gates, renormalize=True, counts=counts, tokens=tokens, dloss=loss)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0), step(1)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            outs.append(step(i))
    for seed in range(4):
        for i in (0, 1):
            x[i].copy_(_randn(dev, *x[i].shape, seed=50 + seed))
            l[i].copy_(torch.randn(l[i].shape, device=dev))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for i in (1, 0):
            for a, b in zip(outs[i], step(i)):
                assert torch.equal(a, b)
