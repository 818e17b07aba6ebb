"""MoeLayer's gradient over token counts that change, eager and captured."""
import pytest
import torch

import sparse_mixture_experts_50_amd as moe
import workloads
from parity import device

pytestmark = pytest.mark.gpu


def make_layer(seed=1):
    w = workloads.scaled(
        workloads.get("deepseek_v3"), T=64, d=256, E=8, k=2, d_ff=256,
        dtype="bf16", n_shared=1, activation="swiglu", expert_bias="none",
        seed=seed)
    inp = workloads.make_inputs(w, device())
    return moe.MoeLayer(moe.Weights.from_dict(inp), w.k)


def tokens(T, seed):
    g = torch.Generator(device=device()).manual_seed(100 * T + seed)
    return [torch.randn(T, 256, generator=g, device=device()).bfloat16()
            for _ in range(2)]


def step(lay, x, dy):
    _, r = lay.forward(x)
    return lay.backward(x, r, dy, z_scale=0.1)


def test_changing_token_counts():
    """One layer over many token counts, up and down, gives what a layer of
    its own gives for each."""
    lay = make_layer()
    for i, T in enumerate((100, 3, 700, 100, 701, 1, 1500, 64)):
        x, dy = tokens(T, i)
        got = {n: t.clone() for n, t in step(lay, x, dy).as_dict().items()}
        want = step(make_layer(), x, dy).as_dict()
        assert sorted(got) == sorted(want)
        for n, t in want.items():
            assert torch.equal(got[n], t), (T, n)


def test_captured_step_outlives_larger_calls():
    """A captured step replays right after eager calls of more tokens have
    grown the layer's buffers, and leaves its results where they were."""
    dev, lay, T = device(), make_layer(), 96
    x, dy = tokens(T, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(lay, x, dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = step(lay, x, dy)
    for i, more in enumerate((500, 2000, 96, 40)):
        a, b = tokens(more, i)
        step(lay, a, b)
        filled = torch.full((1 << 20,), 7.0, device=dev)   # takes what is free
        xi, di = tokens(T, 10 + i)
        x.copy_(xi)
        dy.copy_(di)
        graph.replay()
        torch.cuda.synchronize()
        want = step(make_layer(), xi, di).as_dict()
        assert lay.grad_buffers(T)[1] is g
        for n, t in want.items():
            assert torch.equal(getattr(g, n), t), (more, n)
        assert bool((filled == 7.0).all())


def test_two_forwards_before_their_backwards():
    """As pipelining or a layer used twice runs them: with a clone of the
    first routing both backwards give what a layer of their own gives;
    without, the first one is refused."""
    lay = make_layer()
    (xa, da), (xb, db) = tokens(120, 1), tokens(120, 2)
    _, ra = lay.forward(xa)
    kept = ra.clone()
    _, rb = lay.forward(xb)
    with pytest.raises(ValueError, match="earlier forward"):
        lay.backward(xa, ra, da)
    for x, r, dy in ((xa, kept, da), (xb, rb, db)):
        got = {n: t.clone() for n, t in lay.backward(
            x, r, dy, z_scale=0.1).as_dict().items()}
        for n, t in step(make_layer(), x, dy).as_dict().items():
            assert torch.equal(got[n], t), n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act,shared", [("gelu", 0), ("silu", 1),
                                        ("swiglu", 0)])
def test_gradients_of_weights_that_the_layer_lacks(act, shared, dtype):
    """Wanted all the same they are zeros, also of calls that want nothing
    else."""
    dev, T, d, E, F = device(), 40, 128, 4, 128
    desc = moe.make_desc(T, d, E, 2, F, dtype, n_shared=shared,
                         activation=act)

    def z(*s):
        return torch.randn(s, device=dev).mul_(0.1).to(dtype)

    w = moe.Weights(z(E, d), z(E, F, d), z(E, d, F),
                    ws1=z(F, d) if shared else None,
                    ws2=z(d, F) if shared else None,
                    w3=z(E, F, d) if act == "swiglu" else None)
    lay = moe.MoeLayer(w, 2, activation=act)
    x, dy = z(T, d), z(T, d)
    _, r = lay.forward(x)
    want = {n: t.clone() for n, t in lay.backward(x, r, dy).as_dict().items()}
    lacks = ([] if act == "swiglu" else ["w3", "b3"]) + \
        ([] if shared else ["ws1", "bs1", "ws2", "bs2"]) + \
        ([] if shared and act == "swiglu" else ["ws3", "bs3"])
    ws = torch.empty(moe.moe_grad_workspace_size(desc), dtype=torch.uint8,
                     device=dev)
    for names in (lacks, [*lacks, *want], lacks[-1:]):
        g = moe.Grads(desc, dev, names)
        for t in g.as_dict().values():
            t.fill_(7.0)
        moe.moe_backward(desc, x, w, r, dy, g, ws, aux_scale=1.0)
        for n in names:
            got = getattr(g, n)
            if n in lacks:
                assert not got.any(), n
            else:
                assert torch.equal(got, want[n]), n
