"""GPU: two layers from logits to output, and two routings' gradients, on two streams at once, with nothing
waiting between them: each bit for bit what it gives alone."""
import pytest
import torch

from gpu_helpers import say
from test_gpu_route_mx_use import FORMS, Layer, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


@pytest.mark.parametrize("i,j", [(0, 1), (1, 3), (2, 2), (3, 3), (2, 3)])
def test_two_layers(moe, i, j):
    say(f"[mx layer] {FORMS[i]} beside {FORMS[j]}")
    layers = [Layer(moe, 70 + n, **FORMS[f]) for n, f in enumerate((i, j))]
    want = []
    for L in layers:
        L.run()
        torch.cuda.synchronize()
        want.append(L.results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        for L in layers:
            for t in (L.hid, L.hs, L.y, L.out, L.wts, L.ids):
                t.fill_(7)
        torch.cuda.synchronize()
        for _ in range(8):  # (calls of both in turn, so that they overlap)
            for L, s in zip(layers, streams):
                L.run(stream=s)
        torch.cuda.synchronize()
        for L, res in zip(layers, want):
            assert all(same(a, b) for a, b in zip(res, L.results())), turn


def test_two_gradients(moe):
    n, e, k = 9000, 128, 8
    g = torch.Generator("cuda").manual_seed(8)
    p, r = moe.problem(n, 8, k, e, 1), moe.router("sigmoid")
    sets = []
    for _ in range(2):
        l = torch.randn(n, e, generator=g, device="cuda")
        ids = torch.argsort(l, dim=1, descending=True)[:, :k].int().contiguous()
        dw, ds = torch.randn(n, k, generator=g, device="cuda"), torch.randn(n, e, generator=g, device="cuda")
        sets.append((l, ids, torch.zeros_like(l), dw, ds))
    want = []
    for l, ids, dl, dw, ds in sets:
        moe.moe_route_backward(p, r, l, ids, dl, dweights=dw, dscores=ds)
        torch.cuda.synchronize()
        want.append(dl.clone())
        dl.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (l, ids, dl, dw, ds), s in zip(sets, streams):
            moe.moe_route_backward(p, r, l, ids, dl, dweights=dw, dscores=ds, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(s[2], w) for s, w in zip(sets, want))
