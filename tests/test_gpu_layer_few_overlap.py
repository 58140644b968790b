"""ExpertLayer.few on one layer by several streams and graphs at once: each call gets its own
result, bit for bit that of the call alone."""
import pytest

import moe_expert_routing_ids_gb300 as topo
from test_gpu_layer_few import EIGHT, MX, NV, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
SIZES = (1, 13, 4, 32)


def case(fmt):
    layer, x, logits, _ = make(64, 16, 4, 4, 1, 512, 256, fmt)
    ins = [(x[i:i + n].clone(), logits[i:i + n].clone()) for i, n in enumerate(SIZES)]
    want = [layer.few(*a).clone() for a in ins]
    torch.cuda.synchronize()
    return layer, ins, want


@pytest.mark.parametrize("fmt", [EIGHT, MX, NV])
def test_calls_on_several_streams(fmt):
    layer, ins, want = case(fmt)
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(5):
        got = [[] for _ in ins]
        for s in streams:                                         # all of them begin together
            with torch.cuda.stream(s):
                torch.cuda._sleep(3_000_000)
        for _ in range(20):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[i].append(layer.few(*ins[i]))
        torch.cuda.synchronize()
        assert all(torch.equal(g, want[i]) for i, gs in enumerate(got) for g in gs)
    assert layer.error() == 0


@pytest.mark.parametrize("fmt", [EIGHT, NV])
def test_graphs_replayed_beside_each_other_and_beside_calls(fmt):
    layer, ins, want = case(fmt)
    graphs, outs = [], []
    for a in ins[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([layer.few(*a) for _ in range(8)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        for os in outs:
            for o in os:
                o.zero_()
        torch.cuda.synchronize()
        for s in streams:
            with torch.cuda.stream(s):
                torch.cuda._sleep(3_000_000)
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = [layer.few(*ins[3]) for _ in range(8)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[i]) for i in (0, 1) for o in outs[i])
        assert all(torch.equal(o, want[3]) for o in eager)


def test_few_beside_a_forward():
    layer, x, logits, _ = make(64, 16, 4, 4, 1, 512, 256, MX)
    whole, part = layer.forward(x, logits).clone(), layer.few(x[:9], logits[:9]).clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for s in (a, b):
            with torch.cuda.stream(s):
                torch.cuda._sleep(3_000_000)
        ys, zs = [], []
        for _ in range(4):
            with torch.cuda.stream(a):
                ys.append(layer.forward(x, logits))
            with torch.cuda.stream(b):
                zs.append(layer.few(x[:9], logits[:9]))
        torch.cuda.synchronize()
        assert all(torch.equal(y, whole) for y in ys) and all(torch.equal(z, part) for z in zs)


def test_a_layer_holds_no_buffers_for_few():
    layer, x, logits, _ = make(16, 16, 4, 4, 1, 512, 256, EIGHT)
    held = sum(v.numel() * v.element_size() for v in vars(layer).values() if isinstance(v, torch.Tensor))
    layer.few(x[:2], logits[:2])
    now = sum(v.numel() * v.element_size() for v in vars(layer).values() if isinstance(v, torch.Tensor))
    assert now - held == 2 * 4 * 4                                # the last call's ids
