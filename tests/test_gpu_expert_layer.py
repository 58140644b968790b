"""The expert layer's whole path on the planned layout, forward and backward,
against plain float64 expressions of the same layer.

Tolerances.  e4m3 rounds a value by at most 2^-4 of it, uniformly: 2^-4 /
sqrt(3) = 0.036 root mean square at the worst exponent position, 0.026 over all.
A product of two such operands sums independent errors: relative error in
2-norm about 0.037.  The forward pass chains two (the activation's error and
the second product's own): below 0.08; a gradient chains up to three more: below
0.15.  The router's gradient starts from dot products of y, with the error of the
forward pass."""
import numpy as np
import pytest

import moe_expert_routing_ids_gb300 as topo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _rel(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


@pytest.mark.parametrize("T,E,k,R,slots,H,I,score,groups,mapped", [
    (96, 8, 2, 4, 1, 128, 64, topo.TOPO_SCORE_SOFTMAX, 1, False),
    (640, 16, 4, 4, 2, 272, 144, topo.TOPO_SCORE_SIGMOID, 4, True),
    (1024, 4, 2, 2, 0, 256, 256, topo.TOPO_SCORE_SOFTMAX, 1, False)])
def test_layer_forward_and_backward(T, E, k, R, slots, H, I, score, groups, mapped):
    from moe_expert_routing_ids_gb300.experts import ExpertLayer
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda:0")
    gen = torch.Generator().manual_seed(T)
    w_up = (torch.randn(E, 2 * I, H, generator=gen) / H ** 0.5).to(torch.bfloat16)
    w_down = (torch.randn(E, H, I, generator=gen) / I ** 0.5).to(torch.bfloat16)
    x = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen) + torch.linspace(1.5, 0, E)
    dout = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    main = torch.randperm(E, generator=gen) % R if mapped else None
    cfg = dict(T=T, E=E, k=k, R=R, ranks_per_node=2, n_slot=slots, tok_bytes=2 * H, expert_bytes=64,
               c_intra=1, c_inter=4, max_refine_iters=0, main_rank=None if main is None else main.int().to(dev))
    opts = topo.make_route(score, groups, max(1, groups // 2), 1 if groups == 1 else 2, True, 1.5)
    bias = torch.zeros(E, device=dev) if groups > 1 else None
    layer = ExpertLayer(cfg, w_up.to(dev), w_down.to(dev), opts, train=True)
    xd, ld = x.to(dev), logits.to(dev)
    out = layer.forward(xd, ld, bias)
    assert layer.error() == 0
    first = out.clone()
    assert torch.equal(layer.forward(xd, ld, bias), first)
    ids = layer.ids[0].cpu().long()
    seg = layer.planner.buf.seg_off[0].cpu()
    if slots:
        assert (layer.seg_w >= 0).sum() > E                     # replicas are in use
    assert int(seg[-1]) == T * k

    xr, lr = x.double().requires_grad_(), logits.double().requires_grad_()
    ur, dr = w_up.double().requires_grad_(), w_down.double().requires_grad_()
    s = torch.softmax(lr, -1) if score == topo.TOPO_SCORE_SOFTMAX else torch.sigmoid(lr)
    w = torch.gather(s, 1, ids)
    w = w / w.sum(-1, keepdim=True) * 1.5
    want = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = xr[t] @ ur[e].T
        a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        want = want.index_add(0, t, (a @ dr[e].T) * w[t, j][:, None])
    assert _rel(out, want.detach()) < 0.08
    want.backward(dout.double())
    dx, dl, du, dd = layer.backward(xd, ld, dout.to(dev))
    assert layer.error() == 0
    assert _rel(dx, xr.grad) < 0.15
    assert _rel(du, ur.grad) < 0.15
    assert _rel(dd, dr.grad) < 0.15
    assert _rel(dl, lr.grad) < 0.15


def test_layer_shapes_are_checked():
    from moe_expert_routing_ids_gb300.experts import ExpertLayer
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda:0")
    cfg = dict(T=16, E=4, k=2, R=2, ranks_per_node=1, n_slot=0, tok_bytes=64, expert_bytes=64, c_intra=1, c_inter=1)
    up = torch.zeros(4, 64, 32, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        ExpertLayer(cfg, up, torch.zeros(4, 32, 16, dtype=torch.bfloat16, device=dev), topo.make_route(0))
    layer = ExpertLayer(cfg, up, torch.zeros(4, 32, 32, dtype=torch.bfloat16, device=dev), topo.make_route(0))
    x, lg = torch.zeros(16, 32, dtype=torch.bfloat16, device=dev), torch.zeros(16, 4, device=dev)
    assert float(layer.forward(x, lg).float().abs().max()) == 0.0
    with pytest.raises(RuntimeError):
        layer.backward(x, lg, x)
    with pytest.raises(TypeError):
        layer.planner.route(lg.double(), layer.ids, layer.weights, layer.route)
    assert np.array_equal(layer.planner.instance_experts().cpu().numpy(), [[0, 1, 2, 3]])


def _layer(T, E, k, R, slots, H, I, opts, seed=0, stream=None, hot=0.0):
    """A training layer and inputs x, logits (expert 0 ahead by hot), dout."""
    from moe_expert_routing_ids_gb300.experts import ExpertLayer
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda:0")
    gen = torch.Generator().manual_seed(seed)
    up = (torch.randn(E, 2 * I, H, generator=gen) / H ** 0.5).to(torch.bfloat16).to(dev)
    down = (torch.randn(E, H, I, generator=gen) / I ** 0.5).to(torch.bfloat16).to(dev)
    x = torch.randn(T, H, generator=gen).to(torch.bfloat16).to(dev)
    logits = torch.randn(T, E, generator=gen)
    logits[:, 0] += hot
    dout = torch.randn(T, H, generator=gen).to(torch.bfloat16).to(dev)
    cfg = dict(T=T, E=E, k=k, R=R, ranks_per_node=2, n_slot=slots, tok_bytes=2 * H, expert_bytes=64,
               c_intra=1, c_inter=4, max_refine_iters=0)
    if T % R:                                                   # ranks of unequal token counts
        cfg["rank_offsets"] = np.linspace(0, T, R + 1).astype(np.int64)
    return ExpertLayer(cfg, up, down, opts, train=True, stream=stream), x, logits.to(dev), dout


def test_layer_on_a_stream_of_its_own():
    """Built with a stream, the layer gives what it gives on the current one,
    whichever of the two is busy and however late the inputs come."""
    args = (640, 8, 2, 2, 1, 256, 128, topo.make_route(topo.TOPO_SCORE_SOFTMAX))
    plain, x, logits, dout = _layer(*args, hot=4.0)
    want = [plain.forward(x, logits).clone(), *plain.backward(x, logits, dout)]
    assert int((plain.seg_w >= 0).sum()) > 8                    # replicas are in use
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        torch.cuda._sleep(10_000_000)
        layer, *_ = _layer(*args, hot=4.0, stream=stream)
        for _ in range(3):
            late = [torch.full_like(v, float("nan")) for v in (x, logits, dout)]
            torch.cuda._sleep(10_000_000)
            for v, t in zip(late, (x, logits, dout)):
                v.copy_(t)
            with torch.cuda.stream(s):
                torch.cuda._sleep(10_000_000)
            got = [layer.forward(*late[:2]).clone(), *layer.backward(*late)]
            late = [v.zero_() for v in late]                    # the caller's next step on its tensors
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert layer.error() == 0
        assert torch.equal(layer.planner.instance_experts(), plain.planner.instance_experts())


def test_layer_arguments_are_checked():
    """Types, sizes, layouts and devices that a call would misread are refused;
    other strides and types of dout, which torch reads, are not."""
    from moe_expert_routing_ids_gb300.experts import ExpertLayer, ExpertWeights
    T, E, k, H, I = 64, 8, 2, 128, 64
    route = topo.make_route(topo.TOPO_SCORE_SIGMOID)
    layer, x, logits, dout = _layer(T, E, k, 4, 1, H, I, route)
    dev = x.device
    bias = torch.zeros(E, device=dev)
    want = layer.forward(x, logits, bias).clone()
    grads = layer.backward(x, logits, dout)
    assert torch.equal(layer.forward(x[None], logits[None], bias), want)

    def refused(kind, f, *args):
        with pytest.raises(kind):
            f(*args)

    short = torch.zeros(T - 1, H, dtype=torch.bfloat16, device=dev)
    for bad, kind in ((x.float(), TypeError), (None, TypeError), (x.half(), TypeError), (short, ValueError),
                      (x.t().contiguous().t(), ValueError), (x.t().contiguous(), ValueError), (x.cpu(), ValueError),
                      (torch.zeros(T, 2 * H, dtype=torch.bfloat16, device=dev)[:, :H], ValueError)):
        refused(kind, layer.forward, bad, logits)
        refused(kind, layer.backward, bad, logits, dout)
    for bad, kind in ((logits.double(), TypeError), (logits[:-1], ValueError), (logits[:, :4], ValueError),
                      (logits.t().contiguous().t(), ValueError), (logits.cpu(), ValueError)):
        refused(kind, layer.forward, x, bad)
        refused(kind, layer.backward, x, bad, dout)
    for bad, kind in ((bias.double(), TypeError), (bias[:4], ValueError), (bias.cpu(), ValueError)):
        refused(kind, layer.forward, x, logits, bad)
    for bad, kind in ((short, ValueError), (dout.long(), TypeError), (None, TypeError), (dout.cpu(), ValueError)):
        refused(kind, layer.backward, x, logits, bad)
    layer.forward(x, logits, bias)
    for same in (dout.float(), dout.t().contiguous().t(), dout[None]):
        assert all(torch.equal(a, b) for a, b in zip(layer.backward(x, logits, same), grads))

    P, ids, w = layer.planner, layer.ids, layer.weights
    for i, w_ in ((ids.long(), w), (ids, w.double()), (ids[:, 1:], w), (ids, w[:, 1:])):
        refused((TypeError, ValueError), P.route, logits, i, w_, route)
    refused(ValueError, P.route_grad, logits, ids, w[:, 1:], torch.empty_like(logits), route)
    refused(TypeError, P.route_grad, logits, ids, w, torch.empty_like(logits, dtype=torch.bfloat16), route)

    up = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device=dev)
    down = torch.zeros(E, H, I, dtype=torch.bfloat16, device=dev)
    cfg = dict(T=T, E=E, k=k, R=4, ranks_per_node=2, n_slot=1, tok_bytes=64, expert_bytes=64, c_intra=1, c_inter=1)
    for u, d, kind in ((up.float(), down, TypeError), (up, down.float(), TypeError), (up.cpu(), down, ValueError),
                       (up, down.cpu(), ValueError), (up.transpose(1, 2).contiguous().transpose(1, 2), down, ValueError),
                       (up[:4], down[:4], ValueError), (up[0], down, ValueError)):
        refused(kind, ExpertLayer, cfg, u, d, route)
    refused(TypeError, ExpertWeights, up.float())
    refused(ValueError, ExpertWeights, up[0])
    refused(ValueError, ExpertWeights, up.cpu())
    assert layer.error() == 0


def test_backward_repeats_bit_for_bit():
    """Four instances of one expert: their weight gradients are added in one order."""
    layer, x, logits, dout = _layer(2048, 8, 2, 8, 1, 256, 128, topo.make_route(topo.TOPO_SCORE_SOFTMAX), hot=6.0)
    layer.forward(x, logits)
    assert int((layer.seg_w == 0).sum()) >= 4
    first = [g.clone() for g in layer.backward(x, logits, dout)]
    for _ in range(8):
        for a, b in zip(layer.backward(x, logits, dout), first):
            assert torch.equal(a, b)
    assert layer.error() == 0


def test_weight_gradients_of_instances_are_added_in_order(monkeypatch):
    """An expert's gradient is its main instance's plus its replicas', by rank."""
    from moe_expert_routing_ids_gb300 import experts
    layer, x, logits, dout = _layer(2048, 8, 2, 8, 2, 256, 128, topo.make_route(topo.TOPO_SCORE_SOFTMAX), hot=6.0)
    layer.forward(x, logits)
    seen, call = [], experts.topo_expert_wgrad

    def watched(*args):
        call(*args)
        seen.append(args[10].clone())

    monkeypatch.setattr(experts, "topo_expert_wgrad", watched)
    *_, up, down = layer.backward(x, logits, dout)
    seg = layer.seg_w.reshape(8, -1).cpu()
    nm = 1                                                      # mains of a rank
    assert int((seg == 0).sum()) >= 4
    for inst, got in zip(seen, (down, up)):
        inst = inst.reshape(8, seg.shape[1], *inst.shape[1:])
        for e in range(8):
            want = inst[e, 0]
            for r in range(8):
                for j in range(nm, seg.shape[1]):
                    if seg[r, j] == e:
                        want = want + inst[r, j]
            assert torch.equal(got[e], want)
    assert layer.error() == 0


def test_an_output_outlives_the_next_call():
    layer, x, logits, _ = _layer(64, 8, 2, 4, 1, 128, 64, topo.make_route(topo.TOPO_SCORE_SOFTMAX))
    a = layer.forward(x, logits)
    kept = a.clone()
    b = layer.forward(-x, logits)
    assert torch.equal(a, kept) and not torch.equal(a, b)


@pytest.mark.parametrize("own", [False, True])
def test_new_weights(own):
    """set_weights gives what a layer built from those weights gives."""
    args = (96, 8, 2, 4, 1, 128, 64, topo.make_route(topo.TOPO_SCORE_SIGMOID))
    stream = torch.cuda.Stream() if own and torch.cuda.is_available() else None
    layer, x, logits, dout = _layer(*args, stream=stream)
    other = _layer(*args, seed=1)[0]
    gen = torch.Generator().manual_seed(1)                      # the weights of seed 1
    up = (torch.randn(8, 128, 128, generator=gen) / 128 ** 0.5).to(torch.bfloat16).to(x.device)
    down = (torch.randn(8, 128, 64, generator=gen) / 64 ** 0.5).to(torch.bfloat16).to(x.device)
    before = layer.forward(x, logits)
    layer.set_weights(up, down)
    got = [layer.forward(x, logits), *layer.backward(x, logits, dout)]
    want = [other.forward(x, logits), *other.backward(x, logits, dout)]
    assert not torch.equal(before, got[0])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for u, d, kind in ((up.float(), down, TypeError), (up[:4], down[:4], ValueError), (up, down.transpose(1, 2), ValueError),
                       (up.cpu(), down, ValueError)):
        with pytest.raises(kind):
            layer.set_weights(u, d)
    assert layer.error() == 0


@pytest.mark.parametrize("T,E,k,R,score,groups,renorm,bf16", [
    (384, 16, 4, 4, topo.TOPO_SCORE_SOFTMAX, 4, True, False), (384, 16, 4, 4, topo.TOPO_SCORE_SOFTMAX, 4, False, True),
    (200, 8, 3, 2, topo.TOPO_SCORE_SIGMOID, 1, False, True), (1, 8, 2, 4, topo.TOPO_SCORE_SIGMOID, 1, True, False)])
def test_layer_with_other_routers(T, E, k, R, score, groups, renorm, bf16):
    """Softmax with groups, weights that are shares of the whole row, logits in
    bf16, one token; the gradient of bf16 logits is rounded to 2^-9 of itself."""
    H, I, scale = 256, 128, 2.0
    top = 2 if groups > 1 else 1
    layer, x, logits, dout = _layer(T, E, k, R, 1, H, I, topo.make_route(score, groups, max(1, groups // 2), top, renorm, scale),
                                    hot=1.0)
    if bf16:
        logits = logits.to(torch.bfloat16)
    out = layer.forward(x, logits)
    dx, dl, du, dd = layer.backward(x, logits, dout)
    assert layer.error() == 0 and dl.dtype == logits.dtype
    gen = torch.Generator().manual_seed(0)                      # the weights again
    ur = (torch.randn(E, 2 * I, H, generator=gen) / H ** 0.5).to(torch.bfloat16).double().requires_grad_()
    dr = (torch.randn(E, H, I, generator=gen) / I ** 0.5).to(torch.bfloat16).double().requires_grad_()
    xr, lr = x.double().cpu().requires_grad_(), logits.double().cpu().requires_grad_()
    ids = layer.ids[0].cpu().long()
    s = torch.softmax(lr, -1) if score == topo.TOPO_SCORE_SOFTMAX else torch.sigmoid(lr)
    w = torch.gather(s, 1, ids)
    w = (w / w.sum(-1, keepdim=True) if renorm else w) * scale
    want = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = xr[t] @ ur[e].T
        want = want.index_add(0, t, (torch.nn.functional.silu(h[:, :I]) * h[:, I:] @ dr[e].T) * w[t, j][:, None])
    assert _rel(out, want.detach()) < 0.08
    want.backward(dout.double().cpu())
    for got, ref in ((dx, xr.grad), (dl, lr.grad), (du, ur.grad), (dd, dr.grad)):
        assert _rel(got, ref) < 0.15


def test_layer_without_tokens():
    layer, x, logits, dout = _layer(0, 8, 2, 4, 1, 128, 64, topo.make_route(topo.TOPO_SCORE_SOFTMAX))
    assert layer.forward(x, logits).shape == (0, 128)
    dx, dl, du, dd = layer.backward(x, logits, dout)
    assert dx.shape == (0, 128) and dl.shape == (0, 8)
    assert torch.all(du == 0) and torch.all(dd == 0) and du.shape == (8, 128, 128) and dd.shape == (8, 128, 64)
    assert layer.error() == 0
