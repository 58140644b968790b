"""The expert layer with weights in 4 bits, and its call for a few tokens: each step of the
path against a plain float64 form of that step on the step's own input, and the whole
against the layer of the weights' values."""
import pytest

import moe_expert_routing_ids_gb300 as topo
from test_gpu_micro import values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
EIGHT, MX, NV = topo.TOPO_FMT_EIGHT, topo.TOPO_FMT_MX, topo.TOPO_FMT_NV


def make(T, E, k, R, slots, H, I, fmt, seed=0, stream=None, opts=None):
    from moe_expert_routing_ids_gb300.experts import ExpertLayer
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda:0")
    gen = torch.Generator().manual_seed(seed)
    up = (torch.randn(E, 2 * I, H, generator=gen) / H ** 0.5).to(torch.bfloat16).to(dev)
    down = (torch.randn(E, H, I, generator=gen) / I ** 0.5).to(torch.bfloat16).to(dev)
    x = torch.randn(T, H, generator=gen).to(torch.bfloat16).to(dev)
    logits = (torch.randn(T, E, generator=gen) + torch.linspace(1.5, 0, E)).to(dev)
    cfg = dict(T=T, E=E, k=k, R=R, ranks_per_node=2, n_slot=slots, tok_bytes=2 * H, expert_bytes=64, c_intra=1, c_inter=4)
    opts = opts or topo.make_route(topo.TOPO_SCORE_SOFTMAX, scale=1.5)
    return ExpertLayer(cfg, up, down, opts, stream=stream, fmt=fmt), x, logits, (up, down)


def held(w):
    """The values that a layer's weights stand for, float64 [E, N, K]."""
    if w.fmt == EIGHT:
        s = w.scale.double().repeat_interleave(128, 1)[:, :w.N].repeat_interleave(128, 2)[..., :w.K]
        return (w.q.view(torch.float8_e4m3fn).double() * s).cpu()
    return torch.as_tensor(values(w.q.cpu().numpy(), w.scale.cpu().numpy(), None if w.row is None else w.row.cpu().double().numpy(), w.fmt))


def near(got, want, A, K):
    """A bf16 product of the tensor cores (bounds of the products' own test)."""
    tol = (K / 64 + K / 8192 + 4) * 2.0 ** -23 * A + 2.0 ** -8 * want.abs()
    return bool(((got.double().cpu() - want).abs() <= tol).all())


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("T,E,k,R,slots,H,I", [(96, 8, 2, 4, 1, 128, 64), (640, 16, 4, 4, 2, 288, 160), (12, 4, 3, 2, 0, 256, 1056)])
def test_layer_in_four_bits(T, E, k, R, slots, H, I, fmt):
    layer, x, logits, _ = make(T, E, k, R, slots, H, I, fmt)
    out = layer.forward(x, logits)
    assert layer.error() == 0
    assert torch.equal(layer.forward(x, logits), out)
    P, rows = layer.planner, T * k

    def rows_of(q, s, r):
        return torch.as_tensor(values(q.cpu().numpy(), s.cpu().numpy(), None if r is None else r.cpu().double().numpy(), fmt))

    pair = P.buf.sorted_pairs[0].long()
    q, s = torch.empty_like(layer.xq), torch.empty_like(layer.xs)
    r = None if layer.xr is None else torch.empty_like(layer.xr)
    topo.topo_quantize_rows_micro(rows, H, fmt, x[pair // k].contiguous(), q, s, r)
    assert torch.equal(q, layer.xq) and torch.equal(s, layer.xs) and (r is None or torch.equal(r, layer.xr))
    off, seg = P.buf.seg_off[0].cpu().tolist(), layer.seg_w.reshape(-1).cpu().tolist()
    for w, a, got, K in ((held(layer.up), rows_of(q, s, r), layer.h, H), (held(layer.down), rows_of(layer.aq, layer.as_, layer.ar), layer.y, I)):
        for i, e in enumerate(seg):
            if off[i + 1] > off[i]:
                v = a[off[i]:off[i + 1]]
                assert near(got[off[i]:off[i + 1]], v @ w[e].T, v.abs() @ w[e].abs().T, K)
    q, s = torch.empty_like(layer.aq), torch.empty_like(layer.as_)
    r = None if layer.ar is None else torch.empty_like(layer.ar)
    topo.topo_swiglu_quantize_micro(rows, I, fmt, layer.h, q, s, r)
    assert torch.equal(q, layer.aq) and torch.equal(s, layer.as_)
    # combine: k terms in float32, rounded once
    y, wt = layer.y.double(), layer.weights.reshape(-1)[pair].double()[:, None]
    want = torch.zeros(T, H, dtype=torch.float64, device=x.device).index_add(0, pair // k, y * wt)
    mag = torch.zeros(T, H, dtype=torch.float64, device=x.device).index_add(0, pair // k, (y * wt).abs())
    assert bool(((out.double() - want).abs() <= (k + 1) * 2.0 ** -23 * mag + 2.0 ** -8 * want.abs()).all())


@pytest.mark.parametrize("fmt", [EIGHT, MX, NV])
@pytest.mark.parametrize("score,groups", [(topo.TOPO_SCORE_SOFTMAX, 1), (topo.TOPO_SCORE_SIGMOID, 4)])
def test_few_tokens_of_a_layer(fmt, score, groups):
    """In 2-norm: f16 activations and bf16 results leave 2^-11 and 2^-8 of the value at most;
    the sums cancel by less than a factor of four on these inputs' random signs."""
    opts = topo.make_route(score, groups, max(1, groups // 2), 1 if groups == 1 else 2, True, 1.5)
    layer, x, logits, _ = make(64, 16, 4, 4, 1, 288, 160, fmt, opts=opts)
    bias = torch.linspace(0.1, -0.1, 16, device=x.device) if groups > 1 else None
    layer.forward(x, logits, bias)
    ids, weights = layer.ids[0].cpu().long(), layer.weights[0].cpu().double()
    vu, vd = held(layer.up), held(layer.down)
    want = torch.zeros(64, 288, dtype=torch.float64)
    for t in range(64):
        for j in range(4):
            h = vu[ids[t, j]] @ x[t].cpu().double()
            want[t] += weights[t, j] * (vd[ids[t, j]] @ (torch.nn.functional.silu(h[:160]) * h[160:]))
    for n in (1, 2, 8, 13, 32):
        got = layer.few(x[:n], logits[:n], bias)
        assert layer.error() == 0 and got.shape == (n, 288) and got.dtype == torch.bfloat16
        assert torch.equal(layer.few_ids[:n].cpu().long(), ids[:n])
        assert float((got.double().cpu() - want[:n]).norm() / want[:n].norm()) < 4 * (2.0 ** -11 + 2.0 ** -8)
        assert torch.equal(layer.few(x[:n], logits[:n], bias), got)
    assert layer.few(x[:0], logits[:0], bias).shape == (0, 288)
    got = layer.few(x[:3], logits[:3].to(torch.bfloat16), bias)
    assert bool(torch.isfinite(got).all()) and layer.error() == 0


def test_few_after_set_weights_and_on_a_stream():
    s = torch.cuda.Stream() if torch.cuda.is_available() else None
    for fmt in (EIGHT, NV):
        plain, x, logits, (up, down) = make(32, 8, 2, 2, 0, 256, 128, fmt)
        layer, *_ = make(32, 8, 2, 2, 0, 256, 128, fmt, seed=9, stream=s)
        other = layer.few(x[:4], logits[:4])
        layer.set_weights(up, down)
        want = plain.few(x[:4], logits[:4])
        assert not torch.equal(other, want)
        for _ in range(3):
            late = torch.full_like(x[:4], float("nan"))
            torch.cuda._sleep(10_000_000)
            late.copy_(x[:4])
            got = layer.few(late, logits[:4])
            late.zero_()
            assert torch.equal(got, want)


def test_few_in_a_graph():
    layer, x, logits, _ = make(32, 16, 4, 2, 0, 512, 256, MX)
    want = [layer.few(x[8 * i:8 * i + 8], logits[8 * i:8 * i + 8]) for i in range(2)]
    src, lg = x[:8].clone(), logits[:8].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer.few(src, lg)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer.few(src, lg)
    for i in (1, 0, 1):
        src.copy_(x[8 * i:8 * i + 8])
        lg.copy_(logits[8 * i:8 * i + 8])
        g.replay()
        assert torch.equal(out, want[i])
    assert layer.error() == 0


def test_refusals_of_the_layer():
    layer, x, logits, (up, down) = make(64, 16, 4, 4, 0, 288, 160, MX)
    from moe_expert_routing_ids_gb300.experts import ExpertLayer, ExpertWeights
    cfg = layer.planner.cfg_dict
    with pytest.raises(ValueError):
        ExpertLayer(cfg, up, down, layer.route, train=True, fmt=MX)
    with pytest.raises(ValueError):
        ExpertLayer(cfg, up, down, layer.route, fmt=3)
    with pytest.raises(ValueError):
        ExpertWeights(up[:, :, :272].contiguous(), fmt=NV)
    with pytest.raises(RuntimeError):
        layer.backward(x, logits, x)
    with pytest.raises(ValueError):
        layer.few(x[:33], logits[:33])
    with pytest.raises(ValueError):
        layer.few(x[:4], logits[:3])
    with pytest.raises(ValueError):
        layer.few(x[:4, :256], logits[:4])
    with pytest.raises(ValueError):
        layer.few(x[:8:2], logits[:4])
    with pytest.raises(TypeError):
        layer.few(x[:4].float(), logits[:4])
    with pytest.raises(TypeError):
        layer.few(x[:4], logits[:4].double())
    with pytest.raises(ValueError):
        layer.few(x[:4].cpu(), logits[:4])
    with pytest.raises(ValueError):
        layer.few(x[0], logits[0])
