"""The expert layer in 4 bits as a whole, against the layer of the values that its weights stand
for, in 64 bits."""
import pytest

from test_gpu_layer_few import MX, NV, held, make

import moe_expert_routing_ids_gb300 as topo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("T,E,k,R,slots,H,I", [(96, 8, 2, 4, 1, 128, 64), (200, 16, 4, 4, 2, 288, 160), (12, 4, 3, 2, 0, 256, 1056)])
def test_layer_as_a_whole(T, E, k, R, slots, H, I, fmt):
    """Only the rows x and the activations are rounded.  A value is off by a quarter of itself at
    most where it is at least its block's scale, by a quarter of the scale below: 0.144 of a row in
    2-norm at the worst place of its values between two scales.  Through silu(g) u the first counts
    1.5 times at most in 2-norm (g and u one time each, sqrt(2), and silu's slope of up to 1.1): with
    the second, independent of it, sqrt((1.5 * 0.144)^2 + 0.144^2) = 0.26.  A layer that lost a scale
    would be off by half and more: 0.35."""
    layer, x, logits, _ = make(T, E, k, R, slots, H, I, fmt)
    out = layer.forward(x, logits)
    assert layer.error() == 0
    if fmt == NV:                                                 # the activation's row scales, in the layer's buffer
        q, s, r = torch.empty_like(layer.aq), torch.empty_like(layer.as_), torch.empty_like(layer.ar)
        topo.topo_swiglu_quantize_micro(T * k, I, fmt, layer.h, q, s, r)
        assert torch.equal(r, layer.ar)
        g, u = layer.h[:, :I].double(), layer.h[:, I:].double()
        amax = (g * torch.sigmoid(g) * u).abs().amax(1)
        n = torch.log2(amax / 2688).ceil()                        # 2^-20 of it from a border it may be either
        near = (torch.log2(amax / 2688 * (1 - 2.0 ** -20)).ceil() != torch.log2(amax / 2688 * (1 + 2.0 ** -20)).ceil())
        assert bool(((layer.ar.double() == torch.exp2(n)) | near).all())
    ids, w = layer.ids[0].cpu().long(), layer.weights[0].cpu().double()
    vu, vd, xs = held(layer.up), held(layer.down), x.cpu().double()
    want = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            h = vu[ids[t, j]] @ xs[t]
            want[t] += w[t, j] * (vd[ids[t, j]] @ (torch.nn.functional.silu(h[:I]) * h[I:]))
    err = out.cpu().double() - want
    assert float(err.norm() / want.norm()) < 0.35
    few = layer.few(x[:12], logits[:12])                          # the same layer, its rows not rounded
    assert float((few.cpu().double() - want[:12]).norm() / want[:12].norm()) < 4 * (2.0 ** -11 + 2.0 ** -8)
