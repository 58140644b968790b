"""Rows and products in 4 bits at the ends of their ranges."""
import numpy as np
import pytest

import moe_expert_routing_ids_gb300 as topo
from test_gpu_micro import BLOCK, E4M3, MX, NV, _dev, bf16, buffers, least_power, values

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows,I", [(9, 32), (13, 96), (40, 512), (21, 768), (12, 1408), (9, 2048), (9, 8192)])
def test_activation_of_gates_near_the_largest(rows, I, fmt):
    """silu(g) u is finite for gates past float32's largest over log2(e), 2.358e38, as long as
    the product is.  Such a gate's 1 + exp(-g) is 1: a product with u is all that is rounded,
    2^-24 of itself, below the bounds of the activation's own test (scale: 8 * 2^-24 of the
    value, value: half of e2m1's step and 11 * 2^-24)."""
    dev = _dev()
    rng = np.random.default_rng([rows, I, 23])
    h = bf16(rng.standard_normal((rows, 2 * I)) * 3)
    gates = [2.3e38, 2.36e38, 2.4e38, 3e38, 3.38e38, 1.7e38, 1e38, 128.0]
    for i, u in enumerate((0.5, -0.25, 2.0 ** -20, 2.0 ** -120, 0.0, 0.9)):
        for j, v in enumerate(gates):
            c = (j * 5 + i) % I
            h[i, c], h[i, I + c] = v, u
    h[6], h[6, :I] = 2.0 ** -127, 3.38e38                     # a whole row of them
    h[7, I - 1], h[7, 2 * I - 1] = float("inf"), 0.5          # not finite: its block's scale is NaN
    q, s, g = buffers(rows, I, fmt, dev)
    topo.topo_swiglu_quantize_micro(rows, I, fmt, h.to(dev), q, s, g)
    x = h.double().numpy()
    with np.errstate(over="ignore"):
        a = x[:, :I] / (1 + np.exp(-x[:, :I])) * x[:, I:]
    blk, d, dq = BLOCK[fmt], 8 * 2.0 ** -24, 11 * 2.0 ** -24
    p = a.reshape(rows, -1, blk)
    bad = ~np.isfinite(p).all(-1)
    assert bad.sum() == 1 and np.abs(a[np.isfinite(a)]).max() < 3.39e38
    p = np.where(bad[..., None], 0.0, p)
    mag = np.abs(p)
    amax = mag.max(-1)
    sb = s.cpu().numpy()[:, :I // blk]
    gs = np.ones(rows) if g is None else g.cpu().double().numpy()
    v = values(q.cpu().numpy(), s.cpu().numpy(), None if g is None else gs, fmt).reshape(p.shape)
    assert np.array_equal(np.isnan(v).all(-1), bad) and np.array_equal(np.isnan(v).any(-1), bad)
    if fmt == MX:
        sc = np.exp2(sb.astype(np.float64) - 127)
        ok = (sc == least_power(amax * (1 - d), 6.0)) | (sc == least_power(amax * (1 + d), 6.0))
    else:
        # the row's largest may lie beside an infinity, in the block that is NaN
        with np.errstate(invalid="ignore"):
            row = np.where(np.isfinite(a), np.abs(a), 0.0).max(1)
        assert np.all((gs == least_power(row * (1 - d), 2688.0)) | (gs == least_power(row * (1 + d), 2688.0)))
        e = E4M3[np.minimum(sb, 126)]
        lo = np.where(sb > 0, E4M3[np.maximum(sb.astype(int), 1) - 1], 0)
        sc = e * gs[:, None]
        ok = (amax == 0) | ((amax <= 6 * sc * (1 + d)) & (amax * (1 + d) >= 6 * lo * gs[:, None]))
    assert np.all(ok | bad)
    step = np.where(mag < 2 * sc[..., None], 0.25, np.where(mag < 4 * sc[..., None], 0.5, 1.0)) * sc[..., None]
    assert np.all((np.abs(v - p) <= step * (1 + d) + dq * mag) | bad[..., None])
