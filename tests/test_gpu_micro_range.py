"""Rows and products in 4 bits at the ends of their ranges: gates near bf16's largest, row
scales whose product float32 does not hold, every scale byte."""
import numpy as np
import pytest

import moe_expert_routing_ids_gb300 as topo
from test_gpu_micro import BLOCK, E4M3, MX, NV, _dev, bf16, buffers, least_power, product, random_rows, segments, values

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


@gpu
@pytest.mark.parametrize("bf", [False, True])
@pytest.mark.parametrize("rows,n_seg,N,K", [(70, 1, 144, 288), (200, 3, 272, 96), (300, 20, 1040, 64)])
@pytest.mark.parametrize("ea,ew", [(-118, -40), (-126, -30), (120, -120), (-120, 118), (100, 20), (127, -126), (-140, 100), (-60, -70), (0, 0)])
def test_row_scales_whose_product_float32_does_not_hold(ea, ew, rows, n_seg, N, K, bf):
    """Any float32 row scales: out = ra rw sum.  The sum's bound is that of the products' own
    test; each scale is one multiplication (2^-24; a power of two taken out of it none), and
    what ends below float32's normal numbers is off by 2^-149 at most.  Sums past float32's
    range are infinite; rows and columns of a scale 0 stay 0."""
    dev = _dev()
    rng = np.random.default_rng([rows, N, abs(ea), abs(ew)])
    off = segments(rng, n_seg, rows)

    def scales(n, e):
        m = np.exp2(np.clip(e + rng.integers(-3, 4, n), -149, 127)) * np.where(rng.random(n) < 0.5, 1.0, rng.uniform(1, 1.9, n))
        return np.where(rng.random(n) < 0.05, 0.0, np.minimum(m, 3.4e38)).astype(np.float32)

    a, w = list(random_rows(rng, rows, K, NV)), list(random_rows(rng, n_seg * N, K, NV))
    a[2], w[2] = scales(rows, ea), scales(n_seg * N, ew)
    if rows > 100:
        a[2][40:100] = scales(60, 0)                          # rows of a warp with different ranges
    got, err = product(a, w, off, None, n_seg, N, K, NV, bf, dev)
    assert err == 0
    got = got.double().cpu()
    ones = (np.ones(rows, np.float32), np.ones(n_seg * N, np.float32))
    va = torch.as_tensor(values(a[0], a[1], ones[0], NV))
    vw = torch.as_tensor(values(w[0], w[1], ones[1], NV)).reshape(n_seg, N, K)
    ra, rw = torch.as_tensor(a[2]).double(), torch.as_tensor(w[2]).double().reshape(n_seg, N)
    for i in range(n_seg):
        r0, r1 = int(off[i]), int(off[i + 1])
        f = ra[r0:r1, None] * rw[i]
        want, A = (va[r0:r1] @ vw[i].T) * f, (va[r0:r1].abs() @ vw[i].abs().T) * f
        tol = (K / 64 + K / 8192 + 4) * 2.0 ** -23 * A + (2.0 ** -8 * want.abs() if bf else 0) + (2.0 ** -133 if bf else 2.0 ** -149)
        inside = (want.abs() + tol) < 3.38e38
        far = (want.abs() - tol) > 3.41e38
        g = got[r0:r1]
        assert not bool(torch.isnan(g).any())
        assert bool(((g - want).abs() <= tol)[inside].all())
        assert bool((g.abs() == float("inf"))[far].all()) and bool((torch.sign(g) == torch.sign(want))[far].all())


@gpu
@pytest.mark.parametrize("rows,n_seg,N,K", [(3, 1, 48, 32), (150, 2, 272, 288), (130, 1, 128, 1056), (70, 9, 1040, 544)])
@pytest.mark.parametrize("fmt,a_bytes,w_bytes", [(NV, (0, 127), (0, 127)), (NV, (0, 8), (0, 127)), (NV, (0, 127), (0, 8)), (NV, (0, 8), (0, 8)),
                                                 (MX, (0, 24), (231, 255)), (MX, (231, 255), (0, 24)), (MX, (87, 168), (87, 168)),
                                                 (MX, (1, 255), (127, 128)), (MX, (127, 128), (1, 252))])
def test_products_of_every_scale_byte(fmt, a_bytes, w_bytes, rows, n_seg, N, K):
    """Subnormal e4m3 scales and 0 (bytes below 8), powers of two to the ends.  The bound of the
    products' own test, of the terms' magnitudes: a product is 0 or far above 2^-149 but for the
    last two sets, where what is lost below float32's numbers is 2^-149 a product and more."""
    dev = _dev()
    rng = np.random.default_rng([rows, N, K, *a_bytes, *w_bytes])
    off = segments(rng, n_seg, rows)
    a, w = list(random_rows(rng, rows, K, fmt)), list(random_rows(rng, n_seg * N, K, fmt))
    for t, b in ((a, a_bytes), (w, w_bytes)):
        t[1][:, :K // BLOCK[fmt]] = rng.integers(*b, (len(t[1]), K // BLOCK[fmt]))
    got, err = product(a, w, off, None, n_seg, N, K, fmt, False, dev)
    assert err == 0
    got = got.double().cpu()
    va, vw = torch.as_tensor(values(*a, fmt)), torch.as_tensor(values(*w, fmt)).reshape(n_seg, N, K)
    for i in range(n_seg):
        r0, r1 = int(off[i]), int(off[i + 1])
        if r0 == r1:
            continue
        want, A = va[r0:r1] @ vw[i].T, va[r0:r1].abs() @ vw[i].abs().T
        tol = (K / 64 + K / 8192 + 4) * 2.0 ** -23 * A + K * 2.0 ** -149
        inside = A < 3.4e38                                       # a partial sum may pass float32's range
        g = got[r0:r1]
        assert bool(((g - want).abs() <= tol)[inside].all())
        assert bool(inside.any())
