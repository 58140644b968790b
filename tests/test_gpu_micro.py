"""Rows and weights in microscaled 4 bits against the formulas in 64 bits: the
quantised codes and scales exactly, the values they stand for, the experts'
products, and the refusals of arguments.

A product's float32 sum of K terms is compared to the sum of the terms'
magnitudes A: the tensor core adds 64 products at a time with at least 24 bits
below the largest, sums of 8192 values are added in float32, and the two row
scales are one multiplication each: |error| <= (K / 64 + K / 8192 + 4) * 2^-23 * A;
a bf16 output adds 2^-8 of the value."""
import numpy as np
import pytest

import moe_expert_routing_ids_gb300 as topo

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
MX, NV = topo.TOPO_FMT_MX, topo.TOPO_FMT_NV
BLOCK = {MX: 32, NV: 16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def e4m3_values():
    i = np.arange(127)
    e, m = i >> 3, i & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))


E4M3 = e4m3_values()


def least_power(amax, top):
    """Smallest power of two s (exponent at least -126) with amax <= top * s; 1 for 0."""
    s = np.full(amax.shape, 2.0 ** -126)
    while np.any(s * top < amax):
        s = np.where(s * top < amax, s * 2, s)
    return np.where(amax > 0, s, 1.0)


def to_e2m1(y):
    """Codes of y (float64): nearest, ties to the even code."""
    a = np.abs(y)
    d = np.abs(a[..., None] - E2M1)
    lo = d.argmin(-1)                                         # the lower of two that are as near
    hi = np.minimum(lo + 1, 7)
    tie = (np.take_along_axis(d, lo[..., None], -1) == np.take_along_axis(d, hi[..., None], -1))[..., 0] & (hi > lo)
    return (np.where(tie & (lo % 2 == 1), hi, lo) | np.where(np.signbit(y), 8, 0)).astype(np.uint8)


def quant(v, fmt):
    """v float64 [rows, C]: packed codes, scale bytes [rows, pitch], row scales, and blocks that are NaN."""
    rows, C = v.shape
    blk = BLOCK[fmt]
    p = v.reshape(rows, C // blk, blk)
    fin = np.isfinite(p)
    bad = ~fin.all(-1)
    mag = np.where(fin, np.abs(p), 0.0)
    amax = mag.max(-1)
    sb = np.full((rows, topo.topo_micro_pitch(C, fmt)), 127 if fmt == MX else 0x38, np.uint8)
    if fmt == MX:
        s = np.where(bad, 1.0, least_power(amax, 6.0))
        sb[:, :C // blk] = np.where(bad, 255, 127 + np.log2(s))
        g = None
    else:
        g = least_power(mag.max((1, 2)), 6.0 * 448.0)
        code = np.searchsorted(E4M3, amax / g[:, None] / 6.0)
        # the quotient by 6 is rounded: the code is the least with amax <= 6 s g
        code = np.where((code > 0) & (6 * E4M3[np.maximum(code, 1) - 1] * g[:, None] >= amax), code - 1, code)
        code = np.where(6 * E4M3[np.minimum(code, 126)] * g[:, None] < amax, code + 1, code)
        code = np.where(amax > 0, code, 0x38)
        s = E4M3[np.minimum(code, 126)] * g[:, None]
        sb[:, :C // blk] = np.where(bad, 0x7f, code)
    with np.errstate(invalid="ignore"):
        q = to_e2m1(np.where(fin, p, 0.0) / s[..., None]).reshape(rows, C)
    return q[:, ::2] | (q[:, 1::2] << 4), sb, g, bad


def values(q, sb, g, fmt):
    """Float64 values of packed rows (any leading shape)."""
    c = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    blk = BLOCK[fmt]
    sb = sb[..., :c.shape[-1] // blk]
    if fmt == MX:
        s = np.where(sb == 255, np.nan, np.exp2(sb.astype(np.float64) - 127))
    else:
        s = np.where((sb & 127) == 127, np.nan, E4M3[np.minimum(sb & 127, 126)] * np.where(sb & 128, -1.0, 1.0)) * g[..., None]
    return v * np.repeat(s, blk, -1)


def bf16(v):
    return torch.as_tensor(v.astype(np.float32)).to(torch.bfloat16)


def hard_rows(rng, rows, C):
    """Rows over many magnitudes with zeros, NaN, infinities, subnormals, ties and block maxima on the scales' edges."""
    v = rng.standard_normal((rows, C)) * np.exp(rng.standard_normal((rows, 1)) * 4)
    v = bf16(v).float().numpy().astype(np.float64)
    v[:, ::7] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6], (rows, len(range(0, C, 7))))
    if rows > 10:
        v[0] = 0.0
        v[1, 5] = np.nan
        v[2, C - 1] = np.inf
        v[3] = -np.inf
        v[4] = 2.0 ** -133                                    # subnormal bf16
        v[5] = 6.0 * 2.0 ** -3
        v[6] = 6.0625
        v[7] = 3.3e38
        v[8] = -2.0 ** -126
        v[9, :16] *= 2.0 ** -12                               # a block far below its row's largest
        v[10, 1:] = 0.0
    if rows > 16:
        v[11, 0], v[11, 16:32] = 3e38, 2.0 ** -130            # a quotient that underflows
        v[12, :16] = 2.0 ** -115 * 3                          # the quotients' own scaling
        v[13] = np.ldexp(v[14] / np.abs(v[14]).max(), -118)
    with np.errstate(over="ignore", invalid="ignore"):
        return bf16(v).double().numpy()                       # the oracle's values are those that the call gets


def buffers(rows, C, fmt, dev):
    return (torch.full((rows, C // 2), 0x55, dtype=torch.uint8, device=dev),
            torch.full((rows, topo.topo_micro_pitch(C, fmt)), 0xEE, dtype=torch.uint8, device=dev),
            torch.full((rows,), -1.0, device=dev) if fmt == NV else None)


def check_rows(v, q, s, g, fmt):
    wq, ws, wg, bad = quant(v, fmt)
    assert np.array_equal(s.cpu().numpy(), ws)
    if fmt == NV:
        assert np.array_equal(g.cpu().numpy().astype(np.float64), wg)
    keep = np.repeat(~bad, BLOCK[fmt] // 2, -1)               # the codes of a NaN block are not fixed
    assert np.array_equal(q.cpu().numpy()[keep], wq[keep])


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows,C", [(1, 32), (3, 128), (17, 160), (40, 1408), (11, 7168), (700, 288), (20000, 64), (5000, 1056), (19, 20512)])
def test_quantize_rows(rows, C, fmt):
    dev = _dev()
    v = hard_rows(np.random.default_rng([rows, C]), rows, C)
    q, s, g = buffers(rows, C, fmt, dev)
    topo.topo_quantize_rows_micro(rows, C, fmt, bf16(v).to(dev), q, s, g)
    check_rows(v, q, s, g, fmt)


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("L,T,k,H", [(1, 1, 1, 32), (1, 5, 8, 7168), (2, 33, 3, 288), (1, 100, 40, 160), (2, 4097, 2, 1024),
                                     (1, 2100, 40, 1056)])
def test_permute_quantize(L, T, k, H, fmt):
    dev = _dev()
    rng = np.random.default_rng([L, T, k, H])
    v = hard_rows(rng, L * T, H)
    sp = np.stack([rng.permutation(T * k) for _ in range(L)]).astype(np.int32)
    cfg = topo.make_cfg(T=T, E=8, k=k, R=1, ranks_per_node=1, n_slot=0)
    nb = topo.topo_workspace_bytes(cfg, L, topo.TOPO_CALL_PACK)
    ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
    q, s, g = buffers(L * T * k, H, fmt, dev)
    topo.topo_permute_quantize_micro(cfg, L, H, fmt, bf16(v).to(dev), torch.as_tensor(sp, device=dev), q, s, g, ws, nb)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == 0
    a, b, c = buffers(L * T, H, fmt, dev)
    topo.topo_quantize_rows_micro(L * T, H, fmt, bf16(v).to(dev), a, b, c)
    at = torch.as_tensor((np.arange(L)[:, None] * T + sp // k).reshape(-1), device=dev)
    assert torch.equal(s, b[at])
    if fmt == NV:
        assert torch.equal(g, c[at])
    assert torch.equal(q, a[at])                              # (tested against the formulas above)


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("T,H", [(64, 64), (3000, 1024)])
def test_permute_quantize_reports_bad_pairs(T, H, fmt):
    dev = _dev()
    k = 2
    cfg = topo.make_cfg(T=T, E=8, k=k, R=1, ranks_per_node=1, n_slot=0)
    nb = topo.topo_workspace_bytes(cfg, 1, topo.TOPO_CALL_PACK)
    ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
    sp = torch.arange(T * k, dtype=torch.int32, device=dev)
    sp[5] = T * k
    q, s, g = buffers(T * k, H, fmt, dev)
    topo.topo_permute_quantize_micro(cfg, 1, H, fmt, torch.zeros(T, H, dtype=torch.bfloat16, device=dev), sp, q, s, g, ws, nb)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == topo.TOPO_ESTATE


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows,I", [(1, 32), (37, 160), (333, 1408), (5000, 288), (3, 8192), (2000, 6688)])
def test_swiglu_quantize(rows, I, fmt):
    """a is formed in float32: 2^x within 2^-22.5 (2.9 * 2^-24) and four more roundings of 2^-24,
    the reciprocal's step another: within 8 * 2^-24 of itself (d); expf within 2 units in the last
    place (4 * 2^-24), a sum, a quotient and a product stay below that too.  A scale then is that of
    an amax within d.  The quotient by a scale is a product with its approximate inverse, one unit
    in the last place and a rounding: 3 * 2^-24 more, so a code's value is within half of e2m1's
    step (0.25 below 2, 0.5 below 4, 1 above) and 11 * 2^-24 of the value (dq)."""
    dev = _dev()
    rng = np.random.default_rng([rows, I, 7])
    h = bf16(rng.standard_normal((rows, 2 * I)) * 3)
    h[0] = 0
    if rows > 4:
        h[1, :3] = torch.tensor([-200.0, 80.0, -88.5])
        h[2, 4] = float("nan")
        h[3, I + 40] = float("inf")
    q, s, g = buffers(rows, I, fmt, dev)
    topo.topo_swiglu_quantize_micro(rows, I, fmt, h.to(dev), q, s, g)
    x = h.double().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        a = x[:, :I] / (1 + np.exp(-x[:, :I])) * x[:, I:]
    blk, d, dq = BLOCK[fmt], 8 * 2.0 ** -24, 11 * 2.0 ** -24
    p = a.reshape(rows, -1, blk)
    bad = ~np.isfinite(p).all(-1)
    mag = np.where(np.isfinite(p), np.abs(p), 0.0)
    q, sb = q.cpu().numpy(), s.cpu().numpy()
    assert np.all(np.isnan(values(q, sb, g.cpu().double().numpy() if g is not None else None, fmt)).reshape(rows, -1, blk).all(-1) == bad)
    amax = mag.max(-1)
    if fmt == MX:
        sc = np.exp2(sb[:, :I // blk].astype(np.float64) - 127)
        ok = (sc == least_power(amax * (1 - d), 6.0)) | (sc == least_power(amax * (1 + d), 6.0))
        assert np.all(ok | bad)
        sc = np.where(bad, 1.0, sc)
    else:
        gs = g.cpu().double().numpy()
        row = mag.max((1, 2))
        assert np.all((gs == least_power(row * (1 - d), 2688.0)) | (gs == least_power(row * (1 + d), 2688.0)))
        e = E4M3[np.minimum(sb[:, :I // blk], 126)]
        lo = np.where(sb[:, :I // blk] > 0, E4M3[np.maximum(sb[:, :I // blk].astype(int), 1) - 1], 0)
        inside = (amax <= 6 * e * gs[:, None] * (1 + d)) & (amax * (1 + d) >= 6 * lo * gs[:, None])
        assert np.all(inside | bad | (amax == 0))
        sc = np.where(bad, 1.0, e * gs[:, None])
    v = np.nan_to_num(values(q, sb, g.cpu().double().numpy() if g is not None else None, fmt)).reshape(p.shape)
    step = np.where(mag < 2 * sc[..., None], 0.25, np.where(mag < 4 * sc[..., None], 0.5, 1.0)) * sc[..., None]
    with np.errstate(invalid="ignore"):
        err = np.abs(v - p)
    assert np.all((err <= step * (1 + d) + dq * mag) | bad[..., None])


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows,C", [(513, 32), (2, 64), (257, 96), (65, 128), (130, 256), (33, 480), (4099, 512), (18, 544)])
def test_quantize_narrow_rows(rows, C, fmt):
    """Several rows to a warp, the last warp's not all there."""
    test_quantize_rows(rows, C, fmt)


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("L,T,k,H", [(1, 3, 2, 64), (2, 35, 5, 96), (1, 70001, 2, 32), (2, 9000, 40, 224), (1, 16385, 3, 128)])
def test_permute_quantize_narrow_rows(L, T, k, H, fmt):
    test_permute_quantize(L, T, k, H, fmt)


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("T,H", [(65, 32), (16400, 128)])
def test_permute_quantize_narrow_rows_leaves_bad_pairs(T, H, fmt):
    """A pair out of range: an error, and no row of it or its token; the others are there."""
    dev = _dev()
    rng = np.random.default_rng([T, H, 3])
    k, by_token = 2, T * H * 2 > 4 << 20
    cfg = topo.make_cfg(T=T, E=8, k=k, R=1, ranks_per_node=1, n_slot=0)
    nb = topo.topo_workspace_bytes(cfg, 1, topo.TOPO_CALL_PACK)
    ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
    x = bf16(hard_rows(rng, T, H)).to(dev)
    sp = rng.permutation(T * k).astype(np.int32)
    lost = sp[5] // k
    sp[5] = T * k + 7
    q, s, g = buffers(T * k, H, fmt, dev)
    topo.topo_permute_quantize_micro(cfg, 1, H, fmt, x, torch.as_tensor(sp, device=dev), q, s, g, ws, nb)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == topo.TOPO_ESTATE
    a, b, c = buffers(T, H, fmt, dev)
    topo.topo_quantize_rows_micro(T, H, fmt, x, a, b, c)
    keep = np.arange(T * k) != 5
    if by_token:
        keep &= sp // k != lost
    at, rows = torch.as_tensor(sp[keep] // k, dtype=torch.int64, device=dev), torch.as_tensor(np.flatnonzero(keep), device=dev)
    assert torch.equal(q[rows], a[at]) and torch.equal(s[rows], b[at])
    assert fmt == MX or torch.equal(g[rows], c[at])
    if not by_token:
        assert bool((q[5] == 0x55).all()) and bool((s[5] == 0xEE).all())


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows,I", [(4, 32), (300, 64), (33, 96), (129, 256), (70, 480), (600, 512), (9, 544), (40, 768), (21, 1536),
                                    (11, 2560), (7, 6144)])
def test_swiglu_quantize_narrow_rows_and_three_groups_to_a_lane(rows, I, fmt):
    test_swiglu_quantize(rows, I, fmt)
    dev = _dev()
    q, s, g = buffers(rows, I, fmt, dev)
    topo.topo_swiglu_quantize_micro(rows, I, fmt, torch.ones(rows, 2 * I, dtype=torch.bfloat16, device=dev), q, s, g)
    assert bool((s[:, I // BLOCK[fmt]:] == (127 if fmt == MX else 0x38)).all())
    n = 1041                                                  # a row's values do not depend on its place
    h = (torch.randn(n, 2 * I, generator=torch.Generator().manual_seed(I)) * 3).to(torch.bfloat16).to(dev)
    whole = buffers(n, I, fmt, dev)
    topo.topo_swiglu_quantize_micro(n, I, fmt, h, *whole)
    for at in (0, 1, 515, n - 4):
        four = buffers(4, I, fmt, dev)
        topo.topo_swiglu_quantize_micro(4, I, fmt, h[at:at + 4], *four)
        for x, y in zip(whole, four):
            assert x is None or torch.equal(x[at:at + 4], y)


@gpu
def test_quantised_rows_in_the_order_of_any_launch():
    """Rows split over warps and whole rows give the same bytes."""
    dev = _dev()
    v = bf16(hard_rows(np.random.default_rng(1), 3000, 7168)).to(dev)
    for fmt in (MX, NV):
        a, b = buffers(3000, 7168, fmt, dev), buffers(3000, 7168, fmt, dev)
        topo.topo_quantize_rows_micro(3000, 7168, fmt, v, *a)
        for r in range(0, 3000, 300):
            topo.topo_quantize_rows_micro(300, 7168, fmt, v[r:r + 300], *(t if t is None else t[r:r + 300] for t in b))
        assert all(x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
def test_dequantize_every_code_and_scale(fmt):
    dev = _dev()
    rows, C = 256, 512
    rng = np.random.default_rng(3)
    q = np.tile(np.arange(256, dtype=np.uint8), (rows, 1))
    sb = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, topo.topo_micro_pitch(C, fmt)))
    g = np.exp2(rng.integers(-20, 20, rows)).astype(np.float32) if fmt == NV else None
    out = torch.empty(rows, C, dtype=torch.bfloat16, device=dev)
    topo.topo_dequantize_micro(rows, C, fmt, torch.as_tensor(q, device=dev), torch.as_tensor(sb, device=dev),
                               None if g is None else torch.as_tensor(g, device=dev), out)
    want = values(q, sb, None if g is None else g.astype(np.float64), fmt)
    got = out.cpu().double().numpy()
    with np.errstate(over="ignore"):
        want = torch.as_tensor(want.astype(np.float32)).to(torch.bfloat16).double().numpy()   # past bf16's range only
    assert np.array_equal(got, want, equal_nan=True)


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows,C", [(1, 32), (35, 32), (4097, 96), (700, 160), (33, 1408), (9, 20512), (3, 65568)])
def test_dequantize_rows_of_any_length(rows, C, fmt):
    """A product of a code (2 bits), a scale (4 bits) and a power of two is a bf16 value: equal."""
    dev = _dev()
    q, sb, g = random_rows(np.random.default_rng([rows, C, 5]), rows, C, fmt)
    sb[:, C // BLOCK[fmt]:] = 0xEE                            # the padding is not a value's scale
    out = torch.full((rows + 1, C), 7.0, dtype=torch.bfloat16, device=dev)
    topo.topo_dequantize_micro(rows, C, fmt, torch.as_tensor(q, device=dev), torch.as_tensor(sb, device=dev),
                               None if g is None else torch.as_tensor(g, device=dev), out)
    want = values(q, sb, None if g is None else g.astype(np.float64), fmt)
    assert np.array_equal(out[:rows].cpu().double().numpy(), want)
    assert bool((out[rows] == 7).all())


def segments(rng, n_seg, rows, empty=True):
    cuts = np.sort(rng.integers(0, rows + 1, n_seg - 1)) if n_seg > 1 else np.empty(0, np.int64)
    off = np.concatenate([[0], cuts, [rows]]).astype(np.int32)
    if empty and n_seg > 3:
        off[2] = off[1]
    return off


def random_rows(rng, rows, K, fmt, spread=6):
    """Random codes and scales: packed rows, scale bytes, row scales."""
    q = rng.integers(0, 256, (rows, K // 2)).astype(np.uint8)
    pitch = topo.topo_micro_pitch(K, fmt)
    if fmt == MX:
        return q, rng.integers(127 - spread, 128 + spread, (rows, pitch)).astype(np.uint8), None
    return q, rng.integers(8, 127, (rows, pitch)).astype(np.uint8), np.exp2(rng.integers(-3, 4, rows)).astype(np.float32)


def product(a, w, off, seg_w, n_w, N, K, fmt, bf, dev, fill=7.0):
    rows = a[0].shape[0]
    t = [None if x is None else torch.as_tensor(x, device=dev) for x in (*a, *w)]
    out = torch.full((rows, N), fill, dtype=torch.bfloat16 if bf else torch.float32, device=dev)
    n_seg = len(off) - 1
    nb = topo.topo_expert_workspace_bytes(n_seg, rows, N, K)
    ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
    topo.topo_expert_gemm_micro(n_seg, rows, n_w, N, K, fmt, *t[:3], torch.as_tensor(off, device=dev),
                                None if seg_w is None else torch.as_tensor(seg_w, device=dev), *t[3:], out,
                                topo.TOPO_DTYPE_BF16 if bf else topo.TOPO_DTYPE_F32, ws, nb)
    torch.cuda.synchronize()
    return out, topo.topo_read_error(ws)


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows,n_seg,n_w,N,K,bf", [
    (1, 1, 1, 16, 32, False), (5, 3, 3, 48, 64, True), (130, 2, 2, 272, 288, False), (700, 8, 5, 528, 1408, True),
    (257, 4, 4, 1040, 544, False), (300, 2, 2, 256, 7168, True), (40, 400, 7, 64, 96, False), (200, 1, 1, 144, 17408, False),
    (33, 40, 9, 4096, 160, True)])
def test_products(rows, n_seg, n_w, N, K, bf, fmt):
    dev = _dev()
    rng = np.random.default_rng([rows, n_seg, N, K])
    off = segments(rng, n_seg, rows)
    seg_w = rng.integers(0, n_w, n_seg).astype(np.int32) if n_w != n_seg else None
    a = random_rows(rng, rows, K, fmt)
    w = random_rows(rng, n_w * N, K, fmt)
    got, err = product(a, w, off, seg_w, n_w, N, K, fmt, bf, dev)
    assert err == 0
    va, vw = torch.as_tensor(values(*a, fmt)), torch.as_tensor(values(*w, fmt)).reshape(n_w, N, K)
    got = got.double().cpu()
    for i in range(n_seg):
        r0, r1 = int(off[i]), int(off[i + 1])
        if r0 == r1:
            continue
        m = vw[i if seg_w is None else int(seg_w[i])]
        want, A = va[r0:r1] @ m.T, va[r0:r1].abs() @ m.abs().T
        tol = (K / 64 + K / 8192 + 4) * 2.0 ** -23 * A + (2.0 ** -8 * want.abs() if bf else 0)
        assert bool(((got[r0:r1] - want).abs() <= tol).all()), float(((got[r0:r1] - want).abs() / A).max())


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
def test_product_skips_bad_segments_and_leaves_other_rows(fmt):
    dev = _dev()
    rng = np.random.default_rng(11)
    a, w = random_rows(rng, 100, 64, fmt), random_rows(rng, 2 * 32, 64, fmt)
    off = np.array([10, 30, 50, 90], np.int32)
    got, err = product(a, w, off, np.array([0, 5, 1], np.int32), 2, 32, 64, fmt, False, dev)
    assert err == topo.TOPO_ERANGE
    assert bool((got[:10] == 7).all() and (got[30:50] == 7).all() and (got[90:] == 7).all())
    assert not bool((got[10:30] == 7).all()) and not bool((got[50:90] == 7).all())
    off = np.array([10, 30, 20, 101], np.int32)
    got, err = product(a, w, off, np.array([0, 1, 1], np.int32), 2, 32, 64, fmt, False, dev)
    assert err == topo.TOPO_ESTATE
    assert bool((got[:10] == 7).all() and (got[30:] == 7).all())


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
def test_product_of_rows_that_are_nan(fmt):
    """A block's NaN scale makes its row's outputs NaN and no other's."""
    dev = _dev()
    rng = np.random.default_rng(12)
    v = rng.standard_normal((300, 320))
    v[7, 300] = np.nan
    v[200, 3] = np.inf
    q, s, g = buffers(300, 320, fmt, dev)
    topo.topo_quantize_rows_micro(300, 320, fmt, bf16(v).to(dev), q, s, g)
    w = random_rows(rng, 48, 320, fmt)
    a = [None if x is None else x.cpu().numpy() for x in (q, s, g)]
    got, err = product(a, w, np.array([0, 300], np.int32), None, 1, 48, 320, fmt, False, dev)
    assert err == 0
    nan = torch.isnan(got).cpu()
    assert bool(nan[7].all() and nan[200].all()) and int(nan.sum()) == 96


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
def test_products_repeat_and_do_not_depend_on_other_rows(fmt):
    dev = _dev()
    rng = np.random.default_rng(13)
    a, w = random_rows(rng, 900, 1056, fmt), random_rows(rng, 3 * 272, 1056, fmt)
    off = np.array([0, 301, 600, 900], np.int32)
    one, _ = product(a, w, off, None, 3, 272, 1056, fmt, True, dev)
    two, _ = product(a, w, off, None, 3, 272, 1056, fmt, True, dev)
    assert torch.equal(one, two)
    part, _ = product(a, w, np.array([310, 320], np.int32), np.array([1], np.int32), 3, 272, 1056, fmt, True, dev)
    assert torch.equal(part[310:320], one[310:320])


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows,n_seg,n_w,N,K,bf", [(89, 3, 3, 1536, 4064, True), (400, 1, 1, 144, 288, False), (2, 1, 1, 512, 5024, True),
                                                   (150, 2, 3, 1040, 544, False), (19, 19, 2, 1024, 96, True)])
def test_products_of_few_tiles(rows, n_seg, n_w, N, K, bf, fmt):
    """Tiles of half as many columns."""
    test_products(rows, n_seg, n_w, N, K, bf, fmt)


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("n_seg", [17, 18, 19, 20, 38, 39])
def test_products_do_not_depend_on_the_tiles_width(n_seg, fmt):
    """4 or 8 tiles a segment: narrow ones for a single segment, wide ones for many."""
    dev = _dev()
    rng = np.random.default_rng(19)
    n, N, K = 39, 1008, 800
    a, w = random_rows(rng, 2 * n, K, fmt), random_rows(rng, 3 * N, K, fmt)
    seg_w = rng.integers(0, 3, n).astype(np.int32)
    off = np.arange(0, 2 * n + 1, 2).astype(np.int32)
    got, err = product(a, w, off[:n_seg + 1], seg_w[:n_seg], 3, N, K, fmt, False, dev)
    assert err == 0 and bool((got[2 * n_seg:] == 7).all())
    for i in (0, 5, n_seg - 1):
        one, _ = product(a, w, off[i:i + 2], seg_w[i:i + 1], 3, N, K, fmt, False, dev)
        assert torch.equal(one[2 * i:2 * i + 2], got[2 * i:2 * i + 2])


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
def test_calls_captured_in_a_graph(fmt):
    dev = _dev()
    rng = np.random.default_rng(14)
    rows, C, N = 200, 1408, 256
    w = [None if t is None else torch.as_tensor(t, device=dev) for t in random_rows(rng, 2 * N, C, fmt)]
    x = [bf16(rng.standard_normal((rows, C))).to(dev) for _ in range(2)]
    off = torch.tensor([0, 90, rows], dtype=torch.int32, device=dev)
    buf, out = buffers(rows, C, fmt, dev), torch.empty(rows, N, device=dev)
    nb = topo.topo_expert_workspace_bytes(2, rows, N, C)
    ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
    src = x[0].clone()

    def step():
        s = torch.cuda.current_stream().cuda_stream
        topo.topo_quantize_rows_micro(rows, C, fmt, src, *buf, s)
        topo.topo_expert_gemm_micro(2, rows, 2, N, C, fmt, *buf, off, None, *w, out, topo.TOPO_DTYPE_F32, ws, nb, s)

    want = []
    for v in x:
        src.copy_(v)
        step()
        want.append(out.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 1, 0):
        src.copy_(x[i])
        graph.replay()
        assert torch.equal(out, want[i])
    assert topo.topo_read_error(ws) == 0


def _refused(fn, *args, code=topo.TOPO_EINVAL):
    with pytest.raises(topo.TopoError) as ex:
        fn(*args)
    assert ex.value.code == code


def test_refusals():
    """Before anything is enqueued: no GPU is touched."""
    try:
        topo.lib()
    except RuntimeError:
        pytest.skip("library not built")
    p, odd = 1 << 20, (1 << 20) + 8
    assert topo.topo_micro_pitch(1408, MX) == 48 and topo.topo_micro_pitch(1408, NV) == 96
    assert topo.topo_micro_pitch(32, MX) == 16 and topo.topo_micro_pitch(512, MX) == 16 and topo.topo_micro_pitch(544, MX) == 32
    for C, fmt in ((16, MX), (0, NV), (-32, MX), (48, NV), (64, 0), (64, 3)):
        assert topo.topo_micro_pitch(C, fmt) == 0
        for fn in (topo.topo_quantize_rows_micro, topo.topo_swiglu_quantize_micro):
            _refused(fn, 4, C, fmt, p, p, p, p if fmt == NV else None)
    for fn in (topo.topo_quantize_rows_micro, topo.topo_swiglu_quantize_micro):
        _refused(fn, -1, 64, MX, p, p, p)
        _refused(fn, 1 << 31, 64, MX, p, p, p)
        _refused(fn, 4, 64, MX, None, p, p)
        _refused(fn, 4, 64, MX, odd, p, p)
        _refused(fn, 4, 64, MX, p, odd, p)
        _refused(fn, 4, 64, MX, p, p, odd)
        _refused(fn, 4, 64, MX, p, p, p, p)                   # MX has no row scales
        _refused(fn, 4, 64, NV, p, p, p, None)
        _refused(fn, 4, 64, NV, p, p, p, p + 2)
        assert fn(0, 64, MX, None, None, None) == 0
    _refused(topo.topo_dequantize_micro, 4, 64, MX, p, p, None, None)
    _refused(topo.topo_dequantize_micro, 4, 64, NV, p, p, None, p)
    _refused(topo.topo_dequantize_micro, 4, 64, MX, p, p, None, odd)
    assert topo.topo_dequantize_micro(0, 64, MX, None, None, None, None) == 0
    cfg = topo.make_cfg(T=4, E=4, k=2, R=1, ranks_per_node=1, n_slot=0)
    nb = topo.topo_workspace_bytes(cfg, 1, topo.TOPO_CALL_PACK)
    _refused(topo.topo_permute_quantize_micro, cfg, 1, 48, MX, p, p, p, p, None, p, nb)
    _refused(topo.topo_permute_quantize_micro, cfg, 1, 64, MX, p, p, p, None, None, p, nb)
    _refused(topo.topo_permute_quantize_micro, cfg, 1, 64, NV, p, p, p, p, None, p, nb)
    _refused(topo.topo_permute_quantize_micro, cfg, 1, 64, MX, p, p, p, p, None, p, nb - 1, code=topo.TOPO_ENOSPC)
    ok = [2, 8, 2, 32, 64, MX, p, p, None, p, None, p, p, None, p, topo.TOPO_DTYPE_F32, p, 256]

    def gemm(code=topo.TOPO_EINVAL, **change):
        names = ("n_seg rows n_w N K fmt a a_scale a_row seg_off seg_w w w_scale w_row out dtype ws nb").split()
        args = list(ok)
        for n, v in change.items():
            args[names.index(n)] = v
        _refused(topo.topo_expert_gemm_micro, *args, code=code)

    for change in (dict(n_seg=-1), dict(rows=-1), dict(N=24), dict(K=48), dict(fmt=0), dict(fmt=3), dict(a=None), dict(a=odd),
                   dict(a_scale=odd), dict(a_row=p), dict(seg_off=None), dict(seg_off=p + 2), dict(seg_w=p + 1), dict(w=None),
                   dict(w_scale=None), dict(w_row=p), dict(out=None), dict(out=odd), dict(dtype=2), dict(ws=None), dict(n_w=0),
                   dict(n_seg=3), dict(fmt=NV), dict(fmt=NV, a_row=p), dict(fmt=NV, w_row=p), dict(fmt=NV, a_row=p, w_row=odd),
                   dict(N=1 << 23), dict(K=1 << 23), dict(n_w=1 << 28)):
        gemm(**change)
    gemm(code=topo.TOPO_ENOSPC, nb=255)
    args = list(ok)
    args[0] = 0
    assert topo.topo_expert_gemm_micro(*args) == 0
