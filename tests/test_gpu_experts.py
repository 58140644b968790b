"""The 8-bit operands and the experts' products against the formulas in 64
bits (numpy), at ragged sizes and segments, and the refusals of their arguments.

Quantised bytes and scales are compared exactly: the scale is a power of two,
so each value is rounded once.  A product's float32 sum of K terms is compared
to the sum of the terms' magnitudes A: the tensor core adds 32 products at a
time with at least 24 bits below the largest, the blocks' sums are added in
float32, so |error| <= (K / 32 + 3 * ceil(K / 128) + 2) * 2^-23 * A bounds it;
a bf16 output adds 2^-8 of the value."""
import numpy as np
import pytest

import moe_expert_routing_ids_gb300 as topo

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
B = 128


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _kb(n):
    return (n + B - 1) // B


# ---------------------------------------------------------- e4m3 on the host
def _table():
    v = np.empty(256, np.float64)
    for i in range(256):
        s, e, m = i >> 7, (i >> 3) & 15, i & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[i] = np.nan if (e == 15 and m == 7) else (-x if s else x)
    return v


E4M3 = _table()


def scale_of(amax):
    """Smallest power of two >= amax / 448, exponent >= -126; 1 for 0."""
    m, e = np.frexp(np.where(amax > 0, amax, 1.0) / 448.0)
    n = np.maximum(np.where(m == 0.5, e - 1, e), -126)
    return np.where(amax > 0, np.ldexp(1.0, n), 1.0)


def to_e4m3(y):
    """Bytes of y (float64) rounded to nearest, ties to even; not finite: NaN."""
    pos = E4M3[:127]                                        # 0 .. 448, ascending
    a = np.abs(np.where(np.isfinite(y), y, 0.0))
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    out = np.where(np.signbit(y), pick | 128, pick)
    return np.where(np.isfinite(y), out, 127).astype(np.uint8)


def quant(v):
    """v float64 [rows, C]: bytes and scales along the rows."""
    rows, C = v.shape
    q, s = np.empty((rows, C), np.uint8), np.empty((rows, _kb(C)))
    for b in range(_kb(C)):
        p = v[:, b * B:(b + 1) * B]
        s[:, b] = scale_of(np.where(np.isfinite(p), np.abs(p), 0.0).max(1))
        with np.errstate(invalid="ignore"):
            q[:, b * B:(b + 1) * B] = to_e4m3(p / s[:, b:b + 1])
    return q, s


def same_bytes(got, want):
    """Equal bytes, any NaN pattern for a NaN."""
    nan = (want & 127) == 127
    return np.array_equal(got[~nan], want[~nan]) and np.all((got[nan] & 127) == 127)


def bf16(v):
    return torch.as_tensor(v.astype(np.float32)).to(torch.bfloat16)


def hard_rows(rng, rows, C):
    """Rows over many magnitudes with zeros, NaN, infinities, subnormals and block maxima on the scale's edges."""
    v = rng.standard_normal((rows, C)) * np.exp(rng.standard_normal((rows, 1)) * 4)
    v = bf16(v).float().numpy().astype(np.float64)
    if rows > 8:
        v[0] = 0.0
        v[1, :5] = np.nan
        v[2, C - 1] = np.inf
        v[3] = -np.inf
        v[4] = 2.0 ** -133                                    # subnormal bf16
        v[5] = 448.0 * 2.0 ** -3
        v[6] = 450.0
        v[7] = 3.3e38
        v[8] = -2.0 ** -126
    return v


@gpu
@pytest.mark.parametrize("rows,C", [(1, 16), (3, 128), (17, 144), (40, 1408), (9, 7168), (700, 272), (20000, 128)])
def test_quantize_rows(rows, C):
    dev = _dev()
    v = hard_rows(np.random.default_rng([rows, C]), rows, C)
    x = bf16(v).to(dev)
    q = torch.full((rows, C), 0x55, dtype=torch.uint8, device=dev)
    s = torch.full((rows, _kb(C)), -1.0, device=dev)
    topo.topo_quantize_rows(rows, C, x, q, s)
    wq, ws = quant(v)
    assert np.array_equal(s.cpu().numpy().astype(np.float64), ws)
    assert same_bytes(q.cpu().numpy(), wq)


@gpu
@pytest.mark.parametrize("L,T,k,H", [(1, 1, 1, 16), (1, 5, 8, 7168), (2, 33, 3, 272), (1, 100, 40, 144),
                                     (1, 3000, 6, 1408), (2, 4097, 2, 1024), (1, 2100, 40, 1024)])
def test_permute_quantize(L, T, k, H):
    dev = _dev()
    rng = np.random.default_rng([L, T, k, H])
    v = hard_rows(rng, L * T, H)
    cfg = topo.make_cfg(T=T, E=max(k, 2), k=k, R=1, ranks_per_node=1, n_slot=0)
    sp = np.stack([rng.permutation(T * k) for _ in range(L)]).astype(np.int32)
    nb = topo.topo_workspace_bytes(cfg, L, topo.TOPO_CALL_PACK)
    ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
    q = torch.full((L, T * k, H), 0x55, dtype=torch.uint8, device=dev)
    s = torch.full((L, T * k, _kb(H)), -1.0, device=dev)
    topo.topo_permute_quantize(cfg, L, H, bf16(v).to(dev), torch.as_tensor(sp, device=dev), q, s, ws, nb)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == 0
    wq, wsc = quant(v)
    for l in range(L):
        t = l * T + sp[l] // k
        assert np.array_equal(s[l].cpu().numpy().astype(np.float64), wsc[t])
        assert same_bytes(q[l].cpu().numpy(), wq[t])


@gpu
@pytest.mark.parametrize("T,H", [(8, 32), (2100, 1024)])
def test_permute_quantize_reports_pairs_outside_the_layer(T, H):
    dev = _dev()
    k = 2
    cfg = topo.make_cfg(T=T, E=4, k=k, R=1, ranks_per_node=1, n_slot=0)
    nb = topo.topo_workspace_bytes(cfg, 1, topo.TOPO_CALL_PACK)
    for bad in (-1, T * k):
        ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
        sp = torch.arange(T * k, dtype=torch.int32, device=dev)
        sp[3] = bad
        q = torch.zeros((T * k, H), dtype=torch.uint8, device=dev)
        s = torch.zeros((T * k, _kb(H)), device=dev)
        topo.topo_permute_quantize(cfg, 1, H, torch.zeros((T, H), dtype=torch.bfloat16, device=dev), sp, q, s, ws, nb)
        torch.cuda.synchronize()
        assert topo.topo_read_error(ws) == topo.TOPO_ESTATE


@gpu
@pytest.mark.parametrize("n_w,N,K", [(1, 16, 16), (2, 128, 256), (3, 144, 272), (1, 400, 1040)])
def test_quantize_weight_and_its_transpose(n_w, N, K):
    dev = _dev()
    rng = np.random.default_rng([n_w, N, K])
    v = bf16(rng.standard_normal((n_w, N, K)) * 0.02).float().numpy().astype(np.float64)
    v[0, 0, 0] = np.nan
    q, qt = (torch.full(s, 0x55, dtype=torch.uint8, device=dev) for s in ((n_w, N, K), (n_w, K, N)))
    s, st = torch.full((n_w, _kb(N), _kb(K)), -1.0, device=dev), torch.full((n_w, _kb(K), _kb(N)), -1.0, device=dev)
    topo.topo_quantize_weight(n_w, N, K, bf16(v).to(dev), q, s, qt, st)
    only, os = torch.zeros_like(q), torch.zeros_like(s)
    topo.topo_quantize_weight(n_w, N, K, bf16(v).to(dev), only, os)
    assert torch.equal(only, q) and torch.equal(os, s)
    assert torch.equal(qt, q.transpose(1, 2)) and torch.equal(st, s.transpose(1, 2))
    got, sc = q.cpu().numpy(), s.cpu().numpy()
    for i in range(n_w):
        for a in range(_kb(N)):
            for b in range(_kb(K)):
                blk = v[i, a * B:(a + 1) * B, b * B:(b + 1) * B]
                w = scale_of(np.array(np.nanmax(np.abs(blk))))
                assert sc[i, a, b] == w
                assert same_bytes(got[i, a * B:(a + 1) * B, b * B:(b + 1) * B], to_e4m3(blk / w))


@gpu
@pytest.mark.parametrize("rows,I", [(1, 16), (33, 144), (130, 1408), (4000, 256)])
def test_swiglu_quantize_and_gradient(rows, I):
    """The activation is formed in float32 (four roundings and exp within 2 ulp:
    8 * 2^-24 relative): its bytes may differ from the 64-bit ones only where the
    value is that near to a rounding edge."""
    dev = _dev()
    rng = np.random.default_rng([rows, I])
    h = bf16(rng.standard_normal((rows, 2 * I)) * 3)
    hv = h.float().numpy().astype(np.float64)
    q = torch.full((rows, I), 0x55, dtype=torch.uint8, device=dev)
    s = torch.full((rows, _kb(I)), -1.0, device=dev)
    topo.topo_swiglu_quantize(rows, I, h.to(dev), q, s)
    g, u = hv[:, :I], hv[:, I:]
    sg = 1.0 / (1.0 + np.exp(-g))
    a = g * sg * u
    lo, hi = quant(a * (1 - 8 * 2.0 ** -24)), quant(a * (1 + 8 * 2.0 ** -24))
    sv = s.cpu().numpy().astype(np.float64)
    assert np.all((sv == lo[1]) | (sv == hi[1]))
    same = np.repeat((lo[1] == hi[1]) & (sv == lo[1]), B, 1)[:, :I]
    got = q.cpu().numpy()
    assert np.all((got == lo[0]) | (got == hi[0]) | ~same)
    assert same.mean() > 0.99

    dy = bf16(rng.standard_normal((rows, I)))
    dh = torch.full((rows, 2 * I), float("nan"), dtype=torch.bfloat16, device=dev)
    topo.topo_swiglu_grad(rows, I, h.to(dev), dy.to(dev), dh)
    y = dy.float().numpy().astype(np.float64)
    # terms' magnitudes: 1 + g (1 - s) cancels near its zero
    want = np.concatenate([y * u * sg * (1 + g * (1 - sg)), y * g * sg], 1)
    size = np.concatenate([np.abs(y * u * sg) * (1 + np.abs(g) * (1 - sg)), np.abs(y * g * sg)], 1)
    got = dh.float().cpu().numpy()
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size + 1e-37)


@gpu
def test_swiglu_gradient_against_differences():
    dev = _dev()
    rng = np.random.default_rng(2)
    I, e = 16, 1e-4
    h = bf16(rng.standard_normal((4, 2 * I)))
    dy = bf16(rng.standard_normal((4, I)))
    dh = torch.empty((4, 2 * I), dtype=torch.bfloat16, device=dev)
    topo.topo_swiglu_grad(4, I, h.to(dev), dy.to(dev), dh)
    v, y = h.double().numpy(), dy.double().numpy()

    def f(z):
        g, u = z[:, :I], z[:, I:]
        return g / (1 + np.exp(-g)) * u * y

    num = np.empty_like(v)
    for j in range(2 * I):
        d = np.zeros_like(v)
        d[:, j] = e
        num[:, j] = ((f(v + d) - f(v - d)) / (2 * e))[:, j % I]
    assert np.all(np.abs(dh.double().cpu().numpy() - num) <= 2.0 ** -8 * np.abs(num) + 1e-5)


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def product(lens, n_w, N, K, out, seg_w=None, seed=0, lead=0, tail=0, stream=None, want_error=0, so=None):
    """Runs topo_expert_gemm on random operands; checks every row against 64 bits."""
    dev = _dev()
    rng = np.random.default_rng([seed, N, K, len(lens)])
    rows = int(sum(lens)) + lead + tail
    a = (rng.integers(0, 255, (rows, K), dtype=np.uint8) & 0xBF) if rows else np.zeros((0, K), np.uint8)
    w = rng.integers(0, 255, (n_w, N, K), dtype=np.uint8) & 0xBF      # |value| below 2, no NaN
    sa = np.exp(rng.standard_normal((rows, _kb(K)))).astype(np.float32)
    sw = np.exp(rng.standard_normal((n_w, _kb(N), _kb(K)))).astype(np.float32)
    so = offsets(lens) + lead if so is None else so
    dt = torch.bfloat16 if out == topo.TOPO_DTYPE_BF16 else torch.float32
    y = torch.full((rows, N), -777.0, dtype=dt, device=dev)
    nb = topo.topo_expert_workspace_bytes(len(lens), rows, N, K)
    ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
    t = lambda z: torch.as_tensor(z, device=dev)  # noqa: E731
    args = [t(z) for z in (a, sa, so, w, sw)]
    sw_d = None if seg_w is None else t(np.asarray(seg_w, np.int32))
    torch.cuda.synchronize()
    topo.topo_expert_gemm(len(lens), rows, n_w, N, K, args[0], args[1], args[2], sw_d, args[3], args[4], y, out, ws, nb,
                          stream)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == want_error
    if want_error:
        return y
    got = y.float().cpu().numpy().astype(np.float64)
    assert np.all(got[:lead] == -777.0) and np.all(got[rows - tail:] == -777.0)
    fac = (K / 32 + 3 * _kb(K) + 2) * 2.0 ** -23
    for i, n in enumerate(lens):
        if not n:
            continue
        e = i if seg_w is None else seg_w[i]
        r = slice(so[i], so[i + 1])
        av, wv = E4M3[a[r]], E4M3[w[e]]
        av = av * np.repeat(sa[r].astype(np.float64), B, 1)[:, :K]
        wv = wv * np.repeat(np.repeat(sw[e].astype(np.float64), B, 0)[:N], B, 1)[:, :K]
        want, size = av @ wv.T, np.abs(av) @ np.abs(wv).T
        tol = fac * size + (2.0 ** -8 * np.abs(want) if dt == torch.bfloat16 else 0.0)
        assert np.all(np.abs(got[r] - want) <= tol), (i, n, np.max(np.abs(got[r] - want) - tol))
    return y


F32, BF = topo.TOPO_DTYPE_F32, topo.TOPO_DTYPE_BF16


@gpu
@pytest.mark.parametrize("out", [F32, BF])
@pytest.mark.parametrize("lens,N,K", [
    ([1], 16, 16), ([0, 1, 0], 16, 128), ([6], 128, 144), ([3, 0, 17, 1], 272, 1408), ([16, 15, 33, 2, 64], 144, 400),
    ([31, 32, 33, 100], 400, 256), ([129, 0, 60, 255], 256, 640), ([200, 300, 190], 528, 272), ([128, 256, 512], 256, 128),
    ([777, 0, 1, 129, 640], 272, 400), ([1500], 16, 4096), ([5, 2000], 1040, 144)])
def test_products_of_ragged_segments(lens, N, K, out):
    product(lens, len(lens), N, K, out)


@gpu
@pytest.mark.parametrize("lens", [[3, 5, 0, 2], [300, 0, 260, 1]])
def test_products_of_replicas_and_of_a_part_of_the_rows(lens):
    """Segments that share weights, and rows before and after the segments left alone."""
    product(lens, 3, 144, 272, F32, seg_w=[2, 0, 0, 2], lead=7, tail=21)


@gpu
@pytest.mark.parametrize("per", [1, 200])
def test_products_of_more_segments_than_one_launch_holds(per):
    n = 1300 if per == 1 else 1030
    lens = [per if i % 3 else 0 for i in range(n)]
    lens[-1] = 5
    product(lens, 4, 32, 32, F32, seg_w=[i % 4 for i in range(n)])


@gpu
def test_products_on_another_stream_and_twice():
    a = product([40, 0, 300], 3, 272, 400, BF, stream=torch.cuda.Stream())
    b = product([40, 0, 300], 3, 272, 400, BF)
    assert torch.equal(a, b)


@gpu
def test_products_skip_and_report_bad_segments():
    product([4, 4], 2, 16, 32, F32, seg_w=[0, 2], want_error=topo.TOPO_ERANGE)
    product([4, 4], 2, 16, 32, F32, seg_w=[-1, 0], want_error=topo.TOPO_ERANGE)
    y = product([4, 4, 4], 3, 16, 32, F32, so=np.array([0, 4, 2, 12], np.int32), want_error=topo.TOPO_ESTATE)
    assert not torch.any(y[:4] == -777.0)                      # the good segment is there
    product([4, 4], 2, 16, 32, F32, so=np.array([0, 4, 9], np.int32), want_error=topo.TOPO_ESTATE)
    product([4, 4], 2, 16, 32, F32, so=np.array([-4, 4, 8], np.int32), want_error=topo.TOPO_ESTATE)


@gpu
def test_a_nan_or_infinite_scale_stays_in_its_row():
    dev = _dev()
    rows, N, K = 40, 32, 256
    a = torch.full((rows, K), 0x38, dtype=torch.uint8, device=dev)      # 1.0
    w = torch.full((1, N, K), 0x38, dtype=torch.uint8, device=dev)
    sa = torch.ones((rows, 2), device=dev)
    sa[3, 0] = float("nan")
    sa[9, 1] = float("inf")
    a[5, 200] = 0x7F                                                    # e4m3 NaN
    y = torch.empty((rows, N), device=dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    for n in (1, 2):                                                    # few rows, and many for one segment
        so = torch.tensor([0, rows], dtype=torch.int32, device=dev)
        if n == 2:
            a, sa = a.repeat(10, 1), sa.repeat(10, 1)
            so[1] = 10 * rows
            y = torch.empty((10 * rows, N), device=dev)
        topo.topo_expert_gemm(1, y.shape[0], 1, N, K, a, sa, so, None, w, torch.ones((1, 1, 2), device=dev), y, F32, ws, 256)
        v = y.cpu().numpy()[:rows]
        bad = np.zeros(rows, bool)
        bad[[3, 5]] = True
        assert np.all(np.isnan(v[bad])) and np.all(np.isinf(v[9]))
        bad[9] = True
        assert np.all(v[~bad] == K)


# ------------------------------------------------------------ weight gradient
def cols_reference(v, so, cap):
    """Transposed bytes [C, cap] and scales [cap / 128, C] (rows of blocks that exist)."""
    C = v.shape[1]
    q, s, b = np.zeros((C, cap), np.uint8), np.ones((cap // B, C)), 0
    for i in range(len(so) - 1):
        for r in range(so[i], so[i + 1], B):
            part = v[r:min(r + B, so[i + 1])]
            pq, ps = quant(part.T)
            q[:, b * B:b * B + len(part)] = pq
            s[b] = ps[:, 0]
            b += 1
    return q, s, b


@gpu
@pytest.mark.parametrize("lens,C", [([1], 16), ([0, 127, 0, 129], 144), ([128, 256], 128), ([5, 300, 77], 272),
                                    ([700, 0, 1300, 3], 528)])
def test_quantize_cols(lens, C):
    dev = _dev()
    so = offsets(lens)
    rows = int(so[-1])
    v = hard_rows(np.random.default_rng([rows, C]), rows, C)
    cap = topo.topo_cols_capacity(len(lens), rows)
    q = torch.full((C, cap), 0x55, dtype=torch.uint8, device=dev)
    s = torch.full((cap // B, C), -1.0, device=dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    topo.topo_quantize_cols(len(lens), rows, C, bf16(v).to(dev), torch.as_tensor(so, device=dev), cap, q, s, ws, 256)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == 0
    wq, wsc, nb = cols_reference(v, so, cap)
    assert np.array_equal(s[:nb].cpu().numpy().astype(np.float64), wsc[:nb])
    assert same_bytes(q.cpu().numpy()[:, :nb * B], wq[:, :nb * B])


def wgrad(lens, N, K, seed=0):
    dev = _dev()
    rng = np.random.default_rng([seed, N, K, len(lens)])
    so = offsets(lens)
    rows = int(so[-1])
    dy = bf16(rng.standard_normal((rows, N)) * 1e-3)
    x = bf16(rng.standard_normal((rows, K)))
    cap = topo.topo_cols_capacity(len(lens), rows)
    sod = torch.as_tensor(so, device=dev)
    nb = topo.topo_expert_workspace_bytes(len(lens), rows, N, K)
    ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
    ops = []
    for v, C in ((dy, N), (x, K)):
        q = torch.full((C, cap), 0x7F, dtype=torch.uint8, device=dev)   # NaN where nothing is written
        s = torch.full((cap // B, C), float("nan"), device=dev)
        topo.topo_quantize_cols(len(lens), rows, C, v.to(dev), sod, cap, q, s, ws, nb)
        ops += [q, s]
    dw = torch.full((len(lens), N, K), float("nan"), device=dev)
    topo.topo_expert_wgrad(len(lens), rows, N, K, cap, *ops, sod, dw, ws, nb)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == 0
    q = [o.cpu().numpy().astype(np.float64) if o.dtype == torch.float32 else E4M3[o.cpu().numpy()] for o in ops]
    b = 0
    for i, n in enumerate(lens):
        want, size = np.zeros((N, K)), np.zeros((N, K))
        for _ in range(_kb(n)):
            c = slice(b * B, (b + 1) * B)
            A, X = q[0][:, c] * q[1][b][:, None], q[2][:, c] * q[3][b][:, None]
            want += A @ X.T
            size += np.abs(A) @ np.abs(X).T
            b += 1
        fac = (_kb(n) * 4 + 4 * _kb(n) + 2) * 2.0 ** -23
        assert np.all(np.abs(dw[i].cpu().numpy() - want) <= fac * size), i
    return dw, dy, x, so


@gpu
@pytest.mark.parametrize("lens,N,K", [([1], 16, 16), ([0, 5, 0], 16, 272), ([127, 129, 0, 300], 144, 400),
                                      ([128, 512], 128, 256), ([600, 33], 272, 528), ([2000], 400, 16)])
def test_weight_gradients_of_ragged_segments(lens, N, K):
    dw, *_ = wgrad(lens, N, K)
    for i, n in enumerate(lens):
        if n == 0:
            assert torch.all(dw[i] == 0)


@gpu
def test_weight_gradients_of_more_segments_than_one_launch_holds():
    wgrad([(i * 37) % 140 if i % 2 else 0 for i in range(1100)], 16, 16)


@gpu
def test_gradients_against_differences():
    """The products are linear, so a unit difference of one operand gives the
    gradient: dX from the transposed weights, dW from the columns; values on the
    e4m3 grid make the quantisation exact, and the sums are small integers."""
    dev = _dev()
    rng = np.random.default_rng(1)
    rows, N, K = 40, 32, 48
    x = rng.integers(-4, 5, (rows, K)).astype(np.float64)
    w = rng.integers(-4, 5, (1, N, K)).astype(np.float64)
    c = rng.integers(-4, 5, (rows, N)).astype(np.float64)               # loss = sum of c * y
    x[:, 0], w[:, :, 0], c[:, 0] = 4, 4, 4
    x[0], c[0] = 4, 4
    so = torch.tensor([0, rows], dtype=torch.int32, device=dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    u8 = torch.uint8

    def loss(xx, ww):
        return float((c * (xx @ ww[0].T)).sum())

    wq, wt = torch.empty((1, N, K), dtype=u8, device=dev), torch.empty((1, K, N), dtype=u8, device=dev)
    s, st = torch.empty((1, 1, 1), device=dev), torch.empty((1, 1, 1), device=dev)
    topo.topo_quantize_weight(1, N, K, bf16(w).to(dev), wq, s, wt, st)
    cq, cs = torch.empty((rows, N), dtype=u8, device=dev), torch.empty((rows, 1), device=dev)
    topo.topo_quantize_rows(rows, N, bf16(c).to(dev), cq, cs)
    dx = torch.empty((rows, K), device=dev)
    topo.topo_expert_gemm(1, rows, 1, K, N, cq, cs, so, None, wt, st, dx, F32, ws, 256)
    cap = topo.topo_cols_capacity(1, rows)
    ops = []
    for v, C in ((c, N), (x, K)):
        q, sc = torch.empty((C, cap), dtype=u8, device=dev), torch.empty((cap // B, C), device=dev)
        topo.topo_quantize_cols(1, rows, C, bf16(v).to(dev), so, cap, q, sc, ws, 256)
        ops += [q, sc]
    dw = torch.empty((1, N, K), device=dev)
    topo.topo_expert_wgrad(1, rows, N, K, cap, *ops, so, dw, ws, 256)
    dx, dw = dx.cpu().numpy(), dw.cpu().numpy()
    for i, j in ((0, 0), (7, 31), (39, 47), (20, 16)):
        d = np.zeros_like(x)
        d[i, j] = 1
        assert dx[i, j] == loss(x + d, w) - loss(x, w)
    for n, j in ((0, 0), (31, 47), (5, 16)):
        d = np.zeros_like(w)
        d[0, n, j] = 1
        assert dw[0, n, j] == loss(x, w + d) - loss(x, w)


# -------------------------------------------------------------------- refusals
def test_arguments_are_checked_on_the_host():
    try:
        topo.lib()
    except RuntimeError:
        pytest.skip("library not built")
    a = 1 << 20                                                 # never dereferenced
    assert topo.topo_expert_workspace_bytes(4, 100, 32, 32) == 256
    assert topo.topo_expert_workspace_bytes(4, 100, 24, 32) == 0
    assert topo.topo_cols_capacity(0, 0) == 128 and topo.topo_cols_capacity(3, 2) == 256
    assert topo.topo_cols_capacity(2, 256) == 384 and topo.topo_cols_capacity(-1, 5) == 0

    def refused(code, f, *args):
        with pytest.raises(topo.TopoError) as ex:
            f(*args)
        assert ex.value.code == code, (f.__name__, args)

    E, S = topo.TOPO_EINVAL, topo.TOPO_ENOSPC
    good = [4, 100, 4, 32, 48, a, a, a, None, a, a, a, F32, a, 256]
    for i, v in ((0, -1), (0, 5), (1, -1), (1, 1 << 31), (2, -1), (2, 0), (3, 24), (3, 0), (4, 8), (5, None), (5, a + 8),
                 (6, None), (6, a + 2), (7, None), (7, a + 1), (9, None), (9, a + 4), (10, None), (11, None), (11, a + 4),
                 (12, 2), (13, None)):
        args = list(good)
        args[i] = v
        refused(E, topo.topo_expert_gemm, *args)
    refused(S, topo.topo_expert_gemm, *good[:-1], 255)
    refused(E, topo.topo_expert_gemm, *[4, 100, 1 << 27, 32, 48], *good[5:])
    cap = topo.topo_cols_capacity(4, 100)
    good = [4, 100, 32, 48, cap, a, a, a, a, a, a, a, 256]
    for i, v in ((0, -1), (2, 8), (3, 20), (4, cap + 128), (5, None), (5, a + 4), (6, None), (8, a + 2), (9, None),
                 (10, None), (10, a + 8), (11, None)):
        args = list(good)
        args[i] = v
        refused(E, topo.topo_expert_wgrad, *args)
    refused(S, topo.topo_expert_wgrad, *good[:-1], 255)
    good = [4, 100, 32, a, a, cap, a, a, a, 256]
    for i, v in ((0, -1), (1, -1), (2, 24), (3, a + 2), (4, None), (5, cap - 128), (6, None), (7, None), (8, None)):
        args = list(good)
        args[i] = v
        refused(E, topo.topo_quantize_cols, *args)
    refused(S, topo.topo_quantize_cols, *good[:-1], 255)
    for f in (topo.topo_quantize_rows, topo.topo_swiglu_quantize):
        for args in ((-1, 32, a, a, a), (4, 24, a, a, a), (4, 0, a, a, a), (4, 32, None, a, a), (4, 32, a + 8, a, a),
                     (4, 32, a, a + 8, a), (4, 32, a, a, None), (4, 32, a, a, a + 2)):
            refused(E, f, *args)
        f(0, 32, None, None, None)                              # no rows: nothing to do
    refused(E, topo.topo_swiglu_grad, 4, 32, a, None, a)
    refused(E, topo.topo_swiglu_grad, 4, 32, a, a, a + 8)
    for args in ((1, 32, 24, a, a, a), (1, 32, 32, None, a, a), (1, 32, 32, a, a, a, a, None), (1, 32, 32, a, a, a, None, a),
                 (1, 32, 32, a, a, a, a + 8, a), (-1, 32, 32, a, a, a)):
        refused(E, topo.topo_quantize_weight, *args)
    c = topo.make_cfg(T=8, E=4, k=2, R=1, ranks_per_node=1, n_slot=0)
    nb = topo.topo_workspace_bytes(c, 1, topo.TOPO_CALL_PACK)
    refused(E, topo.topo_permute_quantize, c, 1, 24, a, a, a, a, a, nb)
    refused(E, topo.topo_permute_quantize, c, 1, 32, a, a, a, None, a, nb)
    refused(E, topo.topo_permute_quantize, c, 1, 32, a + 8, a, a, a, a, nb)
    refused(S, topo.topo_permute_quantize, c, 1, 32, a, a, a, a, a, nb - 1)


@gpu
def test_weight_gradients_of_offsets_out_of_order():
    """Offsets that go back: that segment is empty, and so is every segment whose
    blocks the operands do not hold; the ones before them are whole."""
    dev = _dev()
    rng = np.random.default_rng(4)
    so, rows, N, K = np.array([0, 300, 0, 300], np.int32), 300, 144, 272
    n = len(so) - 1
    cap = topo.topo_cols_capacity(n, rows)
    assert cap == 5 * B                                        # 3 blocks of the first segment, 2 of the third's 3
    sod = torch.as_tensor(so, device=dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    ops = []
    for C in (N, K):
        q, s = torch.full((C, cap), 0x7F, dtype=torch.uint8, device=dev), torch.full((cap // B, C), float("nan"), device=dev)
        topo.topo_quantize_cols(n, rows, C, bf16(rng.standard_normal((rows, C))).to(dev), sod, cap, q, s, ws, 256)
        ops += [q, s]
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == topo.TOPO_ESTATE
    ws.zero_()
    dw = torch.full((n, N, K), float("nan"), device=dev)
    topo.topo_expert_wgrad(n, rows, N, K, cap, *ops, sod, dw, ws, 256)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == topo.TOPO_ESTATE
    q = [o.cpu().numpy().astype(np.float64) if o.dtype == torch.float32 else E4M3[o.cpu().numpy()] for o in ops]
    want, size = np.zeros((N, K)), np.zeros((N, K))
    for b in range(3):
        c = slice(b * B, (b + 1) * B)
        A, X = q[0][:, c] * q[1][b][:, None], q[2][:, c] * q[3][b][:, None]
        want += A @ X.T
        size += np.abs(A) @ np.abs(X).T
    assert np.all(np.abs(dw[0].cpu().numpy() - want) <= (4 * 3 + 4 * 3 + 2) * 2.0 ** -23 * size)
    assert torch.all(dw[1:] == 0)


@gpu
def test_weight_gradients_of_offsets_that_go_back_many_times():
    """The same 2^24 rows 2^14 times over: 2^31 blocks, of which the operands hold
    the first segment's 2^17.  Ones make its sum exact."""
    dev = _dev()
    rows, n, C = 1 << 24, 1 << 15, 16
    so = torch.zeros(n + 1, dtype=torch.int32, device=dev)
    so[1::2] = rows
    cap = topo.topo_cols_capacity(n, rows)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    x = torch.ones((rows, C), dtype=torch.bfloat16, device=dev)
    q, s = torch.empty((C, cap), dtype=torch.uint8, device=dev), torch.empty((cap // B, C), device=dev)
    topo.topo_quantize_cols(n, rows, C, x, so, cap, q, s, ws, 256)
    dw = torch.full((n, C, C), float("nan"), device=dev)
    topo.topo_expert_wgrad(n, rows, C, C, cap, q, s, q, s, so, dw, ws, 256)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == topo.TOPO_ESTATE
    assert torch.all(dw[0] == rows) and torch.all(dw[1:] == 0)


def test_columns_past_32_bit_coordinates_are_refused():
    try:
        topo.lib()
    except RuntimeError:
        pytest.skip("library not built")
    a, rows = 1 << 20, (1 << 31) - 1                            # never dereferenced
    for n in (2, 500):
        cap = topo.topo_cols_capacity(n, rows)
        assert cap > 1 << 31
        with pytest.raises(topo.TopoError) as ex:
            topo.topo_expert_wgrad(n, rows, 16, 16, cap, a, a, a, a, a, a, a, 256)
        assert ex.value.code == topo.TOPO_EINVAL


@gpu
@pytest.mark.parametrize("lens,N,K", [([2049, 0, 3], 16, 272), ([4096, 130], 144, 16), ([7, 5000, 0, 2176], 272, 144)])
def test_weight_gradients_of_long_segments(lens, N, K):
    """More than 2048 rows: the sum leaves tensor memory more than once."""
    wgrad(lens, N, K)


@gpu
def test_weight_gradients_of_many_tiles():
    """Several tiles to a CTA, of different depths, with ragged edges: 2 segments
    x 9 x 17 tiles, the last of 16 rows and of 16 columns."""
    wgrad([300, 2200], 1040, 4112)


@gpu
@pytest.mark.parametrize("out", [F32, BF])
def test_products_of_many_tiles(out):
    """Several tiles to a CTA, 11 blocks each, few rows and many, ragged columns."""
    lens = [(37 * i) % 150 if i % 5 else 0 for i in range(36)]
    lens[7] = 300
    product(lens, 3, 2064, 1408, out, seg_w=[i % 3 for i in range(36)])
