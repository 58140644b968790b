"""topo_route / topo_route_grad against the formulas in 64 bits (numpy), at the
sizes, ties and masks where routing can go wrong, and the refusals of their
arguments.

Tolerances.  Weights and gradients are short float32 expressions of exp and a
division: each of the at most E + 20 roundings is 2^-24 relative, exp is within
2 ulp, so 64 * 2^-24 covers a weight, and a gradient is compared to the size of
the terms it is the difference of.  Where the choice depends on rounded scores
the test only uses rows whose 64-bit scores differ by more than 1e-5."""
import numpy as np
import pytest

import moe_expert_routing_ids_gb300 as topo

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
SOFT, SIG = topo.TOPO_SCORE_SOFTMAX, topo.TOPO_SCORE_SIGMOID
U = 2.0 ** -24


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def scores(x, score):
    x = x.astype(np.float64)
    with np.errstate(all="ignore"):
        if score == SIG:
            return 1.0 / (1.0 + np.exp(-x))
        m = np.max(x, -1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(m), 0.0, m))
        t = e.sum(-1, keepdims=True)
        return np.where(t == 0, 0.0, e / np.where(t == 0, 1.0, t))


def order(v):
    """Indices in descending order of v: equal values by index, NaN last."""
    idx = np.arange(v.shape[-1])
    return np.array([np.array(sorted(idx, key=lambda i: (np.isnan(r[i]), -r[i] if not np.isnan(r[i]) else 0.0, i)))
                     for r in v])


def reference(x, k, score, bias=None, groups=1, kept=1, top=1, renorm=True, scale=1.0):
    """ids [T, k], weights [T, k] and the selection values, in 64 bits."""
    T, E = x.shape
    s = scores(x, score)
    c = x.astype(np.float64) if bias is None and top == 1 else s + (0.0 if bias is None else bias.astype(np.float64))
    c = np.where(np.isneginf(x), -np.inf, c)
    drop = np.zeros((T, E), bool)
    gs = None
    if groups > 1:
        low = np.where(np.isnan(c), -np.inf, c)                # NaN ranks below every number
        v = np.sort(low.reshape(T, groups, -1), -1)[:, :, ::-1][:, :, :top].sum(-1)
        keep = order(v)[:, :kept]
        drop = np.ones((T, groups), bool)
        np.put_along_axis(drop, keep, False, 1)
        drop = np.repeat(drop, E // groups, 1)
        gs = v
    ids = np.empty((T, k), np.int64)
    for t in range(T):
        live = np.flatnonzero(~drop[t])
        ids[t] = live[order(c[t, live][None])[0][:k]]
    sk = np.take_along_axis(s, ids, 1)
    if score == SOFT and renorm:                       # softmax over the chosen logits: no underflow
        sk = scores(np.take_along_axis(x, ids, 1), SOFT)
    S = sk.sum(-1, keepdims=True)
    w = np.where(S == 0, 0.0, sk / np.where(S == 0, 1.0, S) * scale) if renorm else sk * scale
    return ids, w, c, gs, drop


def run(x, k, score, bias=None, groups=1, kept=1, top=1, renorm=True, scale=1.0, bf16=False, L=1, hist=False, R=1,
        stream=None):
    """x float32 [L * T, E]; returns ids, weights (and hist) as numpy."""
    dev = _dev()
    T, E = x.shape[0] // L, x.shape[1]
    cfg = topo.make_cfg(T=T, E=E, k=k, R=R, ranks_per_node=1, n_slot=0)
    o = topo.make_route(score, groups, kept, top, renorm, scale)
    xd = torch.as_tensor(x, device=dev)
    if bf16:
        xd = xd.to(torch.bfloat16)
    nb = topo.topo_workspace_bytes(cfg, L, topo.TOPO_CALL_GATE) if hist else 256
    ws = torch.zeros(nb, dtype=torch.uint8, device=dev)
    ids = torch.full((L, T, k), -7, dtype=torch.int32, device=dev)
    w = torch.full((L, T, k), -7.0, dtype=torch.float32, device=dev)
    h = torch.full((L, R, E), -7, dtype=torch.int32, device=dev) if hist else None
    b = None if bias is None else torch.as_tensor(bias, device=dev)
    topo.topo_route(cfg, L, o, xd, topo.TOPO_DTYPE_BF16 if bf16 else topo.TOPO_DTYPE_F32, b, ids, w, h, ws, nb, stream)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == 0
    out = ids.cpu().numpy().reshape(L * T, k), w.cpu().numpy().reshape(L * T, k)
    return out + (h.cpu().numpy(),) if hist else out


def clear_rows(c, gs, drop, k, kept, gap):
    """Rows whose choice does not hang on less than gap."""
    ok = np.ones(len(c), bool)
    for t in range(len(c)):
        v = np.sort(np.where(drop[t], -np.inf, c[t]))[::-1][:k + 1]
        v = v[np.isfinite(v)]
        ok[t] = len(v) < 2 or np.min(-np.diff(v)) > gap
        if gs is not None and kept < gs.shape[1]:
            g = np.sort(gs[t])[::-1]
            ok[t] &= g[kept - 1] - g[kept] > gap
    return ok


CASES = [
    # T, E, k, score, bias, groups, kept, top, renorm, scale, bf16
    (1, 8, 1, SOFT, False, 1, 1, 1, True, 1.0, False),
    (7, 8, 8, SOFT, False, 1, 1, 1, True, 1.0, False),
    (33, 13, 9, SIG, True, 1, 1, 1, False, 1.0, False),
    (65, 60, 6, SIG, False, 1, 1, 1, True, 2.5, True),
    (129, 64, 8, SOFT, False, 1, 1, 1, False, 1.0, True),
    (200, 128, 8, SOFT, True, 1, 1, 1, True, 1.0, False),
    (90, 139, 5, SOFT, False, 1, 1, 1, True, 1.5, False),
    (300, 256, 8, SIG, True, 8, 4, 2, True, 2.5, False),
    (300, 256, 8, SIG, True, 8, 4, 2, True, 2.5, True),
    (64, 160, 6, SOFT, False, 8, 3, 1, False, 16.0, False),
    (50, 60, 4, SIG, True, 4, 3, 2, False, 1.0, False),
    (40, 96, 12, SIG, True, 32, 9, 2, True, 1.0, False),
    (40, 64, 16, SOFT, False, 4, 1, 1, True, 1.0, False),
    (257, 512, 10, SOFT, False, 1, 1, 1, True, 1.0, False),
    (31, 512, 10, SIG, True, 8, 2, 2, True, 1.0, True),
    (9, 1024, 64, SOFT, False, 1, 1, 1, True, 1.0, False),
    (9, 1000, 33, SIG, True, 4, 2, 2, False, 1.0, False),
    (12, 1023, 17, SIG, False, 1, 1, 1, True, 1.0, True),
]


@gpu
@pytest.mark.parametrize("T,E,k,score,has_bias,groups,kept,top,renorm,scale,bf16", CASES)
def test_route_and_gradient(T, E, k, score, has_bias, groups, kept, top, renorm, scale, bf16):
    rng = np.random.default_rng([T, E, k])
    x = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    if bf16:
        x = torch.as_tensor(x).to(torch.bfloat16).float().numpy()
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32) if has_bias else None
    ids, w = run(x, k, score, bias, groups, kept, top, renorm, scale, bf16)
    rid, rw, c, gs, drop = reference(x, k, score, bias, groups, kept, top, renorm, scale)
    exact = bias is None and top == 1                   # ranked by the logits themselves
    ok = np.ones(T, bool) if exact else clear_rows(c, gs, drop, k, kept, 1e-5)
    assert ok.mean() > 0.9 or E >= 512
    assert np.array_equal(ids[ok], rid[ok])
    assert np.all(np.abs(w[ok] - rw[ok]) <= 64 * U * np.abs(rw[ok]) + 1e-30)
    for t in range(T):                                  # every row: k distinct experts of range
        assert len(set(ids[t])) == k and ids[t].min() >= 0 and ids[t].max() < E

    # the gradient, against the formula in 64 bits for the ids that were chosen
    dev = _dev()
    g = rng.standard_normal((T, k)).astype(np.float32)
    dx = grad(x, ids, g, score, renorm, scale, bf16)
    want, size = grad_reference(x, ids, g, score, renorm, scale)
    tol = (2.0 ** -8 if bf16 else 0.0) * np.abs(want) + 128 * U * size + 1e-30
    assert np.all(np.abs(dx - want) <= tol)
    assert dev.type == "cuda"


def grad(x, ids, g, score, renorm, scale, bf16=False, want_error=0):
    dev = _dev()
    T, E = x.shape
    k = ids.shape[1]
    cfg = topo.make_cfg(T=T, E=E, k=k, R=1, ranks_per_node=1, n_slot=0)
    o = topo.make_route(score, 1, 1, 1, renorm, scale)
    dt = torch.bfloat16 if bf16 else torch.float32
    xd = torch.as_tensor(x, device=dev).to(dt)
    out = torch.full((1, T, E), float("nan"), dtype=dt, device=dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    topo.topo_route_grad(cfg, 1, o, xd, topo.TOPO_DTYPE_BF16 if bf16 else topo.TOPO_DTYPE_F32,
                         torch.as_tensor(ids.astype(np.int32), device=dev), torch.as_tensor(g, device=dev), out, ws, 256)
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == want_error
    return out[0].float().cpu().numpy()


def grad_reference(x, ids, g, score, renorm, scale):
    """The gradient, and the sum of the magnitudes of its terms (dense [T, E])."""
    T, E = x.shape
    g = g.astype(np.float64)
    if score == SOFT and renorm:
        s = np.zeros((T, E))
        np.put_along_axis(s, ids, scores(np.take_along_axis(x, ids, 1), SOFT), 1)
    else:
        s = scores(x, score)
    p = np.take_along_axis(s, ids, 1)
    if renorm:
        S = p.sum(-1, keepdims=True)
        safe = np.where(S == 0, 1.0, S)
        dp = np.where(S == 0, 0.0, scale * (g - (g * p).sum(-1, keepdims=True) / safe) / safe)
        ap = np.where(S == 0, 0.0, scale * (np.abs(g) + (np.abs(g) * p).sum(-1, keepdims=True) / safe) / safe)
    else:
        dp, ap = scale * g, np.abs(scale * g)
    d, a = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(d, ids, dp, 1)
    np.put_along_axis(a, ids, ap, 1)
    if score == SOFT:
        return s * (d - (d * s).sum(-1, keepdims=True)), s * (a + (a * s).sum(-1, keepdims=True))
    return d * s * (1 - s), a * s


@gpu
@pytest.mark.parametrize("score,renorm", [(SOFT, True), (SOFT, False), (SIG, True), (SIG, False)])
def test_gradient_against_differences(score, renorm):
    """Central differences of the 64-bit weights with the ids held fixed; their
    error is h^2 / 6 times a third derivative below 8 in magnitude per term."""
    rng = np.random.default_rng(5)
    T, E, k, scale, h = 6, 24, 5, 2.5, 1e-4
    x = rng.standard_normal((T, E)).astype(np.float32)
    g = rng.standard_normal((T, k)).astype(np.float32)
    ids, _ = run(x, k, score, renorm=renorm, scale=scale)

    def f(xx):
        s = scores(xx, score)
        p = np.take_along_axis(s, ids, 1)
        return ((p / p.sum(-1, keepdims=True) if renorm else p) * scale * g).sum(-1)

    num = np.empty((T, E))
    for e in range(E):
        d = np.zeros((T, E))
        d[:, e] = h
        num[:, e] = (f(x.astype(np.float64) + d) - f(x.astype(np.float64) - d)) / (2 * h)
    dx = grad(x, ids, g, score, renorm, scale)
    size = scale * np.abs(g).sum(-1, keepdims=True)
    assert np.all(np.abs(dx - num) <= size * (8 * h * h / 6 + 128 * U) + 1e-10)


@gpu
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("E", [13, 64, 256, 512])
def test_ties_go_to_the_lowest_expert(score, E):
    k = 6
    x = np.zeros((4, E), np.float32)
    x[1, ::2] = 1.0
    x[2] = -0.0
    x[2, 3] = 0.0                                       # -0 equals +0
    x[3, E - 3:] = 2.0
    bias = np.zeros(E, np.float32)
    for b in (None, bias):
        ids, w = run(x, k, score, b)
        rid, rw, *_ = reference(x, k, score, b)
        assert np.array_equal(ids, rid)
        assert np.allclose(w, rw, rtol=64 * U, atol=0)
    g = 4 if E % 4 == 0 else 1
    ids, _ = run(x, k, score, bias, g, max(1, g // 2), 2)
    assert np.array_equal(ids, reference(x, k, score, bias, g, max(1, g // 2), 2)[0])


@gpu
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,groups,kept", [(16, 1, 1), (64, 8, 2), (256, 8, 4), (500, 1, 1)])
def test_masked_experts(score, renorm, E, groups, kept):
    """-inf logits: masked experts come last whatever their bias, rows with
    fewer than k others give them weight 0, rows without any give only 0."""
    rng = np.random.default_rng(E)
    k = 4
    x = rng.standard_normal((6, E)).astype(np.float32)
    x[0, : E // 2] = -np.inf
    x[1] = -np.inf
    x[2] = -np.inf
    x[2, E - 2] = 0.5
    x[3] = np.finfo(np.float32).min                      # a mask of the lowest finite value
    x[4] = np.finfo(np.float32).min
    x[4, 1] = -3.0
    bias = np.linspace(0.5, -0.5, E).astype(np.float32)
    top = 2 if groups > 1 else 1
    ids, w = run(x, k, score, bias, groups, kept, top, renorm)
    rid, rw, c, gs, drop = reference(x, k, score, bias, groups, kept, top, renorm)
    assert np.array_equal(ids[1:5], rid[1:5])
    assert np.all(np.isfinite(w))
    assert np.allclose(w[1:5], rw[1:5], rtol=64 * U, atol=1e-30)
    assert np.all(w[1] == 0)
    live = np.isfinite(np.take_along_axis(x, ids.astype(np.int64), 1))
    assert np.all(w[~live] == 0)
    dx = grad(x, ids, np.ones((6, k), np.float32), score, renorm, 1.0)
    assert np.all(np.isfinite(dx)) and np.all(dx[1] == 0)


@gpu
@pytest.mark.parametrize("E", [16, 256, 512])
def test_nan_ranks_below_every_number(E):
    rng = np.random.default_rng(E)
    x = rng.standard_normal((5, E)).astype(np.float32)
    x[0, 5] = np.nan
    x[1, : E - 2] = np.nan
    x[2] = np.nan
    ids, w = run(x, 4, SIG)
    assert np.array_equal(ids, order(x)[:, :4])
    assert np.all(np.isfinite(w[0])) and np.all(np.isfinite(w[3:]))
    assert np.all(np.isnan(w[2]))


@gpu
@pytest.mark.parametrize("E,groups,kept", [(24, 1, 1), (256, 8, 4), (160, 8, 3)])
def test_biases_that_mask_experts(E, groups, kept):
    """A bias of -inf takes an expert out of the choice, NaN ranks it last."""
    rng = np.random.default_rng(E)
    x = rng.standard_normal((40, E)).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
    bias[rng.permutation(E)[: E // 3]] = -np.inf
    for b in (bias, np.where(np.arange(E) == 5, np.nan, bias).astype(np.float32)):
        args = (x, 4, SIG, b, groups, kept, 2 if groups > 1 else 1)
        ids, w = run(*args)
        rid, rw, c, gs, drop = reference(*args)
        ok = clear_rows(np.nan_to_num(c, nan=-np.inf), None if gs is None else np.nan_to_num(gs, nan=-1e9), drop, 4, kept, 1e-5)
        assert ok.mean() > 0.9
        assert np.array_equal(ids[ok], rid[ok])
        assert np.all(np.abs(w[ok] - rw[ok]) <= 64 * U * rw[ok])


@gpu
@pytest.mark.parametrize("gap", [0.0, 3e-8, 1e-6, 1e-5])
def test_groups_that_are_nearly_equal(gap):
    """Groups whose scores differ by less than a cheap evaluation could tell: the
    choice is that of the scores as defined, every operation rounded to float32."""
    E, G, kept, k, T = 64, 8, 3, 4, 64
    rng = np.random.default_rng(8)
    x = np.tile(rng.standard_normal((T, 1, E // G)), (1, G, 1)).reshape(T, E).astype(np.float32)
    bias = np.repeat(rng.permutation(G) * gap, E // G).astype(np.float32)
    x += (rng.standard_normal((T, E)) * gap).astype(np.float32)
    ids, _ = run(x, k, SIG, bias, G, kept, 2)
    dev = _dev()
    xd = torch.as_tensor(x, device=dev)
    c = 1.0 / (1.0 + torch.exp(-xd)) + torch.as_tensor(bias, device=dev)      # the definition in float32
    top = torch.sort(c.reshape(T, G, -1), dim=-1, descending=True).values
    keep = torch.sort(top[..., 0] + top[..., 1], dim=-1, descending=True, stable=True).indices[:, :kept]
    on = torch.zeros(T, G, dtype=torch.bool, device=dev).scatter_(1, keep, True).repeat_interleave(E // G, 1)
    want = torch.sort(c.masked_fill(~on, -torch.inf), dim=-1, descending=True, stable=True).indices[:, :k]
    assert np.array_equal(ids, want.cpu().numpy())


@gpu
def test_layers_histogram_and_another_stream():
    rng = np.random.default_rng(3)
    L, T, E, k, R = 3, 96, 32, 4, 4
    x = rng.standard_normal((L * T, E)).astype(np.float32)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ids, w, h = run(x, k, SOFT, L=L, hist=True, R=R, stream=s)
    assert np.array_equal(ids, reference(x, k, SOFT)[0])
    want = np.zeros((L, R, E), np.int32)
    for l in range(L):
        for t in range(T):
            for e in ids[l * T + t]:
                want[l, t // (T // R), e] += 1
    assert np.array_equal(h, want)


@gpu
def test_unaligned_logits_and_no_tokens():
    """Rows that start off a 16-byte boundary take the scalar loads."""
    dev = _dev()
    rng = np.random.default_rng(9)
    T, E, k = 17, 64, 6
    buf = torch.zeros(T * E + 1, dtype=torch.float32, device=dev)
    x = rng.standard_normal((T, E)).astype(np.float32)
    buf[1:] = torch.as_tensor(x.reshape(-1), device=dev)
    cfg = topo.make_cfg(T=T, E=E, k=k, R=1, ranks_per_node=1, n_slot=0)
    o = topo.make_route(SOFT)
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    topo.topo_route(cfg, 1, o, buf.data_ptr() + 4, topo.TOPO_DTYPE_F32, None, ids, w, None, ws, 256)
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), reference(x, k, SOFT)[0])
    empty = topo.make_cfg(T=0, E=E, k=k, R=1, ranks_per_node=1, n_slot=0)
    topo.topo_route(empty, 1, o, None, topo.TOPO_DTYPE_F32, None, None, None, None, ws, 256)
    topo.topo_route_grad(empty, 1, o, None, topo.TOPO_DTYPE_F32, None, None, None, ws, 256)


@gpu
def test_gradient_reports_an_id_outside_the_experts():
    x = np.zeros((2, 8), np.float32)
    ids = np.array([[0, 8], [1, 2]])
    dx = grad(x, ids, np.ones((2, 2), np.float32), SIG, False, 1.0, want_error=topo.TOPO_ERANGE)
    assert np.array_equal(dx[0], [0.25] + [0.0] * 7)     # the valid slot's gradient, nothing else


def test_arguments_are_checked_on_the_host():
    try:
        topo.lib()
    except RuntimeError:
        pytest.skip("library not built")
    a = 1 << 20                                           # never dereferenced
    c = topo.make_cfg(T=8, E=64, k=6, R=1, ranks_per_node=1, n_slot=0)

    def call(cfg=c, o=topo.make_route(SOFT), dt=topo.TOPO_DTYPE_F32, x=a, bias=None, ids=a, w=a, hist=None, ws=a, nb=256):
        topo.topo_route(cfg, 1, o, x, dt, bias, ids, w, hist, ws, nb)

    bad = [dict(o=topo.make_route(2)), dict(o=topo.make_route(SOFT, 0)), dict(o=topo.make_route(SOFT, 7)),
           dict(o=topo.make_route(SOFT, 64, 8)), dict(o=topo.make_route(SOFT, 8, 9)), dict(o=topo.make_route(SOFT, 8, 0)),
           dict(o=topo.make_route(SOFT, 8, 4, 3)), dict(o=topo.make_route(SOFT, 8, 4, 0)),
           dict(o=topo.make_route(SOFT, 32, 2)),          # 2 groups of 2 experts hold no 6
           dict(o=topo.make_route(SOFT, scale=float("inf"))), dict(dt=2), dict(x=a + 2), dict(bias=a + 1), dict(ids=a + 2),
           dict(x=None), dict(ids=None), dict(w=None), dict(ws=None),
           dict(cfg=topo.make_cfg(T=8, E=2048, k=2, R=1, ranks_per_node=1, n_slot=0)),
           dict(cfg=topo.make_cfg(T=8, E=8, k=9, R=1, ranks_per_node=1, n_slot=0))]
    for kw in bad:
        with pytest.raises(topo.TopoError) as ex:
            call(**kw)
        assert ex.value.code == topo.TOPO_EINVAL, kw
    for kw in (dict(nb=255), dict(hist=a)):
        with pytest.raises(topo.TopoError) as ex:
            call(**kw)
        assert ex.value.code == topo.TOPO_ENOSPC
    with pytest.raises(topo.TopoError) as ex:
        topo.topo_route_grad(c, 1, topo.make_route(SOFT), a, topo.TOPO_DTYPE_F32, a, None, a, a, 256)
    assert ex.value.code == topo.TOPO_EINVAL
    with pytest.raises(topo.TopoError) as ex:
        topo.topo_route_grad(c, 1, topo.make_route(SOFT), a, topo.TOPO_DTYPE_F32, a, a, a + 2, a, 256)
    assert ex.value.code == topo.TOPO_EINVAL


@gpu
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E", [8, 64, 256, 500])
def test_softmax_weights_of_rows_far_from_zero(E, bf16):
    """Weights that are not renormalised are shares of the whole row: logits far
    from zero, rows masked to -1e9 or the type's lowest value in whole or in part,
    rows near the type's largest.  The logits of a row that count lie within 16 of
    its largest, whose differences are exact to 16 roundings: the 64 above hold."""
    rng = np.random.default_rng([E, bf16])
    k, scale = 4, 2.5
    low = float(torch.finfo(torch.bfloat16 if bf16 else torch.float32).min)
    x = rng.standard_normal((14, E)).astype(np.float32)
    for i, v in enumerate((100.0, -100.0, 1e4, -1e4, 1e6)):
        x[i] += v
    for i, v in enumerate((-1e9, low, -low, 2.5e38, -1e4, 0.0)):
        x[5 + i] = v
    x[11, : E // 2] = -1e9
    x[12, : E // 2] = low
    x[13] = -np.inf
    x[13, 3] = 300.0
    if bf16:
        x = torch.as_tensor(x).to(torch.bfloat16).float().numpy()
    ids, w = run(x, k, SOFT, renorm=False, scale=scale, bf16=bf16)
    rid, rw, *_ = reference(x, k, SOFT, renorm=False, scale=scale)
    assert np.array_equal(ids, rid)
    assert np.all(np.abs(w - rw) <= 64 * U * rw)
    g = rng.standard_normal(ids.shape).astype(np.float32)
    dx = grad(x, ids, g, SOFT, False, scale, bf16)
    want, size = grad_reference(x, ids, g, SOFT, False, scale)
    assert np.all(np.abs(dx - want) <= (2.0 ** -8 if bf16 else 0.0) * np.abs(want) + 128 * U * size + 1e-30)


@gpu
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_gradient_of_large_logits(renorm):
    """The derivative s (1 - s) is 1 - s near 1: it is held to its own size, to
    which exp and three roundings of each of the two factors count, not to s's."""
    rng = np.random.default_rng(11)
    T, E, k, scale = 40, 24, 5, 2.5
    x = rng.uniform(5, 30, (T, E)).astype(np.float32)
    x[20:] = rng.uniform(-30, 30, (20, E))
    ids, _ = run(x, k, SIG, renorm=renorm, scale=scale)
    g = rng.standard_normal((T, k)).astype(np.float32)
    dx = grad(x, ids, g, SIG, renorm, scale)
    p = np.take_along_axis(scores(x, SIG), ids, 1)
    q = np.take_along_axis(scores(-x, SIG), ids, 1)      # 1 - p
    S = p.sum(-1, keepdims=True) if renorm else np.ones((T, 1))
    dot = (g * p).sum(-1, keepdims=True) / S if renorm else 0.0
    size = (np.abs(g) * p).sum(-1, keepdims=True) / S if renorm else 0.0
    got = np.take_along_axis(dx, ids, 1)
    assert np.all(np.abs(got - scale * (g - dot) * p * q / S) <= 128 * U * scale * (np.abs(g) + size) * p * q / S + 1e-30)


@gpu
@pytest.mark.parametrize("k,scale", [(1, 2.5), (4, 2.5), (4, 1.0), (20, 16.0)])
def test_sigmoid_weights_of_scores_near_underflow(k, scale):
    """Renormalised weights are finite and sum to scale while any chosen score is
    above 0; a score is 0 in float32 below a logit of -88.72, and from -86 down
    it has 21 bits or more: half a unit of the last is 2^-22 = 4 * 2^-24."""
    E, T = 64, 30
    rng = np.random.default_rng(k)
    x = rng.uniform(-88.7, -86, (T, E)).astype(np.float32)
    x[10:] = -95.0
    x[10:20, 7] = np.linspace(-88.7, -86, 10)
    x[10:20, 40] = -88.7
    ids, w = run(x, k, SIG, renorm=True, scale=scale)
    assert np.array_equal(ids, reference(x, k, SIG)[0])
    p = np.where(np.take_along_axis(x, ids, 1) < -88.72, 0.0, np.take_along_axis(scores(x, SIG), ids, 1))
    S = p.sum(-1, keepdims=True)
    want = np.where(S == 0, 0.0, scale * p / np.where(S == 0, 1.0, S))
    assert np.all(np.abs(w - want) <= 64 * U * want)
    g = rng.standard_normal((T, k)).astype(np.float32)
    got = np.take_along_axis(grad(x, ids, g, SIG, True, scale), ids, 1)
    r = want / scale
    dot, size = (g * r).sum(-1, keepdims=True), (np.abs(g) * r).sum(-1, keepdims=True)
    assert np.all(np.abs(got - scale * r * (g - dot)) <= 128 * U * scale * r * (np.abs(g) + size) + 1e-30)


def group_choice(x, bias, G, kept, k):
    """The ids of the definition in float32, every operation rounded."""
    xd = torch.as_tensor(x, device=_dev())
    c = 1.0 / (1.0 + torch.exp(-xd)) + torch.as_tensor(bias, device=xd.device)
    T, E = x.shape
    top = torch.sort(c.reshape(T, G, -1), dim=-1, descending=True).values
    keep = torch.sort(top[..., 0] + top[..., 1], dim=-1, descending=True, stable=True).indices[:, :kept]
    on = torch.zeros(T, G, dtype=torch.bool, device=xd.device).scatter_(1, keep, True).repeat_interleave(E // G, 1)
    return torch.sort(c.masked_fill(~on, -torch.inf), dim=-1, descending=True, stable=True).indices[:, :k].cpu().numpy()


@gpu
@pytest.mark.parametrize("which", ["all", "one"])
@pytest.mark.parametrize("size", [32.0, 64.0, 500.0, 1e6])
def test_group_scores_whose_biases_cancel(size, which):
    """The two largest values of a group near +size and -size: their sum is
    small, its rounding is not.  Groups alike up to a few such roundings."""
    E, G, kept, k, T = 64, 8, 3, 4, 4096
    rng = np.random.default_rng([int(size), which == "one"])
    x = np.tile(rng.standard_normal((T, 1, E // G)), (1, G, 1)).reshape(T, E)
    x = (x + rng.standard_normal((T, E)) * size * 2.0 ** -22).astype(np.float32)
    bias = np.full((G, E // G), -size, np.float32)
    bias[:, 0] = size
    if which == "one":                                   # the others reach the same sums without cancelling
        bias[1:] = np.array([0.0, 0.0] + [-4.0] * (E // G - 2), np.float32)
        x = x.reshape(T, G, -1)
        x[:, :, 1:] = np.minimum(x[:, :, 1:], x[:, :, 1:2])
        x = x.reshape(T, E)
    bias = bias.reshape(-1)
    ids, _ = run(x, k, SIG, bias, G, kept, 2)
    assert np.array_equal(ids, group_choice(x, bias, G, kept, k))


@gpu
def test_group_scores_that_overflow():
    """Sums of two biases past the largest float32 are equal: the lower group stays."""
    E, G, k, T = 64, 8, 4, 33
    x = np.random.default_rng(3).standard_normal((T, E)).astype(np.float32)
    bias = np.zeros(E, np.float32)
    bias[[17, 18, 41, 42]] = 3e38
    ids, _ = run(x, k, SIG, bias, G, 1, 2)
    assert np.array_equal(ids, group_choice(x, bias, G, 1, k))
    assert np.all(ids // 8 == 2)
