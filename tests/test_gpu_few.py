"""The experts applied to a few tokens, in 8 and in 4 bits, against the formulas in
64 bits on the values that the weights' codes and scales stand for.

Tolerances.  u = 2^-24.  A product of K terms is summed in float32, 16 products at a
time with at least 23 bits below the largest, and each block's sum is scaled and
added (three roundings): |error| <= c(K) * A with c(K) = (K / 16 + 3 K / 16 + 8) * 2 u and A the sum
of the terms' magnitudes (splitting the contraction adds less than the 8).  The
tokens' f16 form is exact for bf16 values within 2^-28 of the row's largest and off by
2^-39 of that one otherwise (down to f16's step 2^-24 below 2^14): it adds 2^-38 *
max|x| * sum|w|.  a = silu(g) u with errors dg, du is off by
1.1 |u| dg + (|silu(g)| + 1.1 dg) du + 2^-20 |a| (|silu'| <= 1.1; expf within 2 units, two divisions'
roundings), and 2^-11 |a| more as f16, 2^-38 max|a| for small ones.  The weighted sum
adds (k + 1) u of its terms, bf16 2^-8 of the result."""
import numpy as np
import pytest

import moe_expert_routing_ids_gb300 as topo
from test_gpu_micro import values

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
EIGHT, MX, NV = topo.TOPO_FMT_EIGHT, topo.TOPO_FMT_MX, topo.TOPO_FMT_NV


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def weights(gen, E, N, K, fmt, dev):
    """(q, scale, row scales) on the device and their values in float64 [E, N, K]."""
    w = (torch.randn(E, N, K, generator=gen) / K ** 0.5 * torch.exp(torch.randn(E, N, 1, generator=gen))).to(torch.bfloat16).to(dev)
    if fmt == EIGHT:
        kb, nb = (K + 127) // 128, (N + 127) // 128
        q = torch.empty(E, N, K, dtype=torch.uint8, device=dev)
        s = torch.empty(E, nb, kb, device=dev)
        topo.topo_quantize_weight(E, N, K, w, q, s)
        s *= torch.rand(E, nb, kb, generator=gen).to(dev) + 0.5    # any float32
        v = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[..., :K]
        return (q, s, None), v.cpu()
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=dev)
    s = torch.empty(E, N, topo.topo_micro_pitch(K, fmt), dtype=torch.uint8, device=dev)
    r = torch.empty(E, N, device=dev) if fmt == NV else None
    topo.topo_quantize_rows_micro(E * N, K, fmt, w, q, s, r)
    v = values(q.cpu().numpy(), s.cpu().numpy(), None if r is None else r.cpu().double().numpy(), fmt)
    return (q, s, r), torch.as_tensor(v)


class Case:
    def __init__(self, T, E, k, H, I, fmt, seed=0, hot=False):
        self.dims, self.fmt, self.dev = (T, E, k, H, I), fmt, _dev()
        gen = torch.Generator().manual_seed(seed)
        self.up, self.vu = weights(gen, E, 2 * I, H, fmt, self.dev)
        self.down, self.vd = weights(gen, E, H, I, fmt, self.dev)
        self.x = (torch.randn(T, H, generator=gen) * torch.exp(2 * torch.randn(T, 1, generator=gen))).to(torch.bfloat16)
        self.ids = torch.rand(T, E, generator=gen).argsort(1)[:, :k].to(torch.int32) if k <= E else torch.randint(0, E, (T, k), generator=gen).to(torch.int32)
        if hot:
            self.ids = torch.randint(0, 2, (T, k), generator=gen).to(torch.int32)
        self.w = torch.rand(T, k, generator=gen)

    def buffers(self):
        T, E, k, H, I = self.dims
        nb = topo.topo_few_workspace_bytes(T, E, k, H, I)
        ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device=self.dev)
        topo.topo_ws_reset(ws, nb)
        return torch.full((T, H), 7.0, dtype=torch.bfloat16, device=self.dev), ws, nb

    def run(self, buf=None, x=None, stream=None):
        T, E, k, H, I = self.dims
        out, ws, nb = buf or self.buffers()
        on = [t.to(self.dev) for t in (self.x if x is None else x, self.ids, self.w)]
        topo.topo_expert_few(T, E, k, H, I, self.fmt, *on, *self.up, *self.down, out, ws, nb, stream)
        return out, ws

    def want(self):
        T, E, k, H, I = self.dims
        u = 2.0 ** -24
        x, w = self.x.double(), self.w.double()
        out, tol = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
        for t in range(T):
            for j in range(k):
                e = int(self.ids[t, j])
                if not 0 <= e < E:
                    continue
                m, d = self.vu[e], self.vd[e]
                c = (4 * H / 16 + 8) * 2 * u
                h = m @ x[t]
                dh = c * (m.abs() @ x[t].abs()) + 2.0 ** -38 * x[t].abs().max() * m.abs().sum(1)
                g, v = h[:I], h[I:]
                s = g * torch.sigmoid(g)
                a = s * v
                da = 1.1 * v.abs() * dh[:I] + (s.abs() + 1.1 * dh[:I]) * dh[I:] + 2.0 ** -20 * a.abs()
                da = da + 2.0 ** -11 * (a.abs() + da) + 2.0 ** -38 * (a.abs() + da).max()
                y, A = d @ a, d.abs() @ (a.abs() + da)
                out[t] += w[t, j] * y
                tol[t] += w[t, j] * (d.abs() @ da + (4 * I / 16 + 8 + k + 1) * 2 * u * A)
        return out, tol + 2.0 ** -8 * out.abs()


@gpu
@pytest.mark.parametrize("fmt", [EIGHT, MX, NV])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 32, 32), (1, 8, 2, 1024, 768), (2, 5, 3, 160, 96), (8, 16, 4, 288, 1056),
                                       (7, 64, 6, 512, 64), (9, 12, 8, 256, 128), (32, 40, 2, 96, 320), (3, 4, 64, 64, 32),
                                       (5, 300, 2, 32, 64), (1, 9, 8, 7168, 256), (4, 3, 2, 64, 4096), (8, 6, 6, 8224, 64),
                                       (8, 1024, 8, 64, 32), (32, 3, 2, 7168, 32), (20, 2, 1, 5152, 64), (32, 20, 16, 7168, 32),
                                       (3, 2, 2, 32768, 32), (32, 2, 1, 8224, 32), (5, 2, 2, 64, 16416), (1, 1, 1, 32, 32768),
                                       (32, 1, 1, 64, 9248), (20, 6, 64, 64, 32), (17, 1, 1, 32768, 32),
                                       (32, 2, 16, 7168, 32), (32, 2, 16, 64, 9248), (32, 200, 16, 4128, 32)])
def test_few(T, E, k, H, I, fmt):
    c = Case(T, E, k, H, I, fmt)
    got, ws = c.run()
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == 0
    want, tol = c.want()
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@gpu
@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 16, 16), (6, 7, 3, 144, 272), (8, 3, 2, 4112, 48)])
def test_few_in_eight_bits_at_multiples_of_16(T, E, k, H, I):
    c = Case(T, E, k, H, I, EIGHT, seed=1)
    got, ws = c.run()
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == 0
    want, tol = c.want()
    assert bool(((got.double().cpu() - want).abs() <= tol).all())


@gpu
@pytest.mark.parametrize("fmt", [EIGHT, MX, NV])
def test_an_expert_named_twice_and_all_tokens_on_two(fmt):
    c = Case(8, 6, 4, 128, 160, fmt, seed=2, hot=True)
    got, ws = c.run()
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == 0
    want, tol = c.want()
    assert bool(((got.double().cpu() - want).abs() <= tol).all())


@gpu
@pytest.mark.parametrize("fmt", [EIGHT, NV])
def test_ids_outside_and_tokens_without_an_expert(fmt):
    c = Case(5, 6, 3, 64, 32, fmt, seed=3)
    c.ids[0] = torch.tensor([-1, 6, 1 << 30])
    c.ids[1, 2] = 70000
    got, ws = c.run()
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == topo.TOPO_ERANGE
    want, tol = c.want()
    assert bool(((got.double().cpu() - want).abs() <= tol).all()) and not bool(got[0].any())
    c.ids[:] = -1
    got, ws = c.run()
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == topo.TOPO_ERANGE and not bool(got.any())


@gpu
@pytest.mark.parametrize("fmt", [EIGHT, MX, NV])
def test_rows_of_zeros_small_large_and_not_finite(fmt):
    c = Case(8, 6, 2, 256, 96, fmt, seed=4)
    c.w[3] = 0.0
    c.x[0] = 0
    c.x[1] *= 2.0 ** -60
    c.x[2] = (c.x[2].float() * 2.0 ** 20).to(torch.bfloat16)
    c.x[4, 7] = 2.0 ** -133
    plain, _ = c.run()
    want, tol = c.want()
    assert bool(((plain.double().cpu() - want).abs() <= tol + 2.0 ** -133).all())
    bad = c.x.clone()
    bad[5, 9], bad[6, 250] = float("nan"), float("-inf")
    got, _ = c.run(x=bad)
    fin = torch.isfinite(got).all(1).cpu()
    assert fin.tolist() == [True] * 5 + [False, False, True]
    keep = [0, 1, 2, 3, 4, 7]
    assert torch.equal(got[keep], plain[keep]) and not bool(torch.isfinite(got[5:7]).any())


@gpu
@pytest.mark.parametrize("fmt", [EIGHT, MX, NV])
def test_weights_that_are_nan_reach_their_tokens_only(fmt):
    """A NaN weight (8 bits) or scale (4 bits) of expert 2 in W_up's gate rows, then in W_down."""
    c = Case(8, 6, 2, 256, 96, fmt, seed=9)
    plain, _ = c.run()
    for part, row in (("up", 17), ("down", 40)):
        t = list(getattr(c, part))
        i = 0 if fmt == EIGHT else 1
        kept = t[i].clone()
        t[i][2, row, 0] = {EIGHT: 0x7f, MX: 0xff, NV: 0x7f}[fmt]
        got, ws = c.run()
        t[i].copy_(kept)
        hit = (c.ids == 2).any(1)
        assert hit.any() and not hit.all()
        fin = torch.isfinite(got).cpu()
        assert bool(fin[~hit].all()) and torch.equal(got[~hit], plain[~hit])
        # through W_up a NaN activation reaches all of a token, through W_down the row's column
        assert not bool(fin[hit].any()) if part == "up" else fin[hit].sum(1).eq(255).all() and not bool(fin[hit][:, 40].any())


@gpu
@pytest.mark.parametrize("fmt", [EIGHT, MX, NV])
def test_few_repeats_and_a_workspace_is_used_again(fmt):
    c = Case(8, 32, 6, 1024, 256, fmt, seed=5)
    buf = c.buffers()
    first = c.run(buf)[0].clone()
    small = Case(3, 8, 2, 64, 32, fmt, seed=6)
    want = small.run()[0].clone()
    for _ in range(20):
        assert torch.equal(c.run(buf)[0], first)
        T, E, k, H, I = small.dims
        assert torch.equal(small.run((torch.empty(T, H, dtype=torch.bfloat16, device=c.dev), buf[1], buf[2]))[0], want)
    assert topo.topo_read_error(buf[1]) == 0


@gpu
@pytest.mark.parametrize("fmt", [EIGHT, MX])
def test_a_token_alone_and_in_a_batch(fmt):
    """The tokens beside it do not change a token's bits but through the order of the sums (f32)."""
    c = Case(8, 16, 4, 512, 256, fmt, seed=7)
    both, _ = c.run()
    one = Case(8, 16, 4, 512, 256, fmt, seed=7)
    one.dims, one.x, one.ids, one.w = (1, 16, 4, 512, 256), c.x[3:4], c.ids[3:4], c.w[3:4]
    got, _ = one.run()
    want, tol = one.want()
    assert bool(((got.double().cpu() - want).abs() <= tol).all())
    assert float((got.float() - both[3:4].float()).abs().max()) <= 2.0 ** -7 * float(both[3].float().abs().max())


@gpu
@pytest.mark.parametrize("fmt", [EIGHT, NV])
def test_two_calls_at_once_on_two_streams_and_in_graphs(fmt):
    cs = [Case(4, 16, 4, 512, 256, fmt, seed=8 + i) for i in range(2)]
    want = [c.run()[0].clone() for c in cs]
    torch.cuda.synchronize()
    on = [[t.to(c.dev) for t in (c.x, c.ids, c.w)] for c in cs]
    bufs, streams = [c.buffers() for c in cs], [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()

    def call(i, stream):
        out, ws, nb = bufs[i]
        topo.topo_expert_few(*cs[i].dims, fmt, *on[i], *cs[i].up, *cs[i].down, out, ws, nb, stream)

    for _ in range(10):
        for i in (0, 1):
            bufs[i][0].zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for i in (0, 1):
                call(i, streams[i])
        torch.cuda.synchronize()
        assert all(torch.equal(bufs[i][0], want[i]) for i in (0, 1))
    graphs = []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, torch.cuda.current_stream())
            call(i, torch.cuda.current_stream())
        graphs.append(g)
    for _ in range(3):
        for i in (0, 1):
            bufs[i][0].zero_()
            graphs[i].replay()
        assert all(torch.equal(bufs[i][0], want[i]) for i in (0, 1))


def test_refusals():
    """Before anything is enqueued: no GPU is touched."""
    try:
        topo.lib()
    except RuntimeError:
        pytest.skip("library not built")
    p, odd = 1 << 20, (1 << 20) + 8
    names = "T E k H I fmt x ids w up us ur down ds dr out ws nb".split()
    nb = topo.topo_few_workspace_bytes(4, 8, 2, 64, 32)
    assert nb > 4 * 2 * (64 + 32) * 4
    ok = dict(zip(names, [4, 8, 2, 64, 32, MX, p, p, p, p, p, None, p, p, None, p, p, nb]))

    def refused(code=topo.TOPO_EINVAL, **change):
        with pytest.raises(topo.TopoError) as ex:
            topo.topo_expert_few(*{**ok, **change}.values())
        assert ex.value.code == code

    for change in (dict(T=-1), dict(T=33), dict(E=0), dict(E=1025), dict(k=0), dict(k=65), dict(H=48), dict(I=16), dict(H=0),
                   dict(H=1 << 16), dict(I=1 << 16), dict(fmt=3), dict(fmt=-1), dict(fmt=EIGHT, H=40), dict(x=None), dict(x=odd),
                   dict(ids=None), dict(ids=p + 2), dict(w=None), dict(w=p + 1), dict(up=None), dict(up=odd), dict(us=None),
                   dict(us=odd), dict(ur=p), dict(dr=p), dict(fmt=NV), dict(fmt=NV, ur=p), dict(fmt=EIGHT, ur=p), dict(down=odd),
                   dict(ds=odd), dict(out=None), dict(out=odd), dict(ws=None), dict(ws=odd)):
        refused(**change)
    refused(code=topo.TOPO_ENOSPC, nb=nb - 1)
    assert topo.topo_expert_few(*{**ok, "T": 0}.values()) == 0
    for H, I, k in ((7168, 2048, 8), (32768, 32768, 64), (64, 32, 2), (4112, 48, 6), (5152, 9248, 3)):
        sizes = [topo.topo_few_workspace_bytes(T, 64, k, H, I) for T in range(33)]
        assert sizes == sorted(sizes) and sizes[1] > 256          # one made for more tokens serves fewer
    for dims in ((-1, 8, 2, 64, 32), (33, 8, 2, 64, 32), (4, 0, 2, 64, 32), (4, 8, 65, 64, 32), (4, 8, 2, 8, 32), (4, 8, 2, 64, 1 << 16)):
        assert topo.topo_few_workspace_bytes(*dims) == 0
