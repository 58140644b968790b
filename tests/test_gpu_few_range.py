"""The experts of a few tokens with weights and tokens far from 1: the row scales' order and
every scale byte.  Bounds are those of the call's own test."""
import pytest

import moe_expert_routing_ids_gb300 as topo
from test_gpu_few import MX, NV, Case
from test_gpu_micro import BLOCK, values

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


def check(c):
    got, ws = c.run()
    torch.cuda.synchronize()
    assert topo.topo_read_error(ws) == 0
    want, tol = c.want()
    assert float(want.abs().max()) < 3e38 and bool((want != 0).any())
    assert bool(((got.double().cpu() - want).abs() <= tol + 2.0 ** -133).all())   # bf16's last step of all


@gpu
@pytest.mark.parametrize("T,k,H,I", [(1, 2, 128, 64), (8, 2, 512, 96), (32, 3, 96, 160)])
@pytest.mark.parametrize("up,x,down", [(112, -112, 0), (-100, 100, 0), (0, -10, 112), (90, -100, 100), (-60, 60, -90), (112, -118, 112), (0, 0, 0)])
def test_row_scales_far_from_one(up, x, down, T, k, H, I):
    """The sums are over a power of two of the token's row, which may take back what the weights'
    row scale adds: neither order of the two alone stays inside float32's range."""
    c = Case(T, 6, k, H, I, NV, seed=11)
    for part, v, e in (("up", "vu", up), ("down", "vd", down)):
        t = getattr(c, part)
        t[2].mul_(2.0 ** e)
        assert bool(((t[2] > 0) & torch.isfinite(t[2])).all())
        setattr(c, v, getattr(c, v) * 2.0 ** e)
    c.x = (c.x.double() * 2.0 ** x).to(torch.bfloat16)
    check(c)


@gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("T,k,H,I", [(1, 2, 128, 64), (8, 2, 544, 96), (32, 3, 96, 288)])
def test_every_scale_byte(fmt, T, k, H, I):
    """Subnormal e4m3 scales and 0; powers of two down to 2^-127, and of W_down up to 2^99."""
    c = Case(T, 6, k, H, I, fmt, seed=12)
    gen = torch.Generator().manual_seed(13)
    for part, v, K, top in (("up", "vu", H, 127), ("down", "vd", I, 227)):
        q, s, r = getattr(c, part)
        n = K // BLOCK[fmt]
        s[..., :n] = torch.randint(0, 127 if fmt == NV else top, (*s.shape[:-1], n), generator=gen).to(torch.uint8).to(c.dev)
        if fmt == MX and part == "up":                            # near 1 in every third block, far below elsewhere
            s[..., :n:3] = torch.randint(118, 126, s[..., :n:3].shape, generator=gen).to(torch.uint8).to(c.dev)
        setattr(c, v, torch.as_tensor(values(q.cpu().numpy(), s.cpu().numpy(), None if r is None else r.cpu().double().numpy(), fmt)))
    check(c)
