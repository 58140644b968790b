"""Cases of the expert layer's operators: routing, 8-bit quantisation, the experts' products and the gated activation.

Each case is one call (or one training step's calls) of the expert layer; the sizes are those of the framework's
workloads (hidden 1024 / 2048 / 4096 / 7168, 8 to 512 experts, k = 2 to 10) or generic.  With ``own`` false, ``run``
computes the operators from their formulas with elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False
BLOCK = 128          # values along the contraction that share one scale
DEV = "cuda"


# ------------------------------------------------------------------------------------------------- cases
def _route(name, T, E, k, score, dtype="f32", bias=False, groups=1, kept=1, group_top=1, renorm=True, scale=1.0,
           grad=False):
    return dict(name=name, op="route", T=T, E=E, k=k, score=score, dtype=dtype, bias=bias, groups=groups, kept=kept,
                group_top=group_top, renorm=renorm, scale=scale, grad=grad)


def listed():
    return [
        # one decoding step of a small batch: sigmoid scores with a balance bias, 4 of 8 groups
        _route("route_decode", 48, 256, 8, "sigmoid", bias=True, groups=8, kept=4, group_top=2, scale=2.5),
        # a prefill chunk with the same router
        _route("route_prefill_groups", 65536, 256, 8, "sigmoid", bias=True, groups=8, kept=4, group_top=2, scale=2.5),
        # a training microbatch of a million tokens: softmax router, forward and gradient
        _route("route_train_softmax", 1048576, 512, 10, "softmax", grad=True),
        # dispatch of a decoding batch to odd hidden sizes, and of a long prefill
        dict(name="dispatch_small", op="dispatch", T=333, E=64, k=6, H=1408),
        dict(name="dispatch_prefill", op="dispatch", T=65536, E=256, k=8, H=7168),
        # one token's pairs through the down projection: latency
        dict(name="product_one_token", op="product", rows=6, E=64, N=4096, K=1408, skew=0.0, out="bf16"),
        # a decoding batch: every expert gets a few rows, the weights are the traffic
        dict(name="product_decode", op="product", rows=1536, E=64, N=2816, K=4096, skew=0.6, out="bf16"),
        # prefill of 16384 tokens, k = 8, experts unevenly loaded
        dict(name="product_prefill", op="product", rows=131072, E=128, N=4096, K=7168, skew=0.8, out="bf16"),
        # the activation between the two products: a decoding batch, and a training step with its gradient
        dict(name="swiglu_decode", op="swiglu", rows=1000, I=1408, grad=False),
        dict(name="swiglu_train", op="swiglu", rows=131072, I=2048, grad=True),
        # weight gradients of a small layer with ragged experts, and of a 16384-token microbatch, k = 6
        dict(name="wgrad_small", op="wgrad", rows=8190, E=8, N=1536, K=1024, skew=1.0),
        dict(name="wgrad_train", op="wgrad", rows=98304, E=64, N=2816, K=4096, skew=0.8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, hi, units=(16, 128, 512)):
    """An odd multiple of 16, 128 or 512, up to hi: whole and partial scale blocks."""
    unit = rng.choice([u for u in units if u <= hi])
    return unit * (2 * _log(rng, 1, (hi // unit + 1) // 2) - 1)


def draw(rng):
    op = rng.choice(["route", "route", "dispatch", "product", "product", "product", "swiglu", "wgrad"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        score = "sigmoid" if groups > 1 else rng.choice(["softmax", "sigmoid"])
        E = groups * _log(rng, 8, 512 // groups) if groups > 1 else _log(rng, 8, 512)
        kept = rng.randint(max(1, groups // 2), groups)
        renorm = rng.random() < 0.7
        k = rng.randint(2 if renorm else 1, min(10, kept * (E // groups)))     # one renormalised weight has no gradient
        return dict(op="route", T=_log(rng, 1, 262144), E=E, k=k, score=score, dtype=rng.choice(["f32", "f32", "bf16"]),
                    bias=score == "sigmoid" and rng.random() < 0.7, groups=groups, kept=kept,
                    group_top=2 if groups > 1 else 1, renorm=renorm, scale=rng.choice([1.0, 2.5]),
                    grad=rng.random() < 0.5)
    if op == "dispatch":
        E = _log(rng, 8, 256)
        return dict(op="dispatch", T=_log(rng, 1, 32768), E=E, k=rng.randint(1, 8), H=_size(rng, 7168))
    if op == "product":
        E = _log(rng, 1, 128)
        return dict(op="product", rows=_log(rng, 1, 65536), E=E, N=_size(rng, 4096), K=_size(rng, 7168),
                    skew=rng.choice([0.0, 0.6, 1.2]), out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "swiglu":
        return dict(op="swiglu", rows=_log(rng, 1, 131072), I=_size(rng, 2048, (16, 128)), grad=rng.random() < 0.5)
    return dict(op="wgrad", rows=_log(rng, 1, 65536), E=_log(rng, 1, 64), N=_size(rng, 2816),
                K=_size(rng, 4096), skew=rng.choice([0.0, 0.6, 1.2]))


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ------------------------------------------------------------------------------------------------ inputs
def _counts(seed, rows, E, skew):
    """Rows of each expert: a multinomial draw over Zipf(skew) shares in a seeded order."""
    r = np.random.default_rng([seed, rows, E])
    p = np.arange(1, E + 1, dtype=np.float64) ** -skew
    p = r.permutation(p / p.sum())
    return r.multinomial(rows, p)


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), device=DEV)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _rows8(gen, rows, K):
    """Quantised activation rows: e4m3 values whose blocks reach up to 448, with a power of two for each block."""
    KB = _blocks(K)
    q = (_randn(gen, rows, K) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    e = torch.randint(-10, -5, (rows, KB), generator=gen, device=DEV)
    return q, torch.exp2(e.float())


def _weights8(gen, E, N, K):
    """Quantised expert weights [E, N, K] with a float32 scale for each 128 x 128 block."""
    q = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    for e in range(E):
        q[e] = (_randn(gen, N, K) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s = torch.rand((E, _blocks(N), _blocks(K)), generator=gen, device=DEV) * 1e-4 + 1e-4
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, st = case["op"], dict(case=case)
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        x = _randn(gen, 1, T, E).mul_(1.5)
        st["logits"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        st["bias"] = _randn(gen, E) * 0.05 if case["bias"] else None
        st["grad"] = _randn(gen, 1, T, k) if case["grad"] else None
    elif op == "dispatch":
        T, E, k, H = case["T"], case["E"], case["k"], case["H"]
        st["x"] = (_randn(gen, T, H) * torch.exp(_randn(gen, T, 1))).to(torch.bfloat16)
        ids = torch.rand((T, E), generator=gen, device=DEV).topk(k, dim=1).indices.reshape(-1)
        st["sorted_pairs"] = torch.sort(ids, stable=True).indices.to(torch.int32)
    elif op == "product":
        counts = _counts(seed, case["rows"], case["E"], case["skew"])
        st["lens"] = [int(c) for c in counts]
        st["seg_off"] = _offsets(counts)
        st["a"], st["a_scale"] = _rows8(gen, case["rows"], case["K"])
        st["w"], st["w_scale"] = _weights8(gen, case["E"], case["N"], case["K"])
    elif op == "swiglu":
        st["h"] = (_randn(gen, case["rows"], 2 * case["I"]) * 2).to(torch.bfloat16)
        st["dy"] = _randn(gen, case["rows"], case["I"]).to(torch.bfloat16) if case["grad"] else None
    else:
        counts = _counts(seed, case["rows"], case["E"], case["skew"])
        st["lens"] = [int(c) for c in counts]
        st["seg_off"] = _offsets(counts)
        st["dy"] = (_randn(gen, case["rows"], case["N"]) * 1e-3).to(torch.bfloat16)
        st["x"] = _randn(gen, case["rows"], case["K"]).to(torch.bfloat16)
    return st


# -------------------------------------------------------------------------------------------- plain forms
def _scale_of(amax):
    """The smallest power of two that is at least amax / 448 (exponent at least -126; 1 for amax = 0)."""
    m, e = torch.frexp(amax)                                   # amax = m * 2^e, m in [0.5, 1)
    n = (e.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)).clamp(min=-126)
    s = ((n + 127) << 23).view(torch.float32)
    return torch.where(amax > 0, s, torch.ones_like(s))


def _quant(x):
    """x float32 [..., C] -> (e4m3 [..., C], scale [..., ceil(C / 128)])."""
    C, KB = x.shape[-1], _blocks(x.shape[-1])
    p = torch.nn.functional.pad(x, (0, KB * BLOCK - C)).reshape(*x.shape[:-1], KB, BLOCK)
    s = _scale_of(torch.where(torch.isfinite(p), p.abs(), torch.zeros_like(p)).amax(-1))
    q = (p * (1.0 / s)[..., None]).reshape(*x.shape[:-1], KB * BLOCK)[..., :C]
    return q.to(torch.float8_e4m3fn), s


def _dequant_rows(q, s):
    return q.float() * s.repeat_interleave(BLOCK, dim=-1)[..., :q.shape[-1]]


def _plain_route(st):
    c = st["case"]
    E, k, G, scale = c["E"], c["k"], c["groups"], c["scale"]
    x = st["logits"][0].float()
    if c["score"] == "softmax":
        m = x.amax(-1, keepdim=True)
        ex = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
        tot = ex.sum(-1, keepdim=True)
        s = torch.where(tot > 0, ex / tot, torch.zeros_like(ex))
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    sel = x if st["bias"] is None and c["group_top"] == 1 else s + (st["bias"] if st["bias"] is not None else 0.0)
    sel = torch.where(torch.isneginf(x), x, sel)
    if G > 1:
        top = torch.sort(sel.reshape(-1, G, E // G), dim=-1, descending=True).values
        gs = top[..., 0] + top[..., 1] if c["group_top"] == 2 else top[..., 0]
        keep = torch.sort(gs, dim=-1, descending=True, stable=True).indices[:, :c["kept"]]
        on = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, keep, True).repeat_interleave(E // G, dim=1)
        sel = torch.where(on, sel, torch.full_like(sel, -math.inf))
    ids = torch.sort(sel, dim=-1, descending=True, stable=True).indices[:, :k]
    sk = torch.gather(s, 1, ids)
    S = sk.sum(-1, keepdim=True)
    w = torch.where(S > 0, sk * (scale / S), torch.zeros_like(sk)) if c["renorm"] else sk * scale
    out = dict(ids=ids.to(torch.int32)[None], weights=w[None])
    if st["grad"] is not None:
        g = st["grad"][0]
        dx = torch.zeros_like(x)
        if c["score"] == "softmax" and not c["renorm"]:
            dx = -s * (g * w).sum(-1, keepdim=True)
            dx.scatter_add_(1, ids, g * w)
        elif c["score"] == "softmax":
            dx.scatter_(1, ids, w * (g - (g * w).sum(-1, keepdim=True) / scale))
        elif c["renorm"]:
            d = sk * (1 - sk) * (g * scale - (g * w).sum(-1, keepdim=True)) / S
            dx.scatter_(1, ids, torch.where(S > 0, d, torch.zeros_like(d)))
        else:
            dx.scatter_(1, ids, g * scale * sk * (1 - sk))
        out["grad_logits"] = dx.to(st["logits"].dtype)[None]
    return out


def _plain_dispatch(st):
    q, s = _quant(st["x"].float())
    t = (st["sorted_pairs"] // st["case"]["k"]).long()
    return dict(q=q.view(torch.uint8)[t].view(torch.float8_e4m3fn), scale=s[t])


def _plain_product(st):
    c = st["case"]
    N, K = c["N"], c["K"]
    out = torch.empty((c["rows"], N), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
    a = _dequant_rows(st["a"], st["a_scale"])
    at = 0
    for e, n in enumerate(st["lens"]):                         # one product for each expert's rows
        if n:
            ws = st["w_scale"][e].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
            out[at:at + n] = (a[at:at + n] @ (st["w"][e].float() * ws).t()).to(out.dtype)
            at += n
    return out


def _plain_swiglu(st):
    I = st["case"]["I"]
    g, u = st["h"][:, :I].float(), st["h"][:, I:].float()
    q, s = _quant(g / (1.0 + torch.exp(-g)) * u)
    out = dict(q=q, scale=s)
    if st["dy"] is not None:
        dy, sg = st["dy"].float(), 1.0 / (1.0 + torch.exp(-g))
        out["dh"] = torch.cat([dy * u * sg * (1.0 + g * (1.0 - sg)), dy * g * sg], 1).to(torch.bfloat16)
    return out


def _block_quant_cols(x, lens):
    """Rows quantised down each column over 128-row blocks counted from each segment's first row, dequantised."""
    C = x.shape[1]
    starts, at, pos = [], 0, 0
    rows = np.empty(x.shape[0], np.int64)                      # padded position of each row
    for n in lens:
        rows[at:at + n] = pos + np.arange(n)
        at, pos = at + n, pos + _blocks(n) * BLOCK
    rows = torch.as_tensor(rows, device=DEV)
    p = torch.zeros((pos, C), dtype=torch.float32, device=DEV)
    p[rows] = x.float()
    p = p.reshape(-1, BLOCK, C)
    s = _scale_of(torch.where(torch.isfinite(p), p.abs(), torch.zeros_like(p)).amax(1))
    q = (p * (1.0 / s)[:, None, :]).to(torch.float8_e4m3fn)
    return (q.float() * s[:, None, :]).reshape(-1, C)[rows]


def _plain_wgrad(st):
    c = st["case"]
    dy, x = _block_quant_cols(st["dy"], st["lens"]), _block_quant_cols(st["x"], st["lens"])
    dw = torch.zeros((c["E"], c["N"], c["K"]), dtype=torch.float32, device=DEV)
    at = 0
    for e, n in enumerate(st["lens"]):                         # one product for each expert's rows
        if n:
            dw[e] = dy[at:at + n].t() @ x[at:at + n]
            at += n
    return dw


# ------------------------------------------------------------------------------- the framework's operators
def _kept(st, key, make):
    """What a program that makes this call each step keeps between the steps: output buffers, options, workspace."""
    if key not in st:
        st[key] = make()
    return st[key]


def _empty(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _header(topo):
    n = topo.topo_workspace_bytes(None, 0, topo.TOPO_CALL_COOCCUR)
    return torch.zeros(n, dtype=torch.uint8, device=DEV), n


def _own_route(topo, st, stream):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = st["logits"]
    dt = topo.TOPO_DTYPE_BF16 if x.dtype == torch.bfloat16 else topo.TOPO_DTYPE_F32

    def make():
        cfg = topo.make_cfg(T=T, E=E, k=k, R=1, ranks_per_node=1, n_slot=0)
        opts = topo.make_route(topo.TOPO_SCORE_SOFTMAX if c["score"] == "softmax" else topo.TOPO_SCORE_SIGMOID,
                               n_group=c["groups"], topk_group=c["kept"], group_top=c["group_top"],
                               renorm=c["renorm"], scale=c["scale"])
        out = dict(ids=_empty(1, T, k, dtype=torch.int32), weights=_empty(1, T, k, dtype=torch.float32))
        if c["grad"]:
            out["grad_logits"] = torch.empty_like(x)
        return cfg, opts, out, _header(topo)

    cfg, opts, out, (ws, nb) = _kept(st, "own", make)
    topo.topo_route(cfg, 1, opts, x, dt, st["bias"], out["ids"], out["weights"], None, ws, nb, stream)
    if c["grad"]:
        topo.topo_route_grad(cfg, 1, opts, x, dt, out["ids"], st["grad"], out["grad_logits"], ws, nb, stream)
    return out


def _own_dispatch(topo, st, stream):
    c = st["case"]
    T, k, H = c["T"], c["k"], c["H"]

    def make():
        cfg = topo.make_cfg(T=T, E=c["E"], k=k, R=1, ranks_per_node=1, n_slot=0)
        nb = topo.topo_workspace_bytes(cfg, 1, topo.TOPO_CALL_PACK)
        return (cfg, torch.zeros(nb, dtype=torch.uint8, device=DEV), nb,
                dict(q=_empty(T * k, H, dtype=torch.float8_e4m3fn), scale=_empty(T * k, _blocks(H), dtype=torch.float32)))

    cfg, ws, nb, out = _kept(st, "own", make)
    topo.topo_permute_quantize(cfg, 1, H, st["x"], st["sorted_pairs"], out["q"], out["scale"], ws, nb, stream)
    return out


def _own_product(topo, st, stream):
    c = st["case"]
    rows, E, N, K = c["rows"], c["E"], c["N"], c["K"]

    def make():
        dt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        nb = topo.topo_expert_workspace_bytes(E, rows, N, K)
        return _empty(rows, N, dtype=dt), torch.zeros(nb, dtype=torch.uint8, device=DEV), nb

    out, ws, nb = _kept(st, "own", make)
    topo.topo_expert_gemm(E, rows, E, N, K, st["a"], st["a_scale"], st["seg_off"], None, st["w"], st["w_scale"], out,
                          topo.TOPO_DTYPE_BF16 if c["out"] == "bf16" else topo.TOPO_DTYPE_F32, ws, nb, stream)
    return out


def _own_swiglu(topo, st, stream):
    c = st["case"]
    rows, I = c["rows"], c["I"]

    def make():
        out = dict(q=_empty(rows, I, dtype=torch.float8_e4m3fn), scale=_empty(rows, _blocks(I), dtype=torch.float32))
        if c["grad"]:
            out["dh"] = torch.empty_like(st["h"])
        return out

    out = _kept(st, "own", make)
    topo.topo_swiglu_quantize(rows, I, st["h"], out["q"], out["scale"], stream)
    if c["grad"]:
        topo.topo_swiglu_grad(rows, I, st["h"], st["dy"], out["dh"], stream)
    return out


def _own_wgrad(topo, st, stream):
    c = st["case"]
    rows, E, N, K = c["rows"], c["E"], c["N"], c["K"]

    def make():
        cap = topo.topo_cols_capacity(E, rows)
        f8, f32 = torch.float8_e4m3fn, torch.float32
        nb = topo.topo_expert_workspace_bytes(E, rows, N, K)
        return (cap, _empty(N, cap, dtype=f8), _empty(cap // BLOCK, N, dtype=f32), _empty(K, cap, dtype=f8),
                _empty(cap // BLOCK, K, dtype=f32), _empty(E, N, K, dtype=f32),
                torch.zeros(nb, dtype=torch.uint8, device=DEV), nb)

    cap, dyt, dys, xt, xs, dw, ws, nb = _kept(st, "own", make)
    topo.topo_quantize_cols(E, rows, N, st["dy"], st["seg_off"], cap, dyt, dys, ws, nb, stream)
    topo.topo_quantize_cols(E, rows, K, st["x"], st["seg_off"], cap, xt, xs, ws, nb, stream)
    topo.topo_expert_wgrad(E, rows, N, K, cap, dyt, dys, xt, xs, st["seg_off"], dw, ws, nb, stream)
    return dw


def run(state):
    op = state["case"]["op"]
    if not own:
        return dict(route=_plain_route, dispatch=_plain_dispatch, product=_plain_product, swiglu=_plain_swiglu,
                    wgrad=_plain_wgrad)[op](state)
    import moe_expert_routing_ids_gb300 as topo
    f = dict(route=_own_route, dispatch=_own_dispatch, product=_own_product, swiglu=_own_swiglu, wgrad=_own_wgrad)[op]
    return f(topo, state, torch.cuda.current_stream().cuda_stream)


# -------------------------------------------------------------------------------------------------- floors
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        esz = 2 if case["dtype"] == "bf16" else 4
        b = T * (E * esz + 8 * k) + (4 * E if case["bias"] else 0)
        if case["grad"]:                                       # read the upstream gradient, write the logits' gradient
            b += T * (E * esz + 4 * k)
        return dict(bytes=b, flops=4 * T * E * (2 if case["grad"] else 1))
    if op == "dispatch":
        T, k, H = case["T"], case["k"], case["H"]
        return dict(bytes=T * H * 2 + T * k * (4 + H + 4 * _blocks(H)), flops=2 * T * H)
    if op == "swiglu":
        rows, I = case["rows"], case["I"]
        b = rows * (4 * I + I + 4 * _blocks(I)) + (rows * 6 * I if case["grad"] else 0)
        return dict(bytes=b, flops=rows * I * (20 if case["grad"] else 8))
    rows, E, N, K = case["rows"], case["E"], case["N"], case["K"]
    if op == "product":
        used = min(E, rows)                                    # experts that can hold a row
        b = rows * (K + 4 * _blocks(K)) + used * (N * K + 4 * _blocks(N) * _blocks(K))
        b += rows * N * (2 if case["out"] == "bf16" else 4) + 4 * (E + 1)
    else:
        b = rows * (N + K) * 2 + E * N * K * 4 + 4 * (E + 1)
    return dict(bytes=b, flops=2 * rows * N * K)


# ------------------------------------------------------------------------- the definitions in 64 bits
def _exact_quant(v, axis):
    """v float64; scale over 128-blocks of the last axis (axis=1) or of the first (axis=0, v already one segment)."""
    if axis == 0:
        q, s = _exact_quant(v.t().contiguous(), 1)
        return q.t(), s.t()
    power = torch.tensor([math.ldexp(1.0, i) for i in range(-400, 401)], dtype=torch.float64, device=DEV)
    out_q = torch.empty_like(v)
    out_s = []
    for b in range(0, v.shape[1], BLOCK):
        part = v[:, b:b + BLOCK]
        amax = part.abs().max(dim=1).values
        m, n = torch.frexp(amax / 448.0)                       # m * 2^n with m in [0.5, 1): 2^(n-1) only for m = 0.5
        n = torch.where(m == 0.5, n - 1, n).clamp(min=-126).long()
        s = torch.where(amax > 0, power[n + 400], torch.ones_like(amax))
        y = part / s[:, None]
        # e4m3: 3 bits after the leading one, exponents from -6 (below: multiples of 2^-9), to nearest, ties to even
        ulp = power[torch.frexp(y.abs().clamp(min=2.0 ** -6))[1].long() - 4 + 400]
        out_q[:, b:b + BLOCK] = torch.round(y / ulp) * ulp
        out_s.append(s)
    return out_q, torch.stack(out_s, 1)


def exact(case, seed):
    st, op, f64 = prepare(case, seed), case["op"], torch.float64
    if op == "route":
        if case["T"] * case["E"] > 1 << 28:                    # a 64-bit sort of this many rows takes too long
            step = 1 << 17
        else:
            step = case["T"]
        parts = [_exact_route(case, st, a, min(case["T"], a + step)) for a in range(0, case["T"], step)]
        out = dict(ids=None, weights=torch.cat([p[0] for p in parts])[None])
        if case["grad"]:
            out["grad_logits"] = torch.cat([p[1] for p in parts])[None]
        return out
    if op == "dispatch":
        T, H = case["T"], case["H"]
        q = torch.empty((T, H), dtype=torch.float32, device=DEV)
        s = torch.empty((T, _blocks(H)), dtype=torch.float32, device=DEV)
        for a in range(0, T, 8192):
            q[a:a + 8192], s[a:a + 8192] = _exact_quant(st["x"][a:a + 8192].to(f64), 1)
        t = torch.div(st["sorted_pairs"].long(), case["k"], rounding_mode="floor")
        return dict(q=q[t], scale=s[t])
    if op == "swiglu":
        I = case["I"]
        q, s, d = [], [], []
        for a in range(0, case["rows"], 16384):
            h = st["h"][a:a + 16384].to(f64)
            g, u = h[:, :I], h[:, I:]
            sg = torch.sigmoid(g)
            p = _exact_quant(g * sg * u, 1)
            q.append(p[0].float())
            s.append(p[1].float())
            if case["grad"]:
                dy = st["dy"][a:a + 16384].to(f64)
                d.append(torch.cat([dy * u * (sg + g * sg * (1 - sg)), dy * g * sg], 1).float())
        out = dict(q=torch.cat(q), scale=torch.cat(s))
        if case["grad"]:
            out["dh"] = torch.cat(d)
        return out
    if 2.0 * case["rows"] * case["N"] * case["K"] > 9e12:
        return None
    rows, N, K, at = case["rows"], case["N"], case["K"], 0
    if op == "product":
        out = torch.empty((rows, N), dtype=f64, device=DEV)
        for e, n in enumerate(st["lens"]):
            if not n:
                continue
            w = st["w"][e].to(f64)
            y = torch.zeros((n, N), dtype=f64, device=DEV)
            sa = st["a_scale"][at:at + n].to(f64)
            wb = st["w_scale"][e].to(f64).repeat_interleave(BLOCK, 0)[:N]
            a = st["a"][at:at + n].to(f64)
            for b in range(_blocks(K)):
                i = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
                y += (a[:, i] @ w[:, i].t()) * sa[:, b:b + 1] * wb[:, b]
            out[at:at + n] = y
            at += n
        return out
    out = torch.zeros((case["E"], N, K), dtype=f64, device=DEV)
    for e, n in enumerate(st["lens"]):
        for b in range(at, at + n, BLOCK):
            i = slice(b, min(at + n, b + BLOCK))
            (dy, sd), (x, sx) = _exact_quant(st["dy"][i].to(f64), 0), _exact_quant(st["x"][i].to(f64), 0)
            out[e] += (dy * sd).t() @ (x * sx)
        at += n
    return out


def _exact_route(case, st, a, b):
    f64, E, k, G = torch.float64, case["E"], case["k"], case["groups"]
    x = st["logits"][0, a:b].to(f64)
    s = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    c = x if st["bias"] is None and case["group_top"] == 1 else s if st["bias"] is None else s + st["bias"].to(f64)
    if G > 1:
        v = c.reshape(b - a, G, E // G).topk(case["group_top"], dim=-1).values.sum(-1)
        out = torch.ones((b - a, G), dtype=torch.bool, device=DEV).scatter_(1, v.topk(case["kept"], dim=1).indices, False)
        c = c.masked_fill(out[:, :, None].expand(b - a, G, E // G).reshape(b - a, E), -math.inf)
    order = torch.sort(c, dim=-1, descending=True, stable=True).indices[:, :k]
    p = torch.gather(s, 1, order)
    scale = case["scale"]
    w = p / p.sum(-1, keepdim=True) * scale if case["renorm"] else p * scale
    if not case["grad"]:
        return w, None
    g = st["grad"][0, a:b].to(f64)
    # chain rule through w(p), then p(x)
    dp = scale * (g - (g * p).sum(-1, keepdim=True) / p.sum(-1, keepdim=True)) / p.sum(-1, keepdim=True) if case["renorm"] else scale * g
    full = torch.zeros_like(s).scatter_(1, order, dp)
    dx = s * (full - (full * s).sum(-1, keepdim=True)) if case["score"] == "softmax" else full * s * (1 - s)
    return w, dx.float()
