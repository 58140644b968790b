"""Cases of the expert layer in 4 bits and of the expert layer of a few tokens.

Quantisation to microscaled 4-bit values, the experts' products of such rows and weights, the gated activation between
two of them, and the whole set of experts applied to a few tokens.  The sizes are those of the framework's workloads
(hidden 1024 / 2048 / 4096 / 7168, 8 to 512 experts, k = 2 to 10) or generic.  With ``own`` false, ``run`` computes the
operators from their formulas with elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
E4M3, MX, NV = "e4m3", "mx", "nv"      # 8 bits with a scale per 128 x 128; 4 bits by 32 (power of two); 4 bits by 16 (e4m3)


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # rows of a decoding batch at an odd count: latency
        dict(name="rows_small", op="rows", rows=333, C=1408, fmt=NV),
        # the expert weights of a layer, turned to 4 bits and looked at: 64 experts of 2816 x 4096
        dict(name="weights_large", op="rows", rows=64 * 2816, C=4096, fmt=MX),
        # dispatch of a prefill chunk straight into 4 bits
        dict(name="dispatch_prefill", op="dispatch", T=16384, E=256, k=8, H=7168, fmt=NV),
        # the activation between the two products: a decoding batch, a prefill chunk
        dict(name="swiglu_decode", op="swiglu", rows=1000, I=1408, fmt=MX),
        dict(name="swiglu_prefill", op="swiglu", rows=131072, I=2048, fmt=NV),
        # one token's pairs through the down projection: latency
        dict(name="product_one_token", op="product", rows=6, E=64, N=4096, K=1408, skew=0.0, out="f32", fmt=MX),
        # a decoding batch: every expert gets a few rows, the weights are the traffic
        dict(name="product_decode", op="product", rows=1536, E=64, N=2816, K=4096, skew=0.6, out="bf16", fmt=NV),
        # prefill of 16384 tokens, k = 8, experts unevenly loaded
        dict(name="product_prefill", op="product", rows=131072, E=128, N=4096, K=7168, skew=0.8, out="bf16", fmt=NV),
        # one token through a large layer's experts, weights in 8 bits: the weights of 8 experts are the traffic
        dict(name="few_one_token", op="few", T=1, E=256, k=8, H=7168, I=2048, fmt=E4M3),
        # one token through a small layer: latency
        dict(name="few_one_token_small", op="few", T=1, E=128, k=8, H=2048, I=768, fmt=MX),
        # a small decoding batch, weights in 4 bits
        dict(name="few_batch", op="few", T=8, E=64, k=6, H=4096, I=1408, fmt=NV),
        # the most tokens the call takes: nearly every expert is used
        dict(name="few_most", op="few", T=32, E=256, k=8, H=7168, I=2048, fmt=MX),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, hi, units=(32, 128, 512)):
    """An odd multiple of 32, 128 or 512, up to hi: whole and partial scale blocks and tiles."""
    unit = rng.choice([u for u in units if u <= hi])
    return unit * (2 * _log(rng, 1, (hi // unit + 1) // 2) - 1)


def draw(rng):
    op = rng.choice(["rows", "dispatch", "swiglu", "product", "product", "product", "few", "few", "few"])
    fmt = rng.choice([MX, NV])
    if op == "rows":
        return dict(op="rows", rows=_log(rng, 1, 131072), C=_size(rng, 7168), fmt=fmt)
    if op == "dispatch":
        return dict(op="dispatch", T=_log(rng, 1, 16384), E=_log(rng, 8, 256), k=rng.randint(1, 8), H=_size(rng, 7168), fmt=fmt)
    if op == "swiglu":
        return dict(op="swiglu", rows=_log(rng, 1, 131072), I=_size(rng, 2048), fmt=fmt)
    if op == "product":
        return dict(op="product", rows=_log(rng, 1, 65536), E=_log(rng, 1, 128), N=_size(rng, 4096), K=_size(rng, 7168),
                    skew=rng.choice([0.0, 0.6, 1.2]), out=rng.choice(["bf16", "bf16", "f32"]), fmt=fmt)
    E = _log(rng, 8, 256)
    return dict(op="few", T=_log(rng, 1, 32), E=E, k=rng.randint(1, 8), H=_size(rng, 7168), I=_size(rng, 2048),
                fmt=rng.choice([E4M3, MX, NV]))


# ------------------------------------------------------------------------------------------------ inputs
def _cdiv(a, b):
    return (a + b - 1) // b


def _block(fmt):
    return 32 if fmt == MX else 16


def _pitch(C, fmt):
    """Bytes of a row's scales: one a block, filled up to a multiple of 16."""
    return _cdiv(C // _block(fmt), 16) * 16


def _counts(seed, rows, E, skew):
    """Rows of each expert: a multinomial draw over Zipf(skew) shares in a seeded order."""
    r = np.random.default_rng([seed, rows, E])
    p = np.arange(1, E + 1, dtype=np.float64) ** -skew
    return r.multinomial(rows, r.permutation(p / p.sum()))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _power(n):
    """2^n in float32 for whole numbers n from -126 to 127."""
    return ((n.to(torch.int32) + 127) << 23).view(torch.float32)


def _weights(gen, n, N, K, fmt):
    """Weights [n, N, K] as a program holds them, made a matrix at a time: packed values, scales, row scales."""
    if fmt == E4M3:
        q = torch.empty((n, N, K), dtype=torch.float8_e4m3fn, device=DEV)
        for e in range(n):
            q[e] = (_randn(gen, N, K) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s = torch.rand((n, _cdiv(N, 128), _cdiv(K, 128)), generator=gen, device=DEV)
        return q, (s + 0.5) * (0.01 / K ** 0.5), None
    q = torch.empty((n, N, K // 2), dtype=torch.uint8, device=DEV)
    nb = K // _block(fmt)
    s = torch.full((n, N, _pitch(K, fmt)), 127 if fmt == MX else 0x38, dtype=torch.uint8, device=DEV)
    base = -int(round(math.log2(4 * K ** 0.5)))
    for e in range(n):
        # magnitudes 0 .. 6 about as often as in normal values whose block reaches 4 to 6
        c = (_randn(gen, N, K) * 3).abs_().clamp_(max=7).to(torch.uint8)
        c |= torch.randint(0, 2, (N, K), generator=gen, device=DEV, dtype=torch.uint8) << 3
        q[e] = c[:, 0::2] | (c[:, 1::2] << 4)
        if fmt == MX:
            s[e, :, :nb] = torch.randint(126 + base, 129 + base, (N, nb), generator=gen, device=DEV).to(torch.uint8)
        else:
            s[e, :, :nb] = (torch.rand((N, nb), generator=gen, device=DEV) * 300 + 100).to(torch.float8_e4m3fn).view(torch.uint8)
    r = None if fmt == MX else _power(torch.randint(base - 9, base - 6, (n, N), generator=gen, device=DEV))
    return q, s, r


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, st = case["op"], dict(case=case)
    if op == "rows":
        rows, C = case["rows"], case["C"]
        st["x"] = (_randn(gen, rows, C) * torch.exp(_randn(gen, rows, 1))).to(torch.bfloat16)
    elif op == "dispatch":
        T, E, k, H = case["T"], case["E"], case["k"], case["H"]
        st["x"] = (_randn(gen, T, H) * torch.exp(_randn(gen, T, 1))).to(torch.bfloat16)
        ids = torch.rand((T, E), generator=gen, device=DEV).topk(k, dim=1).indices.reshape(-1)
        st["sorted_pairs"] = torch.sort(ids, stable=True).indices.to(torch.int32)
    elif op == "swiglu":
        st["h"] = (_randn(gen, case["rows"], 2 * case["I"]) * 2).to(torch.bfloat16)
    elif op == "product":
        counts = _counts(seed, case["rows"], case["E"], case["skew"])
        st["lens"] = [int(c) for c in counts]
        st["seg_off"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), device=DEV)
        st["x"] = (_randn(gen, case["rows"], case["K"]) * torch.exp(_randn(gen, case["rows"], 1))).to(torch.bfloat16)
        st["w"], st["w_scale"], st["w_row"] = _weights(gen, case["E"], case["N"], case["K"], case["fmt"])
    else:
        T, E, k, H, I, fmt = (case[n] for n in ("T", "E", "k", "H", "I", "fmt"))
        st["x"] = (_randn(gen, T, H) * torch.exp(0.5 * _randn(gen, T, 1))).to(torch.bfloat16)
        ids = torch.rand((T, E), generator=gen, device=DEV).topk(k, dim=1).indices
        st["ids"], st["host_ids"] = ids.to(torch.int32), sorted(set(ids.reshape(-1).tolist()))
        w = torch.rand((T, k), generator=gen, device=DEV) + 0.05
        st["weights"] = w / w.sum(-1, keepdim=True)
        st["up"], st["up_scale"], st["up_row"] = _weights(gen, E, 2 * I, H, fmt)
        st["down"], st["down_scale"], st["down_row"] = _weights(gen, E, H, I, fmt)
    return st


# -------------------------------------------------------------------------------------------- plain forms
def _values():
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=DEV)


def _least_power(amax, top):
    """The smallest power of two s with amax <= top * s (exponent at least -126; 1 for amax = 0)."""
    f, p = math.frexp(top)                                     # top = f * 2^p, f in [0.5, 1)
    m, e = torch.frexp(amax)
    n = torch.where(m > f, e - p + 1, e - p).clamp(min=-126)
    return torch.where(amax > 0, _power(n), torch.ones_like(amax))


def _round4(y):
    """Magnitudes y <= 6 to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even mantissa."""
    return torch.where(y < 2, torch.round(y * 2) * 0.5, torch.where(y < 4, torch.round(y), torch.round(y * 0.5) * 2))


def _quant4(x, fmt):
    """x float32 [R, C] (finite) as the values that its 4-bit form stands for, float32."""
    p = x.reshape(x.shape[0], -1, _block(fmt))
    amax = p.abs().amax(-1, keepdim=True)
    if fmt == MX:
        s = _least_power(amax, 6.0)
    else:
        g = _least_power(amax.amax(1, keepdim=True), 6.0 * 448.0)
        t = amax / (6.0 * g)
        ulp = _power(torch.frexp(t)[1].clamp(min=-5) - 4)      # the smallest e4m3 value that is at least t
        s = torch.ceil(t / ulp) * ulp
        s = torch.where(amax > 0, s, torch.ones_like(s)) * g
    return (torch.copysign(_round4((p / s).abs()), p) * s).reshape(x.shape)


def _unpack(q, scale, row, fmt, values):
    """Packed rows [R, K / 2] with their scales as float32 [R, K]."""
    R, K = q.shape[0], 2 * q.shape[1]
    v = values[torch.stack([q & 15, q >> 4], -1).reshape(R, K).int()]
    nb = K // _block(fmt)
    s = scale[:, :nb]
    s = _power(s.to(torch.int32) - 127) if fmt == MX else s.contiguous().view(torch.float8_e4m3fn).float() * row[:, None]
    return (v.reshape(R, nb, -1) * s[..., None]).reshape(R, K)


def _matrix(q, scale, row, fmt, values):
    """One expert's weights [N, K] as float32."""
    if fmt != E4M3:
        return _unpack(q, scale, row, fmt, values)
    N, K = q.shape
    return q.float() * scale.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def _swiglu(h, I):
    g, u = h[..., :I], h[..., I:]
    return g / (1.0 + torch.exp(-g)) * u


def _plain_product(st):
    c, values = st["case"], _values()
    out = torch.empty((c["rows"], c["N"]), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
    a, at = _quant4(st["x"].float(), c["fmt"]), 0
    for e, n in enumerate(st["lens"]):                         # one product for each expert's rows
        if n:
            w = _unpack(st["w"][e], st["w_scale"][e], None if st["w_row"] is None else st["w_row"][e], c["fmt"], values)
            out[at:at + n] = (a[at:at + n] @ w.t()).to(out.dtype)
            at += n
    return out


def _plain_few(st):
    c, values = st["case"], _values()
    x = st["x"].float()
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float32, device=DEV)
    for e in st["host_ids"]:                                   # one set of products for each expert in use
        up = _matrix(st["up"][e], st["up_scale"][e], None if st["up_row"] is None else st["up_row"][e], c["fmt"], values)
        down = _matrix(st["down"][e], st["down_scale"][e], None if st["down_row"] is None else st["down_row"][e], c["fmt"], values)
        y = _swiglu(x @ up.t(), c["I"]) @ down.t()
        out += y * torch.where(st["ids"] == e, st["weights"], torch.zeros_like(st["weights"])).sum(1, keepdim=True)
    return out.to(torch.bfloat16)


def _plain(st):
    c, op = st["case"], st["case"]["op"]
    if op == "rows":
        return _quant4(st["x"].float(), c["fmt"]).to(torch.bfloat16)
    if op == "dispatch":
        return _quant4(st["x"].float(), c["fmt"]).to(torch.bfloat16)[torch.div(st["sorted_pairs"].long(), c["k"], rounding_mode="floor")]
    if op == "swiglu":
        return _quant4(_swiglu(st["h"].float(), c["I"]), c["fmt"]).to(torch.bfloat16)
    return _plain_product(st) if op == "product" else _plain_few(st)


# ------------------------------------------------------------------------------- the framework's operators
def _kept(st, make):
    """What a program that makes this call each step keeps between the steps: output buffers, workspace."""
    if "own" not in st:
        st["own"] = make()
    return st["own"]


def _empty(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _fmt(topo, fmt):
    return dict(e4m3=topo.TOPO_FMT_EIGHT, mx=topo.TOPO_FMT_MX, nv=topo.TOPO_FMT_NV)[fmt]


def _rows4(topo, rows, C, fmt):
    """Buffers of rows in 4 bits: values, scales, row scales."""
    return (_empty(rows, C // 2), _empty(rows, topo.topo_micro_pitch(C, _fmt(topo, fmt))),
            _empty(rows, dtype=torch.float32) if fmt == NV else None)


def _own_rows(topo, st, stream):
    c, f = st["case"], _fmt(topo, st["case"]["fmt"])
    op = c["op"]
    C = c["C"] if op == "rows" else c["H"] if op == "dispatch" else c["I"]
    rows = c["T"] * c["k"] if op == "dispatch" else c["rows"]

    def make():
        more = None
        if op == "dispatch":
            cfg = topo.make_cfg(T=c["T"], E=c["E"], k=c["k"], R=1, ranks_per_node=1, n_slot=0)
            nb = topo.topo_workspace_bytes(cfg, 1, topo.TOPO_CALL_PACK)
            more = cfg, torch.zeros(nb, dtype=torch.uint8, device=DEV), nb
        return *_rows4(topo, rows, C, c["fmt"]), _empty(rows, C, dtype=torch.bfloat16), more

    q, s, r, out, more = _kept(st, make)
    if op == "rows":
        topo.topo_quantize_rows_micro(rows, C, f, st["x"], q, s, r, stream)
    elif op == "dispatch":
        cfg, ws, nb = more
        topo.topo_permute_quantize_micro(cfg, 1, C, f, st["x"], st["sorted_pairs"], q, s, r, ws, nb, stream)
    else:
        topo.topo_swiglu_quantize_micro(rows, C, f, st["h"], q, s, r, stream)
    topo.topo_dequantize_micro(rows, C, f, q, s, r, out, stream)
    return out


def _own_product(topo, st, stream):
    c, f = st["case"], _fmt(topo, st["case"]["fmt"])
    rows, E, N, K = c["rows"], c["E"], c["N"], c["K"]
    bf16 = c["out"] == "bf16"

    def make():
        nb = topo.topo_expert_workspace_bytes(E, rows, N, K)
        return (*_rows4(topo, rows, K, c["fmt"]), _empty(rows, N, dtype=torch.bfloat16 if bf16 else torch.float32),
                torch.zeros(nb, dtype=torch.uint8, device=DEV), nb)

    q, s, r, out, ws, nb = _kept(st, make)
    topo.topo_quantize_rows_micro(rows, K, f, st["x"], q, s, r, stream)
    topo.topo_expert_gemm_micro(E, rows, E, N, K, f, q, s, r, st["seg_off"], None, st["w"], st["w_scale"], st["w_row"], out,
                                topo.TOPO_DTYPE_BF16 if bf16 else topo.TOPO_DTYPE_F32, ws, nb, stream)
    return out


def _own_few(topo, st, stream):
    c = st["case"]
    T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]

    def make():
        nb = topo.topo_few_workspace_bytes(T, E, k, H, I)
        return _empty(T, H, dtype=torch.bfloat16), torch.zeros(nb, dtype=torch.uint8, device=DEV), nb

    out, ws, nb = _kept(st, make)
    topo.topo_expert_few(T, E, k, H, I, _fmt(topo, c["fmt"]), st["x"], st["ids"], st["weights"], st["up"], st["up_scale"],
                         st["up_row"], st["down"], st["down_scale"], st["down_row"], out, ws, nb, stream)
    return out


def run(state):
    if not own:
        return _plain(state)
    import moe_expert_routing_ids_gb300 as topo
    f = dict(product=_own_product, few=_own_few).get(state["case"]["op"], _own_rows)
    return f(topo, state, torch.cuda.current_stream().cuda_stream)


# -------------------------------------------------------------------------------------------------- floors
def _weight_bytes(n, N, K, fmt):
    if fmt == E4M3:
        return n * (N * K + 4 * _cdiv(N, 128) * _cdiv(K, 128))
    return n * N * (K // 2 + K // _block(fmt) + (4 if fmt == NV else 0))


def work(case):
    op = case["op"]
    if op == "rows":
        return dict(bytes=case["rows"] * case["C"] * 4, flops=2 * case["rows"] * case["C"])
    if op == "dispatch":
        T, k, H = case["T"], case["k"], case["H"]
        return dict(bytes=T * H * 2 + T * k * (4 + 2 * H), flops=2 * T * H)
    if op == "swiglu":
        return dict(bytes=case["rows"] * case["I"] * 6, flops=10 * case["rows"] * case["I"])
    if op == "product":
        rows, E, N, K = case["rows"], case["E"], case["N"], case["K"]
        b = rows * K * 2 + _weight_bytes(min(E, rows), N, K, case["fmt"]) + rows * N * (2 if case["out"] == "bf16" else 4)
        return dict(bytes=b + 4 * (E + 1), flops=2 * rows * N * K)
    T, E, k, H, I = case["T"], case["E"], case["k"], case["H"], case["I"]
    used = E * (1.0 - (1.0 - k / E) ** T)                      # experts that T tokens name, on average
    b = used * (_weight_bytes(1, 2 * I, H, case["fmt"]) + _weight_bytes(1, H, I, case["fmt"])) + T * (4 * H + 8 * k)
    return dict(bytes=b, flops=6 * T * k * H * I)


# ------------------------------------------------------------------------- the definitions in 64 bits
def _nearest(y):
    """The e2m1 value nearest each float64 in y, by the midpoints between neighbours; a midpoint goes to the even code."""
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    mid = (mag[1:] + mag[:-1]) / 2
    a = y.abs().contiguous()
    up, down = torch.bucketize(a, mid, right=True), torch.bucketize(a, mid)   # a midpoint counted, not counted
    return torch.where(y < 0, -1.0, 1.0) * mag[torch.where(up == down, up, up & ~1)]


def _exact_quant(v, fmt):
    """v float64 [R, C] -> the float64 values of its 4-bit form."""
    R, C = v.shape
    blk = 32 if fmt == MX else 16
    b = v.view(R, C // blk, blk)
    top = b.abs().max(-1).values
    if fmt == MX:
        s = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 6.0) - 1e-12).clamp(min=-126.0))
    else:
        row = top.max(-1, keepdim=True).values
        g = torch.exp2(torch.ceil(torch.log2(row.clamp(min=1e-300) / 2688.0) - 1e-12).clamp(min=-126.0))
        g = torch.where(row > 0, g, torch.ones_like(g))
        codes = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).to(torch.float64)
        at = torch.bucketize((top / (6.0 * g)).contiguous(), codes)            # the first e4m3 value that is no smaller
        s = codes[at.clamp(max=126)] * g
    s = torch.where(top > 0, s, torch.ones_like(s))[..., None]
    return (_nearest(b / s) * s).view(R, C)


def _exact_weights(q, scale, row, fmt):
    f64 = torch.float64
    if fmt == E4M3:
        N, K = q.shape
        w = q.to(f64)
        for b in range(scale.shape[1]):
            w[:, 128 * b:128 * b + 128] *= scale[:, b].to(f64).repeat_interleave(128)[:N, None]
        return w
    N, K = q.shape[0], 2 * q.shape[1]
    w = torch.empty((N, K), dtype=f64, device=DEV)
    for half in (0, 1):
        c = (q >> (4 * half)).to(torch.int64)
        e, m = (c >> 1) & 3, (c & 1).to(f64)
        mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).to(f64)))
        w[:, half::2] = torch.where((c & 8) != 0, -mag, mag)
    blk = 32 if fmt == MX else 16
    s = scale[:, :K // blk]
    s = torch.exp2(s.to(f64) - 127) if fmt == MX else s.contiguous().view(torch.float8_e4m3fn).to(f64) * row.to(f64)[:, None]
    return w * s.repeat_interleave(blk, 1)


def _pick(st, name, e):
    r = st[name + "_row"]
    return st[name][e], st[name + "_scale"][e], None if r is None else r[e], st["case"]["fmt"]


def exact(case, seed):
    op, f64 = case["op"], torch.float64
    if op == "product" and 2.0 * case["rows"] * case["N"] * case["K"] > 4e12:
        return None
    st = prepare(case, seed)
    if op in ("rows", "swiglu", "dispatch"):
        src, parts = st["h"] if op == "swiglu" else st["x"], []
        for a in range(0, src.shape[0], 8192):
            v = src[a:a + 8192].to(f64)
            if op == "swiglu":
                g, u = v.chunk(2, 1)
                v = g * torch.sigmoid(g) * u
            parts.append(_exact_quant(v, case["fmt"]).float())
        out = torch.cat(parts)
        return out[torch.div(st["sorted_pairs"].long(), case["k"], rounding_mode="floor")] if op == "dispatch" else out
    if op == "product":
        out, at = torch.empty((case["rows"], case["N"]), dtype=f64, device=DEV), 0
        for e, n in enumerate(st["lens"]):
            if n:
                out[at:at + n] = _exact_quant(st["x"][at:at + n].to(f64), case["fmt"]) @ _exact_weights(*_pick(st, "w", e)).t()
                at += n
        return out
    out, I = torch.zeros((case["T"], case["H"]), dtype=f64, device=DEV), case["I"]
    for e in st["host_ids"]:
        t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        h = st["x"][t].to(f64) @ _exact_weights(*_pick(st, "up", e)).t()
        y = (h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]) @ _exact_weights(*_pick(st, "down", e)).t()
        out.index_add_(0, t, y * st["weights"][t, j].to(f64)[:, None])
    return out
