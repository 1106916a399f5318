"""Measured cases of the fp8 expert path's operators.

Four operators that sit around a MoE layer whose experts are held in 8-bit
floating point (e4m3) with one fp32 scale per block of 128:

  norm   residual addition + root-mean-square norm, with an e4m3 output that
         carries one scale per token and 128 channels
  gate   scores from router logits, balance bias, expert groups, top-k,
         renormalised weights
  gemm   grouped matrix product of block-scaled e4m3 operands
  ffn    the experts' FFN on routed tokens: gathered rows, first product,
         SwiGLU, block-scaled e4m3 again, second product

``run`` computes each in its plain form (elementary torch operations in fp32,
rounded once at the end), or, where ``own`` is set, through the package's
public binding.  ``exact`` restates them in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128                      # channels per scale
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100         # a block of zeros takes the scale of this amax
CLOSED = -1e30                   # a logit at or below this closes the expert for the token
F32_MAX = 3.4028234663852886e38

# The largest listed case: the repository's full-layer configuration.
FULL = dict(T=16384, H=7168, E=128, K=8, N=4096)


def listed():
    return [
        # router of one decoded token: pure latency; sigmoid scores with a
        # balance bias, 256 experts in 8 groups of which 4 stay
        dict(name="gate 1 token", op="gate", T=1, E=256, K=8, score="sigmoid", bias=True, G=8,
             KG=4, group="top2", renorm=True, scale=2.5, dtype="f32", mask=False, closed=0.0),
        # a prefill batch's router: softmax over bf16 logits (exact ties are common)
        dict(name="gate prefill", op="gate", T=32768, E=256, K=8, score="softmax", bias=False,
             G=1, KG=1, group="max", renorm=True, scale=1.0, dtype="bf16", mask=False, closed=0.0),
        # many experts, odd sizes, some experts closed to some tokens, padding tokens masked
        dict(name="gate odd", op="gate", T=4097, E=1000, K=16, score="sigmoid", bias=True, G=20,
             KG=7, group="max", renorm=True, scale=1.0, dtype="f32", mask=True, closed=0.05),
        # one decoded token between attention and the experts
        dict(name="norm 1 token", op="norm", T=1, H=7168, residual=True, y=True, q=True, w="bf16"),
        # a prefill batch, all four outputs: bounded by HBM
        dict(name="norm prefill", op="norm", T=16384, H=7168, residual=True, y=True, q=True,
             w="bf16"),
        # a width that ends inside a block, codes only, fp32 weight
        dict(name="norm odd", op="norm", T=1023, H=1000, residual=False, y=False, q=True, w="f32"),
        # one dense projection for a handful of tokens: reading the weights bounds it
        dict(name="gemm 16 rows", op="gemm", rows=16, E=1, N=4096, Kd=7168, skew=0.0, out="bf16"),
        # the same kind of projection for a prefill batch: the tensor cores bound it
        dict(name="gemm 8192 rows", op="gemm", rows=8192, E=1, N=7168, Kd=2048, skew=0.0,
             out="bf16"),
        # ragged groups, edges that end inside a tile and inside a block, fp32 output
        dict(name="gemm ragged", op="gemm", rows=1533, E=7, N=1000, Kd=1456, skew=1.0, out="f32"),
        # one decoded token through its 8 of 128 experts
        dict(name="ffn 1 token", op="ffn", T=1, H=7168, E=128, K=8, N=4096, skew=0.0, mask=False),
        # the repository's small-batch layer: 8 rows per expert on average, every expert read once
        dict(name="ffn 128 tokens", op="ffn", T=128, H=7168, E=128, K=8, N=4096, skew=0.3,
             mask=True),
        # the repository's full-layer configuration: the tensor cores bound it
        dict(name="ffn prefill", op="ffn", skew=0.1, mask=False, **FULL),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step`, its factor spread evenly over the logarithm of [lo, hi]."""
    v = step * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["gate", "norm", "gemm", "ffn"])
    if op == "gate":
        G = rng.choice([1, 1, 4, 8, 10])
        per = _log(rng, 4, 1000 // G)
        E = G * per
        KG = rng.randint(1, G)
        K = rng.randint(1, min(16, KG * per))
        return dict(op=op, T=_log(rng, 1, 32768), E=E, K=K, score=rng.choice(["sigmoid", "softmax"]),
                    bias=rng.random() < 0.5, G=G, KG=KG, group=rng.choice(["max", "top2"]),
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["f32", "bf16"]), mask=rng.random() < 0.3,
                    closed=rng.choice([0.0, 0.05]))
    if op == "norm":
        res, y, q = rng.choice([(True, True, True), (True, False, True), (False, True, True),
                                (True, True, False), (False, False, True)])
        return dict(op=op, T=_log(rng, 1, 16384), H=_log(rng, 8, 1024, 8), residual=res, y=y, q=q,
                    w=rng.choice(["bf16", "f32"]))
    if op == "gemm":
        E = _log(rng, 1, 64)
        return dict(op=op, rows=_log(rng, 1, 16384), E=E, N=_log(rng, 16, 900, 8),
                    Kd=_log(rng, 8, 448, 16), skew=rng.choice([0.0, 0.5, 1.0]),
                    out=rng.choice(["bf16", "f32"]))
    E = _log(rng, 8, 128)
    return dict(op=op, T=_log(rng, 1, 8192), H=_log(rng, 16, 448, 16), E=E,
                K=rng.randint(1, 8), N=_log(rng, 1, 16, 256), skew=rng.choice([0.0, 0.3]),
                mask=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _codes(g, *shape):
    """e4m3 codes as a block-scaled tensor holds them: a normal distribution
    whose largest values reach the format's end."""
    return (_randn(g, *shape) * 110.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _scales(g, typical, *shape):
    """Block scales spread over about a factor of four around `typical`."""
    return typical * torch.exp(0.35 * _randn(g, *shape))


def _weights(g, E, N, Kd):
    w = torch.empty((E, N, Kd), dtype=torch.float8_e4m3fn, device=DEV)
    for e in range(E):
        w[e] = _codes(g, N, Kd)
    return w, _scales(g, 0.02 / 110.0, E, _blocks(N), _blocks(Kd))


def _gate_keys64(c, logits, bias):
    """Selection keys and scores in 64 bits (closed experts: key -inf)."""
    l = logits.double()
    valid = l > CLOSED
    l = l.clamp(max=F32_MAX)
    if c["score"] == "sigmoid":
        s = torch.special.expit(l)
    else:
        s = torch.softmax(l.masked_fill(~valid, -math.inf), dim=1).nan_to_num(0.0)
    s = s.masked_fill(~valid, 0.0)
    key = (s if bias is None else s + bias.double()).masked_fill(~valid, -math.inf)
    if c["G"] > 1:
        per = key.view(key.shape[0], c["G"], -1)
        top = per.topk(min(2, per.shape[2]) if c["group"] == "top2" else 1, dim=2).values
        gs = top.masked_fill(top == -math.inf, 0.0).sum(2)
        gs = gs.masked_fill(per.amax(2) == -math.inf, -math.inf)
        order = torch.sort(gs, dim=1, descending=True, stable=True)
        keep = torch.zeros_like(gs, dtype=torch.bool)
        keep.scatter_(1, order.indices[:, :c["KG"]], True)
        key = key.masked_fill(~keep.repeat_interleave(per.shape[2], 1), -math.inf)
        return key, s, valid, order.values
    return key, s, valid, None


def _close(v):
    """Rows of descending values with two neighbours so near that rounding in
    32 bits alone could order them (equal values are ties, and stay)."""
    a, b = v[:, :-1], v[:, 1:]
    d = a - b
    return ((d > 0) & (d < 3e-6 * a.abs())).any(1)


def _prepare_gate(c, seed):
    g = _gen(seed)
    T, E = c["T"], c["E"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    popular = 0.4 * _randn(g, E)
    bias = 0.1 * _randn(g, E) if c["bias"] else None

    def fresh(n):
        l = (1.3 * _randn(g, n, E) + popular).to(dt)
        if c["closed"]:
            u = torch.rand(n, E, generator=g, device=DEV)
            l[u < c["closed"]] = -math.inf
            l[u > 1 - c["closed"] / 2] = torch.finfo(dt).min
        return l

    logits = fresh(T)
    # A token whose choice hangs on the rounding of its scores has no choice
    # that every correct 32-bit evaluation agrees on: draw it again.
    for _ in range(40):
        key, _, _, groups = _gate_keys64(c, logits, bias)
        bad = _close(key.topk(min(c["K"] + 1, E), dim=1).values)
        if groups is not None:
            bad |= _close(groups[:, :c["KG"] + 1])
        n = int(bad.sum())
        if n == 0:
            break
        logits[bad] = fresh(n)
    if c["closed"] and T >= 64:
        logits[5::97] = -math.inf            # tokens that every expert is closed to
    mask = None
    if c["mask"]:
        mask = (torch.rand(T, generator=g, device=DEV) < 0.9).to(torch.uint8)
        logits[mask == 0] = math.nan         # padding rows hold anything
    out = dict(expert_ids=torch.empty(T, c["K"], dtype=torch.int32, device=DEV),
               expert_scales=torch.empty(T, c["K"], device=DEV),
               route_mask=torch.empty(T, c["K"], dtype=torch.uint8, device=DEV))
    return dict(logits=logits, bias=bias, mask=mask, out=out)


def _prepare_norm(c, seed):
    g = _gen(seed)
    T, H = c["T"], c["H"]
    # a few channels far larger than the rest, as hidden states have them
    spread = torch.where(torch.rand(H, generator=g, device=DEV) < 0.01, 20.0, 1.0)
    x = (_randn(g, T, H) * spread).bfloat16()
    residual = (3.0 * _randn(g, T, H) * spread).bfloat16() if c["residual"] else None
    w = 1.0 + 0.2 * _randn(g, H)
    if c["w"] == "bf16":
        w = w.bfloat16()
    out = {}
    if c["y"]:
        out["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    if c["residual"]:
        out["residual_out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    if c["q"]:
        out["q"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=DEV)
        out["scales"] = torch.empty(T, _blocks(H), device=DEV)
    return dict(x=x, residual=residual, weight=w, out=out)


def _prepare_gemm(c, seed):
    g = _gen(seed)
    rows, E, N, Kd = c["rows"], c["E"], c["N"], c["Kd"]
    p = torch.exp(c["skew"] * _randn(g, E)).cpu()
    p = p / p.sum()
    if E > 3 and c["skew"]:
        p[2] = 0.0                           # an expert without rows
    pick = torch.multinomial(p, rows, replacement=True,
                             generator=torch.Generator().manual_seed(int(seed)))
    counts = torch.bincount(pick, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    w, ws = _weights(g, E, N, Kd)
    return dict(a=_codes(g, rows, Kd), a_scales=_scales(g, 1.0 / 110.0, rows, _blocks(Kd)), w=w,
                w_scales=ws, offsets=offsets.to(DEV), most=int(counts.max()),
                out=torch.empty(rows, N, device=DEV,
                                dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32))


def _prepare_ffn(c, seed):
    g = _gen(seed)
    T, H, E, K, N = c["T"], c["H"], c["E"], c["K"], c["N"]
    # K distinct experts a token (Gumbel top-k over the experts' popularity)
    u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-12, 1 - 1e-7)
    ids = (c["skew"] * _randn(g, E) - torch.log(-torch.log(u))).topk(K, dim=1).indices
    on = torch.ones(T, dtype=torch.bool, device=DEV)
    if c["mask"] and T > 1:
        on = torch.rand(T, generator=g, device=DEV) < 0.9
        on[0] = True
    # the dispatch bookkeeping a program has at this point: rows by expert,
    # then token, then slot; (partition, token, slot) of each row
    code = torch.where(on[:, None], ids, E).reshape(-1)
    order = torch.sort(code, stable=True).indices
    counts = torch.bincount(code, minlength=E + 1)[:E]
    R = int(counts.sum())
    order = order[:R]
    assist = torch.zeros(T * K, 3, dtype=torch.int32, device=DEV)
    assist[:R, 1] = (order // K).int()
    assist[:R, 2] = (order % K).int()
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    w1, s1 = _weights(g, E, N, H)
    w2, s2 = _weights(g, E, H, N // 2)
    return dict(x=_codes(g, T, H), x_scales=_scales(g, 1.0 / 110.0, T, _blocks(H)), assist=assist,
                offsets=offsets, R=R, most=int(counts.max()), w1=w1, w1_scales=s1, w2=w2,
                w2_scales=s2, y=torch.zeros(T * K, H, dtype=torch.bfloat16, device=DEV))


def prepare(case, seed):
    s = {"gate": _prepare_gate, "norm": _prepare_norm, "gemm": _prepare_gemm,
         "ffn": _prepare_ffn}[case["op"]](case, seed)
    s["case"] = dict(case)
    return s


# ------------------------------------------------------------------ plain forms

def _expand(s, n, dim):
    """Block scales -> one per element along `dim` (the last block may be short)."""
    return s.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def _rows32(q, s):
    return q.float() * _expand(s, q.shape[1], 1)


def _weights32(w, s):
    return w.float() * _expand(_expand(s, w.shape[1], 1), w.shape[2], 2)


def _quantise(v):
    """fp32 rows -> e4m3 codes and one fp32 scale per row and 128 channels."""
    n, H = v.shape
    nb = _blocks(H)
    p = torch.zeros(n, nb * BLOCK, device=v.device)
    p[:, :H] = v
    p = p.view(n, nb, BLOCK)
    amax = p.abs().amax(2).clamp(min=AMAX_FLOOR)
    q = (p * (E4M3_MAX / amax)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(n, nb * BLOCK)[:, :H].contiguous(), amax / E4M3_MAX


def _plain_gate(s):
    c = s["case"]
    l = s["logits"].float()
    T, E = l.shape
    K = c["K"]
    valid = l > CLOSED
    if s["mask"] is not None:
        valid = valid & (s["mask"] != 0)[:, None]
    l = torch.where(valid, l.clamp(max=F32_MAX), -math.inf)
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = l.amax(1, keepdim=True).clamp(min=-F32_MAX)
        e = torch.exp(l - m)
        score = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    key = score if s["bias"] is None else score + s["bias"]
    key = torch.where(valid, key, -math.inf)
    if c["G"] > 1:
        per = key.view(T, c["G"], E // c["G"])
        if c["group"] == "top2":
            top = torch.sort(per, dim=2, descending=True).values[:, :, :2]
        else:
            top = per.amax(2, keepdim=True)
        gs = torch.where(top == -math.inf, 0.0, top).sum(2)
        gs = torch.where(top[:, :, 0] == -math.inf, -math.inf, gs)
        best = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["KG"]]
        keep = torch.zeros(T, c["G"], dtype=torch.bool, device=l.device).scatter_(1, best, True)
        key = torch.where(keep.repeat_interleave(E // c["G"], 1), key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True)    # ties: lowest index
    open_ = order.values[:, :K] > -math.inf
    ids = torch.where(open_, order.indices[:, :K], -1)
    w = torch.where(open_, score.gather(1, order.indices[:, :K]), 0.0)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return dict(expert_ids=ids.int(), expert_scales=w * c["scale"],
                route_mask=open_.to(torch.uint8))


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    out = {}
    if c["residual"]:
        h = h + s["residual"].float()
        out["residual_out"] = h.bfloat16()
    v = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    if c["y"]:
        out["y"] = v.bfloat16()
    if c["q"]:
        out["q"], out["scales"] = _quantise(v)
    return out


def _grouped32(rows, offsets, most, w):
    """Row r of expert e times w[e]^T: every expert's rows padded to the fullest expert's."""
    E = offsets.numel() - 1
    r = torch.arange(rows.shape[0], device=rows.device)
    e = torch.searchsorted(offsets, r.int(), right=True) - 1
    at = r - offsets[e]
    padded = torch.zeros(E, most, rows.shape[1], device=rows.device)
    padded[e, at] = rows
    return torch.bmm(padded, w.transpose(1, 2))[e, at]


def _plain_gemm(s):
    y = _grouped32(_rows32(s["a"], s["a_scales"]), s["offsets"], s["most"],
                   _weights32(s["w"], s["w_scales"]))
    return y.to(s["out"].dtype)


def _plain_ffn(s):
    R, Nh = s["R"], s["case"]["N"] // 2
    x = _rows32(s["x"], s["x_scales"])[s["assist"][:R, 1].long()]
    h = _grouped32(x, s["offsets"], s["most"], _weights32(s["w1"], s["w1_scales"]))
    gate = h[:, :Nh]
    q, qs = _quantise(gate / (1.0 + torch.exp(-gate)) * h[:, Nh:])
    y = torch.zeros_like(s["y"])                  # rows past the routed ones are not written
    y[:R] = _grouped32(_rows32(q, qs), s["offsets"], s["most"],
                       _weights32(s["w2"], s["w2_scales"])).bfloat16()
    return y


# ------------------------------------------------------------------ the package's operators

def _own_gate(s):
    from combine_route_count_prefix_gb300 import binding as B
    c = s["case"]
    return B.gate(s["logits"], c["K"], bias=s["bias"], mask=s["mask"], score=c["score"],
                  groups=c["G"], topk_groups=c["KG"], group_score=c["group"],
                  renormalize=c["renorm"], scale=c["scale"], out=s["out"])


def _own_norm(s):
    from combine_route_count_prefix_gb300 import binding as B
    return B.add_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=1e-6, out=s["out"])


def _own_gemm(s):
    from combine_route_count_prefix_gb300 import binding as B
    out, s["ws"] = B.grouped_gemm_fp8(s["offsets"], s["a"], s["a_scales"], s["w"], s["w_scales"],
                                      ws=s.get("ws"), out=s["out"])
    return out


def _own_ffn(s):
    from combine_route_count_prefix_gb300 import binding as B
    c = s["case"]
    if "shape" not in s:
        s["shape"] = B.make_shape(c["T"], 1, c["H"], c["E"], c["K"], c["N"])
    y, s["ws"] = B.grouped_ffn_fp8(s["shape"], s["x"], s["x_scales"], s["offsets"], s["w1"],
                                   s["w1_scales"], s["w2"], s["w2_scales"], assist=s["assist"],
                                   ws=s.get("ws"), y=s["y"])
    return y


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gate": _own_gate, "norm": _own_norm, "gemm": _own_gemm, "ffn": _own_ffn}[op](state)
    return {"gate": _plain_gate, "norm": _plain_norm, "gemm": _plain_gemm,
            "ffn": _plain_ffn}[op](state)


# ------------------------------------------------------------------ floors

def work(case):
    c = case
    if c["op"] == "gate":
        n = c["T"] * c["E"]
        b = n * (4 if c["dtype"] == "f32" else 2) + (4 * c["E"] if c["bias"] else 0)
        b += (c["T"] if c["mask"] else 0) + c["T"] * c["K"] * 9
        return {"bytes": b, "flops": 5 * n}
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        b = n * (2 + (4 if c["residual"] else 0) + (2 if c["y"] else 0) + (1 if c["q"] else 0))
        b += c["H"] * (2 if c["w"] == "bf16" else 4) + (4 * c["T"] * _blocks(c["H"]) if c["q"] else 0)
        return {"bytes": b, "flops": 6 * n}
    if c["op"] == "gemm":
        R, E, N, Kd = c["rows"], c["E"], c["N"], c["Kd"]
        hit = E * (1 - (1 - 1 / E) ** R)          # experts with rows, on average
        b = R * (Kd + 4 * _blocks(Kd)) + hit * (N * Kd + 4 * _blocks(N) * _blocks(Kd))
        return {"bytes": b + R * N * (2 if c["out"] == "bf16" else 4), "flops": 2 * R * N * Kd}
    T, H, E, K, N = c["T"], c["H"], c["E"], c["K"], c["N"]
    if c["mask"]:
        T = max(1, 0.9 * T)
    hit = E * (1 - (1 - K / E) ** T)
    R = T * K
    return {"bytes": T * (H + 4 * _blocks(H)) + hit * (N * H + H * N // 2) + R * (2 * H + 12),
            "flops": R * (2 * N * H + N * H)}


# ------------------------------------------------------------------ 64 bits

def _quantise64(v):
    """The values that e4m3 codes with block scales stand for, without the
    rounding of the scale itself: codes (rounded to e4m3) and scales."""
    q, s = torch.empty_like(v), v.new_empty(v.shape[0], _blocks(v.shape[1]))
    for b in range(s.shape[1]):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        s[:, b] = part.abs().amax(1).clamp(min=AMAX_FLOOR) / E4M3_MAX
        u = part / s[:, b:b + 1]
        step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, b * BLOCK:(b + 1) * BLOCK] = torch.round(u / step) * step
    return q, s


def _product64(rows, row_scales, w, w_scales):
    """[n, Kd] x [N, Kd]^T with block scales, block by block of the inner dimension."""
    N, Kd = w.shape
    acc = torch.zeros(rows.shape[0], N, dtype=torch.float64, device=rows.device)
    cs = w_scales.double().repeat_interleave(BLOCK, 0)[:N]
    for b in range(_blocks(Kd)):
        k = slice(b * BLOCK, min(Kd, (b + 1) * BLOCK))
        acc += (rows[:, k].double() @ w[:, k].double().T) * row_scales[:, b:b + 1].double() * cs[:, b]
    return acc


def exact(case, seed):
    c = case
    if c["op"] in ("gemm", "ffn") and work(c)["flops"] > 3e12:
        return None                               # over about 20 seconds in 64 bits
    s = prepare(c, seed)
    if c["op"] == "gate":
        logits = s["logits"].double().nan_to_num(nan=-math.inf, neginf=-math.inf)
        key, score, valid, _ = _gate_keys64(c, logits, s["bias"])
        top, ids = torch.sort(key, dim=1, descending=True, stable=True)
        top, ids = top[:, :c["K"]], ids[:, :c["K"]]
        open_ = torch.isfinite(top)
        w = score.gather(1, ids) * open_
        if c["renorm"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        return dict(expert_ids=ids.masked_fill(~open_, -1).int(), expert_scales=w * c["scale"],
                    route_mask=open_.to(torch.uint8))
    if c["op"] == "norm":
        h = s["x"].double()
        out = {}
        if c["residual"]:
            h = h + s["residual"].double()
            out["residual_out"] = h
        v = h / (h.square().sum(1, keepdim=True) / c["H"] + 1e-6).sqrt() * s["weight"].double()
        if c["y"]:
            out["y"] = v
        if c["q"]:
            out["q"], out["scales"] = _quantise64(v)
        return out
    off = s["offsets"].tolist()
    if c["op"] == "gemm":
        return torch.cat([_product64(s["a"][a:b], s["a_scales"][a:b], s["w"][e], s["w_scales"][e])
                          for e, (a, b) in enumerate(zip(off, off[1:]))])
    y, Nh = torch.zeros_like(s["y"], dtype=torch.float64), c["N"] // 2
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if a == b:
            continue
        tok = s["assist"][a:b, 1].long()
        h = _product64(s["x"].view(torch.uint8)[tok].view(torch.float8_e4m3fn), s["x_scales"][tok],
                       s["w1"][e], s["w1_scales"][e])
        q, qs = _quantise64(h[:, :Nh] * torch.special.expit(h[:, :Nh]) * h[:, Nh:])
        y[a:b] = _product64(q, qs, s["w2"][e], s["w2_scales"][e])
    return y
