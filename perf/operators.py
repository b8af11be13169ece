"""Operators of an attention layer around the chunked attention: what is measured.

Three operators, each in the directions that training needs:

``linear_*``     the projections, Y = act(X W + b) + R, with the gradients of X and of W, b
``rope_*``       per-head norm of queries and keys, rotary positions and the write into the caches,
                 with its backward
``adamw``        one AdamW step over many tensors, states in 32 or in 8 bits

``run`` computes them in elementary torch operations (``own = False``) or calls the framework
(``own = True``).  ``exact`` gives the same values in 64 bits, written from the definitions.
"""

import math

import torch

own = False

HEAD_SHAPES = ((32, 8, 128), (64, 8, 128), (16, 2, 64), (8, 8, 64), (32, 8, 64))   # Hq, Hkv, head_dim
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # the fused Q/K/V projection of one new token (the shortest chunk): latency and the weight's bytes
        dict(name="linear-fwd-one-token", op="linear_fwd", rows=1, k=4096, n=6144, bias=True, act="none",
             residual=False, keep_z=False),
        # an MLP's first product over a partition of about 500 rows, sizes off every tile grid
        dict(name="linear-fwd-silu-ragged", op="linear_fwd", rows=501, k=4104, n=10248, bias=True, act="silu",
             residual=False, keep_z=True),
        # the output projection of a 2048-row chunk, added to the residual stream
        dict(name="linear-fwd-residual-2048", op="linear_fwd", rows=2048, k=4096, n=4096, bias=False, act="none",
             residual=True, keep_z=False),
        # the gradient of the fused projection's input for a 2048-row chunk
        dict(name="linear-dgrad-2048", op="linear_dgrad", rows=2048, k=4096, n=6144, act="none", residual=True),
        # the fused projection's weight gradient over four 2048-row chunks' rows
        dict(name="linear-wgrad-8192", op="linear_wgrad", rows=8192, k=4096, n=6144, bias=True),
        # one new token for each of eight sequences: the smallest call
        dict(name="rope-fwd-token-b8", op="rope_fwd", batch=8, start=2000, rows=1, hq=32, hkv=8, d=128, rot=128,
             axes=1, interleaved=False, norm=True, dtype="bf16"),
        # the last chunk of a 131072-token pass with 64 query heads
        dict(name="rope-fwd-4096-of-131072", op="rope_fwd", batch=1, start=126976, rows=4096, hq=64, hkv=8, d=128,
             rot=128, axes=1, interleaved=False, norm=True, dtype="bf16"),
        # a 2048-row chunk's way back from the attention to the projection
        dict(name="rope-bwd-2048", op="rope_bwd", batch=1, start=6144, rows=2048, hq=32, hkv=8, d=128, rot=128,
             axes=1, interleaved=False, norm=True, dtype="bf16"),
        # image and video positions (time, height, width), float32, two sequences, a 500-row partition
        dict(name="rope-bwd-axes-f32", op="rope_bwd", batch=2, start=1000, rows=500, hq=16, hkv=2, d=64, rot=64,
             axes=3, interleaved=True, norm=True, dtype="fp32"),
        # one layer's projections, biases and head norms
        dict(name="adamw-layer-32", op="adamw", layers=1, d_model=4096, qkv=6144, bits=32, g_dtype="fp32"),
        dict(name="adamw-layer-8", op="adamw", layers=1, d_model=4096, qkv=6144, bits=8, g_dtype="fp32"),
        # the head norms and biases of 36 layers alone: many small tensors
        dict(name="adamw-small-tensors-8", op="adamw", layers=36, d_model=0, qkv=6144, bits=8, g_dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear_fwd", "linear_fwd", "linear_dgrad", "linear_wgrad", "rope_fwd", "rope_bwd", "adamw"))
    if op.startswith("linear"):
        k, n = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024)
        rows = min(_log(rng, 1, 16384), int(4.1e11 / (2 * k * n)))
        case = dict(op=op, rows=rows, k=k, n=n)
        if op == "linear_fwd":
            case.update(bias=rng.random() < 0.5, act=rng.choice(ACTS), residual=rng.random() < 0.5,
                        keep_z=rng.random() < 0.5)
        elif op == "linear_dgrad":
            case.update(act=rng.choice(ACTS), residual=rng.random() < 0.5)
        else:
            case.update(bias=rng.random() < 0.5)
        return case
    if op.startswith("rope"):
        hq, hkv, d = rng.choice(HEAD_SHAPES)
        batch = rng.choice((1, 1, 2, 3, 8))
        return dict(op=op, batch=batch, start=_log(rng, 1, 131072 // batch) - 1,
                    rows=_log(rng, 1, max(1, 4096 // batch)), hq=hq, hkv=hkv, d=d, rot=rng.choice((d, d, d // 2)),
                    axes=rng.choice((1, 1, 2, 3)), interleaved=rng.random() < 0.3, norm=rng.random() < 0.7,
                    dtype=rng.choice(("bf16", "bf16", "fp32")))
    return dict(op="adamw", layers=_log(rng, 1, 36), d_model=rng.choice((0, 8 * _log(rng, 4, 96))),
                qkv=8 * _log(rng, 8, 192), bits=rng.choice((32, 8)), g_dtype=rng.choice(("fp32", "bf16")))


# ------------------------------------------------------------------ inputs

LR, BETA1, BETA2, EPS, STEP, GRAD_SCALE = 3e-4, 0.9, 0.95, 1e-8, 10, 0.5
DECAY = 0.1
BLOCK = 256                       # elements of a tensor that share one scale of an 8-bit state
NORM_EPS = 1e-6
BASE = 1e6                        # rotary base


def _axis_of_pairs(pairs, axes):
    """Pairs dealt to the axes in contiguous sections, the first one the longest."""
    return [min(axes - 1, i * axes // pairs) for i in range(pairs)]


def _inv_freq(case):
    rot = case["rot"]
    return [BASE ** (-2.0 * i / rot) for i in range(rot // 2)]


def _tensor_sizes(case):
    """(elements, decayed) of every tensor of one optimizer step."""
    dm, qkv = case["d_model"], case["qkv"]
    layer = [(128, False), (128, False), (qkv, False)]
    if dm:
        layer += [(dm * qkv, True), (dm * dm, True), (dm + 5, False)]
    return layer * case["layers"]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(shape, generator=gen, device=dev, dtype=torch.float32) * std).to(dtype)

    s = dict(case=case)
    op = case["op"]
    if op.startswith("linear"):
        rows, k, n = case["rows"], case["k"], case["n"]
        if op != "linear_dgrad":
            s["x"] = normal(rows, k)
        if op != "linear_fwd":
            s["g"] = normal(rows, n, std=0.02)
        if op != "linear_wgrad":
            s["w"] = normal(k, n, std=k ** -0.5)
        if op == "linear_fwd":
            s["y"] = torch.empty(rows, n, dtype=torch.bfloat16, device=dev)
            s["bias"] = normal(n, std=0.5) if case["bias"] else None
            s["residual"] = normal(rows, n) if case["residual"] else None
            s["z"] = torch.empty_like(s["y"]) if case["keep_z"] else None
        elif op == "linear_dgrad":
            s["dx"] = torch.empty(rows, k, dtype=torch.bfloat16, device=dev)
            s["z"] = normal(rows, k) if case["act"] != "none" else None
            s["residual"] = normal(rows, k, std=0.02) if case["residual"] else None
        else:
            s["dw"] = normal(k, n, dtype=torch.float32, std=0.1)
            s["dbias"] = normal(n, dtype=torch.float32, std=0.1) if case["bias"] else None
    elif op.startswith("rope"):
        B, c, hq, hkv, d = case["batch"], case["rows"], case["hq"], case["hkv"], case["d"]
        T = case["start"] + c
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # one row of the fused projection's output: Hq query, Hkv key and Hkv value heads
        s["qkv"] = normal(B, c, hq + 2 * hkv, d, dtype=dt, std=2.0)
        s["gamma_q"] = 1 + normal(d, dtype=dt, std=0.2) if case["norm"] else None
        s["gamma_k"] = 1 + normal(d, dtype=dt, std=0.2) if case["norm"] else None
        s["inv_freq"] = torch.tensor(_inv_freq(case), dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor(_axis_of_pairs(case["rot"] // 2, case["axes"]), device=dev)
        s["positions"] = None
        if case["axes"] > 1:
            s["positions"] = torch.randint(0, T, (case["axes"], B, c), generator=gen, device=dev)
        if op == "rope_fwd":
            s["q"] = torch.empty(B, c, hq, d, dtype=dt, device=dev)
            s["k_cache"] = normal(B, T, hkv, d, dtype=dt)
            s["v_cache"] = normal(B, T, hkv, d, dtype=dt)
        else:
            s["dq"] = normal(B, c, hq, d, dtype=torch.float32, std=0.1)
            s["dk"] = normal(B, T, hkv, d, dtype=torch.float32, std=0.3)
            s["dv"] = normal(B, T, hkv, d, dtype=torch.float32, std=0.3)
            s["dqkv"] = torch.empty_like(s["qkv"])
            s["dgamma_q"] = normal(d, dtype=torch.float32) if case["norm"] else None
            s["dgamma_k"] = normal(d, dtype=torch.float32) if case["norm"] else None
        if own:
            from long_context_attention_seqattn_gb300 import binding
            s["plan"] = binding.rope_plan(_inv_freq(case), _axis_of_pairs(case["rot"] // 2, case["axes"]),
                                          case["interleaved"])
    else:
        sizes = _tensor_sizes(case)
        starts, at = [], 0
        for n, _ in sizes:
            starts.append(at)
            at += -(-n // BLOCK) * BLOCK
        # every tensor is a view of one flat array, on a boundary of 256 elements; the gaps hold zeros
        blocks = torch.arange(0, at, BLOCK, device=dev)
        first = torch.tensor(starts, device=dev)
        which = torch.searchsorted(first, blocks, right=True) - 1
        left = torch.tensor([n for n, _ in sizes], device=dev)[which] - (blocks - first[which])
        real = torch.arange(BLOCK, device=dev)[None, :] < left[:, None]

        def flat(std):
            return (normal(at // BLOCK, BLOCK, dtype=torch.float32, std=std) * real).reshape(-1)

        s["wd"] = torch.tensor([DECAY if d else 0.0 for _, d in sizes], device=dev)[which]   # of each block
        s["p"] = flat(0.02)
        s["lowp"] = s["p"].to(torch.bfloat16)
        # gradients over several orders of magnitude, as rows of a real weight have
        spread = torch.exp(normal(at // BLOCK, 1, dtype=torch.float32, std=1.5)).expand(-1, BLOCK).reshape(-1)
        s["g"] = (flat(1e-3) * spread).to(torch.float32 if case["g_dtype"] == "fp32" else torch.bfloat16)
        m, u = flat(3e-4) * spread, flat(1e-3).abs() * spread
        if case["bits"] == 8:
            s["m"], s["m_scale"] = _to_8bit(m)
            s["v"], s["v_scale"] = _to_8bit(u, keep_nonzero=True)
        else:
            s["m"], s["v"] = m, u * u
            s["m_scale"] = s["v_scale"] = None
        spans = [(a, a + n) for a, (n, _) in zip(starts, sizes)]
        views = lambda t: [t[a:b] for a, b in spans]                                    # noqa: E731
        sviews = lambda t: [t[a // BLOCK:-(-b // BLOCK)] for a, b in spans]             # noqa: E731
        if own:
            from long_context_attention_seqattn_gb300 import binding
            scales = {}
            if case["bits"] == 8:
                scales = dict(m_scale=sviews(s["m_scale"]), v_scale=sviews(s["v_scale"]))
            s["optimizer"] = binding.AdamW(views(s["p"]), views(s["g"]), lowp=views(s["lowp"]),
                                           state_bits=case["bits"], m=views(s["m"]), v=views(s["v"]),
                                           weight_decay=[DECAY if d else 0.0 for _, d in sizes], **scales)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return {"linear_fwd": _linear_fwd, "linear_dgrad": _linear_dgrad, "linear_wgrad": _linear_wgrad,
            "rope_fwd": _rope_fwd, "rope_bwd": _rope_bwd, "adamw": _adamw}[state["case"]["op"]](state)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.7071067811865476)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    if act == "gelu_tanh":
        t = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.7978845608028654 * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _linear_fwd(s):
    act = s["case"]["act"]
    if own:
        from long_context_attention_seqattn_gb300 import binding
        binding.linear_fwd(s["x"], s["w"], s["y"], bias=s["bias"], act=act, residual=s["residual"], z=s["z"])
        return {"y": s["y"], "z": s["z"]}
    z = s["x"].float() @ s["w"].float()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, act)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(torch.bfloat16), "z": z.to(torch.bfloat16) if s["z"] is not None else None}


def _linear_dgrad(s):
    act = s["case"]["act"]
    if own:
        from long_context_attention_seqattn_gb300 import binding
        binding.linear_dgrad(s["g"], s["w"], s["dx"], act=act, z=s["z"], residual=s["residual"])
        return s["dx"]
    dx = s["g"].float() @ s["w"].float().t()
    if act != "none":
        dx = dx * _act_grad(s["z"].float(), act)
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return dx.to(torch.bfloat16)


def _linear_wgrad(s):
    if own:
        from long_context_attention_seqattn_gb300 import binding
        binding.linear_wgrad(s["x"], s["g"], s["dw"], dbias=s["dbias"])
    else:
        g = s["g"].float()
        s["dw"] += s["x"].float().t() @ g
        if s["dbias"] is not None:
            s["dbias"] += g.sum(0)
    return {"dw": s["dw"], "dbias": s["dbias"]}


def _cos_sin(s):
    """cos and sin of every row's pairs, [B, c, 1, rot / 2]; angles in 64 bits (positions reach 131072)."""
    c = s["case"]
    if s["positions"] is None:
        pos = torch.arange(c["start"], c["start"] + c["rows"], device="cuda").expand(1, c["batch"], -1)
    else:
        pos = s["positions"]
    ang = pos.double()[s["axis"]].permute(1, 2, 0) * s["inv_freq"]
    return torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]


def _halves(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _joined(a, b, rest, interleaved):
    pair = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((pair, rest), -1)


def _rotated(x, cos, sin, rot, interleaved):
    a, b = _halves(x, rot, interleaved)
    return _joined(a * cos - b * sin, b * cos + a * sin, x[..., rot:], interleaved)


def _rope_fwd(s):
    c = s["case"]
    hq, hkv, start, end = c["hq"], c["hkv"], c["start"], c["start"] + c["rows"]
    q_in, k_in, v_in = s["qkv"].split((hq, hkv, hkv), 2)
    if own:
        from long_context_attention_seqattn_gb300 import binding
        binding.qk_norm_rope_fwd(q_in, k_in, v_in, s["q"], s["k_cache"], s["v_cache"], start, gamma_q=s["gamma_q"],
                                 gamma_k=s["gamma_k"], eps=NORM_EPS, plan=s["plan"], positions=s["positions"])
        return {"q": s["q"], "k": s["k_cache"], "v": s["v_cache"]}
    cos, sin = _cos_sin(s)

    def one(x, gamma):
        x = x.float()
        if gamma is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * gamma.float()
        return _rotated(x, cos, sin, c["rot"], c["interleaved"])

    s["q"].copy_(one(q_in, s["gamma_q"]))
    s["k_cache"][:, start:end].copy_(one(k_in, s["gamma_k"]))
    s["v_cache"][:, start:end].copy_(v_in)
    return {"q": s["q"], "k": s["k_cache"], "v": s["v_cache"]}


def _rope_bwd(s):
    c = s["case"]
    hq, hkv, start, end = c["hq"], c["hkv"], c["start"], c["start"] + c["rows"]
    q_in, k_in, _ = s["qkv"].split((hq, hkv, hkv), 2)
    dq_in, dk_in, dv_in = s["dqkv"].split((hq, hkv, hkv), 2)
    if own:
        from long_context_attention_seqattn_gb300 import binding
        binding.qk_norm_rope_bwd(q_in, k_in, s["dq"], s["dk"], s["dv"], dq_in, dk_in, dv_in, start,
                                 gamma_q=s["gamma_q"], gamma_k=s["gamma_k"], dgamma_q=s["dgamma_q"],
                                 dgamma_k=s["dgamma_k"], eps=NORM_EPS, plan=s["plan"], positions=s["positions"])
    else:
        cos, sin = _cos_sin(s)

        def one(x, dy, gamma, dgamma, dx):
            dn = _rotated(dy, cos, -sin, c["rot"], c["interleaved"])
            if gamma is not None:
                x = x.float()
                r = torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS)
                xhat = x * r
                dgamma += (dn * xhat).sum((0, 1, 2))
                dn = dn * gamma.float()
                dn = r * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))
            dx.copy_(dn)

        one(q_in, s["dq"], s["gamma_q"], s["dgamma_q"], dq_in)
        one(k_in, s["dk"][:, start:end], s["gamma_k"], s["dgamma_k"], dk_in)
        dv_in.copy_(s["dv"][:, start:end])
    return {"dqkv": s["dqkv"], "dgamma_q": s["dgamma_q"], "dgamma_k": s["dgamma_k"]}


def _to_8bit(x, keep_nonzero=False):
    """e4m3 codes of each 256 elements over their scale max |x| / 448 (zeros where the maximum is under 1e-30);
    with ``keep_nonzero`` a positive value is never stored as zero (2^-9 is the smallest code)."""
    b = x.reshape(-1, BLOCK)
    top = b.abs().amax(1)
    top = torch.where(top < 1e-30, torch.zeros_like(top), top)
    scale = top / 448
    inv = torch.where(top > 0, 448 / top, torch.zeros_like(top))
    codes = (b * inv[:, None]).to(torch.float8_e4m3fn)
    if keep_nonzero:
        low = (codes.float() == 0) & (b > 0) & (top[:, None] > 0)
        codes = torch.where(low, 2.0 ** -9, codes.float()).to(torch.float8_e4m3fn)
    return codes.reshape(-1), scale


def _adamw(s):
    c = s["case"]
    if own:
        s["optimizer"].step(LR, STEP, beta1=BETA1, beta2=BETA2, eps=EPS, grad_scale=GRAD_SCALE)
    else:
        shape = (-1, BLOCK)
        g = s["g"].float() * GRAD_SCALE
        if c["bits"] == 8:
            m = (s["m"].float().reshape(shape) * s["m_scale"][:, None]).reshape(-1)
            u = (s["v"].float().reshape(shape) * s["v_scale"][:, None]).reshape(-1)
            v = u * u
        else:
            m, v = s["m"], s["v"]
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + ((1 - BETA2) * g) * g
        root = torch.sqrt(v)
        step = (LR / (1 - BETA1 ** STEP)) * (m / (root / math.sqrt(1 - BETA2 ** STEP) + EPS))
        p = s["p"].reshape(shape) * (1 - LR * s["wd"])[:, None] - step.reshape(shape)
        s["p"].copy_(p.reshape(-1))
        s["lowp"].copy_(s["p"])
        if c["bits"] == 8:
            for name, x, keep in (("m", m, False), ("v", root, True)):
                codes, scale = _to_8bit(x, keep)
                s[name].copy_(codes)
                s[name + "_scale"].copy_(scale)
        else:
            s["m"].copy_(m)
            s["v"].copy_(v)
    return {"p": s["p"], "lowp": s["lowp"], "m": s["m"], "v": s["v"], "m_scale": s["m_scale"],
            "v_scale": s["v_scale"]}


# ------------------------------------------------------------------ what one pass cannot do without

def work(case):
    op = case["op"]
    if op.startswith("linear"):
        r, k, n = case["rows"], case["k"], case["n"]
        flops = 2 * r * k * n
        if op == "linear_fwd":
            byte = 2 * (r * k + k * n + r * n * (1 + case["residual"] + case["keep_z"]) + n * case["bias"])
        elif op == "linear_dgrad":
            byte = 2 * (r * n + k * n + r * k * (1 + case["residual"] + (case["act"] != "none")))
        else:
            byte = 2 * (r * k + r * n) + 8 * k * n + 8 * n * case["bias"]
        return {"bytes": byte, "flops": flops}
    if op.startswith("rope"):
        e = 2 if case["dtype"] == "bf16" else 4
        rows, d = case["batch"] * case["rows"], case["d"]
        rotated, values = rows * (case["hq"] + case["hkv"]) * d, rows * case["hkv"] * d
        pos = 8 * rows * case["axes"] if case["axes"] > 1 else 0
        if op == "rope_fwd":
            return {"bytes": 2 * e * (rotated + values) + pos, "flops": 8 * rotated}
        return {"bytes": rotated * ((e if case["norm"] else 0) + 4 + e) + values * (4 + e) + pos,
                "flops": 16 * rotated}
    n = sum(x for x, _ in _tensor_sizes(case))
    g = 4 if case["g_dtype"] == "fp32" else 2
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (8 + 2 + g + state), "flops": 16 * n}


# ------------------------------------------------------------------ the definitions in 64 bits

def _e4m3(x):
    """Nearest e4m3 value (ties to even) of |x| <= 448, in float64."""
    mant, exp = torch.frexp(x)
    exp = torch.clamp(exp, min=-5)                  # below 2^-6 the spacing stays 2^-9
    ulp = torch.ldexp(torch.ones_like(x), exp - 4)
    return torch.clamp(torch.round(x / ulp) * ulp, -448, 448)


def _exact_act(z, act):
    phi = lambda t: torch.special.ndtr(t)           # noqa: E731
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if act == "gelu":
        return z * phi(z), phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        s = torch.sigmoid(2 * a * (z + 0.044715 * z ** 3))
        return z * s, s + z * s * (1 - s) * 2 * a * (1 + 0.134145 * z ** 2)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    f = lambda t: None if t is None else t.double()       # noqa: E731
    op = case["op"]
    if op == "linear_fwd":
        z = f(s["x"]) @ f(s["w"]) + (f(s["bias"]) if s["bias"] is not None else 0)
        y = _exact_act(z, case["act"])[0] + (f(s["residual"]) if s["residual"] is not None else 0)
        return {"y": y, "z": z if s["z"] is not None else None}
    if op == "linear_dgrad":
        dx = torch.einsum("rn,kn->rk", f(s["g"]), f(s["w"]))
        if s["z"] is not None:
            dx = dx * _exact_act(f(s["z"]), case["act"])[1]
        return dx + (f(s["residual"]) if s["residual"] is not None else 0)
    if op == "linear_wgrad":
        dw = f(s["dw"]) + torch.einsum("rk,rn->kn", f(s["x"]), f(s["g"]))
        db = None if s["dbias"] is None else f(s["dbias"]) + torch.einsum("rn->n", f(s["g"]))
        return {"dw": dw, "dbias": db}
    if op.startswith("rope"):
        return _exact_rope(case, s, f)
    return _exact_adamw(case, s, f)


def _exact_rope(case, s, f):
    hq, hkv, rot, a, b = case["hq"], case["hkv"], case["rot"], case["start"], case["start"] + case["rows"]
    B, c, d = case["batch"], case["rows"], case["d"]
    if s["positions"] is None:
        pos = torch.arange(a, b, device="cuda").repeat(1, B, 1)
    else:
        pos = s["positions"]
    axis = _axis_of_pairs(rot // 2, case["axes"])
    ang = torch.stack([pos[axis[i]].double() * w for i, w in enumerate(_inv_freq(case))], -1)
    turn = torch.polar(torch.ones_like(ang), ang)[:, :, None]            # e^{i angle}, [B, c, 1, rot / 2]

    def rotate(x, turn):
        if case["interleaved"]:
            w = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * turn
            head = torch.view_as_real(w).reshape(*x.shape[:-1], rot)
        else:
            w = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            head = torch.cat((w.real, w.imag), -1)
        return torch.cat((head, x[..., rot:]), -1)

    x = f(s["qkv"])
    parts = ((x[:, :, :hq], f(s["gamma_q"])), (x[:, :, hq:hq + hkv], f(s["gamma_k"])))
    root = [torch.sqrt((h ** 2).sum(-1, keepdim=True) / d + NORM_EPS) for h, _ in parts]
    if case["op"] == "rope_fwd":
        out = [rotate(h / r * g if g is not None else h, turn) for (h, g), r in zip(parts, root)]
        k, v = f(s["k_cache"]).clone(), f(s["v_cache"]).clone()
        k[:, a:b], v[:, a:b] = out[1], x[:, :, hq + hkv:]
        return {"q": out[0], "k": k, "v": v}
    grads, dgam = [], []
    for (h, g), r, dy, old in zip(parts, root, (f(s["dq"]), f(s["dk"])[:, a:b]),
                                  (f(s["dgamma_q"]), f(s["dgamma_k"]))):
        back = rotate(dy, turn.conj())
        if g is None:
            grads.append(back)
            dgam.append(None)
            continue
        # y = g h / r with r = sqrt(mean h^2 + eps): dh = g back / r - h sum(g back h) / (d r^3)
        dot = (g * back * h).sum(-1, keepdim=True)
        grads.append(g * back / r - h * dot / (d * r ** 3))
        dgam.append(old + (back * h / r).sum((0, 1, 2)))
    return {"dqkv": torch.cat((*grads, f(s["dv"])[:, a:b]), 2), "dgamma_q": dgam[0], "dgamma_k": dgam[1]}


def _exact_adamw(case, s, f):
    rows = lambda t: f(t).reshape(-1, BLOCK)              # noqa: E731
    g, m, v = rows(s["g"]) * GRAD_SCALE, rows(s["m"]), rows(s["v"])
    if case["bits"] == 8:
        m, v = m * f(s["m_scale"])[:, None], (v * f(s["v_scale"])[:, None]) ** 2
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g ** 2 - v)
    mhat, vhat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
    p = rows(s["p"])
    p = p - LR * (mhat / (vhat.sqrt() + EPS) + f(s["wd"])[:, None] * p)
    out = {"p": p.reshape(-1), "lowp": p.reshape(-1), "m_scale": None, "v_scale": None}
    if case["bits"] == 32:
        return {**out, "m": m.reshape(-1), "v": v.reshape(-1)}
    for name, x in (("m", m), ("v", v.sqrt())):
        top = x.abs().amax(1, keepdim=True)
        code = _e4m3(x * (448 / top.clamp(min=1e-300)))
        if name == "v":
            code = torch.where((code == 0) & (x > 0), 2.0 ** -9, code)
        out[name], out[name + "_scale"] = code.reshape(-1), top.reshape(-1) / 448
    return out
