"""The operators together, as a trainer uses them: a whole attention layer
(projection, head norm, rotary positions, chunked attention, output
projection) with its backward and optimizer step, against float64 autograd of
the layer written out.

Bars: rel-L2 <= 2e-2 per tensor, the bar of the bf16 attention path.  A tensor
passes at most eight bf16 roundings on its way (x, w, q or k, p, o, d_o, ds,
d_qkv), each 2^-8 at most and 2^-9 / sqrt(3) in the root mean square, so
sqrt(8) 1.1e-3 = 3.2e-3, times a condition number that the norm and softmax
keep to a few."""

import math

import numpy as np
import pytest
import torch

from long_context_attention_seqattn_gb300 import binding
from long_context_attention_seqattn_gb300.block import AttentionBlock

pytestmark = pytest.mark.gpu

REL = 2e-2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_attention_seqattn_gb300 import build
    build.build()
    binding.load_library()
    yield
    binding.sync_status()


def _rel(name, got, ref):
    rel = float((got.double().cpu() - ref).norm() / ref.norm())
    assert rel <= REL, f"{name}: rel-L2 {rel:.3e}"


def _make(B, T, dm, Hq, Hkv, d, chunk, axes=1, qk_norm=True, bias=False, state_bits=32, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).bfloat16()      # noqa: E731
    inv = [1e4 ** (-2.0 * i / d) for i in range(d // 2)]
    axis = [i * axes // (d // 2) for i in range(d // 2)]
    pos = torch.randint(0, 5000, (axes, B, T), generator=g) if axes > 1 else None
    block = AttentionBlock(B, T, dm, Hq, Hkv, d, chunk, plan=binding.rope_plan(inv, axis),
                           positions=None if pos is None else pos.cuda(), qk_norm=qk_norm, bias=bias,
                           state_bits=state_bits, weight_decay=0.1)
    w = {"w_qkv": r(dm, (Hq + 2 * Hkv) * d, std=dm ** -0.5), "w_o": r(Hq * d, dm, std=(Hq * d) ** -0.5)}
    if bias:
        w["b_qkv"] = r((Hq + 2 * Hkv) * d, std=0.3)
    if qk_norm:
        w["gamma_q"], w["gamma_k"] = (1 + r(d, std=0.1).float()).bfloat16(), (1 + r(d, std=0.1).float()).bfloat16()
    block.load(**{n: t.cuda() for n, t in w.items()})
    x, dy = r(B, T, dm), r(B, T, dm)
    p64 = pos if pos is not None else torch.arange(T).expand(1, B, T)
    ang = torch.stack([p64[a].double() * f for a, f in zip(axis, inv)], -1)[:, :, None]
    return block, w, x, dy, ang


def _layer64(w, x, ang, Hq, Hkv, d, eps=1e-6):
    B, T, _ = x.shape
    qkv = x @ w["w_qkv"] + w.get("b_qkv", 0)
    q, k, v = qkv.view(B, T, Hq + 2 * Hkv, d).split((Hq, Hkv, Hkv), 2)

    def norm_rope(h, gamma):
        if gamma is not None:
            h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * gamma
        a, b = h[..., :d // 2], h[..., d // 2:]
        c, s = torch.cos(ang), torch.sin(ang)
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    q, k = norm_rope(q, w.get("gamma_q")), norm_rope(k, w.get("gamma_k"))
    k, v = k.repeat_interleave(Hq // Hkv, 2), v.repeat_interleave(Hq // Hkv, 2)
    sc = torch.einsum("bqhd,bkhd->bhqk", q, k) / math.sqrt(d)
    sc = sc.masked_fill(torch.ones(T, T).triu(1).bool(), -math.inf)
    o = torch.einsum("bhqk,bkhd->bqhd", sc.softmax(-1), v)
    return x + o.reshape(B, T, Hq * d) @ w["w_o"]


CASES = [
    dict(B=1, T=300, dm=256, Hq=4, Hkv=2, d=64, chunk=128),
    dict(B=2, T=200, dm=200, Hq=4, Hkv=1, d=128, chunk=70, axes=3, bias=True),
    dict(B=1, T=129, dm=136, Hq=2, Hkv=2, d=128, chunk=128, qk_norm=False),     # last chunk: a single row
    dict(B=1, T=96, dm=64, Hq=8, Hkv=2, d=64, chunk=1, bias=True),              # token by token
]


@pytest.mark.parametrize("case", CASES)
def test_layer_forward_and_gradients(case):
    block, w, x, dy, ang = _make(**case)
    y = block.forward(x.cuda())
    dx = block.backward(dy.cuda())
    binding.sync_status()
    w64 = {n: t.double().requires_grad_(True) for n, t in w.items()}
    x64 = x.double().requires_grad_(True)
    ref = _layer64(w64, x64, ang, case["Hq"], case["Hkv"], case["d"])
    (ref * dy.double()).sum().backward()
    _rel("y", y, ref.detach())
    _rel("dx", dx, x64.grad)
    for n in w:
        _rel("d" + n, block.grads[n], w64[n].grad)


def test_layer_gradient_is_the_definitions_slope():
    """dx and the weights' gradients against central differences of the
    float64 layer along a random direction."""
    case = CASES[0]
    block, w, x, dy, ang = _make(**case, seed=3)
    block.forward(x.cuda())
    dx = block.backward(dy.cuda())
    args = (ang, case["Hq"], case["Hkv"], case["d"])
    g = torch.Generator().manual_seed(9)
    for name in ("x", "w_qkv", "w_o", "gamma_q"):
        base = x if name == "x" else w[name]
        got = dx if name == "x" else block.grads[name]
        # a direction with a share of the gradient itself, so that the slope is not a sum that cancels
        e = torch.randn(base.shape, generator=g, dtype=torch.float64) * got.double().cpu().square().mean().sqrt()
        e = e + got.double().cpu()
        h = 1e-4 / float(e.square().mean().sqrt())

        def loss(sign):
            ws = {n: t.double() for n, t in w.items()}
            xs = x.double()
            if name == "x":
                xs = xs + sign * h * e
            else:
                ws[name] = ws[name] + sign * h * e
            return float((_layer64(ws, xs, *args) * dy.double()).sum())

        slope = (loss(1) - loss(-1)) / (2 * h)
        mine = float((got.double().cpu() * e).sum())
        assert abs(slope - mine) <= REL * float(got.double().norm().cpu() * e.norm()), (name, slope, mine)


@pytest.mark.parametrize("state_bits", [32, 8])
def test_optimizer_step_on_the_layers_gradients(state_bits):
    block, w, x, dy, ang = _make(**CASES[1], state_bits=state_bits, seed=4)
    block.forward(x.cuda())
    block.backward(dy.cuda())
    before = {n: t.double().cpu() for n, t in block.masters.items()}
    block.step(1e-3, 1, grad_scale=0.5)
    torch.cuda.synchronize()
    for n, old in before.items():
        g = block.grads[n].double().cpu() * 0.5
        decay = 0.1 if n.startswith("w_") else 0.0
        # first step: m / (1 - b1) = g and v / (1 - b2) = g^2
        want = old * (1 - 1e-3 * decay) - 1e-3 * g / (g.abs() + 1e-8)
        off = (block.masters[n].double().cpu() - want).abs()
        assert float((off - 2.0 ** -22 * (old.abs() + 1e-3)).max()) <= 0, n
        assert torch.equal(block.weights[n], block.masters[n].to(torch.bfloat16))


def test_chunk_size_and_reruns_agree():
    """The same layer in one chunk, in odd chunks, and run again: the chunk
    bounds move only float32 sums; a rerun adds the same gradients again."""
    outs = []
    for chunk in (300, 77):
        block, w, x, dy, ang = _make(**dict(CASES[0], chunk=chunk), seed=5)
        y = block.forward(x.cuda())
        dx = block.backward(dy.cuda())
        torch.cuda.synchronize()
        first = {n: t.clone() for n, t in block.grads.items()}
        block.forward(x.cuda())
        block.backward(dy.cuda())
        torch.cuda.synchronize()
        for n, t in block.grads.items():
            _rel("twice d" + n, t, 2 * first[n].double().cpu())
        outs.append((y, dx, first))
    (y0, dx0, g0), (y1, dx1, g1) = outs
    _rel("y", y1, y0.double().cpu())
    _rel("dx", dx1, dx0.double().cpu())
    for n in g0:
        _rel("d" + n, g1[n], g0[n].double().cpu())


def test_training_step_replays_from_a_graph():
    """Forward, backward and AdamW captured once and replayed with new inputs
    in the same buffers, the step number and rate read from the device."""
    eager, w, x, dy, ang = _make(**CASES[0], seed=6)
    other, _, _, _, _ = _make(**CASES[0], seed=6)
    lr = torch.tensor([1e-3], device="cuda")
    step = torch.tensor([1], dtype=torch.int64, device="cuda")
    xs, dys = x.cuda(), dy.cuda()

    def train(block, n, rate):
        block.zero_grad()
        y = block.forward(xs)
        dx = block.backward(dys)
        block.step(rate, n)
        return y, dx

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):              # kernels loaded outside the capture
        other.forward(xs)
        other.backward(dys)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y_g, dx_g = train(other, step, lr)
    for n in (1, 2, 3):
        step.fill_(n)
        lr.fill_(float(np.float32(1e-3 / n)))
        xs.copy_(_noise(100 + n, xs.shape))
        dys.copy_(_noise(200 + n, dys.shape))
        y, dx = train(eager, n, float(np.float32(1e-3 / n)))
        graph.replay()
        torch.cuda.synchronize()
        _rel("y", y_g, y.double().cpu())
        _rel("dx", dx_g, dx.double().cpu())
    for n in w:
        _rel(n, other.masters[n], eager.masters[n].double().cpu())


def _noise(seed, shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def test_block_refuses():
    block, w, x, dy, ang = _make(**CASES[0])
    with pytest.raises(ValueError, match="shape"):
        block.forward(x.cuda()[:, :10])
    with pytest.raises(ValueError, match="positions"):
        AttentionBlock(1, 64, 64, 1, 1, 64, 32, positions=torch.zeros((1, 1, 63), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="dy has shape"):
        block.backward(torch.zeros((x.shape[0], x.shape[1] + 8, x.shape[2]), dtype=torch.bfloat16, device="cuda"))
