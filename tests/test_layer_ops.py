"""The layer's operators on the GPU against plain 64-bit implementations.

Tolerances count roundings (u = half a step: bf16 2^-8, e4m3 2^-4, fp32 2^-24,
relative to the value):

linear    one bf16 rounding of the result, plus the float32 sums: the tensor
          core's additions of 16 products each may truncate, so k / 16 + 16
          additions (two more for bias and residual) of at most 2^-23 of the
          sum of magnitudes S; the activations' fast exponential adds
          2^-20 (1 + |z|) (its argument's rounding grows with |z|).
weights   float32: products are summed for at most 768 rows on the tensor
          core (48 additions of 2^-23) and those sums are added in float32
          (one 2^-24 each, fewer than rows / 512 + 2 of them).
rope      one rounding to the element type; in float32 about 24 roundings of
          a value no larger than the head's largest rotated pair.
adamw     float32 states: at most 8 roundings of a term each.  8-bit states:
          half an e4m3 step of the value, half the smallest step (2^-10) of the
          scale for subnormal codes (2^-9 for u, never rounded to zero).
"""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from long_context_attention_seqattn_gb300 import binding

pytestmark = pytest.mark.gpu

U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_attention_seqattn_gb300 import build
    build.build()
    binding.load_library()
    yield
    binding.sync_status()


def _rand(seed, *shape, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def _within(name, got, ref, tol):
    """|got - ref| <= tol element by element (a NaN fails)."""
    off = (got.double().cpu() - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((off / tol.clamp(min=1e-300)).nan_to_num(nan=math.inf).max()):.3g} of the bound")


# ============================================================== linear

def _act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _act_grad64(z, act):
    z = z.clone().requires_grad_(True)
    _act64(z, act).sum().backward()
    return z.grad


def _sum_tol(k, mags):
    return (k / 16 + 16) * 2.0 ** -23 * mags


LINEAR_SIZES = [
    (1, 64, 64), (1, 8, 8), (3, 4096, 40), (17, 72, 264), (128, 128, 128), (129, 136, 1000), (500, 2048, 512),
    (257, 520, 776), (2, 16, 2056), (1030, 328, 648),
]


@pytest.mark.parametrize("rows,k,n", LINEAR_SIZES)
@pytest.mark.parametrize("act,bias,residual,keep_z", [
    ("none", False, False, False), ("none", True, True, False), ("silu", True, False, True),
    ("gelu", False, True, True), ("relu", True, True, True), ("gelu_tanh", True, False, False),
])
def test_linear_fwd(rows, k, n, act, bias, residual, keep_z):
    x, w = _rand(1, rows, k), _rand(2, k, n, std=k ** -0.5)
    b = _rand(3, n) if bias else None
    r = _rand(4, rows, n) if residual else None
    y = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    z = torch.full_like(y, float("nan")) if keep_z else None
    binding.linear_fwd(x.cuda(), w.cuda(), y, bias=None if b is None else b.cuda(), act=act,
                       residual=None if r is None else r.cuda(), z=z)
    z64 = x.double() @ w.double()
    mags = x.double().abs() @ w.double().abs()
    if bias:
        z64, mags = z64 + b.double(), mags + b.double().abs()
    y64 = _act64(z64, act)
    tol = _sum_tol(k, mags)
    if act != "none":
        tol = 1.13 * tol + 2.0 ** -20 * (1 + z64.abs())
    if residual:
        y64 = y64 + r.double()
        tol = tol + U_F32 * (y64.abs() + r.double().abs())
    _within("y", y, y64, U_BF16 * y64.abs() + tol + 1e-38)
    if keep_z:
        _within("z", z, z64, U_BF16 * z64.abs() + _sum_tol(k, mags) + 1e-38)


@pytest.mark.parametrize("rows,k,n", LINEAR_SIZES)
@pytest.mark.parametrize("act,residual", [("none", False), ("silu", True), ("gelu", False), ("relu", False),
                                          ("gelu_tanh", True)])
def test_linear_dgrad(rows, k, n, act, residual):
    g, w = _rand(5, rows, n), _rand(6, k, n, std=n ** -0.5)
    z = _rand(7, rows, k, std=2.0) if act != "none" else None
    r = _rand(8, rows, k) if residual else None
    dx = torch.full((rows, k), float("nan"), dtype=torch.bfloat16, device="cuda")
    binding.linear_dgrad(g.cuda(), w.cuda(), dx, act=act, z=None if z is None else z.cuda(),
                         residual=None if r is None else r.cuda())
    ref = g.double() @ w.double().t()
    tol = _sum_tol(n, g.double().abs() @ w.double().abs().t())
    if z is not None:
        d = _act_grad64(z.double(), act)
        tol = 1.13 * tol + 2.0 ** -20 * (1 + z.double().abs()) * ref.abs()
        ref = ref * d
    if residual:
        ref = ref + r.double()
        tol = tol + U_F32 * (ref.abs() + r.double().abs())
    _within("dx", dx, ref, U_BF16 * ref.abs() + tol + 1e-38)


@pytest.mark.parametrize("rows,k,n", LINEAR_SIZES + [(5000, 136, 264)])
@pytest.mark.parametrize("bias", [False, True])
def test_linear_wgrad(rows, k, n, bias):
    x, g = _rand(9, rows, k), _rand(10, rows, n)
    dw = _rand(11, k, n, dtype=torch.float32)
    db = _rand(12, n, dtype=torch.float32)
    dw_d, db_d = dw.cuda(), db.cuda()
    binding.linear_wgrad(x.cuda(), g.cuda(), dw_d, dbias=db_d if bias else None)
    ref = dw.double() + x.double().t() @ g.double()
    mags = dw.double().abs() + x.double().abs().t() @ g.double().abs()
    _within("dw", dw_d, ref, (32 + 16) * 2.0 ** -23 * mags + (rows / 512 + 2) * U_F32 * mags)
    dref = db.double() + (g.double().sum(0) if bias else 0)
    # rows / 128 serial additions, a tree of 7, the old value
    dmags = db.double().abs() + g.double().abs().sum(0)
    _within("dbias", db_d, dref, (rows / 128 + 10) * U_F32 * dmags if bias else torch.zeros_like(dref) + 1e-300)


def test_linear_wgrad_keeps_float32_over_long_contractions():
    """Over thousands of rows of one sign a running sum on the tensor core
    alone would drift by a truncation per addition; the bound here is the one
    of the module's head, 2^-18 at 16384 rows, and the drift would pass it."""
    rows, k, n = 16384, 128, 256
    x, g = _rand(13, rows, k).abs(), _rand(14, rows, n).abs()
    dw = torch.zeros((k, n), device="cuda")
    binding.linear_wgrad(x.cuda(), g.cuda(), dw)
    ref = x.double().t() @ g.double()
    _within("dw", dw, ref, ((32 + 16) * 2.0 ** -23 + (rows / 512 + 2) * U_F32) * ref)


@pytest.mark.parametrize("cols", [1800, 1856])
def test_linear_with_several_waves_of_tiles(cols):
    """Some 88 tiles of 256 x 256 over a long contraction: more than run at
    once, with a rest that is computed in other shapes.  References in float64
    on the GPU; same bits on a second run."""
    rows, k = 2570, 4104
    x, w = _rand(210, rows, k).cuda(), _rand(211, k, cols, std=k ** -0.5).cuda()
    r, b = _rand(212, rows, cols).cuda(), _rand(213, cols).cuda()
    for act, res in (("silu", r), ("none", None)):
        outs = []
        for _ in range(2):
            y, z = torch.full_like(r, float("nan")), torch.full_like(r, float("nan"))
            binding.linear_fwd(x, w, y, bias=b, act=act, residual=res, z=z)
            outs.append((y, z))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        z64 = x.double() @ w.double() + b.double()
        tol = _sum_tol(k, x.double().abs() @ w.double().abs() + b.double().abs())
        y64 = _act64(z64, act) + (res.double() if res is not None else 0)
        ytol = 1.13 * tol + 2.0 ** -20 * (1 + z64.abs()) if act != "none" else tol
        if res is not None:
            ytol = ytol + U_F32 * (y64.abs() + res.double().abs())
        _within("z", outs[0][1], z64.cpu(), (U_BF16 * z64.abs() + tol).cpu())
        _within("y", outs[0][0], y64.cpu(), (U_BF16 * y64.abs() + ytol).cpu())
    # dx [2570, cols] = g [2570, 4104] wt^T
    g, wt = x, w.t().contiguous()
    dx = r.clone()
    binding.linear_dgrad(g, wt, dx, residual=dx)
    ref = g.double() @ wt.double().t() + r.double()
    tol = _sum_tol(k, g.double().abs() @ wt.double().abs().t()) + U_F32 * (ref.abs() + r.double().abs())
    _within("dx", dx, ref.cpu(), (U_BF16 * ref.abs() + tol).cpu())
    # dw [2568, cols] += a^T g over 4104 rows
    a, gg = _rand(214, k, 2568).cuda(), _rand(215, k, cols).cuda()
    dws = [torch.zeros((2568, cols), device="cuda") for _ in range(2)]
    for dw in dws:
        binding.linear_wgrad(a, gg, dw)
    assert torch.equal(*dws)
    mags = a.double().abs().t() @ gg.double().abs()
    _within("dw", dws[0], (a.double().t() @ gg.double()).cpu(),
            (((32 + 16) * 2.0 ** -23 + (k / 512 + 2) * U_F32) * mags).cpu())


def test_linear_strided_operands_and_neighbours():
    """Rows of wider matrices: what lies between and behind the rows is NaN
    and must neither be read into the result nor written."""
    rows, k, n, pad = 150, 200, 264, 24
    nan = float("nan")

    def wide(t, extra_rows=3):
        buf = torch.full((t.shape[0] + extra_rows, t.shape[1] + pad), nan, dtype=t.dtype)
        buf[:t.shape[0], :t.shape[1]] = t
        buf = buf.cuda()
        return buf, buf[:t.shape[0], :t.shape[1]]

    x, w, g = _rand(20, rows, k), _rand(21, k, n, std=k ** -0.5), _rand(22, rows, n)
    r, z = _rand(23, rows, n), torch.zeros(rows, n, dtype=torch.bfloat16)
    (_, xs), (_, gs), (rb, rs), (zb, zs) = wide(x), wide(g), wide(r), wide(z)
    yb, ys = wide(torch.zeros_like(z))
    binding.linear_fwd(xs, w.cuda(), ys, act="relu", residual=rs, z=zs)
    z64 = x.double() @ w.double()
    tol = _sum_tol(k, x.double().abs() @ w.double().abs())
    y64 = z64.clamp(min=0) + r.double()
    _within("z", zs, z64, U_BF16 * z64.abs() + tol)
    _within("y", ys, y64, U_BF16 * y64.abs() + tol + U_F32 * (y64.abs() + r.double().abs()))
    dxb, dxs = wide(torch.zeros_like(x))
    binding.linear_dgrad(gs, w.cuda(), dxs)
    ref = g.double() @ w.double().t()
    _within("dx", dxs, ref, U_BF16 * ref.abs() + _sum_tol(n, g.double().abs() @ w.double().abs().t()))
    dw, db = torch.zeros((k, n), device="cuda"), torch.zeros(n, device="cuda")
    binding.linear_wgrad(xs, gs, dw, dbias=db)
    mags = x.double().abs().t() @ g.double().abs()
    _within("dw", dw, x.double().t() @ g.double(), 50 * 2.0 ** -23 * mags)
    _within("dbias", db, g.double().sum(0), 20 * U_F32 * g.double().abs().sum(0))
    for buf, cols in ((yb, n), (zb, n), (dxb, k), (rb, n)):
        assert torch.isnan(buf[:rows, cols:]).all() and torch.isnan(buf[rows:]).all()


def test_linear_three_dimensional_rows_and_refused_strides():
    B, c, k, n = 2, 5, 64, 72
    x, w = _rand(24, B, c, k).cuda(), _rand(25, k, n).cuda()
    y = torch.empty((B, c, n), dtype=torch.bfloat16, device="cuda")
    binding.linear_fwd(x, w, y)
    flat = torch.empty((B * c, n), dtype=torch.bfloat16, device="cuda")
    binding.linear_fwd(x.reshape(B * c, k), w, flat)
    assert torch.equal(y.reshape(B * c, n), flat)
    cut = _rand(26, B, c + 2, k).cuda()[:, :c]             # rows at two different strides
    with pytest.raises(ValueError, match="uniform stride"):
        binding.linear_fwd(cut, w, y)
    with pytest.raises(ValueError, match="contiguous"):
        binding.linear_fwd(x.reshape(B * c, k).t().contiguous().t(), w, flat)
    with pytest.raises(ValueError, match="contiguous"):
        binding.linear_fwd(x, w.t().contiguous().t(), y)
    with pytest.raises(ValueError, match="rows"):
        binding.linear_fwd(x, w, flat[:3])
    with pytest.raises(ValueError, match="columns"):
        binding.linear_fwd(x[..., :32], w, y)
    with pytest.raises(binding.SeqattnError, match="stride"):
        binding.linear_fwd(torch.zeros((4, 68), dtype=torch.bfloat16, device="cuda")[:, :64], w, y[0, :4])
    with pytest.raises(binding.SeqattnError, match="aligned"):
        binding.linear_fwd(torch.zeros(64 * 9, dtype=torch.bfloat16, device="cuda")[4:4 + 64 * 5].view(5, 64), w, y[0])
    with pytest.raises(ValueError, match="z is needed"):
        binding.linear_dgrad(y, w, x, act="relu")
    empty = torch.empty((0, k), dtype=torch.bfloat16, device="cuda")
    binding.linear_fwd(empty, w, torch.empty((0, n), dtype=torch.bfloat16, device="cuda"))


def test_linear_sums_into_its_residual():
    rows, k, n = 300, 256, 384
    g, w = _rand(27, rows, n).cuda(), _rand(28, k, n, std=n ** -0.5).cuda()
    r = _rand(29, rows, k).cuda()
    apart = torch.empty_like(r)
    binding.linear_dgrad(g, w, apart, residual=r)
    binding.linear_dgrad(g, w, r, residual=r)
    assert torch.equal(apart, r)


def test_linear_special_values():
    """A NaN or an infinity of x reaches its own row only; activations take
    their limits for large arguments."""
    rows, k, n = 140, 64, 136
    x, w = _rand(30, rows, k), _rand(31, k, n)
    x[3, 5], x[131, 0] = float("nan"), float("inf")
    y = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    binding.linear_fwd(x.cuda(), w.cuda(), y, act="relu")
    fin = torch.isfinite(y).all(1).cpu()
    assert not fin[3] and not fin[131] and int((~fin).sum()) == 2
    assert torch.isnan(y[3]).all()
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        big = torch.tensor([[1e4, -1e4, 1e19, -1e19, 3e38, -3e38, 0.0, 200.0]], dtype=torch.bfloat16)
        one = torch.zeros((8, 8), dtype=torch.bfloat16).cuda()
        g = torch.ones((1, 8), dtype=torch.bfloat16).cuda()
        dx = torch.empty((1, 8), dtype=torch.bfloat16, device="cuda")
        one.fill_diagonal_(1.0)
        binding.linear_dgrad(g, one, dx, act=act, z=big.cuda())
        want = [1, 0, 1, 0, 1, 0, 0.0 if act == "relu" else 0.5, 1]
        assert dx[0].tolist() == want, (act, dx[0].tolist())


def test_linear_dgrad_of_relu_drops_infinities():
    """Where relu was off its gradient is zero whatever comes back; a NaN of z
    is kept."""
    w = torch.eye(8).bfloat16().cuda()
    z = torch.tensor([[1.0, -1.0, 1.0, -1.0, 0.0, float("nan"), -float("inf"), float("inf")]]).bfloat16()
    g = torch.full((1, 8), 2.0).bfloat16()
    g_inf = torch.full((1, 8), float("inf")).bfloat16()
    for rows in (1, 130):
        dx = torch.empty((rows, 8), dtype=torch.bfloat16, device="cuda")
        zz = z.expand(rows, 8).contiguous().cuda()
        binding.linear_dgrad(g.expand(rows, 8).contiguous().cuda(), w, dx, act="relu", z=zz)
        assert torch.isnan(dx[:, 5]).all()
        assert dx[0, [0, 1, 2, 3, 4, 6, 7]].tolist() == [2, 0, 2, 0, 0, 0, 2]
        # infinite and NaN products (inf * 0)
        binding.linear_dgrad(g_inf.expand(rows, 8).contiguous().cuda(), w, dx, act="relu", z=zz)
        assert dx[0, [1, 3, 4, 6]].tolist() == [0, 0, 0, 0]


def test_adamw_refuses_tensors_that_overlap():
    buf, g = torch.zeros(64, device="cuda"), torch.zeros(32, device="cuda")
    a, b = buf[:32], buf[16:48]
    binding.AdamW([a, buf[32:]], [g, g])                         # one gradient for two tensors is only read
    for params, grads, kw in (([a, a], [g, g], {}), ([a, b], [g, g], {}), ([a], [b], {}),
                              ([a], [g], dict(m=[buf[32:]], v=[buf[32:]])),
                              ([a], [g], dict(lowp=[a.view(torch.bfloat16)[:32]]))):
        with pytest.raises(ValueError, match="overlaps"):
            binding.AdamW(params, grads, **kw)


def test_linear_is_reproducible_and_replays():
    """Same bits on every run, on another stream and from a replayed graph
    with new inputs in the same buffers."""
    rows, k, n = 700, 1024, 520
    x, w, g = _rand(32, rows, k).cuda(), _rand(33, k, n, std=k ** -0.5).cuda(), _rand(34, rows, n).cuda()
    y, dx = torch.empty_like(g), torch.empty_like(x)
    dw, db = torch.zeros((k, n), device="cuda"), torch.zeros(n, device="cuda")

    def run(stream=None):
        binding.linear_fwd(x, w, y, act="gelu", stream=stream)
        binding.linear_dgrad(g, w, dx, stream=stream)
        binding.linear_wgrad(x, g, dw, dbias=db, stream=stream)

    run()
    torch.cuda.synchronize()
    first = [t.clone() for t in (y, dx, dw, db)]
    side = torch.cuda.Stream()
    dw.zero_(), db.zero_()
    side.wait_stream(torch.cuda.current_stream())
    run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw, db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    x.copy_(_rand(35, rows, k).cuda())
    dw.zero_(), db.zero_()
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (y, dx, dw, db)]
    dw.zero_(), db.zero_()
    run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(replayed, (y, dx, dw, db)))
    assert not torch.equal(first[0], y)


def test_linear_calls_side_by_side():
    """Two products of one weight on two streams at once."""
    k, n = 2048, 1024
    w = _rand(36, k, n, std=k ** -0.5).cuda()
    xs = [_rand(37 + i, 300 + 40 * i, k).cuda() for i in range(2)]
    ys = [torch.empty((x.shape[0], n), dtype=torch.bfloat16, device="cuda") for x in xs]
    want = [torch.empty_like(y) for y in ys]
    for x, y in zip(xs, want):
        binding.linear_fwd(x, w, y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        for st, x, y in zip(streams, xs, ys):
            binding.linear_fwd(x, w, y, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))


@pytest.mark.parametrize("rows,k,n", [(70, 264, 136), (700, 512, 1032)])
def test_linear_waits_run_out_and_recover(rows, k, n):
    """A one-cycle wait limit: the status says so once, and the same calls
    succeed afterwards."""
    x, w, g = _rand(60, rows, k).cuda(), _rand(61, k, n, std=k ** -0.5).cuda(), _rand(62, rows, n).cuda()
    y, dx, dw = torch.empty_like(g), torch.empty_like(x), torch.zeros((k, n), device="cuda")
    binding.sync_status()
    for call in (lambda: binding.linear_fwd(x, w, y), lambda: binding.linear_dgrad(g, w, dx),
                 lambda: binding.linear_wgrad(x, g, dw)):
        try:
            binding.set_wait_limit(1)
            call()
            with pytest.raises(binding.SeqattnError) as e:
                binding.sync_status()
            assert e.value.status == binding.SEQATTN_ERR_TIMEOUT
        finally:
            binding.set_wait_limit(0)
        binding.sync_status()
    dw.zero_()
    binding.linear_fwd(x, w, y)
    binding.linear_dgrad(g, w, dx)
    binding.linear_wgrad(x, g, dw)
    binding.sync_status()
    ref = x.double().cpu() @ w.double().cpu()
    _within("y", y, ref, U_BF16 * ref.abs() + _sum_tol(k, x.double().cpu().abs() @ w.double().cpu().abs()))
    ref = x.double().cpu().t() @ g.double().cpu()
    _within("dw", dw, ref, 50 * 2.0 ** -23 * (x.double().cpu().abs().t() @ g.double().cpu().abs()))


@pytest.mark.parametrize("rows,k,n", [(40, 512, 264), (300, 64, 136), (2570, 520, 1800)])
def test_linear_writes_nothing_after_an_error(rows, k, n):
    """Calls that find the error word set leave their outputs alone, and the
    next ones after it has been read and cleared are whole."""
    x, w, g = _rand(63, rows, k).cuda(), _rand(64, k, n, std=k ** -0.5).cuda(), _rand(65, rows, n).cuda()
    y, dx, dw = torch.full_like(g, 7.0), torch.full_like(x, 7.0), torch.full((k, n), 7.0, device="cuda")
    first = torch.empty_like(g)
    binding.sync_status()
    try:
        binding.set_wait_limit(1)
        binding.linear_fwd(x, w, first)
    finally:
        binding.set_wait_limit(0)
    binding.linear_fwd(x, w, y)
    binding.linear_dgrad(g, w, dx)
    binding.linear_wgrad(x, g, dw)
    with pytest.raises(binding.SeqattnError):
        binding.sync_status()
    assert (y == 7).all() and (dx == 7).all() and (dw == 7).all()
    binding.linear_fwd(x, w, y)
    binding.sync_status()
    ref = x.double() @ w.double()
    _within("y", y, ref.cpu(), (U_BF16 * ref.abs() + _sum_tol(k, x.double().abs() @ w.double().abs())).cpu())


# ============================================================== head norm + rotary positions

def _angles(positions, inv_freq, axis):
    """[B, c, 1, pairs] in float64; positions [axes, B, c]."""
    return torch.stack([positions[a].double() * f for a, f in zip(axis, inv_freq)], -1)[:, :, None]


def _rope64(x, ang, inter):
    rot = 2 * ang.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    c, s = torch.cos(ang), torch.sin(ang)
    y = (a * c - b * s, b * c + a * s)
    y = torch.stack(y, -1).flatten(-2) if inter else torch.cat(y, -1)
    return torch.cat((y, x[..., rot:]), -1)


def _norm_rope64(x, gamma, eps, ang, inter):
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma
    return _rope64(x, ang, inter) if ang is not None else x


ROPE_CASES = [
    # B, start, c, tail, Hq, Hkv, d, rot, axes, interleaved, norm, dtype
    (1, 0, 1, 0, 1, 1, 128, 128, 1, False, True, "bf16"),
    (2, 37, 5, 3, 4, 2, 128, 128, 1, False, True, "bf16"),
    (1, 131000, 33, 0, 32, 8, 128, 128, 1, False, True, "bf16"),
    (3, 7, 50, 11, 5, 5, 64, 64, 1, True, True, "fp32"),
    (2, 0, 64, 0, 3, 1, 64, 32, 3, False, True, "fp32"),
    (1, 100, 40, 9, 8, 2, 128, 64, 2, True, False, "bf16"),
    (1, 5, 17, 1, 7, 7, 128, 16, 1, False, False, "fp32"),
    (1, 3, 200, 2, 16, 2, 64, 0, 1, False, True, "bf16"),
    (2, 0, 600, 0, 6, 3, 128, 128, 3, True, True, "bf16"),
]


def _rope_case(B, start, c, tail, Hq, Hkv, d, rot, axes, inter, norm, dtype, seed=40):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T = start + c + tail
    inv = [1e4 ** (-2.0 * i / rot) for i in range(rot // 2)] if rot else None
    axis = [i * axes // (rot // 2) for i in range(rot // 2)] if rot else None
    plan = binding.rope_plan(inv, axis, inter) if rot else None
    pos = None
    if axes > 1:
        g = torch.Generator().manual_seed(seed)
        pos = torch.randint(-5, 200000, (axes, B, c), generator=g)
    p64 = pos if pos is not None else torch.arange(start, start + c).expand(1, B, c)
    ang = _angles(p64, inv, axis) if rot else None
    qkv = _rand(seed + 1, B, c, Hq + 2 * Hkv, d, dtype=dt, std=1.5)
    gq = (1 + _rand(seed + 2, d, dtype=torch.float32, std=0.3)).to(dt) if norm else None
    gk = (1 + _rand(seed + 3, d, dtype=torch.float32, std=0.3)).to(dt) if norm else None
    return dt, T, plan, pos, ang, qkv, gq, gk


def _dev(t):
    return None if t is None else t.cuda()


def _scale_of(x):
    """Largest magnitude of each head, the size that rounding errors of a rotated pair are relative to."""
    return x.abs().amax(-1, keepdim=True)


@pytest.mark.parametrize("case", ROPE_CASES)
def test_norm_rope_fwd(case):
    B, start, c, tail, Hq, Hkv, d, rot, axes, inter, norm, dtype = case
    dt, T, plan, pos, ang, qkv, gq, gk = _rope_case(*case)
    q_in, k_in, v_in = qkv.cuda().split((Hq, Hkv, Hkv), 2)
    k_old, v_old = _rand(44, B, T, Hkv, d, dtype=dt), _rand(45, B, T, Hkv, d, dtype=dt)
    q = torch.full((B, c, Hq, d), float("nan"), dtype=dt, device="cuda")
    k, v = k_old.cuda(), v_old.cuda()
    binding.qk_norm_rope_fwd(q_in, k_in, v_in, q, k, v, start, gamma_q=_dev(gq), gamma_k=_dev(gk), eps=1e-5, plan=plan,
                             positions=_dev(pos))
    u = U_BF16 if dt == torch.bfloat16 else U_F32
    for name, got, x, gamma in (("q", q, qkv[:, :, :Hq], gq), ("k", k[:, start:start + c], qkv[:, :, Hq:Hq + Hkv], gk)):
        ref = _norm_rope64(x.double(), None if gamma is None else gamma.double(), 1e-5, ang, inter)
        _within(name, got, ref, u * ref.abs() + 24 * U_F32 * _scale_of(ref) + 1e-30)
    assert torch.equal(v[:, start:start + c].cpu(), qkv[:, :, Hq + Hkv:])
    for got, old in ((k, k_old), (v, v_old)):                   # rows of other chunks stay
        assert torch.equal(got[:, :start].cpu(), old[:, :start])
        assert torch.equal(got[:, start + c:].cpu(), old[:, start + c:])


@pytest.mark.parametrize("case", ROPE_CASES)
def test_norm_rope_bwd(case):
    B, start, c, tail, Hq, Hkv, d, rot, axes, inter, norm, dtype = case
    dt, T, plan, pos, ang, qkv, gq, gk = _rope_case(*case)
    dq = _rand(46, B, c, Hq, d, dtype=torch.float32)
    dk, dv = _rand(47, B, T, Hkv, d, dtype=torch.float32), _rand(48, B, T, Hkv, d, dtype=torch.float32)
    dgq, dgk = _rand(49, d, dtype=torch.float32), _rand(50, d, dtype=torch.float32)
    q_in, k_in, _ = qkv.cuda().split((Hq, Hkv, Hkv), 2)
    out = torch.full((B, c, Hq + 2 * Hkv, d), float("nan"), dtype=dt, device="cuda")
    oq, ok, ov = out.split((Hq, Hkv, Hkv), 2)
    dgq_d, dgk_d = dgq.cuda(), dgk.cuda()
    binding.qk_norm_rope_bwd(q_in if norm else None, k_in if norm else None, dq.cuda(), dk.cuda(), dv.cuda(), oq, ok, ov,
                             start, gamma_q=_dev(gq), gamma_k=_dev(gk), dgamma_q=dgq_d, dgamma_k=dgk_d, eps=1e-5,
                             plan=plan, positions=_dev(pos))
    u = U_BF16 if dt == torch.bfloat16 else U_F32
    rows = slice(start, start + c)
    for name, got, x, gamma, dy, old, dg in (("q", oq, qkv[:, :, :Hq], gq, dq, dgq, dgq_d),
                                             ("k", ok, qkv[:, :, Hq:Hq + Hkv], gk, dk[:, rows], dgk, dgk_d)):
        x64 = x.double().requires_grad_(True)
        g64 = None if gamma is None else gamma.double().requires_grad_(True)
        y = _norm_rope64(x64, g64, 1e-5, ang, inter)
        (y * dy.double()).sum().backward()
        size = _scale_of(dy.double())
        if norm:    # r gamma dn and r xhat mean(gamma dn xhat), each of the head's size
            r = 1 / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-5)
            size = size * r * gamma.double().abs().max() * (2 + (x.double() * r).abs())
        _within("d" + name, got, x64.grad, u * x64.grad.abs() + 32 * U_F32 * size + 1e-30)
        if norm:
            # each term 12 roundings; a thread adds at most its rows' heads in turn, then warps and blocks
            xhat = x.double() * r
            mags = (_scale_of(dy.double()) * 2 * xhat.abs()).sum((0, 1, 2)) + old.double().abs()
            _within("dgamma_" + name, dg, old.double() + g64.grad, (12 + 40) * U_F32 * mags)
        else:
            assert torch.equal(dg.cpu(), old)
    _within("dv", ov, dv[:, rows].double(), u * dv[:, rows].double().abs() + 1e-40)


def test_norm_rope_gradient_is_the_forwards_slope():
    """Central differences of the float32 forward kernel along random directions."""
    case = (2, 11, 9, 0, 4, 2, 64, 64, 1, False, True, "fp32")
    dt, T, plan, pos, ang, qkv, gq, gk = _rope_case(*case)
    B, start, c, _, Hq, Hkv, d = case[:7]
    wq, wk = _rand(51, B, c, Hq, d, dtype=dt).cuda(), _rand(52, B, T, Hkv, d, dtype=dt).cuda()
    qkv, gq, gk = qkv.cuda(), gq.cuda(), gk.cuda()

    def loss(t, a, b):
        q = torch.empty((B, c, Hq, d), device="cuda")
        k = torch.zeros((B, T, Hkv, d), device="cuda")
        binding.qk_norm_rope_fwd(t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], None, q, k, None, start, gamma_q=a, gamma_k=b,
                                 plan=plan)
        return (q.double() * wq.double()).sum() + (k.double() * wk.double())[:, start:].sum()

    dx, dgq, dgk = torch.zeros_like(qkv), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")
    binding.qk_norm_rope_bwd(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], wq, wk, None, dx[:, :, :Hq], dx[:, :, Hq:Hq + Hkv],
                             None, start, gamma_q=gq, gamma_k=gk, dgamma_q=dgq, dgamma_k=dgk, plan=plan)
    h = 2.0 ** -7
    for seed in range(3):
        e = _rand(53 + seed, *qkv.shape, dtype=dt).cuda()
        eq, ek = _rand(56 + seed, d, dtype=dt).cuda(), _rand(59 + seed, d, dtype=dt).cuda()
        slope = (loss(qkv + h * e, gq + h * eq, gk + h * ek) - loss(qkv - h * e, gq - h * eq, gk - h * ek)) / (2 * h)
        parts = torch.stack([(dx.double() * e.double()).sum(), (dgq.double() * eq.double()).sum(),
                             (dgk.double() * ek.double()).sum()])
        # h^2 times third derivatives (order one per element), summed over 4608 elements at random signs,
        # and float32 roundings of the loss' 3456 terms over 2 h
        assert abs(float(slope - parts.sum())) <= 20 * h * h * math.sqrt(qkv.numel()) + 3456 ** 0.5 * 8 * U_F32 / h


def test_norm_rope_replays_reproduces_and_keeps_values_optional():
    B, start, c, Hq, Hkv, d = 1, 64, 300, 8, 2, 128
    dt, T, plan, pos, ang, qkv, gq, gk = _rope_case(B, start, c, 0, Hq, Hkv, d, d, 1, False, True, "bf16")
    qkv, gq, gk = qkv.cuda(), gq.cuda(), gk.cuda()
    q_in, k_in, v_in = qkv.split((Hq, Hkv, Hkv), 2)
    q = torch.empty((B, c, Hq, d), dtype=dt, device="cuda")
    k, v = torch.zeros((B, T, Hkv, d), dtype=dt, device="cuda"), torch.zeros((B, T, Hkv, d), dtype=dt, device="cuda")
    dq = _rand(70, B, c, Hq, d, dtype=torch.float32).cuda()
    dk = _rand(71, B, T, Hkv, d, dtype=torch.float32).cuda()
    dx, dgq, dgk = torch.zeros_like(qkv), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")
    oq, ok, ov = dx.split((Hq, Hkv, Hkv), 2)
    ws = torch.empty(binding.qk_norm_rope_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")

    def run(stream=None, workspace=ws):
        binding.qk_norm_rope_fwd(q_in, k_in, v_in, q, k, v, start, gamma_q=gq, gamma_k=gk, plan=plan, stream=stream)
        binding.qk_norm_rope_bwd(q_in, k_in, dq, dk, dk, oq, ok, ov, start, gamma_q=gq, gamma_k=gk, dgamma_q=dgq,
                                 dgamma_k=dgk, plan=plan, workspace=workspace, stream=stream)

    outs = (q, k, v, dx, dgq, dgk)
    run()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    for t in outs:
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(side, None)                                             # its own temporary workspace
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    # without values: the rest is the same, the value cache is left alone
    v.fill_(7.0)
    q.zero_()
    binding.qk_norm_rope_fwd(q_in, k_in, None, q, k, None, start, gamma_q=gq, gamma_k=gk, plan=plan)
    dx.fill_(9.0), dgq.zero_(), dgk.zero_()
    binding.qk_norm_rope_bwd(q_in, k_in, dq, dk, None, oq, ok, None, start, gamma_q=gq, gamma_k=gk, dgamma_q=dgq,
                             dgamma_k=dgk, plan=plan)
    torch.cuda.synchronize()
    assert torch.equal(q, first[0]) and (v == 7).all() and (ov == 9).all()
    # dgamma adds the same terms, but the values' heads are no longer among those dealt to the warps,
    # so in another order: two sums of terms |dn xhat| <= 2 max|dy| |xhat|, 40 additions deep each
    x = qkv[:, :, :Hq].double()
    xhat = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + 1e-6)
    mags = (_scale_of(dq.double()) * 2 * xhat.abs()).sum((0, 1, 2)).cpu()
    _within("dgamma_q", dgq, first[4].double().cpu(), 2 * 40 * U_F32 * mags)


def test_norm_rope_binding_refuses():
    B, c, Hq, Hkv, d, T = 2, 4, 4, 2, 64, 8
    qkv = torch.zeros((B, c, Hq + 2 * Hkv, d), device="cuda")
    q_in, k_in, v_in = qkv.split((Hq, Hkv, Hkv), 2)
    q, k = torch.zeros((B, c, Hq, d), device="cuda"), torch.zeros((B, T, Hkv, d), device="cuda")
    f = binding.qk_norm_rope_fwd
    with pytest.raises(ValueError, match="both be given"):
        f(q_in, k_in, v_in, q, k, None, 0)
    with pytest.raises(ValueError, match="both be given"):
        f(q_in, k_in, v_in, q, k, k.clone(), 0, gamma_q=torch.ones(d, device="cuda"))
    with pytest.raises(ValueError, match="uniform stride"):
        f(torch.zeros((B, c + 1, Hq, d), device="cuda")[:, :c], k_in, v_in, q, k, k.clone(), 0)
    with pytest.raises(ValueError, match="dense"):
        f(torch.zeros((B, c, d, Hq), device="cuda").transpose(2, 3), k_in, v_in, q, k, k.clone(), 0)
    with pytest.raises(ValueError, match="positions"):
        f(q_in, k_in, v_in, q, k, k.clone(), 0, positions=torch.zeros((B, c + 1), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="int64"):
        f(q_in, k_in, v_in, q, k, k.clone(), 0, positions=torch.zeros((B, c), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        f(q_in.bfloat16(), k_in, v_in, q, k, k.clone(), 0)
    with pytest.raises(binding.SeqattnError, match="seq_capacity"):
        f(q_in, k_in, v_in, q, k, k.clone(), T - c + 1)
    with pytest.raises(binding.SeqattnError, match="rot_dim"):
        f(q_in, k_in, v_in, q, k, k.clone(), 0, plan=binding.rope_plan([1.0] * 64))


# ============================================================== AdamW

def _e4m3(x):
    """All of x's nearest e4m3 values' magnitudes and half steps: (value, half the local step)."""
    mant, exp = np.frexp(np.abs(x))
    ulp = np.ldexp(1.0, np.maximum(exp, -5) - 4)
    return ulp / 2


ADAMW_SIZES = [1, 3, 255, 256, 257, 2048, 5000, 128, 0, 4097]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [ADAMW_SIZES, [77] * 450, [1]])
def test_adamw_steps(bits, g_dtype, sizes):
    lr, b1, b2, eps, gs = 1e-2, 0.9, 0.95, 1e-8, 0.25
    p = [_rand(80 + i, n, dtype=torch.float32) for i, n in enumerate(sizes)]
    decay = [0.1 * (i % 3) for i in range(len(sizes))]
    dev = [t.cuda() for t in p]
    grads = [torch.zeros(n, dtype=g_dtype, device="cuda") for n in sizes]
    lowp = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") if i % 4 else None for i, n in enumerate(sizes)]
    opt = binding.AdamW(dev, grads, lowp=lowp, state_bits=bits, weight_decay=decay)
    for step in range(1, 4):
        for i, g in enumerate(grads):
            g.copy_(_rand(1000 * step + i, *g.shape, dtype=torch.float32).mul(10.0 ** (i % 5 - 2)).to(g_dtype))
        old_p = [t.double().cpu() for t in dev]
        if bits == 32:
            old_m, old_v = [t.double().cpu() for t in opt.m], [t.double().cpu() for t in opt.v]
        else:
            old_m = [_dequant(c, s) for c, s in zip(opt.m, opt.m_scale)]
            old_v = [_dequant(c, s) ** 2 for c, s in zip(opt.v, opt.v_scale)]
        opt.step(lr, step, beta1=b1, beta2=b2, eps=eps, grad_scale=gs)
        torch.cuda.synchronize()
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            g = grads[i].double().cpu() * gs
            m = b1 * old_m[i] + (1 - b1) * g
            v = b2 * old_v[i] + (1 - b2) * g * g
            mm = b1 * old_m[i].abs() + (1 - b1) * g.abs()         # magnitudes that m's roundings are relative to
            denom = v.sqrt() / math.sqrt(1 - b2 ** step) + eps
            ratio = m / denom
            ref = old_p[i] * (1 - lr * decay[i]) - lr / (1 - b1 ** step) * ratio
            tol = 4 * U_F32 * old_p[i].abs() + 16 * U_F32 * lr / (1 - b1 ** step) * mm / denom + 1e-30
            _within(f"p[{i}]", dev[i], ref, tol)
            if lowp[i] is not None:
                assert torch.equal(lowp[i], dev[i].to(torch.bfloat16))
            if bits == 32:
                _within(f"m[{i}]", opt.m[i], m, 8 * U_F32 * mm + 1e-40)
                _within(f"v[{i}]", opt.v[i], v, 8 * U_F32 * v + 1e-40)
                continue
            for name, code, scale, want, least in (("m", opt.m[i], opt.m_scale[i], m, 0.5),
                                                   ("u", opt.v[i], opt.v_scale[i], v.sqrt(), 1.0)):
                pad = torch.zeros(-(-n // 256) * 256, dtype=torch.float64)
                pad[:n] = want
                top = pad.reshape(-1, 256).abs().amax(1)
                slack = (8 * U_F32 * mm).max() if name == "m" else 0.0
                _within(f"{name}_scale[{i}]", scale, top / 448, 12 * U_F32 * top / 448 + slack / 448 + 1e-40)
                s = scale.double().cpu().repeat_interleave(256)[:n]
                half = torch.from_numpy(_e4m3((want / s).clamp(-448, 448).numpy())) * s
                tol = torch.maximum(half, least * 2.0 ** -9 * s) * (1 + 1e-5) + 8 * U_F32 * mm.max()
                _within(f"{name}[{i}]", _dequant(code, scale), want, tol)
                if name == "u":
                    assert ((code.float().cpu() != 0) | (want == 0)).all()


def _dequant(code, scale):
    n = code.numel()
    return code.float().double().cpu() * scale.double().cpu().repeat_interleave(256)[:n]


def test_adamw_state_extremes():
    """Zero gradients, a block of zeros, tiny and huge magnitudes in one
    block, a NaN: each stays where it is."""
    n = 1024
    p = torch.ones(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    g[256] = 1e-25                       # alone in its block
    g[512], g[513] = 1e4, 1e-9           # far more apart than e4m3's range
    g[768] = float("nan")
    opt = binding.AdamW([p], [g], state_bits=8)
    opt.step(1e-3, 1)
    torch.cuda.synchronize()
    assert (p[:256] == 1).all() and opt.m_scale[0][0] == 0 and (opt.m[0][:256].float() == 0).all()
    want = 1 - 1e-3 * 1e-25 / (1e-25 + 1e-8)
    assert abs(float(p[256]) - want) < 1e-7 and (p[257:512] == 1).all()
    assert float(opt.v[0][513].float()) == 2.0 ** -9       # kept above zero
    assert (p[514:768] == 1).all()
    assert torch.isnan(p[768]) and torch.isfinite(p[769:]).all()
    for step in range(2, 6):
        opt.step(1e-3, step)
    torch.cuda.synchronize()
    assert torch.isfinite(p[:768]).all() and float((p[:768] - 1).abs().max()) < 6e-3


def test_adamw_guards_its_neighbours():
    """Odd tails of views in one flat array: the gaps between them stay."""
    sizes, starts, at = [5, 1000, 300], [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // 256) * 256
    flat = {k: torch.full((at,), 3.0, dtype=dt, device="cuda") for k, dt in
            (("p", torch.float32), ("lo", torch.bfloat16), ("g", torch.float32))}
    codes = {k: torch.zeros(at, device="cuda").to(torch.float8_e4m3fn) for k in ("m", "v")}
    scales = {k: torch.zeros(at // 256, device="cuda") for k in ("m", "v")}
    cut = lambda t: [t[a:a + n] for a, n in zip(starts, sizes)]                          # noqa: E731
    scut = lambda t: [t[a // 256:a // 256 + -(-n // 256)] for a, n in zip(starts, sizes)]   # noqa: E731
    opt = binding.AdamW(cut(flat["p"]), cut(flat["g"]), lowp=cut(flat["lo"]), state_bits=8, m=cut(codes["m"]),
                        v=cut(codes["v"]), m_scale=scut(scales["m"]), v_scale=scut(scales["v"]))
    opt.step(0.5, 1)
    torch.cuda.synchronize()
    gap = torch.ones(at, dtype=torch.bool)
    for a, n in zip(starts, sizes):
        gap[a:a + n] = False
    assert (flat["p"].cpu()[gap] == 3).all() and (flat["lo"].cpu()[gap] == 3).all()
    assert (codes["m"].float().cpu()[gap] == 0).all() and (codes["v"].float().cpu()[gap] == 0).all()
    assert (flat["p"].cpu()[~gap] != 3).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_replays_with_device_scalars(bits):
    """A captured step that takes its step number, rate and gradient scale
    from the device gives what eager steps with numbers give."""
    sizes = [1000, 64]
    p0 = [_rand(90 + i, n, dtype=torch.float32) for i, n in enumerate(sizes)]
    g = [_rand(95 + i, n, dtype=torch.float32).cuda() for i, n in enumerate(sizes)]
    a, b = [t.cuda() for t in p0], [t.cuda() for t in p0]
    eager, captured = binding.AdamW(a, g, state_bits=bits), binding.AdamW(b, g, state_bits=bits)
    lr, scale = torch.tensor([0.0], device="cuda"), torch.tensor([0.0], device="cuda")
    step = torch.tensor([0], dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step(lr, step, grad_scale=scale)
    for i in range(1, 4):
        rate, gs = float(np.float32(0.01 / i)), 0.5 ** i
        eager.step(rate, i, grad_scale=gs)
        lr.fill_(rate), scale.fill_(gs), step.fill_(i)
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(a + eager.m + eager.v, b + captured.m + captured.v):
        assert torch.equal(x.float(), y.float())


def test_adamw_refuses():
    p, g = [torch.zeros(300, device="cuda")], [torch.zeros(300, device="cuda")]
    with pytest.raises(ValueError, match="elements"):
        binding.AdamW(p, [torch.zeros(299, device="cuda")])
    with pytest.raises(TypeError):
        binding.AdamW(p, [g[0].half()])
    with pytest.raises(ValueError, match="contiguous"):
        binding.AdamW(p, [torch.zeros(600, device="cuda")[::2]])
    opt = binding.AdamW(p, g)
    with pytest.raises(binding.SeqattnError, match="step"):
        opt.step(1e-3, 0)
    with pytest.raises(ValueError, match="int64"):
        opt.step(1e-3, torch.ones(1, device="cuda"))
    with pytest.raises(binding.SeqattnError, match="beta"):
        opt.step(1e-3, 1, beta1=1.0)
    with pytest.raises(binding.SeqattnError, match="aligned"):
        binding.AdamW([torch.zeros(301, device="cuda")[1:]], g).step(1e-3, 1)
    binding.AdamW([], []).step(1e-3, 1)


# ============================================================== offsets past 32 bits

def test_norm_rope_in_a_cache_of_more_than_2_31_elements():
    """Rows near the end of 4.4 GB caches: the same bits as the same rows of a
    short cache, given the same positions."""
    B, c, Hq, Hkv, d, T = 1, 3, 64, 64, 128, 270000
    start = T - c
    assert start * Hkv * d > 2 ** 31
    qkv = _rand(110, B, c, Hq + 2 * Hkv, d).cuda()
    q_in, k_in, v_in = qkv.split((Hq, Hkv, Hkv), 2)
    gamma = (1 + _rand(111, d, dtype=torch.float32, std=0.2)).bfloat16().cuda()
    plan = binding.rope_plan([1e4 ** (-i / 64) for i in range(64)])
    pos = torch.arange(start, T, device="cuda")[None, None]
    outs = []
    for rows, at, p in ((T, start, None), (c, 0, pos)):
        q = torch.zeros((B, c, Hq, d), dtype=torch.bfloat16, device="cuda")
        k = torch.zeros((B, rows, Hkv, d), dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        binding.qk_norm_rope_fwd(q_in, k_in, v_in, q, k, v, at, gamma_q=gamma, gamma_k=gamma, plan=plan, positions=p)
        assert int((k[:, :at] != 0).sum()) == 0 and int((v[:, :at] != 0).sum()) == 0
        outs.append((q, k[:, at:].clone(), v[:, at:].clone()))
        del k, v
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    dq = _rand(112, B, c, Hq, d, dtype=torch.float32).cuda()
    rows_dk = _rand(113, B, c, Hkv, d, dtype=torch.float32).cuda()
    outs = []
    for rows, at, p in ((T, start, None), (c, 0, pos)):
        dk = torch.empty((B, rows, Hkv, d), device="cuda")
        dk[:, at:] = rows_dk
        dx, dgq, dgk = torch.zeros_like(qkv), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")
        oq, ok, _ = dx.split((Hq, Hkv, Hkv), 2)
        binding.qk_norm_rope_bwd(q_in, k_in, dq, dk, None, oq, ok, None, at, gamma_q=gamma, gamma_k=gamma,
                                 dgamma_q=dgq, dgamma_k=dgk, plan=plan, positions=p)
        outs.append((dx, dgq, dgk))
        del dk
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_linear_with_more_than_2_31_elements():
    rows, k, n = 270000, 64, 8192
    x, w = _rand(114, 4096, k).cuda().repeat(66, 1)[:rows], _rand(115, k, n).cuda()
    y = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    binding.linear_fwd(x, w, y)
    ref = x[:4096].double() @ w.double()
    tol = U_BF16 * ref.abs() + _sum_tol(k, x[:4096].double().abs() @ w.double().abs())
    for at in (0, 4096 * 63, 4096 * 64):
        off = (y[at:at + 4096].double() - ref).abs()
        assert bool((off <= tol).all())
    assert torch.equal(y[4096 * 65:], y[:rows - 4096 * 65])
    dx = torch.empty_like(x)
    binding.linear_dgrad(y, w, dx)                      # reads the long matrix
    assert torch.equal(dx[4096 * 64:4096 * 65], dx[:4096])
    assert torch.equal(dx[4096 * 65:], dx[:rows - 4096 * 65])
    dw, part = torch.zeros((k, n), device="cuda"), torch.zeros((k, n), device="cuda")
    tail = rows - 4096 * 65
    y[:rows - tail] = 0                                 # only the last rows count
    binding.linear_wgrad(x, y, dw)
    binding.linear_wgrad(x[rows - tail:], y[rows - tail:], part)
    mags = x[rows - tail:].double().abs().t() @ y[rows - tail:].double().abs()
    _within("dw", dw, part.double().cpu(), 2 * (48 * 2.0 ** -23 + (rows / 512 + 2) * U_F32) * mags.cpu())


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_tensor_of_more_than_2_31_elements(bits):
    n, cut = 2 ** 31 + 256 * 5 + 77, 2 ** 31 - 256
    tail_p = _rand(116, n - cut, dtype=torch.float32).cuda()
    tail_g = _rand(117, n - cut).cuda()
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[cut:], g[cut:] = tail_p, tail_g
    big, small = binding.AdamW([p], [g], state_bits=bits), binding.AdamW([tail_p], [tail_g], state_bits=bits)
    for step in (1, 2):
        big.step(1e-2, step)
        small.step(1e-2, step)
    torch.cuda.synchronize()
    assert torch.equal(p[cut:], tail_p) and int((p[:cut] != 0).sum()) == 0
    assert torch.equal(big.m[0][cut:].float(), small.m[0].float())
    assert torch.equal(big.v[0][cut:].float(), small.v[0].float())
    if bits == 8:
        assert torch.equal(big.m_scale[0][cut // 256:], small.m_scale[0])


# ============================================================== side by side

def test_all_operators_on_two_streams_at_once():
    """Two streams run the same chain of different data over shared weights,
    several times; each gets what it gets alone."""
    k, n, rows, H, d = 512, 6 * 64, 300, 2, 64
    w = _rand(120, k, n, std=k ** -0.5).cuda()
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    plan = binding.rope_plan([1e4 ** (-i / 32) for i in range(32)])

    def state(seed):
        z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")        # noqa: E731
        return dict(x=_rand(seed, rows, k).cuda(), qkv=z(rows, n, dt=torch.bfloat16),
                    q=z(1, rows, H, d, dt=torch.bfloat16), k=z(1, rows, H, d, dt=torch.bfloat16),
                    v=z(1, rows, H, d, dt=torch.bfloat16), dq=_rand(seed + 1, 1, rows, H, d, dtype=torch.float32).cuda(),
                    dx=z(1, rows, 3 * H, d, dt=torch.bfloat16), dh=z(rows, k, dt=torch.bfloat16), dw=z(k, n),
                    db=z(n), dgq=z(d), dgk=z(d), p=z(k, n))

    def chain(s, opt, stream):
        with torch.cuda.stream(stream):
            for t in (s["dw"], s["db"], s["dgq"], s["dgk"]):
                t.zero_()
            binding.linear_fwd(s["x"], w, s["qkv"])
            q_in, k_in, v_in = s["qkv"].view(1, rows, 3 * H, d).split((H, H, H), 2)
            binding.qk_norm_rope_fwd(q_in, k_in, v_in, s["q"], s["k"], s["v"], 0, gamma_q=gamma, gamma_k=gamma, plan=plan)
            oq, ok, ov = s["dx"].split((H, H, H), 2)
            binding.qk_norm_rope_bwd(q_in, k_in, s["dq"], s["dq"], s["dq"], oq, ok, ov, 0, gamma_q=gamma, gamma_k=gamma,
                                     dgamma_q=s["dgq"], dgamma_k=s["dgk"], plan=plan)
            flat = s["dx"].view(rows, n)
            binding.linear_dgrad(flat, w, s["dh"])
            binding.linear_wgrad(s["x"], flat, s["dw"], dbias=s["db"])
            opt.step(1e-2, 1)

    def run(streams):
        states = [state(130), state(140)]
        opts = [binding.AdamW([s["p"]], [s["dw"]], state_bits=8) for s in states]
        torch.cuda.synchronize()
        for _ in range(4):
            for s, o, st in zip(states, opts, streams):
                chain(s, o, st)
        torch.cuda.synchronize()
        return states

    main = torch.cuda.current_stream()
    alone, together = run([main, main]), run([torch.cuda.Stream(), torch.cuda.Stream()])
    for a, b in zip(alone, together):
        for name in a:
            assert torch.equal(a[name], b[name]), name


def test_first_calls_may_be_captured():
    """In a new process, calls that have never run are captured into a graph
    and replayed."""
    code = """
import torch
from long_context_attention_seqattn_gb300 import binding
def new(*shape):
    return torch.randn(shape, device="cuda").bfloat16()
xs, w = [new(r, 512) for r in (1, 40, 2570)], new(512, 1800) / 32
ys = [torch.zeros(len(x), 1800, device="cuda", dtype=torch.bfloat16) for x in xs]
dw = torch.zeros_like(w, dtype=torch.float32)
qkv = new(1, 64, 6, 128)
q, k, v = (torch.zeros(1, 64, h, 128, device="cuda", dtype=torch.bfloat16) for h in (4, 1, 1))
p, g = torch.zeros(1000, device="cuda"), torch.ones(1000, device="cuda")
opt = binding.AdamW([p], [g], state_bits=8)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for x, y in zip(xs, ys):
        binding.linear_fwd(x, w, y)
    binding.linear_wgrad(xs[1], ys[1], dw)
    binding.qk_norm_rope_fwd(*qkv.split((4, 1, 1), 2), q, k, v, 0, plan=binding.rope_plan([0.0] * 64))
    opt.step(0.5, 1)
graph.replay()
binding.sync_status()
for x, y in zip(xs, ys):
    ref = x.double() @ w.double()
    assert ((y - ref).abs() <= 2.0 ** -8 * ref.abs() + 48 * 2.0 ** -23 * (x.double().abs() @ w.double().abs())).all()
ref = xs[1].double().t() @ ys[1].double()
assert ((dw - ref).abs() <= 50 * 2.0 ** -23 * (xs[1].double().abs().t() @ ys[1].double().abs())).all()
assert torch.equal(torch.cat((q, k, v), 2), qkv)
assert torch.allclose(p, torch.full_like(p, -0.5), rtol=2.0 ** -20)    # 16 roundings
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
