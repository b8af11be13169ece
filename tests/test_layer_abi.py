"""Refusals of the layer's operators (linear products, head norm with rotary
positions, AdamW) on the host, before anything is launched: the C ABI with
fake device addresses that are never dereferenced, and the binding's checks
that need no GPU."""

import ctypes
import math

import pytest
import torch

from long_context_attention_seqattn_gb300 import binding, build

P = 0x10000          # aligned fake device address
MIS = 0x10004
INV = binding.SEQATTN_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def _call(f, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return f(*a.values())


FWD = dict(rows=16, k=64, n=128, x=P, ldx=64, w=P, bias=None, act=0, residual=None, ldr=0, z=None, ldz=0, y=P,
           ldy=128, stream=None)
DGRAD = dict(rows=16, k=64, n=128, g=P, ldg=128, w=P, act=0, z=None, ldz=0, residual=None, ldr=0, dx=P, lddx=64,
             stream=None)
WGRAD = dict(rows=16, k=64, n=128, x=P, ldx=64, g=P, ldg=128, dw=P, dbias=None, stream=None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=2 ** 31 - 512), dict(k=0), dict(k=60), dict(n=-8), dict(n=4), dict(act=5), dict(act=-1),
    dict(ldx=56), dict(ldx=65), dict(ldy=120), dict(x=None), dict(w=None), dict(y=None), dict(x=MIS), dict(y=MIS),
    dict(bias=MIS), dict(residual=P, ldr=64), dict(residual=MIS, ldr=128), dict(z=P, ldz=0), dict(z=MIS, ldz=128),
])
def test_linear_fwd_refuses(lib, kw):
    assert _call(lib.seqattn_linear_fwd, FWD, kw) == INV
    assert lib.seqattn_last_error()


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(k=12), dict(n=0), dict(act=9), dict(act=2), dict(act=2, z=P, ldz=56), dict(act=2, z=MIS, ldz=64),
    dict(ldg=64), dict(lddx=60), dict(g=None), dict(w=MIS), dict(dx=None), dict(residual=P, ldr=8),
])
def test_linear_dgrad_refuses(lib, kw):
    assert _call(lib.seqattn_linear_dgrad, DGRAD, kw) == INV


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(k=4), dict(n=20), dict(ldx=8), dict(ldg=100), dict(x=None), dict(g=MIS), dict(dw=None),
    dict(dw=MIS), dict(dbias=MIS),
])
def test_linear_wgrad_refuses(lib, kw):
    assert _call(lib.seqattn_linear_wgrad, WGRAD, kw) == INV


def test_linear_without_rows_is_a_no_op(lib):
    assert _call(lib.seqattn_linear_fwd, FWD, dict(rows=0, x=None, y=None)) == 0
    assert _call(lib.seqattn_linear_dgrad, DGRAD, dict(rows=0, act=1)) == INV      # its stride is still checked
    assert _call(lib.seqattn_linear_dgrad, DGRAD, dict(rows=0, g=None)) == 0
    assert _call(lib.seqattn_linear_wgrad, WGRAD, dict(rows=0, dw=None)) == 0


def _pb(**kw):
    base = dict(batch=1, num_q_heads=4, num_kv_heads=2, head_dim=128, seq_capacity=1024, dtype=0)
    base.update(kw)
    return binding.Problem(**base)


def _plan(**kw):
    plan = binding.rope_plan([1.0 / (i + 1) for i in range(64)])
    for name, v in kw.items():
        setattr(plan, name, v)
    return plan


RFWD = dict(pb=_pb(), q_start=0, q_len=16, q_in=P, ld_q=512, k_in=P, ld_k=256, v_in=P, ld_v=256, gamma_q=P, gamma_k=P,
            eps=1e-6, plan=_plan(), positions=None, q=P, k_cache=P, v_cache=P, stream=None)
RBWD = dict(pb=_pb(), q_start=0, q_len=16, q_in=P, ld_q=512, k_in=P, ld_k=256, gamma_q=P, gamma_k=P, eps=1e-6,
            plan=_plan(), positions=None, dq=P, dk=P, dv=P, dq_in=P, ld_dq=512, dk_in=P, ld_dk=256, dv_in=P,
            ld_dv=256, dgamma_q=P, dgamma_k=P, workspace=P, bytes=1 << 20, stream=None)
ROPE_BAD = [
    dict(pb=None), dict(pb=_pb(head_dim=96)), dict(pb=_pb(num_q_heads=3)), dict(q_start=-1), dict(q_len=-1),
    dict(q_start=1020), dict(gamma_q=None), dict(gamma_k=None), dict(gamma_q=MIS), dict(eps=-1.0),
    dict(eps=math.nan), dict(eps=math.inf), dict(positions=MIS), dict(q_in=None), dict(k_in=MIS), dict(ld_q=504),
    dict(ld_k=257), dict(plan=_plan(rot_dim=8)), dict(plan=_plan(rot_dim=24)), dict(plan=_plan(rot_dim=256)),
    dict(plan=_plan(axes=0)), dict(plan=_plan(axes=65)), dict(plan=_plan(interleaved=2)), dict(plan=_plan(reserved=1)),
    dict(plan=binding.RopePlan(128, 1, 0, 0, (0,) * 64, (1,) * 64)),       # an axis that does not exist
]


@pytest.mark.parametrize("kw", ROPE_BAD + [dict(v_in=None), dict(v_cache=None), dict(ld_v=8), dict(v_in=MIS),
                                           dict(q=None), dict(k_cache=MIS), dict(v_cache=MIS)])
def test_norm_rope_fwd_refuses(lib, kw):
    assert _call(lib.seqattn_qk_norm_rope_fwd, RFWD, kw) == INV


@pytest.mark.parametrize("kw", ROPE_BAD + [dict(dv=None), dict(dv_in=None), dict(ld_dv=0), dict(ld_dq=8),
                                           dict(ld_dk=260), dict(dq=None), dict(dk=MIS), dict(dq_in=None),
                                           dict(dgamma_q=None), dict(dgamma_k=MIS), dict(workspace=None),
                                           dict(bytes=1024)])
def test_norm_rope_bwd_refuses(lib, kw):
    assert _call(lib.seqattn_qk_norm_rope_bwd, RBWD, kw) == INV


def test_norm_rope_without_rows_is_a_no_op(lib):
    assert _call(lib.seqattn_qk_norm_rope_fwd, RFWD, dict(q_len=0, q_in=None, q=None)) == 0
    assert _call(lib.seqattn_qk_norm_rope_bwd, RBWD, dict(q_len=0, dq=None, workspace=None)) == 0
    assert lib.seqattn_qk_norm_rope_bwd_workspace_size(_pb(head_dim=96)) == 0
    assert lib.seqattn_qk_norm_rope_bwd_workspace_size(_pb()) > 0


def _tensor(**kw):
    base = dict(param=P, lowp=None, grad=P, m=P, v=P, m_scale=P, v_scale=P, n=8, weight_decay=0.0, grad_bf16=0)
    base.update(kw)
    return binding.AdamwTensor(**base)


def _params(**kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, grad_scale=1.0, step=1)
    base.update(kw)
    return binding.AdamwParams(**base)


@pytest.mark.parametrize("tensor,params,bits", [
    (dict(n=-1), {}, 32), (dict(n=2 ** 41), {}, 32), (dict(param=None), {}, 32), (dict(grad=MIS), {}, 32),
    (dict(m=None), {}, 32), (dict(v=MIS), {}, 8), (dict(lowp=MIS), {}, 32), (dict(m_scale=None), {}, 8),
    (dict(v_scale=0x10002), {}, 8), (dict(weight_decay=math.nan), {}, 32), (dict(grad_bf16=2), {}, 32),
    ({}, dict(beta1=1.0), 32), ({}, dict(beta2=-0.1), 32), ({}, dict(eps=-1.0), 32), ({}, dict(lr=math.inf), 32),
    ({}, dict(grad_scale=math.nan), 32), ({}, dict(step=0), 32), ({}, {}, 16), ({}, dict(lr_dev=0x10002), 32),
    ({}, dict(step_dev=MIS), 32),
])
def test_adamw_refuses(lib, tensor, params, bits):
    list_ = (binding.AdamwTensor * 2)(_tensor(), _tensor(**tensor))
    assert lib.seqattn_adamw_step(list_, 2, bits, _params(**params), None) == INV


def test_adamw_without_work_is_a_no_op(lib):
    assert lib.seqattn_adamw_step(None, 0, 32, _params(), None) == 0
    assert lib.seqattn_adamw_step(None, 1, 32, _params(), None) == INV
    assert lib.seqattn_adamw_step(None, -1, 32, _params(), None) == INV
    empty = (binding.AdamwTensor * 1)(_tensor(n=0, param=None))
    assert lib.seqattn_adamw_step(empty, 1, 8, _params(), None) == 0


def _message(lib):
    return lib.seqattn_last_error().decode()


A = [0x100000 * (i + 2) for i in range(16)]      # fake addresses, all different


@pytest.mark.parametrize("kw,words", [
    (dict(y=A[0]), "y is the memory of x"), (dict(y=A[1]), "y is the memory of w"),
    (dict(z=A[0], ldz=128), "z is the memory of x"), (dict(z=A[2], ldz=128), "y and z"),
    (dict(residual=A[3], ldr=128, z=A[3], ldz=128), "z is the memory of residual"),
    (dict(residual=A[2], ldr=256), "another row stride"),
])
def test_linear_fwd_refuses_shared_memory(lib, kw, words):
    assert _call(lib.seqattn_linear_fwd, dict(FWD, x=A[0], w=A[1], y=A[2]), kw) == INV
    assert words in _message(lib)


@pytest.mark.parametrize("kw,words", [
    (dict(dx=A[0]), "dx is the memory of g"), (dict(act=2, z=A[2], ldz=64), "dx is the memory of z"),
    (dict(residual=A[2], ldr=128), "another row stride"),
])
def test_linear_dgrad_refuses_shared_memory(lib, kw, words):
    assert _call(lib.seqattn_linear_dgrad, dict(DGRAD, g=A[0], w=A[1], dx=A[2]), kw) == INV
    assert words in _message(lib)


@pytest.mark.parametrize("kw,words", [(dict(dw=A[0]), "dw is the memory of x"), (dict(dbias=A[2]), "dw and dbias")])
def test_linear_wgrad_refuses_shared_memory(lib, kw, words):
    assert _call(lib.seqattn_linear_wgrad, dict(WGRAD, x=A[0], g=A[1], dw=A[2]), kw) == INV
    assert words in _message(lib)


RFWD_APART = dict(RFWD, q_in=A[0], k_in=A[1], v_in=A[2], gamma_q=A[3], gamma_k=A[3], q=A[5], k_cache=A[6],
                  v_cache=A[7])
RBWD_APART = dict(RBWD, q_in=A[0], k_in=A[1], gamma_q=A[2], gamma_k=A[2], dq=A[4], dk=A[5], dv=A[6], dq_in=A[7],
                  dk_in=A[8], dv_in=A[9], dgamma_q=A[10], dgamma_k=A[11], workspace=A[12])


@pytest.mark.parametrize("kw,words", [
    (dict(q=A[0]), "q is the memory of q_in"), (dict(k_cache=A[1]), "k_cache is the memory of k_in"),
    (dict(k_cache=A[7]), "k_cache and v_cache"),
])
def test_norm_rope_fwd_refuses_shared_memory(lib, kw, words):
    assert _call(lib.seqattn_qk_norm_rope_fwd, RFWD_APART, kw) == INV
    assert words in _message(lib)


@pytest.mark.parametrize("kw,words", [
    (dict(dgamma_k=A[10]), "dgamma_q and dgamma_k"), (dict(dq_in=A[0]), "dq_in is the memory of q_in"),
    (dict(dk_in=A[9]), "dk_in and dv_in"), (dict(dq_in=A[4]), "dq_in is the memory of dq"),
    (dict(workspace=A[10]), "dgamma_q and workspace"),
])
def test_norm_rope_bwd_refuses_shared_memory(lib, kw, words):
    assert _call(lib.seqattn_qk_norm_rope_bwd, RBWD_APART, kw) == INV
    assert words in _message(lib)


@pytest.mark.parametrize("kw", [dict(q_start=2 ** 63 - 1), dict(q_len=2 ** 63 - 1, q_start=1),
                                dict(q_start=2 ** 63 - 1, q_len=2 ** 63 - 1),
                                dict(pb=_pb(num_q_heads=2 ** 30, num_kv_heads=1), ld_q=2 ** 36)])
def test_norm_rope_refuses_sizes_past_their_integers(lib, kw):
    assert _call(lib.seqattn_qk_norm_rope_fwd, RFWD_APART, kw) == INV
    assert _call(lib.seqattn_qk_norm_rope_bwd, RBWD_APART, {k: v for k, v in kw.items()}) == INV


@pytest.mark.parametrize("q_start,q_len", [(2 ** 63 - 1, 1), (1, 2 ** 63 - 1), (2 ** 63 - 1, 2 ** 63 - 1), (1009, 16)])
def test_chunk_calls_refuse_rows_past_the_cache(lib, q_start, q_len):
    pb = _pb()
    assert lib.seqattn_chunk_fwd(pb, q_start, q_len, 0, 0.1, P, P, P, P, P, None) == INV
    assert "exceeds seq_capacity" in _message(lib)
    assert lib.seqattn_chunk_bwd(pb, q_start, q_len, 0, 0.1, P, P, P, P, P, P, P, P, P, P, 2 ** 62, None) == INV
    assert "exceeds seq_capacity" in _message(lib)


# ------------------------------------------------------------------ the binding's own checks

@pytest.mark.parametrize("outs,ins,want", [
    ([(100, 10), (110, 10)], [(120, 5), (122, 5)], False),       # side by side; inputs may overlap
    ([(100, 10), (109, 10)], [], True), ([(100, 10), (100, 10)], [], True), ([(100, 50), (120, 5)], [], True),
    ([(100, 10)], [(95, 6)], True), ([(100, 10)], [(90, 40)], True), ([(100, 10)], [(90, 10)], False),
    ([(100, 10)], [(104, 2)], True), ([(100, 10)], [(90, 40), (200, 5)], True), ([(0, 0), (0, 0)], [(0, 0)], False),
    ([(100, 10), (105, 0)], [], False),
])
def test_ranges_that_collide(outs, ins, want):
    assert binding._collide(outs, ins) is want


def test_rope_plan_turns():
    """A frequency f is kept as round(f / 2 pi * 2^64) modulo a turn."""
    plan = binding.rope_plan([2 * math.pi * 0.25, 1.0, -1.0] + [0.0] * 5, [0, 1, 2] + [0] * 5, interleaved=True)
    assert (plan.rot_dim, plan.axes, plan.interleaved) == (16, 3, 1)
    assert abs(plan.turns[0] / 2 ** 64 - 0.25) < 2 ** -52        # the argument itself is rounded to 53 bits
    assert (plan.turns[1] + plan.turns[2]) % 2 ** 64 == 0        # -f is the turn's complement
    # a whole position's angle: position * turns mod 2^64 against float64 of a reduced argument
    pos = 1_000_003
    turn = (pos * plan.turns[1] % 2 ** 64) / 2 ** 64
    assert abs(math.cos(2 * math.pi * turn) - math.cos(float(pos))) < 1e-9
    assert list(plan.axis[:3]) == [0, 1, 2]


@pytest.mark.parametrize("args", [([1.0] * 7,), ([1.0] * 72,), ([],), ([math.inf] + [1.0] * 7,),
                                  ([1.0] * 8, [0] * 7), ([1.0] * 8, [64] * 8), ([1.0] * 8, [-1] * 8)])
def test_rope_plan_refuses(args):
    with pytest.raises(ValueError):
        binding.rope_plan(*args)


def test_binding_refuses_host_tensors_and_bad_choices():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((64, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.linear_fwd(x, w, x)
    with pytest.raises(ValueError, match="CUDA"):
        binding.linear_dgrad(x, w, x)
    with pytest.raises(ValueError, match="CUDA"):
        binding.linear_wgrad(x, x, torch.zeros((64, 64)))
    with pytest.raises(ValueError, match="activation"):
        binding._act_code("swish2")
    p = [torch.zeros(8)]
    with pytest.raises(ValueError, match="CUDA"):
        binding.AdamW(p, p)
    with pytest.raises(ValueError, match="state_bits"):
        binding.AdamW(p, p, state_bits=16)
    with pytest.raises(ValueError, match="all be given"):
        binding.AdamW(p, p, m=p)
    with pytest.raises(ValueError, match="entries"):
        binding.AdamW(p, [])


def test_structures_mirror_the_header(lib):
    assert ctypes.sizeof(binding.AdamwTensor) == 72
    assert ctypes.sizeof(binding.RopePlan) == 16 + 64 * 8 + 64
    assert ctypes.sizeof(binding.AdamwParams) == 72
