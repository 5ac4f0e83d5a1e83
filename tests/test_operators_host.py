"""Host-side checks of adamw_step, token_logprobs and balance_loss (no GPU):
sizes, no-ops and every refusal, with fake device addresses that no call gets
as far as touching; and the binding's own checks."""

import ctypes

import pytest
import torch

from newton_schulz_08_gb300 import muon

A = 0x7F0000000000
STEP = 0x10000000


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(muon.LIB_PATH):
        from newton_schulz_08_gb300 import build
        build.build()
    return muon.lib()


def at(k, off=0):
    return A + k * STEP + off


# ------------------------------------------------------------------- adamw
def adamw_desc(k=0, numel=1000, bits=32, **kw):
    d = dict(param=at(6 * k), grad=at(6 * k + 1), exp_avg=at(6 * k + 2), exp_avg_sq=at(6 * k + 3),
             exp_avg_scale=at(6 * k + 4) if bits == 8 else 0, exp_avg_sq_scale=at(6 * k + 5) if bits == 8 else 0,
             numel=numel, lr=1e-3, weight_decay=0.1, param_dtype=muon.MUON_F32, grad_dtype=muon.MUON_BF16,
             state_bits=bits, reserved=0)
    d.update(kw)
    return muon.adamw_tensor_desc(*[d[f[0]] for f in muon.adamw_tensor_desc._fields_])


def adamw_call(L, descs, n=None, beta1=0.9, beta2=0.95, eps=1e-8, step=1, scale=None):
    arr = (muon.adamw_tensor_desc * max(len(descs), 1))(*descs)
    return L.adamw_step(arr, len(descs) if n is None else n, beta1, beta2, eps, 0, step, 0,
                        ctypes.c_void_p(scale), None)


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kw,code", [
    (dict(param=0), "INVALID_ARG"), (dict(grad=0), "INVALID_ARG"), (dict(exp_avg=0), "INVALID_ARG"),
    (dict(exp_avg_sq=0), "INVALID_ARG"), (dict(numel=-1), "INVALID_ARG"), (dict(param_dtype=2), "INVALID_ARG"),
    (dict(grad_dtype=-1), "INVALID_ARG"), (dict(state_bits=16), "INVALID_ARG"), (dict(reserved=1), "INVALID_ARG"),
    (dict(lr=INF), "INVALID_ARG"), (dict(weight_decay=NAN), "INVALID_ARG"),
    (dict(exp_avg_scale=at(4)), "INVALID_ARG"),                        # scales with 32-bit moments
    (dict(bits=8, exp_avg_sq_scale=0), "INVALID_ARG"),                 # and none with 8-bit ones
    (dict(numel=(1 << 40) + 1), "TOO_LARGE"),
    (dict(param=at(0, 2)), "MISALIGNED"), (dict(grad=at(1, 1)), "MISALIGNED"), (dict(exp_avg=at(2, 1)), "MISALIGNED"),
    (dict(bits=8, exp_avg_scale=at(4, 2)), "MISALIGNED"),
    (dict(grad=at(0, 64)), "ALIASING"), (dict(exp_avg_sq=at(2, 3996)), "ALIASING"),
    (dict(bits=8, exp_avg_sq_scale=at(4, 12)), "ALIASING"),
])
def test_adamw_refuses(L, kw, code):
    assert adamw_call(L, [adamw_desc(1), adamw_desc(0, **kw)]) == getattr(muon, "MUON_ERR_" + code)


@pytest.mark.parametrize("kw", [dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1e-8), dict(eps=INF),
                                dict(n=-1), dict(beta1=NAN)])
def test_adamw_refuses_scalars(L, kw):
    assert adamw_call(L, [adamw_desc()], **kw) == muon.MUON_ERR_INVALID_ARG


def test_adamw_refuses_misaligned_grad_scale_and_null_list(L):
    assert adamw_call(L, [adamw_desc()], scale=at(9, 2)) == muon.MUON_ERR_MISALIGNED
    assert L.adamw_step(None, 3, 0.9, 0.95, 1e-8, 0, 1, 0, None, None) == muon.MUON_ERR_INVALID_ARG


def test_adamw_nothing_to_do(L):
    assert adamw_call(L, []) == muon.MUON_OK
    # tensors without elements need no pointers
    assert adamw_call(L, [adamw_desc(numel=0, param=0, grad=0, exp_avg=0, exp_avg_sq=0)]) == muon.MUON_OK


def test_adamw_plan_checks(L):
    plan = ctypes.c_void_p()
    arr = (muon.adamw_tensor_desc * 2)(adamw_desc(0, grad=0), adamw_desc(1))
    assert L.adamw_plan_create(arr, 2, None) == muon.MUON_ERR_INVALID_ARG
    assert L.adamw_plan_create(arr, -1, ctypes.byref(plan)) == muon.MUON_ERR_INVALID_ARG and not plan
    assert L.adamw_plan_create(arr, 2, ctypes.byref(plan)) == muon.MUON_OK and plan
    step = lambda: L.adamw_plan_step(plan, 0.9, 0.95, 1e-8, 0, 1, 0, None, None)  # noqa: E731
    assert step() == muon.MUON_ERR_INVALID_ARG  # a gradient is missing
    ptr, kind = (ctypes.c_void_p * 2), (ctypes.c_int32 * 2)(muon.MUON_F32, muon.MUON_BF16)
    assert L.adamw_plan_set_grads(plan, ptr(at(1), 0), kind) == muon.MUON_ERR_INVALID_ARG
    assert L.adamw_plan_set_grads(plan, ptr(at(0), at(7)), kind) == muon.MUON_ERR_ALIASING
    assert L.adamw_plan_set_grads(plan, ptr(at(1, 2), at(7)), kind) == muon.MUON_ERR_MISALIGNED
    assert step() == muon.MUON_ERR_INVALID_ARG  # unchanged by the refusals
    double = ctypes.c_double * 2
    assert L.adamw_plan_set_rates(plan, double(1.0, INF), double(0, 0)) == muon.MUON_ERR_INVALID_ARG
    assert L.adamw_plan_set_rates(plan, double(1.0, 2.0), double(0, 0)) == muon.MUON_OK
    L.adamw_plan_destroy(plan)
    L.adamw_plan_destroy(None)
    assert L.adamw_plan_step(None, 0.9, 0.95, 1e-8, 0, 1, 0, None, None) == muon.MUON_ERR_INVALID_ARG


def test_adamw_many_tensors_are_checked_against_each_other(L):
    """600 disjoint tensors, then one whose moment lies in the middle of another's gradient."""
    descs = [adamw_desc(k, numel=256) for k in range(600)]
    plan = ctypes.c_void_p()
    arr = (muon.adamw_tensor_desc * 600)(*descs)
    assert L.adamw_plan_create(arr, 600, ctypes.byref(plan)) == muon.MUON_OK
    L.adamw_plan_destroy(plan)
    arr[431] = adamw_desc(431, numel=256, exp_avg=at(6 * 17 + 1, 64))
    assert L.adamw_plan_create(arr, 600, ctypes.byref(plan)) == muon.MUON_ERR_ALIASING
    arr[431] = adamw_desc(431, numel=256, grad=at(6 * 17 + 1))  # shared gradients are fine
    assert L.adamw_plan_create(arr, 600, ctypes.byref(plan)) == muon.MUON_OK
    L.adamw_plan_destroy(plan)


# ---------------------------------------------------------------- logprobs
def score_call(L, x=at(0), dtype=muon.MUON_BF16, rows=4, vocab=100, stride=100, y=at(1), scale=1.0, top=3, lp=at(2),
               lse=at(3), h=at(4), tlp=at(5), ids=at(6)):
    v = ctypes.c_void_p
    return L.token_logprobs(v(x), dtype, rows, vocab, stride, v(y), scale, top, v(lp), v(lse), v(h), v(tlp), v(ids), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), "INVALID_ARG"), (dict(y=0), "INVALID_ARG"), (dict(lp=0), "INVALID_ARG"), (dict(lse=0), "INVALID_ARG"),
    (dict(h=0), "INVALID_ARG"), (dict(tlp=0), "INVALID_ARG"), (dict(ids=0), "INVALID_ARG"),
    (dict(dtype=2), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"), (dict(vocab=0), "INVALID_ARG"),
    (dict(stride=99), "INVALID_ARG"), (dict(scale=0.0), "INVALID_ARG"), (dict(scale=NAN), "INVALID_ARG"),
    (dict(scale=2e6), "INVALID_ARG"), (dict(top=33), "INVALID_ARG"), (dict(top=-1), "INVALID_ARG"),
    (dict(vocab=2, top=3), "INVALID_ARG"),
    (dict(vocab=(1 << 30) + 1, stride=1 << 31), "TOO_LARGE"), (dict(rows=1 << 31), "TOO_LARGE"),
    (dict(stride=(1 << 32) + 1), "TOO_LARGE"),
    (dict(x=at(0, 1)), "MISALIGNED"), (dict(dtype=muon.MUON_F32, x=at(0, 2)), "MISALIGNED"),
    (dict(y=at(1, 4)), "MISALIGNED"), (dict(ids=at(6, 4)), "MISALIGNED"), (dict(lse=at(3, 2)), "MISALIGNED"),
    (dict(lp=at(0, 400)), "ALIASING"), (dict(lse=at(2, 12)), "ALIASING"), (dict(ids=at(1, 24)), "ALIASING"),
])
def test_logprobs_refuses(L, kw, code):
    assert score_call(L, **kw) == getattr(muon, "MUON_ERR_" + code)


def grad_call(L, x=at(0), dtype=muon.MUON_BF16, rows=4, vocab=100, stride=100, y=at(1), scale=1.0, lse=at(3), h=at(4),
              gl=at(5), ge=at(6), grad=at(7), gs=100):
    v = ctypes.c_void_p
    return L.token_logprobs_backward(v(x), dtype, rows, vocab, stride, v(y), scale, v(lse), v(h), v(gl), v(ge), v(grad),
                                     gs, None)


def loss_call(L, x=at(0), dtype=muon.MUON_BF16, rows=4, vocab=100, stride=100, y=at(1), scale=1.0, top=2, gl=at(5),
              ge=at(6), grad=at(7), gs=100, lse=at(3)):
    v = ctypes.c_void_p
    return L.token_logprobs_loss(v(x), dtype, rows, vocab, stride, v(y), scale, top, v(gl), v(ge), v(at(2)), v(lse),
                                 v(at(4)), v(at(8)), v(at(9)), v(grad), gs, None)


@pytest.mark.parametrize("call", [grad_call, loss_call])
@pytest.mark.parametrize("kw,code", [
    (dict(gl=0), "INVALID_ARG"), (dict(grad=0), "INVALID_ARG"), (dict(lse=0), "INVALID_ARG"), (dict(gs=99), "INVALID_ARG"),
    (dict(scale=-1.0), "INVALID_ARG"), (dict(grad=at(7, 1)), "MISALIGNED"), (dict(gl=at(5, 2)), "MISALIGNED"),
    (dict(grad=at(0), gs=104), "ALIASING"), (dict(grad=at(0, 2)), "ALIASING"), (dict(grad=at(5, 8)), "ALIASING"),
    (dict(gs=(1 << 32) + 1), "TOO_LARGE"),
])
def test_logprobs_gradient_refuses(L, call, kw, code):
    assert call(L, **kw) == getattr(muon, "MUON_ERR_" + code)


def test_logprobs_gradient_of_entropy_needs_it(L):
    assert grad_call(L, h=0) == muon.MUON_ERR_INVALID_ARG


def test_logprobs_no_rows(L):
    assert score_call(L, rows=0, x=0, y=0, lp=0) == muon.MUON_OK
    assert grad_call(L, rows=0, x=0, grad=0) == muon.MUON_OK
    assert loss_call(L, rows=0) == muon.MUON_OK


# ----------------------------------------------------------------- balance
def bal_call(L, x=at(0), dtype=muon.MUON_F32, tokens=64, experts=8, stride=8, ids=at(1), top=2, mask=0, groups=4,
             stats=at(2), counts=at(3), n=at(4), mean=at(5), weights=at(6), ws=at(7), wsb=1 << 30):
    v = ctypes.c_void_p
    return L.balance_loss(v(x), dtype, tokens, experts, stride, v(ids), top, v(mask), groups, v(stats), v(counts), v(n),
                          v(mean), v(weights), v(ws), wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), "INVALID_ARG"), (dict(ids=0), "INVALID_ARG"), (dict(stats=0), "INVALID_ARG"), (dict(ws=0), "INVALID_ARG"),
    (dict(weights=0), "INVALID_ARG"), (dict(dtype=5), "INVALID_ARG"), (dict(tokens=-4), "INVALID_ARG"),
    (dict(experts=0), "INVALID_ARG"), (dict(experts=1025, stride=1025), "INVALID_ARG"), (dict(stride=7), "INVALID_ARG"),
    (dict(top=0), "INVALID_ARG"), (dict(top=9), "INVALID_ARG"), (dict(groups=0), "INVALID_ARG"),
    (dict(groups=5), "INVALID_ARG"), (dict(tokens=1 << 31), "TOO_LARGE"), (dict(tokens=1 << 30), "TOO_LARGE"),
    (dict(x=at(0, 2)), "MISALIGNED"), (dict(ids=at(1, 4)), "MISALIGNED"), (dict(ws=at(7, 128)), "MISALIGNED"),
    (dict(stats=at(2, 1)), "MISALIGNED"), (dict(wsb=256), "WORKSPACE_TOO_SMALL"),
    (dict(stats=at(0, 64)), "ALIASING"), (dict(weights=at(5, 64)), "ALIASING"), (dict(mask=at(7, 32)), "ALIASING"),
])
def test_balance_refuses(L, kw, code):
    assert bal_call(L, **kw) == getattr(muon, "MUON_ERR_" + code)


def balg_call(L, x=at(0), tokens=64, experts=8, stride=8, mask=0, groups=4, stats=at(2), weights=at(6), gb=at(3), gz=at(4),
              grad=at(8), gs=8):
    v = ctypes.c_void_p
    return L.balance_loss_backward(v(x), muon.MUON_F32, tokens, experts, stride, v(mask), groups, v(stats), v(weights),
                                   v(gb), v(gz), v(grad), gs, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), "INVALID_ARG"), (dict(gb=0), "INVALID_ARG"), (dict(grad=0), "INVALID_ARG"), (dict(gs=7), "INVALID_ARG"),
    (dict(groups=3), "INVALID_ARG"), (dict(grad=at(8, 2)), "MISALIGNED"), (dict(gz=at(4, 2)), "MISALIGNED"),
    (dict(grad=at(0), gs=9), "ALIASING"), (dict(grad=at(6, 64)), "ALIASING"), (dict(mask=at(8)), "ALIASING"),
])
def test_balance_gradient_refuses(L, kw, code):
    assert balg_call(L, **kw) == getattr(muon, "MUON_ERR_" + code)


def test_balance_sizes(L):
    assert muon.balance_loss_workspace_size(-1, 8, 1) == 0 and muon.balance_loss_workspace_size(8, 2000, 1) == 0
    assert muon.balance_loss_workspace_size(10, 8, 3) == 0
    assert muon.balance_loss_workspace_size(0, 8, 1) > 0
    assert 0 < muon.balance_loss_workspace_size(64, 8, 1) <= muon.balance_loss_workspace_size(1 << 20, 8, 1) < 1 << 20
    assert balg_call(L, tokens=0, x=0, grad=0) == muon.MUON_OK


# ----------------------------------------------------------------- binding
def test_binding_refuses_bad_tensors():
    x, y = torch.zeros((4, 8)), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        muon.token_logprobs(x, y)                        # not CUDA tensors
    with pytest.raises(ValueError):
        muon.token_logprobs(x.t(), y)                    # columns are not contiguous
    with pytest.raises(ValueError):
        muon.token_logprobs(x[0], y)                     # not 2-D
    with pytest.raises(ValueError):
        muon.token_logprobs(x[:1].expand(4, 8), y)       # rows overlap
    with pytest.raises(ValueError):
        muon.token_logprobs_backward(x, y, y.float(), y.float(), grad_entropy=y.float())  # needs entropy
    with pytest.raises(ValueError):
        muon.token_logprobs_backward(x, y, y.float(), y.float(), out=torch.zeros((4, 9)))
    with pytest.raises(ValueError):
        muon.balance_loss(x, y)                          # ids must be tokens x top
    with pytest.raises(ValueError):
        muon.balance_loss(x, torch.zeros((4, 1), dtype=torch.int32))
    with pytest.raises(ValueError):
        muon.AdamW([])


def test_binding_adamw_checks():
    p = torch.zeros(300)
    s32, s8 = muon.adamw_state(p), muon.adamw_state(p, 8)
    assert [t.dtype for t in s8] == [torch.float8_e4m3fn, torch.float32, torch.float8_e5m2, torch.float32]
    assert s8[1].numel() == 2 and all(bool((v == 0).all()) for v in muon.adamw_state_values(s8))
    with pytest.raises(ValueError):
        muon.adamw_state(p, 4)
    for bad in (dict(states=[s32, s32]), dict(states=[s32[:1]]), dict(states=[(s32[0], s32[1].half())]),
                dict(states=[(s8[0], s8[1][:1], s8[2], s8[3])]), dict(grads=[p[:5]]), dict(lr=[1e-3, 1e-3]),
                dict(grads=[torch.zeros(600)[::2]])):
        kw = dict(grads=[p], states=[s32], lr=1e-3)
        kw.update(bad)
        with pytest.raises(ValueError):
            muon.adamw_step([p], kw["grads"], kw["states"], 1, lr=kw["lr"])
    with pytest.raises(ValueError):
        muon.adamw_step([p], [p], [s32], 1)              # not CUDA tensors
    muon.adamw_step([], [], [], 1)
