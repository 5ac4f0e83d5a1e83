"""Host-side check of AdamW's clipping factor (no GPU): it may not lie in what
the step writes, at whatever end, for the single call and for a plan."""

import ctypes

import pytest

from newton_schulz_08_gb300 import muon
from tests.test_operators_host import L, adamw_call, adamw_desc, at  # noqa: F401


@pytest.mark.parametrize("where", [at(0), at(0, 2000), at(0, 3996), at(2), at(3, 3996), at(8, 996), at(9), at(10), at(10, 12), at(11, 8)])
def test_grad_scale_in_a_written_array_is_refused(L, where):  # noqa: F811
    descs = [adamw_desc(0), adamw_desc(1, bits=8)]  # 1000 elements: 4000 bytes, 1000 of codes, 16 of scales
    assert adamw_call(L, descs, scale=where) == muon.MUON_ERR_ALIASING
    plan, arr = ctypes.c_void_p(), (muon.adamw_tensor_desc * 2)(*descs)
    assert L.adamw_plan_create(arr, 2, ctypes.byref(plan)) == muon.MUON_OK
    assert L.adamw_plan_step(plan, 0.9, 0.95, 1e-8, 0, 1, 0, ctypes.c_void_p(where), None) == muon.MUON_ERR_ALIASING
    grads, kinds = (ctypes.c_void_p * 2)(at(20), at(21)), (ctypes.c_int32 * 2)(muon.MUON_F32, muon.MUON_F32)
    assert L.adamw_plan_set_grads(plan, grads, kinds) == muon.MUON_OK  # the same arrays are written
    assert L.adamw_plan_step(plan, 0.9, 0.95, 1e-8, 0, 1, 0, ctypes.c_void_p(where), None) == muon.MUON_ERR_ALIASING
    L.adamw_plan_destroy(plan)


@pytest.mark.parametrize("where", [at(0, 4000), at(0) - 4, at(1, 40), at(8, 1000), at(10, 16), at(20)])
def test_grad_scale_beside_the_written_arrays_is_not(L, where):  # noqa: F811
    """Past an array's end, before its beginning, in a gradient: the missing gradient, which is found later, is what is told."""
    empty = [adamw_desc(0), adamw_desc(1, bits=8, grad=0)]  # the missing gradient is found after the factor
    plan, arr = ctypes.c_void_p(), (muon.adamw_tensor_desc * 2)(*empty)
    assert L.adamw_plan_create(arr, 2, ctypes.byref(plan)) == muon.MUON_OK
    assert L.adamw_plan_step(plan, 0.9, 0.95, 1e-8, 0, 1, 0, ctypes.c_void_p(where), None) == muon.MUON_ERR_INVALID_ARG
    L.adamw_plan_destroy(plan)
