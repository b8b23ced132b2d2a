"""Refusals of the speculative step's entry points that need views of their
own, on the CPU: the host checks run and no kernel is launched."""
import ctypes

import pytest
import torch

from gated_deltanet_recurrent_sigmoid_b200 import binding, speculative as spec
from test_spec_abi import make_commit, make_maps, make_verify, refused

I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib(gdn_lib):
    return spec.load()


STATE = 128 * 128


@pytest.mark.parametrize("slots,heads,slot,head", [
    (2, 2, STATE, STATE),                # slot 0's head 1 is slot 1's head 0
    (5, 2, STATE, 4 * STATE),            # slot 4's head 0 is slot 0's head 1
    (3, 3, 2 * STATE, STATE),            # slot 0's head 2 is slot 1's head 0
    (2, 2, STATE + 4, STATE),            # in part
])
def test_commit_refuses_pools_whose_states_share_addresses(slots, heads, slot, head):
    pool = torch.zeros(64 * STATE).as_strided((slots, heads, 128, 128), (slot, head, 128, 1))
    refused(binding.ERR_SHAPE, lambda: make_commit(N=2, HV=heads, slots=slots), state_pool=pool)


@pytest.mark.parametrize("slots,heads,slot,head", [
    (5, 2, STATE, 5 * STATE),            # heads outside slots
    (3, 3, 3 * STATE, STATE),
    (3, 2, 2 * STATE + 8, STATE + 4),
    (1, 3, 0, STATE),                    # the stride of one entry does not matter
    (4, 1, STATE, 0),
])
def test_commit_takes_pools_whose_states_lie_apart(slots, heads, slot, head):
    pool = torch.zeros(64 * STATE).as_strided((slots, heads, 128, 128), (slot, head, 128, 1))
    fn, args = make_commit(N=2, HV=heads, slots=slots)
    with pytest.raises(ValueError):      # every check of the library passes; host tensors are refused by the binding
        fn(**{**args, "state_pool": pool})


@pytest.mark.parametrize("n,d,strides", [(3, 2, (2, 1)), (3, 2, (1, 2)), (3, 2, (3, 0)), (2, 2, (1, 1))])
def test_verify_refuses_outputs_that_share_addresses(n, d, strides):
    out = torch.zeros(32, dtype=I32).as_strided((n, d + 1), strides)
    refused(binding.ERR_SHAPE, lambda: make_verify(N=n, D=d), out_tokens=out)


def far_vector(n, place, dtype=3):
    """A descriptor of n entries at an address of its own; nothing reads it."""
    d = binding.GdnTensor()
    d.data, d.dtype, d.ndim = (place + 1) << 40, dtype, 1
    d.shape[0], d.stride[0] = n, 1
    return d


@pytest.mark.parametrize("n,status", [(2**31 - 2, binding.ERR_SHAPE), (2**31 - 1024, binding.ERR_SHAPE),
                                      (2**31 - 1025, binding.OK), (2**30, binding.OK), (0, binding.OK)])
def test_maps_refuses_more_requests_than_its_counters_hold(n, status):
    """The kernel counts requests in 32 bits, 1024 at a time."""
    call = spec.GdnStepMapsCall()
    names = ("lengths", "context", "slots", "cu_seqlens", "state_indices", "row_seq", "positions")
    descs = [far_vector(n + 1 if k == "cu_seqlens" else 64 if k in ("row_seq", "positions") else n, i) for i, k in enumerate(names)]
    for k, d in zip(names, descs):
        setattr(call, k, ctypes.pointer(d))
    call.flags = spec.CHECK_ONLY
    assert spec.load().gdn_step_maps(ctypes.byref(call)) == status
