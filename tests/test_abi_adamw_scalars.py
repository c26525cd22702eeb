"""The AdamW step's numbers on the device have to be aligned as their types: refused on the
host, on the CPU (the call's tensor is refused too, so that no kernel is launched)."""
import ctypes

import pytest

from sparse_expert_routing_amd import _lib

P = 0x1000  # an address that no call gets to read


@pytest.mark.parametrize("name,off", [("grad_scale", 1), ("grad_scale", 2), ("lr_ptr", 2), ("lr_ptr", 3), ("step_ptr", 4), ("step_ptr", 1)])
def test_misaligned_numbers(name, off):
    def status(**kw):
        rule = _lib.AdamW(1e-3, 0.9, 0.999, 1e-8, 0.1, 1, 0, None, None, None)
        for n, v in kw.items():
            setattr(rule, n, v)
        far = _lib.AdamWTensor(P, P, P, P, None, None, None, 1 << 35, 0, 0, 32)  # more elements than a call takes
        return _lib.load().moe_adamw(ctypes.byref(rule), ctypes.byref(far), 1, None)

    assert status(**{name: P}) == _lib.MOE_ENOTSUP and status(**{name: P + off}) == _lib.MOE_EINVAL
