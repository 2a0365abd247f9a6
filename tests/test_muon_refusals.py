"""Parameters of the Muon step that only fail once they are fp32 values, and
reserved ones, on the CPU (refused before a launch; run only where no GPU is
visible)."""
import ctypes

import pytest

from tests.test_lib_host import cpu_only
from tests.test_muon_host import EINVAL, status
from zero_sharded_mixed_flatten_amd import _muon


@cpu_only
@pytest.mark.parametrize("op", ["upd", "upd_dc"])
@pytest.mark.parametrize("scale", [1e39, -1e39, 1e300, 3.4028236e38])
def test_an_update_scale_beyond_fp32_is_refused(op, scale):
    assert status(op, scale=scale) == EINVAL


@cpu_only
@pytest.mark.parametrize("reserved", [1, -1, 1 << 30])
def test_a_reserved_field_that_is_not_zero_is_refused(reserved):
    assert status("orth", ns=ctypes.byref(_muon._NsParams(5, reserved, 1e-7, None))) == EINVAL
