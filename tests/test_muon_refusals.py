"""Parameters of the Muon step that only fail once they are fp32 values, on the
CPU (refused before a launch; run only where no GPU is visible)."""
import pytest

from tests.test_lib_host import cpu_only
from tests.test_muon_host import EINVAL, status


@cpu_only
@pytest.mark.parametrize("op", ["upd", "upd_dc"])
@pytest.mark.parametrize("scale", [1e39, -1e39, 1e300, 3.4028236e38])
def test_an_update_scale_beyond_fp32_is_refused(op, scale):
    assert status(op, scale=scale) == EINVAL
