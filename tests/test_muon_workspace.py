"""The orthogonalisation's workspace: what it asks for where one workgroup does a
matrix (CPU), and that no path writes behind it (GPU)."""
import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs


@pytest.mark.parametrize("count,r,c", [(1, 1, 1), (1000, 64, 64), (48, 1024, 64), (3, 77, 333),
                                       (300, 128, 448)])
def test_a_matrix_of_one_workgroup_needs_its_low_half_alone(count, r, c):
    rp, cp = (r + 63) // 64 * 64, (c + 63) // 64 * 64
    need = zs.zero_orthogonalize_workspace_bytes(count, r, c)
    assert 2 * count * rp * cp <= need < 2 * count * rp * cp + 256


@pytest.mark.gpu
@pytest.mark.parametrize("count,r,c", [(1, 1, 1), (5, 64, 64), (2, 1024, 64), (3, 77, 333),
                                       (2, 128, 448), (1, 64, 2000), (2, 100, 1500), (3, 200, 130),
                                       (1, 700, 2300)])
def test_nothing_behind_the_workspace_is_written(count, r, c):
    g = torch.Generator(device="cuda")
    g.manual_seed(r)
    need = zs.zero_orthogonalize_workspace_bytes(count, r, c)
    buf = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    u = torch.randn(count, r, c, generator=g, device="cuda")
    o, p = (torch.empty(count, r, c, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    zs.zero_orthogonalize(u, o, workspace=buf[2048:2048 + need])
    zs.zero_orthogonalize(u, p)
    assert (buf[:2048] == 77).all() and (buf[2048 + need:] == 77).all()
    assert torch.equal(o, p) and torch.isfinite(o).all()
    with pytest.raises(ValueError):
        zs.zero_orthogonalize(u, o, workspace=buf[2048:2048 + need - 16])
