"""Further host-side checks of the many-tensor entry points: what they refuse
and what their sizes count, before anything is launched (no GPU needed)."""
import numpy as np
import pytest

import dimuon_optimizer_b200 as dm
from oracle import adamw_oracle as ao
from test_many_host import fake_grad, fake_tensor


def test_an_eps_the_kernels_cannot_divide_by_is_refused():
    """Subnormal ones and those whose reciprocal is subnormal; 0 is allowed."""
    for eps in (0.0, 2.0 ** -126, 1e-30, 1e-8, 2.0 ** 125):
        assert dm.dm_adamw_workspace_size([fake_tensor()], dm.dm_adamw_default_hparams(eps=eps))
    for eps in (1e-45, 1e-40, 2.0 ** -126 - 2.0 ** -149, 2.0 ** 125 * (1 + 2.0 ** -23), 3e38):
        hp = dm.dm_adamw_default_hparams(eps=eps)
        with pytest.raises(dm.DimuonError, match="invalid argument"):
            dm.dm_adamw_workspace_size([fake_tensor()], hp)
        # a step that were to run would find no workspace
        assert dm.dm_adamw_step([fake_tensor()], hp, (0, 0), stream=0) == dm.DM_ERR_INVALID_ARG


def test_the_oracle_holds_second_moments_at_the_largest_code():
    inf, nan, top = np.inf, np.nan, ao.LARGEST
    m = np.array([1.0, 1.0, inf, nan, nan, 1.0, 1.0])
    v = np.array([inf, 3.4e38, inf, inf, nan, nan, top])
    np.testing.assert_array_equal(ao.hold(m, v), [top, top, inf, inf, nan, nan, top])
    _, _, c2, s2 = ao.pack_moments(m[:2], v[:2], 1, 1, 0)
    assert (c2 == 123).all() and s2[0] == 2.0 ** 112 and ao.unpack(c2, s2, ao.E5M2)[0] == top
    # the next larger number of the format at that scale is none of fp32
    assert 65536.0 * 2.0 ** 112 > float(np.finfo(np.float32).max)


def test_tile_numbers_of_a_norm_launch_stay_within_32_bits():
    """A CTA of the norm pass goes from tile to tile in steps of the grid (1184
    at most), up to one step past the last: a launch's tiles end that far below 2^31.
    (One gradient may be listed often, so lists longer than the memory are calls.)"""
    tile, grid = 256 * 16 * 4, 1184
    full = (1 << 40) // tile + 1  # tiles of the longest tensor, at any offset
    rest = (1 << 31) - 31 * full
    header = dm.dm_grad_clip_workspace_size([])

    def launches(total):
        ts = [fake_grad(numel=1 << 40)] * 31 + [fake_grad(numel=(total - 31 * full) * tile - 15)]
        return (dm.dm_grad_clip_workspace_size(ts) - header) // (8 * grid)

    assert 0 < rest < full
    assert launches((1 << 31) - 1 - grid) == 1
    for total in ((1 << 31) - grid, (1 << 31) - 1):
        assert launches(total) == 2
