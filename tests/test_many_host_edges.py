"""Further host-side checks of the many-tensor entry points: what they refuse
and what their sizes count, before anything is launched (no GPU needed)."""
import pytest

import dimuon_optimizer_b200 as dm
from test_many_host import fake_tensor


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
