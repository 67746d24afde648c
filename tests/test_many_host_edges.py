"""Further host-side checks of the many-tensor entry points: what they refuse
and what their sizes count, before anything is launched (no GPU needed)."""
import types

import numpy as np
import pytest
import torch

import dimuon_optimizer_b200 as dm
from oracle import adamw_oracle as ao
from test_many_host import WS, fake_grad, fake_tensor


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


class OnDevice:
    """Stands in for a CUDA tensor of 8 elements on device `index`."""

    def __init__(self, index, dtype=torch.float32, numel=8):
        self.device = types.SimpleNamespace(index=index)
        self.dtype, self._numel, self.is_cuda = dtype, numel, True

    def numel(self):
        return self._numel

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100000


@pytest.fixture
def devices(monkeypatch):
    """.current is the current device; .calls counts what reached the library."""
    st = types.SimpleNamespace(current=0, calls=0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: st.current)

    def reached(*args):
        st.calls += 1
        return dm.DM_OK

    monkeypatch.setattr(dm, "_lib", types.SimpleNamespace(
        dm_adamw_step=reached, dm_grad_clip=reached,
        dm_adamw_default_hparams=dm._lib.dm_adamw_default_hparams))
    return st


@pytest.mark.parametrize("kept", [False, True])
def test_descriptors_of_another_device_are_refused(devices, kept):
    """Made while device 0 was current, called while device 1 is."""
    a = dm.dm_adamw_tensor(*(OnDevice(0) for _ in range(4)))
    g = dm.dm_grad_tensor(OnDevice(0))
    ts, gs = ([a], [g]) if not kept else (dm.dm_adamw_tensors([a]), dm.dm_grad_tensors([g]))
    hp = dm.dm_adamw_default_hparams()
    scaled = dm.dm_adamw_default_hparams(grad_scale=OnDevice(0, numel=1))

    def calls():
        ws, res = OnDevice(devices.current, torch.uint8, 4096), OnDevice(devices.current, numel=2)
        yield lambda: dm.dm_adamw_step(ts, hp, ws, stream=0)
        yield lambda: dm.dm_adamw_step(ts, hp, WS, stream=0)
        yield lambda: dm.dm_adamw_step([], scaled, ws, stream=0)
        yield lambda: dm.dm_grad_clip(gs, 1.0, res, ws, stream=0)

    for c in calls():
        assert c() == dm.DM_OK
    assert devices.calls == 4
    devices.current = 1
    for c in calls():
        with pytest.raises(ValueError, match="cuda:0.*current CUDA device"):
            c()
    assert devices.calls == 4


def test_lists_over_two_devices_are_refused(devices):
    a = dm.dm_adamw_tensor(*(OnDevice(0) for _ in range(4)))
    devices.current = 1
    b = dm.dm_adamw_tensor(*(OnDevice(1) for _ in range(4)))
    for ts in ([a, b], [b, a], dm.dm_adamw_tensors([a, b])):
        with pytest.raises(ValueError, match="cuda:0"):
            dm.dm_adamw_step(ts, dm.dm_adamw_default_hparams(), OnDevice(1, torch.uint8, 4096), stream=0)
    assert devices.calls == 0


def test_a_generator_of_descriptors_is_one_list(devices):
    """Looked at for its devices and then handed over whole."""
    got = []
    dm._lib.dm_adamw_step = lambda arr, n, *rest: got.append(n) or dm.DM_OK
    gen = (dm.dm_adamw_tensor(*(OnDevice(0) for _ in range(4))) for _ in range(3))
    dm.dm_adamw_step(gen, dm.dm_adamw_default_hparams(), WS, stream=0)
    assert got == [3]


def test_hyper_parameters_of_other_names_are_refused():
    """torch's betas=(0.9, 0.95), say, must not leave the defaults in place."""
    for name in ("betas", "wd", "Lr", "_keep"):
        with pytest.raises(TypeError, match="no field"):
            dm.dm_adamw_default_hparams(**{name: (0.9, 0.95)})
    assert dm.dm_adamw_default_hparams(seed=3, step_counter=None).seed == 3
