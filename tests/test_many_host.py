"""Host-side checks of the many-tensor entry points (dm_adamw_step,
dm_grad_clip): struct layouts, defaults, and refusals, which come back before
anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import dimuon_optimizer_b200 as dm

WS = (0x100000, 1 << 30)


def fake_tensor(numel=1000, state=dm.DM_STATE_FP32, at=0):
    t = dm.dm_adamw_tensor_t()
    t.numel = numel
    t.weight, t.grad = 0x10000 + at, 0x20000 + at
    t.moment1, t.moment2 = 0x30000 + at, 0x40000 + at
    t.weight_dtype = t.grad_dtype = dm.DM_BF16
    t.state = state
    if state == dm.DM_STATE_8BIT:
        t.scale1, t.scale2 = 0x50000 + at, 0x60000 + at
    t.lr_mult = t.decay_mult = 1.0
    return t


def fake_grad(numel=1000, out=None):
    t = dm.dm_grad_t()
    t.numel, t.grad, t.grad_dtype = numel, 0x10000, dm.DM_BF16
    t.out, t.out_dtype = out, dm.DM_BF16
    return t


def test_struct_layouts():
    assert ctypes.sizeof(dm.dm_adamw_tensor_t) == 80
    assert dm.dm_adamw_tensor_t.weight_dtype.offset == 56
    assert ctypes.sizeof(dm.dm_adamw_hparams_t) == 64
    assert dm.dm_adamw_hparams_t.step.offset == 24
    assert dm.dm_adamw_hparams_t.reserved.offset == 56
    assert ctypes.sizeof(dm.dm_grad_t) == 32


def test_defaults():
    hp = dm.dm_adamw_default_hparams()
    assert [round(x, 9) for x in (hp.lr, hp.beta1, hp.beta2, hp.weight_decay)] == \
        [0.001, pytest.approx(0.9), pytest.approx(0.999), pytest.approx(0.01)]
    assert hp.eps == pytest.approx(1e-8) and hp.step == 1 and hp.seed == 0
    assert not hp.step_counter and not hp.lr_dev and not hp.grad_scale
    assert dm.dm_adamw_default_hparams(lr=0.5, step=7).step == 7
    assert dm.dm_adamw_workspace_size([fake_tensor()], hp) >= 256
    assert dm.dm_adamw_workspace_size([], hp) >= 256


@pytest.mark.parametrize("mutate,code", [
    (lambda t, h: setattr(t, "numel", -1), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "numel", (1 << 40) + 1), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "weight", None), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "grad", None), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "moment1", None), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "moment2", None), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "scale1", None), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "scale2", 0x60002), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "weight", 0x10001), dm.DM_ERR_INVALID_ARG),   # not on an element
    (lambda t, h: setattr(t, "grad", 0x20001), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "weight_dtype", 2), dm.DM_ERR_UNSUPPORTED),
    (lambda t, h: setattr(t, "grad_dtype", -1), dm.DM_ERR_UNSUPPORTED),
    (lambda t, h: setattr(t, "state", 2), dm.DM_ERR_UNSUPPORTED),
    (lambda t, h: setattr(t, "lr_mult", float("nan")), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "decay_mult", float("inf")), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "reserved0", 1), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(t, "moment1", t.weight), dm.DM_ERR_INVALID_ARG),  # written twice
    (lambda t, h: setattr(t, "scale2", t.scale1), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(h, "lr", float("inf")), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(h, "beta1", 1.0), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(h, "beta2", -0.1), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(h, "beta2", float("nan")), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(h, "eps", -1e-8), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(h, "step", 0), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: setattr(h, "step_counter", 0x1004), dm.DM_ERR_INVALID_ARG),  # not on 8 bytes
    (lambda t, h: setattr(h, "grad_scale", 0x1002), dm.DM_ERR_INVALID_ARG),
    (lambda t, h: h.reserved.__setitem__(1, 1), dm.DM_ERR_INVALID_ARG),
])
def test_adamw_refusals(mutate, code):
    t, hp = fake_tensor(state=dm.DM_STATE_8BIT), dm.dm_adamw_default_hparams()
    mutate(t, hp)
    assert dm.dm_adamw_step([t], hp, WS, stream=0) == code


def test_fp32_moments_on_an_element():
    t, hp = fake_tensor(), dm.dm_adamw_default_hparams()
    t.moment2 += 2
    assert dm.dm_adamw_step([t], hp, WS, stream=0) == dm.DM_ERR_INVALID_ARG


def test_the_same_tensor_twice_is_refused():
    hp = dm.dm_adamw_default_hparams()
    a, b = fake_tensor(), fake_tensor(at=0x100000)
    b.moment2 = a.moment2
    assert dm.dm_adamw_step([a, b], hp, WS, stream=0) == dm.DM_ERR_INVALID_ARG
    assert dm.dm_adamw_step([a, a], hp, WS, stream=0) == dm.DM_ERR_INVALID_ARG
    g = fake_grad(out=0x70000)
    assert clip([g, g], 1.0, 0x200000) == dm.DM_ERR_INVALID_ARG


def test_gradients_that_are_written_are_refused():
    hp = dm.dm_adamw_default_hparams()
    a, b = fake_tensor(), fake_tensor(at=0x100000)
    b.grad = a.weight
    assert dm.dm_adamw_step([a, b], hp, WS, stream=0) == dm.DM_ERR_INVALID_ARG
    # one tensor's output is another's gradient; a gradient in place that another reads
    x, y = fake_grad(out=0x20000), fake_grad()
    y.grad = 0x20000
    assert clip([x, y], 1.0, 0x200000) == dm.DM_ERR_INVALID_ARG
    assert clip([y, x], 1.0, 0x200000) == dm.DM_ERR_INVALID_ARG
    x, y = fake_grad(out=0x10000), fake_grad(out=0x20000)
    assert clip([x, y], 1.0, 0x200000) == dm.DM_ERR_INVALID_ARG


def clip(ts, max_norm, result, ws=WS):
    arr, n = dm._list(ts, dm.dm_grad_t)
    return dm._lib.dm_grad_clip(arr, n, max_norm, result, ws[0], ws[1], None)


@pytest.mark.parametrize("mutate,code", [
    (lambda t: setattr(t, "numel", -1), dm.DM_ERR_INVALID_ARG),
    (lambda t: setattr(t, "numel", 1 << 41), dm.DM_ERR_INVALID_ARG),
    (lambda t: setattr(t, "grad", None), dm.DM_ERR_INVALID_ARG),
    (lambda t: setattr(t, "grad", 0x10001), dm.DM_ERR_INVALID_ARG),
    (lambda t: setattr(t, "out", 0x20001), dm.DM_ERR_INVALID_ARG),
    (lambda t: setattr(t, "grad_dtype", 5), dm.DM_ERR_UNSUPPORTED),
    (lambda t: setattr(t, "out_dtype", 5), dm.DM_ERR_UNSUPPORTED),
    # in place in another type
    (lambda t: (setattr(t, "out", t.grad), setattr(t, "out_dtype", dm.DM_FP32)),
     dm.DM_ERR_INVALID_ARG),
])
def test_clip_refusals(mutate, code):
    t = fake_grad(out=0x20000)
    mutate(t)
    assert clip([t], 1.0, 0x200000) == code


def test_clip_scalar_refusals():
    t = fake_grad()
    for bad in (0.0, -1.0, float("nan")):
        assert clip([t], bad, 0x200000) == dm.DM_ERR_INVALID_ARG
    assert clip([t], 1.0, None) == dm.DM_ERR_INVALID_ARG
    assert clip([t], 1.0, 0x200002) == dm.DM_ERR_INVALID_ARG


def test_workspace_refusals():
    hp = dm.dm_adamw_default_hparams()
    t, g = fake_tensor(), fake_grad()
    need = dm.dm_adamw_workspace_size([t], hp)
    for ws in ((0, need), (0x100010, need), (0x100000, need - 1)):
        assert dm.dm_adamw_step([t], hp, ws, stream=0) == dm.DM_ERR_WORKSPACE
    need = dm.dm_grad_clip_workspace_size([g])
    for ws in ((0, need), (0x100010, need), (0x100000, need - 1)):
        assert clip([g], 1.0, 0x200000, ws) == dm.DM_ERR_WORKSPACE
    # more launches leave more partial sums
    assert dm.dm_grad_clip_workspace_size([g] * 2000) > need
    assert dm.dm_grad_clip_workspace_size([]) >= 256


def test_sizes_refuse_like_the_calls():
    hp = dm.dm_adamw_default_hparams(beta1=2.0)
    with pytest.raises(dm.DimuonError):
        dm.dm_adamw_workspace_size([fake_tensor()], hp)
    with pytest.raises(dm.DimuonError):
        dm.dm_grad_clip_workspace_size([fake_grad(numel=-5)])


def test_binding_refuses_what_would_fault():
    """Host tensors, other dtypes, sizes and layouts never reach the kernels."""
    w, g, m, v = (torch.zeros(8) for _ in range(4))
    with pytest.raises(ValueError, match="CUDA"):
        dm.dm_adamw_tensor(w, g, m, v)
    with pytest.raises(ValueError, match="elements"):
        dm.dm_adamw_tensor(w, torch.zeros(7), m, v)
    with pytest.raises(TypeError, match="moments"):
        dm.dm_adamw_tensor(w, g, m.half(), v)
    with pytest.raises(TypeError, match="moments"):
        dm.dm_adamw_tensor(w, g, m.to(torch.float8_e5m2), v.to(torch.float8_e5m2))
    with pytest.raises(ValueError, match="scales"):
        dm.dm_adamw_tensor(w, g, m, v, scale1=torch.zeros(1))
    e1, e2 = m.to(torch.float8_e4m3fn), v.to(torch.float8_e5m2)
    with pytest.raises(ValueError, match="scales"):
        dm.dm_adamw_tensor(w, g, e1, e2)
    with pytest.raises(ValueError, match="scales"):
        dm.dm_adamw_tensor(w, g, e1, e2, torch.zeros(2), torch.zeros(2))
    with pytest.raises(TypeError):
        dm.dm_adamw_tensor(w.half(), g, m, v)
    with pytest.raises(ValueError, match="CUDA"):
        dm.dm_grad_tensor(g)
    with pytest.raises(ValueError, match="elements"):
        dm.dm_grad_tensor(g, torch.zeros(9))
    with pytest.raises(ValueError, match="two"):
        dm.dm_grad_clip([], 1.0, torch.zeros(3), WS, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        dm.dm_grad_clip([], 1.0, torch.zeros(2), WS, stream=0)
    with pytest.raises(ValueError, match="step_counter"):
        dm.dm_adamw_default_hparams(step_counter=torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA"):
        dm.dm_adamw_default_hparams(grad_scale=torch.zeros(1))
    with pytest.raises(ValueError):
        dm.dm_adamw_state(w, 5)


def test_state_shapes():
    m, v = dm.dm_adamw_state(torch.zeros(3, 5))
    assert m.shape == v.shape == (3, 5) and m.dtype == v.dtype == torch.float32
    m, v, s1, s2 = dm.dm_adamw_state(torch.zeros(3, 100), dm.DM_STATE_8BIT)
    assert (m.dtype, v.dtype) == (torch.float8_e4m3fn, torch.float8_e5m2)
    assert m.shape == (3, 100) and s1.numel() == s2.numel() == 3 and not s1.any()
