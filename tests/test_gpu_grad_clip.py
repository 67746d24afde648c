"""dm_grad_clip on the GPU against float64, and the clipped training step:
one norm over the gradients of both groups, Muon on the matrices, AdamW on the
rest.

Tolerances (u = 2^-24): a square and a running sum of 16 of them in fp32 round
at most 17 times, so the sum of squares is off by 17 u relative and the norm by
half of that, plus its rounding to fp32: 10 u.  The coefficient adds one
rounding, a clipped gradient its product and half a step of its type.
"""
import math

import numpy as np
import pytest
import torch

import dimuon_optimizer_b200 as dm
import oracle as orc
from gpu_harness import TOL_BF16, Group, oracle_hp, rel_fro, to_dev, to_host
from oracle import adamw_oracle as ao
from test_gpu_adamw import Buf, check_fp32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
SIZES = [1, 2, 7, 8, 9, 15, 16, 17, 31, 500, 4095, 4096, 4097, 8191, 20011, 0]


def call(ts, max_norm, status=dm.DM_OK, stream=None):
    ts = list(ts)
    res = torch.full((2,), -1.0, device="cuda")
    ws = torch.full((dm.dm_grad_clip_workspace_size(ts),), 0xFF, dtype=torch.uint8, device="cuda")
    dm.check(dm.dm_grad_clip(ts, max_norm, res, ws, stream=stream))
    assert dm.dm_read_device_status(ws, stream=stream) == status
    return res


@pytest.mark.parametrize("gdt", [BF, F32])
@pytest.mark.parametrize("odt", [None, BF, F32, "in_place"])
@pytest.mark.parametrize("layout", ["aligned", "same_offset", "mixed_offset"])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_norm_and_clip(gdt, odt, layout, max_norm):
    rng = np.random.default_rng(1)
    gb, ob = [], []
    for i, n in enumerate(SIZES):
        s, o = (0, 0) if layout == "aligned" else (i % 8, i % 8) if layout == "same_offset" else \
            (i % 8, (i + 3) % 8)
        gb.append(Buf(n, gdt, s, rng.standard_normal(n)))
        ob.append(gb[-1] if odt == "in_place" else None if odt is None else Buf(n, odt, o))
    host = [to_host(g.t) for g in gb]
    norm, c, _ = ao.grad_clip(host, max_norm)
    res = call([dm.dm_grad_tensor(g.t, o.t if o else None) for g, o in zip(gb, ob)], max_norm)
    assert abs(res[0].item() - norm) <= 10 * U * norm
    assert abs(res[1].item() - c) <= (0 if c == 1.0 else 11 * U * c)
    for g, o, h in zip(gb, ob, host):
        g.check()
        if odt != "in_place":
            assert np.array_equal(to_host(g.t), h)
        if o:
            o.check()
            half = torch.finfo(o.t.dtype).eps / 2
            want = h * c
            assert np.all(np.abs(to_host(o.t) - want) <= (13 * U + half * (1 + 13 * U)) * np.abs(want))


def test_more_tensors_than_a_launch_holds():
    rng = np.random.default_rng(2)
    gs = [torch.from_numpy(rng.standard_normal(int(n))).to(BF).cuda()
          for n in rng.integers(0, 9000, 1100)]
    out = [torch.empty_like(g) for g in gs]
    norm, c, want = ao.grad_clip([to_host(g) for g in gs], 2.0, ["bf16"] * len(gs))
    # every second gradient has an output
    res = call([dm.dm_grad_tensor(g, o if i % 2 else None)
                for i, (g, o) in enumerate(zip(gs, out))], 2.0)
    assert abs(res[0].item() - norm) <= 10 * U * norm
    for o, w in list(zip(out, want))[1::2]:
        assert np.all(np.abs(to_host(o) - w) <= 2.0 ** -7 * np.abs(w))  # one bf16 step


@pytest.mark.parametrize("size", [1e30, 1e-30, 1e-42])
def test_sizes_whose_squares_leave_fp32(size):
    rng = np.random.default_rng(3)
    g = torch.from_numpy(rng.standard_normal(100003) * size).float().cuda()
    h = to_host(g)
    norm = math.sqrt((h ** 2).sum())
    res = call([dm.dm_grad_tensor(g)], size)
    # subnormal results carry an absolute error of half a subnormal step
    assert abs(res[0].item() - norm) <= 10 * U * norm + 2.0 ** -150
    assert abs(res[1].item() - min(1.0, float(np.float32(size)) / norm)) <= 11 * U
    # next to ordinary gradients the small ones count as nothing, the large ones as all
    res = call([dm.dm_grad_tensor(g), dm.dm_grad_tensor(torch.ones(64, device="cuda"))], 1.0)
    assert abs(res[0].item() - math.sqrt(norm ** 2 + 64)) <= 10 * U * math.sqrt(norm ** 2 + 64)


def test_zero_and_no_gradients():
    z = torch.zeros(5000, device="cuda")
    o = torch.ones(5000, device="cuda")
    res = call([dm.dm_grad_tensor(z, o)], 1.0)
    assert res.tolist() == [0.0, 1.0] and not o.any()
    for ts in ([], [dm.dm_grad_tensor(torch.zeros(0, device="cuda"))]):
        assert call(ts, 1.0).tolist() == [0.0, 1.0]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("in_place", [False, True])
def test_non_finite_gradients_write_nothing(bad, in_place):
    g = torch.ones(70001, device="cuda")
    g[65000] = bad
    o = g if in_place else torch.full_like(g, 7.0)
    keep = o.clone()
    res = call([dm.dm_grad_tensor(g, o)], 1.0, dm.DM_ERR_NONFINITE)
    assert not math.isfinite(res[0].item()) and math.isnan(res[1].item())
    assert torch.equal(o.view(torch.int32), keep.view(torch.int32))
    # a norm beyond fp32 counts as not finite
    call([dm.dm_grad_tensor(torch.full((100,), 3e38, device="cuda"))], 1.0, dm.DM_ERR_NONFINITE)


def test_the_same_bits_every_time():
    gs = [torch.randn(n, device="cuda").to(BF) for n in (3_000_001, 77, 1_234_567)]
    ts = [dm.dm_grad_tensor(g) for g in gs]
    first = call(ts, 1.0)
    for _ in range(5):
        assert torch.equal(call(ts, 1.0), first)


def test_infinite_limit_copies():
    g = torch.randn(10007, device="cuda")
    o = torch.empty_like(g)
    res = call([dm.dm_grad_tensor(g, o)], math.inf)
    assert torch.equal(g, o) and res[1].item() == 1.0


@pytest.mark.slow
def test_offsets_past_32_bits():
    n = (1 << 32) + 777
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[-5:] = 2.0
    g[0] = 1.0
    o = torch.empty_like(g)
    res = call([dm.dm_grad_tensor(g, o)], 1.0)
    want = math.sqrt(21.0)
    assert abs(res[0].item() - want) <= 10 * U * want
    half = 2.0 ** -8
    for i, x in ((0, 1.0), (n - 1, 2.0), (n - 5, 2.0), (n - 6, 0.0), (1 << 32, 0.0)):
        assert abs(o[i].item() - x / want) <= 2 * half * x / want
    assert int(o.count_nonzero()) == 6


@pytest.mark.parametrize("state", [dm.DM_STATE_FP32, dm.DM_STATE_8BIT])
@pytest.mark.parametrize("captured", [False, True])
def test_a_clipped_training_step(state, captured):
    """Three steps as a training loop makes them: one norm over all gradients
    (Muon's clipped in place, AdamW's scaled by the coefficient), then both
    optimizers; each step against the oracles from the state before it.  The third step's
    gradients hold a NaN: AdamW skips it, and so does the caller's Muon."""
    shapes = [(64, 96), (8, 512)]
    vecs = [768, 101, 4096 + 5]
    rng = np.random.default_rng(8)
    grp = Group(shapes, dm.DM_BF16, dm.DM_BF16, dm.DM_FP32, seed=8)
    mg = [torch.zeros(s, dtype=BF, device="cuda") for s in shapes]
    W = [torch.randn(n, device="cuda").to(BF) for n in vecs]
    ag = [torch.zeros(n, dtype=BF, device="cuda") for n in vecs]
    st = [dm.dm_adamw_state(w, state) for w in W]
    res = torch.zeros(2, device="cuda")
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    hp = dm.dm_default_hparams(weight_decay=0.1)
    ha = dm.dm_adamw_default_hparams(lr=0.01, seed=5, step_counter=counter, grad_scale=res[1:])
    mats = grp.matrices(mg)
    ts = dm.dm_adamw_tensors([dm.dm_adamw_tensor(w, g, *s) for w, g, s in zip(W, ag, st)])
    cl = dm.dm_grad_tensors([dm.dm_grad_tensor(g, g) for g in mg] + [dm.dm_grad_tensor(g) for g in ag])
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
        dm.dm_workspace_size(mats, hp, 0), dm.dm_adamw_workspace_size(ts, ha),
        dm.dm_grad_clip_workspace_size(cl))]

    def clip_and_adamw():
        dm.check(dm.dm_grad_clip(cl, 3.0, res, ws[2]))
        dm.check(dm.dm_adamw_step(ts, ha, ws[1]))

    run = clip_and_adamw
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            clip_and_adamw()
        run = graph.replay
    p = ao.AdamWParams(ha.lr, ha.beta1, ha.beta2, ha.eps, ha.weight_decay)
    for step in (1, 2, 3):
        for g in mg + ag:
            g.copy_(torch.from_numpy(rng.standard_normal(tuple(g.shape))))
        if step == 3:
            ag[1][50] = float("nan")
        gh = [to_host(g) for g in mg + ag]
        before = [(to_host(w), to_host(g)) for w, g in zip(W, ag)]
        moments = []
        for s in st:
            if state == dm.DM_STATE_FP32:
                moments.append((to_host(s[0]), to_host(s[1])))
            else:
                moments.append((ao.unpack(s[0].view(torch.uint8).cpu().numpy(), to_host(s[2]), ao.E4M3),
                                ao.unpack(s[1].view(torch.uint8).cpu().numpy(), to_host(s[3]), ao.E5M2)))
        mom = [to_host(m) for m in grp.M], [to_host(w) for w in grp.W]
        run()
        if step == 3:
            assert dm.dm_read_device_status(ws[2]) == dm.DM_ERR_NONFINITE
            assert dm.dm_read_device_status(ws[1]) == dm.DM_ERR_NONFINITE
            assert counter.item() == 2
            assert all(np.array_equal(to_host(w), b[0]) for w, b in zip(W, before))
            break
        dm.check(dm.dm_muon_step(mats, hp, ws[0]))
        for k in range(3):
            assert dm.dm_read_device_status(ws[k]) == dm.DM_OK
        norm, c, _ = ao.grad_clip(gh, 3.0)
        assert c < 1 and abs(res[0].item() - norm) <= 10 * U * norm
        coef = res[1].item()
        assert abs(coef - c) <= 11 * U * c and counter.item() == step
        for w, s, b, m in zip(W, st, before, moments):
            fp = state == dm.DM_STATE_FP32
            check_fp32(*b, *m, ha, step, to_host(w), to_host(s[0]) if fp else None,
                       to_host(s[1]) if fp else None, BF, coef)
        for i in range(len(shapes)):
            assert np.all(np.abs(to_host(mg[i]) - gh[i] * c) <= (2.0 ** -8 + 13 * U) * np.abs(gh[i] * c))
            r = orc.optimizer_step(mom[1][i], to_host(mg[i]), mom[0][i], oracle_hp(hp), conditioned=False,
                                   momentum_dtype="fp32", weight_dtype="bf16")
            assert np.array_equal(to_host(grp.M[i]), r.M)
            assert rel_fro(to_host(grp.upd[i]), r.O) <= TOL_BF16
