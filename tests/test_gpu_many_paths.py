"""Launch forms of dm_adamw_step and dm_grad_clip that only certain lists
reach: parameter blocks by the number of tensors, four passes per CTA of the
8-bit form, one buffer off its boundary, gradients at any offset of 16.

Tolerances are those derived in test_gpu_adamw and test_gpu_grad_clip; 8-bit
codes and scales equal the oracle's.
"""
import numpy as np
import pytest
import torch

import dimuon_optimizer_b200 as dm
from gpu_harness import to_host
from oracle import adamw_oracle as ao
from test_gpu_adamw import BF, F32, U, Buf, check_fp32, draw, workspace
from test_gpu_grad_clip import call

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def params(hp):
    return ao.AdamWParams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay)


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


class Eight:
    """A tensor with 8-bit moments: weight, gradient and both moments at their
    element offsets, random codes as they stand after some steps."""

    def __init__(self, n, wdt, gdt, shifts, seed):
        rng = np.random.default_rng(seed)
        blocks = -(-n // 128)
        W, G, _, _ = draw(n, seed)
        self.bufs = [Buf(n, dt, s) for dt, s in zip((wdt, gdt, E4, E5), shifts)]
        self.bufs += [Buf(blocks, F32), Buf(blocks, F32)]
        W, G = (torch.from_numpy(x) for x in (W, G))
        self.bufs[0].t.copy_(W)
        self.bufs[1].t.copy_(G)
        for k, top in ((2, 127), (3, 124)):
            c = rng.integers(0, top, n, dtype=np.uint8)
            if k == 2:
                c |= (rng.random(n) < 0.5).astype(np.uint8) << 7
            self.bufs[k].t.view(torch.uint8).copy_(torch.from_numpy(c))
        for k, base in ((4, -9), (5, -17)):
            self.bufs[k].t.copy_(torch.from_numpy(2.0 ** (base + rng.integers(-3, 4, blocks))))
        self.before = None

    def descriptor(self):
        return dm.dm_adamw_tensor(*(b.t for b in self.bufs))

    def remember(self):
        w, g, c1, c2, s1, s2 = (b.t for b in self.bufs)
        self.before = (to_host(w), to_host(g), ao.unpack(codes(c1), to_host(s1), ao.E4M3),
                       ao.unpack(codes(c2), to_host(s2), ao.E5M2))

    def check(self, hp, t, index, wdt, gs=1.0):
        for b in self.bufs:
            b.check()
        w0, g, m0, v0 = self.before
        m32, v32 = ao.moments_f32(g, m0, v0, params(hp), gs)
        want = ao.pack_moments(m32.astype(np.float64), v32.astype(np.float64), hp.seed, t, index)
        w, grad, c1, c2, s1, s2 = (b.t for b in self.bufs)
        for got, x in zip((codes(c1), to_host(s1), codes(c2), to_host(s2)), want):
            np.testing.assert_array_equal(got, x)
        assert np.array_equal(to_host(grad), g)
        check_fp32(w0, g, m0, v0, hp, t, to_host(w), None, None, wdt, gs)


@pytest.mark.parametrize("moved", [0, 1, 2, 3])
@pytest.mark.parametrize("shift", [1, 8, 16])
@pytest.mark.parametrize("wdt,gdt", [(BF, BF), (F32, F32)])
def test_8bit_one_buffer_off_its_boundary(moved, shift, wdt, gdt):
    hp = dm.dm_adamw_default_hparams(lr=3e-3, weight_decay=0.1, seed=4, step=7)
    items = [Eight(n, wdt, gdt, [shift if k == moved else 0 for k in range(4)], 300 + n)
             for n in (1, 15, 16, 17, 128, 4097, 8192, 9001)]
    ts = [x.descriptor() for x in items]
    for x in items:
        x.remember()
    dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
    for i, x in enumerate(items):
        x.check(hp, 7, i, wdt)


@pytest.mark.parametrize("wdt,gdt", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_8bit_long_lists(wdt, gdt):
    """Just over 2^24 elements of one pair of types, from where a CTA takes
    four passes: whole and ragged tensors, one of them at an offset."""
    gs = torch.tensor([0.75], device="cuda")
    hp = dm.dm_adamw_default_hparams(lr=3e-3, weight_decay=0.1, seed=6, step=40, grad_scale=gs)
    sizes = [((1 << 23) + 4097, 0), ((1 << 22) + 77, 3), (5, 0), (1 << 22, 0), (3 * 16384, 0),
             (16385, 0), (12288, 1), (4095, 0)]
    assert sum(n for n, _ in sizes) >= 1 << 24
    items = [Eight(n, wdt, gdt, [s] * 4, 400 + i) for i, (n, s) in enumerate(sizes)]
    ts = [x.descriptor() for x in items]
    for x in items:
        x.remember()
    ws = workspace(ts, hp)
    dm.check(dm.dm_adamw_step(ts, hp, ws))
    assert dm.dm_read_device_status(ws) == dm.DM_OK
    for i, x in enumerate(items):
        x.check(hp, 40, i, wdt, 0.75)


@pytest.mark.parametrize("count", [24, 25, 100, 160, 161])
@pytest.mark.parametrize("wdt,gdt", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_adamw_lists_of_every_parameter_block(count, wdt, gdt):
    """`count` tensors of each moment format: the blocks hold 24, 160 and 448."""
    hp = dm.dm_adamw_default_hparams(lr=3e-3, weight_decay=0.1, seed=12, step=3)
    rng = np.random.default_rng(count)
    eight = [Eight(int(n), wdt, gdt, [0] * 4, 500 + i)
             for i, n in enumerate(rng.integers(1, 900, count))]
    fp32 = []
    for i, n in enumerate(rng.integers(1, 5000, count)):
        x = draw(int(n), 700 + i)
        fp32.append([Buf(int(n), dt, i % 8, y) for y, dt in zip(x, (wdt, gdt, F32, F32))])
    host = [[to_host(b.t) for b in x] for x in fp32]
    for x in eight:
        x.remember()
    ts = [x.descriptor() for x in eight] + [dm.dm_adamw_tensor(*(b.t for b in x)) for x in fp32]
    dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
    for i, x in enumerate(eight):
        x.check(hp, 3, i, wdt)
    for x, h in zip(fp32, host):
        for b in x:
            b.check()
        check_fp32(*h, hp, 3, to_host(x[0].t), to_host(x[2].t), to_host(x[3].t), wdt)


@pytest.mark.parametrize("count", [24, 25, 100, 160, 161])
@pytest.mark.parametrize("gdt,odt", [(BF, None), (F32, None), (BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_clip_lists_of_every_parameter_block(count, gdt, odt):
    """... with offsets 0 to 15 of gradient and output, equal in every second tensor."""
    rng = np.random.default_rng(count)
    gb, ob = [], []
    for i in range(count):
        n = int(rng.integers(1, 40000 if i % 10 == 0 else 300))
        gb.append(Buf(n, gdt, i % 16, rng.standard_normal(n)))
        ob.append(Buf(n, odt, i % 16 if i % 2 else (i + 5) % 16) if odt else None)
    host = [to_host(g.t) for g in gb]
    norm, c, _ = ao.grad_clip(host, 0.5)
    res = call([dm.dm_grad_tensor(g.t, o.t if o else None) for g, o in zip(gb, ob)], 0.5)
    assert abs(res[0].item() - norm) <= 10 * U * norm
    assert abs(res[1].item() - c) <= 11 * U * c
    for g, o, h in zip(gb, ob, host):
        g.check()
        assert np.array_equal(to_host(g.t), h)
        if o:
            o.check()
            half = torch.finfo(odt).eps / 2
            want = h * c
            assert np.all(np.abs(to_host(o.t) - want) <= (13 * U + half * (1 + 13 * U)) * np.abs(want))


@pytest.mark.parametrize("gdt", [BF, F32])
@pytest.mark.parametrize("shift", range(16))
def test_norm_at_every_offset(gdt, shift):
    """Lengths that end groups of 16 at every place, gradients in place."""
    rng = np.random.default_rng(shift)
    gb = [Buf(n, gdt, shift, rng.standard_normal(n)) for n in list(range(1, 34)) + [16383, 16384, 16400]]
    host = [to_host(g.t) for g in gb]
    norm, c, _ = ao.grad_clip(host, 3.0)
    res = call([dm.dm_grad_tensor(g.t, g.t) for g in gb], 3.0)
    assert abs(res[0].item() - norm) <= 10 * U * norm
    half = torch.finfo(gdt).eps / 2
    for g, h in zip(gb, host):
        g.check()
        want = h * c
        assert np.all(np.abs(to_host(g.t) - want) <= (13 * U + half * (1 + 13 * U)) * np.abs(want))
