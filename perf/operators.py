"""Cases of the library's many-tensor operators: the AdamW step with its
moments in 32 bits or in 8, and the global gradient norm with clipping.

A case is a parameter set of `tables` equal matrices (embeddings, heads or
LoRA factors, rows x width each) followed by `vectors` vectors of about `width`
elements (biases, norms).  All tensors of a kind lie in one flat buffer at a
fixed stride, so a kind is also a (count, stride) matrix: the plain forms work on
that matrix, the library on one descriptor per tensor.  With `packed` the
stride is the tensor's own length (an odd one puts every other tensor on an
unaligned address), else it is rounded up to 128 elements and the gaps hold
zeros, which every operator here maps to zeros.
"""
import math

import torch

own = False  # true: run() calls the library; false: it computes the plain form

BLOCK = 128          # elements that share one scale of an 8-bit moment
E4M3_MAX = 448.0
E5M2_MAX = 57344.0
GOLDEN = 0x9E3779B9  # 2^32 / golden ratio, odd
M32 = 0xFFFFFFFF

BETA1, BETA2, EPS = 0.9, 0.999, 1e-8
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _adamw(name, op, tables, rows, width, vectors, weight="bf16", grad="bf16", ragged=False,
           packed=False, step=1000):
    return {"name": name, "op": op, "tables": tables, "rows": rows, "width": width,
            "vectors": vectors, "weight": weight, "grad": grad, "ragged": ragged,
            "packed": packed, "step": step}


def _clip(name, tables, rows, width, vectors, grad="bf16", out="none", ragged=False, packed=False,
          max_norm=1.0):
    return {"name": name, "op": "clip", "tables": tables, "rows": rows, "width": width,
            "vectors": vectors, "grad": grad, "out": out, "ragged": ragged, "packed": packed,
            "max_norm": max_norm}


def listed():
    return [
        # one bias vector alone, first step (all moments zero): launch latency
        _adamw("adamw32 one vector", "adamw32", 0, 0, 768, 1, step=1),
        # the biases and norms of twelve layers packed back to back at an odd
        # length, so that most tensors start on an unaligned address
        _adamw("adamw32 vectors packed", "adamw32", 0, 0, 771, 148, packed=True),
        # embedding and head of a small model with its vectors
        _adamw("adamw32 embeddings small", "adamw32", 2, 50257, 768, 98, ragged=True),
        # LoRA factors in fp32 with fp32 gradients
        _adamw("adamw32 lora fp32", "adamw32", 448, 8, 4096, 0, weight="fp32", grad="fp32"),
        # embedding and head of a large model: pure bandwidth
        _adamw("adamw32 embeddings large", "adamw32", 2, 32000, 4096, 130),
        # 8-bit moments: one short vector, a ragged last block
        _adamw("adamw8 one vector", "adamw8", 0, 0, 1001, 1, ragged=True, step=3),
        # LoRA factors of rank 32, fp32 weights kept by the optimizer, bf16 gradients
        _adamw("adamw8 lora fp32 weights", "adamw8", 448, 32, 4096, 0, weight="fp32"),
        # embedding and head of a large model with 8-bit moments: pure bandwidth
        _adamw("adamw8 embeddings large", "adamw8", 2, 32000, 4096, 130, ragged=True),
        # norm of a few vectors only (result read by the AdamW step): latency
        _clip("clip norm vectors", 0, 0, 768, 98, ragged=True),
        # norm over the hidden matrices of a large batch of layers
        _clip("clip norm matrices", 16, 4096, 4096, 130, max_norm=0.5),
        # fp32 accumulated gradients clipped into the bf16 gradients that the
        # orthogonalised matrices' step reads
        _clip("clip fp32 to bf16", 24, 1024, 4099, 51, grad="fp32", out="bf16"),
        # bf16 gradients clipped into a second bf16 buffer, packed at an odd length
        _clip("clip bf16 packed", 0, 0, 100003, 257, out="bf16", packed=True),
    ]


def draw(rng):
    op = rng.choice(["adamw32", "adamw8", "clip"])

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    width = log(64, 8192)
    if rng.random() < 0.5:
        width |= 1
    vectors = log(1, 400)
    tables, rows = 0, 0
    kind = rng.choice(["vectors", "factors", "tables"])
    if kind == "factors":
        tables, rows = log(8, 448), rng.choice([2, 4, 8, 16, 32, 5])
    elif kind == "tables":
        tables = rng.randint(1, 4)
        rows = log(100, 64000)
        rows = max(1, min(rows, 200_000_000 // (tables * width)))
    if op == "clip":
        out = rng.choice(["none", "bf16", "fp32"])
        c = _clip("", tables, rows, width, vectors, grad=rng.choice(["bf16", "fp32"]), out=out,
                  ragged=rng.random() < 0.5, packed=rng.random() < 0.3,
                  max_norm=rng.choice([0.25, 1.0, 1e6]))
    else:
        c = _adamw("", op, tables, rows, width, vectors, weight=rng.choice(["bf16", "fp32"]),
                   grad=rng.choice(["bf16", "fp32"]), ragged=rng.random() < 0.5,
                   packed=op == "adamw32" and rng.random() < 0.3, step=log(1, 100000))
    if c["packed"]:
        c["ragged"] = False
    del c["name"]
    return c


def _stride(case, n):
    return n if case["packed"] else -(-n // BLOCK) * BLOCK


def _kinds(case):
    """(count, stride, longest length) of the tables and of the vectors."""
    n = case["rows"] * case["width"]
    return [(case["tables"], _stride(case, n), n),
            (case["vectors"], _stride(case, case["width"]), case["width"])]


def _lengths(case):
    """Length of every tensor, the tables first."""
    n = case["rows"] * case["width"]
    vec = [max(1, case["width"] - (i % 37 if case["ragged"] else 0))
           for i in range(case["vectors"])]
    return [n] * case["tables"] + vec


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _pow2_scale(largest, top):
    """Smallest power of two s with largest <= top * s (1 where largest is 0)."""
    s = torch.exp2(torch.ceil(torch.log2(largest.double() / top)))
    return torch.where(largest > 0, s, torch.ones_like(s)).float()


def _pack(x, top, dtype):
    b = x.view(-1, BLOCK)
    scale = _pow2_scale(b.abs().amax(1), top)
    return (b / scale[:, None]).to(dtype).view(-1), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(n):
        return torch.randn(n, generator=gen, device="cuda")

    kinds, lengths = _kinds(case), _lengths(case)
    total = sum(c * s for c, s, _ in kinds)
    first_vec = kinds[0][0] * kinds[0][1]
    live = torch.ones(total, dtype=torch.bool, device="cuda")
    starts, pos = [], 0
    for c, s, _ in kinds:
        starts += [pos + i * s for i in range(c)]
        pos += c * s
    if case["tables"]:
        live[:first_vec].view(case["tables"], -1)[:, kinds[0][2]:] = False
    if case["vectors"]:
        n = torch.tensor(lengths[case["tables"]:], device="cuda")
        live[first_vec:] = (torch.arange(kinds[1][1], device="cuda") < n[:, None]).view(-1)
    # gradients: each run of 64 elements has its own size over three decades,
    # and in the tables two runs in five saw no token in this batch
    runs = -(-total // 64)
    size = torch.exp(1.7 * normal(runs))
    seen = torch.rand(runs, generator=gen, device="cuda") >= 0.4
    seen[first_vec // 64:] = True
    per = torch.repeat_interleave(size, 64)[:total]
    g = normal(total) * per * 1e-3 * live
    g *= torch.repeat_interleave(seen, 64)[:total]
    st = {"case": case, "starts": starts, "lengths": lengths, "kinds": kinds,
          "G": g.to(DTYPES[case["grad"]])}
    del g, seen
    if case["op"] == "clip":
        st["result"] = torch.zeros(2, device="cuda")
        if case["out"] != "none":
            st["out"] = torch.zeros(total, dtype=DTYPES[case["out"]], device="cuda")
    else:
        st["W"] = (0.02 * normal(total) * live).to(DTYPES[case["weight"]])
        later = 1.0 if case["step"] > 1 else 0.0
        m = normal(total) * per * (3e-4 * later) * live
        v = (1e-3 * per).square() * (0.5 + torch.rand(total, generator=gen, device="cuda")) \
            * later * live
        if case["op"] == "adamw8":
            st["M"], st["MS"] = _pack(m, E4M3_MAX, torch.float8_e4m3fn)
            st["V"], st["VS"] = _pack(v, E5M2_MAX, torch.float8_e5m2)
        else:
            st["M"], st["V"] = m, v
        del m, v
        st["clip"] = torch.full((), 0.37 + 0.01 * (seed % 50), device="cuda")
        st["step"] = case["step"] - 1
        st["seed"] = (seed * 2654435761 + 12345) & M32
    del per, live, size
    if own:
        _descriptors(st)
    return st


def _mults(case, i):
    """(learning-rate multiplier, weight-decay multiplier) of tensor i: the
    vectors are not decayed and move at half the rate."""
    return (1.0, 1.0) if i < case["tables"] else (0.5, 0.0)


LR, DECAY = 3e-4, 0.1


def _descriptors(st):
    """The library's descriptors and workspace, which a program keeps from
    step to step."""
    import dimuon_optimizer_b200 as dm
    case = st["case"]

    def part(name, i):
        return st[name][st["starts"][i]:st["starts"][i] + st["lengths"][i]]

    def scales(name, i):
        a = st["starts"][i] // BLOCK
        return st[name][a:a - (-st["lengths"][i] // BLOCK)]

    idx = range(len(st["lengths"]))
    if case["op"] == "clip":
        st["tensors"] = dm.dm_grad_tensors(
            [dm.dm_grad_tensor(part("G", i), part("out", i) if "out" in st else None) for i in idx])
        size = dm.dm_grad_clip_workspace_size(st["tensors"])
    else:
        ts = []
        for i in idx:
            lr, wd = _mults(case, i)
            sc = (scales("MS", i), scales("VS", i)) if case["op"] == "adamw8" else (None, None)
            ts.append(dm.dm_adamw_tensor(part("W", i), part("G", i), part("M", i), part("V", i),
                                         *sc, lr_mult=lr, decay_mult=wd))
        st["tensors"] = dm.dm_adamw_tensors(ts)
        st["hp"] = dm.dm_adamw_default_hparams(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                                               weight_decay=DECAY, seed=st["seed"],
                                               grad_scale=st["clip"])
        size = dm.dm_adamw_workspace_size(st["tensors"], st["hp"])
    st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(st):
    case = st["case"]
    if case["op"] == "clip":
        if own:
            import dimuon_optimizer_b200 as dm
            dm.check(dm.dm_grad_clip(st["tensors"], case["max_norm"], st["result"], st["ws"]))
        else:
            _plain_clip(st)
        return [st["result"], st["out"]] if "out" in st else [st["result"]]
    st["step"] += 1
    if own:
        import dimuon_optimizer_b200 as dm
        st["hp"].step = st["step"]
        dm.check(dm.dm_adamw_step(st["tensors"], st["hp"], st["ws"]))
    else:
        first_vec = st["kinds"][0][0] * st["kinds"][0][1]
        if case["tables"]:
            _plain_adamw(st, 0, st["kinds"][0], 0)
        if case["vectors"]:
            _plain_adamw(st, first_vec, st["kinds"][1], case["tables"])
    out = [st["W"], st["M"], st["V"]]
    return out + [st["MS"], st["VS"]] if case["op"] == "adamw8" else out


def _plain_clip(st):
    norm = st["G"].float().square().sum(dtype=torch.float64).sqrt()
    coef = torch.clamp(st["case"]["max_norm"] / norm, max=1.0).float()
    st["result"][0], st["result"][1] = norm, coef
    if "out" in st:
        st["out"].copy_(st["G"].float() * coef)


def _f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def _plain_adamw(st, at, kind, first):
    """The step of `kind`'s tensors, a (count, stride) matrix from element
    `at` on; `first` is the number of the first of them."""
    case, (count, stride, _) = st["case"], kind
    shape, cut = (count, stride), slice(at, at + count * stride)
    b1, b2 = _f32(BETA1), _f32(BETA2)
    c1, c2 = _f32(1.0 - b1), _f32(1.0 - b2)
    t = st["step"]
    lr_mult, wd_mult = _mults(case, first)
    lr = _f32(_f32(LR) * lr_mult)
    W, G = st["W"][cut].view(shape), st["G"][cut].view(shape)
    M, V = st["M"][cut].view(shape), st["V"][cut].view(shape)
    eight = case["op"] == "adamw8"
    m, v = M.float(), V.float()
    if eight:
        blocks = slice(at // BLOCK, (at + count * stride) // BLOCK)
        MS, VS = st["MS"][blocks], st["VS"][blocks]
        m = (m.view(-1, BLOCK) * MS[:, None]).view(shape)
        v = (v.view(-1, BLOCK) * VS[:, None]).view(shape)
    g = G.float() * st["clip"]
    m = m * b1 + g * c1
    v = v * b2 + (g * g) * c2
    denom = v.sqrt() * (1.0 / math.sqrt(1.0 - b2 ** t)) + _f32(EPS)
    W.copy_(W.float() * (1.0 - lr * _f32(_f32(DECAY) * wd_mult))
            - (m / denom) * (lr / (1.0 - b1 ** t)))
    if not eight:
        M.copy_(m)
        V.copy_(v)
        return
    h = _noise(st["seed"], t, count, stride, first)
    ms = _block_scale(m.view(-1, BLOCK), 8)
    vs = _block_scale(v.view(-1, BLOCK), 15)
    MS.copy_(ms)
    VS.copy_(vs)
    x = (m.view(-1, BLOCK).abs() / ms[:, None]).view(shape)
    code = _round_up_or_down(x, 3, 7, (h >> 16) << 4)
    code = torch.where(m < 0, code + 128, code)
    M.view(torch.uint8).copy_(code)
    x = (v.view(-1, BLOCK) / vs[:, None]).view(shape)
    code = _round_up_or_down(x, 2, 15, (h & 0xFFFF) << 5)
    code = torch.where((code == 0) & (v > 0), 1, code)  # a positive v never becomes 0
    V.view(torch.uint8).copy_(code)


def _mix(x):
    """A bijection of 32-bit words in which each bit of the result depends on every bit of x."""
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & M32
    x = ((x ^ (x >> 15)) * 0x846CA68B) & M32
    return x ^ (x >> 16)


def _noise(seed, step, count, stride, first):
    """32 bits for each element: 16 for each moment's rounding."""
    key = _mix((seed + GOLDEN * step) & M32)
    tensor = torch.arange(first, first + count, device="cuda")
    key = _mix((_mix((key + tensor) & M32) + 0) & M32)  # + bits 36 and up of the element
    i = torch.arange(stride, device="cuda")
    x = _mix(key[:, None] ^ (i >> 4)[None, :])
    x = (x + (GOLDEN * (i & 15))[None, :]) & M32
    x = (x * 0x7FEB352D) & M32
    x = ((x ^ (x >> 15)) * 0x846CA68B) & M32
    return x ^ (x >> 16)


def _block_scale(x, top):
    """Smallest power of two s with the row's largest |x| <= 1.75 * 2^top * s, at
    least 2^-110 (so that the least code is a normal number)."""
    bits = x.abs().amax(1).view(torch.int32)
    e = ((bits + 0x1FFFFF) >> 23) - top
    return (torch.clamp(e, min=17) << 23).view(torch.float32)


def _round_up_or_down(x, mantissa, bias, noise):
    """Codes of x >= 0 in a float format with `mantissa` bits and exponent
    `bias`: the neighbour below plus one with the probability of the
    remainder.  Below the least normal number, adding that number puts x on
    the grid of the subnormal codes."""
    least = 2.0 ** (1 - bias)
    small = x < least
    bits = torch.where(small, x + least, x).view(torch.int32).long()
    code = ((bits + noise) >> (23 - mantissa)) - ((127 - bias) << mantissa)
    return torch.where(small, code - (1 << mantissa), code)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    n = sum(_lengths(case))
    gb = 2 if case["grad"] == "bf16" else 4
    if case["op"] == "clip":
        ob = {"none": 0, "bf16": 2, "fp32": 4}[case["out"]]
        return {"bytes": n * (gb + ob), "flops": n * (3 if ob else 2)}
    wb = 2 if case["weight"] == "bf16" else 4
    if case["op"] == "adamw8":
        blocks = sum(-(-k // BLOCK) for k in _lengths(case))
        return {"bytes": n * (gb + 2 * wb + 4) + 16 * blocks, "flops": 30 * n}
    return {"bytes": n * (gb + 2 * wb + 16), "flops": 16 * n}


# ----------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ----------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        g = st["G"].double()
        norm = torch.linalg.vector_norm(g)
        c = min(1.0, case["max_norm"] / float(norm))
        res = torch.tensor([float(norm), c], dtype=torch.float64, device="cuda")
        return [res, g * c] if case["out"] != "none" else [res]
    f = {k: float(torch.tensor(x, dtype=torch.float32))
         for k, x in (("b1", BETA1), ("b2", BETA2), ("eps", EPS), ("lr", LR), ("wd", DECAY))}
    t = case["step"]
    eight = case["op"] == "adamw8"
    W, M, V = (torch.zeros(st["W"].numel(), dtype=torch.float64, device="cuda") for _ in "wmv")
    MS, VS = (torch.ones(st["W"].numel() // BLOCK, dtype=torch.float64, device="cuda")
              for _ in "mv") if eight else (None, None)
    for i, (a, n) in enumerate(zip(st["starts"], st["lengths"])):
        lr_mult, wd_mult = _mults(case, i)
        e = a + (-(-n // BLOCK) * BLOCK if eight else n)  # 8 bits: whole blocks, zeros behind n
        g = st["G"][a:e].double() * st["clip"].double()
        m, v = st["M"][a:e].double(), st["V"][a:e].double()
        if eight:
            bl = slice(a // BLOCK, e // BLOCK)
            m *= st["MS"][bl].double().repeat_interleave(BLOCK)
            v *= st["VS"][bl].double().repeat_interleave(BLOCK)
        m = f["b1"] * m + (1 - f["b1"]) * g
        v = f["b2"] * v + (1 - f["b2"]) * g ** 2
        mhat, vhat = m / (1 - f["b1"] ** t), v / (1 - f["b2"] ** t)
        lr = f["lr"] * lr_mult
        w = st["W"][a:e].double()
        W[a:e] = w - lr * f["wd"] * wd_mult * w - lr * mhat / (torch.sqrt(vhat) + f["eps"])
        if not eight:
            M[a:e], V[a:e] = m, v
            continue
        j = torch.arange(e - a, device="cuda")
        r = _exact_noise(st["seed"], t, i, j)
        M[a:e], MS[bl] = _exact_codes(m, E4M3_MAX, 3, -6, (r // 65536) / 65536)
        V[a:e], VS[bl] = _exact_codes(v, E5M2_MAX, 2, -14, (r % 65536) / 65536, keep=True)
    return [W, M, V, MS, VS] if eight else [W, M, V]


def _exact_codes(x, top, mantissa, least, u, keep=False):
    """(values of the codes, scales): |x| / scale rounded down to its grid
    after u grid steps are added."""
    big = x.abs().view(-1, BLOCK).amax(1)
    k = torch.ceil(torch.log2(big / top))
    scale = torch.exp2(torch.clamp(torch.where(big > 0, k, torch.full_like(k, -1e9)), min=-110.0))
    y = x.abs() / scale.repeat_interleave(BLOCK)
    grid = torch.exp2(torch.clamp(torch.floor(torch.log2(y)), min=float(least)) - mantissa)
    q = torch.floor(y / grid + u) * grid
    if keep:
        q = torch.where((q == 0) & (y > 0), grid, q)
    return torch.copysign(q, x), scale


def _exact_noise(seed, step, tensor, j):
    def mix(x):
        x = x ^ (x // 2 ** 16)
        x = x * 0x7FEB352D % 2 ** 32
        x = x ^ (x // 2 ** 15)
        x = x * 0x846CA68B % 2 ** 32
        return x ^ (x // 2 ** 16)

    key = mix(mix((mix((seed + 0x9E3779B9 * step) % 2 ** 32) + tensor) % 2 ** 32))
    x = (mix((j // 16) ^ key) + (j % 16) * 0x9E3779B9) % 2 ** 32
    x = x * 0x7FEB352D % 2 ** 32
    x = x ^ (x // 2 ** 15)
    x = x * 0x846CA68B % 2 ** 32
    return x ^ (x // 2 ** 16)
