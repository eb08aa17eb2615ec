"""Measured cases of what a training step needs around the vocabulary-sharded
ends of a model: the root-mean-square norm with the residual's addition (its
output as it is or in 8 bits with scales, and its gradient), the norm of all
gradients with the clipping factor, and the AdamW step over many tensors with
its states in 32 bits or in 8.

``listed()`` gives the cases that are always measured, ``draw(rng)`` one more
of the same ranges.  ``prepare(case, seed)`` makes on the GPU what a program
holds before the call, ``run(state)`` makes one call: the library's kernels
where ``own`` is true, elementary torch operations in fp32 otherwise.
``exact(case, seed)`` gives the same outputs from the definitions in fp64.

Definitions (row i, column c, h columns):
    norm:   r = x + residual, rstd = (mean_c r^2 + eps)^(-1/2), y = r rstd w;
            the sum r, rounded to its type, and rstd are outputs too
    in 8 bits: per group of G columns (G = 0: the row) scale = max |y| / 448,
            at least 2^-126, and q = e4m3(y / scale)
    gradient, from the stored r: dr = dresidual + rstd (w dy - r rstd^2 mean_c
            (w dy r)), dw = sum_i dy r rstd
    gradient norm: N = sqrt(sum g^2) over all tensors, factor min(1, max / N),
            0 where N is not finite
    AdamW with g = factor * gradient, step t:
            m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
            p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
            and a bf16 copy of p where one is kept
    states in 8 bits: m and sqrt(v) as e4m3 codes with a scale per 256
            consecutive elements of a tensor, scale = max / 448 (at least
            2^-126).  A value between two neighbouring codes' values lo and hi
            takes hi where (u + 1/2) / 2^16 < (x - lo) / (hi - lo), with u the
            element's 16 random bits; for sqrt(v) the three are squared, and a
            value above 0 takes at least the code 1.  u is half k % 8 (low
            halves first) of the Philox4x32-10 block with key (seed) and
            counter (k / 8, tensor's position, offset) for element k.
"""
import math

import torch

own = False

EPS_NORM = 1e-5
LR, EPS_ADAM, DECAY = 3e-5, 1e-8, 0.1
BLOCK = 256
TINY = 2.0 ** -126


def listed():
    return [
        # one new token of a served model (the hidden size of the repository's
        # s8192_v128256 head): latency counts
        dict(name="norm 1x8192", op="norm", s=1, h=8192, dtype="bf16", residual="bf16", weight="bf16", pad=0),
        # the norm in front of the head over the repository's training batch
        dict(name="norm 8192x8192", op="norm", s=8192, h=8192, dtype="bf16", residual="bf16", weight="bf16", pad=0),
        # a decode batch whose next product runs in 8 bits, one scale per token
        dict(name="norm8 64x8192 row", op="norm8", s=64, h=8192, dtype="bf16", residual="bf16", weight="bf16", pad=0,
             group=0),
        # the same batch as the second case, in 8 bits with a scale per 128 columns
        dict(name="norm8 8192x8192 g128", op="norm8", s=8192, h=8192, dtype="bf16", residual="bf16", weight="bf16",
             pad=0, group=128),
        # a longer batch of a small odd model in fp32 (rows off 16 bytes), no residual stream
        dict(name="dnorm 30001x515 odd f32", op="dnorm", s=30001, h=515, dtype="fp32", residual="none",
             weight="fp32", pad=0),
        # the training batch's backward, the residual stream's gradient added
        dict(name="dnorm 8192x8192", op="dnorm", s=8192, h=8192, dtype="bf16", residual="bf16", weight="bf16", pad=0),
        # a small model's gradients, 48 tensors of odd sizes
        dict(name="gradnorm 8 layers 257", op="gradnorm", kind="layers", layers=8, h=257, param="fp32", grad="fp32",
             copy=False, bits=32, clip=True, b2=0.95),
        # the head's gradient: V = 128256 in four shards, h = 4096
        dict(name="gradnorm 128256x4096", op="gradnorm", kind="shards", V=128256, t=4, h=4096, param="fp32",
             grad="fp32", copy=False, bits=32, clip=True, b2=0.95),
        # the step of the small odd model, bf16 weights and gradients: latency and many tensors
        dict(name="adamw 8 layers 257 bf16", op="adamw", kind="layers", layers=8, h=257, param="bf16", grad="bf16",
             copy=False, bits=32, clip=True, b2=0.95),
        # the step of the head's table: fp32 weights, the bf16 copy that the head reads
        dict(name="adamw 128256x4096", op="adamw", kind="shards", V=128256, t=4, h=4096, param="fp32", grad="fp32",
             copy=True, bits=32, clip=True, b2=0.95),
        # 8-bit states of a model of 72 tensors with bf16 gradients
        dict(name="adamw8 12 layers 512", op="adamw", kind="layers", layers=12, h=512, param="fp32", grad="bf16",
             copy=True, bits=8, clip=True, b2=0.999),
        # 8-bit states of a table of the repository's s4096_v50304 vocabulary
        dict(name="adamw8 50304x4096", op="adamw", kind="shards", V=50304, t=8, h=4096, param="fp32", grad="fp32",
             copy=True, bits=8, clip=True, b2=0.95),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm8", "dnorm", "gradnorm", "adamw", "adamw", "adamw"])
    if op in ("norm", "norm8", "dnorm"):
        h = log_int(64, 16384)
        h += rng.choice([0, (-h) % 64, (-h) % 64])
        s = log_int(1, min(32768, 67_000_000 // h))
        dtype, residual = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "fp32"), ("bf16", "none"),
                                      ("fp32", "fp32"), ("fp32", "none")])
        case = dict(op=op, s=s, h=h, dtype=dtype, residual=residual, weight=rng.choice(["bf16", "fp32"]),
                    pad=rng.choice([0, 0, 64, 1]))
        if op == "norm8":
            case["group"] = rng.choice([0, 64, 128])
        return case
    case = dict(op=op, kind=rng.choice(["layers", "shards"]))
    if case["kind"] == "layers":
        h = log_int(32, 1024)
        case.update(layers=log_int(1, min(24, 1 + 200_000_000 // (11 * h * h))), h=h)
    else:
        h = log_int(64, 8192)
        case.update(V=log_int(1000, min(256000, 200_000_000 // h)), t=rng.choice([1, 2, 3, 8]), h=h)
    param = rng.choice(["fp32", "fp32", "bf16"])
    case.update(param=param, grad=rng.choice(["fp32", "bf16"]), copy=param == "fp32" and rng.random() < 0.5,
                bits=rng.choice([32, 8]), clip=rng.random() < 0.7, b2=rng.choice([0.95, 0.999]))
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows(s, h, pad, dtype, gen, std):
    """[s, h] values in rows of h + pad elements."""
    full = torch.empty(s, h + pad, dtype=dtype, device="cuda")
    full.normal_(0.0, std, generator=gen)
    return full[:, :h]


def _shapes(case):
    """The tensors of a model: (elements, weight decay) of each."""
    h = case["h"]
    if case["kind"] == "layers":
        # a gain, two products in, one out, a gain, the wide pair
        layer = [(h, 0.0), (2 * h * h, DECAY), (h * h, DECAY), (h, 0.0), (4 * h * h, DECAY), (4 * h * h, DECAY)]
        return layer * case["layers"]
    V, t = case["V"], case["t"]
    vs = [0] + [(i * V) // t + (i % 2 if V % t else 0) for i in range(1, t)] + [V]
    return [((vs[i + 1] - vs[i]) * h, DECAY) for i in range(t)]


def _padded(n):
    return -(-n // BLOCK) * BLOCK


def _codes(x):
    """Nearest e4m3 codes of non-negative or signed values, and the scales."""
    b = x.view(-1, BLOCK)
    scale = (b.abs().amax(1) / 448.0).clamp(min=TINY)
    return (b / scale[:, None]).to(torch.float8_e4m3fn).view(-1), scale


def _model(case, gen):
    """Weights, gradients and states of a model in flat buffers, as a program
    that is in its 1000th step has them; each tensor starts at a multiple of
    256 elements, and what lies between tensors is 0."""
    shapes = _shapes(case)
    sizes = [n for n, _ in shapes]
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _padded(n))
    total = starts[-1]
    st = dict(case=case, sizes=sizes, starts=starts, decays=[wd for _, wd in shapes],
              decay=torch.tensor([wd for _, wd in shapes], device="cuda"),
              padded=torch.tensor([_padded(n) for n in sizes], device="cuda"),
              step=torch.full((1,), 1000, dtype=torch.int64, device="cuda"),
              rng=torch.randint(0, 1 << 62, (2,), device="cuda", generator=gen),
              factor=torch.full((1,), 0.7, device="cuda") if case["clip"] else None)
    p = torch.empty(total, device="cuda").normal_(0.0, 0.02, generator=gen)
    g = torch.empty(total, device="cuda").normal_(0.0, 1e-3, generator=gen)
    m = torch.empty(total, device="cuda").normal_(0.0, 3e-4, generator=gen)
    v = torch.empty(total, device="cuda").uniform_(0.2, 2.0, generator=gen).mul_(1e-6)
    for n, a, e in zip(sizes, starts, starts[1:]):
        for x in (p, g, m, v):
            x[a + n:e] = 0.0
    st["p"], st["g"] = p.to(_dtype(case["param"])), g.to(_dtype(case["grad"]))
    st["copy"] = p.to(torch.bfloat16) if case["copy"] else None
    if case["bits"] == 32:
        st.update(m=m, v=v)
    else:
        st["m"], st["m_scale"] = _codes(m)
        st["v"], st["v_scale"] = _codes(v.sqrt_())
    return st


def _views(st, name, per=1):
    """The tensors of a flat buffer (per: elements that one entry stands for)."""
    return [st[name][a // per:-(-(a + n) // per)] for n, a in zip(st["sizes"], st["starts"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("gradnorm", "adamw"):
        st = _model(case, gen)
        if own:  # the handle that such a program keeps: the tensors' addresses and sizes
            from vocab_sharded_lm_gb300 import vpce
            states = dict(exp_avg=_views(st, "m"), exp_avg_sq=_views(st, "v"))
            if case["bits"] == 8:
                states.update(exp_avg_scale=_views(st, "m_scale", BLOCK), exp_avg_sq_scale=_views(st, "v_scale", BLOCK))
            st["plan"] = vpce.vpce_adamw_plan(_views(st, "p"), _views(st, "g"),
                                              copies=_views(st, "copy") if case["copy"] else None,
                                              weight_decay=st["decays"], state_bits=case["bits"], **states)
        return st
    s, h, pad = case["s"], case["h"], case["pad"]
    dt = _dtype(case["dtype"])
    rdt = dt if case["residual"] == "none" else _dtype(case["residual"])
    w = torch.empty(h, device="cuda").normal_(1.0, 0.1, generator=gen).to(_dtype(case["weight"]))
    st = dict(case=case, w=w)
    if op == "dnorm":
        st["x"] = _rows(s, h, pad, rdt, gen, 2.0)
        st["dy"] = _rows(s, h, pad, dt, gen, 1e-3)
        st["dres"] = None if case["residual"] == "none" else _rows(s, h, pad, rdt, gen, 1e-3)
        st["rstd"] = (st["x"].double().square().mean(1) + EPS_NORM).rsqrt().float()
        st["dx"] = torch.empty(s, h, dtype=rdt, device="cuda")
        st["dw"] = torch.empty(h, device="cuda")
        return st
    st["x"] = _rows(s, h, pad, dt, gen, 1.0)
    st["res"] = None if case["residual"] == "none" else _rows(s, h, pad, rdt, gen, 2.0)
    st["sum"] = None if case["residual"] == "none" else torch.empty(s, h, dtype=rdt, device="cuda")
    st["rstd"] = torch.empty(s, device="cuda")
    if op == "norm":
        st["y"] = torch.empty(s, h, dtype=dt, device="cuda")
    else:
        st["q"] = torch.empty(s, h, dtype=torch.float8_e4m3fn, device="cuda")
        st["scale"] = torch.empty(s, -(-h // (case["group"] or h)), device="cuda")
    return st


# ---------------------------------------------------------------------------
# the plain forms (fp32) and the library's calls
# ---------------------------------------------------------------------------
def _plain_norm(st):
    case = st["case"]
    r = st["x"].float()
    out = {}
    if st["res"] is not None:
        r = r + st["res"].float()
        out["sum"] = r.to(st["res"].dtype)
    rstd = (r.square().mean(1) + EPS_NORM).rsqrt()
    out["rstd"] = rstd
    y = r * rstd[:, None] * st["w"].float()
    if case["op"] == "norm":
        out["y"] = y.to(st["x"].dtype)
        return out
    s, h = y.shape
    group = case["group"] or h
    groups = -(-h // group)
    y = torch.nn.functional.pad(y, (0, groups * group - h)).view(s, groups, group)
    scale = (y.abs().amax(2) / 448.0).clamp(min=TINY)
    out["scale"] = scale
    out["q"] = (y / scale[:, :, None]).view(s, groups * group)[:, :h].to(torch.float8_e4m3fn)
    return out


def _plain_dnorm(st):
    r, dy, rstd = st["x"].float(), st["dy"].float(), st["rstd"][:, None]
    wdy = dy * st["w"].float()
    n = r * rstd
    dx = rstd * (wdy - n * (wdy * n).mean(1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(st["x"].dtype), "dw": (dy * n).sum(0)}


def _plain_gradnorm(st):
    norm = st["g"].float().square().sum(dtype=torch.float64).sqrt()
    factor = torch.where(norm.isfinite(), (1.0 / norm).clamp(max=1.0), 0.0)
    return {"norm": norm.float(), "factor": factor.float()}


def _philox_halves(c0, c1, rng):
    """The 8 random 16-bit values of each counter (c0, c1, offset)."""
    M32 = 0xFFFFFFFF
    k0, k1 = rng[0] & M32, (rng[0] >> 32) & M32
    c2, c3 = rng[1] & M32, (rng[1] >> 32) & M32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & M32) ^ c1 ^ k0, p1 & M32, ((p0 >> 32) & M32) ^ c3 ^ k1, p0 & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16],
                       dim=1).view(-1, BLOCK)


def _e4m3(code):
    return code.to(torch.uint8).view(torch.float8_e4m3fn).float()


def _round_up(a, u, power):
    """e4m3 codes of 0 <= a <= 448, rounded up where the random bits say so."""
    code = torch.where(a >= 2.0 ** -6, (a.view(torch.int32) >> 20) - 960, (a * 512.0).int()).clamp(max=126)
    lo, hi = _e4m3(code).pow(power), _e4m3(code + 1).pow(power)
    up = (u.float() + 0.5) < (a.pow(power) - lo) / (hi - lo) * 65536.0
    return code + (up & (code < 126)).int()


def _plain_adamw(st):
    case = st["case"]
    b1, b2 = 0.9, case["b2"]
    t = st["step"].double()
    bias1, bias2 = (1.0 - b1 ** t).float(), (1.0 - b2 ** t).float()
    g = st["g"].float()
    if st["factor"] is not None:
        g = g * st["factor"]
    if case["bits"] == 32:
        m, v = st["m"], st["v"]
    else:
        m = (st["m"].float().view(-1, BLOCK) * st["m_scale"][:, None]).view(-1)
        v = (st["v"].float().view(-1, BLOCK) * st["v_scale"][:, None]).view(-1).square()
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    keep = torch.repeat_interleave(1.0 - LR * st["decay"], st["padded"], output_size=g.numel())
    p = st["p"].float() * keep - (LR / bias1) * (m / ((v / bias2).sqrt() + EPS_ADAM))
    st["p"].copy_(p)
    out = {"p": st["p"], "m": st["m"], "v": st["v"]}
    if case["copy"]:
        st["copy"].copy_(p)
        out["copy"] = st["copy"]
    if case["bits"] == 32:
        st["m"].copy_(m)
        st["v"].copy_(v)
        return out
    groups = st["padded"] // 8
    tensor = torch.repeat_interleave(torch.arange(groups.numel(), device="cuda"), groups, output_size=g.numel() // 8)
    first = (groups.cumsum(0) - groups)[tensor]
    u = _philox_halves(torch.arange(g.numel() // 8, device="cuda") - first, tensor, st["rng"])
    m, r = m.view(-1, BLOCK), v.sqrt().view(-1, BLOCK)
    m_scale = (m.abs().amax(1) / 448.0).clamp(min=TINY)
    r_scale = (r.amax(1) / 448.0).clamp(min=TINY)
    mc = _round_up(m.abs() / m_scale[:, None], u, 1) + torch.where(m < 0, 128, 0)
    rc = torch.maximum(_round_up(r / r_scale[:, None], u, 2), (r > 0).int())
    st["m"].copy_(mc.to(torch.uint8).view(torch.float8_e4m3fn).view(-1))
    st["v"].copy_(rc.to(torch.uint8).view(torch.float8_e4m3fn).view(-1))
    st["m_scale"].copy_(m_scale)
    st["v_scale"].copy_(r_scale)
    out.update(m_scale=st["m_scale"], v_scale=st["v_scale"])
    return out


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "norm8": _plain_norm, "dnorm": _plain_dnorm, "gradnorm": _plain_gradnorm,
                "adamw": _plain_adamw}[op](st)
    from vocab_sharded_lm_gb300 import vpce
    if op == "norm":
        r = vpce.vpce_rmsnorm_forward(st["x"], st["w"], st["res"], eps=EPS_NORM, out=st["y"], residual_out=st["sum"],
                                      rstd_out=st["rstd"])
        out = {"rstd": r.rstd, "y": r.out}
        if st["res"] is not None:
            out["sum"] = r.residual
        return out
    if op == "norm8":
        r = vpce.vpce_rmsnorm_quantized_forward(st["x"], st["w"], st["res"], eps=EPS_NORM, group=case["group"],
                                                q_out=st["q"], scale_out=st["scale"], residual_out=st["sum"],
                                                rstd_out=st["rstd"])
        out = {"rstd": r.rstd, "q": r.q, "scale": r.scale}
        if st["res"] is not None:
            out["sum"] = r.residual
        return out
    if op == "dnorm":
        dx, dw = vpce.vpce_rmsnorm_backward(st["dy"], st["x"], st["w"], st["rstd"], grad_residual=st["dres"],
                                            grad_in=st["dx"], grad_weight=st["dw"])
        return {"dx": dx, "dw": dw}
    if op == "gradnorm":
        norm, factor = vpce.vpce_grad_norm(st["plan"], 1.0)
        return {"norm": norm, "factor": factor}
    vpce.vpce_adamw_step(st["plan"], st["step"], lr=LR, betas=(0.9, case["b2"]), eps=EPS_ADAM,
                         grad_scale=st["factor"], rng=st["rng"] if case["bits"] == 8 else None)
    out = {k: st[k] for k in ("p", "m", "v")}
    if case["copy"]:
        out["copy"] = st["copy"]
    if case["bits"] == 8:
        out.update(m_scale=st["m_scale"], v_scale=st["v_scale"])
    return out


# ---------------------------------------------------------------------------
# floors
# ---------------------------------------------------------------------------
def work(case):
    size = {"bf16": 2, "fp32": 4, "none": 0}
    op, h = case["op"], case["h"]
    if op in ("gradnorm", "adamw"):
        n = float(sum(n for n, _ in _shapes(case)))
        if op == "gradnorm":
            return {"bytes": n * size[case["grad"]], "flops": 2.0 * n}
        state = 8.0 if case["bits"] == 32 else 2.0 + 8.0 / BLOCK
        # gradients read; weights and states read and written; the copy written
        per = size[case["grad"]] + 2 * size[case["param"]] + 2 * state + (2 if case["copy"] else 0)
        return {"bytes": n * per, "flops": 16.0 * n}
    s, b, r, w = case["s"], size[case["dtype"]], size[case["residual"]], size[case["weight"]] * h
    if op == "dnorm":
        rr = r or b
        # dy and the sum read, the residual stream's gradient read, dx written, dw written
        return {"bytes": float(s * h * (b + rr + r + rr) + 4 * s + w + 4 * h), "flops": 10.0 * s * h}
    read, kept = s * h * (b + r) + w, s * h * r + 4 * s
    out = s * h * b if op == "norm" else s * (h + 4 * -(-h // (case["group"] or h)))
    return {"bytes": float(read + kept + out), "flops": 5.0 * s * h}


# ---------------------------------------------------------------------------
# the same outputs in fp64
# ---------------------------------------------------------------------------
def _grid():
    """The 127 finite non-negative e4m3 values in order, and the largest once more."""
    v = [k * 2.0 ** -9 for k in range(8)] + [(8 + k) * 2.0 ** (e - 10) for e in range(1, 16) for k in range(8)]
    return torch.tensor(v[:127] + [v[126]], dtype=torch.float64, device="cuda")


def _exact_codes(x, u, squared):
    """Values of the codes that |x| takes, x and u [blocks, 256], and the scales."""
    grid = _grid()
    top = x.abs().max(dim=1).values
    scale = torch.maximum(top / 448, torch.full_like(top, TINY))
    a = x.abs() / scale[:, None]
    at = (torch.searchsorted(grid[:127], a, right=True) - 1).clamp(min=0, max=126)
    lo, hi = grid[at], grid[at + 1]
    part = (a * a - lo * lo) / (hi * hi - lo * lo) if squared else (a - lo) / (hi - lo)
    c = torch.where((at < 126) & ((u + 0.5) / 65536 < part), hi, lo)
    if squared:
        c = torch.where(x > 0, c.clamp(min=grid[1].item()), c)
    return torch.copysign(c, x), scale


def _exact_halves(n, tensor, rng):
    """16 random bits of n elements of one tensor, products on 16-bit limbs."""
    seed, offset = (int(v) % (1 << 64) for v in rng.tolist())

    def mul(a, const):
        lo, hi = (a % 65536) * const, (a // 65536) * const
        mid = hi % 65536 * 65536 + lo
        return hi // 65536 + mid // (1 << 32), mid % (1 << 32)

    k = torch.arange(n // 8, device="cuda")
    x = [k, torch.full_like(k, tensor), torch.full_like(k, offset % (1 << 32)), torch.full_like(k, offset >> 32)]
    ka, kb = seed % (1 << 32), seed >> 32
    for i in range(10):
        h0, l0 = mul(x[0], 3528531795)
        h1, l1 = mul(x[2], 3449720151)
        a, b = (ka + i * 2654435769) % (1 << 32), (kb + i * 3144134277) % (1 << 32)
        x = [h1 ^ x[1] ^ a, l1, h0 ^ x[3] ^ b, l0]
    bits = torch.empty(n // 8, 8, dtype=torch.int64, device="cuda")
    for j in range(8):
        bits[:, j] = (x[j // 2] // (65536 if j % 2 else 1)) % 65536
    return bits.view(-1, BLOCK)


def _exact_adamw(st):
    case = st["case"]
    total, t = st["starts"][-1], int(st["step"].item())
    c1, c2 = 1 - 0.9 ** t, 1 - case["b2"] ** t
    factor = 1.0 if st["factor"] is None else float(st["factor"].item())
    out = {k: torch.zeros(total, dtype=torch.float64, device="cuda") for k in ("p", "m", "v")}
    if case["bits"] == 8:
        out.update({k: torch.zeros(total // BLOCK, dtype=torch.float64, device="cuda") for k in ("m_scale", "v_scale")})
    for i, (a, e) in enumerate(zip(st["starts"], st["starts"][1:])):
        g, m, v = st["g"][a:e].double() * factor, st["m"][a:e].double(), st["v"][a:e].double()
        if case["bits"] == 8:
            of = slice(a // BLOCK, e // BLOCK)
            m = (m.view(-1, BLOCK) * st["m_scale"][of, None].double()).view(-1)
            v = (v.view(-1, BLOCK) * st["v_scale"][of, None].double()).view(-1) ** 2
        m, v = 0.9 * m + (1 - 0.9) * g, case["b2"] * v + (1 - case["b2"]) * g * g
        old = st["p"][a:e].double()
        out["p"][a:e] = old - LR * st["decays"][i] * old - LR * (m / c1) / (torch.sqrt(v / c2) + EPS_ADAM)
        if case["bits"] == 32:
            out["m"][a:e], out["v"][a:e] = m, v
            continue
        u = _exact_halves(e - a, i, st["rng"])
        for k, x, sq in (("m", m, False), ("v", torch.sqrt(v), True)):
            c, scale = _exact_codes(x.view(-1, BLOCK), u, sq)
            out[k][a:e], out[k + "_scale"][of] = c.view(-1), scale
    if case["copy"]:
        out["copy"] = out["p"]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(st)
    if op == "gradnorm":
        norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in _views(st, "g")))
        return {"norm": torch.tensor(norm, dtype=torch.float64),
                "factor": torch.tensor(min(1.0, 1.0 / norm), dtype=torch.float64)}
    w, h = st["w"].double(), case["h"]
    if op == "dnorm":
        n = st["x"].double() * st["rstd"].double()[:, None]
        gy = st["dy"].double()
        along = torch.einsum("sh,sh,h->s", gy, n, w) / h
        dx = st["rstd"].double()[:, None] * (gy * w - along[:, None] * n)
        return {"dx": dx if st["dres"] is None else dx + st["dres"].double(), "dw": torch.einsum("sh,sh->h", gy, n)}
    r = st["x"].double() if st["res"] is None else st["x"].double() + st["res"].double()
    rstd = 1 / torch.sqrt(torch.einsum("sh,sh->s", r, r) / h + EPS_NORM)
    y = torch.einsum("sh,s,h->sh", r, rstd, w)
    out = {"rstd": rstd, "y": y} if op == "norm" else {"rstd": rstd}
    if st["res"] is not None:
        out["sum"] = r
    if op == "norm8":
        group = case["group"] or h
        parts = y.split(group, dim=1)
        scale = torch.stack([q.abs().max(dim=1).values / 448 for q in parts], dim=1)
        out["scale"] = torch.maximum(scale, torch.full_like(scale, TINY))
        a = torch.cat([q / out["scale"][:, j:j + 1] for j, q in enumerate(parts)], dim=1)
        grid = _grid()[:127]
        at = torch.searchsorted((grid[1:] + grid[:-1]) / 2, a.abs())
        out["q"] = torch.copysign(grid[at], a)
    return out
