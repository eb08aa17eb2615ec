"""Measured cases of the token scores (log probabilities, entropy, top
alternatives, and their gradient) and of the scaled embedding with dropout.

``listed()`` gives the cases that are always measured, ``draw(rng)`` one more
of the same ranges.  ``prepare(case, seed)`` makes on the GPU what a program
holds before the call, ``run(state)`` makes one call: the library's kernels
where ``own`` is true, elementary torch operations in fp32 otherwise.
``exact(case, seed)`` gives the same outputs from the definitions in fp64.

Definitions (row r, column k, temperature T, V columns in t shards):
    x_k = z_rk / T,  lse = log sum_k exp(x_k),  p_k = exp(x_k - lse)
    logp = x_y - lse,  entropy = -sum_k p_k log p_k,
    top: the `top` columns of largest z (ties: lowest column first) and x - lse
    dz_k = (g_logp ([k = y] - p_k) + sum_j g_top_j ([k = id_j] - p_k)
            - g_entropy p_k (log p_k + entropy)) / T
Rows whose target is -100 have logp, entropy and top log probabilities 0, top
ids -1 and zero gradients.
Embedding: out_rc = scale m_rc E[id_r, c]; the gradient of table row v is the
sum over r with id_r = v of scale m_rc g_rc; ids equal to the padding id give
zero rows and no gradient.  m_rc = 65536 / (65536 - D) or 0 with
D = round(65536 p): 0 where the 16-bit half c % 8 (low halves first) of the
Philox4x32-10 block with key (seed) and counter (c / 8, r, offset) is < D.
"""
import math

import numpy as np
import torch

own = False

IGNORE = -100


def listed():
    return [
        # one new token of a served model scored with its 20 best alternatives
        # (the repository's s8192_v128256 head): latency counts
        dict(name="logprob 1x128256 top20", op="logprob", s=1, V=128256, t=8, dtype="bf16", top=20, layout="dense",
             ignored=0, banned=0, temperature=1.0),
        # a decode batch: one token of each of 64 sequences, sampled at a temperature
        dict(name="logprob 64x128256 top5", op="logprob", s=64, V=128256, t=8, dtype="bf16", top=5, layout="dense",
             ignored=0, banned=512, temperature=0.7),
        # the repository's tiny workload: fp32 logits of 64 rows
        dict(name="logprob 64x1000 f32 top8", op="logprob", s=64, V=1000, t=2, dtype="fp32", top=8, layout="dense",
             ignored=4, banned=0, temperature=1.0),
        # uneven shards as column blocks of one odd-width tensor (rows and
        # shards off 16 bytes), a constrained vocabulary, greedy token only
        dict(name="logprob 1021x50259 odd top1", op="logprob", s=1021, V=50259, t=3, dtype="bf16", top=1,
             layout="columns", ignored=100, banned=20000, temperature=1.3),
        # scoring a training batch: the s8192_v128256 logits, the prompt's rows ignored
        dict(name="logprob 8192x128256 top20", op="logprob", s=8192, V=128256, t=8, dtype="bf16", top=20,
             layout="dense", ignored=512, banned=0, temperature=1.0),
        # fp32 logits as the s16384_v152064 workload has them, a quarter of its rows, the longest list
        dict(name="logprob 4096x152064 f32 top32", op="logprob", s=4096, V=152064, t=8, dtype="fp32", top=32,
             layout="dense", ignored=200, banned=0, temperature=1.0),
        # the policy-gradient step's backward over the same batch: log
        # probabilities and an entropy bonus
        dict(name="dlogprob 8192x128256", op="dlogprob", s=8192, V=128256, t=8, dtype="bf16", top=0, layout="dense",
             ignored=512, banned=0, temperature=1.0),
        # a distillation term on the top alternatives, odd sizes, fp32
        dict(name="dlogprob 515x50259 odd f32 top8", op="dlogprob", s=515, V=50259, t=3, dtype="fp32", top=8,
             layout="columns", ignored=50, banned=3000, temperature=1.3),
        # the input side of the same training batch (8192 tokens, hidden 8192), dropout 0.1
        dict(name="embed 8192x8192 drop", op="embed", s=8192, V=128256, t=8, h=8192, dtype="bf16", out="bf16", p=0.1,
             scale=90.5, pads=512),
        # a decode batch's lookup: no dropout, fp32 table, bf16 activations
        dict(name="embed 64x4096 f32 to bf16", op="embed", s=64, V=50304, t=4, h=4096, dtype="fp32", out="bf16",
             p=0.0, scale=64.0, pads=0),
        # the training batch's table gradient, Zipf ids, every table row written
        dict(name="dembed 8192x8192 drop", op="dembed", s=8192, V=128256, t=8, h=8192, dtype="bf16", p=0.1,
             scale=90.5, pads=512),
        # a longer batch on a small odd model, fp32 gradients
        dict(name="dembed 30001x515 odd f32", op="dembed", s=30001, V=50259, t=3, h=515, dtype="fp32", p=0.25,
             scale=1.0, pads=1000),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["logprob", "logprob", "dlogprob", "embed", "dembed"])
    t = rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    eb = 2 if dtype == "bf16" else 4
    if op in ("logprob", "dlogprob"):
        V = log_int(1000, 256000)
        V += rng.choice([0, (-V) % 64, (-V) % 64])
        s = log_int(1, min(16384, 2_000_000_000 // (V * eb)))
        return dict(op=op, s=s, V=V, t=t, dtype=dtype, top=rng.choice([0, 1, 5, 8, 20, 32]),
                    layout=rng.choice(["dense", "columns"]), ignored=rng.choice([0, s // 16]),
                    banned=rng.choice([0, V // 50, V // 3]), temperature=rng.choice([1.0, 0.6, 1.5]))
    h = log_int(64, 8192)
    h += rng.choice([0, (-h) % 64, (-h) % 64])
    s = log_int(1, min(32768, 66_000_000 // h))
    V = log_int(1000, min(256000, 1_000_000_000 // h))
    case = dict(op=op, s=s, V=V, t=t, h=h, dtype=dtype, p=rng.choice([0.0, 0.1, 0.3]), scale=rng.choice([1.0, 22.6]),
                pads=rng.choice([0, s // 16]))
    if op == "embed":
        case["out"] = rng.choice(["bf16", "fp32"])
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _starts(V, t):
    """t shards; an odd vocabulary is split unevenly."""
    if V % t == 0:
        return [i * (V // t) for i in range(t + 1)]
    return [0] + [(i * V) // t + (i % 2) for i in range(1, t)] + [V]


def _zipf_ids(s, V, gen):
    """Token ids with P(rank k) ~ k^-1.1 (natural text's spread)."""
    w = torch.arange(1, V + 1, device="cuda", dtype=torch.float64).pow(-1.1).cumsum(0)
    u = torch.rand(s, device="cuda", dtype=torch.float64, generator=gen) * w[-1]
    return torch.searchsorted(w, u).clamp_(max=V - 1)


def _logits(case, gen):
    """Logits of a trained head: noise of deviation 3, the target's raised
    in a third of the rows, banned columns at -inf."""
    s, V, t = case["s"], case["V"], case["t"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    vs = _starts(V, t)
    y = torch.randint(0, V, (s,), device="cuda", generator=gen)
    ban = torch.zeros(V, dtype=torch.bool, device="cuda")
    if case["banned"]:
        ban[torch.randperm(V, device="cuda", generator=gen)[: case["banned"]]] = True
        ban[y] = False
    full = torch.empty(s, V, dtype=dt, device="cuda")
    full.normal_(0.0, 3.0, generator=gen)
    full.masked_fill_(ban, float("-inf"))
    rows = torch.arange(0, s, 3, device="cuda")
    full[rows, y[rows]] += 12.0
    if case["ignored"]:
        y[torch.randperm(s, device="cuda", generator=gen)[: case["ignored"]]] = IGNORE
    if case["layout"] == "columns":
        return full, list(full.split([vs[i + 1] - vs[i] for i in range(t)], dim=1)), vs, y
    return None, [full[:, vs[i]:vs[i + 1]].contiguous() for i in range(t)], vs, y


def _row_stats(shards, y, inv_t):
    """What the forward leaves for the backward: per row the largest logit,
    the log of the sum of exp((z - max) / T), the entropy, and 0."""
    z = torch.cat(shards, dim=1) if len(shards) > 1 else shards[0]
    out = torch.zeros(z.shape[0], 4, device="cuda")
    for r in range(0, z.shape[0], 1024):
        x = z[r:r + 1024].double()
        m = x.amax(1)
        u = (x - m[:, None]).mul_(inv_t)
        e = u.exp()
        S = e.sum(1)
        T = torch.where(e > 0, u * e, 0.0).sum(1)
        out[r:r + 1024, 0] = m.float()
        out[r:r + 1024, 1] = S.log().float()
        out[r:r + 1024, 2] = (S.log() - T / S).float()
    out[y == IGNORE] = 0.0
    return out


def _top_ids(z, top):
    """Columns of the `top` largest values of each row, largest first, equal
    values in column order."""
    zf = z.float()
    b = torch.where(zf == 0, 0.0, zf).view(torch.int32).long()
    key = torch.where(b >= 0, b, b ^ 0x7FFFFFFF) * (1 << 32)
    key += (1 << 32) - 1 - torch.arange(z.shape[1], device=z.device)
    return key.topk(top, dim=1, sorted=True).indices


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, s, V, t = case["op"], case["s"], case["V"], case["t"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    st = dict(case=case)
    if op in ("logprob", "dlogprob"):
        full, shards, vs, y = _logits(case, gen)
        top = case["top"]
        st.update(full=full, shards=shards, vs=vs, y=y)
        if op == "logprob":
            st["buffers"] = dict(
                logp_out=torch.empty(s, device="cuda"), entropy_out=torch.empty(s, device="cuda"),
                stats_out=torch.empty(s, 4, device="cuda"),
                top_ids_out=torch.empty(s, top, dtype=torch.int64, device="cuda") if top else None,
                top_logp_out=torch.empty(s, top, device="cuda") if top else None)
            return st
        st["stats"] = _row_stats(shards, y, 1.0 / case["temperature"])
        st["g_logp"] = torch.randn(s, device="cuda", generator=gen) / s
        st["g_entropy"] = torch.full((s,), -0.01 / s, device="cuda")
        st["top_ids"] = st["g_top"] = None
        if top:
            z = full if full is not None else torch.cat(shards, dim=1)
            ids = torch.cat([_top_ids(z[r:r + 1024], top) for r in range(0, s, 1024)])
            ids[y == IGNORE] = -1
            st["top_ids"] = ids
            st["g_top"] = torch.randn(s, top, device="cuda", generator=gen) / s
        grad = torch.empty(s, V, dtype=dt, device="cuda")
        st["grad"] = [grad[:, vs[i]:vs[i + 1]] if full is not None else torch.empty_like(shards[i]) for i in range(t)]
        return st
    h = case["h"]
    vs = _starts(V, t)
    ids = _zipf_ids(s, V, gen)
    st["padding"] = V - 1
    ids[ids == V - 1] = 0
    if case["pads"]:
        ids[torch.randperm(s, device="cuda", generator=gen)[: case["pads"]]] = V - 1
    st.update(vs=vs, ids=ids, rng=torch.randint(0, 1 << 62, (2,), device="cuda", generator=gen))
    if op == "embed":
        odt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        full = torch.empty(V, h, dtype=dt, device="cuda")
        full.normal_(0.0, 1.0 / math.sqrt(h), generator=gen)
        st.update(full=full, table=[full[vs[i]:vs[i + 1]] for i in range(t)],
                  out=torch.empty(s, h, dtype=odt, device="cuda"))
        return st
    g = torch.empty(s, h, dtype=dt, device="cuda")
    g.normal_(0.0, 1.0, generator=gen)
    st["g"] = g
    st["grads"] = [torch.empty(vs[i + 1] - vs[i], h, device="cuda") for i in range(t)]
    return st


# ---------------------------------------------------------------------------
# the plain forms (fp32) and the library's calls
# ---------------------------------------------------------------------------
def _philox_keep(rows, h, p, rng):
    """Keep mask [rows, h] of the dropout (Philox4x32-10, 16 bits a value)."""
    drop = int(math.floor(p * 65536 + 0.5))
    M32 = 0xFFFFFFFF
    nb = (h + 7) // 8
    k0, k1 = rng[0] & M32, (rng[0] >> 32) & M32
    c0 = torch.arange(nb, device="cuda")[None, :].expand(rows, nb)
    c1 = torch.arange(rows, device="cuda")[:, None].expand(rows, nb)
    c2, c3 = rng[1] & M32, (rng[1] >> 32) & M32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & M32) ^ c1 ^ k0, p1 & M32, ((p0 >> 32) & M32) ^ c3 ^ k1, p0 & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    halves = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16],
                         dim=2)
    return halves.view(rows, nb * 8)[:, :h] >= drop


def _mask(case, st):
    """The dropout's factor per element, 1 without dropout."""
    if case["p"] == 0:
        return 1.0
    drop = int(math.floor(case["p"] * 65536 + 0.5))
    return _philox_keep(case["s"], case["h"], case["p"], st["rng"]).float() * (65536.0 / (65536 - drop))


def _plain_logprob(st):
    case = st["case"]
    top, inv_t, y = case["top"], 1.0 / case["temperature"], st["y"]
    z = st["full"] if st["full"] is not None else torch.cat(st["shards"], dim=1)
    zf = z.float()
    m = zf.amax(1)
    u = (zf - m[:, None]) * inv_t
    e = u.exp()
    S = e.sum(1)
    log_s = S.log()
    valid = y != IGNORE
    logp = u.gather(1, y.clamp(min=0)[:, None])[:, 0] - log_s
    entropy = log_s - torch.where(e > 0, u * e, 0.0).sum(1) / S
    out = dict(logp=torch.where(valid, logp, 0.0), entropy=torch.where(valid, entropy, 0.0),
               stats=torch.where(valid[:, None], torch.stack([m, log_s, entropy, torch.zeros_like(m)], 1), 0.0))
    if top:
        ids = _top_ids(z, top)
        out["top_logp"] = torch.where(valid[:, None], u.gather(1, ids) - log_s[:, None], 0.0)
        out["top_ids"] = torch.where(valid[:, None], ids, -1)
    return out


def _plain_dlogprob(st):
    case = st["case"]
    top, inv_t, y = case["top"], 1.0 / case["temperature"], st["y"]
    z = st["full"] if st["full"] is not None else torch.cat(st["shards"], dim=1)
    m, log_s, ent = st["stats"][:, 0:1], st["stats"][:, 1:2], st["stats"][:, 2:3]
    lp = (z.float() - m) * inv_t - log_s
    p = lp.exp()
    valid = (y != IGNORE)[:, None]
    gl, ge = st["g_logp"][:, None], st["g_entropy"][:, None]
    weight = gl + st["g_top"].sum(1, keepdim=True) if top else gl
    d = -p * weight - torch.where(p > 0, p * (lp + ent), 0.0) * ge
    d.scatter_add_(1, y.clamp(min=0)[:, None], gl)
    if top:
        d.scatter_add_(1, st["top_ids"].clamp(min=0), st["g_top"])
    d = torch.where(valid, d * inv_t, 0.0).to(z.dtype)
    return list(d.split([st["vs"][i + 1] - st["vs"][i] for i in range(case["t"])], dim=1))


def _plain_embed(st):
    case = st["case"]
    x = st["full"][st["ids"]].float()
    x = x * (_mask(case, st) * case["scale"])
    return torch.where((st["ids"] == st["padding"])[:, None], 0.0, x).to(st["out"].dtype)


def _plain_dembed(st):
    case = st["case"]
    g = st["g"].float() * (_mask(case, st) * case["scale"])
    g = torch.where((st["ids"] == st["padding"])[:, None], 0.0, g)
    full = torch.zeros(case["V"], case["h"], device="cuda").index_add_(0, st["ids"], g)
    return list(full.split([st["vs"][i + 1] - st["vs"][i] for i in range(case["t"])], dim=0))


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"logprob": _plain_logprob, "dlogprob": _plain_dlogprob, "embed": _plain_embed,
                "dembed": _plain_dembed}[op](st)
    from vocab_sharded_lm_gb300 import vpce
    if op == "logprob":
        r = vpce.vpce_logprob_forward(st["shards"], st["y"], st["vs"], ignore_index=IGNORE,
                                      temperature=case["temperature"], top=case["top"], **st["buffers"])
        out = dict(logp=r.logp, entropy=r.entropy, stats=r.stats)
        if case["top"]:
            out.update(top_ids=r.top_ids, top_logp=r.top_logp)
        return out
    if op == "dlogprob":
        return vpce.vpce_logprob_backward(st["shards"], st["y"], st["stats"], st["vs"], ignore_index=IGNORE,
                                          temperature=case["temperature"], grad_logp=st["g_logp"],
                                          grad_entropy=st["g_entropy"], top_ids=st["top_ids"],
                                          grad_top_logp=st["g_top"], grad_shards=st["grad"])
    rng = st["rng"] if case["p"] else None
    if op == "embed":
        return vpce.vpce_embedding_dropout_forward(st["table"], st["ids"], st["vs"], scale=case["scale"], p=case["p"],
                                                   rng=rng, padding_id=st["padding"], out=st["out"])
    return vpce.vpce_embedding_dropout_backward(st["g"], st["ids"], st["grads"], st["vs"], scale=case["scale"],
                                                p=case["p"], rng=rng, padding_id=st["padding"], accumulate=False)


# ---------------------------------------------------------------------------
# floors
# ---------------------------------------------------------------------------
def _distinct(s, V):
    """Expected number of distinct ids among s Zipf draws."""
    w = np.arange(1, V + 1, dtype=np.float64) ** -1.1
    return float(-np.expm1(s * np.log1p(-w / w.sum())).sum())


def work(case):
    s, V, op = case["s"], case["V"], case["op"]
    eb = 2 if case["dtype"] == "bf16" else 4
    if op in ("logprob", "dlogprob"):
        valid, top = s - case["ignored"], case["top"]
        if op == "logprob":
            # logits read; targets read; logp, entropy, statistics and alternatives written
            return {"bytes": valid * V * eb + s * (8 + 4 + 4 + 16 + 12 * top), "flops": 6.0 * valid * V}
        # logits of the valid rows read, every row's gradient written
        return {"bytes": valid * V * eb + s * V * eb + s * (8 + 16 + 8 + 12 * top), "flops": 8.0 * valid * V}
    h, live = case["h"], s - case["pads"]
    if op == "embed":
        ob = 2 if case["out"] == "bf16" else 4
        return {"bytes": s * h * ob + _distinct(live, V) * h * eb + 8 * s, "flops": float(live * h)}
    # gradient rows read, every table row written in fp32
    return {"bytes": live * h * eb + V * h * 4 + 8 * s, "flops": 2.0 * live * h}


# ---------------------------------------------------------------------------
# the same outputs in fp64
# ---------------------------------------------------------------------------
def _exact_factor(case, rng):
    """Dropout factors in fp64, the generator on 16-bit limbs."""
    s, h, p = case["s"], case["h"], case["p"]
    if p == 0:
        return 1.0
    seed, offset = (int(v) % (1 << 64) for v in rng.tolist())
    nb = -(-h // 8)

    def mul(a, const):
        """(high, low) 32 bits of a * const, a < 2^32, without 64-bit overflow"""
        lo, hi = (a % 65536) * const, (a // 65536) * const
        mid = hi % 65536 * 65536 + lo
        return hi // 65536 + mid // (1 << 32), mid % (1 << 32)

    shape = (s, nb)
    x = [torch.arange(nb, device="cuda").expand(shape), torch.arange(s, device="cuda")[:, None].expand(shape),
         torch.full(shape, offset % (1 << 32), device="cuda"), torch.full(shape, offset >> 32, device="cuda")]
    ka, kb = seed % (1 << 32), seed >> 32
    for i in range(10):
        h0, l0 = mul(x[0], 3528531795)
        h1, l1 = mul(x[2], 3449720151)
        a, b = (ka + i * 2654435769) % (1 << 32), (kb + i * 3144134277) % (1 << 32)
        x = [h1 ^ x[1] ^ a, l1, h0 ^ x[3] ^ b, l0]
    bits = torch.empty(s, nb, 8, dtype=torch.int64, device="cuda")
    for j in range(8):
        bits[:, :, j] = (x[j // 2] // (65536 if j % 2 else 1)) % 65536
    drop = int(math.floor(p * 65536 + 0.5))
    return (bits.reshape(s, nb * 8)[:, :h] >= drop).double() * (65536.0 / (65536 - drop))


def exact(case, seed):
    st = prepare(case, seed)
    op, s = case["op"], case["s"]
    if op in ("logprob", "dlogprob"):
        y, T, top = st["y"], case["temperature"], case["top"]
        parts = {k: [] for k in ("logp", "entropy", "stats", "top_logp", "d")}
        for r0 in range(0, s, 1024):
            r1 = min(s, r0 + 1024)
            z = torch.cat([q[r0:r1] for q in st["shards"]], dim=1).double()
            live = (y[r0:r1] != IGNORE)
            yy = torch.where(live, y[r0:r1], 0)
            lse = torch.logsumexp(z / T, dim=1)
            lp = z / T - lse[:, None]
            p = torch.exp(lp)
            plp = torch.where(p > 0, p * lp, torch.zeros_like(p))
            ent = -plp.sum(1)
            if op == "logprob":
                m = z.max(dim=1).values
                parts["logp"].append(torch.where(live, lp[torch.arange(r1 - r0, device="cuda"), yy], 0.0))
                parts["entropy"].append(torch.where(live, ent, 0.0))
                parts["stats"].append(torch.where(live[:, None], torch.stack([m, lse - m / T, ent, 0 * m], 1), 0.0))
                if top:
                    best = torch.topk(lp, top, dim=1).values
                    parts["top_logp"].append(torch.where(live[:, None], best, 0.0))
                continue
            gl, ge = st["g_logp"][r0:r1].double(), st["g_entropy"][r0:r1].double()
            d = -ge[:, None] * (plp + p * ent[:, None]) - gl[:, None] * p
            d[torch.arange(r1 - r0, device="cuda"), yy] += gl
            if top:
                gt, ids = st["g_top"][r0:r1].double(), st["top_ids"][r0:r1].clamp(min=0)
                d = d - gt.sum(1)[:, None] * p
                d.scatter_add_(1, ids, gt)
            parts["d"].append(torch.where(live[:, None], d / T, 0.0))
        if op == "dlogprob":
            d = torch.cat(parts["d"])
            return [d[:, st["vs"][i]:st["vs"][i + 1]] for i in range(case["t"])]
        out = {k: torch.cat(parts[k]) for k in ("logp", "entropy", "stats")}
        if top:
            out.update(top_logp=torch.cat(parts["top_logp"]), top_ids=None)
        return out
    factor = _exact_factor(case, st["rng"])
    live = (st["ids"] != st["padding"]).double()[:, None]
    if op == "embed":
        return st["full"][st["ids"]].double() * case["scale"] * factor * live
    g = st["g"].double() * case["scale"] * factor * live
    table = torch.zeros(case["V"], case["h"], dtype=torch.float64, device="cuda")
    table.index_put_((st["ids"],), g, accumulate=True)
    return [table[st["vs"][i]:st["vs"][i + 1]] for i in range(case["t"])]
