"""The operators of a paged cache beyond plain decode attention, as cases that can be measured.

Four operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and as the calls a user makes:

``rotary_store``      rotary positions of a step's q and k, and the write of the
                      rotated k and of v to their slots of the paged cache;
``latent_store``      the same for a cache of one latent row a token
                      ([latent | shared rotated key part]);
``latent_attention``  attention over the paged latent rows in absorbed form: the
                      row is every head's key, its first part every head's value;
``latent_prefill``    attention of prompts in expanded form: per-head keys and
                      values, and one rotated key part that all heads share.
"""

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"
LOW_TURNS, HIGH_TURNS = 1.0, 32.0  # by-parts scaling: the turns over the original length between which it blends


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rotary(name, n, hq, hkv, d, rot, page, layout, scaling, factor, far, dtype):
    return dict(name=name, op="rotary_store", n=n, hq=hq, hkv=hkv, d=d, rot=rot, page=page, layout=layout, scaling=scaling,
                factor=factor, far=far, dtype=dtype)


def _latent_store(name, n, hq, dc, dr, page, layout, scaling, factor, far, dtype):
    return dict(name=name, op="latent_store", n=n, hq=hq, dc=dc, dr=dr, page=page, layout=layout, scaling=scaling,
                factor=factor, far=far, dtype=dtype)


def _latent(name, b, m, hq, lo, hi, page, raw, window, sinks, dtype="bf16", dc=512, dr=64):
    return dict(name=name, op="latent_attention", b=b, m=m, hq=hq, lo=lo, hi=hi, page=page, raw=raw, window=window,
                sinks=sinks, dc=dc, dr=dr, dtype=dtype)


def _expanded(name, b, hq, qlo, qhi, plo, phi, dtype="bf16", dn=128, dr=64, dv=128):
    return dict(name=name, op="latent_prefill", b=b, hq=hq, qlo=qlo, qhi=qhi, plo=plo, phi=phi, dn=dn, dr=dr, dv=dv,
                dtype=dtype)


def listed():
    return [
        # one decode step of 64 requests: latency
        _rotary("rotary_decode64", 64, 32, 8, 128, 128, 16, "half", "none", 1.0, 4096, "bf16"),
        # a chunked-prefill step of 16 requests, 512 tokens each, on a context stretched eightfold
        _rotary("rotary_chunk8192", 8192, 32, 8, 128, 128, 16, "half", "by_parts", 8.0, 65536, "bf16"),
        # a long-context load: half of each head rotated, pairs side by side, positions near a million
        _rotary("rotary_load65537", 65537, 64, 8, 128, 64, 1, "interleaved", "linear", 4.0, 1 << 20, "bf16"),
        # fp32 caches, as numerics checks use them
        _rotary("rotary_f32_3001", 3001, 16, 2, 64, 64, 4, "interleaved", "ntk", 2.0, 32768, "f32"),
        # one decode step of 256 requests on a latent cache
        _latent_store("latent_store256", 256, 16, 512, 64, 16, "interleaved", "none", 1.0, 16384, "bf16"),
        # the chunk of many prompts at once
        _latent_store("latent_store16461", 16461, 32, 512, 64, 64, "half", "by_parts", 40.0, 131072, "bf16"),
        # one chat request: latency
        _latent("latent_decode_b1", 1, 1, 16, 777, 777, 16, False, 0, 0),
        # the batch of the GQA decode configuration (64 requests of 512 to 4096 tokens) on latents
        _latent("latent_decode_b64", 64, 1, 32, 512, 4096, 16, False, 0, 0),
        # long documents, raw token locations, every head on one GPU
        _latent("latent_decode_long", 32, 1, 128, 8192, 32768, 1, True, 0, 0),
        # four drafted tokens of each request verified at once
        _latent("latent_verify4", 64, 4, 64, 512, 4096, 16, False, 0, 0),
        # a few short prompts that arrive together
        _expanded("expanded_short", 5, 16, 33, 600, 0, 0),
        # the chunk of the prefill configuration: 512 new tokens of 16 requests on prefixes up to 2048
        _expanded("expanded_chunk512", 16, 32, 512, 512, 0, 2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary_store", "latent_store", "latent_attention", "latent_attention", "latent_prefill"])
    scaling = rng.choice(["none", "linear", "ntk", "by_parts"])
    factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 40.0])
    layout = rng.choice(["half", "interleaved"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    page = rng.choice([1, 4, 16, 32, 64])
    far = _log(rng, 1024, 1 << 20)
    if op == "rotary_store":
        hkv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 128])
        c = _rotary("", _log(rng, 1, 16384), hkv * rng.choice([1, 4, 8]), hkv, d, rng.choice([d, d, d // 2]), page, layout,
                    scaling, factor, far, dtype)
    elif op == "latent_store":
        c = _latent_store("", _log(rng, 1, 16384), rng.choice([8, 16, 32, 64]), 512, 64, page, layout, scaling, factor, far,
                          dtype)
    elif op == "latent_attention":
        hi = _log(rng, 8, 8192)
        window = rng.choice([0, 0, 0, max(4, hi // 3)])
        hq, m, b = rng.choice([8, 16, 32, 64, 128]), rng.choice([1, 1, 1, 2, 4, 7]), _log(rng, 1, 64)
        if dtype == "f32":
            b, hi, hq, m = min(b, 8), min(hi, 1024), min(hq, 16), min(m, 2)
        c = _latent("", b, m, hq, max(m, rng.randint(m, max(m, hi))), max(m, hi), page, rng.random() < 0.3, window,
                    rng.choice([0, 2]) if window else 0, dtype)
        c["lo"] = min(c["lo"], c["hi"])
        while c["b"] * m * hq * c["hi"] > 64_000_000:  # no more work than the largest listed case
            c["b"] //= 2
    else:
        b, hq = _log(rng, 1, 16), rng.choice([4, 8, 16, 32])
        qhi = _log(rng, 1, 1024)
        if dtype == "f32":
            b, hq, qhi = min(b, 4), min(hq, 8), min(qhi, 200)
        c = _expanded("", b, hq, rng.randint(1, qhi), qhi, 0, rng.choice([0, 0, 300, 1500]), dtype)
        while c["b"] * hq * qhi * (c["phi"] + qhi) > 280_000_000:
            c["b"] //= 2
    del c["name"]
    return c


def _lengths(case, lo, hi, what):
    """Lengths belong to the case: the same for every seed."""
    r = random.Random("%s %s" % (what, sorted((k, str(v)) for k, v in case.items() if k != "name")))
    return [r.randint(lo, hi) for _ in range(case["b"])]


# ---------------------------------------------------------------------------
# what a user has in hand before the call
# ---------------------------------------------------------------------------
def _inverse_frequencies(dim, base, scaling, factor, original):
    """theta_i = base^(-2 i / dim) of pair i, stretched for long contexts (64 bits)."""
    i = torch.arange(dim // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    f = base ** (-2.0 * i / dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        turns = original * f / (2 * math.pi)
        keep = ((turns - LOW_TURNS) / (HIGH_TURNS - LOW_TURNS)).clamp(0.0, 1.0)
        f = keep * f + (1 - keep) * (f / factor)
    return f


def _rope_facts(case, dim):
    attn = 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "by_parts" else 1.0
    return dict(dim=dim, base=10000.0, scaling=case["scaling"], factor=case["factor"], original=4096, attn=attn)


def _plan(case, dim):
    """The handle that a user's program makes once: the kernels' own, or the frequencies of the plain form."""
    f = _rope_facts(case, dim)
    if own:
        from paged_decode_attention_store_gb300 import binding as kb

        return kb.RotaryPlan(dim, base=f["base"], layout=case["layout"], scaling=f["scaling"], factor=f["factor"],
                             original_len=f["original"], low_turns=LOW_TURNS, high_turns=HIGH_TURNS, attn_factor=f["attn"],
                             device=DEV)
    return _inverse_frequencies(dim, f["base"], f["scaling"], f["factor"], f["original"]).to(DEV), f["attn"]


def _slots(g, n, page, pages):
    """n slots, page after page in a random order of the pages, as requests' tails lie in a used pool."""
    order = torch.randperm(pages, generator=g, device=DEV)
    i = torch.arange(n, device=DEV)
    return (order[i // page] * page + i % page).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt = DT[case["dtype"]]
    rnd = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dt)  # noqa: E731
    s = {"case": case}
    op = case["op"]
    if op in ("rotary_store", "latent_store"):
        n, page = case["n"], case["page"]
        pages = -(-n // page) + 3
        s["out_loc"] = _slots(g, n, page, pages)
        s["positions"] = torch.randint(0, case["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
        if op == "rotary_store":
            hq, hkv, d = case["hq"], case["hkv"], case["d"]
            qkv = rnd(n, hq + 2 * hkv, d)  # one projection's output: q, k and v are views of it
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            s["cache"] = torch.zeros((2, 1, pages, page, hkv, d), dtype=dt, device=DEV)
            s["q_out"] = torch.empty((n, hq, d), dtype=dt, device=DEV)
            s["rope"] = _plan(case, case["rot"])
        else:
            dc, dr = case["dc"], case["dr"]
            down = rnd(n, dc + dr)  # the down projection's output: latent and key part
            s["latent"], s["k_pe"] = down[:, :dc], down[:, dc:]
            s["q_pe"] = rnd(n, case["hq"], dr)
            s["q_full"] = torch.zeros((n, case["hq"], dc + dr), dtype=dt, device=DEV)  # the queries of the attention
            s["cache"] = torch.zeros((1, pages, page, dc + dr), dtype=dt, device=DEV)
            s["rope"] = _plan(case, dr)
    elif op == "latent_attention":
        b, m, page, width = case["b"], case["m"], case["page"], case["dc"] + case["dr"]
        lens = _lengths(case, case["lo"], case["hi"], "lens")
        need = [-(-x // page) for x in lens]
        pages = sum(need) + 3
        s["cache"] = rnd(1, pages, page, width)
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        cols = max(need)
        block = torch.full((b, cols), -1, dtype=torch.int32)
        at = 0
        for i, x in enumerate(need):
            block[i, :x] = torch.arange(at, at + x, dtype=torch.int32)
            at += x
        block = block.to(DEV)
        block = torch.where(block >= 0, order[block.clamp(min=0).long()], block)
        if case["raw"]:  # token locations: page * P + offset
            raw = block.repeat_interleave(page, dim=1)
            offs = torch.arange(cols * page, device=DEV, dtype=torch.int32) % page
            block = torch.where(raw >= 0, raw * page + offs, raw)
        s["table"] = block.contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = rnd(b, m, case["hq"], width)
        s["out"] = torch.empty((b, m, case["hq"], case["dc"]), dtype=dt, device=DEV)
        s["scale"] = 1.0 / math.sqrt(128 + case["dr"])
    else:
        ql = _lengths(case, case["qlo"], case["qhi"], "q")
        kl = [a + p for a, p in zip(ql, _lengths(case, case["plo"], case["phi"], "prefix"))]
        hq, dn, dr, dv = case["hq"], case["dn"], case["dr"], case["dv"]
        tq, tk = sum(ql), sum(kl)
        up = rnd(tk, hq, dn + dv)  # the up projection's output: per head key part and value
        s["k"], s["v"] = up[..., :dn], up[..., dn:]
        s["k_pe"] = rnd(tk, 512 + dr)[:, 512:]  # of the latent rows
        s["q"] = rnd(tq, hq, dn + dr)
        s["out"] = torch.empty((tq, hq, dv), dtype=dt, device=DEV)
        start = lambda xs: torch.tensor([sum(xs[:i]) for i in range(len(xs) + 1)], dtype=torch.int32, device=DEV)  # noqa: E731
        s["q_start"], s["k_start"] = start(ql), start(kl)
        s["max_q"], s["max_k"] = max(ql), max(kl)
        s["scale"] = 1.0 / math.sqrt(dn + dr)
    if own:
        from paged_decode_attention_store_gb300 import binding as kb

        kdt = kb.KVP_BF16 if case["dtype"] == "bf16" else kb.KVP_F32
        if op == "rotary_store":
            s["pool"] = kb.Pool(s["cache"], case["page"], kdt)
        elif op != "latent_prefill":
            s["pool"] = kb.LatentPool(s["cache"], case["dc"], kdt)
        if op == "latent_attention":
            s["workspace"] = kb.alloc_latent_workspace(s["pool"], case["b"], case["m"], case["hq"], device=DEV)
        if op == "latent_prefill":
            s["error_word"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _rotated(x, dim, positions, rope, layout):
    """The first ``dim`` entries of each head turned by position x frequency, the rest as they are (32 bits; the
    angles, which grow with the position, in 64)."""
    freq, attn = rope
    angle = positions.double()[:, None] * freq
    cos, sin = (angle.cos() * attn).float()[:, None, :], (angle.sin() * attn).float()[:, None, :]
    x = x.float()
    if layout == "half":
        a, b = x[..., :dim // 2], x[..., dim // 2:dim]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:dim:2], x[..., 1:dim:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., dim:]), -1)


def _run_rotary_store(s):
    c, loc, cache = s["case"], s["out_loc"].long(), s["cache"]
    s["q_out"].copy_(_rotated(s["q"], c["rot"], s["positions"], s["rope"], c["layout"]))
    rows = cache.view(2, -1, c["hkv"], c["d"])
    rows[0, loc] = _rotated(s["k"], c["rot"], s["positions"], s["rope"], c["layout"]).to(cache.dtype)
    rows[1, loc] = s["v"]
    return {"q": s["q_out"], "cache": cache}


def _run_latent_store(s):
    c, loc, cache = s["case"], s["out_loc"].long(), s["cache"]
    s["q_full"][..., c["dc"]:] = _rotated(s["q_pe"], c["dr"], s["positions"], s["rope"], c["layout"]).to(cache.dtype)
    rows = cache.view(-1, c["dc"] + c["dr"])
    key = _rotated(s["k_pe"][:, None], c["dr"], s["positions"], s["rope"], c["layout"])[:, 0]
    rows[loc] = torch.cat((s["latent"], key.to(cache.dtype)), -1)
    return {"q": s["q_full"], "cache": cache}


def _attended(p, t, window, sinks):
    """Whether the query at position p attends position t: causal, within the window, or a sink row."""
    ok = t <= p
    if window > 0:
        ok = ok & ((t > p - (window - sinks)) | (t < sinks))
    return ok


def _run_latent_attention(s):
    c, table = s["case"], s["table"].long()
    rows = s["cache"].view(-1, c["dc"] + c["dr"])
    t = torch.arange(c["hi"], device=DEV)
    slot = table[:, t.clamp(max=table.shape[1] - 1)] if c["raw"] else (
        table[:, (t // c["page"]).clamp(max=table.shape[1] - 1)] * c["page"] + t % c["page"])
    live = t[None, :] < s["lens"][:, None]
    x = rows[torch.where(live, slot, 0)].float()  # [b, t, width]
    score = torch.einsum("bmhd,btd->bmht", s["q"].float(), x) * s["scale"]
    p = s["lens"][:, None].long() - c["m"] + torch.arange(c["m"], device=DEV)
    ok = live[:, None, :] & _attended(p[:, :, None], t, c["window"], c["sinks"])
    w = torch.exp(torch.where(ok[:, :, None, :], score, float("-inf")) - torch.where(
        ok[:, :, None, :], score, float("-inf")).amax(-1, keepdim=True))
    o = torch.einsum("bmht,btd->bmhd", w, x[..., :c["dc"]]) / w.sum(-1, keepdim=True)
    s["out"].copy_(o)
    return s["out"]


def _run_latent_prefill(s):
    qs, ks = s["q_start"].long(), s["k_start"].long()
    j, t = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    ql, kl = qs[1:] - qs[:-1], ks[1:] - ks[:-1]
    qi = (qs[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)  # padded to the longest
    ki = (ks[:-1, None] + t).clamp(max=s["k"].shape[0] - 1)
    q, k, v, pe = s["q"][qi].float(), s["k"][ki].float(), s["v"][ki].float(), s["k_pe"][ki].float()
    dn = k.shape[-1]
    score = torch.einsum("bjhd,bthd->bhjt", q[..., :dn], k) + torch.einsum("bjhd,btd->bhjt", q[..., dn:], pe)
    ok = (t <= (kl - ql)[:, None, None] + j[:, None]) & (j < ql[:, None])[:, :, None]
    ok = ok | (j >= ql[:, None])[:, :, None] & (t == 0)  # rows of the padding: dropped below
    score = torch.where(ok[:, None], score * s["scale"], float("-inf"))
    w = torch.exp(score - score.amax(-1, keepdim=True))
    o = torch.einsum("bhjt,bthd->bjhd", w / w.sum(-1, keepdim=True), v)
    s["out"].copy_(o[j < ql[:, None]])
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        from paged_decode_attention_store_gb300 import binding as kb

        s, c = state, state["case"]
        if op == "rotary_store":
            kb.rotary_store_cache(s["pool"], 0, s["q"], s["k"], s["v"], s["positions"], s["out_loc"], s["rope"], s["q_out"])
            return {"q": s["q_out"], "cache": s["cache"]}
        if op == "latent_store":
            kb.rotary_store_latent(s["pool"], 0, s["q_pe"], s["latent"], s["k_pe"], s["positions"], s["out_loc"], s["rope"],
                                   s["q_full"][..., c["dc"]:])
            return {"q": s["q_full"], "cache": s["cache"]}
        if op == "latent_attention":
            kb.paged_latent_attention(s["pool"], 0, s["q"], s["table"],
                                      kb.KVP_RAW_LOCATIONS if c["raw"] else kb.KVP_BLOCK_TABLE, s["lens"], c["window"],
                                      s["scale"], s["out"], s["workspace"], sinks=c["sinks"])
            return s["out"]
        kb.latent_prefill_attention(s["q"], s["k"], s["k_pe"], s["v"], s["q_start"], s["k_start"], s["max_q"], s["scale"],
                                    s["out"], error_word=s["error_word"])
        return s["out"]
    if op == "rotary_store":
        return _run_rotary_store(state)
    if op == "latent_store":
        return _run_latent_store(state)
    if op == "latent_attention":
        return _run_latent_attention(state)
    return _run_latent_prefill(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _count(L, m, window, sinks):
    """Positions that the m newest of L tokens attend, all together, and those that any of them does."""
    each = [range(L - m + j + 1) for j in range(m)]
    if window <= 0:
        return sum(len(r) for r in each), L
    total, lows = 0, []
    for r in each:
        lo = max(0, len(r) - (window - sinks))
        total += len(r) - lo + min(sinks, lo)
        lows.append(lo)
    return total, L - min(lows) + min(sinks, min(lows))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "rotary_store":
        n, heads = case["n"], case["hq"] + case["hkv"]
        return {"bytes": n * (2 * e * case["d"] * (heads + case["hkv"]) + 8), "flops": 3 * n * heads * case["rot"]}
    if op == "latent_store":
        n = case["n"]
        return {"bytes": n * (2 * e * (case["hq"] * case["dr"] + case["dc"] + case["dr"]) + 8),
                "flops": 3 * n * (case["hq"] + 1) * case["dr"]}
    if op == "latent_attention":
        width = case["dc"] + case["dr"]
        pairs = rows = entries = 0
        for L in _lengths(case, case["lo"], case["hi"], "lens"):
            a, r = _count(L, case["m"], case["window"], case["sinks"])
            pairs, rows = pairs + a, rows + r
            entries += r if case["raw"] else -(-r // case["page"])
        io = case["b"] * case["m"] * case["hq"] * (width + case["dc"]) * e
        return {"bytes": rows * width * e + io + 4 * (entries + case["b"]),
                "flops": 2 * pairs * case["hq"] * (width + case["dc"])}
    ql = _lengths(case, case["qlo"], case["qhi"], "q")
    kl = [a + p for a, p in zip(ql, _lengths(case, case["plo"], case["phi"], "prefix"))]
    pairs = sum((k - q) * q + q * (q + 1) // 2 for q, k in zip(ql, kl))
    hq, dn, dr, dv = case["hq"], case["dn"], case["dr"], case["dv"]
    return {"bytes": e * (sum(ql) * hq * (dn + dr + dv) + sum(kl) * (hq * (dn + dv) + dr)) + 8 * (case["b"] + 1),
            "flops": 2 * pairs * hq * (dn + dr + dv)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _turn(x, case, dim, positions):
    """Each pair (a, b) as a complex number, times attn * exp(i * position * theta)."""
    f = _rope_facts(case, dim)
    theta = []
    for i in range(dim // 2):
        base = f["base"] * (f["factor"] ** (dim / (dim - 2)) if f["scaling"] == "ntk" else 1.0)
        th = math.exp(-2.0 * i / dim * math.log(base))
        if f["scaling"] == "linear":
            th /= f["factor"]
        if f["scaling"] == "by_parts":
            g = (f["original"] * th / (2 * math.pi) - LOW_TURNS) / (HIGH_TURNS - LOW_TURNS)
            g = min(1.0, max(0.0, g))
            th = th * (g + (1 - g) / f["factor"])
        theta.append(th)
    ang = positions.double()[:, None] * torch.tensor(theta, dtype=torch.float64, device=positions.device)
    unit = torch.polar(torch.full_like(ang, f["attn"]), ang)[:, None, :]
    y = x.double().clone()
    if case["layout"] == "half":
        z = torch.complex(y[..., :dim // 2].contiguous(), y[..., dim // 2:dim].contiguous()) * unit
        y[..., :dim // 2], y[..., dim // 2:dim] = z.real, z.imag
    else:
        z = torch.view_as_complex(y[..., :dim].reshape(*y.shape[:-1], dim // 2, 2)) * unit
        y[..., :dim] = torch.view_as_real(z).flatten(-2)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op, dev = case["op"], s["cache"].device if "cache" in s else s["q"].device
    if op == "rotary_store":
        cache = s["cache"].double()
        flat = cache.view(2, -1, case["hkv"], case["d"])
        flat[0].index_copy_(0, s["out_loc"].long(), _turn(s["k"], case, case["rot"], s["positions"]))
        flat[1].index_copy_(0, s["out_loc"].long(), s["v"].double())
        return {"q": _turn(s["q"], case, case["rot"], s["positions"]), "cache": cache}
    if op == "latent_store":
        cache, q = s["cache"].double(), s["q_full"].double()
        flat = cache.view(-1, case["dc"] + case["dr"])
        row = torch.cat((s["latent"].double(), _turn(s["k_pe"][:, None], case, case["dr"], s["positions"])[:, 0]), 1)
        flat.index_copy_(0, s["out_loc"].long(), row)
        q[..., case["dc"]:] = _turn(s["q_pe"], case, case["dr"], s["positions"])
        return {"q": q, "cache": cache}
    if op == "latent_attention":
        flat = s["cache"].view(-1, case["dc"] + case["dr"])
        table, lens, m = s["table"].cpu(), s["lens"].tolist(), case["m"]
        if sum(lens) * case["hq"] * m > 1 << 28:
            return None
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
        for b, L in enumerate(lens):
            row = table[b].tolist()
            where = [row[t] if case["raw"] else row[t // case["page"]] * case["page"] + t % case["page"] for t in range(L)]
            x = flat[torch.tensor(where, device=dev)].double()
            for j in range(m):
                p = L - m + j
                lo = max(0, p + 1 - (case["window"] - case["sinks"])) if case["window"] > 0 else 0
                keep = list(range(min(case["sinks"], lo))) + list(range(lo, p + 1)) if lo else None
                y = x[:p + 1] if keep is None else x[torch.tensor(keep, device=dev)]
                pr = torch.softmax(s["q"][b, j].double() @ y.T * s["scale"], -1)
                out[b, j] = pr @ y[:, :case["dc"]]
        return out
    qs, ks = s["q_start"].tolist(), s["k_start"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
    for b in range(case["b"]):
        q0, q1, k0, k1 = qs[b], qs[b + 1], ks[b], ks[b + 1]
        after = torch.ones((q1 - q0, k1 - k0), dtype=torch.bool, device=dev).triu(k1 - k0 - (q1 - q0) + 1)
        for h in range(case["hq"]):
            key = torch.cat((s["k"][k0:k1, h], s["k_pe"][k0:k1]), 1).double()
            sc = (s["q"][q0:q1, h].double() @ key.T * s["scale"]).masked_fill(after, float("-inf"))
            out[q0:q1, h] = torch.softmax(sc, -1) @ s["v"][k0:k1, h].double()
    return out
