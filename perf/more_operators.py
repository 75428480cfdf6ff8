"""The operators of a four-bit paged cache, and rotary positions of several axes, as cases that can be measured.

Four operators, each in its plain form (elementary torch operations in 32
bits, in 64 where a value is rounded to four bits) and as the calls a user
makes:

``rotary_axes``    rotary positions with several axes (time, height, width) of
                   a step's q and k, and the store of the rotated k and of v;
``fp4_store``      the same into a cache of four bits (blocks of 16 entries, each
                   e2m1, with an e4m3 scale), and the rows read back;
``fp4_attention``  decode and verify attention over the rows of such a cache;
``fp4_prefill``    chunks of new tokens, causal, over the rows of such a cache.
"""

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"
K_SCALE, V_SCALE = 1.0, 0.5  # what a cache's block scales are multiples of: powers of two


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _axes(name, n, hq, hkv, d, rot, page, layout, sections, interleave, far, dtype):
    return dict(name=name, op="rotary_axes", n=n, hq=hq, hkv=hkv, d=d, rot=rot, page=page, layout=layout,
                sections=sections, interleave=interleave, far=far, dtype=dtype)


def _store(name, n, hq, hkv, d, rot, page, layout, sections, interleave, far, dtype):
    return dict(_axes(name, n, hq, hkv, d, rot, page, layout, sections, interleave, far, dtype), op="fp4_store")


def _attention(name, b, m, hq, hkv, lo, hi, page, raw, window, sinks, dtype="bf16", d=128):
    return dict(name=name, op="fp4_attention", b=b, m=m, hq=hq, hkv=hkv, d=d, lo=lo, hi=hi, page=page, raw=raw,
                window=window, sinks=sinks, qlo=m, qhi=m, dtype=dtype)


def _prefill(name, b, hq, hkv, qlo, qhi, plo, phi, page, raw, window, sinks, dtype="bf16", d=128):
    return dict(name=name, op="fp4_prefill", b=b, m=qhi, hq=hq, hkv=hkv, d=d, lo=plo, hi=phi, page=page, raw=raw,
                window=window, sinks=sinks, qlo=qlo, qhi=qhi, dtype=dtype)


def listed():
    return [
        # one decode step of 64 requests whose prompts held images: latency
        _axes("axes_decode64", 64, 32, 8, 128, 128, 16, "half", "16,24,24", False, 4096, "bf16"),
        # the chunk of several images' prompts, the axes dealt to the pairs in turn
        _axes("axes_chunk8205", 8205, 32, 8, 128, 128, 16, "half", "24,20,20", True, 32768, "bf16"),
        # one decode step of 64 requests into four bits: latency
        _store("fp4_store64", 64, 32, 8, 128, 128, 16, "half", "64", False, 4096, "bf16"),
        # a chunked-prefill step of 16 requests, 512 tokens each
        _store("fp4_store8192", 8192, 32, 8, 128, 128, 16, "half", "64", False, 65536, "bf16"),
        # an odd load, half of each head turned, token by token, positions of three axes
        _store("fp4_store30011", 30011, 64, 8, 128, 64, 1, "interleaved", "8,12,12", False, 4096, "bf16"),
        # one chat request: latency
        _attention("fp4_decode_b1", 1, 1, 32, 8, 777, 777, 16, False, 0, 0),
        # the batch of the GQA decode configuration
        _attention("fp4_decode_b64", 64, 1, 32, 8, 512, 4096, 16, False, 0, 0),
        # long documents in a window with two first tokens that stay
        _attention("fp4_decode_sinks", 32, 1, 32, 8, 8192, 32768, 16, False, 4096, 2),
        # long documents, raw token locations, eight query heads a key head
        _attention("fp4_decode_long", 32, 1, 64, 8, 8192, 32768, 1, True, 0, 0),
        # four drafted tokens of each request verified at once
        _attention("fp4_verify4", 64, 4, 32, 8, 512, 4096, 16, False, 0, 0),
        # a few short prompts that arrive together
        _prefill("fp4_chunk_short", 5, 32, 8, 33, 600, 0, 0, 16, False, 0, 0),
        # the chunk of the prefill configuration: 512 new tokens of 16 requests on prefixes up to 2048
        _prefill("fp4_chunk512", 16, 32, 8, 512, 512, 0, 2048, 16, False, 0, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary_axes", "fp4_store", "fp4_attention", "fp4_attention", "fp4_attention", "fp4_prefill"])
    page = rng.choice([1, 4, 16, 16, 32, 64])
    dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 4, 8, 8])
    hq = hkv * rng.choice([1, 4, 8] if hkv > 1 else [4, 8, 16])
    if op in ("rotary_axes", "fp4_store"):
        d = rng.choice([64, 128, 128])
        if hkv * d < 128:
            d = 128
        rot = rng.choice([d, d, d // 2])
        a = rng.choice([1, 2, 3])
        part = rot // 2 // a
        sections = [rot // 2 - part * (a - 1)] + [part] * (a - 1)
        make = _axes if op == "rotary_axes" else _store
        c = make("", _log(rng, 1, 8192), hq, hkv, d, rot, page, rng.choice(["half", "interleaved"]),
                 ",".join(map(str, sections)), rng.random() < 0.5, _log(rng, 1024, 1 << 17), dtype)
    elif op == "fp4_attention":
        hi, m, b = _log(rng, 8, 8192), rng.choice([1, 1, 1, 1, 2, 4, 7]), _log(rng, 1, 64)
        window = rng.choice([0, 0, 0, max(4, hi // 3)])
        if dtype == "f32":
            b, hi, hq, m = min(b, 8), min(hi, 1024), min(hq, 4 * hkv), min(m, 2)
        hi = max(m, hi)
        c = _attention("", b, m, hq, hkv, rng.randint(m, hi), hi, page, rng.random() < 0.3, window,
                       rng.choice([0, 2, 4]) if window else 0, dtype)
        c["sinks"] = min(c["sinks"], max(0, window - 1))
    else:
        b, qhi = _log(rng, 1, 16), _log(rng, 8, 1024)
        phi = rng.choice([0, 0, 300, 1500])
        window = rng.choice([0, 0, 0, 500])
        if dtype == "f32":
            b, hq, qhi, phi = min(b, 4), min(hq, 4 * hkv), min(qhi, 100), min(phi, 300)
        c = _prefill("", b, hq, hkv, rng.randint(1, qhi), qhi, 0, phi, page, rng.random() < 0.3, window,
                     rng.choice([0, 2]) if window else 0, dtype)
        while c["b"] * hq * qhi * (phi + qhi) > 280_000_000:
            c["b"] //= 2
    del c["name"]
    return c


def _lengths(case, lo, hi, what):
    """Lengths belong to the case: the same for every seed."""
    r = random.Random("%s %s" % (what, sorted((k, str(v)) for k, v in case.items() if k != "name")))
    return [r.randint(lo, hi) for _ in range(case["b"])]


def _queries_and_contexts(case):
    if case["op"] == "fp4_attention":
        return [case["m"]] * case["b"], _lengths(case, case["lo"], case["hi"], "lens")
    q = _lengths(case, case["qlo"], case["qhi"], "q")
    q[0] = case["qhi"]
    return q, [a + p for a, p in zip(q, _lengths(case, case["lo"], case["hi"], "prefix"))]


# ---------------------------------------------------------------------------
# four bits
# ---------------------------------------------------------------------------
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between them; a tie goes to the even code


def _e4m3(x):
    """x >= 0 to the nearest e4m3 value (ties to even, 448 at most), in x's own precision."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    # log2 may be off next to a power of two: there a step too small or too large by two is put right
    step = torch.where(x >= 16 * step, 2 * step, torch.where((x < 8 * step) & (step > 2.0 ** -9), step / 2, step))
    return (torch.round(x / step) * step).clamp(max=448.0)


def _codes(x, g):
    """x [..., blocks, 16] -> (codes 0 .. 7 of |x| [..., blocks, 16], scales [..., blocks, 1])."""
    s = _e4m3(x.abs().amax(-1, keepdim=True) / (6.0 * g))
    r = torch.where(s > 0, x.abs() / torch.where(s > 0, s * g, 1.0), 0.0)
    c = torch.zeros_like(r, dtype=torch.uint8)
    for i, b in enumerate(BORDERS):
        c += (r > b) if i % 2 == 0 else (r >= b)
    return c, s


def _through_four_bits(x, g):
    """The values that x [..., d] comes back as."""
    y = x.unflatten(-1, (-1, 16))
    c, s = _codes(y, g)
    v = torch.tensor(E2M1, dtype=x.dtype, device=x.device)[c.int()]
    return (torch.where(y < 0, -v, v) * s * g).flatten(-2)


def _packed(g, slots, hkv, d):
    """A cache of random rows: codes [slots, hkv, 2, d / 2] (entry 2 i in the low half of byte i; K, then V) and block
    scales [ceil(slots / 16), hkv, 16, 2, d / 16]."""
    codes = torch.empty((slots, hkv, 2, d // 2), dtype=torch.uint8, device=DEV)
    groups = -(-slots // 16)
    scales = torch.zeros((groups * 16, hkv, 2, d // 16), dtype=torch.uint8, device=DEV)
    for at in range(0, slots, 1 << 16):
        n = min(1 << 16, slots - at)
        x = torch.randn((n, hkv, 2, d // 16, 16), generator=g, device=DEV)
        x[:, :, 0] *= 1.0 + torch.rand((hkv, d // 16, 1), generator=g, device=DEV)  # keys' channels differ in size
        for part, gs in ((0, K_SCALE), (1, V_SCALE)):
            c, s = _codes(x[:, :, part], gs)
            c = (c | (x[:, :, part] < 0).to(torch.uint8) * 8).flatten(-2)
            codes[at:at + n, :, part] = c[..., 0::2] | (c[..., 1::2] << 4)
            scales[at:at + n, :, part] = s[..., 0].to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scales.view(groups, 16, hkv, 2, d // 16).transpose(1, 2).contiguous()


def _read(s, slot, dtype=torch.float32):
    """K and V [..., hkv, d] of the given slots."""
    c = s["case"]
    hkv, d = c["hkv"], c["d"]
    byte = s["codes"].view(-1, hkv, 2, d // 2)[slot].int()
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=dtype, device=byte.device)
    x = torch.stack((lut[byte & 15], lut[byte >> 4]), -1).flatten(-2)  # [..., hkv, 2, d]
    scale = s["scales"].view(-1, hkv, 16, 2, d // 16)[slot // 16, :, slot % 16]
    x = x.unflatten(-1, (-1, 16)) * scale.view(torch.float8_e4m3fn).to(dtype)[..., None]
    x = x.flatten(-2)
    return x[..., 0, :] * K_SCALE, x[..., 1, :] * V_SCALE


# ---------------------------------------------------------------------------
# what a user has in hand before the call
# ---------------------------------------------------------------------------
def _pair_axes(case):
    """The axis of each pair: the sections one after another, or dealt in turn until each is used up."""
    left = [int(x) for x in case["sections"].split(",")]
    if not case["interleave"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out, a = [], 0
    while sum(left):
        if left[a]:
            out.append(a)
            left[a] -= 1
        a = (a + 1) % len(left)
    return out


def _plan(case):
    """The handle that a user's program makes once: the kernels' own, or frequencies and axes of the plain form."""
    if own:
        from paged_decode_attention_store_gb300 import binding as kb

        return kb.RotaryPlan(case["rot"], base=10000.0, layout=case["layout"], device=DEV,
                             sections=[int(x) for x in case["sections"].split(",")], interleave=case["interleave"])
    i = torch.arange(case["rot"] // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / case["rot"])).to(DEV), torch.tensor(_pair_axes(case), device=DEV)


def _positions(g, case):
    """Text, whose axes are equal, and images: one time, rows and columns of patches."""
    n, axes = case["n"], len(case["sections"].split(","))
    start = torch.randint(0, case["far"], (-(-n // 100),), generator=g, device=DEV).repeat_interleave(100)[:n]
    i = torch.arange(n, device=DEV)
    image = (i // 100) % 2 == 1
    text = start + i % 100
    grid = [start, start + i % 100 // 10, start + i % 10][:axes]
    p = torch.stack([torch.where(image, x, text) if axes > 1 else text for x in grid])
    return p.to(torch.int32) if axes > 1 else p[0].to(torch.int32)


def _slots(g, n, page, pages):
    """n slots, page after page in a random order of the pages, as requests' tails lie in a used pool."""
    order = torch.randperm(pages, generator=g, device=DEV)
    i = torch.arange(n, device=DEV)
    return (order[i // page] * page + i % page).to(torch.int32)


def _table(g, case, lens):
    page = case["page"]
    need = [-(-x // page) for x in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    cols = max(need)
    block = torch.full((case["b"], cols), -1, dtype=torch.int32)
    at = 0
    for i, x in enumerate(need):
        block[i, :x] = torch.arange(at, at + x, dtype=torch.int32)
        at += x
    block = block.to(DEV)
    block = torch.where(block >= 0, order[block.clamp(min=0).long()], block)
    if case["raw"]:  # token locations: page * P + offset
        raw = block.repeat_interleave(page, dim=1)
        block = torch.where(raw >= 0, raw * page + torch.arange(cols * page, device=DEV, dtype=torch.int32) % page, raw)
    return block.contiguous(), pages


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt = DT[case["dtype"]]
    rnd = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dt)  # noqa: E731
    s = {"case": case}
    op, hq, hkv, d, page = case["op"], case["hq"], case["hkv"], case["d"], case["page"]
    if op in ("rotary_axes", "fp4_store"):
        n = case["n"]
        pages = -(-n // page) + 3
        s["out_loc"] = _slots(g, n, page, pages)
        s["positions"] = _positions(g, case)
        qkv = rnd(n, hq + 2 * hkv, d)  # one projection's output: q, k and v are views of it
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.empty((n, hq, d), dtype=dt, device=DEV)
        s["rope"] = _plan(case)
        if op == "rotary_axes":
            s["cache"] = torch.zeros((2, 1, pages, page, hkv, d), dtype=dt, device=DEV)
        else:
            s["k_out"], s["v_out"] = (torch.empty((n, hkv, d), dtype=dt, device=DEV) for _ in range(2))
    else:
        ql, lens = _queries_and_contexts(case)
        s["table"], pages = _table(g, case, lens)
        s["codes"], s["scales"] = _packed(g, pages * page, hkv, d)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q_lens"] = torch.tensor(ql, dtype=torch.int32, device=DEV) if op == "fp4_prefill" else None
        s["q"] = rnd(case["b"], case["m"], hq, d)
        s["out"] = torch.zeros((case["b"], case["m"], hq, d), dtype=dt, device=DEV)
        s["scale"] = 1.0 / math.sqrt(d)
        s["longest"] = max(lens)
    if own:
        from paged_decode_attention_store_gb300 import binding as kb

        kdt = kb.KVP_BF16 if case["dtype"] == "bf16" else kb.KVP_F32
        if op == "rotary_axes":
            s["pool"] = kb.Pool(s["cache"], page, kdt)
        elif op == "fp4_store":
            s["pool"] = kb.kv_fp4_pool_create(pages, page, hkv, d, kdt, 1, k_scale=K_SCALE, v_scale=V_SCALE, device=DEV)
        else:
            s["pool"] = kb.Fp4Pool(s["codes"].view(1, pages, page, hkv, 2, d // 2),
                                   s["scales"].view(1, -1, hkv, 16, 2, d // 16), kdt, k_scale=K_SCALE, v_scale=V_SCALE)
            s["workspace"] = kb.alloc_fp4_workspace(s["pool"], case["b"], case["m"], hq, s["longest"], device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _rotated(x, s, dtype):
    """The first entries of each head turned by position x frequency, each pair by its axis' position; the rest as they
    are. In 32 bits (the angles, which grow with the position, in 64), or all in 64."""
    c = s["case"]
    freq, axis = s["rope"]
    rot = c["rot"]
    p = s["positions"] if s["positions"].dim() == 2 else s["positions"][None]
    angle = p.double()[axis].T * freq
    cos, sin = angle.cos().to(dtype)[:, None, :], angle.sin().to(dtype)[:, None, :]
    x = x.to(dtype)
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _run_rotary_axes(s):
    c, loc, cache = s["case"], s["out_loc"].long(), s["cache"]
    s["q_out"].copy_(_rotated(s["q"], s, torch.float32))
    rows = cache.view(2, -1, c["hkv"], c["d"])
    rows[0, loc] = _rotated(s["k"], s, torch.float32).to(cache.dtype)
    rows[1, loc] = s["v"]
    return {"q": s["q_out"], "cache": cache}


def _run_fp4_store(s):
    s["q_out"].copy_(_rotated(s["q"], s, torch.float32))
    s["k_out"].copy_(_through_four_bits(_rotated(s["k"], s, torch.float64), K_SCALE))  # in 64: values next to a border
    s["v_out"].copy_(_through_four_bits(s["v"].double(), V_SCALE))
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _attended(p, t, window, sinks):
    """Whether the query at position p attends position t: causal, within the window, or a sink row."""
    ok = t <= p
    if window > 0:
        ok = ok & ((t > p - (window - sinks)) | (t < sinks))
    return ok


def _run_attention(s):
    c, table = s["case"], s["table"].long()
    b, m, hkv, d = c["b"], c["m"], c["hkv"], c["d"]
    t = torch.arange(s["longest"], device=DEV)
    slot = table[:, t] if c["raw"] else table[:, t // c["page"]] * c["page"] + t % c["page"]
    live = t < s["lens"][:, None]
    k, v = _read(s, torch.where(live, slot, 0))  # [b, t, hkv, d]
    ql = s["lens"].new_full((b,), m) if s["q_lens"] is None else s["q_lens"]
    j = torch.arange(m, device=DEV)
    p = (s["lens"] - ql)[:, None] + j
    real = j < ql[:, None]
    ok = live[:, None, :] & _attended(p[:, :, None], t, c["window"], c["sinks"]) | (~real[:, :, None] & (t == 0))
    q = s["q"].float().view(b, m, hkv, -1, d)
    score = torch.einsum("bmhgd,bthd->bhgmt", q, k) * s["scale"]
    score = torch.where(ok[:, None, None], score, float("-inf"))
    w = torch.exp(score - score.amax(-1, keepdim=True))
    o = torch.einsum("bhgmt,bthd->bmhgd", w / w.sum(-1, keepdim=True), v).reshape(s["out"].shape)
    s["out"].copy_(torch.where(real[:, :, None, None], o, s["out"].float()))
    return s["out"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        from paged_decode_attention_store_gb300 import binding as kb

        if op == "rotary_axes":
            kb.rotary_store_cache(s["pool"], 0, s["q"], s["k"], s["v"], s["positions"], s["out_loc"], s["rope"], s["q_out"])
            return {"q": s["q_out"], "cache": s["cache"]}
        if op == "fp4_store":
            kb.rotary_store_fp4(s["pool"], 0, s["q"], s["k"], s["v"], s["positions"], s["out_loc"], s["rope"], s["q_out"])
            kb.load_cache_fp4(s["pool"], 0, s["out_loc"], s["k_out"], s["v_out"])
            return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
        kb.paged_fp4_attention(s["pool"], 0, s["q"], s["table"], kb.KVP_RAW_LOCATIONS if c["raw"] else kb.KVP_BLOCK_TABLE,
                               s["lens"], c["window"], s["scale"], s["out"], s["workspace"], q_lens=s["q_lens"],
                               sinks=c["sinks"], max_context=s["longest"])
        return s["out"]
    if op == "rotary_axes":
        return _run_rotary_axes(s)
    if op == "fp4_store":
        return _run_fp4_store(s)
    return _run_attention(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _pairs_and_rows(L, m, window, sinks):
    """(query, position) pairs of the m newest of L tokens, and the positions that any of them attends."""
    if window <= 0:
        return sum(range(L - m + 1, L + 1)), L
    total, lows = 0, []
    for n in range(L - m + 1, L + 1):
        lo = max(0, n - (window - sinks))
        total += n - lo + min(sinks, lo)
        lows.append(lo)
    return total, L - min(lows) + min(sinks, min(lows))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, hq, hkv, d = case["op"], case["hq"], case["hkv"], case["d"]
    if op in ("rotary_axes", "fp4_store"):
        n, axes = case["n"], len(case["sections"].split(","))
        q, kv, back = 2 * e * hq * d, 2 * e * hkv * d, 0
        if op == "rotary_axes":
            put = kv
        else:
            put = 2 * hkv * (d // 2 + d // 16)  # written, then read back and given out
            back = put + kv + 4
        return {"bytes": n * (q + kv + put + back + 4 * axes + 4), "flops": 3 * n * (hq + hkv) * case["rot"]}
    pairs = rows = entries = queries = 0
    for m, L in zip(*_queries_and_contexts(case)):
        a, r = _pairs_and_rows(L, m, case["window"], case["sinks"])
        pairs, rows, queries = pairs + a, rows + r, queries + m
        entries += r if case["raw"] else -(-r // case["page"])
    return {"bytes": rows * 2 * hkv * (d // 2 + d // 16) + 2 * e * queries * hq * d + 4 * (entries + case["b"]),
            "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _turn(x, case, positions):
    """Each pair (a, b) as a complex number, times exp(i * position * theta) of its axis."""
    rot = case["rot"]
    theta = torch.tensor([math.exp(-2.0 * i / rot * math.log(10000.0)) for i in range(rot // 2)], dtype=torch.float64,
                         device=positions.device)
    p = positions.double().reshape(-1, positions.shape[-1])
    ang = torch.stack([p[a] * theta[i] for i, a in enumerate(_pair_axes(case))], -1)
    unit = torch.polar(torch.ones_like(ang), ang)[:, None, :]
    y = x.double().clone()
    if case["layout"] == "half":
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * unit
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2)) * unit
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    return y


def _nearest(x, values):
    """The nearest of the ascending values; of two as near, the one of even index."""
    lo = torch.searchsorted(values, x.contiguous(), right=True) - 1
    hi = (lo + 1).clamp(max=len(values) - 1)
    below, above = x - values[lo], values[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return values[torch.where(up & (hi > lo), hi, lo)]


def _rounded(x, g):
    dev = x.device
    e4m3 = torch.arange(127, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()
    y = x.reshape(*x.shape[:-1], -1, 16) / g
    s = _nearest(y.abs().max(-1, keepdim=True).values / 6, e4m3)
    z = _nearest(torch.where(s > 0, y.abs() / s, torch.zeros_like(y)), torch.tensor(E2M1, dtype=torch.float64, device=dev))
    return (torch.copysign(z, y) * s * g).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary_axes":
        cache = s["cache"].double()
        flat = cache.view(2, -1, case["hkv"], case["d"])
        flat[0].index_copy_(0, s["out_loc"].long(), _turn(s["k"], case, s["positions"]))
        flat[1].index_copy_(0, s["out_loc"].long(), s["v"].double())
        return {"q": _turn(s["q"], case, s["positions"]), "cache": cache}
    if op == "fp4_store":
        return {"q": _turn(s["q"], case, s["positions"]), "k": _rounded(_turn(s["k"], case, s["positions"]), K_SCALE),
                "v": _rounded(s["v"].double(), V_SCALE)}
    table, (ql, lens) = s["table"].cpu(), _queries_and_contexts(case)
    hkv, page, G = case["hkv"], case["page"], case["hq"] // case["hkv"]
    if sum(a * b for a, b in zip(ql, lens)) * case["hq"] > 1 << 29 or sum(ql) * case["b"] > 1 << 20:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for b, (m, L) in enumerate(zip(ql, lens)):
        row = table[b].tolist()
        where = [row[t] if case["raw"] else row[t // page] * page + t % page for t in range(L)]
        k, v = _read(s, torch.tensor(where, device=DEV), torch.float64)
        p = torch.arange(L - m, L, device=DEV)[:, None]
        t = torch.arange(L, device=DEV)
        keep = t <= p
        if case["window"] > 0:
            keep &= (p - t < case["window"] - case["sinks"]) | (t < case["sinks"])
        for h in range(case["hq"]):
            sc = (s["q"][b, :m, h].double() @ k[:, h // G].T * s["scale"]).masked_fill(~keep, float("-inf"))
            out[b, :m, h] = torch.softmax(sc, -1) @ v[:, h // G]
    return out
