"""Workloads of the paged K/V cache operators: page allocation and release, the append of new K/V rows, and the
attention of one new token per sequence over the pages.

``run`` computes an operator in elementary torch operations when ``own`` is false, and through this package's entry
points when it is true. ``exact`` is the operator's definition in 64 bits. Head layouts are those of the models in
``synth/configs.py``: 20 query heads over 4 K/V heads of 128 (the 2B model), 16 over 4 of 128 (the sparse-MoE model),
4 over 4 and 4 over 2 of 64 (the tiny models).
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4, "e4m3": 1}
E4M3_MAX = 448.0
NO_SCALE = 2.0 ** -126  # the scale of an all-zero row


def listed():
    return [
        # The 2B model's decode at the end of its benchmark (128 prompt + 1,024 new tokens), one request: latency.
        attention("attention: 2B, one of 1,152", 1, 20, 4, 128, 16, 1152, 1152, "fp16", "fp32"),
        # The long-context decode (8,192 prompt + 512 new tokens), one request: the split over the length.
        attention("attention: 2B, one of 8,704", 1, 20, 4, 128, 64, 8704, 8704, "fp16", "fp32"),
        # A serving batch whose requests are of every age, from the first token to the longest context.
        attention("attention: 2B, 32 ragged", 32, 20, 4, 128, 16, 1, 8704, "fp16", "fp16"),
        # A full serving batch of the sparse-MoE model's heads: the largest.
        attention("attention: MoE heads, 256", 256, 16, 4, 128, 64, 128, 4096, "bf16", "bf16"),
        # A long-context batch on an 8-bit cache.
        attention("attention: 2B, 61 on e4m3", 61, 20, 4, 128, 32, 513, 8704, "e4m3", "fp16"),
        # One decode step of a small batch: latency.
        append("append: 2B, 32 tokens", 32, 0, 20, 4, 128, 16, "fp16", "fp16"),
        # A long prompt's rows at once, from the framework's fp32 activations.
        append("append: MoE heads, 8,192 tokens", 8192, 0, 16, 4, 128, 64, "fp16", "fp32"),
        # A mixed step of odd size into an 8-bit cache, padded to a captured size.
        append("append: 2B, 4,097 on e4m3", 4097, 63, 20, 4, 128, 32, "e4m3", "bf16"),
        # One decode step of a full batch: a token each.
        extend("extend: 256 of one token", 256, 1, 1, 16, 8704, 0),
        # Prompts of every length next to running requests, one more than a captured size.
        extend("extend: 1,025 mixed", 1025, 1, 512, 32, 2048, 77),
        # A few of a full batch have ended.
        release("release: 256", 256, 16, 8704, 9),
        # Most of a large batch has ended.
        release("release: 2,047", 2047, 32, 2048, 2),
    ]


def attention(name, seqs, hq, hkv, dh, block, lo, hi, cache, q, window=0):
    return dict(name=name, op="attention", seqs=seqs, hq=hq, hkv=hkv, dh=dh, block=block, lo=lo, hi=hi, cache=cache,
                q=q, window=window)


def append(name, rows, pad, hq, hkv, dh, block, cache, x):
    return dict(name=name, op="append", rows=rows, pad=pad, hq=hq, hkv=hkv, dh=dh, block=block, cache=cache, x=x)


def extend(name, seqs, lo, hi, block, longest, pad):
    return dict(name=name, op="extend", seqs=seqs, lo=lo, hi=hi, block=block, longest=longest, pad=pad)


def release(name, seqs, block, longest, every):
    return dict(name=name, op="release", seqs=seqs, block=block, longest=longest, every=every)


def draw(rng):
    def log(lo, hi):
        return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4))))))

    op = rng.choice(["attention", "attention", "attention", "append", "append", "extend", "release"])
    hq, hkv, dh = rng.choice([(20, 4, 128), (16, 4, 128), (4, 4, 64), (4, 2, 64), (8, 1, 128), (7, 7, 128)])
    block = rng.choice([16, 32, 48, 64, 128])
    if op == "attention":
        seqs = log(1, 256)
        hi = log(1, min(16384, (1 << 20) // seqs))
        cache, q = rng.choice([("fp16", "fp16"), ("fp16", "fp32"), ("bf16", "bf16"), ("e4m3", "fp32"),
                               ("e4m3", "bf16"), ("e4m3", "fp16")])
        window = rng.choice([0, 0, 0, log(1, 4096)])
        c = attention("", seqs, hq, hkv, dh, block, log(1, hi), hi, cache, q, window)
    elif op == "append":
        cache, x = rng.choice([("fp16", "fp16"), ("fp16", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"),
                               ("e4m3", "fp32"), ("e4m3", "bf16"), ("e4m3", "fp16")])
        c = append("", log(1, 8192), rng.choice([0, log(1, 64)]), hq, hkv, dh, block, cache, x)
    elif op == "extend":
        seqs = log(1, 1025)
        hi = log(1, 512)
        c = extend("", seqs, log(1, hi), hi, block, log(64, 2048), rng.choice([0, log(1, 100)]))
    else:
        c = release("", log(1, 2047), block, log(1, 2048), rng.choice([1, 2, 3, 9]))
    del c["name"]
    return c


def _spread(n, lo, hi):
    """n whole numbers from hi down to lo, evenly over the logarithm (the case alone decides them)."""
    if n == 1:
        return [hi]
    return [max(lo, min(hi, int(round(hi * (lo / hi) ** (i / (n - 1)))))) for i in range(n)]


def _shuffled(values, g):
    t = torch.tensor(values, dtype=torch.int32, device="cuda")
    return t[torch.randperm(len(values), generator=g, device="cuda")]


def _ceil(a, b):
    return -(-a // b)


def _seen(length, window):
    return min(length, window) if window else length


def _draw_rows(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _table_of(lens, block, width, g, spare=7):
    """A block table over randomly placed pages for the given lengths (-1 where there is no page), and the other pages."""
    pages = (lens + block - 1) // block
    total = int(pages.sum())
    order = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    first = torch.cumsum(pages, 0) - pages
    mine = col[None] < pages[:, None]
    at = torch.where(mine, first[:, None] + col[None], 0)
    return torch.where(mine, order[at], -1).to(torch.int32).contiguous(), order[total:].contiguous(), total + spare


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "attention":
        B, hq, hkv, dh, bs = (case[k] for k in ("seqs", "hq", "hkv", "dh", "block"))
        s["lens"] = _shuffled(_spread(B, case["lo"], case["hi"]), g)
        s["table"], _, n = _table_of(s["lens"].long(), bs, _ceil(case["hi"], bs), g)
        s["q"] = _draw_rows((B, hq, dh), TYPES[case["q"]], g) * 2
        for x in ("k", "v"):
            rows = torch.randn((n, hkv, bs, dh), generator=g, device="cuda", dtype=torch.float32)
            s[x + "_scale"] = None
            if case["cache"] == "e4m3":
                s[x + "_scale"] = rows.abs().amax(-1) / E4M3_MAX
                rows = rows / s[x + "_scale"][..., None]
            s[x] = rows.to(TYPES[case["cache"]])
            # what a page holds behind its sequence's end was never written: nothing may depend on it
            last = (s["lens"].long() - 1).clamp(min=0)
            page = s["table"].gather(1, (last // bs)[:, None])[:, 0].long()
            dead = (torch.arange(bs, device="cuda")[None] > (last % bs)[:, None])[:, None, :, None]
            s[x].view(torch.uint8 if case["cache"] == "e4m3" else torch.int16)[page] |= (
                dead * (0x7F if case["cache"] == "e4m3" else 0x7FFF)).to(
                    torch.uint8 if case["cache"] == "e4m3" else torch.int16)
            del rows
    elif case["op"] == "append":
        T, pad, hq, hkv, dh, bs = (case[k] for k in ("rows", "pad", "hq", "hkv", "dh", "block"))
        n = _ceil(T, bs) + 5
        dt = TYPES[case["x"]]
        s["q"], s["k"], s["v"] = (_draw_rows((T + pad, h, dh), dt, g) for h in (hq, hkv, hkv))
        s["q_out"] = torch.zeros_like(s["q"])
        s["slots"] = torch.full((T + pad,), -1, dtype=torch.int32, device="cuda")
        s["slots"][:T] = torch.randperm(n * bs, generator=g, device="cuda")[:T]
        s["positions"] = torch.full((T + pad,), -1, dtype=torch.int32, device="cuda")
        s["positions"][:T] = torch.randint(0, 8704, (T,), generator=g, device="cuda")
        angle = torch.arange(8704, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, dh, 2, device="cuda", dtype=torch.float64) / dh)
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()
        for x in ("k", "v"):
            s[x + "_cache"] = torch.zeros((n, hkv, bs, dh), dtype=TYPES[case["cache"]], device="cuda")
            s[x + "_scale"] = (torch.ones((n, hkv, bs), dtype=torch.float32, device="cuda")
                               if case["cache"] == "e4m3" else None)
    elif case["op"] == "extend":
        R, bs = case["seqs"], case["block"]
        new = _spread(R, case["lo"], case["hi"])
        s["new_lens"] = _shuffled(new, g)
        s["lens"] = torch.randint(0, case["longest"] + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
        s["rows"] = sum(new) + case["pad"]
        s["table"], free, n = _table_of(s["lens"].long(), bs, _ceil(case["longest"] + case["hi"], bs), g)
        more = _ceil(case["hi"], bs) * R + R  # pages enough for every request
        s["free"] = torch.cat([free, torch.arange(n, n + more, dtype=torch.int32, device="cuda")])
        s["n_free"] = torch.tensor([s["free"].numel()], dtype=torch.int32, device="cuda")
    else:
        R, bs = case["seqs"], case["block"]
        s["lens"] = _shuffled(_spread(R, 1, case["longest"]), g)
        s["table"], free, n = _table_of(s["lens"].long(), bs, _ceil(case["longest"], bs), g)
        s["done"] = torch.randint(0, case["every"], (R,), generator=g, device="cuda") == 0
        s["free"] = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        s["free"][: free.numel()] = free
        s["n_free"] = torch.tensor([free.numel()], dtype=torch.int32, device="cuda")
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"attention": _plain_attention, "append": _plain_append, "extend": _plain_extend,
            "release": _plain_release}[s["op"]](s)


def _run_own(s):
    import persistent_monokernel_decode_gb300 as kie
    if s["op"] == "attention":
        return kie.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], window=s["window"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True)
    if s["op"] == "append":
        kie.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], positions=s["positions"],
                         rope=s["rope"], q=s["q"], q_out=s["q_out"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["k_cache"], s["v_cache"], s["q_out"], s["k_scale"], s["v_scale"]
    if s["op"] == "extend":
        step = kie.paged_extend(s["new_lens"], s["lens"], s["table"], s["free"], s["n_free"], s["block"], s["rows"])
        return (s["table"], step.lens, step.n_free, step.admitted, step.row_start, step.slots, step.positions,
                step.seqs)
    lens, n_free = kie.paged_release(s["done"], s["lens"], s["table"], s["free"], s["n_free"], s["block"])
    return s["free"], lens, n_free


# ---- plain forms -------------------------------------------------------------------------------------------

def _plain_attention(s):
    B, hq, hkv, dh, bs = (s[k] for k in ("seqs", "hq", "hkv", "dh", "block"))
    page = s["table"].clamp(min=0).long()
    lens = s["lens"].long()
    pos = torch.arange(page.shape[1] * bs, device="cuda")
    live = pos[None] < lens[:, None]
    if s["window"]:
        live &= pos[None] >= (lens - s["window"])[:, None]

    def gather(x, scale):
        x = s[x][page].float()  # [B, pages, hkv, bs, dh]
        if scale is not None:
            x = x * scale[page][..., None]
        x = x.transpose(1, 2).reshape(B, hkv, -1, dh)
        return x.masked_fill_(~live[:, None, :, None], 0.0)

    q = s["q"].float().view(B, hkv, hq // hkv, dh)
    score = torch.matmul(q, gather("k", s["k_scale"]).transpose(2, 3)) / math.sqrt(dh)
    score = score.masked_fill_(~live[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, gather("v", s["v_scale"])) / total.clamp(min=1e-30)
    lse = (top + torch.log(total))[..., 0]
    return o.reshape(B, hq, dh).to(s["q"].dtype), lse.reshape(B, hq)


def _rotate(x, rope):
    c, sn = rope[:, None, :, 0], rope[:, None, :, 1]
    a, b = x.float().chunk(2, -1)
    return torch.cat([a * c - b * sn, b * c + a * sn], -1)


def _plain_append(s):
    T, bs = s["rows"], s["block"]
    rope = s["rope"][s["positions"][:T].long()]
    slot = s["slots"][:T].long()
    page, at = slot // bs, slot % bs
    s["q_out"][:T] = _rotate(s["q"][:T], rope).to(s["q_out"].dtype)
    for x, rows in (("k", _rotate(s["k"][:T], rope)), ("v", s["v"][:T].float())):
        if s[x + "_scale"] is not None:
            top = rows.abs().amax(-1, keepdim=True)
            scale = torch.where(top > 0, top / E4M3_MAX, NO_SCALE)
            rows = (rows / scale).clamp(-E4M3_MAX, E4M3_MAX)
            s[x + "_scale"][page, :, at] = scale[..., 0]
            s[x + "_cache"].view(torch.uint8)[page, :, at] = rows.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            s[x + "_cache"][page, :, at] = rows.to(s[x + "_cache"].dtype)
    return s["k_cache"], s["v_cache"], s["q_out"], s["k_scale"], s["v_scale"]


def _plain_extend(s):
    bs, T, W = s["block"], s["rows"], s["table"].shape[1]
    lens, new, n_free = s["lens"].long(), s["new_lens"].long(), s["n_free"].long()
    ends = torch.cumsum(new, 0)
    have = (lens + bs - 1) // bs
    fits = (lens + new <= W * bs) & (ends <= T)
    need = torch.where(fits, (lens + new + bs - 1) // bs - have, 0)
    after = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (after <= n_free))
    need = torch.where(ok, need, 0)
    first = after - need
    col = torch.arange(W, device="cuda")
    fresh = (col[None] >= have[:, None]) & (col[None] < (have + need)[:, None])
    index = n_free - 1 - (first - have)[:, None] - col[None]
    s["table"].copy_(torch.where(fresh, s["free"][index.clamp(0, s["free"].numel() - 1)], s["table"]))
    row = torch.arange(T, device="cuda")
    seq = torch.searchsorted(ends, row, right=True)
    at = seq.clamp(max=lens.numel() - 1)
    live = (seq < lens.numel()) & ok[at]
    pos = lens[at] + row - (ends - new)[at]
    page = s["table"][at, (pos // bs).clamp(0, W - 1)]
    slot = page * bs + pos % bs
    start = torch.cat([torch.zeros_like(ends[:1]), ends])
    return (s["table"], torch.where(ok, lens + new, lens).int(), (n_free - need.sum()).int(), ok, start.int(),
            torch.where(live, slot, -1).int(), torch.where(live, pos, -1).int(), torch.where(live, at, -1).int())


def _plain_release(s):
    bs, W = s["block"], s["table"].shape[1]
    lens = s["lens"].long()
    pages = torch.where(s["done"], (lens + bs - 1) // bs, 0)
    after = torch.cumsum(pages, 0)
    col = torch.arange(W, device="cuda")
    mine = col[None] < pages[:, None]
    to = s["n_free"].long() + (after - pages)[:, None] + col[None]
    room = torch.cat([s["free"], s["free"][:1]])  # one place more, for what is not written
    room[torch.where(mine, to, s["free"].numel())] = s["table"]
    s["free"].copy_(room[:-1])
    return s["free"], torch.where(s["done"], 0, s["lens"]), (s["n_free"] + after[-1:]).int()


# ---- what a pass cannot do without ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "attention":
        n = sum(_seen(x, case["window"]) for x in _spread(case["seqs"], case["lo"], case["hi"]))
        row = case["dh"] * BYTES[case["cache"]] + (4 if case["cache"] == "e4m3" else 0)
        heads = case["seqs"] * case["hq"]
        pages = _ceil(n, case["block"])
        return {"bytes": 2 * n * case["hkv"] * row + heads * (2 * case["dh"] * BYTES[case["q"]] + 4) + 4 * pages,
                "flops": 4 * n * case["hq"] * case["dh"]}
    if case["op"] == "append":
        T, dh = case["rows"], case["dh"]
        row = dh * BYTES[case["cache"]] + (4 if case["cache"] == "e4m3" else 0)
        x = BYTES[case["x"]]
        return {"bytes": T * (2 * case["hq"] * dh * x + 2 * case["hkv"] * (dh * x + row) + 8 + dh * 4),
                "flops": 3 * T * (case["hq"] + case["hkv"]) * dh}
    if case["op"] == "extend":
        new = _spread(case["seqs"], case["lo"], case["hi"])
        pages = sum(new) // case["block"] + 1
        return {"bytes": 12 * (sum(new) + case["pad"]) + 21 * case["seqs"] + 8 * pages, "flops": sum(new)}
    lens = _spread(case["seqs"], 1, case["longest"])
    pages = sum(_ceil(x, case["block"]) for x in lens) // case["every"]
    return {"bytes": 8 * pages + 9 * case["seqs"], "flops": case["seqs"]}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    if case["op"] == "append":
        return _exact_append(s)
    return None  # whole numbers only


def _exact_attention(s):
    group, bs, dh = s["hq"] // s["hkv"], s["block"], s["dh"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - s["window"]) if s["window"] else 0
        at = torch.arange(lo, n, device="cuda")
        page = s["table"][b].long()[at // bs]
        rows = {}
        for x in ("k", "v"):
            rows[x] = s[x][page].double() if s[x].dtype != torch.float8_e4m3fn else s[x][page].float().double()
            rows[x] = rows[x][torch.arange(n - lo, device="cuda"), :, at % bs]  # [n, hkv, dh]
            if s[x + "_scale"] is not None:
                rows[x] = rows[x] * s[x + "_scale"][page, :, at % bs].double()[..., None]
        for h in range(s["hkv"]):
            heads = slice(h * group, (h + 1) * group)
            score = (s["q"][b, heads].double() @ rows["k"][:, h].T) / math.sqrt(dh)
            lse[b, heads] = torch.logsumexp(score, -1)
            out[b, heads] = torch.softmax(score, -1) @ rows["v"][:, h]
    return out, lse


def _exact_append(s):
    T, bs, half = s["rows"], s["block"], s["dh"] // 2
    cs = s["rope"].double()[s["positions"][:T].long()]
    c, sn = cs[:, None, :, 0], cs[:, None, :, 1]

    def turned(x):
        x = x[:T].double()
        return torch.cat([x[..., :half] * c - x[..., half:] * sn, x[..., half:] * c + x[..., :half] * sn], -1)

    q = s["q_out"].double()
    q[:T] = turned(s["q"])
    got = []
    scales = []
    page, at = s["slots"][:T].long() // bs, s["slots"][:T].long() % bs
    for x, rows in (("k", turned(s["k"])), ("v", s["v"][:T].double())):
        cache = s[x + "_cache"].float().double()
        if s[x + "_scale"] is None:
            cache[page, :, at] = rows
            scales.append(None)
        else:
            scale = rows.abs().amax(-1) / E4M3_MAX
            scale[scale == 0] = NO_SCALE
            held = s[x + "_scale"].double()
            held[page, :, at] = scale
            cache[page, :, at] = _nearest_e4m3(rows / scale[..., None])
            scales.append(held)
        got.append(cache)
    return got[0], got[1], q, scales[0], scales[1]


def _nearest_e4m3(x):
    """The nearest value of three fraction bits, exponents from -6 on (below, steps of 2^-9); ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
