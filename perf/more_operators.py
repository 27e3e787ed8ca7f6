"""Workloads of the operators for several continuations of one prompt: attention that reads a shared prefix once, forking
and freeing of sequences whose pages are shared, copies of pages, compaction of the cache, and log probabilities of tokens.

``run`` computes an operator in elementary torch operations when ``own`` is false, and through this package's entry
points when it is true. ``exact`` is the operator's definition in 64 bits. Head layouts and vocabularies are those of the
models in ``synth/configs.py``: 20 query heads over 4 K/V heads of 128, 25 layers (the 2B model), 16 over 4 of 128, 24
layers (the sparse-MoE model), 4 over 4 and 4 over 2 of 64 (the tiny models); 32,000 and 4,096 tokens.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4, "e4m3": 1}
E4M3_MAX = 448.0


def listed():
    return [
        # A beam search of four over one prompt of the 2B model's benchmark length, early on: latency.
        attention("prefix attention: 2B, 4 beams of 1,024", 4, 1, 0, 20, 4, 128, 16, 1024, 1024, 1, 128, "fp16", "fp32"),
        # 64 samples of one long prompt, up to the long-context benchmark's 512 new tokens each.
        attention("prefix attention: 2B, 64 samples of 8,192", 64, 1, 0, 20, 4, 128, 16, 8192, 8192, 1, 512, "fp16", "fp16"),
        # A full serving batch of the sparse-MoE model's heads under eight system prompts: the largest.
        attention("prefix attention: MoE heads, 256 under 8", 256, 8, 0, 16, 4, 128, 64, 4096, 4096, 16, 1024, "bf16", "bf16"),
        # A batch of odd size on an 8-bit cache, prompts of every length and shared by few or many, six requests alone.
        attention("prefix attention: 2B, 61 under 5 on e4m3", 61, 5, 6, 20, 4, 128, 32, 513, 8191, 1, 777, "e4m3", "fp16"),
        # A step of a beam search of eight over four prompts: latency.
        fork("fork: 32 rows in beams of 8", 32, 8, 16, 128, 1152),
        # A step of a large batch of beam searches with contexts up to the longest, one row more than whole beams.
        fork("fork: 1,025 rows in beams of 4", 1025, 4, 16, 64, 8704),
        # The half-filled last pages of a beam search's new rows, in every layer of the 2B model.
        copy("copy: 2B, 24 open pages", 24, 25, 4, 128, 16, "fp16", True),
        # A compaction of the sparse-MoE model's 8-bit cache: whole pages of every layer.
        copy("copy: MoE, 256 pages on e4m3", 256, 24, 4, 128, 64, "e4m3", False),
        # A small cache, half empty.
        compact("compact: 512 pages", 512, 32, 16, 64, 50),
        # A large cache after many requests have ended, to be shrunk.
        compact("compact: 100,003 pages", 100003, 1025, 16, 2048, 37),
        # The next step of four beams over the 2B model's vocabulary: latency.
        logprobs("log probabilities: 4 beams", 4, 32000, 8, "fp32"),
        # A long prompt's tokens scored with their alternatives, the logits in 16 bits, padded to a captured size.
        logprobs("log probabilities: 8,191 rows", 8191, 32000, 20, "bf16"),
    ]


def attention(name, seqs, groups, alone, hq, hkv, dh, block, prefix_lo, prefix_hi, lo, hi, cache, q):
    return dict(name=name, op="attention", seqs=seqs, groups=groups, alone=alone, hq=hq, hkv=hkv, dh=dh, block=block,
                prefix_lo=prefix_lo, prefix_hi=prefix_hi, lo=lo, hi=hi, cache=cache, q=q)


def fork(name, rows, beams, block, lo, hi):
    return dict(name=name, op="fork", rows=rows, beams=beams, block=block, lo=lo, hi=hi)


def copy(name, pairs, layers, hkv, dh, block, cache, part):
    return dict(name=name, op="copy", pairs=pairs, layers=layers, hkv=hkv, dh=dh, block=block, cache=cache, part=part)


def compact(name, pages, rows, block, longest, percent):
    return dict(name=name, op="compact", pages=pages, rows=rows, block=block, longest=longest, percent=percent)


def logprobs(name, rows, vocab, top, logits):
    return dict(name=name, op="logprobs", rows=rows, vocab=vocab, top=top, logits=logits)


def draw(rng):
    def log(lo, hi):
        return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4))))))

    op = rng.choice(["attention", "attention", "attention", "fork", "copy", "compact", "logprobs", "logprobs"])
    hq, hkv, dh = rng.choice([(20, 4, 128), (16, 4, 128), (4, 4, 64), (4, 2, 64), (8, 1, 128), (7, 7, 128)])
    block = rng.choice([16, 32, 48, 64, 128])
    if op == "attention":
        seqs = log(1, 256)
        groups = log(1, max(1, seqs // 2))
        alone = rng.choice([0, 0, log(1, seqs) // 2])
        prefix = log(1, min(8192, (1 << 20) // seqs))
        cache, q = rng.choice([("fp16", "fp16"), ("fp16", "fp32"), ("bf16", "bf16"), ("e4m3", "fp32"),
                               ("e4m3", "bf16"), ("e4m3", "fp16")])
        lo = log(1, 256)
        c = attention("", seqs, min(groups, seqs - alone), alone, hq, hkv, dh, block, log(1, prefix), prefix, lo,
                      lo + log(1, 512), cache, q)
    elif op == "fork":
        lo = log(1, 2048)
        c = fork("", log(1, 1025), rng.choice([1, 2, 3, 4, 8, 16]), block, lo, log(lo, 4096))
    elif op == "copy":
        c = copy("", log(1, 128), log(1, 24), hkv, dh, rng.choice([16, 32, 48, 64]), rng.choice(["fp16", "bf16", "e4m3"]),
                 rng.choice([True, False]))
    elif op == "compact":
        c = compact("", log(2, 100003), log(1, 1025), block, log(1, 2048), rng.randint(0, 100))
    else:
        rows = log(1, 4096)
        c = logprobs("", rows, log(32, min(200000, (1 << 27) // rows)), rng.choice([0, 1, 5, 20, 32]),
                     rng.choice(["fp32", "fp16", "bf16"]))
    del c["name"]
    return c


def _spread(n, lo, hi):
    """n whole numbers from hi down to lo, evenly over the logarithm (the case alone decides them)."""
    if n == 1:
        return [hi]
    return [max(lo, min(hi, int(round(hi * (lo / hi) ** (i / (n - 1)))))) for i in range(n)]


def _sizes(n, groups):
    """n rows in groups of very different sizes, one row each at least."""
    weights = [i + 1 for i in range(groups)]
    total = sum(weights)
    cuts = [min(n - (groups - i - 1), max(i + 1, n * sum(weights[: i + 1]) // total)) for i in range(groups)]
    cuts = [0] + cuts[:-1] + [n] if groups else []
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _ceil(a, b):
    return -(-a // b)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prefixes(case):
    return _spread(case["groups"], case["prefix_lo"], case["prefix_hi"]) if case["groups"] else []


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"attention": _prepare_attention, "fork": _prepare_fork, "copy": _prepare_copy, "compact": _prepare_compact,
            "logprobs": _prepare_logprobs}[case["op"]](dict(case), g)


def _prepare_attention(s, g):
    """Sequences in groups of neighbours, each group's prefix in pages that its table rows share as far as they are full;
    behind it each sequence has pages of its own. The sequences that are alone come last."""
    B, hq, hkv, dh, bs = (s[k] for k in ("seqs", "hq", "hkv", "dh", "block"))
    sizes, prefixes = _sizes(B - s["alone"], s["groups"]), _prefixes(s)
    tails = torch.tensor(_spread(B, s["lo"], s["hi"]))[torch.randperm(B, generator=torch.Generator().manual_seed(B))].tolist()
    table, lens, n = [], [], 0
    for size, prefix in zip(sizes + [1] * s["alone"], prefixes + [0] * s["alone"]):
        shared = list(range(n, n + prefix // bs))
        n += len(shared)
        for _ in range(size):
            length = prefix + tails[len(lens)]
            mine = _ceil(length, bs) - len(shared)
            table.append(shared + list(range(n, n + mine)))
            lens.append(length)
            n += mine
    order = torch.randperm(n + 7, generator=g, device="cuda").to(torch.int32)
    width = max(len(r) for r in table)
    at = _ints([r + [-1] * (width - len(r)) for r in table])
    s["table"] = torch.where(at >= 0, order[at.clamp(min=0).long()], -1).contiguous()
    s["lens"] = _ints(lens)
    starts = [0]
    for size in sizes:
        starts.append(starts[-1] + size)
    s["group_start"], s["prefix_lens"] = _ints(starts), _ints(prefixes)
    s["q"] = (torch.randn((B, hq, dh), generator=g, device="cuda") * 2).to(TYPES[s["q"]])
    last = (s["lens"].long() - 1).clamp(min=0)
    page = s["table"].long().gather(1, (last // bs)[:, None])[:, 0]
    dead = (torch.arange(bs, device="cuda")[None] > (last % bs)[:, None])[:, None, :, None]
    for x in ("k", "v"):
        rows = torch.randn((n + 7, hkv, bs, dh), generator=g, device="cuda")
        s[x + "_scale"] = None
        bits, nan = (torch.uint8, 0x7F) if s["cache"] == "e4m3" else (torch.int16, 0x7FFF)
        if s["cache"] == "e4m3":
            s[x + "_scale"] = rows.abs().amax(-1) / E4M3_MAX
            rows = rows / s[x + "_scale"][..., None]
        s[x] = rows.to(TYPES[s["cache"]])
        # what a page holds behind its sequence's end was never written: nothing may depend on it
        s[x].view(bits)[page] |= (dead * nan).to(bits)
    return s


def _prepare_fork(s, g):
    """Requests of `beams` rows each, all of a request's rows of one length: three quarters of it, as far as pages are
    full, in pages that the rows share, the rest in pages of their own. Every row continues a random row of its request;
    one request in eight has ended."""
    R, beams, bs = s["rows"], s["beams"], s["block"]
    requests = _ceil(R, beams)
    of = torch.arange(R, device="cuda") // beams
    length = _ints(_spread(requests, s["lo"], s["hi"])).long()[torch.randperm(requests, generator=g, device="cuda")]
    lens, shared = length[of], (length * 3 // 4 // bs)
    first = torch.cumsum(shared, 0) - shared
    mine = (lens + bs - 1) // bs - shared[of]
    own_first = shared.sum() + torch.cumsum(mine, 0) - mine
    width = _ceil(s["hi"], bs) + 1
    col = torch.arange(width, device="cuda")[None]
    at = torch.where(col < shared[of][:, None], first[of][:, None] + col, own_first[:, None] + col - shared[of][:, None])
    live = col < (shared[of] + mine)[:, None]
    n = int(shared.sum() + mine.sum())
    total = int(shared.sum() + beams * ((length + bs - 1) // bs - shared).sum()) + R + 9
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.where(live, order[torch.where(live, at, 0)], -1).contiguous()
    s["lens"] = lens.int()
    holders = torch.zeros(total, dtype=torch.int32, device="cuda")
    holders.scatter_add_(0, s["table"][live].long(), torch.ones(int(live.sum()), dtype=torch.int32, device="cuda"))
    s["shares"] = (holders - 1).clamp(min=0)
    s["free"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    s["free"][: total - n] = order[n:]
    s["n_free"] = _ints([total - n])
    size = torch.minimum(torch.full_like(of, beams), R - of * beams)
    pick = of * beams + torch.randint(0, 1 << 20, (R,), generator=g, device="cuda") % size
    ended = (torch.randint(0, 8, (requests,), generator=g, device="cuda") == 0)[of]
    s["parents"] = torch.where(ended, -1, pick).int()
    return s


def _prepare_copy(s, g):
    N, bs = s["pairs"], s["block"]
    shape = (s["layers"], 2 * N + 5, s["hkv"], bs, s["dh"])
    order = torch.randperm(2 * N + 5, generator=g, device="cuda").to(torch.int32)
    s["src"], s["dst"] = order[:N].contiguous(), order[N:2 * N].contiguous()
    if N > 2:
        s["src"][N // 2] = -1  # a row that needs no copy
    s["n_rows"] = torch.randint(1, bs, (N,), generator=g, device="cuda", dtype=torch.int32) if s["part"] else None
    for x in ("k", "v"):
        if s["cache"] == "e4m3":
            s[x] = torch.randint(0, 127, shape, generator=g, device="cuda", dtype=torch.uint8).view(TYPES["e4m3"])
            s[x + "_scale"] = torch.rand(shape[:4], generator=g, device="cuda")
        else:
            s[x] = torch.randn(shape, generator=g, device="cuda").to(TYPES[s["cache"]])
            s[x + "_scale"] = None
    return s


def _prepare_compact(s, g):
    """A cache of which `percent` per cent of the pages are free, wherever they lie; rows hold the others (as far as the
    table goes), the first page of each row being shared with the row before it."""
    n, R, bs = s["pages"], s["rows"], s["block"]
    free = max(1, min(n - 1, n * s["percent"] // 100))
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    s["free"] = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    s["free"][:free] = order[:free]
    s["n_free"] = _ints([free])
    held = order[free:]
    width = _ceil(s["longest"], bs) + 1
    pages = torch.randint(0, max(1, min(width, _ceil(n - free, R)) + 1), (R,), generator=g, device="cuda").clamp(max=width)
    first = torch.cumsum(pages, 0) - pages
    col = torch.arange(width, device="cuda")[None]
    at = first[:, None] + col
    live = (col < pages[:, None]) & (at < held.numel())
    s["table"] = torch.where(live, held[torch.where(live, at, 0)], -1).contiguous()
    s["lens"] = (live.sum(1) * bs - torch.randint(0, bs, (R,), generator=g, device="cuda")).clamp(min=0).int()
    s["shares"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    s["shares"][held.long()] = torch.randint(0, 3, (held.numel(),), generator=g, device="cuda", dtype=torch.int32)
    return s


def _prepare_logprobs(s, g):
    N, V = s["rows"], s["vocab"]
    s["logits"] = torch.empty((N, V), dtype=TYPES[s["logits"]], device="cuda")
    for i in range(0, N, 1024):
        s["logits"][i:i + 1024] = torch.randn((min(1024, N - i), V), generator=g, device="cuda") * 3
    s["logits"][:, V // 3:V // 3 + V // 50] = -math.inf  # tokens that a grammar rules out
    s["tokens"] = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    s["tokens"][N - N // 7:] = -1  # padding: nothing was drawn there
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"attention": _plain_attention, "fork": _plain_fork, "copy": _plain_copy, "compact": _plain_compact,
            "logprobs": _plain_logprobs}[s["op"]](s)


def _run_own(s):
    import persistent_monokernel_decode_gb300 as kie
    if s["op"] == "attention":
        return kie.paged_prefix_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["group_start"], s["prefix_lens"],
                                          k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True)
    if s["op"] == "fork":
        f = kie.paged_fork(s["parents"], s["lens"], s["table"], s["shares"], s["free"], s["n_free"], s["block"])
        return s["table"], s["shares"], s["free"], f.lens, f.n_free, f.ok, f.copy_src, f.copy_dst, f.copy_rows
    if s["op"] == "copy":
        kie.paged_copy(s["src"], s["dst"], s["k"], s["v"], rows=s["n_rows"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["k"], s["v"], s["k_scale"], s["v_scale"]
    if s["op"] == "compact":
        m = kie.paged_compact(s["lens"], s["table"], s["shares"], s["free"], s["n_free"], s["block"])
        return s["table"], s["shares"], s["free"], m.n_free, m.src, m.dst, m.page_map
    p = kie.token_logprobs(s["logits"], s["tokens"], top=s["top"])
    return p.logprob, p.entropy, p.top_ids, p.top_logprobs


# ---- plain forms -------------------------------------------------------------------------------------------

def _prefix_of_rows(s):
    """Per row: the length of its prefix (0 where it is alone), and the row whose pages hold it."""
    row = torch.arange(s["seqs"], device="cuda")
    if not s["groups"]:
        return torch.zeros_like(row), row
    start = s["group_start"].long()
    group = torch.searchsorted(start, row, right=True) - 1
    inside = (group >= 0) & (group < s["groups"])
    group = group.clamp(0, s["groups"] - 1)
    return torch.where(inside, s["prefix_lens"].long()[group], 0), torch.where(inside, start[group], row)


def _plain_attention(s):
    B, hq, hkv, dh, bs = (s[k] for k in ("seqs", "hq", "hkv", "dh", "block"))
    prefix, head = _prefix_of_rows(s)
    lens = s["lens"].long()
    pos = torch.arange(s["table"].shape[1] * bs, device="cuda")
    live = pos[None] < lens[:, None]
    table = s["table"].long()
    through = torch.where(pos[None] < prefix[:, None], head[:, None], torch.arange(B, device="cuda")[:, None])
    page = table[through, (pos // bs)[None]].clamp(min=0)
    offset = (pos % bs)[None].expand_as(page)

    def gather(x, scale):
        x = s[x][page, :, offset].float()  # [B, positions, hkv, dh]
        if scale is not None:
            x = x * scale[page, :, offset][..., None]
        return x.transpose(1, 2).masked_fill(~live[:, None, :, None], 0.0)

    q = s["q"].float().view(B, hkv, hq // hkv, dh)
    score = torch.matmul(q, gather("k", s["k_scale"]).transpose(2, 3)) / math.sqrt(dh)
    score = score.masked_fill_(~live[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, gather("v", s["v_scale"])) / total.clamp(min=1e-30)
    lse = (top + torch.log(total))[..., 0]
    return o.reshape(B, hq, dh).to(s["q"].dtype), lse.reshape(B, hq)


def _plain_fork(s):
    bs, (R, W), n = s["block"], s["table"].shape, s["shares"].numel()
    row = torch.arange(R, device="cuda")
    lens, n_free, old = s["lens"].long(), s["n_free"].long(), s["table"].clone()
    parent = torch.where(s["parents"].long() >= R, row, s["parents"].long())
    live = parent >= 0
    at = parent.clamp(min=0)
    kids = torch.zeros_like(row).scatter_add(0, at, live.long())
    first = torch.full_like(row, R).scatter_reduce(0, at, torch.where(live, row, R), "amin")
    keeper = torch.where(parent == row, row, first)
    pages = ((lens.clamp(min=0) + bs - 1) // bs).clamp(max=W)
    part = (lens > 0) & (lens % bs != 0) & (lens <= W * bs)  # the last page is not full
    need = live & part[at] & (keeper[at] != row)
    rank = torch.cumsum(need.long(), 0) - need.long()
    total = need.long().sum()
    ok = total <= n_free
    fresh = s["free"][(n_free - 1 - rank).clamp(0, s["free"].numel() - 1)]
    need = need & ok
    col = torch.arange(W, device="cuda")[None]
    last = (pages - 1)[:, None]
    taken = torch.where(need[:, None] & (col == last[at]), fresh[:, None], old[at])
    moved = (live & (at != row) & ok)[:, None] & (col < pages[at][:, None])
    s["table"].copy_(torch.where(moved, taken, old))
    change = torch.where(part[:, None] & (col == last), kids.clamp(max=1)[:, None], kids[:, None]) - 1
    counted = (col < pages[:, None]) & (old >= 0) & (old < n) & ok
    shares = s["shares"].long().scatter_add(0, torch.where(counted, old, 0).long().view(-1),
                                            torch.where(counted, change, 0).view(-1))
    freed = (shares < 0) & ok
    s["shares"].copy_(torch.where(freed, 0, shares))
    to = n_free - total + torch.cumsum(freed.long(), 0) - 1
    room = torch.cat([s["free"], s["free"][:1]])  # one place more, for what is not written
    cap = s["free"].numel()
    room[torch.where(freed & (to < cap), to, cap)] = torch.arange(n, device="cuda", dtype=torch.int32)
    s["free"].copy_(room[:-1])
    left = torch.where(ok, (n_free - total + freed.sum()).clamp(max=cap), n_free).int()
    copies = [torch.where(need, x.int(), none) for x, none in (
        (old[at].gather(1, last[at].clamp(min=0))[:, 0], -1), (fresh, -1), (lens[at] % bs, 0))]
    return (s["table"], s["shares"], s["free"],
            torch.where(ok, torch.where(live, lens[at], 0), lens).int(), left, ok, *copies)


def _plain_copy(s):
    bs = s["block"]
    use = (s["src"] >= 0) & (s["dst"] >= 0)
    src, dst = s["src"][use].long(), s["dst"][use].long()
    rows = torch.full_like(src, bs) if s["n_rows"] is None else s["n_rows"][use].long()
    mask = (torch.arange(bs, device="cuda")[None] < rows[:, None])[None, :, None, :]
    for x in ("k", "v"):
        c = s[x].view(torch.uint8) if s["cache"] == "e4m3" else s[x]
        c[:, dst] = torch.where(mask[..., None], c[:, src], c[:, dst])
        if s[x + "_scale"] is not None:
            c = s[x + "_scale"]
            c[:, dst] = torch.where(mask, c[:, src], c[:, dst])
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def _plain_compact(s):
    bs, W, n = s["block"], s["table"].shape[1], s["shares"].numel()
    page = torch.arange(n, device="cuda")
    stack = s["free"].long()
    listed_free = (torch.arange(stack.numel(), device="cuda") < s["n_free"].long()) & (stack >= 0) & (stack < n)
    free = torch.zeros(n + 1, dtype=torch.bool, device="cuda")
    free[torch.where(listed_free, stack, n)] = True
    free = free[:n]
    live = (~free).long().sum()
    hole, high = free & (page < live), ~free & (page >= live)
    most = n // 2
    rank_hole, rank_high = torch.cumsum(hole.long(), 0) - 1, torch.cumsum(high.long(), 0) - 1
    dst = torch.full((n + 1,), -1, dtype=torch.int64, device="cuda")
    src = dst.clone()
    dst[torch.where(hole, rank_hole, n)] = page
    src[torch.where(high, rank_high, n)] = page
    moves = high.long().sum()
    index = torch.arange(most, device="cuda")
    dst, src = (torch.where(index < moves, x[:most], -1) for x in (dst, src))
    to = torch.where(high, dst[rank_high.clamp(0, max(most - 1, 0))], page) if most else page
    page_map = torch.where(free, -1, to)
    col = torch.arange(W, device="cuda")[None]
    held = (col < ((s["lens"].long().clamp(min=0) + bs - 1) // bs)[:, None]) & (s["table"] >= 0) & (s["table"] < n)
    there = page_map[torch.where(held, s["table"], 0).long()]
    s["table"].copy_(torch.where(held & (there >= 0), there, s["table"]))
    shares = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    shares[torch.where(free, n, to)] = s["shares"]
    s["shares"].copy_(shares[:n])
    place = torch.arange(stack.numel(), device="cuda")
    s["free"].copy_(torch.where(place < n - live, n - 1 - place, stack))
    left = (n - live).clamp(max=stack.numel())
    return s["table"], s["shares"], s["free"], left.int()[None], src.int(), dst.int(), page_map.int()


def _plain_logprobs(s):
    N, V, k = s["rows"], s["vocab"], s["top"]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    logp = x - lse
    entropy = -torch.where(e > 0, logp * (e / total), 0.0).sum(1)
    asked = s["tokens"] >= 0
    mine = logp.gather(1, s["tokens"].clamp(min=0).long()[:, None])[:, 0]
    value, index = torch.sort(x, dim=1, descending=True, stable=True)  # equal logits: the lowest index first
    return torch.where(asked, mine, 0.0), entropy, index[:, :k].int(), value[:, :k] - lse


# ---- what a pass cannot do without ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "attention":
        B, sizes = case["seqs"], _sizes(case["seqs"] - case["alone"], case["groups"])
        tails = sum(_spread(B, case["lo"], case["hi"]))
        prefixes = _prefixes(case)
        row = case["dh"] * BYTES[case["cache"]] + (4 if case["cache"] == "e4m3" else 0)
        read = sum(prefixes) + tails
        seen = sum(a * b for a, b in zip(sizes, prefixes)) + tails
        heads = B * case["hq"]
        return {"bytes": 2 * read * case["hkv"] * row + heads * (2 * case["dh"] * BYTES[case["q"]] + 4) +
                4 * _ceil(read, case["block"]), "flops": 4 * seen * case["hq"] * case["dh"]}
    if case["op"] == "fork":
        lens = _spread(_ceil(case["rows"], case["beams"]), case["lo"], case["hi"])
        pages = sum(_ceil(x, case["block"]) for x in lens) * case["beams"]
        every = sum(x * 3 // 4 // case["block"] for x in lens) + pages // 4
        return {"bytes": 8 * pages + 8 * every + 24 * case["rows"], "flops": pages}
    if case["op"] == "copy":
        row = case["dh"] * BYTES[case["cache"]] + (4 if case["cache"] == "e4m3" else 0)
        rows = case["pairs"] * (case["block"] // 2 if case["part"] else case["block"])
        return {"bytes": 4 * rows * row * case["hkv"] * case["layers"], "flops": rows}
    if case["op"] == "compact":
        n, free = case["pages"], max(1, case["pages"] * case["percent"] // 100)
        return {"bytes": 8 * free + 12 * n + 8 * min(n - free, case["rows"] * _ceil(case["longest"], case["block"])),
                "flops": n}
    N, V = case["rows"], case["vocab"]
    return {"bytes": N * V * BYTES[case["logits"]] + N * (12 + 8 * case["top"]), "flops": 6 * N * V}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    return None  # whole numbers and copies only


def _exact_attention(s):
    group, bs, dh = s["hq"] // s["hkv"], s["block"], s["dh"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    starts, prefixes = s["group_start"].tolist(), s["prefix_lens"].tolist()
    first = list(range(s["seqs"]))
    shared = [0] * s["seqs"]
    for a, b, prefix in zip(starts, starts[1:], prefixes):
        for r in range(a, b):
            first[r], shared[r] = a, prefix
    for b, n in enumerate(s["lens"].tolist()):
        at = torch.arange(n, device="cuda")
        cut = min(n, shared[b])
        page = torch.cat([s["table"][first[b]].long()[at[:cut] // bs], s["table"][b].long()[at[cut:] // bs]])
        rows = {}
        for x in ("k", "v"):
            rows[x] = s[x][page, :, at % bs].float().double()  # [n, hkv, dh]; fp32 holds every value exactly
            if s[x + "_scale"] is not None:
                rows[x] = rows[x] * s[x + "_scale"][page, :, at % bs].double()[..., None]
        for h in range(s["hkv"]):
            heads = slice(h * group, (h + 1) * group)
            score = (s["q"][b, heads].double() @ rows["k"][:, h].T) / math.sqrt(dh)
            lse[b, heads] = torch.logsumexp(score, -1)
            out[b, heads] = torch.softmax(score, -1) @ rows["v"][:, h]
    return out, lse


def _exact_logprobs(s):
    N, k = s["rows"], s["top"]
    logprob, entropy = (torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(2))
    top = torch.zeros((N, k), dtype=torch.float64, device="cuda")
    for i in range(0, N, 512):
        x = s["logits"][i:i + 512].double()
        p = torch.log_softmax(x, 1)
        weight = p.exp()
        entropy[i:i + 512] = -torch.where(weight == 0, 0.0, weight * p).sum(1)
        tokens = s["tokens"][i:i + 512].long()
        logprob[i:i + 512] = torch.where(tokens < 0, 0.0, p.gather(1, tokens.clamp(min=0)[:, None])[:, 0])
        top[i:i + 512] = torch.topk(p, k, 1).values
    return logprob, entropy, None, top
