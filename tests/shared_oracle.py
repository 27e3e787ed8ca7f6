"""Plain implementations of the operators for sequences that share pages, and of the log probabilities (Python integers and
fp64 tensors), for the tests."""
import math

import torch

import paged_oracle
from paged_oracle import ceil_div


def fork(parents, lens, table, shares, free, n_free, bs):
    """(table, shares, free, lens, n_free, ok, copy_src, copy_dst, copy_rows) of kie_paged_fork."""
    R, W, n = len(lens), len(table[0]) if table else 0, len(shares)
    old = [list(r) for r in table]
    table, shares, free = [list(r) for r in table], list(shares), list(free)
    parent = [r if p >= R else p for r, p in enumerate(parents)]
    pages = [min(ceil_div(max(l, 0), bs), W) for l in lens]
    part = [l > 0 and l % bs != 0 and ceil_div(l, bs) <= W for l in lens]
    kids = [[r for r in range(R) if parent[r] == p] for p in range(R)]
    keeper = [p if p in kids[p] else kids[p][0] if kids[p] else -1 for p in range(R)]
    need = [r for r in range(R) if parent[r] >= 0 and part[parent[r]] and keeper[parent[r]] != r]
    avail = min(max(n_free, 0), len(free))
    none = ([-1] * R, [-1] * R, [0] * R)
    if len(need) > avail:
        return table, shares, free, list(lens), n_free, False, *none
    src, dst, rows = none
    for r in range(R):
        p = parent[r]
        if p >= 0 and p != r:
            for j in range(pages[p]):
                table[r][j] = old[p][j]
    for k, r in enumerate(need):
        p = parent[r]
        src[r], dst[r], rows[r] = old[p][pages[p] - 1], free[avail - 1 - k], lens[p] % bs
        table[r][pages[p] - 1] = dst[r]
    for p in range(R):
        for j in range(pages[p]):
            last = part[p] and j == pages[p] - 1
            if 0 <= old[p][j] < n:
                shares[old[p][j]] += (min(len(kids[p]), 1) if last else len(kids[p])) - 1
    at = avail - len(need)
    for x in range(n):
        if shares[x] < 0:
            shares[x] = 0
            if at < len(free):
                free[at] = x
            at += 1
    return (table, shares, free, [lens[p] if p >= 0 else 0 for p in parent], min(at, len(free)), True, src, dst, rows)


def compact(lens, table, shares, free, n_free, bs):
    """(table, shares, free, n_free, src, dst, page_map) of kie_paged_compact."""
    n = len(shares)
    table, free = [list(r) for r in table], list(free)
    unused = {x for x in free[:min(max(n_free, 0), len(free))] if 0 <= x < n}
    live = n - len(unused)
    dst = [x for x in range(live) if x in unused]
    src = [x for x in range(live, n) if x not in unused]
    page_map = [-1 if x in unused else x for x in range(n)]
    for a, b in zip(src, dst):
        page_map[a] = b
    out = [0] * n
    for x in range(n):
        if page_map[x] >= 0:
            out[page_map[x]] = shares[x]
    for r, l in enumerate(lens):
        for j in range(min(ceil_div(max(l, 0), bs), len(table[r]))):
            if 0 <= table[r][j] < n and page_map[table[r][j]] >= 0:
                table[r][j] = page_map[table[r][j]]
    left = min(n - live, len(free))
    free[:left] = [n - 1 - i for i in range(left)]
    pad = [-1] * (n // 2 - len(src))
    return table, out, free, left, src + pad, dst + pad, page_map


def prefix_attention(q, k, v, table, lens, start, prefix, scale, k_scale=None, v_scale=None):
    """paged_oracle.attention of the rows' positions, those of a prefix read through the group's longest row: the cache
    taken as pages of one position."""
    B, cap = q.shape[0], table.shape[1] * k.shape[2]
    bs, n = k.shape[2], k.shape[0]
    lens = [min(max(int(l), 0), cap) for l in lens]
    at = torch.arange(cap, device=q.device)
    own = torch.where((table >= 0) & (table < n), table, -1).long()
    slots = torch.where(own[:, at // bs] >= 0, own[:, at // bs] * bs + at % bs, -1)
    edge = 0
    starts = []
    for s in start:
        edge = max(edge, min(max(s, 0), B))
        starts.append(edge)
    for a, b, p in zip(starts, starts[1:], prefix):
        p = min(max(p, 0), cap)
        reach = [min(lens[r], p) for r in range(a, b)]
        if reach:
            slots[a:b, :p] = slots[a + reach.index(max(reach)), :p].clone()
    flat = [x.permute(0, 2, 1, 3).reshape(n * bs, x.shape[1], 1, x.shape[3]) for x in
            ((k, v) if k.dtype != torch.float8_e4m3fn else (k.float(), v.float()))]
    flat_scale = [None if s is None else s.permute(0, 2, 1).reshape(n * bs, -1, 1) for s in (k_scale, v_scale)]
    return paged_oracle.attention(q, *flat, slots.int(), torch.tensor(lens), scale, 0, *flat_scale)


def logprobs(x, tokens, top):
    """fp64 (logprob, entropy, top_ids, top_logprobs) of logits x [N, V], for rows without NaN and +inf."""
    x = x.double()
    d = x - x.amax(1, keepdim=True)  # the log-sum is taken relative to the largest: of logits of 1e30, 64 bits hold no ln 2
    logp = torch.where(torch.isnan(d), -math.inf, d - d.exp().sum(1, keepdim=True).log())
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    inside = (tokens >= 0) & (tokens < x.shape[1])
    mine = logp.gather(1, tokens.clamp(0, x.shape[1] - 1).long()[:, None])[:, 0]
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
    return torch.where(inside, mine, 0.0), entropy, ids, logp.gather(1, ids)


def logprobs_bounds(x):
    """Error bounds (lse, factor of |ln p|, entropy) of kie_token_logprobs for rows of logits x [N, V].

    With d = x - max and w = exp d: d is rounded once (2^-24 relative) and the exponential's argument once more where it
    is formed in powers of two (2^-24), so w is off by |d| 2^-22 + 2^-21 of itself, a generous exponential included. The
    sum of the V weights goes through at most V / 128 + 64 additions on any path (128 threads or more to a row, then
    joins), each off by 2^-24 of the sum. So ln of the sum is off by E|d| 2^-22 + 2^-21 + (V / 128 + 64) 2^-24 plus its own
    rounding, 2^-22 of its size (at most ln V). ln p = d - ln sum: two more roundings, 2^-23 of |ln p| (and of |d|, which
    is no larger). The entropy is ln sum - E d: the sum of w d is off in the same way (its terms' own roundings are 2^-23
    of |d| more, and the errors of the weights now count |d| times: E d^2 2^-22 + E|d| 2^-21), and so is the division."""
    d = x.double() - x.double().amax(1, keepdim=True)
    d = torch.where(torch.isnan(d), 0.0, d)
    w = d.exp()
    total = w.sum(1)
    e1 = torch.where(w > 0, w * d.abs(), 0.0).sum(1) / total
    e2 = torch.where(w > 0, w * d * d, 0.0).sum(1) / total
    adds = (x.shape[1] / 128 + 64) * 2.0 ** -24
    lse = e1 * 2.0 ** -22 + 2.0 ** -21 + adds + 2.0 ** -22 * total.log()
    entropy = lse + e2 * 2.0 ** -22 + e1 * (2.0 ** -21 + e1 * 2.0 ** -22 + 2 * adds + 2.0 ** -21) + 2.0 ** -23 * total.log()
    return lse, 2.0 ** -22, entropy
