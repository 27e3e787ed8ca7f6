"""Plain implementations of the paged-cache operators (Python integers and fp64 tensors), for the tests."""
import math

import torch

NO_SCALE = 2.0 ** -126  # of an all-zero row


def ceil_div(a, b):
    return -(-a // b)


def extend(new_lens, lens, table, free, n_free, bs, n_rows):
    """(table, lens, n_free, admitted, row_start, slots, positions, seqs) of kie_paged_extend, lists of ints."""
    table = [list(r) for r in table]
    out_lens, admitted, starts = [], [], [0]
    slots, positions, seqs = ([-1] * n_rows for _ in range(3))
    rows = pages = taken = 0
    for r, (l, n) in enumerate(zip(lens, new_lens)):
        sane = l >= 0 and n >= 0
        rows += n if sane else 0
        fits = sane and l + n <= len(table[r]) * bs and rows <= n_rows
        need = ceil_div(l + n, bs) - ceil_div(l, bs) if fits else 0
        pages += need
        ok = fits and (need == 0 or pages <= n_free)
        if ok:
            for j in range(need):
                table[r][ceil_div(l, bs) + j] = free[n_free - 1 - taken - j]
            taken += need
            for i in range(n):
                p = l + i
                slots[starts[r] + i] = table[r][p // bs] * bs + p % bs
                positions[starts[r] + i], seqs[starts[r] + i] = p, r
        out_lens.append(l + n if ok else l)
        admitted.append(ok)
        starts.append(rows)
    return table, out_lens, n_free - taken, admitted, starts, slots, positions, seqs


def release(done, lens, table, free, n_free, bs):
    free, out = list(free), []
    for r, (d, l) in enumerate(zip(done, lens)):
        out.append(0 if d else l)
        for j in range(min(ceil_div(max(l, 0), bs), len(table[r])) if d else 0):
            if n_free < len(free):
                free[n_free] = table[r][j]
                n_free += 1
    return free, out, n_free


def attention(q, k, v, table, lens, scale, window=0, k_scale=None, v_scale=None):
    """fp64 (out, lse, spread, reach, n): spread = sum p |v| per output, reach = the largest sum |scale q_i k_i| of a
    row's scores, n = positions attended per sequence (both for the error bounds)."""
    B, H, dh = q.shape
    nb, hkv, bs, _ = k.shape
    G = H // hkv
    out, spread = (torch.zeros(B, H, dh, dtype=torch.float64, device=q.device) for _ in range(2))
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=q.device)
    reach = torch.zeros(B, H, dtype=torch.float64, device=q.device)
    count = []
    for b in range(B):
        L = min(max(int(lens[b]), 0), table.shape[1] * bs)
        row = table[b].tolist()
        at = [p for p in range(max(0, L - window) if window else 0, L) if 0 <= row[p // bs] < nb]
        count.append(len(at))
        if not at:
            continue
        at = torch.tensor(at, device=q.device)
        page, r = table[b].long()[at // bs], at % bs
        kk, vv = (x[page, :, r].float().double() for x in (k, v))  # [n, hkv, dh]
        if k_scale is not None:
            kk, vv = kk * k_scale[page, :, r].double()[..., None], vv * v_scale[page, :, r].double()[..., None]
        for h in range(H):
            qk = q[b, h].double() * scale * kk[:, h // G]
            s = qk.sum(-1)
            p = torch.softmax(s, 0)
            out[b, h], spread[b, h] = p @ vv[:, h // G], p @ vv[:, h // G].abs()
            lse[b, h], reach[b, h] = torch.logsumexp(s, 0), qk.abs().sum(-1).max()
    return out, lse, spread, reach, torch.tensor(count, device=q.device, dtype=torch.float64)


def attention_bounds(q, page_dtype, out, lse, spread, reach, n):
    """Error bounds (out, lse) of the operator against `attention`.

    A score is a sum of head_dim products accumulated in fp32 in steps of at most 16 products: up to dh / 8 + 8
    roundings of 2^-23 (tensor-core accumulation may truncate) of sum |scale q_i k_i|, plus the two-part split of an
    fp32 query (2^-21; exact for 16-bit queries). Its weight is off by the relative size of two such errors (its own
    and the maximum's) plus 2^-20 for the exponential. The weighted sum goes over n positions in steps of 16 or more:
    n / 8 + 128 roundings of 2^-23, and the weights' own split leaves 2^-17 (two bf16 parts) or 2^-20 (two fp16
    parts). The result is rounded once to its type, half a step."""
    dh = q.shape[-1]
    score = reach * ((dh / 8 + 8) * 2.0 ** -23 + (2.0 ** -21 if q.dtype == torch.float32 else 0.0))
    sums = (n / 8 + 128) * 2.0 ** -23
    split = 2.0 ** -17 if page_dtype == torch.bfloat16 else 2.0 ** -20
    rel = 2 * score + sums[:, None] + split
    tiny = torch.finfo(torch.float16).smallest_normal * 2.0 ** -11 if q.dtype == torch.float16 else 2.0 ** -126
    return (torch.finfo(q.dtype).eps / 2 * out.abs() + 1.01 * rel[..., None] * spread + tiny,
            2 * score + sums[:, None] + 2.0 ** -20 + lse.abs() * 2.0 ** -22)


def rotate(x, rope, positions):
    """Rows [T, heads, dh] in fp32, rotated in pairs (i, i + dh / 2) at their positions."""
    half = x.shape[-1] // 2
    cs = rope[positions.long()]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    x = x.float()
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def quantise(rows):
    """fp32 rows [..., dh] -> (E4M3 codes as float8_e4m3fn, fp32 scales): amax / 448, codes of row / scale. The quotient
    by 448 is formed in fp64 and rounded once more, which gives the correctly rounded fp32 quotient (53 >= 2 * 24 + 2
    bits); torch divides an fp32 tensor by a Python number by multiplying with its reciprocal, one step off at times."""
    top = rows.abs().amax(-1)
    scale = torch.where(top == 0, torch.full_like(top, NO_SCALE), (top.double() / 448.0).float())
    return (rows / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale
