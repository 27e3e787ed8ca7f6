"""Attention of rows that share a prefix on the GPU against fp64: types, head layouts, prefixes and tails of every edge
length, rows shorter than their prefix, odd groups, steps, strides, poisoned and bad pages, graphs, streams."""
import numpy as np
import pytest
import torch

import paged_oracle
import persistent_monokernel_decode_gb300 as kie
import shared_oracle as oracle
from test_gpu_paged import BF16, E4M3, F16, F32, HEADS, TYPES, batch, bits, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


def grouped(groups, alone, hq, hkv, dh, bs, cache, qt, seed=0, poison=True, **kw):
    """Sequences in groups [(prefix, lengths)], then `alone` ones. A group's full prefix pages are shared by its rows that
    reach them; whatever else its rows hold of positions in the prefix is NaN, but for the longest row's."""
    lens = [l for _, ls in groups for l in ls] + alone
    q, k, v, table, L, ks, vs = batch(lens, hq, hkv, dh, bs, cache, qt, seed=seed, **kw)
    start, row = [0], 0
    for prefix, ls in groups:
        reach = [min(l, prefix) for l in ls] or [0]
        source = row + reach.index(max(reach))
        for r in range(row, row + len(ls)):
            if r != source and poison:
                for p in range(0, min(lens[r], prefix), bs):
                    page, n = int(table[r, p // bs]), min(bs, prefix - p, lens[r] - p)
                    k[page, :, :n], v[page, :, :n] = float("nan"), float("nan")
            for j in range(min(lens[r], max(reach)) // bs):
                if (j + 1) * bs <= prefix:
                    table[r, j] = table[source, j]
        row += len(ls)
        start.append(row)
    return q, k, v, table, L, ints(start), ints([p for p, _ in groups]), ks, vs


def check(q, k, v, table, lens, start, prefix, ks, vs, scale=None, nan_rows=(), **kw):
    out, lse = kie.paged_prefix_attention(q, k, v, table, lens, start, prefix, scale=scale, k_scale=ks, v_scale=vs,
                                          return_lse=True, **kw)
    compare(out, lse, q, k, v, table, lens, start, prefix, ks, vs, scale, nan_rows)
    return out, lse


def compare(out, lse, q, k, v, table, lens, start, prefix, ks, vs, scale=None, nan_rows=()):
    ref = oracle.prefix_attention(q, k, v, table, lens.tolist(), start.tolist(), prefix.tolist(),
                                  q.shape[-1] ** -0.5 if scale is None else scale, ks, vs)
    tol_out, tol_lse = paged_oracle.attention_bounds(q, k.dtype, *ref)
    good = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    for r in nan_rows:
        good[r] = False
    assert not torch.isnan(out[good]).any()
    err = (out.double() - ref[0]).abs()[good]
    assert torch.all(err <= tol_out[good]), float((err / tol_out[good]).max())
    empty = ref[4] == 0
    assert torch.all(out[empty] == 0) and torch.all(lse[empty] == -torch.inf)
    good &= ~empty
    err = (lse.double() - ref[1]).abs()[good]
    assert torch.all(err <= tol_lse[good]), float((err / tol_lse[good]).max())


EDGES = [(1, [1, 2]), (15, [16, 15, 40]), (16, [17, 16]), (17, [20, 33, 64]), (0, [5, 0]), (127, [128, 300]), (128, [130] * 5),
         (129, [129, 140]), (200, [300, 7, 0, 250]), (256, [257] * 3), (500, [3, 100, 499]), (1000, [1001, 1100, 1000])]


@pytest.mark.parametrize("cache,qt", TYPES)
@pytest.mark.parametrize("hq,hkv,dh", HEADS)
@pytest.mark.parametrize("bs", [16, 48])
def test_edges(cache, qt, hq, hkv, dh, bs):
    check(*grouped(EDGES, [0, 1, 77], hq, hkv, dh, bs, cache, qt, seed=hq + dh))


@pytest.mark.parametrize("cache,qt", TYPES)
@pytest.mark.parametrize("hq,hkv,dh", [(20, 4, 128), (8, 1, 64), (7, 7, 128), (3, 1, 64)])
def test_a_large_group(cache, qt, hq, hkv, dh):
    """More rows than a tile of any layout holds, and tails from none to longer than the prefix."""
    lens = [700 + i * i // 8 for i in range(90)]
    check(*grouped([(700, lens)], [], hq, hkv, dh, 64, cache, qt, seed=3))


@pytest.mark.parametrize("cache,qt", TYPES)
def test_a_long_prefix(cache, qt):
    check(*grouped([(9001, [9002, 9100, 9001])], [40], 20, 4, 128, 16, cache, qt, seed=4, poison=False))


@pytest.mark.parametrize("cache,qt", [(F16, F16), (E4M3, F32)])
def test_many_small_groups(cache, qt):
    rng = np.random.RandomState(5)
    groups = [(p, (p + rng.randint(0, 30, rng.randint(0, 4))).tolist()) for p in rng.randint(0, 90, 400).tolist()]
    check(*grouped(groups, [3, 0, 9], 4, 2, 64, 16, cache, qt, seed=6))


def test_random_batches():
    rng = np.random.RandomState(7)
    for i in range(20):
        groups = []
        for _ in range(rng.randint(1, 8)):
            p = int(np.exp(rng.uniform(0, np.log(1500))))
            groups.append((p, (p + np.exp(rng.uniform(0, np.log(300), rng.randint(1, 30))).astype(int) - 1).tolist()))
        hq, hkv, dh = HEADS[i % len(HEADS)]
        cache, qt = TYPES[i % len(TYPES)]
        check(*grouped(groups, rng.randint(0, 50, rng.randint(0, 5)).tolist(), hq, hkv, dh, int(rng.choice([16, 32, 80, 128])),
                       cache, qt, seed=i))


@pytest.mark.parametrize("cache,qt", TYPES)
def test_large_scores(cache, qt):
    """Scores of a few hundred, so that a few positions, in the prefix or behind it, take all the weight."""
    q, k, *rest = grouped([(300, [340, 301, 500]), (40, [50])], [60], 4, 2, 64, 16, cache, qt, spread=8.0)
    check(q, k, *rest, scale=1.0)


@pytest.mark.parametrize("cache", [F16, E4M3])
def test_rising_scores(cache):
    """Scores that rise along the prefix by 200 nats, so that the softmax's reference moves again and again."""
    q, k, v, table, L, start, prefix, ks, vs = grouped([(800, [810, 805])], [], 4, 2, 64, 16, cache, F16, poison=False)
    ramp = torch.zeros(k.shape[0], k.shape[2], device="cuda")
    for j in range(50):
        ramp[table[0, j].long()] = (torch.arange(16, device="cuda") + 16 * j) / 4.0
    q[:] = 0.0
    q[..., 0] = 1.0
    if cache == F16:
        k[..., 0] = ramp[:, None].to(F16)
    else:
        k.view(torch.uint8)[..., 0] = torch.full_like(ramp, 1.0).to(E4M3).view(torch.uint8)[:, None]
        k.view(torch.uint8)[..., 1:] = 0
        ks[:] = ramp[:, None]
    check(q, k, v, table, L, start, prefix, ks, vs, scale=1.0)


def test_scales_far_apart():
    """E4M3 rows of very different size, and rows of zeros, whose plain scores lie far above the rest."""
    q, k, v, table, lens, start, prefix, ks, vs = grouped([(300, [340, 320]), (40, [90])], [], 8, 2, 128, 16, E4M3, F32,
                                                          poison=False, dead=0.0)
    vs *= 1e-6
    check(q, k, v, table, lens, start, prefix, ks, vs)
    vs[:, :, ::2] *= 1e6
    check(q, k, v, table, lens, start, prefix, ks, vs)
    vs[:, :, ::3] = 2.0 ** -126
    v.view(torch.uint8)[:, :, ::3] = 0
    check(q, k, v, table, lens, start, prefix, ks, vs)


def test_scores_of_zero_rows_far_above():
    """The rows of zeros (scale 2^-126) have scores 100 nats above the others: they take the weight, the output is 0."""
    q, k, v, table, lens, start, prefix, ks, vs = grouped([(200, [210])], [], 4, 2, 64, 16, E4M3, F16, poison=False, dead=0.0)
    q[:], k.view(torch.uint8)[:] = 1.0, torch.tensor(1.0).to(E4M3).view(torch.uint8).item()
    ks[:] = 0.0
    ks[:, :, 5] = 100.0 / 64
    vs[:, :, 5] = 2.0 ** -126
    v.view(torch.uint8)[:, :, 5] = 0
    check(q, k, v, table, lens, start, prefix, ks, vs, scale=1.0)


@pytest.mark.parametrize("factor", [1e-6, 3e5])
def test_queries_of_any_size(factor):
    q, *rest = grouped([(130, [140, 131]), (40, [47])], [], 8, 2, 128, 16, F16, F32)
    check(q * factor, *rest, scale=0.1 / factor)
    q, *rest = grouped([(130, [140, 131]), (40, [47])], [], 8, 2, 128, 16, E4M3, BF16)
    check((q.float() * factor).to(BF16), *rest, scale=0.03 / factor)


@pytest.mark.parametrize("cache,qt", [(F16, F32), (BF16, BF16), (E4M3, F16)])
@pytest.mark.parametrize("order", ["position", "pool"])
def test_page_orders(cache, qt, order):
    check(*grouped([(100, [120, 101]), (33, [40])], [7], 8, 2, 128, 32, cache, qt, order=order))


def test_groups_out_of_range():
    """Starts that fall, lie outside the rows or overlap; negative and huge prefixes; no groups at all."""
    q, k, v, table, lens, _, _, ks, vs = grouped([(64, [100, 90, 80, 70, 65])], [30], 4, 2, 64, 16, F16, F16, poison=False)
    for start, prefix in (([0, 9, 4, 6], [48, 64, 16]), ([-5, 2, 99], [33, 64]), ([3, 1, 5], [64, 16]), ([7, 8], [64]),
                          ([2, 2, 2, 5], [64, 64, 64]), ([0, 5], [2 ** 31 - 1]), ([0, 2, 5], [-3, 64]), ([0, 6], [-2 ** 31])):
        check(q, k, v, table, lens, ints(start), ints(prefix), ks, vs)
    want = kie.paged_attention(q, k, v, table, lens, return_lse=True)
    got = kie.paged_prefix_attention(q, k, v, table, lens, ints([0]), ints([]), return_lse=True)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("cache", [F16, E4M3])
def test_bad_pages_are_left_out(cache):
    q, k, v, table, lens, start, prefix, ks, vs = grouped([(96, [110, 100])], [40], 4, 2, 64, 16, cache, F16)
    table[0, 1], table[0, 3] = -7, 2 ** 30
    check(q, k, v, table, lens, start, prefix, ks, vs)
    table[0, :6] = -1  # nothing of the prefix is left
    check(q, k, v, table, lens, start, prefix, ks, vs)


def test_nan_and_infinity_stay_with_their_group():
    q, k, v, table, lens, start, prefix, ks, vs = grouped([(64, [80, 70]), (64, [90, 66]), (50, [60])], [40], 4, 2, 64, 16, F16,
                                                          F32, poison=False)
    page = table[0, 2].long()
    k[page, :, 3], v[page, :, 5] = float("nan"), float("inf")
    out, lse = check(q, k, v, table, lens, start, prefix, ks, vs, nan_rows=(0, 1))
    assert torch.isnan(out[:2]).any(-1).all()


def test_an_infinity_in_keys_counts_as_a_score():
    """K of -inf against queries of one sign: scores of -inf, weight 0; a head whose every score is -inf is empty."""
    for cache, qt in ((F16, F16), (F16, F32), (BF16, BF16)):
        q, k, v, table, lens, start, prefix, ks, vs = grouped([(64, [64, 64])], [], 2, 2, 64, 16, cache, qt, poison=False)
        q = q.abs() + 0.1
        k[table[0, 1].long(), :, 3, 7] = -torch.inf
        check(q, k, v, table, lens, start, prefix, ks, vs)
        k[table[0, :4].long(), 0, :, 7] = -torch.inf
        out, lse = kie.paged_prefix_attention(q, k, v, table, lens, start, prefix, return_lse=True)
        assert torch.all(out[:, 0] == 0) and torch.all(lse[:, 0] == -torch.inf)
        assert torch.isfinite(lse[:, 1]).all() and torch.isfinite(out).all()


@pytest.mark.parametrize("cache,qt", [(F16, F16), (E4M3, F32), (BF16, BF16)])
def test_steps(cache, qt):
    """Rows of a step: sequences that idle, bring several tokens or were not admitted, padding, a group whose first row is
    none, and rows whose own sequence is out of range."""
    _, k, v, table, lens, _, _, ks, vs = grouped([(64, [100, 90, 80]), (40, [60, 55])], [30], 8, 2, 64, 16, cache, qt, poison=False)
    table[1:3, :4] = table[0, :4]
    table[4, :2] = table[3, :2]
    seqs = [-1, 0, 0, 0, 2, 99, 1, 4, 3, 5, -1, 5]
    positions = [-1, 97, 98, 99, 79, 12, 20, 54, 59, 29, -1, 3]
    q = torch.randn(len(seqs), 8, 64, device="cuda").to(qt)
    out, lse = kie.paged_prefix_attention(q, k, v, table, None, ints([0, 7, 9]), ints([64, 40]), seqs=ints(seqs),
                                          positions=ints(positions), k_scale=ks, v_scale=vs, return_lse=True)
    row_table = table[torch.tensor([s if 0 <= s < 6 else 0 for s in seqs])].contiguous()
    row_lens = ints([p + 1 if 0 <= s < 6 else 0 for s, p in zip(seqs, positions)])
    compare(out, lse, q, k, v, row_table, row_lens, ints([0, 7, 9]), ints([64, 40]), ks, vs)


@pytest.mark.parametrize("cache,qt", [(F16, F32), (E4M3, BF16), (BF16, BF16)])
@pytest.mark.parametrize("cached,rows", [(0, 5), (37, 130), (640, 64), (1000, 1)])
def test_a_part_of_a_prompt(cache, qt, cached, rows):
    """Rows of one sequence, each attending up to itself: what was cached before is the group's prefix."""
    _, k, v, table, lens, _, _, ks, vs = grouped([], [cached + rows], 20, 4, 128, 16, cache, qt)
    q = torch.randn(rows, 20, 128, device="cuda").to(qt)
    seqs, positions = ints([0] * rows), ints(list(range(cached, cached + rows)))
    groups = ints([0, rows]), ints([cached])
    out, lse = kie.paged_prefix_attention(q, k, v, table, None, *groups, seqs=seqs, positions=positions, k_scale=ks, v_scale=vs,
                                          return_lse=True)
    compare(out, lse, q, k, v, table.expand(rows, -1).contiguous(), positions + 1, *groups, ks, vs)


@pytest.mark.parametrize("qt", [F16, F32])
def test_strided_query_and_output_and_in_place(qt):
    q, *rest = grouped([(70, [80, 71, 100])], [5], 4, 2, 64, 16, F16, qt)
    wide = torch.randn(4, 6 * 64 + 1, device="cuda").to(qt)
    strided = wide[:, 1:1 + 4 * 64].unflatten(1, (4, 64))
    strided.copy_(q)
    want, _ = check(q, *rest)
    out = torch.full((4, 6, 64), 7.0, device="cuda", dtype=qt)
    k, v, table, lens, start, prefix, ks, vs = rest
    got = kie.paged_prefix_attention(strided, k, v, table, lens, start, prefix, out=out[:, 1:5])
    assert torch.equal(got, want) and torch.all(out[:, 0] == 7) and torch.all(out[:, 5] == 7)
    assert kie.paged_prefix_attention(strided, k, v, table, lens, start, prefix, out=strided) is strided
    assert torch.equal(strided, want) and torch.equal(wide[:, 0], wide[:, 0])


def test_nothing():
    q, k, v, table, lens, *_ = grouped([], [3], 4, 2, 64, 16, F16, F16)
    assert kie.paged_prefix_attention(q[:0], k, v, table[:0], lens[:0], ints([0, 0]), ints([5])).shape == (0, 4, 64)


def test_past_32_bit_offsets():
    """A cache of more than 2^31 elements, the prefix at its end."""
    n, bs = 140000, 64
    k = torch.zeros((n, 2, bs, 128), dtype=F16, device="cuda")
    v = torch.zeros_like(k)
    k[-4:], v[-4:] = torch.randn_like(k[-4:]), torch.randn_like(v[-4:])
    k[:2], v[:2] = torch.randn_like(k[:2]), torch.randn_like(v[:2])
    table = ints([[n - 1, n - 3, 0], [n - 1, n - 3, n - 2]])
    q = torch.randn(2, 4, 128, device="cuda", dtype=F16)
    lens = ints([130, 190])
    out, lse = kie.paged_prefix_attention(q, k, v, table, lens, ints([0, 2]), ints([128]), return_lse=True)
    small = torch.cat([k[:2], k[-4:]]), torch.cat([v[:2], v[-4:]])
    compare(out, lse, q, *small, ints([[5, 3, 0], [5, 3, 4]]), lens, ints([0, 2]), ints([128]), None, None)


def test_the_same_bits_again_and_any_workspace():
    """The same call gives the same bits, whatever memory its workspace gets."""
    args = grouped([(700, [750] * 30), (90, [100, 95])], [40], 8, 2, 128, 16, F16, F16, poison=False)
    q, k, v, table, lens, start, prefix, _, _ = args
    first = kie.paged_prefix_attention(q, k, v, table, lens, start, prefix, return_lse=True)
    for fill in (0xFF, 0x7F, 0x00):
        junk = torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")
        del junk  # the allocator hands this out again
        again = kie.paged_prefix_attention(q, k, v, table, lens, start, prefix, return_lse=True)
        assert torch.equal(bits(first[0]), bits(again[0])) and torch.equal(first[1], again[1])


def test_a_replayed_graph_follows_its_inputs_and_two_streams_share_nothing():
    sets = [grouped([(300, [400] * 9), (50, [60, 51])], [20], 8, 2, 64, 16, F16, F16, seed=s, poison=False) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in sets]
    graphs, outs = [], []
    for (q, k, v, table, lens, start, prefix, _, _), s in zip(sets, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            kie.paged_prefix_attention(q, k, v, table, lens, start, prefix)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(kie.paged_prefix_attention(q, k, v, table, lens, start, prefix, return_lse=True))
            graphs.append(g)
    torch.cuda.synchronize()
    for new_lens, new_prefix in (([400] * 9 + [60, 51, 20], [300, 50]), ([310] * 9 + [51, 50, 3], [128, 7]), ([0] * 12, [300, 50]),
                                 ([301] * 9 + [55, 51, 1], [0, 49])):
        for s in sets:
            s[4].copy_(ints(new_lens))
            s[6].copy_(ints(new_prefix))
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for (q, k, v, table, lens, start, prefix, ks, vs), (out, lse) in zip(sets, outs):
            compare(out, lse, q, k, v, table, lens, start, prefix, ks, vs)


def test_the_binding_refuses():
    q, k, v, table, lens, start, prefix, _, _ = grouped([(20, [30, 25])], [], 4, 2, 64, 16, F16, F16)
    for bad in ((start.long(), prefix), (start[:1], prefix), (start.cpu(), prefix), (start, prefix.float()), (start, [20])):
        with pytest.raises(ValueError):
            kie.paged_prefix_attention(q, k, v, table, lens, *bad)
    with pytest.raises(ValueError):
        kie.paged_prefix_attention(q.cpu(), k, v, table, lens, start, prefix)
    with pytest.raises(kie.KieError):
        kie.paged_prefix_attention(q, k, v, table, lens, ints([0] * 5000), ints([0] * 4999))
