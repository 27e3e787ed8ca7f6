"""Attention of rows that share a prefix when a wait inside runs out (a block that stops loading, and a short limit): the
results that the block had in hand and had still to do are NaN, all others are as ever, and so is the next call."""
import pytest
import torch

import persistent_monokernel_decode_gb300 as kie
from test_gpu_paged import BF16, E4M3, F16, F32, bits
from test_gpu_prefix import grouped

pytestmark = pytest.mark.gpu

TILE, UNIT, ITEM_COST, MIN_RUN = 128, 64, 2, 2  # kie_paged.cuh, kie_prefix_attn.cu


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    kie.paged_set_timeout_ns(20_000_000)
    yield
    kie.paged_set_timeout_ns(2_000_000_000)


def runs(groups, hq, hkv, lens, blocks):
    """For each block, what it has part in, in order: (first row, end, KV head, units with positions)."""
    members, items, at, row = 2 * (TILE // (hq // hkv)), [], 0, 0
    for prefix, ls in groups:
        units = -(-prefix // UNIT)
        reach = max([min(l, prefix) for l in ls], default=0)
        for t in range(0, len(ls) if units else 0, members):
            for h in range(hkv):
                items.append((at, units, reach, row + t, row + min(t + members, len(ls)), h))
                at += units + ITEM_COST
        row += len(ls)
    per = max(-(-at // blocks), MIN_RUN)
    out = []
    for b in range(blocks):
        mine = []
        for place, units, reach, r0, r1, h in items:
            u0, u1 = max(0, b * per - place - ITEM_COST), min(units, (b + 1) * per - place - ITEM_COST)
            if u1 > u0:
                mine.append((r0, r1, h, max(0, min(u1, -(-reach // UNIT)) - u0)))
        out.append(mine)
    return out


SMALL = [(200 + 30 * (i % 7), [200 + 30 * (i % 7) + i % 4] * (1 + i % 3)) for i in range(400)]  # blocks of several items
LONG = [(6000, [6000, 6010, 5900] * 10), (3000, [3001] * 9)]  # items of several blocks


@pytest.mark.parametrize("cache,qt", [(F16, F16), (F16, F32), (BF16, BF16), (E4M3, F32), (E4M3, F16)])
@pytest.mark.parametrize("groups,hq,hkv,dh", [(SMALL, 8, 2, 64), (LONG, 20, 4, 128)])
def test_a_block_that_loads_no_more(cache, qt, groups, hq, hkv, dh):
    q, k, v, table, lens, start, prefix, ks, vs = grouped(groups, [50], hq, hkv, dh, 64, cache, qt, seed=1, poison=False)
    def call():
        return kie.paged_prefix_attention(q, k, v, table, lens, start, prefix, k_scale=ks, v_scale=vs, return_lse=True)
    want, want_lse = call()
    assert not torch.isnan(want).any()
    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    work = runs(groups, hq, hkv, lens.tolist(), blocks)
    busy = [b for b in range(blocks) if work[b]]
    group = hq // hkv
    for block, half in ((busy[0], 0), (busy[len(busy) // 2], 1), (busy[-1], 2), (busy[3], 5), (busy[7], 12), (busy[5], 7)):
        left, gone = half, torch.zeros(want.shape[:2], dtype=torch.bool, device="cuda")
        for r0, r1, h, units in work[block]:
            left -= 2 * units
            if left < 0:
                for r in range(r0, r1):
                    if min(int(lens[r]), int(prefix[int((start <= r).sum()) - 1])) > 0:
                        gone[r, h * group:(h + 1) * group] = True
        assert kie.lib().kie_paged_debug_stop_loads(block, half) == kie.KIE_OK
        out, lse = call()
        torch.cuda.synchronize()
        assert torch.equal(torch.isnan(out), gone[:, :, None].expand_as(out)) and torch.equal(torch.isnan(lse), gone)
        assert torch.equal(bits(out)[~gone], bits(want)[~gone]) and torch.equal(lse[~gone], want_lse[~gone])
        out, lse = call()
        assert torch.equal(bits(out), bits(want)) and torch.equal(lse, want_lse)
    assert any(len(w) > 1 for w in work) or any(w[0][3] > 1 for w in work if w)


def test_a_captured_call_keeps_what_it_was_given():
    q, k, v, table, lens, start, prefix, _, _ = grouped([(300, [310] * 9)], [], 8, 2, 64, 16, F16, F16, poison=False)
    want = kie.paged_prefix_attention(q, k, v, table, lens, start, prefix)
    # two items of 5 units and 2 places more for 152 blocks: runs of 2 places, of which the first has no unit
    work = runs([(300, [310] * 9)], 8, 2, [310] * 9, torch.cuda.get_device_properties(0).multi_processor_count)
    block = [b for b, w in enumerate(work) if w][0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        assert kie.lib().kie_paged_debug_stop_loads(block, 0) == kie.KIE_OK
        with torch.cuda.graph(g, stream=s):
            out = kie.paged_prefix_attention(q, k, v, table, lens, start, prefix)
    again = kie.paged_prefix_attention(q, k, v, table, lens, start, prefix)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.isnan(out).any() and torch.equal(again, want)


def test_the_hook_is_taken_back():
    q, k, v, table, lens, start, prefix, _, _ = grouped([(300, [310] * 9)], [], 8, 2, 64, 16, F16, F16, poison=False)
    for block in (1, -1):
        assert kie.lib().kie_paged_debug_stop_loads(block, 0) == kie.KIE_OK
    assert not torch.isnan(kie.paged_prefix_attention(q, k, v, table, lens, start, prefix)).any()
