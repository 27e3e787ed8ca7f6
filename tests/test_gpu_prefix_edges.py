"""Attention of rows that share a prefix at its limits: prefixes of nothing, as many groups as there may be, expanded pages,
and steps behind one another on a stream without a wait between them."""
import pytest
import torch

import persistent_monokernel_decode_gb300 as kie
from synth.configs import TINY
from test_gpu_paged import BF16, E4M3, F16, F32, bits, ints
from test_gpu_prefix import check, grouped

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


@pytest.mark.parametrize("cache,qt", [(F16, F32), (BF16, BF16), (E4M3, F16)])
def test_prefixes_of_nothing(cache, qt):
    check(*grouped([(0, [40, 0, 1]), (0, []), (0, [300] * 9)], [5], 8, 2, 64, 16, cache, qt, seed=1))


def test_rows_of_nothing_under_a_prefix():
    check(*grouped([(200, [0, 0, 0]), (64, [0]), (100, [])], [0, 0], 8, 2, 64, 16, F16, F16, seed=2))


def test_as_many_groups_as_there_may_be():
    groups = [(16 * (i % 3), [16 * (i % 3) + i % 5] * (i % 2 + 1)) for i in range(4096)]
    q, k, v, table, lens, start, prefix, ks, vs = grouped(groups, [7], 4, 4, 64, 16, F16, F16, seed=3)
    check(q, k, v, table, lens, start, prefix, ks, vs)
    with pytest.raises((ValueError, kie.KieError)):
        kie.paged_prefix_attention(q, k, v, table, lens, torch.cat([start, start[-1:]]), torch.cat([prefix, prefix[:1]]))


@pytest.mark.parametrize("cache,qt", [(F16, F16), (BF16, BF16)])
def test_pages_whose_heads_are_one(cache, qt):
    q, k, v, table, lens, start, prefix, _, _ = grouped([(150, [160, 170, 150])], [20], 8, 4, 128, 16, cache, qt, seed=4, poison=False)
    k, v = k[:, :1], v[:, :1]
    whole = [x.expand(-1, 4, -1, -1) for x in (k, v)]
    assert whole[0].stride(1) == 0
    try:
        got = kie.paged_prefix_attention(q, *whole, table, lens, start, prefix, return_lse=True)
    except (ValueError, kie.KieError):
        return  # CUDA may refuse a map with a stride of 0
    want = kie.paged_prefix_attention(q, *[x.contiguous() for x in whole], table, lens, start, prefix, return_lse=True)
    assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(got[1], want[1])


def test_steps_behind_one_another():
    """Append, attend, append, attend .. without a wait in between gives the bits of the same with a wait after each call:
    no launch reads pages that an earlier one has still to write, or writes those that one still reads."""
    def run(wait):
        cache = kie.PagedCache(TINY, n_blocks=40 * 24, block_size=16, max_seqs=40, max_blocks=24, shared=True)
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        ks, vs = [torch.randn((26, 300, TINY.n_kv_heads, TINY.head_dim), generator=g, device="cuda").half() for _ in range(2)]
        q = torch.randn((40, TINY.n_heads, TINY.head_dim), generator=g, device="cuda").half()
        outs = []
        first = torch.zeros(40, dtype=torch.int32, device="cuda")
        first[0] = 300
        step = cache.extend(first, 300)
        cache.append(0, ks[25], vs[25], step)
        assert cache.fork(torch.zeros(40, dtype=torch.int32, device="cuda")).ok.all()
        groups = ints([0, 40]), ints([300])
        one = torch.ones_like(first)
        for i in range(25):
            step = cache.extend(one, 40)
            cache.append(0, ks[i, :40], vs[i, :40], step)
            if wait:
                torch.cuda.synchronize()
            outs.append(cache.attention(0, q, step, groups=groups))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs
    for a, b in zip(run(False), run(True)):
        assert torch.equal(bits(a), bits(b))
