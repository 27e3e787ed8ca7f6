"""Attention of rows that share a prefix at its limits: scales and queries next to nothing, pages whose heads are one, what lies
beside an output, steps on E4M3 pages."""
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


@pytest.mark.parametrize("cache,qt", [(F16, F32), (E4M3, F32), (E4M3, BF16), (E4M3, F16), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-20, 1e-38])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-44, -1e-38, 1e-30, -1e-6])
def test_scores_of_next_to_nothing(cache, qt, size, scale):
    """Every position weighs the same; rows that end before their prefix does have masked ones among them."""
    q, *rest = grouped([(150, [160, 170, 130, 1]), (64, [64, 63])], [20, 0], 8, 4, 128, 16, cache, qt, seed=4)
    check((q.float() * size).to(qt), *rest, scale=scale)


@pytest.mark.parametrize("cache,qt", [(F16, F16), (F16, F32), (BF16, BF16), (E4M3, BF16)])
@pytest.mark.parametrize("dh,bs", [(128, 16), (64, 64)])
def test_pages_whose_heads_are_one_give_what_their_copies_give(cache, qt, dh, bs):
    """Expanded heads, with a stride of 0: the results of contiguous pages, or (where CUDA makes no tensor map of them) the
    refusal that says so, and nothing else."""
    q, k, v, table, lens, start, prefix, ks, vs = grouped([(150, [160, 170, 150])], [20], 8, 4, dh, bs, cache, qt, seed=4, poison=False)
    one = [x[:, :1].expand(-1, 4, *[-1] * (x.dim() - 2)) for x in (k, v)]
    scales = {} if ks is None else dict(zip(("k_scale", "v_scale"), [x[:, :1].expand(-1, 4, -1) for x in (ks, vs)]))
    assert one[0].stride(1) == 0
    copies = {name: x.contiguous() for name, x in scales.items()}
    want = kie.paged_prefix_attention(q, *[x.contiguous() for x in one], table, lens, start, prefix, return_lse=True, **copies)
    try:
        got = kie.paged_prefix_attention(q, *one, table, lens, start, prefix, return_lse=True, **scales)
    except kie.KieError as e:
        assert "no tensor map can be made of the pages' strides" in str(e)
        pytest.skip("this driver makes no tensor map with a stride of 0")
    assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("qt", [F16, F32])
def test_what_lies_beside_an_output_stays(qt):
    """In place of strided queries, and into some heads of a wider tensor."""
    q, k, v, table, lens, start, prefix, ks, vs = grouped([(70, [80, 71, 100])], [5], 4, 2, 64, 16, F16, qt)
    wide = torch.randn(4, 6 * 64 + 1, device="cuda").to(qt)
    inner = wide[:, 1:1 + 4 * 64].unflatten(1, (4, 64))
    inner.copy_(q)
    before = wide.clone()
    want = kie.paged_prefix_attention(q, k, v, table, lens, start, prefix)
    assert kie.paged_prefix_attention(inner, k, v, table, lens, start, prefix, out=inner) is inner
    assert torch.equal(inner, want) and not torch.equal(inner, q)
    assert torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, 1 + 4 * 64:], before[:, 1 + 4 * 64:])
    heads = before[:, :6 * 64].clone().unflatten(1, (6, 64))
    kept = heads.clone()
    kie.paged_prefix_attention(q, k, v, table, lens, start, prefix, out=heads[:, 1:5])
    assert torch.equal(heads[:, 1:5], want) and torch.equal(heads[:, [0, 5]], kept[:, [0, 5]])


@pytest.mark.parametrize("cache,qt", [(E4M3, F32), (E4M3, BF16), (BF16, BF16)])
def test_steps_behind_one_another_on_other_pages(cache, qt):
    """Steps on a stream without a wait, whose scales and rows lie beside those that the step before has read, give the bits
    of the same steps with a wait after each call."""
    def run(wait):
        pages = kie.PagedCache(TINY, n_blocks=48 * 24, block_size=32, max_seqs=48, max_blocks=24, dtype=cache, shared=True)
        g = torch.Generator(device="cuda")
        g.manual_seed(6)
        ks, vs = [(torch.randn((41, 300, TINY.n_kv_heads, TINY.head_dim), generator=g, device="cuda") * 3).to(qt) for _ in range(2)]
        q = torch.randn((48, TINY.n_heads, TINY.head_dim), generator=g, device="cuda").to(qt)
        first = torch.zeros(48, dtype=torch.int32, device="cuda")
        first[0] = 300
        step = pages.extend(first, 300)
        pages.append(0, ks[40], vs[40], step)
        assert pages.fork(torch.zeros(48, dtype=torch.int32, device="cuda")).ok.all()
        groups, one, outs = (ints([0, 48]), ints([300])), torch.ones_like(first), []
        for i in range(40):
            step = pages.extend(one, 48)
            pages.append(0, ks[i, :48], vs[i, :48], step)
            if wait:
                torch.cuda.synchronize()
            outs.append(pages.attention(0, q, step, groups=groups))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs
    for a, b in zip(run(False), run(True)):
        assert torch.equal(bits(a), bits(b)) and not torch.isnan(a).any()
