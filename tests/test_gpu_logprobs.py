"""Log probabilities, entropies and top alternatives on the GPU against fp64: types, vocabularies, ties, ruled-out tokens,
infinities and NaN, padding, strides, graphs."""
import math

import numpy as np
import pytest
import torch

import persistent_monokernel_decode_gb300 as kie
import shared_oracle as oracle
from test_gpu_paged import BF16, F16, F32, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


def check(x, tokens, top):
    got = kie.token_logprobs(x, tokens, top=top)
    compare(got, x, tokens, top)
    return got


def compare(got, x, tokens, top):
    lp, h, ids, top_lp = oracle.logprobs(x, tokens, top)
    lse, part, entropy = oracle.logprobs_bounds(x)
    assert torch.equal(got.top_ids.long(), ids)
    for a, b, tol in ((got.logprob, lp, lse + part * lp.abs()), (got.top_logprobs, top_lp, lse[:, None] + part * top_lp.abs()),
                      (got.entropy, h, entropy)):
        same = torch.isinf(b.float()) & (a == b.float())  # -inf, or what fp32 does not hold
        err = torch.where(same, 0.0, (a.double() - b).abs())
        assert torch.all(err <= torch.where(same, 1.0, tol)), float((err / tol).max())


def draw(N, V, dtype, spread=3.0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + V)
    return (torch.randn((N, V), generator=g, device="cuda") * spread).to(dtype), \
        torch.randint(-1, V + 1, (N,), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (2, 31), (5, 33), (7, 255), (4, 1000), (300, 257), (2, 4096), (5, 32000), (1, 50001),
                                 (3, 131072), (1, 262145), (700, 4097), (1300, 32001), (2, 1000003)])
def test_sizes(dtype, N, V):
    x, tokens = draw(N, V, dtype)
    for top in sorted({0, 1, min(V, 20), min(V, 32)}):
        check(x, tokens, top)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("V", [5, 40, 1000, 32000])
def test_ties_go_to_the_lowest_id(dtype, V):
    for x in (torch.zeros(4, V), torch.randint(0, 3, (4, V)).float(), torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0).expand(2, V),
              -torch.arange(V).float().expand(3, V) // 7, (torch.arange(V).float().expand(2, V) // 64)):
        check(x.to(dtype).cuda().contiguous(), ints([0] * len(x)), min(V, 32))


@pytest.mark.parametrize("V", [40, 5000, 32000])
def test_ordered_rows(V):
    """The largest logits all in one place: at the beginning, at the end, every 256th, in one run."""
    base = torch.randn(V, device="cuda")
    rows = [base.sort().values, base.sort(descending=True).values]
    for at in (torch.arange(0, V, 256, device="cuda"), torch.arange(V // 2, min(V, V // 2 + 64), device="cuda")):
        row = base.clone()
        row[at] += 20
        rows.append(row)
    check(torch.stack(rows), ints([0, 1, 2, 3]), 32)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("V", [7, 33, 2000, 32000])
def test_ruled_out_tokens(dtype, V):
    """Tokens at -inf or at the type's lowest value; rows with one token left, or none."""
    x, tokens = draw(6, V, dtype)
    x[0, ::2], x[1, 1:], x[2], x[3, V // 3:] = -math.inf, -math.inf, -math.inf, torch.finfo(dtype).min
    x[4, : V - 1] = -math.inf
    got = check(x, ints([1, 0, 0, 0, V - 1, 2]), min(V, 32))
    assert got.logprob[0] > -math.inf and got.logprob[1] == 0 and got.entropy[1] == 0
    assert got.logprob[2] == -math.inf and got.entropy[2] == 0 and torch.all(got.top_logprobs[2] == -math.inf)
    assert torch.all(check(x, ints([0, 1, 0, V // 3, 0, -1]), 0).logprob[[0, 1, 2, 4]] == -math.inf)


@pytest.mark.parametrize("dtype,spread", [(F32, 1e30), (F32, 1e-30), (BF16, 1e30), (F16, 1e4), (F32, 100.0), (F32, 3e38)])
def test_logits_of_any_size(dtype, spread):
    x, tokens = draw(5, 3000, dtype, 1.0)
    x = (x.float().clamp(-1, 1) * spread).to(dtype)
    x[1] = x[1] + x[1].abs().max()
    x[2, 5] = 0
    check(x.clamp(torch.finfo(dtype).min, torch.finfo(dtype).max), tokens, 9)


def test_nan_and_infinity_stay_in_their_rows():
    x, _ = draw(5, 3000, F32)
    tokens = ints([1, 2, 3, 4, -1])
    x[1, 77], x[2, 5], x[2, 9], x[4, 100] = math.nan, math.inf, math.inf, math.nan
    got = kie.token_logprobs(x, tokens, top=3)
    for r in (1, 2, 4):
        assert torch.isnan(got.entropy[r]) and torch.isnan(got.top_logprobs[r]).all()
    assert torch.isnan(got.logprob[1:3]).all() and got.logprob[4] == 0
    assert got.top_ids[1, 0] == 77 and got.top_ids[2, :2].tolist() == [5, 9] and got.top_ids[4, 0] == 100
    keep = torch.tensor([0, 3], device="cuda")
    compare(kie.TokenLogprobs(*(y[keep] for y in got)), x[keep], tokens[keep], 3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_and_unaligned_rows(dtype):
    """Rows of a wider tensor, starting off a 16-byte boundary, with NaN between them."""
    for V, extra, at in ((1000, 3, 1), (4096, 8, 0), (32000, 5, 3), (33, 100, 50), (9000, 1, 1)):
        wide = torch.full((6, V + extra), math.nan, device="cuda", dtype=dtype)
        x, tokens = draw(6, V, dtype)
        wide[:, at:at + V] = x
        got, want = kie.token_logprobs(wide[:, at:at + V], tokens, top=20), check(x, tokens, 20)
        assert torch.equal(got.top_ids, want.top_ids)
        compare(got, x, tokens, 20)


def test_past_32_bit_offsets():
    x = torch.zeros((3, 1 << 30), device="cuda", dtype=F16)[:, :50000]
    x.copy_(draw(3, 50000, F16)[0])
    got = kie.token_logprobs(x, ints([1, 2, 3]), top=5)
    compare(got, x.contiguous(), ints([1, 2, 3]), 5)


def test_nothing_and_the_same_bits_again():
    x, tokens = draw(9, 32000, BF16)
    assert kie.token_logprobs(x[:0], tokens[:0], top=4).top_ids.shape == (0, 4)
    first = kie.token_logprobs(x, tokens, top=32)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, kie.token_logprobs(x, tokens, top=32)))


def test_a_replayed_graph_follows_its_inputs():
    x, tokens = draw(4, 32000, F32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kie.token_logprobs(x, tokens, top=8)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = kie.token_logprobs(x, tokens, top=8)
    for seed in (1, 2):
        y, t = draw(4, 32000, F32, seed=seed)
        x.copy_(y), tokens.copy_(t)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        compare(got, x, tokens, 8)


def test_the_binding_refuses():
    x, tokens = torch.zeros(3, 50, device="cuda"), ints([0, 1, 2])
    for bad in ((x.double(), tokens, 1), (x.T, tokens, 1), (x[0], tokens, 1), (x, tokens.long(), 1), (x, tokens[:2], 1),
                (x, tokens, 33), (x, tokens, -1), (x[:, :4], tokens, 5), (x.cpu(), tokens, 1), (x, tokens.cpu(), 1)):
        with pytest.raises(ValueError):
            kie.token_logprobs(bad[0], bad[1], top=bad[2])
    with pytest.raises(kie.KieError):
        kie.token_logprobs(x[:1].expand(3, 50), tokens)  # rows that lie over one another
