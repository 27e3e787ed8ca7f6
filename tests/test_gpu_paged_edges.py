"""Paged-cache operators on the GPU where values, rows and arguments are at their limits: E4M3 scales that underflow,
V rows of vanishing and infinite scale, infinite K rows, steps in which not every sequence has a row, and prompts that
do not fit the step they are loaded by."""
import math

import numpy as np
import pytest
import torch

import paged_oracle as oracle
import persistent_monokernel_decode_gb300 as kie
from test_gpu_paged import BF16, E4M3, F16, F32, batch, bits, gen, ints, page_tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


# ---- append --------------------------------------------------------------------------------------------------

def test_append_of_tiny_rows_into_e4m3():
    """fp32 rows with maxima from 2^-149 to 2^-110 that also hold zeros. The scale is max|x| / 448 rounded to fp32, 2^-126
    where that is 0, and no code is NaN. A value is off by half a step of its code (2^-4 of it, or 2^-10 scales), and
    by what the rounding of the scale, 2^-150 at most, can cut from it: 448 * 2^-150."""
    n, dh = 40, 64
    rows = torch.rand((n, 2, dh), generator=torch.Generator().manual_seed(1), dtype=torch.float64) * 2 - 1
    rows[:, :, 7::3] = 0
    top = torch.tensor([[2.0 ** e, -1.75 * 2.0 ** e] for e in range(-149, -109)], dtype=torch.float64)
    rows[:, :, 5] = 1
    rows = (rows * top[..., None]).float()
    (kc, vc), (ks, vs) = page_tensors(3, 2, 16, dh, E4M3)
    kie.paged_append(rows.cuda(), rows.cuda(), kc, vc, torch.arange(n, device="cuda").int(), k_scale=ks, v_scale=vs)
    scale = (rows.abs().amax(-1).double() / 448).float()
    assert torch.any(scale == 0) and torch.any((scale > 0) & (scale < 2.0 ** -126)) and torch.any(scale > 2.0 ** -126)
    scale[scale == 0] = 2.0 ** -126
    codes = (rows.double() / scale.double()[..., None]).float().clamp(-448, 448).to(E4M3)
    for got, got_s in ((kc, ks), (vc, vs)):
        got, got_s = (x.cpu().transpose(1, 2).flatten(0, 1)[:n] for x in (got, got_s))
        assert torch.equal(got_s, scale)
        assert not torch.isnan(got.float()).any()
        assert torch.equal(bits(got), bits(codes))
        err = (got.double() * got_s.double()[..., None] - rows.double()).abs()
        assert torch.all(err <= rows.double().abs() * 2 ** -4 + got_s.double()[..., None] * 2 ** -10 + 448 * 2.0 ** -150)
    out = kie.paged_attention(torch.randn(1, 4, dh, device="cuda"), kc, vc, ints([[0, 1, 2]]), ints([n]), k_scale=ks, v_scale=vs)
    assert torch.all(torch.isfinite(out))


# ---- attention -----------------------------------------------------------------------------------------------

def loud_rows(level, count, v_scale, qt, seed=0):
    """A batch on E4M3 pages (as of `batch`) whose late rows 520, 521, ... score about `level` above the rest in every head,
    with the given V scale."""
    q, k, v, table, lens, ks, vs = batch([700] * 100, 4, 4, 64, 16, E4M3, qt, seed=seed, dead=0.0)
    ks *= 0.02  # the other scores stay below 20
    row = q.float() * (level * 8.0 / (q.float() ** 2).sum(-1, keepdim=True))  # the operator's scale is 1 / 8
    codes, scale = oracle.quantise(row)
    for at in range(520, 520 + count):
        page, r = table[:, at // 16].long(), at % 16
        k.view(torch.uint8)[page, :, r] = codes.view(torch.uint8)
        ks[page, :, r] = scale
        vs[page, :, r] = v_scale
    return q, k, v, table, lens, ks, vs


@pytest.mark.parametrize("qt", [F32, F16, BF16])
@pytest.mark.parametrize("v_scale", [0.0, 2.0 ** -126])
@pytest.mark.parametrize("level", [75, 78, 84, 86, 130, 200])
@pytest.mark.parametrize("count", [1, 3, 40])
def test_attention_where_rows_of_vanishing_scale_dominate(count, level, v_scale, qt):
    """V rows of zeros (as the append stores them) whose weights outweigh the rest by up to e^200.

    To the bounds of the oracle comes what the header says of V scales below 2^-60: weights are held to 2^-32 of the
    largest weight, with the scales counted as 2^-60 at least, so that n positions of values up to 448 may be off by
    n * 448 * 2^-31 times the largest p_j max(scale_j, 2^-60)."""
    q, k, v, table, lens, ks, vs = loud_rows(level, count, v_scale, qt)
    out, lse = kie.paged_attention(q, k, v, table, lens, k_scale=ks, v_scale=vs, return_lse=True)
    ref = oracle.attention(q, k, v, table, lens, 0.125, 0, ks, vs)
    tol_out, tol_lse = oracle.attention_bounds(q, E4M3, *ref)
    # the loud rows have the largest p, which is at most 1, and a scale of 2^-60 counted; every other row a p below
    # e^(20 - level) and a scale below 2^4
    largest = max(2.0 ** -60, 16 * math.exp(20 - level))
    assert not torch.isnan(out).any()
    assert torch.all((lse.double() - ref[1]).abs() <= tol_lse)
    assert torch.all((out.double() - ref[0]).abs() <= tol_out + 700 * 448 * 2.0 ** -31 * largest)


def test_attention_with_an_infinite_scale_of_a_value_row():
    """What the append stores for a V row with an infinity: the head's output there is not finite, its lse is (it does not
    depend on V), and no other head's is touched."""
    q, k, v, table, lens, ks, vs = batch([300, 90, 300], 8, 4, 64, 16, E4M3, F16, dead=0.0)
    clean, lse = kie.paged_attention(q, k, v, table, lens, k_scale=ks, v_scale=vs, return_lse=True)
    vs[table[0, 15].item(), 1, 3] = math.inf
    out, got = kie.paged_attention(q, k, v, table, lens, k_scale=ks, v_scale=vs, return_lse=True)
    assert not torch.any(torch.isfinite(out[0, 2:4]))
    out[0, 2:4] = clean[0, 2:4]
    assert torch.equal(out, clean)
    _, tol = oracle.attention_bounds(q, E4M3, *oracle.attention(q, k, torch.zeros_like(v), table, lens, 0.125, 0, ks, ks))
    assert torch.all((got - lse).abs() <= 2 * tol)


@pytest.mark.parametrize("cache,qt", [(F16, F32), (F16, F16), (BF16, BF16)])
def test_attention_with_infinite_keys(cache, qt):
    """A score of -inf has weight 0: K rows with an infinity against queries of the other sign there count as left out, a
    sequence of such rows alone gives zeros and -inf. A score of +inf makes its head NaN, and only that one."""
    q, k, v, table, lens, ks, vs = batch([300, 40, 20, 90], 4, 2, 64, 16, cache, qt, dead=0.0)
    q[:, :, 9] = q[:, :, 9].abs() + 0.5
    finite = k.clone()
    gone = [torch.arange(0, 300, 7), torch.tensor([39]), torch.arange(20), torch.tensor([], dtype=torch.long)]
    for b, at in enumerate(gone):
        at = at.to("cuda")
        k[table[b].long()[at // 16], :, at % 16, 9] = -math.inf
    out, lse = kie.paged_attention(q, k, v, table, lens, return_lse=True)
    assert torch.all(out[2] == 0) and torch.all(lse[2] == -math.inf)
    for b in (0, 1, 3):  # against the kept positions, moved together
        kept = torch.tensor([p for p in range(int(lens[b])) if p not in gone[b].tolist()], device="cuda")
        page, r = table[b].long()[kept // 16], kept % 16
        n = oracle.ceil_div(kept.numel(), 16)
        pages = [torch.zeros((n, 16, 2, 64), dtype=cache, device="cuda") for _ in range(2)]
        for x, y in zip(pages, (finite, v)):
            x.view(-1, 2, 64)[:kept.numel()] = y[page, :, r]
        pages = [x.transpose(1, 2) for x in pages]
        ref = oracle.attention(q[b:b + 1], *pages, torch.arange(n, device="cuda")[None], ints([kept.numel()]), 0.125)
        tol_out, tol_lse = oracle.attention_bounds(q[b:b + 1], cache, *ref)
        assert torch.all((out[b:b + 1].double() - ref[0]).abs() <= tol_out), b
        assert torch.all((lse[b:b + 1].double() - ref[1]).abs() <= tol_lse), b
    k[table[3, 2].item(), 1, 5, 9] = math.inf
    again = kie.paged_attention(q, k, v, table, lens)
    assert torch.all(torch.isnan(again[3, 2:])) and torch.equal(again[3, :2], out[3, :2]) and torch.equal(again[:3], out[:3])


@pytest.mark.parametrize("cache,qt", [(F16, F32), (F16, F16), (BF16, BF16)])
def test_attention_with_infinite_values(cache, qt):
    """An infinity in V makes its own element of the heads that attend it infinite or NaN, and nothing else."""
    q, k, v, table, lens, ks, vs = batch([70, 700, 70], 4, 2, 64, 16, cache, qt)
    clean, lse = kie.paged_attention(q, k, v, table, lens, return_lse=True)
    v[table[1, 30].item(), 0, 3, 5] = math.inf
    out, got = kie.paged_attention(q, k, v, table, lens, return_lse=True)
    assert not torch.any(torch.isfinite(out[1, :2, 5])) and torch.equal(got, lse)
    out[1, :2, 5] = clean[1, :2, 5]
    assert torch.equal(out, clean)
