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


# ---- rows of a step ------------------------------------------------------------------------------------------

def check_rows(q, k, v, table, seqs, positions, ks=None, vs=None, window=0):
    """Every row against the plain attention over its own sequence's positions up to its own."""
    out, lse = kie.paged_attention(q, k, v, table, None, seqs=seqs, positions=positions, window=window, k_scale=ks,
                                   v_scale=vs, return_lse=True)
    live = (seqs >= 0) & (seqs < table.shape[0]) & (positions >= 0)
    lens = torch.where(live, positions.long() + 1, 0)
    ref = oracle.attention(q, k, v, table[torch.where(live, seqs, 0).long()], lens, q.shape[-1] ** -0.5, window, ks, vs)
    tol_out, tol_lse = oracle.attention_bounds(q, k.dtype, *ref)
    assert torch.all((out.double() - ref[0]).abs() <= tol_out)
    empty = ref[4] == 0
    assert torch.all(out[empty] == 0) and torch.all(lse[empty] == -math.inf) and torch.all(empty[~live])
    assert torch.all((lse.double() - ref[1]).abs()[~empty] <= tol_lse[~empty])
    return out, lse


@pytest.mark.parametrize("cache,qt", [(F16, F16), (F16, F32), (BF16, BF16), (E4M3, F32), (E4M3, F16)])
@pytest.mark.parametrize("window", [0, 20])
def test_attention_of_the_rows_of_a_step(cache, qt, window):
    """Rows in any order, several of a sequence, sequences without a row, and rows that belong to none."""
    lens = [70, 0, 200, 33, 1, 16]
    q, k, v, table, _, ks, vs = batch(lens, 8, 2, 128, 32, cache, qt)
    rows = [(2, 199), (0, 69), (0, 68), (-1, 5), (3, 32), (2, 0), (6, 3), (2 ** 31 - 1, 0), (5, -1), (4, 0), (3, 31), (-1, -1),
            (0, -2 ** 31), (5, 15)] + [(2, p) for p in range(40)]
    q = torch.randn((len(rows), 8, 128), generator=gen(4), device="cuda").to(qt)
    check_rows(q, k, v, table, ints([s for s, _ in rows]), ints([p for _, p in rows]), ks, vs, window)


def test_attention_of_rows_past_the_table_is_cut_there():
    q, k, v, table, lens, ks, vs = batch([64, 64], 4, 2, 64, 16, F16, F16)
    out = kie.paged_attention(q, k, v, table, None, seqs=ints([1, 0]), positions=ints([2 ** 31 - 1, 64]))
    assert torch.equal(out, kie.paged_attention(q, k, v, table.flip(0), lens))


def test_attention_of_rows_as_of_sequences():
    """The rows 0 .. B - 1 at the sequences' last positions: the same bits as with the lengths."""
    q, k, v, table, lens, ks, vs = batch([700, 0, 33, 2000], 20, 4, 128, 16, F16, F32)
    want = kie.paged_attention(q, k, v, table, lens, return_lse=True)
    got = kie.paged_attention(q, k, v, table, None, seqs=torch.arange(4, device="cuda").int(), positions=lens - 1, return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_a_step_with_idle_refused_and_prompt_rows(dtype):
    """Sequences that bring nothing, one token, several or too many: every query attends over its own sequence."""
    from synth.configs import MOE_TINY as M
    cache = kie.PagedCache(M, n_blocks=9, block_size=16, max_seqs=6, max_blocks=3, dtype=dtype)
    # step 2: request 1 is longer than its table row, 5 finds no page; step 3: 3 is idle and 5 is refused again
    for i, (new, n_rows, ok) in enumerate([([5, 16, 0, 31, 1, 0], 60, [1, 1, 1, 1, 1, 1]), ([1, 33, 20, 0, 1, 40], 95, [1, 0, 1, 1, 1, 0]),
                                           ([1, 1, 1, 0, 1, 40], 48, [1, 1, 1, 1, 1, 0]), ([1, 0, 1, 1, 0, 1], 9, [1] * 6)]):
        step = cache.extend(ints(new), n_rows)
        assert step.admitted.tolist() == [bool(x) for x in ok], i
        g = gen(i)
        q, k, v = (torch.randn((n_rows, h, M.head_dim), generator=g, device="cuda") for h in (M.n_heads, M.n_kv_heads, M.n_kv_heads))
        rq = cache.append(0, k, v, step, q=q)
        dead = step.seqs < 0
        rq[dead] = math.nan  # what rows that belong to none hold is of no consequence
        out = cache.attention(0, rq, step)
        scales = (None, None) if cache.k_scale is None else (cache.k_scale[0], cache.v_scale[0])
        want, _ = check_rows(rq, cache.k[0], cache.v[0], cache.block_table, step.seqs, step.positions, *scales)
        assert torch.equal(out, want) and torch.all(out[dead] == 0) and dead.any()
        seqs = [r for r in range(6) if ok[r] for _ in range(new[r])]
        assert step.seqs[step.seqs >= 0].tolist() == seqs


def test_a_captured_step_follows_its_rows():
    """One captured step replayed with another set of sequences each time."""
    from synth.configs import MOE_TINY as M
    n = 6
    cache = kie.PagedCache(M, n_blocks=40, block_size=16, max_seqs=n, max_blocks=4)
    new = ints([1] * n)
    q, k, v = (torch.randn(n, h, M.head_dim, device="cuda") for h in (M.n_heads, M.n_kv_heads, M.n_kv_heads))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step = cache.extend(new, n)
        rq = cache.append(0, k, v, step, q=q)
        out, lse = cache.attention(0, rq, step, return_lse=True)
    rng = np.random.RandomState(0)
    for _ in range(12):
        who = rng.randint(0, 2, n)
        new.copy_(ints(who.tolist()))
        k.normal_(), v.normal_()
        g.replay()
        assert step.seqs.tolist() == np.flatnonzero(who).tolist() + [-1] * int(n - who.sum())
        want = check_rows(rq.nan_to_num(), cache.k[0], cache.v[0], cache.block_table, step.seqs, step.positions)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_a_batched_decode_with_waiting_sequences_matches_the_decoder():
    """Three prompts decoded together where in most steps some sequence waits, and one is refused until another's pages
    are free: every sequence's logits stay those of a Decoder running it alone."""
    import synth
    from synth.configs import TINY as M
    from test_gpu_paged import f16
    weights = synth.model_weights(M)
    w = {k: f16(weights[k]) for k in ("embed", "lm_head", "final_norm")}
    w["layers"] = [{k: f16(v) for k, v in lay.items()} for lay in weights["layers"]]
    prompts = [synth.tokens(s, n, M.vocab) for s, n in ((11, 20), (12, 9), (13, 32))]
    decs = [kie.Decoder(M, weights, max_seq=96) for _ in prompts]
    cache = kie.PagedCache(M, n_blocks=5, block_size=16, max_seqs=3, max_blocks=6)
    for d, p in zip(decs, prompts):
        d.prefill(p)
    step = cache.extend(ints([len(p) for p in prompts]), sum(len(p) for p in prompts))
    for d, at in zip(decs, (0, 20, 29)):
        cache.load(d, step, at)
    current = [d.logits() for d in decs]

    def rms(x, gain):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + M.rms_eps) * gain

    def advance(who):
        """One token of each sequence of `who`; the sequences that were admitted."""
        toks = [int(np.argmax(current[b])) for b in who]
        step = cache.extend(ints([int(b in who) for b in range(3)]), 3)
        x = w["embed"][torch.tensor(toks + [0] * (3 - len(who)), device="cuda")]
        for l, lay in enumerate(w["layers"]):
            u = rms(x, lay["attn_norm"])
            q, k, v = ((u @ lay[n].T).view(3, -1, M.head_dim) for n in ("wq", "wk", "wv"))
            o = cache.attention(l, cache.append(l, k, v, step, q=q), step)
            x = x + o.reshape(3, -1) @ lay["wo"].T
            u = rms(x, lay["ffn_norm"])
            x = x + (torch.nn.functional.silu(u @ lay["w_gate"].T) * (u @ lay["w_up"].T)) @ lay["w_down"].T
        logits = (rms(x, w["final_norm"]) @ w["lm_head"].T).cpu().numpy()
        went = [b for b in who if step.admitted[b]]
        for row, b in enumerate(who):
            if b in went:
                current[b] = decs[b].decode_forced(np.array([toks[row]], dtype=np.int32))[1][0]
                assert np.max(np.abs(logits[row] - current[b])) <= 2e-2, b
        return went

    for who in ([0, 1, 2], [0, 2], [1], [1, 2], [2], [0, 1]):
        # 2 + 1 + 2 pages are all there are: sequence 2 is full at 32 positions and refused
        assert advance(who) == [b for b in who if b != 2]
    assert cache.lens.tolist() == [23, 13, 32]
    cache.release(torch.tensor([True, False, False], device="cuda"))
    for who in ([1, 2], [2], [1, 2]):
        assert advance(who) == who
    assert cache.lens.tolist() == [0, 15, 35]
    for d in decs:
        d.close()


def test_rows_and_lengths_exclude_each_other():
    q, k, v, table, lens, _, _ = batch([20, 3], 4, 2, 64, 16, F16, F16)
    some = ints([0, 1])
    for bad in (dict(lens=lens, seqs=some, positions=some), dict(lens=None), dict(lens=None, seqs=some),
                dict(lens=None, positions=some), dict(lens=lens, positions=some), dict(lens=None, seqs=some[:1], positions=some),
                dict(lens=None, seqs=some, positions=some.long()), dict(lens=None, seqs=some.cpu(), positions=some)):
        with pytest.raises(ValueError):
            kie.paged_attention(q, k, v, table, bad.pop("lens"), **bad)


@pytest.mark.parametrize("cache,qt", [(F16, F32), (E4M3, BF16)])
def test_attention_of_a_prompt_behind_a_prefix(cache, qt):
    """Every row of a prompt of 300 behind 130 cached positions, next to a sequence that decodes."""
    q, k, v, table, _, ks, vs = batch([57, 430], 2, 1, 64, 16, cache, qt)
    q = torch.randn((301, 2, 64), generator=gen(9), device="cuda").to(qt)
    check_rows(q, k, v, table, ints([0] + [1] * 300), ints([56] + list(range(130, 430))), ks, vs)


# ---- prompts of a Decoder ------------------------------------------------------------------------------------

def test_load_refuses_rows_that_are_not_the_prompts():
    """A decoder that has gone past its prompt, a sequence that was not admitted or not empty, another model's decoder:
    nothing is copied."""
    import synth
    from synth.configs import MOE_TINY, TINY as M
    dec = kie.Decoder(M, synth.model_weights(M), max_seq=64)
    dec.prefill(synth.tokens(31, 20, M.vocab))
    cache = kie.PagedCache(M, n_blocks=4, block_size=16, max_seqs=3, max_blocks=3)
    step = cache.extend(ints([20, 20, 1]), 41)  # sequence 2 finds no page
    assert step.admitted.tolist() == [True, True, False]
    for first in (1, 10, 20 + 1, -41, 40, 2 ** 40):
        with pytest.raises(ValueError):
            cache.load(dec, step, first)
    dec.decode(1)
    for first in (0, 20):  # 21 positions for 20 rows
        with pytest.raises(ValueError):
            cache.load(dec, step, first)
    assert not cache.k.any() and not cache.v.any()
    dec.reset()
    dec.prefill(synth.tokens(31, 1, M.vocab))
    with pytest.raises(ValueError):
        cache.load(dec, step, 40)
    step = cache.extend(ints([0, 1, 0]), 1)
    with pytest.raises(ValueError):
        cache.load(dec, step)  # position 20, not 0
    assert not cache.k.any() and not cache.v.any()
    other = kie.PagedCache(MOE_TINY, n_blocks=4, block_size=16, max_seqs=1, max_blocks=3)
    step = other.extend(ints([1]), 1)
    with pytest.raises(ValueError):
        other.load(dec, step)
    dec.close()


# ---- pages that are none -------------------------------------------------------------------------------------

def test_page_ids_outside_the_pages_pass_through_and_are_left_out():
    """Release and extend move ids as they are; rows on such a page get no slot, or one that the append skips, and the
    attention leaves its positions out."""
    bs, n = 16, 5
    bad = [-1, n, 2 ** 31 - 1, -2 ** 31]
    table = ints([[3, bad[0], bad[1], bad[2]], [bad[3], 4, -1, -1]])
    free = torch.full((12,), 7777, dtype=torch.int32, device="cuda")
    lens, n_free = kie.paged_release(torch.ones(2, dtype=torch.bool, device="cuda"), ints([64, 17]), table, free, ints([0]), bs)
    assert free.tolist() == [3, *bad[:3], bad[3], 4] + [7777] * 6 and n_free.tolist() == [6] and lens.tolist() == [0, 0]
    step = kie.paged_extend(ints([96]), ints([0]), (wide := ints([[-1] * 6])), free, n_free, bs, 96)
    assert wide.tolist() == [[4, bad[3], bad[2], bad[1], bad[0], 3]] and step.n_free.tolist() == [0]
    slots = step.slots.tolist()
    assert slots[:16] == list(range(64, 80)) and slots[80:] == list(range(48, 64))
    assert all(s == -1 or s >= n * bs for s in slots[16:80])
    (kc, vc), _ = page_tensors(n, 2, bs, 64, F16)
    rows = torch.randn((96, 2, 64), generator=gen(1), device="cuda")
    kie.paged_append(rows, rows, kc, vc, step.slots)
    for page, at in ((4, 0), (3, 80)):
        assert torch.equal(kc[page].transpose(0, 1), rows[at:at + 16].half())
    assert not kc[:3].any() and not vc[:3].any()
    q = torch.randn((1, 4, 64), generator=gen(2), device="cuda")
    ref = oracle.attention(q, kc, vc, wide, step.lens, 0.125)
    assert ref[4].item() == 32
    out = kie.paged_attention(q, kc, vc, wide, step.lens)
    assert torch.all((out.double() - ref[0]).abs() <= oracle.attention_bounds(q, F16, *ref)[0])
