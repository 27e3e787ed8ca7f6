"""Forks, copies and compaction of a paged cache on the GPU, integers and bytes equal to the plain implementations, and
the operators together: continuations of one prompt decoded side by side."""
import numpy as np
import pytest
import torch

import persistent_monokernel_decode_gb300 as kie
import shared_oracle as oracle
from test_gpu_paged import BF16, E4M3, F16, F32, bits, f16, ints, page_tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


def state(rng, R, top, bs, W=None, spare=None, shared=True):
    """Rows of random lengths on random pages, some first pages of one row's being the next one's too."""
    W = W or max(1, -(-top // bs) + 1)
    lens = rng.randint(0, top + 1, R).tolist()
    pages = [-(-l // bs) for l in lens]
    spare = R + 3 if spare is None else spare
    n = sum(pages) + spare
    pool = rng.permutation(n).tolist()
    table = rng.randint(-5, 2 ** 31 - 1, (R, W)).tolist()
    holders = [0] * n
    for r in range(R):
        for j in range(pages[r]):
            full = r > 0 and shared and lens[r] >= (j + 1) * bs and lens[r - 1] >= (j + 1) * bs and rng.rand() < 0.5
            table[r][j] = table[r - 1][j] if full else pool.pop()
            holders[table[r][j]] += 1
    free = [x for x in pool]
    return lens, table, [max(0, h - 1) for h in holders], free + [-1] * (n - len(free)), len(free)


def check_fork(parents, lens, table, shares, free, n_free, bs):
    want = oracle.fork(parents, lens, table, shares, free, n_free, bs)
    t, s, fr = ints(table).reshape(len(lens), -1), ints(shares), ints(free)
    f = kie.paged_fork(ints(parents), ints(lens), t, s, fr, ints([n_free]), bs)
    got = (t.tolist(), s.tolist(), fr.tolist(), f.lens.tolist(), int(f.n_free), bool(f.ok), f.copy_src.tolist(),
           f.copy_dst.tolist(), f.copy_rows.tolist())
    for name, a, b in zip(("table", "shares", "free", "lens", "n_free", "ok", "src", "dst", "rows"), got, want):
        assert a == b, name
    return want


@pytest.mark.parametrize("R,top,bs", [(1, 40, 16), (2, 0, 16), (7, 100, 16), (33, 300, 48), (256, 700, 64), (1025, 90, 16),
                                      (3000, 20, 16)])
def test_fork(R, top, bs):
    rng = np.random.RandomState(R)
    for kind in range(5):
        lens, table, shares, free, n_free = state(rng, R, top, bs)
        near = np.clip(np.arange(R) // 4 * 4 + rng.randint(0, 4, R), 0, R - 1)
        parents = [rng.randint(-2, R + 2, R), np.arange(R), np.zeros(R, dtype=int), near, rng.permutation(R)][kind].tolist()
        lens, *rest = check_fork(parents, lens, table, shares, free, n_free, bs)[3:5] + (0,), None
        # what a fork has left can be forked again
        lens, table, shares, free, n_free = state(rng, R, top, bs)
        for _ in range(3):
            parents = rng.randint(-1, R, R).tolist()
            table, shares, free, lens, n_free, ok, *_ = check_fork(parents, lens, table, shares, free, n_free, bs)


def test_fork_without_enough_pages_changes_nothing():
    rng = np.random.RandomState(1)
    lens, table, shares, free, n_free = state(rng, 9, 100, 16, shared=False)
    lens = [max(1, l // 16 * 16 + 5) if l < 95 else 90 for l in lens]
    assert not check_fork([0] * 9, lens, table, shares, free, 7, 16)[5]
    assert check_fork([0] * 9, lens, table, shares, free, 8, 16)[5]
    assert check_fork(list(range(9)), lens, table, shares, free, 0, 16)[5]
    assert check_fork(list(range(9)), lens, table, shares, free, -5, 16)[4] == 0


def test_fork_of_odd_states():
    """Lengths below 0 and past the table, entries that are no pages, a list without room, the same page on it twice."""
    table = [[3, 99, -1], [5, 3, 2 ** 31 - 1], [0, 1, 2], [7, 7, 7]]
    for lens in ([-4, 40, 20, 1000], [33, 48, 49, 47], [1, 2, 3, -1]):
        for parents in ([1, 1, 1, 1], [3, 2, 1, 0], [-1, -9, 2, 2 ** 31 - 1], [0, 0, -1, -1]):
            for free in ([4, 6, 8], [4, 4, -1, 70, 6, 0, 0]):
                check_fork(parents, lens, table, [0, 2, 0, 1, -3, 0, 0, 0, 0], free, 3, 16)
                check_fork(parents, lens, table, [0] * 9, free, 100, 16)


def test_fork_of_nothing():
    f = kie.paged_fork(ints([]), ints([]), ints([]).reshape(0, 3), ints([0, -1, 0]), ints([2, -1]), ints([1]), 16)
    assert f.n_free.tolist() == [2] and f.ok.tolist() == [True] and f.lens.numel() == 0


@pytest.mark.parametrize("R,top,bs", [(5, 60, 16), (700, 300, 16), (2049, 90, 48)])
def test_release_of_shared_pages(R, top, bs):
    rng = np.random.RandomState(R)
    lens, table, shares, free, n_free = state(rng, R, top, bs)
    for every in (1, 3):
        done = rng.randint(0, every, R) == 0
        want = oracle.fork([-1 if d else r for r, d in enumerate(done)], lens, table, shares, free, n_free, bs)
        t, s, f = ints(table), ints(shares), ints(free)
        got = kie.paged_release(torch.tensor(done, device="cuda"), ints(lens), t, f, ints([n_free]), bs, s)
        assert t.tolist() == table and s.tolist() == want[1] and f.tolist() == want[2]
        assert got[0].tolist() == want[3] and got[1].tolist() == [want[4]]


@pytest.mark.parametrize("n,R,top,bs,percent", [(1, 1, 16, 16, 100), (2, 1, 16, 16, 50), (37, 3, 60, 16, 50), (1000, 40, 300, 16, 20),
                                                (4096, 100, 700, 32, 90), (30001, 300, 900, 16, 40), (9000, 5, 50, 16, 0)])
def test_compact(n, R, top, bs, percent):
    rng = np.random.RandomState(n)
    W = -(-top // bs)
    order = rng.permutation(n).tolist()
    n_free = n * percent // 100
    held = order[n_free:]
    lens, table = rng.randint(-3, top + 20, R).tolist(), rng.randint(-5, n + 5, (R, W)).tolist()
    for r in range(R):
        for j in range(W):
            if held and rng.rand() < 0.9:
                table[r][j] = held[rng.randint(len(held))]
    shares = rng.randint(0, 5, n).tolist()
    for free in (order[:n_free] + [-1] * (n - n_free), (order[:n_free] + [-1, n, 2 ** 31 - 1] + order[:n_free // 2])[:n], order[:n_free]):
        for count in (n_free, n_free // 2, n + 7):
            want = oracle.compact(lens, table, shares, free, count, bs)
            t, s, f = ints(table), ints(shares), ints(free)
            m = kie.paged_compact(ints(lens), t, s, f, ints([count]), bs)
            got = (t.tolist(), s.tolist(), f.tolist(), int(m.n_free), m.src.tolist(), m.dst.tolist(), m.page_map.tolist())
            for name, a, b in zip(("table", "shares", "free", "n_free", "src", "dst", "map"), got, want):
                assert a == b, name


@pytest.mark.parametrize("cache", [F16, BF16, E4M3])
@pytest.mark.parametrize("hkv,bs,dh,order", [(4, 16, 128, "head"), (2, 48, 64, "position"), (7, 32, 64, "pool"), (1, 1024, 128, "head")])
@pytest.mark.parametrize("part", [False, True])
def test_copy_of_one_layer(cache, hkv, bs, dh, order, part):
    n = 24
    (k, v), (ks, vs) = page_tensors(n, hkv, bs, dh, cache, order)
    for x in (k, v):
        x.copy_(torch.randn(x.shape, device="cuda").to(cache))
    if ks is not None:
        ks.copy_(torch.rand_like(ks)), vs.copy_(torch.rand_like(vs))
    src, dst = [3, -1, 5, 7, 9, 2, 11, 30, 3, 6], [20, 21, -4, 24, 12, 13, 14, 15, 16, 6]  # pairs that are none among them
    rows = [bs, 5, 5, 5, 0, 1, bs - 1, 5, bs + 9, 3] if part else None
    want = [x.clone() for x in (k, v, ks, vs) if x is not None]
    for i, (a, b) in enumerate(zip(src, dst)):
        if 0 <= a < n and 0 <= b < n:
            for x in want:
                r = min(rows[i], bs) if part else bs
                x[b, :, :r] = x[a, :, :r]
    assert kie.paged_copy(ints(src), ints(dst), k, v, rows=ints(rows) if part else None, k_scale=ks, v_scale=vs) is None
    for a, b in zip((x for x in (k, v, ks, vs) if x is not None), want):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("cache", [F16, E4M3])
@pytest.mark.parametrize("layers,pairs", [(1, 1), (3, 70), (25, 7)])
def test_copy_of_all_layers(cache, layers, pairs):
    n = 2 * pairs + 1
    shape = (layers, n, 4, 16, 128)
    k, v = (torch.randn(shape, device="cuda").to(cache) for _ in range(2))
    ks, vs = (torch.rand(shape[:4], device="cuda") if cache == E4M3 else None for _ in range(2))
    order = torch.randperm(n, device="cuda").int()
    src, dst = order[:pairs].contiguous(), order[pairs:2 * pairs].contiguous()
    want = [x.clone() for x in (k, v, ks, vs) if x is not None]
    for x in want:
        x = x.view(torch.uint8) if x.dtype == E4M3 else x
        x[:, dst.long()] = x[:, src.long()]
    kie.paged_copy(src, dst, k, v, k_scale=ks, v_scale=vs)
    for a, b in zip((x for x in (k, v, ks, vs) if x is not None), want):
        assert torch.equal(bits(a), bits(b))
    kie.paged_copy(src[:0], dst[:0], k, v, k_scale=ks, v_scale=vs)


def test_copy_past_32_bit_offsets():
    k = torch.zeros((2, 70000, 2, 64, 128), dtype=F16, device="cuda")
    v = torch.zeros_like(k)
    k[1, 69999], v[1, 69999] = 3.0, 4.0
    kie.paged_copy(ints([69999]), ints([69990]), k, v)
    assert torch.all(k[1, 69990] == 3) and torch.all(v[1, 69990] == 4) and torch.all(k[0, 69990] == 0)


def test_the_binding_refuses():
    table, lens, shares, free = ints([[0, 1]] * 2), ints([3, 3]), ints([0] * 4), ints([2, 3])
    for bad in (dict(parents=ints([0])), dict(parents=ints([0, 1]).long()), dict(shares=shares.float()), dict(n_free=ints([1, 2])),
                dict(lens=lens.cpu())):
        a = dict(parents=ints([0, 1]), lens=lens, block_table=table, shares=shares, free_blocks=free, n_free=ints([2]), block_size=16)
        a.update(bad)
        with pytest.raises(ValueError):
            kie.paged_fork(**a)
    with pytest.raises(kie.KieError):
        kie.paged_fork(ints([0, 1]), lens, table, shares, free, ints([2]), 17)
    with pytest.raises(ValueError):
        kie.paged_compact(lens, table, shares.long(), free, ints([2]), 16)
    with pytest.raises(ValueError):
        kie.paged_release(torch.tensor([True, False], device="cuda"), lens, table, free, ints([2]), 16, shares.long())
    k = torch.zeros((2, 4, 2, 16, 64), dtype=F16, device="cuda")
    for bad in (dict(dst=ints([1, 2])), dict(src=ints([0]).long()), dict(v_cache=k[0]), dict(rows=ints([1, 2])),
                dict(k_scale=torch.ones(2, 4, 2, 16, device="cuda")), dict(k_cache=k.float(), v_cache=k.float())):
        a = dict(src=ints([0]), dst=ints([1]), k_cache=k, v_cache=k.clone())
        a.update(bad)
        with pytest.raises(ValueError):
            kie.paged_copy(**a)
    with pytest.raises(ValueError):
        kie.paged_copy(ints([0]), ints([1]), k.to(E4M3), k.to(E4M3))


# ---- together ------------------------------------------------------------------------------------------------

def model():
    import synth
    from synth.configs import TINY as M
    weights = synth.model_weights(M)
    w = {k: f16(weights[k]) for k in ("embed", "lm_head", "final_norm")}
    w["layers"] = [{k: f16(v) for k, v in lay.items()} for lay in weights["layers"]]
    return M, weights, w


def forward(M, w, cache, step, tokens, groups):
    """The logits [rows, vocab] of a step's tokens: plain fp32 projections around the paged operators."""
    def rms(x, gain):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + M.rms_eps) * gain

    x = w["embed"][tokens.long()]
    for l, lay in enumerate(w["layers"]):
        u = rms(x, lay["attn_norm"])
        q, k, v = ((u @ lay[n].T).view(len(tokens), -1, M.head_dim) for n in ("wq", "wk", "wv"))
        q = cache.append(l, k, v, step, q=q)
        o = cache.attention(l, q, step, groups=groups)
        x = x + o.reshape(len(tokens), -1) @ lay["wo"].T
        u = rms(x, lay["ffn_norm"])
        x = x + (torch.nn.functional.silu(u @ lay["w_gate"].T) * (u @ lay["w_up"].T)) @ lay["w_down"].T
    return rms(x, w["final_norm"]) @ w["lm_head"].T


def test_a_beam_search_over_shared_pages():
    """Two requests of three beams each: the prompts prefilled once, forked into beams, then steps of extend, append,
    attention over the shared prompt, log probabilities with their alternatives, and a fork to the best continuations; once
    in between the cache is compacted. The scores of every beam agree with a Decoder's that is given the beam's tokens (each
    log probability within twice the decoder's own logit tolerance of 2e-2: the token's and the log-sum's), and with the last
    request released every page is free again."""
    M, weights, w = model()
    import synth
    prompts = [synth.tokens(31, 37, M.vocab), synth.tokens(32, 16, M.vocab)]
    B, steps = 3, 12
    cache = kie.PagedCache(M, n_blocks=40, block_size=16, max_seqs=2 * B, max_blocks=6, shared=True)
    dec = kie.Decoder(M, weights, max_seq=96)
    first = []
    for i, p in enumerate(prompts):
        dec.reset()
        dec.prefill(p)
        step = cache.extend(ints([len(p) if r == B * i else 0 for r in range(2 * B)]), len(p))
        cache.load(dec, step)
        first.append(dec.logits())
    f = cache.fork(ints([0, 0, 0, 3, 3, 3]))
    assert f.ok.tolist() == [True] and cache.lens.tolist() == [37] * 3 + [16] * 3
    assert cache.n_free.tolist() == [40 - 3 - 2 - 1] and cache.shares.sum() == 2 * (2 + 1)
    groups = ints([0, B, 2 * B]), ints([len(p) for p in prompts])

    top = kie.token_logprobs(torch.tensor(np.stack(first), device="cuda"), ints([-1, -1]), top=B)
    tokens = top.top_ids.reshape(-1)
    scores = top.top_logprobs.reshape(-1)
    beams = [[int(t)] for t in tokens]
    for i in range(steps):
        step = cache.extend(ints([1] * (2 * B)), 2 * B)
        assert step.admitted.tolist() == [True] * (2 * B)
        logits = forward(M, w, cache, step, tokens, groups)
        p = kie.token_logprobs(logits, ints([-1] * (2 * B)), top=B)
        total = (scores[:, None] + p.top_logprobs).view(2, B * B)
        best = torch.topk(total, B, dim=1)
        parents = (best.indices // B + torch.arange(2, device="cuda")[:, None] * B).view(-1)
        tokens = p.top_ids.view(-1)[(parents * B + best.indices.view(-1) % B)].int().contiguous()
        scores = best.values.reshape(-1)
        beams = [beams[q] + [int(t)] for q, t in zip(parents.tolist(), tokens.tolist())]
        assert cache.fork(parents.int()).ok.tolist() == [True]
        if i == 5:
            held = 40 - int(cache.n_free)
            cache.compact()
            assert cache.n_free.tolist() == [40 - held]
            live = [set(cache.block_table[r, :-(-int(n) // 16)].tolist()) for r, n in enumerate(cache.lens)]
            assert max(max(s) for s in live) == held - 1 and len(set().union(*live)) == held

    for r, beam in enumerate(beams):
        dec.reset()
        dec.prefill(prompts[r // B])
        rows = np.concatenate([dec.logits()[None], dec.decode_forced(np.array(beam[:-1], dtype=np.int32))[1]])
        logp = torch.log_softmax(torch.tensor(rows).double(), 1)
        want = float(logp[torch.arange(len(beam)), torch.tensor(beam)].sum())
        assert abs(want - float(scores[r])) <= len(beam) * 4e-2, r
    cache.release(torch.tensor([True] * B + [False] * B, device="cuda"))
    cache.release(torch.tensor([False] * B + [True] * B, device="cuda"))
    assert cache.n_free.tolist() == [40] and sorted(cache.free_blocks.tolist()) == list(range(40)) and not cache.shares.any()
    dec.close()


def test_a_captured_step_of_forks():
    """extend, append, attention, log probabilities and fork captured once and replayed: as the same steps run eagerly."""
    M, _, w = model()

    def run(captured):
        torch.manual_seed(0)
        cache = kie.PagedCache(M, n_blocks=60, block_size=16, max_seqs=4, max_blocks=8, shared=True)
        step = cache.extend(ints([30, 0, 0, 0]), 30)
        for l in range(M.n_layers):
            k, v = (torch.randn(30, M.n_kv_heads, M.head_dim, device="cuda") for _ in range(2))
            cache.append(l, k, v, step)
        cache.fork(ints([0, 0, 0, 0]))
        groups, ones = (ints([0, 4]), ints([30])), ints([1] * 4)
        tokens, parents = ints([5, 6, 7, 8]), ints([0, 1, 2, 3])

        def one():
            logits = forward(M, w, cache, cache.extend(ones, 4), tokens, groups)
            p = kie.token_logprobs(logits, tokens, top=2)
            tokens.copy_(p.top_ids[:, 1])
            parents.copy_((parents * 3 + 1) % 4)
            cache.fork(parents)

        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                one()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    one()
                for _ in range(20):
                    graph.replay()
            torch.cuda.synchronize()
        else:
            for _ in range(21):
                one()
        return [x.tolist() for x in (cache.lens, cache.block_table, cache.n_free, cache.shares, cache.free_blocks, tokens)]

    assert run(True) == run(False)


def test_a_cache_that_does_not_share():
    M, _, _ = model()
    cache = kie.PagedCache(M, n_blocks=10, block_size=16, max_seqs=2, max_blocks=4)
    with pytest.raises(ValueError):
        cache.fork(ints([0, 0]))
    step = cache.extend(ints([20, 40]), 60)
    k = torch.randn(60, M.n_kv_heads, M.head_dim, device="cuda")
    cache.append(0, k, k, step)
    cache.release(torch.tensor([True, False], device="cuda"))
    before = cache.k[0][cache.block_table[1, :3].long()].clone()
    cache.compact()
    assert sorted(cache.block_table[1, :3].tolist()) == [0, 1, 2] and cache.n_free.tolist() == [7]
    assert torch.equal(cache.k[0][cache.block_table[1, :3].long()], before)
