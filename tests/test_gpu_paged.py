"""Paged-cache operators on the GPU against the plain implementations of paged_oracle (integers equal, values within
bounds derived there): types, head layouts, lengths, strides, dead positions, padding, streams, graphs, and the four
operators together as one batched decode of a model."""
import numpy as np
import pytest
import torch

import paged_oracle as oracle
import persistent_monokernel_decode_gb300 as kie

pytestmark = pytest.mark.gpu

F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---- pages and slots -----------------------------------------------------------------------------------------

def check_extend(new, lens, bs, W, n_free, n_rows, capacity=None, seed=0):
    rng = np.random.RandomState(seed)
    pool = rng.permutation(sum(oracle.ceil_div(max(l, 0), bs) for l in lens) + (capacity or n_free)).tolist()
    table = [[-1] * W for _ in lens]
    for r, l in enumerate(lens):
        for j in range(min(W, oracle.ceil_div(max(l, 0), bs))):
            table[r][j] = pool.pop()
    free = pool[:capacity or n_free]
    want = oracle.extend(new, lens, table, free, n_free, bs, n_rows)
    t = ints(table).reshape(len(lens), W)
    step = kie.paged_extend(ints(new), ints(lens), t, ints(free), ints([n_free]), bs, n_rows)
    for name, got, ref in zip(("table", "lens", "n_free", "admitted", "row_start", "slots", "positions", "seqs"),
                              (t, *step), want):
        ref = [ref] if name == "n_free" else ref
        assert got.tolist() == ref, name


@pytest.mark.parametrize("new,lens,bs,W,n_free,n_rows", [
    ([1], [0], 16, 1, 1, 1),
    ([0], [0], 16, 1, 0, 0),
    ([1, 1, 33, 0], [15, 16, 0, 5], 16, 3, 5, 36),
    ([20, 17, 1, 1], [0, 0, 3, 0], 16, 2, 3, 39),        # pages run out: refused in order
    ([5, 6, 7], [0, 0, 0], 16, 2, 9, 12),                 # rows run out
    ([40, 1], [0, 3], 16, 2, 9, 41),                      # a table row is full
    ([-1, 4, 3], [2, -2, 1], 16, 2, 9, 9),                # negative lengths are not admitted
    ([3, 0, 0, 2], [0, 0, 0, 46], 48, 1, 2, 8)])          # empty requests, a page size that is no power of two
def test_extend_small(new, lens, bs, W, n_free, n_rows):
    check_extend(new, lens, bs, W, n_free, n_rows)


@pytest.mark.parametrize("R,top,bs,short", [(513, 1, 16, 0), (1025, 300, 32, 0), (2100, 40, 16, 900), (300, 700, 64, 5)])
def test_extend_large(R, top, bs, short):
    rng = np.random.RandomState(R)
    new, lens = rng.randint(0, top + 1, R).tolist(), rng.randint(0, 500, R).tolist()
    need = sum(oracle.ceil_div(l + n, bs) - oracle.ceil_div(l, bs) for n, l in zip(new, lens))
    check_extend(new, lens, bs, oracle.ceil_div(500 + top, bs), need - short, sum(new) + 100, capacity=need + 10)


def test_extend_of_nothing():
    step = kie.paged_extend(ints([]), ints([]), ints([]).reshape(0, 3), ints([4, 5]), ints([2]), 16, 7)
    assert step.n_free.tolist() == [2] and step.row_start.tolist() == [0] and step.slots.tolist() == [-1] * 7


@pytest.mark.parametrize("R,top,bs,every", [(1, 40, 16, 1), (700, 300, 16, 3), (2049, 90, 48, 1), (5, 0, 16, 1)])
def test_release(R, top, bs, every):
    rng = np.random.RandomState(R)
    lens, W = rng.randint(0, top + 1, R).tolist(), max(1, oracle.ceil_div(top, bs))
    done = (rng.randint(0, every, R) == 0).tolist()
    table = rng.randint(0, 10 ** 6, (R, W)).tolist()
    for capacity in (10 + R * W, 10 + R * W // 4):  # room for every page, or not
        free = rng.randint(0, 10 ** 6, capacity).tolist()
        f = ints(free)
        got = kie.paged_release(torch.tensor(done, device="cuda"), ints(lens), ints(table).reshape(R, W), f, ints([7]), bs)
        want = oracle.release(done, lens, table, free, 7, bs)
        assert f.tolist() == want[0] and got[0].tolist() == want[1] and got[1].tolist() == [want[2]]


# ---- append --------------------------------------------------------------------------------------------------

def page_tensors(n, hkv, bs, dh, dtype, order="head"):
    if order == "position":  # [n, bs, hkv, dh] in memory
        kv = [torch.zeros((n, bs, hkv, dh), dtype=dtype, device="cuda").permute(0, 2, 1, 3) for _ in range(2)]
    elif order == "pool":    # K and V of a page side by side, several layers in one pool
        pool = torch.zeros((n, 3, 2, hkv, bs, dh), dtype=dtype, device="cuda")
        kv = [pool[:, 1, 0], pool[:, 1, 1]]
    else:
        kv = [torch.zeros((n, hkv, bs, dh), dtype=dtype, device="cuda") for _ in range(2)]
    sc = [torch.full((n, hkv, bs), 7.0, device="cuda") if dtype == E4M3 else None for _ in range(2)]
    return kv, sc


def bits(x):
    return x.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


@pytest.mark.parametrize("T,hq,hkv,dh,bs", [(1, 20, 4, 128, 16), (33, 4, 2, 64, 32), (257, 7, 7, 128, 48), (5, 3, 1, 64, 16)])
@pytest.mark.parametrize("x", [F16, BF16, F32])
@pytest.mark.parametrize("cache", [F16, BF16, E4M3])
def test_append(T, hq, hkv, dh, bs, x, cache):
    g = gen(T + dh)
    n = oracle.ceil_div(T, bs) + 2
    q, k, v = (torch.randn((T, h, dh), generator=g, device="cuda").to(x) for h in (hq, hkv, hkv))
    if T > 3:
        v[2, 0] = 0  # a row of zeros
    pad = T // 5
    slots = torch.randperm(n * bs, generator=g, device="cuda")[:T].int()
    positions = torch.randint(0, 99, (T,), generator=g, device="cuda").int()
    slots[T - pad:] = ints([-1, n * bs, -7, 2 ** 31 - 1] * T)[:pad]  # padding, and slots outside the pages
    if pad > 1:
        slots[0], positions[0] = 3, 99  # a position outside the table
    rope = kie.rope_table(10000.0, dh, 99)
    live = (slots >= 0) & (slots < n * bs) & (positions < 99)
    for order in ("head", "position", "pool"):
        (kc, vc), (ks, vs) = page_tensors(n, hkv, bs, dh, cache, order)
        q_out = torch.full_like(q, 5.0)
        kie.paged_append(k, v, kc, vc, slots, positions=positions, rope=rope, q=q, q_out=q_out, k_scale=ks, v_scale=vs)
        want_q = torch.where(live[:, None, None], oracle.rotate(q, rope, positions.clamp(max=98)).to(x), q_out)
        assert torch.equal(bits(q_out), bits(want_q))
        assert torch.all(q_out[~live] == 5)
        at = slots[live].long()
        for rows, got, got_s in ((oracle.rotate(k, rope, positions.clamp(max=98)), kc, ks), (v.float(), vc, vs)):
            (want, _), (want_s, _) = page_tensors(n, hkv, bs, dh, cache)
            rows = rows[live]
            if cache == E4M3:
                codes, scale = oracle.quantise(rows)
                want.view(torch.uint8)[at // bs, :, at % bs] = codes.view(torch.uint8)
                want_s[at // bs, :, at % bs] = scale
                assert torch.equal(got_s, want_s)
            else:
                want[at // bs, :, at % bs] = rows.to(cache)
            assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("x", [F16, F32])
def test_append_strided_unaligned_and_in_place(x):
    """Rows cut from a wider QKV tensor, one element off a 16-byte boundary, and q rotated in place."""
    g = gen(3)
    T, hq, hkv, dh, bs = 19, 4, 2, 64, 16
    wide = torch.randn(T * ((hq + 2 * hkv) * dh + 3) + 1, generator=g, device="cuda").to(x)[1:]
    wide = wide.view(T, -1)[:, :-3].unflatten(1, (hq + 2 * hkv, dh))
    q, k, v = wide.split((hq, hkv, hkv), 1)
    rope, positions = kie.rope_table(10000.0, dh, 64), torch.arange(T, device="cuda").int()
    slots = torch.randperm(32, generator=g, device="cuda")[:T].int()
    want_q, want_k, want_v = oracle.rotate(q, rope, positions).to(x), oracle.rotate(k, rope, positions).to(F16), v.to(F16)
    (kc, vc), _ = page_tensors(2, hkv, bs, dh, F16)
    assert kie.paged_append(k, v, kc, vc, slots, positions=positions, rope=rope, q=q, q_out=q) is q
    at = slots.long()
    assert torch.equal(q, want_q)
    assert torch.equal(kc[at // bs, :, at % bs], want_k) and torch.equal(vc[at // bs, :, at % bs], want_v)


def test_append_without_rotation_and_of_nothing():
    (kc, vc), _ = page_tensors(2, 2, 16, 64, F16)
    k = torch.randn(3, 2, 64, device="cuda")
    assert kie.paged_append(k, k, kc, vc, ints([31, 0, 5])) is None
    assert torch.equal(kc[1, :, 15], k[0].half()) and torch.equal(vc[0, :, 5], k[2].half())
    before = kc.clone()
    kie.paged_append(k[:0], k[:0], kc, vc, ints([]))
    assert torch.equal(kc, before)


def test_append_infinite_and_nan_rows():
    """A NaN makes its own element (16-bit) or row (E4M3) NaN, and no other; an infinity likewise."""
    k = torch.randn(3, 1, 64, device="cuda")
    k[0, 0, 3], k[1, 0, 7] = float("nan"), float("inf")
    (kc, vc), _ = page_tensors(1, 1, 16, 64, F16)
    kie.paged_append(k, k, kc, vc, ints([0, 1, 2]))
    assert torch.isnan(kc[0, 0, 0]).sum() == 1 and torch.isinf(kc[0, 0, 1]).sum() == 1
    (kc, vc), (ks, vs) = page_tensors(1, 1, 16, 64, E4M3)
    kie.paged_append(k, k, kc, vc, ints([0, 1, 2]), k_scale=ks, v_scale=vs)
    value = kc.float() * ks[..., None]
    assert torch.all(torch.isnan(value[0, 0, 0])) and torch.isnan(value[0, 0, 1, 7])
    assert torch.all(torch.isfinite(value[0, 0, 2])) and torch.all(value[0, 0, 3:] == 0)


# ---- attention -----------------------------------------------------------------------------------------------

def batch(lens, hq, hkv, dh, bs, cache, qt, seed=0, order="head", W=None, spread=1.0, dead=float("nan"), spare=3):
    """Pages for the given lengths: what lies behind a sequence's end and in pages of nobody is `dead`."""
    g = gen(seed)
    pages = [oracle.ceil_div(l, bs) for l in lens]
    W = W or max(1, max(pages))
    n = sum(pages) + spare
    (k, v), (ks, vs) = page_tensors(n, hkv, bs, dh, cache, order)
    perm = torch.randperm(n, generator=g, device="cuda").tolist()
    table = [[2 ** 30 - 1 if i % 2 else -5] * W for i in range(len(lens))]
    alive = torch.zeros((n, bs), dtype=torch.bool, device="cuda")
    for b, l in enumerate(lens):
        for j in range(pages[b]):
            p = perm.pop()
            table[b][j] = p
            alive[p, :l - j * bs] = True
    for i, (x, s) in enumerate(((k, ks), (v, vs))):
        rows = torch.randn((n, hkv, bs, dh), generator=g, device="cuda") * (spread if i == 0 else 1.0)
        if cache == E4M3:
            rows = rows * torch.exp(torch.randn((n, hkv, bs, 1), generator=g, device="cuda"))
            codes, scale = oracle.quantise(rows)
            x.view(torch.uint8).copy_(codes.view(torch.uint8))
            s.copy_(scale)
            s.masked_fill_(~alive[:, None], dead)
            x.view(torch.uint8).masked_fill_(~alive[:, None, :, None], 0x7F if dead != 0 else 0)
        else:
            x.copy_(rows)
            x.masked_fill_(~alive[:, None, :, None], dead)
    q = torch.randn((len(lens), hq, dh), generator=g, device="cuda").to(qt)
    return q, k, v, ints(table), ints(lens), ks, vs


def check_attention(q, k, v, table, lens, ks, vs, scale=None, window=0, **kw):
    out, lse = kie.paged_attention(q, k, v, table, lens, scale=scale, window=window, k_scale=ks, v_scale=vs,
                                   return_lse=True, **kw)
    ref = oracle.attention(q, k, v, table, lens, q.shape[-1] ** -0.5 if scale is None else scale, window, ks, vs)
    tol_out, tol_lse = oracle.attention_bounds(q, k.dtype, *ref)
    assert not torch.isnan(out).any()
    err = (out.double() - ref[0]).abs()
    assert torch.all(err <= tol_out), float((err / tol_out).max())
    empty = ref[4] == 0
    assert torch.all(out[empty] == 0) and torch.all(lse[empty] == -torch.inf)
    err = (lse.double() - ref[1]).abs()[~empty]
    assert torch.all(err <= tol_lse[~empty]), float((err / tol_lse[~empty]).max())
    return out, lse


TYPES = [(F16, F16), (F16, F32), (BF16, BF16), (E4M3, F32), (E4M3, F16), (E4M3, BF16)]
HEADS = [(20, 4, 128), (4, 4, 64), (8, 1, 128), (6, 2, 64), (7, 1, 64), (3, 3, 128)]
EDGES = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 0, 200, 255, 256, 257, 1000]


@pytest.mark.parametrize("cache,qt", TYPES)
@pytest.mark.parametrize("hq,hkv,dh", HEADS)
@pytest.mark.parametrize("bs", [16, 64])
def test_attention_edges(cache, qt, hq, hkv, dh, bs):
    check_attention(*batch(EDGES, hq, hkv, dh, bs, cache, qt, seed=hq + dh))


@pytest.mark.parametrize("cache,qt", TYPES)
@pytest.mark.parametrize("length", [1, 16, 100, 1153, 5000])
def test_attention_of_one_sequence(cache, qt, length):
    check_attention(*batch([length], 20, 4, 128, 16, cache, qt, seed=length))


@pytest.mark.parametrize("cache,qt", TYPES)
@pytest.mark.parametrize("bs", [48, 112, 1024])
def test_attention_of_a_ragged_batch(cache, qt, bs):
    rng = np.random.RandomState(bs)
    lens = np.exp(rng.uniform(0, np.log(3000), 37)).astype(int).tolist()
    check_attention(*batch(lens, 8, 2, 64 if bs == 48 else 128, bs, cache, qt, seed=bs))


@pytest.mark.parametrize("cache,qt", TYPES)
@pytest.mark.parametrize("window", [1, 2, 16, 33, 64, 500, 5000])
def test_attention_window(cache, qt, window):
    check_attention(*batch([0, 1, 2, 17, 33, 34, 640, 1000, 65], 8, 4, 64, 16, cache, qt, seed=window), window=window)


@pytest.mark.parametrize("cache,qt", [(F16, F32), (BF16, BF16), (E4M3, F16)])
@pytest.mark.parametrize("order", ["position", "pool"])
def test_attention_page_orders(cache, qt, order):
    check_attention(*batch([5, 100, 0, 77, 333], 8, 2, 128, 32, cache, qt, order=order))


@pytest.mark.parametrize("cache,qt", TYPES)
def test_attention_with_large_scores(cache, qt):
    """Scores of a few hundred, one position far above the rest, and a scale of 1."""
    q, k, *rest = batch([300, 40, 1], 4, 2, 64, 16, cache, qt, spread=8.0)
    check_attention(q, k, *rest, scale=1.0)


def test_attention_scales_far_apart():
    """E4M3 rows of very different size: values near 1e-6 next to none larger, and rows of zeros."""
    q, k, v, table, lens, ks, vs = batch([300, 90], 8, 2, 128, 16, E4M3, F32, dead=0.0)
    vs *= 1e-6
    check_attention(q, k, v, table, lens, ks, vs)
    vs[:, :, ::2] *= 1e6
    check_attention(q, k, v, table, lens, ks, vs)
    vs[:, :, ::3] = 2.0 ** -126
    v.view(torch.uint8)[:, :, ::3] = 0
    check_attention(q, k, v, table, lens, ks, vs)


@pytest.mark.parametrize("factor", [1e-6, 1.0, 3e5])
def test_attention_of_queries_of_any_size(factor):
    """fp32 queries far from 1 (the scale brings the scores back)."""
    q, *rest = batch([130, 7], 8, 2, 128, 16, F16, F32)
    check_attention(q * factor, *rest, scale=0.1 / factor)
    q, *rest = batch([130, 7], 8, 2, 128, 16, E4M3, BF16)
    check_attention((q.float() * factor).to(BF16), *rest, scale=0.03 / factor)


def test_attention_leaves_out_bad_pages_and_cuts_long_lengths():
    q, k, v, table, lens, ks, vs = batch([100, 100, 64], 4, 2, 64, 16, F16, F16)
    table[0, 2], table[1, 0], table[1, 6] = k.shape[0], -1, 2 ** 31 - 1
    table[2] = -1  # nothing is left
    check_attention(q, k, v, table, lens, ks, vs)
    lens[0], lens[2] = 2 ** 31 - 1, -3
    k.masked_fill_(torch.isnan(k), 0.5), v.masked_fill_(torch.isnan(v), 0.25)  # the cut lengths reach all of the table
    check_attention(q, k, v, table, lens, ks, vs)


def test_attention_nan_and_infinity_stay_with_their_sequence():
    q, k, v, table, lens, ks, vs = batch([70, 70, 70], 4, 2, 64, 16, F16, F16)
    clean = kie.paged_attention(q, k, v, table, lens)
    v[table[1, 1].item(), 0, 3, 5] = float("nan")
    k[table[2, 0].item(), 1, 0] = float("inf")
    out = kie.paged_attention(q, k, v, table, lens)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[1, 2:], clean[1, 2:]) and torch.equal(out[2, :2], clean[2, :2])
    assert torch.all(torch.isnan(out[1, :2, 5])) and not torch.isnan(out[1, :2, :5]).any()
    assert torch.isnan(out[2, 2:]).any()


@pytest.mark.parametrize("qt", [F16, F32])
def test_attention_strided_query_and_output(qt):
    q, k, v, table, lens, ks, vs = batch([70, 3, 150], 4, 2, 64, 16, F16, qt)
    wide = torch.zeros(3 * (4 * 64 + 7) + 1, dtype=qt, device="cuda")[1:].view(3, -1)
    view = wide[:, :256].unflatten(1, (4, 64))
    view.copy_(q)
    room = torch.full((4, 3, 65), 9.0, dtype=qt, device="cuda").transpose(0, 1)[..., :64]
    want = kie.paged_attention(q, k, v, table, lens)
    assert kie.paged_attention(view, k, v, table, lens, out=room) is room
    assert torch.equal(room, want)
    flipped = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(kie.paged_attention(flipped, k, v, table, lens), want)


def test_attention_of_nothing():
    q, k, v, table, lens, ks, vs = batch([5], 4, 2, 64, 16, F16, F16)
    out, lse = kie.paged_attention(q[:0], k, v, table[:0], lens[:0], return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    zero = kie.paged_attention(q, k, v, table, ints([0]))
    assert torch.all(zero == 0)


def test_attention_past_32_bit_offsets():
    """Pages 2^28 elements apart: offsets of 2^31 elements and more."""
    q, k, v, table, lens, ks, vs = batch([100, 20], 4, 2, 64, 16, F16, F32, spare=1)
    n = k.shape[0]
    big = torch.zeros((n - 1) * 2 ** 28 + 2 ** 16, dtype=F16, device="cuda")
    far = big.as_strided(k.shape, (2 ** 28, 16 * 64, 64, 1))
    far_v = big.as_strided(k.shape, (2 ** 28, 16 * 64, 64, 1), 2 ** 15)
    far.copy_(k), far_v.copy_(v)
    assert torch.equal(kie.paged_attention(q, far, far_v, table, lens), kie.paged_attention(q, k, v, table, lens))
    slots = ints([(n - 1) * 16 + 3, 5])
    rows = torch.randn(2, 2, 64, device="cuda")
    kie.paged_append(rows, rows, far, far_v, slots)
    assert torch.equal(far[n - 1, :, 3], rows[0].half()) and torch.equal(far_v[0, :, 5], rows[1].half())


def test_attention_gives_the_same_bits_again():
    args = batch([700, 33, 2000, 1], 20, 4, 128, 16, F16, F32)
    first = kie.paged_attention(*args[:5])
    for _ in range(5):
        assert torch.equal(kie.paged_attention(*args[:5]), first)


def test_two_streams_and_two_graphs_share_nothing():
    """The same call in flight on two streams, and captured into two graphs that are replayed over one another."""
    a, b = (batch(l, 20, 4, 128, 16, F16, F32, seed=i) for i, l in enumerate(([3000, 5], [64, 2500, 700])))
    want = [kie.paged_attention(*x[:5]) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (s, x) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(s):
                got[i].append(kie.paged_attention(*x[:5]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    graphs, outs = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kie.paged_attention(*x[:5]))
        graphs.append(g)
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_a_captured_step_follows_its_inputs():
    """extend, append and attention captured once and replayed: each replay takes the tables and lengths of the last."""
    from synth.configs import MOE_TINY as M
    n, bs = 6, 16
    cache = kie.PagedCache(M, n_blocks=40, block_size=bs, max_seqs=n, max_blocks=4)
    one = ints([1, 1, 0, 1, 1, 1])
    q, k, v = (torch.randn(n, h, M.head_dim, device="cuda") for h in (M.n_heads, M.n_kv_heads, M.n_kv_heads))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step = cache.extend(one, n)
        rq = cache.append(0, k, v, step, q=q)
        out = cache.attention(0, rq)
    want_lens = np.zeros(n, dtype=int)
    for t in range(20):
        g.replay()
        want_lens += np.array(one.tolist())
        assert cache.lens.tolist() == want_lens.tolist()
    ref = oracle.attention(rq, cache.k[0], cache.v[0], cache.block_table, cache.lens, M.head_dim ** -0.5)
    assert torch.all((out.double() - ref[0]).abs() <= oracle.attention_bounds(rq, F16, *ref)[0])
    assert cache.n_free.tolist() == [40 - 5 * 2]


def test_the_first_call_of_a_process_may_be_captured():
    """No kernel has run, or been loaded, when the operators are captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, persistent_monokernel_decode_gb300 as kie
from synth.configs import MOE_TINY as M
n = 3
for dtype in (torch.float16, torch.float8_e4m3fn):
    cache = kie.PagedCache(M, 9, 16, n, 4, dtype=dtype)
    one = torch.ones(n, dtype=torch.int32, device="cuda")
    q, k, v = (torch.ones(n, h, M.head_dim, device="cuda") for h in (M.n_heads, M.n_kv_heads, M.n_kv_heads))
    done = torch.ones(n, dtype=torch.bool, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step = cache.extend(one, n)
        out = cache.attention(0, cache.append(0, k, v, step, q=q))
        cache.release(done)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert cache.n_free.tolist() == [9] and cache.lens.tolist() == [0] * n
        assert torch.allclose(out, torch.ones_like(out), atol=1e-6), out
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def raw_attention(q, k, v, table, lens, workspace):
    """The C entry point itself, with a workspace of the caller's."""
    import ctypes
    out = torch.empty_like(q)
    a = kie.KiePagedAttentionArgs(q=q.data_ptr(), out=out.data_ptr(), block_table=table.data_ptr(), lens=lens.data_ptr(),
                                  table_stride=table.stride(0), workspace=workspace.data_ptr(),
                                  workspace_bytes=workspace.numel(), scale=q.shape[-1] ** -0.5, n_seqs=q.shape[0],
                                  n_heads=q.shape[1], max_blocks=table.shape[1], q_dtype={F16: 0, BF16: 1, F32: 2}[q.dtype])
    a.q_stride[:], a.out_stride[:] = q.stride()[:2], out.stride()[:2]
    p = a.pages
    p.k, p.v, p.dtype = k.data_ptr(), v.data_ptr(), {F16: 0, BF16: 1}[k.dtype]
    p.k_stride[:], p.v_stride[:] = k.stride()[:3], v.stride()[:3]
    p.n_blocks, p.n_kv_heads, p.block_size, p.head_dim = k.shape
    rc = kie.lib().kie_paged_attention(ctypes.byref(a), torch.cuda.current_stream().cuda_stream)
    assert rc == 0, kie.lib().kie_paged_last_error()
    return out


@pytest.mark.parametrize("qt", [F16, F32])
def test_the_workspace_may_hold_anything(qt):
    """Zeros, ones, noise, and what another batch's call left: the results are the same bits."""
    a, b = (batch(l, 20, 4, 128, 16, F16, qt, seed=i) for i, l in enumerate(([9000, 3, 700], [2000, 2500, 64, 1, 3000])))
    want = [kie.paged_attention(*x[:5]) for x in (a, b)]
    size = kie.lib().kie_paged_attention_workspace(20, 4, 128)
    noise = torch.randint(0, 256, (size,), device="cuda", dtype=torch.uint8, generator=gen(5))
    counts = torch.randint(0, 30, (size // 8,), device="cuda", generator=gen(6)).view(torch.uint8)  # small whole numbers
    for fill in (torch.zeros_like(noise), torch.full_like(noise, 255), noise, counts):
        ws = fill.clone() if fill.numel() == size else torch.cat([fill, fill[:size - fill.numel()]])
        for _ in range(3):
            assert torch.equal(raw_attention(*a[:5], ws), want[0])
            assert torch.equal(raw_attention(*b[:5], ws), want[1])


@pytest.mark.parametrize("cache,qt", [(F16, F32), (F16, F16), (E4M3, F16)])
def test_attention_of_one_long_sequence(cache, qt):
    """Pieces of one item on more blocks than are joined at once."""
    check_attention(*batch([40007], 8, 1, 128, 64, cache, qt, seed=2))


@pytest.mark.parametrize("n", [700, 5000])
def test_attention_of_many_short_sequences(n):
    lens = np.random.RandomState(n).randint(0, 4, n).tolist()
    check_attention(*batch(lens, 4, 2, 64, 16, F16, F16, seed=n))


def test_attention_of_random_batches():
    rng = np.random.RandomState(1)
    for i in range(12):
        lens = np.exp(rng.uniform(0, np.log(4000), rng.randint(1, 12))).astype(int).tolist()
        cache, qt = TYPES[i % len(TYPES)]
        hq, hkv, dh = HEADS[rng.randint(len(HEADS))]
        check_attention(*batch(lens, hq, hkv, dh, int(rng.choice([16, 32, 80, 256])), cache, qt, seed=i))


def test_attention_in_place_of_the_query():
    q, k, v, table, lens, ks, vs = batch([3000, 20, 700, 0], 20, 4, 128, 16, F16, F16)
    want = kie.paged_attention(q, k, v, table, lens)
    assert kie.paged_attention(q, k, v, table, lens, out=q) is q
    assert torch.equal(q, want)


def test_a_replayed_graph_follows_the_lengths():
    """One captured call replayed with other lengths each time, so that other blocks share other items."""
    q, k, v, table, lens, ks, vs = batch([4000, 4000, 4000], 20, 4, 128, 16, F16, F32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kie.paged_attention(q, k, v, table, lens)
    rng = np.random.RandomState(3)
    for _ in range(15):
        lens.copy_(ints(rng.randint(0, 4001, 3).tolist()))
        want = kie.paged_attention(q, k, v, table, lens)
        g.replay()
        assert torch.equal(out, want)


# ---- refusals of the binding ---------------------------------------------------------------------------------

def test_the_binding_refuses():
    q, k, v, table, lens, _, _ = batch([20, 3], 4, 2, 64, 16, F16, F16)
    for bad in (dict(q=q.float().double()), dict(q=q.bfloat16()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q.cpu()),
                dict(lens=lens.long()), dict(lens=lens[:1]), dict(table=table[:1]), dict(table=table.t()),
                dict(k=k.float(), v=v.float()), dict(v=v[:1]), dict(k=k.cpu()), dict(k=k.transpose(2, 3), v=v.transpose(2, 3))):
        a = dict(q=q, k=k, v=v, table=table, lens=lens)
        a.update(bad)
        with pytest.raises((ValueError, kie.KieError)):
            kie.paged_attention(a["q"], a["k"], a["v"], a["table"], a["lens"])
    with pytest.raises(ValueError):
        kie.paged_attention(q, k, v, table, lens, k_scale=torch.ones(k.shape[:3], device="cuda"))
    with pytest.raises(ValueError):
        kie.paged_attention(q, k.to(E4M3), v.to(E4M3), table, lens)
    with pytest.raises(kie.KieError):
        kie.paged_attention(q, k, v, table, lens, window=-1)
    rows = torch.zeros(2, 2, 64, device="cuda")
    for bad in (dict(slots=ints([1])), dict(slots=ints([1, 2]).long()), dict(rope=torch.zeros(4, 32, 2, device="cuda")),
                dict(v=rows.half()), dict(k=rows[:, :1], v=rows[:, :1]), dict(q=rows.half())):
        a = dict(k=rows, v=rows, slots=ints([1, 2]))
        a.update(bad)
        with pytest.raises(ValueError):
            kie.paged_append(a.pop("k"), a.pop("v"), k, v, a.pop("slots"), **a)
    with pytest.raises(ValueError):
        kie.paged_extend(lens, lens, table.long(), lens, lens[:1], 16, 4)
    with pytest.raises(kie.KieError):
        kie.paged_extend(lens, lens, table, lens, lens[:1], 17, 4)
    with pytest.raises(ValueError):
        kie.paged_release(lens, lens, table, lens, lens[:1], 16)


# ---- the four together: a batched decode ---------------------------------------------------------------------

def f16(a):
    return torch.from_numpy(np.asarray(a, dtype=np.uint16).view(np.float16).copy()).cuda().float()


def batched_step(M, w, cache, step, tokens, n_rows):
    """One token per sequence through a dense model: plain fp32 projections around the paged operators. Row b of a
    step is sequence b."""
    def rms(x, gain):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + M.rms_eps) * gain

    dh = M.head_dim
    x = w["embed"][tokens.long()]
    for l, lay in enumerate(w["layers"]):
        u = rms(x, lay["attn_norm"])
        q, k, v = ((u @ lay[n].T).view(n_rows, -1, dh) for n in ("wq", "wk", "wv"))
        q = cache.append(l, k, v, step, q=q)
        o = cache.attention(l, q)
        x = x + o.reshape(n_rows, -1) @ lay["wo"].T
        u = rms(x, lay["ffn_norm"])
        x = x + (torch.nn.functional.silu(u @ lay["w_gate"].T) * (u @ lay["w_up"].T)) @ lay["w_down"].T
    return rms(x, w["final_norm"]) @ w["lm_head"].T


def test_a_batched_decode_matches_the_decoder():
    """Three prompts prefilled by a Decoder each, loaded into pages, then decoded together for 20 steps: every
    sequence's logits within the decoder's own logit tolerance of the Decoder running it alone; then one sequence
    ends, its pages go back, and a new prompt takes them."""
    import synth
    from synth.configs import TINY as M
    weights = synth.model_weights(M)
    w = {k: f16(weights[k]) for k in ("embed", "lm_head", "final_norm")}
    w["layers"] = [{k: f16(v) for k, v in lay.items()} for lay in weights["layers"]]
    prompts = [synth.tokens(s, n, M.vocab) for s, n in ((11, 16), (12, 1), (13, 37))]
    decs = [kie.Decoder(M, weights, max_seq=96) for _ in prompts]
    cache = kie.PagedCache(M, n_blocks=13, block_size=16, max_seqs=3, max_blocks=6)
    for d, p in zip(decs, prompts):
        d.prefill(p)
    step = cache.extend(ints([len(p) for p in prompts]), sum(len(p) for p in prompts))
    for d, at in zip(decs, (0, 16, 17)):
        cache.load(d, step, at)
    current = [d.logits() for d in decs]

    def run(steps):
        for _ in range(steps):
            toks = [int(np.argmax(c)) for c in current]
            logits = batched_step(M, w, cache, cache.extend(ints([1, 1, 1]), 3), ints(toks), 3).cpu().numpy()
            for b, d in enumerate(decs):
                current[b] = d.decode_forced(np.array([toks[b]], dtype=np.int32))[1][0]
                assert np.max(np.abs(logits[b] - current[b])) <= 2e-2, b

    run(20)
    assert cache.lens.tolist() == [36, 21, 57] and cache.n_free.tolist() == [13 - 3 - 2 - 4]
    cache.release(torch.tensor([False, False, True], device="cuda"))
    assert cache.lens.tolist() == [36, 21, 0] and cache.n_free.tolist() == [8]
    decs[2].reset()
    prompt = synth.tokens(14, 70, M.vocab)
    decs[2].prefill(prompt)
    step = cache.extend(ints([0, 0, 70]), 70)
    assert step.admitted.tolist() == [True] * 3
    cache.load(decs[2], step)
    current[2] = decs[2].logits()
    run(5)
    for d in decs:
        d.close()


def test_load_from_a_decoder_on_another_stream():
    """The pages hold the prompt although the decoder, on its own stream, takes another one right after."""
    import synth
    from synth.configs import TINY as M
    dec = kie.Decoder(M, synth.model_weights(M), max_seq=64, stream=torch.cuda.Stream())
    cache = kie.PagedCache(M, n_blocks=8, block_size=16, max_seqs=2, max_blocks=4)
    got = []
    for s in (21, 22):
        dec.reset()
        dec.prefill(synth.tokens(s, 50, M.vocab))
        kv = dec._kvbuf.view(F16)[:2 * M.n_layers * M.n_kv_heads * 64 * M.head_dim].view(M.n_layers, 2, M.n_kv_heads, 64, -1)
        got.append(kv[:, :, :, :50].clone())
        step = cache.extend(ints([50, 0] if s == 21 else [0, 50]), 50)
        cache.load(dec, step)
    for b in range(2):
        at = torch.arange(50, device="cuda")
        page = cache.block_table[b].long()[at // 16]
        half = M.head_dim // 2
        for l in range(M.n_layers):
            k, v = (x[l][page, :, at % 16].transpose(0, 1) for x in (cache.k, cache.v))
            assert torch.equal(v, got[b][l, 1])
            assert torch.equal(k[..., :half], got[b][l, 0][..., 0::2]) and torch.equal(k[..., half:], got[b][l, 0][..., 1::2])
    with pytest.raises(ValueError):
        cache.load(dec, step, first_row=1)
    dec.close()
