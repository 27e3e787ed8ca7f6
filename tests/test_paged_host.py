"""Paged-cache operators, host side (no GPU): argument checks of the C entry points refuse before anything is
enqueued, and the plain implementations that the GPU tests compare with hold on cases worked by hand."""
import ctypes
import math

import pytest
import torch

import paged_oracle as oracle
import persistent_monokernel_decode_gb300 as kie

SOME = 4096  # an aligned address that is never read: every call here is refused by the host


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


def pages(dtype=0):
    p = kie.KiePages(k=SOME, v=SOME, k_scale=SOME, v_scale=SOME, n_blocks=8, n_kv_heads=2, block_size=16, head_dim=64,
                     dtype=dtype)
    for s in (p.k_stride, p.v_stride):
        s[:] = (2 * 16 * 64, 16 * 64, 64)
    return p


def refused(fn, args, word):
    assert getattr(kie.lib(), fn)(ctypes.byref(args), None) == kie.KIE_ERR_INVALID
    assert word in kie.lib().kie_paged_last_error().decode()


def extend_args(**change):
    a = kie.KiePagedExtendArgs(*[SOME] * 5, 4, *[SOME + 64 * i for i in range(1, 8)], 3, 4, 16, 5, 8)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,word", [
    (dict(n_seqs=-1), "n_seqs"), (dict(n_rows=-1), "n_rows"), (dict(max_blocks=0), "max_blocks"),
    (dict(block_size=0), "block_size"), (dict(block_size=24), "block_size"), (dict(max_blocks=1 << 27), "2^31"),
    (dict(n_free=None), "n_free"), (dict(lens=None), "requests"), (dict(slots=None), "rows"),
    (dict(free_blocks=None), "free_blocks"), (dict(table_stride=3), "table_stride"), (dict(lens_out=SOME), "must not"),
    (dict(n_free_out=SOME), "must not"), (dict(free_capacity=-1), "free_capacity"), (dict(slots=SOME + 2), "aligned")])
def test_extend_refuses(change, word):
    refused("kie_paged_extend", extend_args(**change), word)


@pytest.mark.parametrize("change,word", [
    (dict(n_seqs=-1), "n_seqs"), (dict(block_size=8), "block_size"), (dict(done=None), "requests"),
    (dict(n_free_out=SOME), "must not"), (dict(lens_out=SOME), "must not"), (dict(table_stride=1), "table_stride"),
    (dict(block_table=SOME + 1), "aligned")])
def test_release_refuses(change, word):
    a = kie.KiePagedReleaseArgs(SOME, SOME, SOME, SOME, 4, SOME, SOME + 64, SOME + 128, 3, 4, 16, 8)
    for k, v in change.items():
        setattr(a, k, v)
    refused("kie_paged_release", a, word)


def append_args(dtype=0):
    a = kie.KiePagedAppendArgs(pages=pages(dtype), k=SOME, v=SOME, q=SOME, q_out=SOME, slots=SOME, positions=SOME,
                               rope=SOME, n_rows=4, n_heads=4, n_pos=32, x_dtype=0)
    return a


BAD_PAGES = [(dict(n_blocks=0), "n_blocks"), (dict(head_dim=96), "head_dim"), (dict(block_size=40), "block_size"),
             (dict(n_blocks=1 << 27), "2^31"), (dict(dtype=2), "KIE_F16"), (dict(k=None), "NULL"),
             (dict(v=SOME + 8), "aligned"), (dict(n_kv_heads=0), "n_kv_heads")]


@pytest.mark.parametrize("change,word", BAD_PAGES)
@pytest.mark.parametrize("fn", ["kie_paged_append", "kie_paged_attention"])
def test_bad_pages_are_refused(fn, change, word):
    a = append_args() if fn == "kie_paged_append" else attention_args()
    for k, v in change.items():
        setattr(a.pages, k, v)
    refused(fn, a, word)


@pytest.mark.parametrize("fn", ["kie_paged_append", "kie_paged_attention"])
def test_page_strides_and_scales_are_checked(fn):
    make = append_args if fn == "kie_paged_append" else attention_args
    a = make()
    a.pages.v_stride[2] = 68
    refused(fn, a, "strides")
    a = make(3)
    a.pages.k_scale = None
    refused(fn, a, "scale")


@pytest.mark.parametrize("change,word", [
    (dict(n_rows=-1), "n_rows"), (dict(x_dtype=3), "KIE_F32"), (dict(q_out=None), "q_out"), (dict(n_heads=0), "n_heads"),
    (dict(slots=None), "slots"), (dict(positions=None), "positions"), (dict(n_pos=0), "n_pos"),
    (dict(rope=SOME + 4), "aligned"), (dict(n_rows=1 << 27), "2^28"), (dict(slots=SOME + 2), "aligned"),
    (dict(k=SOME + 1), "aligned")])
def test_append_refuses(change, word):
    a = append_args()
    for k, v in change.items():
        setattr(a, k, v)
    refused("kie_paged_append", a, word)


def test_append_in_place_needs_equal_strides():
    a = append_args()
    a.q_stride[:], a.q_out_stride[:] = (256, 64), (512, 64)
    refused("kie_paged_append", a, "strides")


def attention_args(dtype=0):
    return kie.KiePagedAttentionArgs(pages=pages(dtype), q=SOME, out=SOME, block_table=SOME, lens=SOME, table_stride=4,
                                     workspace=SOME, workspace_bytes=0, scale=1.0, n_seqs=2, n_heads=4, max_blocks=4)


@pytest.mark.parametrize("change,word", [
    (dict(n_seqs=-1), "n_seqs"), (dict(window=-1), "window"), (dict(max_blocks=0), "max_blocks"),
    (dict(max_blocks=1 << 27), "2^30"), (dict(n_heads=3), "multiple"), (dict(n_heads=18), "more than 8"),
    (dict(q_dtype=3), "KIE_F32"), (dict(q_dtype=1), "F16 pages"), (dict(scale=float("nan")), "finite"),
    (dict(scale=float("inf")), "finite"), (dict(q=None), "NULL"), (dict(lens=None), "NULL"),
    (dict(table_stride=3), "table_stride"), (dict(n_seqs=1 << 30), "2^31"), (dict(lens=SOME + 2), "aligned"),
    (dict(out=SOME + 1), "aligned"), (dict(n_seqs=1 << 20, max_blocks=1 << 26, table_stride=1 << 26), "2^45")])
def test_attention_refuses(change, word):
    a = attention_args()
    for k, v in change.items():
        setattr(a, k, v)
    refused("kie_paged_attention", a, word)


@pytest.mark.parametrize("q_dtype", [0, 2])
def test_bf16_pages_take_bf16_queries_only(q_dtype):
    a = attention_args(1)
    a.q_dtype = q_dtype
    refused("kie_paged_attention", a, "BF16")


@pytest.mark.parametrize("fn", ["kie_paged_extend", "kie_paged_release", "kie_paged_append", "kie_paged_attention"])
def test_null_arguments_are_refused(fn):
    assert getattr(kie.lib(), fn)(None, None) == kie.KIE_ERR_INVALID


@pytest.mark.parametrize("heads", [(0, 1, 64), (4, 0, 64), (5, 2, 64), (18, 2, 64), (4, 2, 96)])
def test_workspace_of_bad_heads_is_zero(heads):
    assert kie.lib().kie_paged_attention_workspace(*heads) == 0


def test_the_oracle_extends_by_hand():
    # bs 16; request 0: 15 + 1 (no page), 1: 16 + 1 (one), 2: 0 + 33 (three), 3: 5 + 0 (none)
    table = [[3, -1, -1], [4, -1, -1], [-1, -1, -1], [5, -1, -1]]
    got = oracle.extend([1, 1, 33, 0], [15, 16, 0, 5], table, [6, 7, 8, 9, 10], 5, 16, 36)
    assert got[0] == [[3, -1, -1], [4, 10, -1], [9, 8, 7], [5, -1, -1]]
    assert got[1] == [16, 17, 33, 5] and got[2] == 1 and got[3] == [True] * 4 and got[4] == [0, 1, 2, 35, 35]
    assert got[5][:3] == [63, 160, 144] and got[5][34] == 7 * 16 and got[5][35] == -1
    assert got[6][:4] == [15, 16, 0, 1] and got[7][1:3] == [1, 2]


def test_the_oracle_refuses_in_order():
    table = [[-1, -1], [-1, -1], [0, -1], [-1, -1]]
    got = oracle.extend([20, 17, 1, 1], [0, 0, 3, 0], table, [1, 2, 3], 3, 16, 39)
    assert got[3] == [True, False, True, False]  # 2 + 2 pages > 3; then one without need; then 5 > 3
    assert got[1] == [20, 0, 4, 0] and got[2] == 1 and got[5][20:37] == [-1] * 17 and got[5][37] == 3


def test_the_oracle_attends_over_equal_keys():
    """Equal keys: the mean of V; lse = s + ln n; an empty sequence: zeros and -inf."""
    k, v = torch.ones(2, 1, 16, 64), torch.randn(2, 1, 16, 64)
    q = torch.ones(2, 1, 64)
    table = torch.tensor([[1, 0], [0, 1]], dtype=torch.int32)
    out, lse, *_ = oracle.attention(q, k, v, table, torch.tensor([18, 0]), 0.5)
    want = torch.cat([v[1, 0], v[0, 0, :2]]).double().mean(0)
    assert torch.allclose(out[0, 0], want) and abs(float(lse[0, 0]) - 32 - math.log(18)) < 1e-12
    assert torch.all(out[1] == 0) and lse[1, 0] == -torch.inf
    out, *_ = oracle.attention(q, k, v, table, torch.tensor([18, 0]), 0.5, window=2)
    assert torch.allclose(out[0, 0], v[0, 0, :2].double().mean(0))


def test_the_oracle_rotates_and_quantises():
    rope = torch.tensor([[[1.0, 0.0]] * 32, [[0.0, 1.0]] * 32])
    x = torch.randn(2, 1, 64)
    y = oracle.rotate(x, rope, torch.tensor([0, 1]))
    assert torch.equal(y[0], x[0])
    assert torch.equal(y[1, 0, :32], -x[1, 0, 32:]) and torch.equal(y[1, 0, 32:], x[1, 0, :32])
    codes, scale = oracle.quantise(torch.stack([x[0, 0], torch.zeros(64)]))
    assert codes[0].float().abs().max() == 448 and scale[1] == 2.0 ** -126 and torch.all(codes[1].float() == 0)
