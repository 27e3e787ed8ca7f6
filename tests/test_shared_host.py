"""Operators for sequences that share pages and the log probabilities, host side (no GPU): the C entry points refuse bad
arguments before anything is enqueued, and the plain implementations that the GPU tests compare with hold by hand."""
import math

import pytest
import torch

import persistent_monokernel_decode_gb300 as kie
import shared_oracle as oracle
from test_paged_host import SOME, attention_args, pages, refused


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


def fork_args(**change):
    a = kie.KiePagedForkArgs(parents=SOME, lens=SOME, n_free=SOME, block_table=SOME, table_stride=4, shares=SOME,
                             free_blocks=SOME, lens_out=2 * SOME, n_free_out=2 * SOME, copy_src=SOME, copy_dst=SOME,
                             copy_rows=SOME, ok=SOME, workspace=SOME, workspace_bytes=48, n_seqs=3, max_blocks=4,
                             block_size=16, n_blocks=8, free_capacity=8)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,word", [
    (dict(n_seqs=-1), "n_seqs"), (dict(n_seqs=16385), "MAX_FORK"), (dict(max_blocks=0), "max_blocks"), (dict(n_blocks=0), "n_blocks"),
    (dict(block_size=24), "block_size"), (dict(max_blocks=1 << 27), "2^31"), (dict(shares=None), "shares"),
    (dict(ok=None), "ok"), (dict(parents=None), "requests"), (dict(copy_rows=None), "requests"),
    (dict(free_blocks=None), "free_blocks"), (dict(table_stride=3), "table_stride"), (dict(lens_out=SOME), "must not"),
    (dict(n_free_out=SOME), "must not"), (dict(shares=SOME + 2), "aligned"), (dict(workspace=None), "workspace"),
    (dict(workspace_bytes=47), "workspace"), (dict(workspace=SOME + 8), "workspace"), (dict(free_capacity=-1), "free_capacity")])
def test_fork_refuses(change, word):
    refused("kie_paged_fork", fork_args(**change), word)


@pytest.mark.parametrize("change,word", [(dict(shares=SOME, n_blocks=0), "n_blocks"), (dict(shares=SOME + 1, n_blocks=4), "aligned"),
                                         (dict(shares=SOME, n_blocks=4, n_seqs=16385), "MAX_FORK")])
def test_release_of_shared_pages_refuses(change, word):
    a = kie.KiePagedReleaseArgs(SOME, SOME, SOME, SOME, 4, SOME, SOME + 64, SOME + 128, 3, 4, 16, 8)
    for k, v in change.items():
        setattr(a, k, v)
    refused("kie_paged_release", a, word)


def copy_args(dtype=0, **change):
    a = kie.KiePagedCopyArgs(pages=pages(dtype), k_layer_stride=16384, v_layer_stride=16384, k_scale_layer_stride=256,
                             v_scale_layer_stride=256, src=SOME, dst=SOME, n_pairs=3, n_layers=2)
    for s in (a.pages.k_scale_stride, a.pages.v_scale_stride):
        s[:] = (32, 16, 1)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,word", [
    (dict(n_pairs=-1), "n_pairs"), (dict(n_layers=0), "n_layers"), (dict(n_pairs=1 << 29), "2^30"), (dict(src=None), "NULL"),
    (dict(dst=SOME + 2), "aligned"), (dict(k_layer_stride=0), "layer strides"), (dict(v_layer_stride=4), "layer strides"),
    (dict(v_layer_stride=1 << 40), "layer strides"), (dict(k_scale_layer_stride=-4, pages=pages(3)), "stride")])
def test_copy_refuses(change, word):
    refused("kie_paged_copy", copy_args(**change), word)


@pytest.mark.parametrize("name", ["k_stride", "v_stride", "k_scale_stride", "v_scale_stride"])
def test_copy_refuses_expanded_pages(name):
    a = copy_args(3)
    getattr(a.pages, name)[1] = 0
    refused("kie_paged_copy", a, "stride of 0")


@pytest.mark.parametrize("change,word", [
    (dict(n_seqs=-1), "n_seqs"), (dict(n_blocks=0), "n_blocks"), (dict(block_size=8), "block_size"), (dict(shares=None), "shares"),
    (dict(page_map=None), "page_map"), (dict(src=None), "src"), (dict(lens=None), "requests"),
    (dict(free_blocks=None), "free_blocks"), (dict(table_stride=1), "table_stride"), (dict(n_free_out=SOME), "must not"),
    (dict(page_map=SOME + 2), "aligned")])
def test_compact_refuses(change, word):
    a = kie.KiePagedCompactArgs(lens=SOME, n_free=SOME, block_table=SOME, table_stride=4, shares=SOME, free_blocks=SOME,
                                n_free_out=2 * SOME, src=SOME, dst=SOME, page_map=SOME, n_seqs=3, max_blocks=4, block_size=16,
                                n_blocks=8, free_capacity=8)
    for k, v in change.items():
        setattr(a, k, v)
    refused("kie_paged_compact", a, word)


def strided_attention_args():
    a = attention_args()
    a.out, a.q_stride[:], a.out_stride[:] = 2 * SOME, (256, 64), (256, 64)
    return a


@pytest.mark.parametrize("change,word", [
    (dict(n_groups=-1), "n_groups"), (dict(n_groups=4097), "n_groups"), (dict(group_start=None), "NULL"),
    (dict(prefix_lens=None), "NULL"), (dict(group_start=SOME + 2), "aligned"), (dict(), "workspace")])
def test_prefix_attention_refuses(change, word):
    p = kie.KiePagedPrefixAttentionArgs(a=strided_attention_args(), group_start=SOME, prefix_lens=SOME, n_groups=2)
    for k, v in change.items():
        setattr(p, k, v)
    if word == "workspace":  # needs a device to tell its size: without one that is what is refused
        assert kie.lib().kie_paged_prefix_attention(kie.ctypes.byref(p), None) != kie.KIE_OK
    else:
        refused("kie_paged_prefix_attention", p, word)


@pytest.mark.parametrize("change,word", [
    (dict(window=5), "window"), (dict(n_heads=18), "more than 8"), (dict(q=None), "NULL"), (dict(q_dtype=1), "F16 pages"),
    (dict(scale=float("nan")), "finite")])
def test_prefix_attention_refuses_what_attention_does(change, word):
    p = kie.KiePagedPrefixAttentionArgs(a=strided_attention_args(), group_start=SOME, prefix_lens=SOME, n_groups=2)
    for k, v in change.items():
        setattr(p.a, k, v)
    refused("kie_paged_prefix_attention", p, word)


@pytest.mark.parametrize("heads", [(3, 0, 1, 64), (3, 4, 0, 64), (3, 5, 2, 64), (3, 18, 2, 64), (3, 4, 2, 96), (-1, 4, 2, 64)])
def test_prefix_workspace_of_bad_heads_is_zero(heads):
    assert kie.lib().kie_paged_prefix_attention_workspace(*heads) == 0


@pytest.mark.parametrize("change,word", [
    (dict(n_rows=-1), "n_rows"), (dict(vocab=0), "vocab"), (dict(vocab=1 << 30), "vocab"), (dict(top=33), "top"),
    (dict(top=-1), "top"), (dict(vocab=4, top=5), "top"), (dict(dtype=3), "KIE_F32"), (dict(row_stride=99), "row_stride"),
    (dict(tokens=None), "together"), (dict(logits=None), "NULL"), (dict(top_ids=None), "NULL"), (dict(logits=SOME + 2), "aligned"),
    (dict(entropy=SOME + 2), "aligned")])
def test_logprobs_refuse(change, word):
    a = kie.KieTokenLogprobsArgs(logits=SOME, row_stride=100, tokens=SOME, logprob=SOME, entropy=SOME, top_logprobs=SOME,
                                 top_ids=SOME, n_rows=3, vocab=100, top=5, dtype=2)
    for k, v in change.items():
        setattr(a, k, v)
    refused("kie_token_logprobs", a, word)


@pytest.mark.parametrize("fn", ["kie_paged_fork", "kie_paged_copy", "kie_paged_compact", "kie_paged_prefix_attention",
                                "kie_token_logprobs"])
def test_null_arguments_are_refused(fn):
    assert getattr(kie.lib(), fn)(None, None) == kie.KIE_ERR_INVALID


def test_the_oracle_forks_by_hand():
    # page size 16; row 0 holds 20 positions on pages 3, 4; row 1 holds 32 on 5, 6; row 2 is empty
    table = [[3, 4, -1], [5, 6, -1], [-1, -1, -1]]
    got = oracle.fork([0, 0, 0], [20, 32, 0], table, [0] * 8, [0, 1, 2, 7], 4, 16)
    assert got[0] == [[3, 4, -1], [3, 7, -1], [3, 2, -1]]      # the full page shared, new pages for the open one
    assert got[1] == [0, 0, 0, 2, 0, 0, 0, 0]                  # two more holders of page 3
    assert got[2] == [0, 1, 5, 6] and got[3] == [20, 20, 20] and got[4] == 4 and got[5]  # row 1's pages are free
    assert got[6:] == ([-1, 4, 4], [-1, 7, 2], [0, 4, 4])
    again = oracle.fork([1, -1, 2], [20, 20, 20], got[0], got[1], got[2] + [-1], 4, 16)
    assert again[0][0] == [3, 7, -1] and again[1][3] == 1 and again[4] == 5 and again[2][4] == 4  # row 0's open page is free
    refused_ = oracle.fork([0, 0, 0], [20, 32, 0], table, [0] * 8, [0], 1, 16)
    assert refused_[0] == table and refused_[3] == [20, 32, 0] and not refused_[5] and refused_[4] == 1


def test_the_oracle_compacts_by_hand():
    got = oracle.compact([20, 16], [[7, 2], [5, 9]], [0, 0, 0, 0, 0, 3, 0, 1], [0, 1, 3, 4, 6], 5, 16)
    assert got[4:6] == ([5, 7, -1, -1], [0, 1, -1, -1]) and got[6] == [-1, -1, 2, -1, -1, 0, -1, 1]
    assert got[0] == [[1, 2], [0, 9]] and got[1] == [3, 1, 0, 0, 0, 0, 0, 0] and got[2] == [7, 6, 5, 4, 3] and got[3] == 5


def test_the_oracle_reads_prefixes_through_the_longest_row():
    """Equal keys: the mean of V over the positions, those of the prefix from the longest row's page."""
    k, v = torch.ones(3, 1, 16, 64), torch.randn(3, 1, 16, 64)
    table, q = torch.tensor([[0], [1], [2]], dtype=torch.int32), torch.ones(3, 1, 64)
    out, *_ = oracle.prefix_attention(q, k, v, table, [2, 9, 9], [0, 2, 3], [4, 0], 1.0)
    assert torch.allclose(out[0, 0], v[1, 0, :2].double().mean(0)) and torch.allclose(out[1, 0], v[1, 0, :9].double().mean(0))
    assert torch.allclose(out[2, 0], v[2, 0, :9].double().mean(0))


def test_the_oracle_of_log_probabilities_by_hand():
    x = torch.tensor([[0.0, 0.0, -math.inf, 0.0], [-math.inf] * 4])
    lp, h, ids, top = oracle.logprobs(x, torch.tensor([2, 9]), 2)
    assert lp.tolist() == [-math.inf, 0.0] and abs(float(h[0]) - math.log(3)) < 1e-12 and h[1] == 0
    assert ids.tolist() == [[0, 1], [0, 1]] and torch.all(top[1] == -math.inf) and abs(float(top[0, 0]) + math.log(3)) < 1e-12
