"""Paged-cache operators, host side (no GPU): refusals of calls that would pair rows with wrong sequences or write an
output over itself, and the build's bookkeeping."""
import pytest

import persistent_monokernel_decode_gb300 as kie
from test_paged_host import SOME, append_args, attention_args, refused


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


@pytest.mark.parametrize("change,word", [
    (dict(seqs=SOME, lens=None), "together"), (dict(positions=SOME, lens=None), "together"),
    (dict(seqs=SOME, positions=SOME), "either"), (dict(lens=None), "either"),
    (dict(seqs=SOME, positions=SOME, lens=None, n_table=-1), "n_table"),
    (dict(seqs=SOME, positions=SOME, lens=None, n_table=2, table_stride=3), "table_stride"),
    (dict(seqs=SOME + 2, positions=SOME, lens=None), "aligned"), (dict(seqs=SOME, positions=SOME + 1, lens=None), "aligned")])
def test_attention_of_rows_refuses(change, word):
    a = attention_args()
    for k, v in change.items():
        setattr(a, k, v)
    refused("kie_paged_attention", a, word)


@pytest.mark.parametrize("out_stride", [(512, 64), (256, 128), (64, 256)])
def test_attention_in_place_needs_equal_strides(out_stride):
    """Another block would read a query that this one has overwritten."""
    a = attention_args()
    a.q_stride[:], a.out_stride[:] = (256, 64), out_stride
    refused("kie_paged_attention", a, "strides")
