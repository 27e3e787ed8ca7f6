"""Log probabilities at the limits of their numbers (NaN, a type's lowest value, large distances), in the form of a block to
a row and in that of a cluster."""
import math

import pytest
import torch

import persistent_monokernel_decode_gb300 as kie
from test_gpu_logprobs import check, draw
from test_gpu_paged import BF16, F16, F32, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


# Rows and vocabulary: a block to a row, two blocks, eight; each thread goes through several rounds of its row.
FORMS = [(300, 32000), (63, 32003), (4, 262147)]


def check_ids(got, x, rows, top):
    """The ids of rows with NaN, which count above +inf, the lowest id first."""
    want = torch.sort(x[rows].double(), dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(got.top_ids[rows].long(), want)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("N,V", FORMS)
@pytest.mark.parametrize("top", [0, 1, 20])
def test_a_nan_anywhere_in_a_row(dtype, N, V, top):
    """In the first round of a thread, in those between and in the last, alone and with others or +inf."""
    at = [0, 1, 7, 3000, V // 3, V // 2 + 1, 5 * V // 8, V - 4097, V - 2, V - 1]
    for i in range(0, len(at), 4):
        x, tokens = draw(N, V, dtype, seed=i)
        tokens[:] = torch.arange(N, device="cuda") % V
        few = at[i:i + 4]
        for r, k in enumerate(few):
            x[r, k] = math.nan
            if i:
                x[r, (k + 12345) % V], x[r, (k + 777) % V] = math.nan, math.inf
        rows = list(range(min(len(few), N)))
        got = kie.token_logprobs(x, tokens, top=top)
        assert torch.isnan(got.logprob[rows]).all() and torch.isnan(got.entropy[rows]).all()
        assert torch.isnan(got.top_logprobs[rows]).all()
        check_ids(got, x, rows, top)
        if N > len(few):
            assert not torch.isnan(got.logprob[len(few):]).any() and not torch.isnan(got.entropy[len(few):]).any()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("N,V", [(5, 10), (5, 1000), (300, 4097), *FORMS])
def test_rows_at_the_lowest_value(dtype, N, V):
    """Masked throughout, masked and ruled out, one token a little above the mask; with and without a piece cut off at either
    end of a row."""
    lowest = torch.finfo(dtype).min
    for at, extra in ((0, 0), (3, 5)):
        wide = torch.zeros((N, V + extra), device="cuda", dtype=dtype)
        x = wide[:, at:at + V]
        x[:] = draw(N, V, dtype)[0]
        near = float(torch.tensor(lowest, dtype=torch.float64) * (1 - torch.finfo(dtype).eps))
        x[0] = lowest
        x[1], x[1, :10] = -math.inf, lowest
        x[2], x[2, V // 2] = lowest, near
        x[3], x[3, ::2] = lowest, -math.inf
        for top in (0, min(V, 9)):
            check(x, ints([1, 1, V // 2, 1] + [0] * (N - 4)), top)


def test_fp16_rows_next_to_the_lowest_value():
    """The largest logit steps of 32 above the lowest: what is at the lowest then counts in full, hardly, or not."""
    x = torch.full((12, 1001), -65504.0, device="cuda").half()
    for r in range(12):
        x[r, r::50] = -65504.0 + 32 * r
    x[6:, 500:] = -math.inf
    check(x, ints([0, 1] * 6), 20)
    check(x[:2].repeat(200, 1), ints([0, 1] * 200), 20)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,V", [(300, 32000), (300, 262147), (4, 1000003)])
@pytest.mark.parametrize("mask", [-9e36, -5e36, -1.5e36, -1e30, -3e38])
def test_rows_that_begin_far_below_the_rest(dtype, N, V, mask):
    """A thread whose first rounds hold a large negative mask, and a few ordinary logits behind: everywhere at the row's
    beginning, and at that of each eighth."""
    x, tokens = draw(N, V, dtype)
    i = torch.arange(V, device="cuda")
    x[0::2, : V * 7 // 8] = mask
    x[1::2, i * 8 % V < V * 9 // 10] = mask
    tokens[:] = V - 1
    check(x, tokens, 4)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("N,V", [(5, 600), (300, 600), (300, 3000), *FORMS])
def test_rows_of_nan_and_a_nan_ahead_of_ties(dtype, N, V):
    """More candidates than a row's list holds, with a NaN at id 0 among them."""
    x, tokens = torch.zeros((N, V), device="cuda", dtype=dtype), ints([0] * N)
    x[0], x[1, 0], x[2, [0, V - 1]], x[3, 0], x[3, 1:] = math.nan, math.nan, math.nan, math.nan, -math.inf
    for top in (1, 8, 32):
        got = kie.token_logprobs(x, tokens, top=top)
        check_ids(got, x, list(range(4)), top)
        assert torch.isnan(got.logprob[:4]).all() and torch.isnan(got.top_logprobs[:4]).all()
        check(x[4:], tokens[4:], top) if N > 4 else None
