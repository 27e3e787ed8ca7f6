"""Decoder.score: log probabilities of a given continuation against fp64 on the decoder's own logits, across the cuts of its
launches, and where it leaves the sequence."""
import numpy as np
import pytest
import torch

import persistent_monokernel_decode_gb300 as kie
import shared_oracle as oracle
import synth
from synth.configs import MOE_TINY, TINY

pytestmark = pytest.mark.gpu

PROMPT = 9
MAX_SEQ = PROMPT + 140


@pytest.fixture(scope="module", params=["tiny", "moe_tiny"])
def decoder(request):
    kie.build()
    cfg, w = (TINY, synth.model_weights(TINY)) if request.param == "tiny" else (MOE_TINY, synth.moe_weights(MOE_TINY))
    dec = kie.Decoder(cfg, w, max_seq=MAX_SEQ)
    yield cfg, dec
    dec.close()


def begin(cfg, dec):
    dec.reset()
    dec.prefill(synth.tokens(cfg.seed, PROMPT, cfg.vocab))


def check(cfg, dec, tokens, cuts, top):
    """Scores of the tokens, taken in pieces that end at `cuts`. How many rows a launch has decides how a row's sums are
    split, so that pieces have to agree with fp64, not bit by bit with each other."""
    n = len(tokens)
    begin(cfg, dec)
    first = dec.logits()
    _, logits = dec.decode_forced(tokens)
    rows = torch.from_numpy(np.concatenate([first[None], logits[:-1]]))
    begin(cfg, dec)
    parts = [dec.score(tokens[a:b], top=top) for a, b in zip((0, *cuts), (*cuts, n))]
    assert dec.position == PROMPT + n and np.array_equal(dec.logits(), logits[-1])
    got = kie.TokenLogprobs(*(np.concatenate([p[k] for p in parts]) for k in range(4)))
    lp, h, ids, top_lp = oracle.logprobs(rows, torch.from_numpy(tokens), top)
    lse, part, entropy = oracle.logprobs_bounds(rows)
    assert got.top_ids.shape == got.top_logprobs.shape == (n, top) and np.array_equal(got.top_ids, ids.numpy())
    for a, b, tol in ((got.logprob, lp, lse + part * lp.abs()), (got.entropy, h, entropy),
                      (got.top_logprobs, top_lp, lse[:, None] + part * top_lp.abs())):
        assert torch.all((torch.from_numpy(a).double() - b).abs() <= tol)


@pytest.mark.parametrize("n,top", [(1, 0), (1, 32), (2, 1), (63, 5), (64, 20), (65, 3), (130, 0), (140, 32)])
def test_scores_are_those_of_the_logits(decoder, n, top):
    check(*decoder, synth.tokens(decoder[0].seed + 1, n, decoder[0].vocab), (), top)


def test_scores_in_pieces(decoder):
    check(*decoder, synth.tokens(decoder[0].seed + 2, 100, decoder[0].vocab), (1, 31, 96), 4)


def test_greedy_tokens_score_as_the_most_probable(decoder):
    cfg, dec = decoder
    begin(cfg, dec)
    tokens = dec.decode(40)
    begin(cfg, dec)
    got = dec.score(tokens, top=1)
    assert np.array_equal(got.top_ids[:, 0], tokens) and np.array_equal(got.top_logprobs[:, 0], got.logprob)


def test_refusals(decoder):
    cfg, dec = decoder
    dec.reset()
    with pytest.raises(kie.KieError) as e:
        dec.score([1])
    assert e.value.code == kie.KIE_ERR_INVALID
    begin(cfg, dec)
    for tokens, top, code in (([], 0, kie.KIE_ERR_INVALID), ([-1], 0, kie.KIE_ERR_INVALID), ([cfg.vocab], 0, kie.KIE_ERR_INVALID),
                              ([1], 33, kie.KIE_ERR_INVALID), ([1], -1, kie.KIE_ERR_INVALID),
                              ([1] * (MAX_SEQ - PROMPT + 1), 0, kie.KIE_ERR_CAPACITY)):
        with pytest.raises(kie.KieError) as e:
            dec.score(tokens, top=top)
        assert e.value.code == code and dec.position == PROMPT
