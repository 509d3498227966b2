"""The example's model: training lowers its loss, generation by single steps
sees what the whole sequence sees, and packed documents do not see each other."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture
def lm(gpu):
    import recurrent_lm
    torch.manual_seed(0)
    return recurrent_lm


def test_training_lowers_the_loss(lm):
    losses = lm.train(lm.Model().cuda(), 60, log=None)
    # ln 128 = 4.85 for a uniform guess; fifteen different bytes occur, ln 15 = 2.71
    assert torch.isfinite(losses).all()
    assert losses[-5:].mean() < 2.7 < losses[0]


def test_steps_see_what_the_scan_sees(lm):
    """Greedy tokens of generate() are the whole pass's.  The log probabilities
    agree to a few bf16 ulp of the projections (2^-8 of values of order one,
    through two layers): 0.05."""
    import selective_state_space_81_amd as ms
    model = lm.Model().cuda()
    lm.train(model, 30, log=None)
    prompt = torch.tensor([list(b"21+34="), list(b"58+67=")], device="cuda")
    tokens, logp, ids, lps = model.generate(prompt, 4)
    assert tokens.shape == (2, 4) and ids.shape == lps.shape == (2, 4, 3)
    assert (lps[:, :, :-1] >= lps[:, :, 1:]).all()
    whole = torch.cat([prompt, tokens.long()], 1)
    with torch.no_grad():
        logits = model(whole[:, :-1].contiguous())
    r = ms.token_logprobs_fwd(logits, whole[:, 1:].reshape(-1).contiguous())
    want = r["logprob"].view(2, -1)[:, -4:]
    assert (want - logp).abs().max() < 0.05


def test_packed_documents_are_apart(lm):
    """The loss of a row of two documents, token by token, is theirs alone
    (the same kernels on other block positions: fp32 sums in another order and
    their bf16 roundings, 0.05)."""
    import selective_state_space_81_amd as ms
    model = lm.Model().cuda()
    a, b = (torch.tensor([list(t)], device="cuda") for t in (b"21+34=55\n", b"58+67=125\n"))
    both = torch.cat([a, b], 1)
    reset = torch.zeros(both.shape, dtype=torch.uint8, device="cuda")
    reset[0, a.shape[1]] = 1
    with torch.no_grad():
        packed = model(both, reset)
        alone = torch.cat([model(a), model(b)])
    t = both.reshape(-1)
    x, y = (ms.token_logprobs_fwd(v, t)["logprob"] for v in (packed, alone))
    assert (x - y).abs().max() < 0.05


def test_loss_of_one_row(lm):
    """The targets of one row are a view into its tokens; the loss is the one
    that two equal rows have (projections of other sizes, 0.05 as above)."""
    model = lm.Model().cuda()
    tokens, reset = (t.cuda() for t in lm.documents(torch.Generator().manual_seed(1), 1, 50))
    one = lm.loss_of(model, tokens, reset, bonus=0.01)
    one.backward()
    two = lm.loss_of(model, tokens.repeat(2, 1), reset.repeat(2, 1), bonus=0.01)
    assert torch.isfinite(one) and abs(float(one - two)) < 0.05
