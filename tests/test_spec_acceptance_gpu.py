"""Drafts that are accepted: single verifications, and the speculative loop of
test_spec_step_gpu.py fed with targets that like the drafts of the rows they
stand at, in every request."""
import copy

import numpy as np
import pytest
import torch

import spec_plain
import test_spec_step_gpu as loop
from gated_deltanet_recurrent_sigmoid_b200 import speculative as spec
from test_spec_gpu import check_verify, problem

pytestmark = pytest.mark.gpu
SLOTS = (4, 9, -1, 0, 7, 2)                              # of the loop's batch
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(gdn_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return spec.load()


@pytest.mark.parametrize("onehot", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,d,vocab", [(40, 2, 2049), (60, 7, 4096), (300, 3, 515), (200, 1, 50021)])
def test_as_many_drafts_are_accepted_as_should_be(n, d, vocab, dtype, onehot):
    """Draft j is accepted with probability a_j = min(1, p(x) / q(x)), the
    uniforms being random, so a sequence keeps k of them or more with
    probability a_1 ... a_k.  The total is within five standard deviations of
    its mean; both kinds of outcome are there."""
    p = problem(n, d, vocab, dtype, 5, onehot)
    kept = check_verify(p) - 1
    x = p["draft_tokens"].long()
    of = p["target_probs"].double().view(n, d + 1, vocab)[:, :d].gather(2, x[..., None])[..., 0]
    by = 1.0 if onehot else p["draft_probs"].double().gather(2, x[..., None])[..., 0]
    at_least = (of / by).clamp(max=1).cumprod(1).cpu().numpy()       # [n, d]: k + 1 drafts or more
    mean = at_least.sum(1)
    square = (at_least * (2 * np.arange(1, d + 1) - 1)).sum(1)       # sum over k of (k^2 - (k - 1)^2) P(kept >= k)
    spread = np.sqrt((square - mean**2).sum())
    assert mean.sum() > 5 * spread or onehot
    assert abs(kept.sum() - mean.sum()) <= 5 * spread, (kept.sum(), mean.sum(), spread)
    assert 0 < kept.sum() < n * d


def accepting(turns):
    """draw_step whose targets favour the drafts at the packed rows that the
    loop is about to run (its next draw from the generator is the lengths)."""

    def draw(rng, n, capacity):
        p, target, draft, tokens, u = plain(rng, n, capacity)
        lengths = copy.deepcopy(rng).integers(1, loop.DRAFTS + 2, n)
        lengths[len(turns) % n] = 0
        runs = np.where(np.array(SLOTS) >= 0, lengths, 0)
        cu = np.concatenate([[0], np.cumsum(runs)])
        for i in range(n):
            for j in range(runs[i] - 1):
                if (i + j + len(turns)) % 4:             # three of four
                    target[cu[i] + j, tokens[i, j]] += 14
        turns.append(runs)
        return p, target, draft, tokens, u

    plain = loop.draw_step
    return draw


@pytest.mark.parametrize("as_graph", [False, True])
def test_loop_with_accepted_drafts(as_graph, monkeypatch):
    turns, counts = [], []
    verify = spec_plain.verify

    def counted(*args):
        got = verify(*args)
        counts.append(got[1])
        return got

    monkeypatch.setattr(loop, "draw_step", accepting(turns))
    monkeypatch.setattr(spec_plain, "verify", counted)
    loop.test_speculative_loop_keeps_the_oracles_state(as_graph)
    runs, num = np.array(turns), np.array(counts)
    accepted, drafts = np.where(runs > 0, num - 1, 0), np.where(runs > 0, runs - 1, 0)
    assert num.shape == (5, 6) and (num[runs == 0] == 0).all()
    live = np.array(SLOTS) >= 0
    assert (accepted.sum(0)[live] >= 1).all(), accepted              # every request with a slot
    assert drafts.sum() // 2 <= accepted.sum() < drafts.sum(), (accepted.sum(), drafts.sum())
