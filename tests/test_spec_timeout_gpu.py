"""Waits of the speculative step's kernels made to run out, in copies of the
library that withhold arrivals (tests/timeout_probe/build_spec_ranks.py): the
status bit is set, nothing wrong is written, the step can be repeated and the
context stays usable."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
TESTS = os.path.dirname(os.path.abspath(__file__))

SETUP = """
import sys, torch
sys.path[:0] = [{root!r}, {tests!r}]
from timeout_probe import build_spec_ranks
from gated_deltanet_recurrent_sigmoid_b200 import build, speculative as spec
kind, vocab, I32 = {kind!r}, {vocab}, torch.int32
good = spec.load()
build.SPEC_LIB_PATH = build_spec_ranks.build(kind)
spec._LIB = None
bad = spec.load()
assert bad is not good
g = torch.Generator(device="cuda").manual_seed(1)
st = torch.zeros(1, dtype=I32, device="cuda")

"""

PROBS = """# probabilities: no entry of a row may be wrong
x = torch.randn(3, vocab, device="cuda", generator=g) * 3
x[:, 0] = 20                                     # the maximum is rank 0's
x[1] = x[1].flip(0)                              # or the last one's
want, p = torch.full_like(x, -1), torch.full_like(x, -1)
spec._LIB = good
spec.token_probs(x, want)
spec._LIB = bad
spec.token_probs(x, p, device_status=st)
torch.cuda.synchronize()
assert int(st) == 4, int(st)
assert bool((p == -1).all()), "written by a cluster that has given up"


spec._LIB = good
st.zero_()
spec.token_probs(x, p, device_status=st)
assert int(st) == 0 and torch.equal(p, want)
print("left as it should be")
"""


def run(code, kind, vocab):
    r = subprocess.run([sys.executable, "-c", (SETUP + code).format(root=os.path.dirname(TESTS), tests=TESTS, kind=kind, vocab=vocab)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "left as it should be" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("kind,vocab", [("exchange", 40000), ("exchange", 500), ("exchange_rank", 40000), ("copy_rank", 40000)])
def test_probabilities_that_time_out(kind, vocab):
    run(PROBS, kind, vocab)


VERIFY = """# verification and commit: num_tokens 0, or the whole answer
n, d = 5, 2
target = torch.softmax(torch.randn(n * (d + 1), vocab, device="cuda", generator=g), -1)
tokens = target.view(n, d + 1, vocab)[:, :d].argmax(-1).to(I32)
u = torch.rand(n, d + 1, device="cuda", generator=g)
u[::2, :d] = 0                                   # all drafts accepted, or none
u[1::2, :d] = 0.999
cu, idx = torch.arange(0, n * (d + 1) + 1, d + 1, dtype=I32, device="cuda"), torch.arange(n, dtype=I32, device="cuda")
idx[3] = -1
new = lambda *s: torch.full(s, 7, dtype=I32, device="cuda")
outs = {{}}
for name, lib in (("good", good), ("bad", bad)):
    spec._LIB = lib
    st.zero_()
    outs[name] = (new(n, d + 1), new(n))
    spec.verify_drafts(target, tokens, None, u, *outs[name], cu_seqlens=cu, state_indices=idx, device_status=st)
    torch.cuda.synchronize()
    outs[name + "_status"] = int(st)
assert outs["good_status"] == 0 and outs["bad_status"] == 4, outs
(out, num), (got, n_got) = outs["good"], outs["bad"]
assert num.tolist() == [3, 1, 3, 0, 3]
for i in range(n):
    if kind == "exchange" or i == 3:                 # (in "exchange_rank" the other CTAs may have finished)
        assert int(n_got[i]) == 0, (i, n_got.tolist())
    elif int(n_got[i]):
        assert int(n_got[i]) == int(num[i]) and torch.equal(got[i], out[i]), i
inter, pool = torch.randn(n * (d + 1), 2, 128, 128, device="cuda"), torch.zeros(n, 2, 128, 128, device="cuda")
spec.commit_states(inter, n_got, pool, idx, cu)
for i in range(n):
    k = int(n_got[i])
    assert torch.equal(pool[i], inter[i * (d + 1) + k - 1]) if k else not bool(pool[i].any())


spec._LIB = good
st.zero_()
spec.verify_drafts(target, tokens, None, u, got, n_got, cu_seqlens=cu, state_indices=idx, device_status=st)
assert int(st) == 0 and torch.equal(n_got, num) and torch.equal(got, out)
print("left as it should be")
"""


@pytest.mark.parametrize("kind,vocab", [("exchange", 40000), ("exchange", 500), ("exchange_rank", 40000)])
def test_verifications_that_time_out(kind, vocab):
    run(VERIFY, kind, vocab)
