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
