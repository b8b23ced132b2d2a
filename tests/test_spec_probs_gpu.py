"""Probabilities against 64 bits with a bound derived from the kernel's own
arithmetic, over temperatures down to the smallest number."""
import numpy as np
import pytest
import torch

import spec_plain
from gated_deltanet_recurrent_sigmoid_b200 import speculative as spec

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib(gdn_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return spec.load()


def bound(x, temperature, want, dtype):
    """|p - want| allowed per entry.  With y = (top - l) / t:
    - the exponent (l - top) c, c = log2(e) / t, carries at most four roundings
      (the constant, the division, the difference, the product), so the power
      is off by 4 * 2^-24 y; a factor 2^k that all powers of a row share cancels
      (|k| <= 2^-4, which moves the exponent's last rounding by 2^-28);
    - the power itself by 2^-22 (the instruction's documented error);
    - the sum by the mean of both under p, and by 2^-24 for each addition in a
      row: a thread's share of a slice, then 5 + 5 + 4 joins;
    - 1 / sum and the product by 2^-24 each, the output by half its step.
    Powers below 2^-126 may become 0.  A thread takes at most V / 128 values (no
    CTA has fewer threads), and not more than 64 up to 262,144 words, V / 4096
    beyond (16 CTAs of 256)."""
    vocab = x.shape[1]
    top = x.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        y = np.where(np.isfinite(x), (top - x) / temperature[:, None], 0)
    y = np.minimum(y, 2000.0)                    # (powers of those are 0 on both sides)
    adds = min(vocab / 128, max(64, vocab / 4096)) + 2 + 14
    mean = (want * y).sum(-1, keepdims=True)
    rel = 4 * 2.0**-24 * (y + mean) + 2 * 2.0**-22 + 2 * 2.0**-28 + adds * 2.0**-24 + 2 * 2.0**-24 + torch.finfo(dtype).eps / 2
    return want * rel + 2.0**-125


def check(logits, temperature, out):
    probs = torch.full(logits.shape, -1.0, device="cuda", dtype=out)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    spec.token_probs(logits, probs, temperature, device_status=st)
    x, t = logits.double().cpu().numpy(), temperature.double().cpu().numpy()
    want, _ = spec_plain.probs(x, t, None, np.zeros(x.shape))
    err, allowed = np.abs(probs.double().cpu().numpy() - want), bound(x, t, want, out)
    assert int(st) == 0 and (err <= allowed).all(), (err / allowed).max()


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab", [(40, 33), (40, 1000), (3, 5003), (600, 8192), (40, 50021), (3, 131072), (2, 300001)])
def test_probabilities_within_their_rounding(rows, vocab, dtype, out):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (torch.randn(rows, vocab, device="cuda", generator=g) * 4).to(dtype)
    t = torch.rand(rows, device="cuda", generator=g) * 1.5 + 0.05
    check(x, t, out)


# either side of where rows go from 8 CTAs to 16
@pytest.mark.parametrize("dtype,vocab", [(F32, 66001), (F32, 112639), (F32, 112641), (BF16, 140001), (BF16, 225279), (BF16, 225283)])
def test_rows_about_the_limit_of_sixteen(dtype, vocab):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (torch.randn(70, vocab, device="cuda", generator=g) * 4).to(dtype)
    check(x, torch.rand(70, device="cuda", generator=g) + 0.3, F32)


# from the smallest number, through c = log2(e) / t out of range, to where it fits
@pytest.mark.parametrize("t", [1e-45, 1e-44, 1e-42, 1e-40, 3e-39, 4.3e-39, 1e-38, 1.2e-38, 1.44e-38, 1e-37, 1e-30])
@pytest.mark.parametrize("base", [0.0, 1.0])
def test_temperatures_down_to_the_smallest(t, base):
    """Logits that are a few temperatures apart, about 0 and (where fp32 holds
    that: only ties are left) about 1."""
    t = float(np.float32(t))
    rng = np.random.default_rng(3)
    x = (base + np.round(rng.uniform(-8, 0, (5, 3001)) * t / 2.0**-149) * 2.0**-149).astype(np.float32)
    x[0, 7] = -np.inf
    x[1, :2000] = -3e38
    x[2, 5] = -1.0
    check(torch.from_numpy(x).cuda(), torch.full((5,), t, device="cuda"), F32)
