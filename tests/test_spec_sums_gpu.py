"""The sums behind a drawn token, on rows where 64 bits decide a tie and fewer
do not.  Every weight is a multiple of one power of two that is at least 2^-52
of their total, so each of their sums, in any order, is exact in fp64: the
expected tokens need no tolerance."""
import pytest
import torch

from gated_deltanet_recurrent_sigmoid_b200 import speculative as spec

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib(gdn_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return spec.load()


def halves(n, half, bits, unit, seed):
    """[n, 2 half] weights: either half of a row holds the same values in an
    order of its own, whole multiples of ``unit`` below 2^bits of it and one
    0.4375."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    values = torch.randint(1, 2**bits, (n, half), device="cuda", generator=g).double() * unit
    values[:, 0] = 0.4375
    order = lambda: torch.rand(n, half, device="cuda", generator=g).argsort(1)    # noqa: E731
    return torch.cat((values.gather(1, order()), values.gather(1, order())), 1)


def drawn(target, **more):
    """The tokens that follow, one sequence a row of ``target``."""
    n, d = target.shape[0] // (2 if more else 1), 1 if more else 0
    out, num = torch.full((n, d + 1), -9, dtype=I32, device="cuda"), torch.full((n,), -9, dtype=I32, device="cuda")
    u = torch.full((n, d + 1), 0.5, device="cuda")
    more = more or dict(draft_tokens=torch.zeros(n, 0, dtype=I32, device="cuda"), draft_probs=None)
    if d:
        u[:, 0] = 0.9
    cu = torch.arange(0, n * (d + 1) + 1, d + 1, dtype=I32, device="cuda")
    st = torch.zeros(1, dtype=I32, device="cuda")
    spec.verify_drafts(target, more["draft_tokens"], more["draft_probs"], u, out, num, cu_seqlens=cu, device_status=st)
    assert int(st) == 0 and bool((num == 1).all())
    return out[:, 0]


# 600 sequences take one CTA each, 128 take eight
@pytest.mark.parametrize("n", [600, 128, 3])
@pytest.mark.parametrize("bits,unit", [(20, 2.0**-46), (20, 2.0**-44), (22, 2.0**-50)])
@pytest.mark.parametrize("shift", [0, 1])
def test_half_of_the_weight(n, bits, unit, shift):
    half = 65536
    w = halves(n, half, bits, unit, n + bits)
    rows = torch.zeros(n, 2 * half + 3, device="cuda")               # rows off the 16-byte boundaries
    rows = rows[:, shift: shift + 2 * half] if shift else rows[:, :2 * half].contiguous()
    rows.copy_(w)
    assert torch.equal(rows.double(), w)
    assert bool((drawn(rows) == half).all())


@pytest.mark.parametrize("n", [600, 40])
def test_half_of_the_weight_bf16(n):
    half = 32768
    w = halves(n, half, 8, 2.0**-46, 3)
    assert torch.equal(w.to(BF16).double(), w)
    assert bool((drawn(w.to(BF16)) == half).all())


@pytest.mark.parametrize("n", [600, 64])
@pytest.mark.parametrize("shift", [0, 1])
def test_half_of_what_a_rejection_leaves(n, shift):
    """Weights p - q; q lies like p in its 16-byte words, or not."""
    half, unit = 30000, 2.0**-46
    w = halves(n, half, 20, unit, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    q = torch.randint(1, 2**20, w.shape, device="cuda", generator=g).double() * unit
    p = w + q
    p[w == 0.4375], q[w == 0.4375] = 0.875, 0.4375
    wide = 2 * half + 8
    target = torch.zeros(2 * n, wide, device="cuda")
    target[::2, 4:4 + 2 * half] = p
    held = torch.zeros(n, 1, wide + shift, device="cuda")
    draft = held[:, :, shift:]
    draft[:, 0, 4:4 + 2 * half] = q
    draft[:, 0, 0] = 0.5                                             # p is 0 there: refused, and no weight
    assert torch.equal(target[::2, 4:4 + 2 * half].double(), p) and torch.equal(draft[:, 0, 4:4 + 2 * half].double(), q)
    tokens = torch.zeros(n, 1, dtype=I32, device="cuda")
    assert bool((drawn(target, draft_tokens=tokens, draft_probs=draft) == 4 + half).all())


def test_uniforms_of_one_draw_the_last_token():
    """u >= 1 counts as the whole weight however its sums round."""
    n, vocab = 600, 40000
    g = torch.Generator(device="cuda").manual_seed(7)
    rows = torch.rand(n, vocab, device="cuda", generator=g) ** 8
    rows[:, -1] = 1e-12
    out, num = torch.zeros(n, 1, dtype=I32, device="cuda"), torch.zeros(n, dtype=I32, device="cuda")
    spec.verify_drafts(rows, torch.zeros(n, 0, dtype=I32, device="cuda"), None, torch.ones(n, 1, device="cuda"), out, num,
                       cu_seqlens=torch.arange(n + 1, dtype=I32, device="cuda"))
    assert bool((out == vocab - 1).all())
