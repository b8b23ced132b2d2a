"""The operators of a speculative step on the GPU, against their 64-bit forms.

Tokens, counts, index arrays and copied states are compared for equality; the
sums behind a drawn token are 64-bit on both sides, and the inputs are random
or exact in few bits, so that the two orders of summation cannot part.
Probabilities have a bound of their own (``probs_bound``).
"""
import subprocess
import sys

import numpy as np
import pytest
import torch

import spec_plain
from gated_deltanet_recurrent_sigmoid_b200 import binding, speculative as spec

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib(gdn_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return spec.load()


def status_word():
    return torch.zeros(1, dtype=I32, device="cuda")


def gpu(x, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else torch.as_tensor(x)
    return t.to(dtype or t.dtype).cuda()


def f64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------- probabilities

@np.errstate(invalid="ignore", divide="ignore")
def probs_bound(logits, temperature, want, dtype):
    """|p - want| allowed per entry.  With x = (l - m) / t the exponent
    ((l - m) c, c = log2(e) / t) carries three roundings of 2^-24, which is
    3 * 2^-24 |x| relative in the result, and 2^x one of 2^-22.  The sum S adds
    the same for its terms (their mean under p), up to n additions of 2^-24
    each, n <= 2^10 (a thread's share of a row is at most 49,152 / 256 values,
    then 5 + 8 + 8 joins), and K <= 200 rescalings by such powers of two, but
    those act on what the running maximum has left behind: a rescaling by f
    < 1 scales all earlier errors by f as well, so at most a few count in
    full; 16 are allowed for.  Two roundings for 1 / S and the product, then
    the output's half step.  Results below 2^-126 may become 0."""
    finite = np.isfinite(logits)
    top = np.where(finite, logits, -np.inf).max(axis=-1, keepdims=True)
    x = np.where(finite, top - logits, 0) / np.where(temperature > 0, temperature, 1)[:, None]
    mean = (want * x).sum(-1, keepdims=True)
    vocab = logits.shape[1]
    adds = min(1024, 64 + vocab // 256)
    rel = 3 * 2.0**-24 * (x + mean) + (2 + 16) * 2.0**-22 + adds * 2.0**-24 + 2 * 2.0**-24 + torch.finfo(dtype).eps / 2
    return want * rel + 2.0**-125


def check_probs(logits, probs, temperature=None, row_seq=None, flags=0):
    before = f64(probs)
    st = status_word()
    spec.token_probs(logits, probs, temperature, row_seq, flags=flags, device_status=st)
    torch.cuda.synchronize()
    l64 = f64(logits)
    want, status = spec_plain.probs(l64, None if temperature is None else f64(temperature),
                                    None if row_seq is None else row_seq.cpu().numpy(), before)
    assert int(st) == status
    temps = np.ones(len(l64))
    if temperature is not None:
        i = np.arange(len(l64)) if row_seq is None else np.clip(row_seq.cpu().numpy(), 0, len(temperature) - 1)
        temps = f64(temperature)[i]
    got = f64(probs)
    untouched = np.zeros(len(l64), bool) if row_seq is None else (row_seq.cpu().numpy() < 0) | (row_seq.cpu().numpy() >= len(temperature))
    assert np.array_equal(got[untouched], before[untouched], equal_nan=True)
    live = ~untouched
    err, bound = np.abs(got - want)[live], probs_bound(l64[live], temps[live], want[live], probs.dtype)
    assert np.isfinite(got[live]).all() and (err <= bound).all(), (err - bound).max()


def logits_of(rows, vocab, dtype, seed, scale=4.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, vocab, device="cuda", generator=g) * scale).to(dtype)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (1, 2), (3, 7), (2, 8), (2, 255), (5, 1000), (1, 1025), (300, 4099), (1, 32768), (2, 50021)])
def test_probs(rows, vocab, dtype, out):
    check_probs(logits_of(rows, vocab, dtype, vocab), torch.full((rows, vocab), -7.0, device="cuda", dtype=out))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab", [(2, 131072), (160, 20011), (1, spec.MAX_VOCAB - 1), (1, spec.MAX_VOCAB)])
def test_probs_wide(rows, vocab, dtype):
    check_probs(logits_of(rows, vocab, dtype, 3), torch.empty(rows, vocab, device="cuda").fill_(-1))


@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F32, F32), (F32, BF16)])
def test_probs_temperatures_and_rows_left_alone(dtype, out):
    rows, vocab = 40, 3001
    temps = gpu(np.array([1, 0, 0.01, 100.0, -1.0, np.inf, np.nan, 0.7, 1e-30, 3e38, 1e-45], np.float32))
    seq = gpu(np.array([i % 13 for i in range(rows)], np.int32))
    seq[::7] = -1
    seq[5] = -2
    seq[6] = 2**31 - 1
    seq[8] = 11                                          # one past the temperatures
    check_probs(logits_of(rows, vocab, dtype, 1, scale=1.0), torch.full((rows, vocab), 9.0, device="cuda", dtype=out), temps, seq)


@pytest.mark.parametrize("temperature", [1.0, 0.0])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_probs_masks_infinities_and_nan(dtype, temperature):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    x = logits_of(12, 2050, dtype, 2)
    x[0] = -inf                                          # nothing left
    x[1] = nan
    x[2, :2049] = -inf                                   # the last one left
    x[3] = low                                           # all at the type's lowest value
    x[4, 5:] = low
    x[5, 7] = inf
    x[6, [3, 2000]] = inf                                # shared by two (the first when greedy)
    x[7, ::2] = nan
    x[8, 1:] = -inf
    x[9] = 0                                             # ties everywhere
    x[10, 100:] = x[10, 100].clone()
    x[11, [1999, 17, 1024]] = 60                         # ties across slices
    check_probs(x, torch.full((12, 2050), 9.0, device="cuda"), torch.full((12,), temperature, device="cuda"))


@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F32, BF16), (F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("shift,pad", [(1, 3), (3, 0), (5, 8), (8, 1)])
def test_probs_strides_and_alignment(dtype, out, shift, pad):
    rows, vocab = 6, 2500
    base = logits_of(1, shift + rows * (vocab + pad), dtype, 4)[0]
    logits = base[shift:].view(rows, vocab + pad)[:, :vocab]
    held = torch.full((rows * (vocab + 2 * pad) + shift + 2,), 5.0, device="cuda", dtype=out)
    probs = held[shift + 2:].view(rows, vocab + 2 * pad)[:, :vocab]
    check_probs(logits, probs)
    rest = held.clone()
    rest[shift + 2:].view(rows, vocab + 2 * pad)[:, :vocab] = 5
    assert (rest == 5).all(), "written outside the rows"


def test_probs_broadcast_temperature_and_shared_logit_row():
    x = logits_of(1, 777, F32, 5).expand(9, 777)
    check_probs(x, torch.empty(9, 777, device="cuda").fill_(0), torch.full((1,), 0.5, device="cuda").expand(9))


def test_probs_rows_past_32_bit_offsets():
    rows, vocab = 2**31 // 65536 + 3, 65536
    x = torch.zeros(rows, vocab, device="cuda", dtype=BF16)
    x[-1] = logits_of(1, vocab, BF16, 6)[0]
    p = torch.zeros(rows, vocab, device="cuda", dtype=BF16)
    spec.token_probs(x, p)
    one = torch.zeros(1, vocab, device="cuda", dtype=BF16)
    spec.token_probs(x[-1:], one)
    assert torch.equal(p[-1], one[0]) and bool((p[-2] == 1 / vocab).all()) and bool((p[0] == 1 / vocab).all())


@pytest.mark.parametrize("dtype,vocab", [(BF16, 4099), (F32, 517), (BF16, 20011)])
def test_probs_more_rows_than_fit_at_once(dtype, vocab):
    """Clusters take several rows, in turn aligned, masked, greedy, plain or
    left out, so that a row's state could leak into the next one's."""
    rows = 3000 if vocab < 5000 else 1200
    rng = np.random.default_rng(vocab)
    x = logits_of(rows, vocab, dtype, 8)
    x[::5] = x[::5].masked_fill(torch.rand_like(x[::5], dtype=F32) < 0.9, -float("inf"))
    x[::11] = -float("inf")
    x[3::17, ::3] = float("nan")
    x[7::19, vocab // 2] = float("inf")
    x[4::23] *= 1e6 if dtype == F32 else 2.0**20
    temps = gpu(np.array([1, 0, 0.5, -1, 2, 0, 1], np.float32))
    seq = gpu(rng.integers(-2, 8, rows).astype(np.int32))
    seq[1500 % rows:1700 % rows] = -1
    check_probs(x, torch.full((rows, vocab), 3.0, device="cuda"), temps, seq)


# ---------------------------------------------------------------- verification

def problem(n, d, vocab, dtype, seed, onehot=False, lens=None, close=0.5):
    """Rows of target and draft probabilities that agree about half the time."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = torch.full((n,), d + 1) if lens is None else torch.as_tensor(lens)
    cu = torch.zeros(n + 1, dtype=I32)
    cu[1:] = lens.cumsum(0)
    total = int(cu[-1])
    t = torch.randn(total, vocab, device="cuda", generator=g) * 2
    q = torch.randn(n, d, vocab, device="cuda", generator=g) * 2
    for i in range(n):
        k = min(int(lens[i]), d)
        q[i, :k] = t[int(cu[i]): int(cu[i]) + k] + close * torch.randn(k, vocab, device="cuda", generator=g)
    t, q = torch.softmax(t * 2, -1).to(dtype), torch.softmax(q * 2, -1).to(dtype)
    tokens = torch.zeros(n, d, dtype=I32, device="cuda")
    if d:
        noise = torch.empty(n, d, vocab, device="cuda").exponential_(generator=g)
        tokens = (q.float() / noise).argmax(-1).to(I32)
    u = torch.rand(n, d + 1, device="cuda", generator=g)
    return dict(target_probs=t, draft_tokens=tokens, draft_probs=None if onehot else q, uniforms=u, cu_seqlens=cu.cuda())


def outputs(n, d):
    return dict(out_tokens=torch.full((n, d + 1), -99, dtype=I32, device="cuda"),
                num_tokens=torch.full((n,), -99, dtype=I32, device="cuda"))


def check_verify(p, cu=None, **more):
    n, d = p["draft_tokens"].shape
    o, st = outputs(n, d), status_word()
    spec.verify_drafts(**p, **o, **more, device_status=st)
    torch.cuda.synchronize()
    t = p["target_probs"]
    if cu is None:
        cu = p["cu_seqlens"].cpu().numpy() if p.get("cu_seqlens") is not None else np.arange(n + 1) * t.shape[1]
    q, idx = p.get("draft_probs"), more.get("state_indices")
    want, num, status = spec_plain.verify(f64(t).reshape(-1, t.shape[-1]), p["draft_tokens"].cpu().numpy(), None if q is None else f64(q),
                                          f64(p["uniforms"]), cu, None if idx is None else idx.cpu().numpy())
    assert np.array_equal(o["num_tokens"].cpu().numpy(), num)
    assert np.array_equal(o["out_tokens"].cpu().numpy(), want)
    assert int(st) == status
    return num


@pytest.mark.parametrize("onehot", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,d,vocab", [(1, 0, 1), (1, 1, 1), (4, 0, 33), (3, 1, 7), (5, 3, 1000), (2, 7, 4096), (40, 2, 2049), (1, 3, 32768), (300, 3, 515), (3, 4, 50021)])
def test_verify(n, d, vocab, dtype, onehot):
    kept = sum(check_verify(problem(n, d, vocab, dtype, seed, onehot)).sum() for seed in (1, 2))
    assert kept >= 2 * n


def test_verify_large_vocab_and_long_drafts():
    check_verify(problem(2, 2, 300007, F32, 3))
    num = check_verify(problem(6, 70, 200, F32, 4, close=0.02))      # past one ballot of 32 drafts
    assert num.max() > 33


@pytest.mark.parametrize("onehot", [False, True])
def test_verify_ragged_padded_and_bad_rows(onehot):
    lens = [1, 4, 0, 2, 3, 4, 1, 4, 2]
    p = problem(9, 3, 901, F32, 5, onehot, lens)
    idx = gpu(np.array([3, 1, 0, -1, 2, 5, 6, -7, 4], np.int32))
    check_verify(p, state_indices=idx)
    p["draft_tokens"][1, 1] = -1                                     # drafts end early
    p["draft_tokens"][4, 0] = 901                                    # outside the vocabulary
    p["draft_tokens"][5, 0] = -2
    check_verify(p)
    p["cu_seqlens"][4] = 9999                                        # sequences 3 and 4 are not usable
    check_verify(p)
    p["cu_seqlens"][4] = p["cu_seqlens"][3]
    p["cu_seqlens"][9] = p["cu_seqlens"][8] + 5                      # longer than D + 1, past the rows
    p["cu_seqlens"][0] = -1
    check_verify(p)


@pytest.mark.parametrize("n,d,vocab,dtype", [(1300, 1, 1500, F32), (600, 1, 5003, BF16), (200, 2, 9000, F32), (150, 1, 12345, F32), (8, 1, 70000, BF16)])
def test_verify_batches_of_every_cluster_size(n, d, vocab, dtype):
    check_verify(problem(n, d, vocab, dtype, 7))


def test_verify_with_nothing_to_judge():
    p = problem(3, 2, 50, F32, 1, lens=[0, 0, 0])
    assert check_verify(p).tolist() == [0, 0, 0]
    p = problem(2, 0, 50, F32, 1)
    check_verify({**p, "draft_probs": torch.zeros(2, 0, 50, device="cuda")})


def test_verify_fixed_length_rows_and_strides():
    n, d, vocab = 4, 3, 1203
    p = problem(n, d, vocab, F32, 6)
    wide = torch.zeros(n * (d + 1), vocab + 5, device="cuda")
    wide[:, 2:2 + vocab] = p["target_probs"]
    steps = torch.zeros(d, n, vocab + 1, device="cuda")              # the draft loop's own order
    steps[:, :, 1:] = p["draft_probs"].transpose(0, 1)
    tokens = p["draft_tokens"].t().contiguous().t()
    uniforms = torch.rand(1, d + 1, device="cuda").expand(n, d + 1)
    q = dict(target_probs=wide[:, 2:2 + vocab].unflatten(0, (n, d + 1)), draft_tokens=tokens, uniforms=uniforms,
             draft_probs=steps[:, :, 1:].transpose(0, 1), cu_seqlens=None)
    check_verify(q)
    q["target_probs"] = q["target_probs"][:, :2]                     # T < D + 1 (a flat [N, T] no more: refused)
    with pytest.raises(binding.GdnError):
        check_verify(q)
    q["target_probs"] = q["target_probs"].contiguous()
    check_verify(q)
    out = torch.full((d + 1, n), -9, dtype=I32, device="cuda").t()   # written by columns
    num = torch.full((2 * n,), -9, dtype=I32, device="cuda")[::2]
    spec.verify_drafts(q["target_probs"], q["draft_tokens"], q["draft_probs"], uniforms, out, num)
    o = outputs(n, d)
    spec.verify_drafts(q["target_probs"], q["draft_tokens"], q["draft_probs"], uniforms, **o)
    assert torch.equal(out, o["out_tokens"]) and torch.equal(num, o["num_tokens"])


def dyadic(rows, vocab, seed, bits=10):
    """Probabilities that are multiples of 2^-bits with sum 1: all sums exact."""
    rng = np.random.default_rng(seed)
    return rng.multinomial(2**bits, np.ones(vocab) / vocab, size=rows).astype(np.float32) / 2**bits


@pytest.mark.parametrize("vocab", [5, 700, 9000])
def test_verify_ties_are_exact(vocab):
    """Products and running sums that meet the goal exactly: the comparisons
    are strict, on both sides of every tie."""
    n, d = 64, 2
    rng = np.random.default_rng(vocab)
    t, q = dyadic(n * 3, vocab, 1), dyadic(n * d, vocab, 2).reshape(n, d, vocab)
    q[::2] = t.reshape(n, 3, vocab)[::2, :d]                         # p = q: u q(x) = p(x) never, u < 1
    tokens = rng.integers(0, vocab, (n, d)).astype(np.int32)
    u = rng.integers(0, 2**10, (n, d + 1)).astype(np.float32) / 2**10
    p = dict(target_probs=gpu(t), draft_tokens=gpu(tokens), draft_probs=gpu(q), uniforms=gpu(u),
             cu_seqlens=gpu(np.arange(0, 3 * n + 1, 3, dtype=np.int32)))
    check_verify(p)
    check_verify({**p, "draft_probs": None})


def test_verify_rows_that_leave_nothing():
    vocab = 300
    t = torch.zeros(12, vocab, device="cuda")
    q = torch.zeros(6, 1, vocab, device="cuda")
    t[0, 5] = 0.25; t[0, 200] = 0.25; q[0, 0] = 1                    # p <= q everywhere: drawn from p
    t[2] = float("nan")                                              # no weight at all
    t[4, 7] = float("inf"); t[4, 9] = 0.5                            # infinite entries weigh nothing
    t[6] = 0                                                         # an empty row
    t[8, 3] = 1; q[4, 0, 3] = float("nan"); t[8, 299] = 1e-30        # NaN drafts are rejected
    t[11] = -1                                                       # negative: nothing
    t[10, 0] = 1
    x = gpu(np.array([[0], [0], [9], [1], [3], [0]], np.int32))
    u = gpu(np.array([[0.9, 0.6], [0.1, 0.5], [0.9, 0.999], [0.5, 0.5], [0.0, 0.0], [0.1, 0.3]], np.float32))
    p = dict(target_probs=t, draft_tokens=x, draft_probs=q, uniforms=u, cu_seqlens=gpu(np.arange(0, 13, 2, dtype=np.int32)))
    check_verify(p)
    check_verify({**p, "draft_probs": None})


def test_verify_uniforms_at_their_ends():
    p = problem(8, 1, 1000, F32, 9)
    p["target_probs"][:, 990:] = 0
    p["uniforms"][:, 1] = gpu(np.array([0, 1 - 2.0**-24, 1, 2, -1, np.nan, 1e-45, np.inf], np.float32))
    check_verify(p)


def test_verify_rows_past_32_bit_offsets():
    n, vocab = 2, 1000
    far = 2**31 + 64
    t = torch.zeros(far + vocab, device="cuda", dtype=BF16).as_strided((n, vocab), (far, 1))
    t[0, 3] = 1
    t[1, 500:] = 0.002
    p = dict(target_probs=t, draft_tokens=torch.zeros(n, 0, dtype=I32, device="cuda"), draft_probs=None,
             uniforms=torch.full((n, 1), 0.5, device="cuda"), cu_seqlens=gpu(np.arange(3, dtype=np.int32)))
    o = outputs(n, 0)
    spec.verify_drafts(**p, **o)
    assert o["out_tokens"].tolist() == [[3], [750]] and o["num_tokens"].tolist() == [1, 1]


def test_verify_draws_with_the_residual_distribution():
    """20,000 sequences over 5 tokens: frequencies of the first emitted token
    follow p whatever q is (4.5 standard deviations)."""
    n, p, q = 20000, np.array([0.1, 0.2, 0.3, 0.15, 0.25]), np.array([0.5, 0.05, 0.05, 0.3, 0.1])
    rng = np.random.default_rng(1)
    tokens = rng.choice(5, size=(n, 1), p=q).astype(np.int32)
    o = outputs(n, 1)
    spec.verify_drafts(gpu(np.tile(p, (2 * n, 1)), F32), gpu(tokens), gpu(np.tile(q, (n, 1, 1)), F32), gpu(rng.random((n, 2)), F32),
                       **o, cu_seqlens=gpu(np.arange(0, 2 * n + 1, 2, dtype=np.int32)))
    seen = np.bincount(o["out_tokens"][:, 0].cpu().numpy(), minlength=5) / n
    assert (np.abs(seen - p) < 4.5 * np.sqrt(p * (1 - p) / n)).all(), seen


# ---------------------------------------------------------------- states

@pytest.mark.parametrize("n,t,heads,varlen", [(1, 1, 1, False), (4, 4, 4, False), (3, 5, 3, True), (64, 2, 8, True), (130, 3, 2, False)])
def test_commit(n, t, heads, varlen):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, t + 1, n) if varlen else np.full(n, t)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    inter = torch.randn(max(1, cu[-1]) if varlen else n * t, heads, 128, 128, device="cuda")
    pool = torch.randn(n + 3, heads, 128, 128, device="cuda")
    num = np.array([rng.integers(0, k + 1) for k in lens], np.int32)
    idx = rng.permutation(n + 3)[:n].astype(np.int32)
    if n > 3:
        idx[[0, 2]] = -1
        idx[3], idx[1] = n + 3, -2                                   # bad slots
        num[-1] = lens[-1] + 1
    want, status = spec_plain.commit(inter.cpu().numpy(), num, pool.cpu().numpy(), idx, cu)
    st = status_word()
    spec.commit_states(inter, gpu(num), pool, gpu(idx), gpu(cu) if varlen else None, device_status=st)
    assert int(st) == status and np.array_equal(pool.cpu().numpy(), want)


def test_commit_strided_states_and_bad_cu_seqlens():
    inter = torch.randn(6, 2, 130, 128, device="cuda")[:, :, :128]
    big = torch.randn(5, 4, 128, 128, device="cuda")
    pool = big[:, ::2]
    cu = np.array([0, 2, -1, 6, 9], np.int32)
    num, idx = np.array([2, 1, 1, 1], np.int32), np.array([4, 0, 1, 2], np.int32)
    want, status = spec_plain.commit(inter.cpu().numpy(), num, pool.cpu().numpy(), idx, cu)
    other = big[:, 1::2].clone()
    st = status_word()
    spec.commit_states(inter, gpu(num), pool, gpu(idx), gpu(cu), device_status=st)
    assert int(st) == status == binding.DEV_BAD_SEQLENS
    assert np.array_equal(pool.cpu().numpy(), want) and torch.equal(big[:, 1::2], other)


def test_commit_states_past_32_bit_offsets():
    tokens = 2**31 // (8 * 16384) + 2
    inter = torch.zeros(tokens, 8, 128, 128, device="cuda")
    inter[-1] = torch.randn(8, 128, 128, device="cuda")
    pool = torch.zeros(2, 8, 128, 128, device="cuda")
    spec.commit_states(inter, gpu(np.array([0, tokens], np.int32)), pool, gpu(np.array([1, 0], np.int32)),
                       gpu(np.array([0, 0, tokens], np.int32)))
    assert torch.equal(pool[0], inter[-1]) and bool((pool[1] == 0).all())


# ---------------------------------------------------------------- index arrays

def maps_problem(n, longest, cached, block, seed, capacity=None, blocks=True, free=None, head=3):
    rng = np.random.default_rng(seed)
    lengths = rng.integers(0, longest + 1, n).astype(np.int32)
    context = rng.integers(0, cached + 1, n).astype(np.int32)
    slots = rng.permutation(2 * n)[:n].astype(np.int32)
    slots[rng.random(n) < 0.1] = -1
    p = dict(lengths=lengths, context=context, slots=slots)
    capacity = int(lengths.sum()) + 5 if capacity is None else capacity
    if blocks:
        held = -(-context // block) + rng.integers(0, 3, n)
        wide = (cached + longest) // block + 4
        ids = rng.permutation(2**20)[: n * wide + 50].astype(np.int32)
        p.update(tables=rng.integers(0, 1000, (n, wide)).astype(np.int32), held=held.astype(np.int32),
                 free=ids if free is None else ids[:free], head=head, block=block)
    return p, capacity


def check_maps(p, capacity, row_stride=0, **more):
    want, status = spec_plain.maps(capacity=capacity, **p)
    n = len(p["lengths"])
    z = lambda *s, dtype=I32: torch.full(s, -77, dtype=dtype, device="cuda")  # noqa: E731
    out = dict(cu_seqlens=z(n + 1), state_indices=z(n), row_seq=z(capacity), positions=z(capacity))
    args = dict(lengths=gpu(p["lengths"]), context=gpu(p["context"]), slots=gpu(p["slots"]))
    if "tables" in p:
        wide = p["tables"].shape[1]
        table = z(n, wide + row_stride)
        table[:, :wide] = gpu(p["tables"])
        out.update(block_tables=table[:, :wide], blocks_held_out=z(n), free_head_out=z(1), slot_map=z(capacity, dtype=torch.int64))
        args.update(blocks_held=gpu(p["held"]), free_blocks=gpu(p["free"]), free_head=gpu(np.array([p["head"]], np.int32)),
                    block_size=p["block"])
    st = status_word()
    spec.step_maps(**args, **out, **more, device_status=st)
    torch.cuda.synchronize()
    for k, v in want.items():
        assert np.array_equal(out[k].cpu().numpy(), v), k
    assert int(st) == status
    if "tables" in p and row_stride:
        assert bool((table[:, wide:] == -77).all())
    return want, status


@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("n,longest,cached,block", [(1, 1, 0, 1), (1, 5000, 3, 7), (2, 3, 100, 16), (33, 40, 64, 16), (128, 4, 3000, 64),
                                                    (1023, 9, 500, 24), (1025, 3, 10, 1), (2500, 2, 40, 128), (7, 3000, 9000, 100), (60, 4000, 5000, 64),
                                                    (257, 700, 100, 48)])
def test_maps(n, longest, cached, block, blocks):
    p, capacity = maps_problem(n, longest, cached, block, n, blocks=blocks)
    check_maps(p, capacity, row_stride=3)


def test_maps_of_nothing():
    p, _ = maps_problem(5, 4, 9, 4, 1)
    p["lengths"][:] = 0
    check_maps(p, 8)
    check_maps(p, 0)
    empty = {k: (v[:0] if k in ("lengths", "context", "slots", "tables", "held") else v) for k, v in p.items()}
    check_maps(empty, 1030)
    check_maps({k: empty[k] for k in ("lengths", "context", "slots")}, 3)
    check_maps({**empty, "head": -1}, 3)


@pytest.mark.parametrize("n,longest", [(40, 30), (2100, 5)])
@pytest.mark.parametrize("short", [1, 0.7, 0.01, 0])
def test_maps_without_room(n, longest, short):
    p, capacity = maps_problem(n, longest, 50, 8, 7)
    full = int(np.where(p["slots"] >= 0, p["lengths"], 0).sum())
    check_maps(p, int(full * short))                                  # rows run out
    free = spec_plain.maps(capacity=capacity, **p)[0]["free_head_out"][0]
    p["free"] = p["free"][: max(3, int(free * short))]                # blocks run out
    check_maps(p, capacity)
    check_maps({k: p[k] for k in ("lengths", "context", "slots")}, int(full * short))


def test_maps_bad_requests():
    p, capacity = maps_problem(60, 20, 100, 16, 8)
    p["lengths"][3], p["context"][5], p["slots"][7] = -4, -1, -3
    p["lengths"][9], p["context"][9] = 2**31 - 1, 7
    p["held"][11], p["held"][13] = -1, p["tables"].shape[1] + 1
    p["context"][15], p["held"][15], p["lengths"][15] = 40, 2, 5      # 40 tokens in 2 blocks of 16
    p["context"][17], p["held"][17], p["lengths"][17] = 16 * p["tables"].shape[1], p["tables"].shape[1], 5
    p["slots"][[11, 13, 15, 17]] = [200, 201, 202, 203]
    p["lengths"][[11, 13]] = 2
    _, status = check_maps(p, capacity + 60)
    assert status == binding.DEV_BAD_SLOT | spec.DEV_BAD_LENGTH | spec.DEV_BAD_BLOCKS
    for head in (-1, len(p["free"]) + 1):
        check_maps({**p, "head": head}, capacity + 60)


def test_maps_places_past_32_bits():
    p, capacity = maps_problem(3, 9, 20, 4096, 9)
    p["free"] = p["free"] + 2**30
    check_maps(p, capacity)
    p["tables"] = p["tables"] + 2**30                                 # the first two requests hold all they need
    want, _ = check_maps(p, capacity)
    assert want["slot_map"].max() > 2**40


# ---------------------------------------------------------------- how they are called

def test_prepared_calls_streams_graphs_and_pdl():
    """Each operator through its prepared call: on a stream of its own, and
    captured together with PDL launches and replayed on new inputs."""
    n, d, vocab = 6, 3, 5000
    p = problem(n, d, vocab, F32, 11)
    logits, probs = logits_of(n * 4, vocab, BF16, 12), torch.zeros(n * 4, vocab, device="cuda")
    inter, pool = torch.randn(n * 4, 2, 128, 128, device="cuda"), torch.zeros(n, 2, 128, 128, device="cuda")
    idx, o = torch.arange(n, dtype=I32, device="cuda"), outputs(n, d)
    z = lambda k: torch.zeros(k, dtype=I32, device="cuda")            # noqa: E731
    lengths, context, cu, seq, pos, at = z(n) + 4, z(n) + 9, z(n + 1), z(n * 4), z(n * 4), z(n)
    temps = torch.rand(n, device="cuda") + 0.5
    st = status_word()
    calls = [spec.PreparedStepMaps(lengths, context, idx, cu, at, seq, pos, flags=binding.LAUNCH_PDL, device_status=st),
             spec.PreparedTokenProbs(logits, probs, temps, seq, flags=binding.LAUNCH_PDL, device_status=st),
             spec.PreparedVerifyDrafts(probs, p["draft_tokens"], p["draft_probs"], p["uniforms"], **o, cu_seqlens=cu,
                                       state_indices=at, flags=binding.LAUNCH_PDL, device_status=st),
             spec.PreparedCommitStates(inter, o["num_tokens"], pool, at, cu, flags=binding.LAUNCH_PDL, device_status=st)]

    def check():
        torch.cuda.synchronize()
        fresh, q = outputs(n, d), torch.zeros_like(probs)
        spec.token_probs(logits, q, temps, torch.arange(n, dtype=I32, device="cuda").repeat_interleave(4))
        assert torch.equal(q, probs)
        want, num, _ = spec_plain.verify(f64(q), p["draft_tokens"].cpu().numpy(), f64(p["draft_probs"]), f64(p["uniforms"]), np.arange(n + 1) * 4)
        assert np.array_equal(o["out_tokens"].cpu().numpy(), want) and np.array_equal(o["num_tokens"].cpu().numpy(), num)
        assert torch.equal(pool, inter[torch.arange(n, device="cuda") * 4 + o["num_tokens"] - 1])
        assert int(st) == 0

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                                     # the current stream is followed
        for c in calls:
            c()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    for seed in (21, 22):
        logits.copy_(logits_of(n * 4, vocab, BF16, seed))
        inter.normal_()
        pool.zero_()
        p["uniforms"].uniform_()
        graph.replay()
        check()


def test_shapes_first_seen_in_a_capture():
    """A graph captured from shapes that no call has run before."""
    x, p = logits_of(77, 9123, F32, 41), torch.zeros(77, 9123, device="cuda")
    q = problem(37, 2, 3111, F32, 42)
    o = outputs(37, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spec.token_probs(x, p)
        spec.verify_drafts(**q, **o)
    graph.replay()
    check = torch.zeros_like(p)
    spec.token_probs(x, check)
    again = outputs(37, 2)
    spec.verify_drafts(**q, **again)
    assert torch.equal(p, check) and torch.equal(o["out_tokens"], again["out_tokens"])


def test_results_do_not_change_from_run_to_run():
    """No order of arrival enters a result: 20 runs, the same bits."""
    x = logits_of(64, 50021, F32, 51)
    p, first = torch.zeros_like(x), None
    q = problem(64, 3, 10007, BF16, 52)
    for _ in range(20):
        o = outputs(64, 3)
        spec.token_probs(x, p)
        spec.verify_drafts(**q, **o)
        got = (p.clone(), o["out_tokens"], o["num_tokens"])
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_two_verifications_at_once():
    """Two streams, two sets of outputs: nothing is shared between calls."""
    a, b = problem(100, 3, 30011, F32, 31), problem(100, 3, 30011, F32, 32)
    oa, ob = outputs(100, 3), outputs(100, 3)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ca, cb = spec.PreparedVerifyDrafts(**a, **oa, stream=sa), spec.PreparedVerifyDrafts(**b, **ob, stream=sb)
    for _ in range(10):
        ca()
        cb()
    torch.cuda.synchronize()
    for p, o in ((a, oa), (b, ob)):
        again = outputs(100, 3)
        spec.verify_drafts(**p, **again)
        assert torch.equal(o["out_tokens"], again["out_tokens"]) and torch.equal(o["num_tokens"], again["num_tokens"])


def test_two_captured_graphs_at_once():
    """Replays of two graphs that overlap on two streams share nothing."""
    sets = []
    for seed in (61, 62):
        x, q = logits_of(300, 20011, F32, seed), problem(90, 2, 20011, F32, seed)
        p, o = torch.zeros(300, 20011, device="cuda"), outputs(90, 2)
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            spec.token_probs(x, p)
            spec.verify_drafts(**q, **o)
        sets.append((x, q, p, o, graph, stream))
    torch.cuda.synchronize()
    for _ in range(5):
        for *_, graph, stream in sets:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for x, q, p, o, *_ in sets:
        check, again = torch.zeros_like(p), outputs(90, 2)
        spec.token_probs(x, check)
        spec.verify_drafts(**q, **again)
        assert torch.equal(p, check) and torch.equal(o["out_tokens"], again["out_tokens"])


def test_first_calls_from_several_threads():
    """A fresh process whose first calls of each kernel come from six threads
    at once (one-time set-up per device, the remembered launch shapes)."""
    code = """
import sys, threading
sys.path[:0] = [{root!r}]
import torch
from gated_deltanet_recurrent_sigmoid_b200 import speculative as spec
spec.load()
jobs, errors, start = [], [], threading.Barrier(6)
for k in range(6):
    vocab = (1000, 40000, 131072)[k % 3]
    x = torch.randn(20, vocab, device="cuda").to((torch.float32, torch.bfloat16)[k % 2])
    jobs.append((x, torch.zeros(20, vocab, device="cuda"), torch.zeros(20, 1, dtype=torch.int32, device="cuda"),
                 torch.zeros(20, dtype=torch.int32, device="cuda"), torch.full((20, 1), 0.5, device="cuda"), torch.cuda.Stream()))
torch.cuda.synchronize()
def run(job):
    x, p, out, num, u, stream = job
    try:
        start.wait()
        for _ in range(20):
            spec.token_probs(x, p, stream=stream)
            spec.verify_drafts(p[:, None], torch.zeros(20, 0, dtype=torch.int32, device="cuda"), None, u, out, num, stream=stream)
        stream.synchronize()
    except Exception as e:
        errors.append(repr(e))
threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
for t in threads: t.start()
for t in threads: t.join()
assert not errors, errors
for x, p, out, num, u, stream in jobs:
    assert torch.allclose(p, torch.softmax(x.double(), -1).float(), atol=1e-6)
    below = p.double().cumsum(-1)
    want = (below > 0.5 * below[:, -1:]).int().argmax(-1)
    assert torch.equal(out[:, 0].long(), want) and bool((num == 1).all())
print("threads agree")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "threads agree" in r.stdout, r.stderr[-2000:]


def test_host_tensors_are_refused():
    with pytest.raises(ValueError):
        spec.token_probs(torch.zeros(1, 8), torch.zeros(1, 8, device="cuda"))


def test_bounded_wait_reports_a_timeout():
    """A copy of the library whose bulk copies are never waited to their end
    (tests/timeout_probe): the call ends with the status bit and the context
    stays usable."""
    code = """
import sys, torch
sys.path[:0] = [{root!r}, {tests!r}]
from timeout_probe import build_spec
from gated_deltanet_recurrent_sigmoid_b200 import build, speculative as spec
good = spec.load()
build.SPEC_LIB_PATH = build_spec.build()
spec._LIB = None
x, p, st = torch.randn(3, 40000, device="cuda"), torch.zeros(3, 40000, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
spec.token_probs(x, p, device_status=st)
torch.cuda.synchronize()
assert int(st) == 4, int(st)
spec._LIB = good
st.zero_()
spec.token_probs(x, p, device_status=st)
assert int(st) == 0 and torch.allclose(p, torch.softmax(x, -1), atol=1e-6)
print("timed out as it should")
"""
    import os
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", code.format(root=os.path.dirname(tests), tests=tests)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "timed out as it should" in r.stdout, r.stderr[-2000:]
