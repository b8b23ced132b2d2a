"""A speculative decode loop on the GPU from end to end: index arrays, state
update with the state after every token, probabilities, verification, commit.
After every step the state pool and the outputs of the kept tokens equal the
oracle's, which runs the kept tokens only and knows nothing of the rest."""
import numpy as np
import pytest
import torch

import spec_plain
from gated_deltanet_recurrent_sigmoid_b200 import binding, speculative as spec
from gpu_helpers import assert_out_close, assert_state_close, bf16_tensor, oracle_on
from helpers import random_problem

pytestmark = pytest.mark.gpu
H, HV, DRAFTS, VOCAB, SLOTS = 2, 4, 3, 1537, 11
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib(gdn_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return spec.load()


def draw_step(rng, n, capacity):
    """One step's activations (by packed row) and model outputs."""
    p = random_problem(rng, lens=[capacity], H=H, HV=HV, K=128, V=128, pad=())
    target = rng.standard_normal((capacity, VOCAB)).astype(np.float32) * 3
    draft = rng.dirichlet(np.full(VOCAB, 0.3), size=(n, DRAFTS)).astype(np.float32)
    tokens = np.array([[rng.choice(VOCAB, p=q / q.sum()) for q in d.astype(np.float64)] for d in draft], np.int32)
    for i in range(n):                                   # rows that like their drafts, mostly
        for j in range(DRAFTS):
            if rng.random() < 0.7:
                target[min(capacity - 1, i * (DRAFTS + 1) + j), tokens[i, j]] += 14
    return p, target, draft, tokens, rng.random((n, DRAFTS + 1)).astype(np.float32)


@pytest.mark.parametrize("as_graph", [False, True])
def test_speculative_loop_keeps_the_oracles_state(as_graph):
    rng = np.random.default_rng(77)
    n, capacity, block = 6, 6 * (DRAFTS + 1), 4
    gpu = lambda x: torch.as_tensor(np.ascontiguousarray(x)).cuda()      # noqa: E731
    slots = np.array([4, 9, -1, 0, 7, 2], np.int32)      # row 2 of the batch has no request
    first = random_problem(rng, lens=[1], H=H, HV=HV, K=128, V=128, pad=())
    pool_ref = (rng.standard_normal((SLOTS, HV, 128, 128)) * 0.1).astype(np.float32)
    z = lambda *s, dtype=I32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    d = dict(lengths=z(n), context=z(n), slots=gpu(slots), cu=z(n + 1), idx=z(n), seq=z(capacity), pos=z(capacity),
             table=z(n, 40), held=z(n), free=torch.randperm(200, device="cuda").to(I32), head=z(1), held_out=z(n),
             head_out=z(1), place=z(capacity, dtype=torch.int64), q=bf(capacity, H, 128), k=bf(capacity, H, 128),
             v=bf(capacity, HV, 128), a=bf(capacity, HV), b=bf(capacity, HV), A_log=gpu(first["A_log"]),
             dt=gpu(first["dt_bias"]), pool=gpu(pool_ref), out=bf(capacity, HV, 128),
             inter=torch.zeros(capacity, HV, 128, 128, device="cuda"), logits=torch.zeros(capacity, VOCAB, device="cuda"),
             probs=torch.zeros(capacity, VOCAB, device="cuda"), temps=torch.ones(n, device="cuda"),
             draft=torch.zeros(n, DRAFTS, VOCAB, device="cuda"), tokens=z(n, DRAFTS), u=torch.zeros(n, DRAFTS + 1, device="cuda"),
             emitted=z(n, DRAFTS + 1), num=z(n), status=z(1))

    def step():
        spec.step_maps(d["lengths"], d["context"], d["slots"], d["cu"], d["idx"], d["seq"], d["pos"], block_tables=d["table"],
                       blocks_held=d["held"], free_blocks=d["free"], free_head=d["head"], blocks_held_out=d["held_out"],
                       free_head_out=d["head_out"], slot_map=d["place"], block_size=block, device_status=d["status"])
        binding.decode_update(d["q"], d["k"], d["v"], d["a"], d["b"], d["A_log"], d["dt"], d["pool"], d["idx"], d["cu"], d["out"],
                              flags=binding.L2NORM_QK | binding.NO_FINAL_WRITEBACK, intermediate_states=d["inter"],
                              device_status=d["status"])
        spec.token_probs(d["logits"], d["probs"], d["temps"], d["seq"], device_status=d["status"])
        spec.verify_drafts(d["probs"], d["tokens"], d["draft"], d["u"], d["emitted"], d["num"], cu_seqlens=d["cu"],
                           state_indices=d["idx"], device_status=d["status"])
        spec.commit_states(d["inter"], d["num"], d["pool"], d["idx"], cu_seqlens=d["cu"], device_status=d["status"])
        d["context"].add_(d["num"])
        d["held"].copy_(d["held_out"])
        d["head"].copy_(d["head_out"])

    graph = None
    context, kept_all = np.zeros(n, np.int64), []
    for turn in range(5):
        p, target, draft, tokens, u = draw_step(rng, n, capacity)
        lengths = rng.integers(1, DRAFTS + 2, n).astype(np.int32)
        lengths[turn % n] = 0                            # one request waits
        for name in ("q", "k", "v", "a", "b"):
            d[name].copy_(bf16_tensor(p[name]))
        for name, x in (("logits", target), ("draft", draft), ("tokens", tokens), ("u", u), ("lengths", lengths)):
            d[name].copy_(gpu(x))
        temps = np.where(np.arange(n) == 1, 0.0, 1.0).astype(np.float32)      # request 1 is greedy
        d["temps"].copy_(gpu(temps))
        if as_graph and graph is None:
            torch.cuda.synchronize()
            keep = {k: d[k].clone() for k in ("pool", "context", "held", "head", "table")}
            step()                                       # loads the libraries before the capture
            for k, v in keep.items():
                d[k].copy_(v)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        graph.replay() if graph is not None else step()
        torch.cuda.synchronize()
        assert int(d["status"]) == 0

        # the same step from the definitions
        runs = np.where(slots >= 0, lengths, 0)
        cu = np.concatenate([[0], np.cumsum(runs)])
        assert np.array_equal(d["cu"].cpu().numpy(), cu)
        idx = np.where(runs > 0, slots, -1).astype(np.int32)
        assert np.array_equal(d["idx"].cpu().numpy(), idx)
        probs = d["probs"].double().cpu().numpy()
        emitted, num, _ = spec_plain.verify(probs, tokens, draft.astype(np.float64), u.astype(np.float64), cu, idx)
        assert np.array_equal(d["emitted"].cpu().numpy(), emitted) and np.array_equal(d["num"].cpu().numpy(), num)
        greedy = target[cu[1] + num[1] - 1] if num[1] else None
        if greedy is not None:
            assert emitted[1, num[1] - 1] == int(np.argmax(greedy))
        context += num
        assert np.array_equal(d["context"].cpu().numpy(), context)
        live = num > 0
        rows = np.concatenate([np.arange(cu[i], cu[i] + num[i]) for i in range(n)]).astype(np.int64)
        kept = dict(q=p["q"][rows], k=p["k"][rows], v=p["v"][rows], a=p["a"][rows], b=p["b"][rows], A_log=first["A_log"],
                    dt_bias=first["dt_bias"], state_pool=pool_ref, state_indices=np.where(live, idx, -1).astype(np.int32),
                    cu_seqlens=np.concatenate([[0], np.cumsum(num)]).astype(np.int32))
        status, o_ref, s_ref, _ = oracle_on(kept)
        assert status == 0
        assert_out_close(d["out"].float().cpu().numpy()[rows], o_ref, f"step {turn} out")
        assert_state_close(d["pool"].cpu().numpy(), s_ref, f"step {turn} state")
        pool_ref = s_ref.astype(np.float32)
        # every kept token's place in the cache is its request's own block
        table, held = d["table"].cpu().numpy(), d["held"].cpu().numpy()
        place, pos = d["place"].cpu().numpy(), d["pos"].cpu().numpy()
        for i in range(n):
            for r in range(cu[i], cu[i + 1]):
                assert place[r] == table[i, pos[r] // block] * block + pos[r] % block and pos[r] // block < held[i]
        used = np.concatenate([table[i, : held[i]] for i in range(n)])
        assert len(set(used.tolist())) == len(used) == int(d["head"])
        kept_all.append(num.sum())
    assert sum(kept_all) > 5 * (n - 2)                   # drafts were accepted, not only drawn
