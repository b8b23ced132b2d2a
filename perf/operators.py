"""The operators of a speculative decode step around the state update, measured.

``token_probs`` turns a step's logits into probabilities, ``verify_drafts``
judges the drafted tokens and draws the next one, ``commit_states`` puts the
state of the last kept token into the pool, ``step_maps`` builds the next
step's index arrays from the requests' lengths.  ``run`` computes each in its
plain form (elementary torch operations) or, with ``own`` set, through the
package's prepared calls.  K = V = 128 throughout.
"""
import math

import numpy as np
import torch

own = False

HEAD = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# share of sequences with a rejected draft in make_verify's inputs (measured
# over the listed cases): those need a row of the draft's probabilities too
REJECTED = 0.33


def listed():
    return [
        # one request's next-token distribution, the latency end
        dict(name="probs_one", op="probs", rows=1, vocab=32768, dtype="bf16", out="f32", greedy=0.0, masked=0.0, skip=0.0),
        # 128 sequences of 4 fed tokens: every row of a speculative step
        dict(name="probs_b128_t4", op="probs", rows=512, vocab=131072, dtype="bf16", out="f32", greedy=0.1, masked=0.0, skip=0.0),
        # odd vocabulary, a mask over part of it, rows of a padded batch left alone
        dict(name="probs_odd_masked", op="probs", rows=200, vocab=50021, dtype="f32", out="f32", greedy=0.2, masked=0.5, skip=0.1),
        # one request, three drafts
        dict(name="verify_one", op="verify", n=1, drafts=3, vocab=32768, dtype="f32", onehot=False, varlen=False),
        # the speculative batch of the decode benchmark
        dict(name="verify_b128_t4", op="verify", n=128, drafts=3, vocab=131072, dtype="f32", onehot=False, varlen=False),
        # drafts looked up in the text (no draft distribution), ragged, odd vocabulary
        dict(name="verify_ragged_lookup", op="verify", n=96, drafts=7, vocab=50021, dtype="bf16", onehot=True, varlen=True),
        # the tiny batch's states
        dict(name="commit_b4_t4", op="commit", n=4, tokens=4, heads=4, pad=0.0, varlen=False),
        # the speculative batch of the decode benchmark
        dict(name="commit_b128_t4", op="commit", n=128, tokens=4, heads=8, pad=0.0, varlen=False),
        # a full decode batch with padded rows and ragged drafts
        dict(name="commit_b512_ragged", op="commit", n=512, tokens=5, heads=8, pad=0.05, varlen=True),
        # index arrays of the speculative batch
        dict(name="maps_b128_t4", op="maps", n=128, longest=4, block=16, cached=2048),
        # the varlen sweep's batch: 1024 requests of 1 to 64 tokens
        dict(name="maps_b1024_varlen", op="maps", n=1024, longest=64, block=16, cached=4096),
        # a prefill batch
        dict(name="maps_prefill", op="maps", n=96, longest=4096, block=64, cached=8192),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("probs", "verify", "commit", "maps"))
    if op == "probs":
        rows = log_int(rng, 1, 512)
        return dict(op=op, rows=rows, vocab=log_int(rng, 500, 131072), dtype=rng.choice(("bf16", "f32")), out=rng.choice(("f32", "f32", "bf16")),
                    greedy=rng.choice((0.0, 0.3)), masked=rng.choice((0.0, 0.7)), skip=rng.choice((0.0, 0.1)))
    if op == "verify":
        return dict(op=op, n=log_int(rng, 1, 128), drafts=rng.randint(0, 7), vocab=log_int(rng, 500, 131072), dtype=rng.choice(("bf16", "f32")),
                    onehot=rng.random() < 0.3, varlen=rng.random() < 0.5)
    if op == "commit":
        heads = rng.choice((2, 4, 8, 16, 32))
        return dict(op=op, n=log_int(rng, 1, 2560 // heads), tokens=rng.randint(1, 8), heads=heads, pad=rng.choice((0.0, 0.1)), varlen=rng.random() < 0.5)
    n = log_int(rng, 1, 1024)
    return dict(op=op, n=n, longest=log_int(rng, 1, max(2, min(4096, 196608 // n))), block=rng.choice((1, 16, 24, 32, 64, 128)), cached=rng.choice((64, 1024, 8192)))


# ---------------------------------------------------------------- inputs

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)


def make_probs(case, seed):
    g = generator(seed)
    rows, vocab = case["rows"], case["vocab"]
    x = torch.randn(rows, vocab, device="cuda", generator=g) * 3
    x[:, : max(1, vocab // 997)] += 4            # a few likely tokens, as a trained model's rows have
    if case["masked"]:
        x.masked_fill_(torch.rand(rows, vocab, device="cuda", generator=g) < case["masked"], -math.inf)
    n = max(1, rows // 4)                        # four rows a sequence
    seq = torch.arange(rows, device="cuda", dtype=torch.int32).div(4, rounding_mode="floor").clamp_(max=n - 1).to(torch.int32)
    skipped = int(case["skip"] * rows)
    if skipped:                                  # rows behind the last sequence
        seq[rows - skipped:] = -1
    temp = torch.rand(n, device="cuda", generator=g) * 0.8 + 0.4
    greedy = int(case["greedy"] * n)
    if greedy:
        temp[torch.randperm(n, device="cuda", generator=g)[:greedy]] = 0
    return dict(logits=x.to(DTYPES[case["dtype"]]), temperature=temp, row_seq=seq, skipped=skipped,
                probs=torch.zeros(rows, vocab, device="cuda", dtype=DTYPES[case["out"]]))


def lengths_of(case, g):
    """Fed tokens per sequence (the last token and the drafts), and cu_seqlens."""
    most = case["drafts"] + 1 if case["op"] == "verify" else case["tokens"]
    if case["varlen"]:
        lens = torch.randint(1, most + 1, (case["n"],), device="cuda", generator=g, dtype=torch.int32)
    else:
        lens = torch.full((case["n"],), most, device="cuda", dtype=torch.int32)
    cu = torch.zeros(case["n"] + 1, device="cuda", dtype=torch.int32)
    cu[1:] = lens.cumsum(0)
    return lens, cu, most


def make_verify(case, seed):
    g = generator(seed)
    n, d, vocab, dt = case["n"], case["drafts"], case["vocab"], DTYPES[case["dtype"]]
    lens, cu, _ = lengths_of(case, g)
    total = int(cu[-1])
    target = torch.randn(total, vocab, device="cuda", generator=g) * 2.5
    target[:, : max(1, vocab // 499)] += 3
    favoured = torch.randint(vocab, (total, 1), device="cuda", generator=g)   # one likely token a row, more or less so
    target.scatter_add_(1, favoured, math.log(vocab) + 3 + 2 * torch.randn(total, 1, device="cuda", generator=g))
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), lens.long(), output_size=total)
    at = torch.arange(total, device="cuda") - cu[seq].long()
    draft = torch.zeros(n, d, vocab, device="cuda")
    inner = at < d
    draft[seq[inner], at[inner]] = target[inner] + torch.randn(int(inner.sum()), vocab, device="cuda", generator=g) * 0.5
    target = torch.softmax(target, -1)
    draft = torch.softmax(draft, -1)
    noise = -torch.log(torch.rand(n, d, vocab, device="cuda", generator=g).clamp_(min=1e-30)) if d else draft
    tokens = (draft / noise).argmax(-1).to(torch.int32) if d else torch.zeros(n, 0, device="cuda", dtype=torch.int32)
    uniforms = torch.rand(n, d + 1, device="cuda", generator=g)
    return dict(target=target.to(dt), tokens=tokens, draft=None if case["onehot"] or not d else draft.to(dt), uniforms=uniforms, cu=cu,
                out=torch.empty(n, d + 1, device="cuda", dtype=torch.int32), num=torch.empty(n, device="cuda", dtype=torch.int32))


def make_commit(case, seed):
    g = generator(seed)
    n, heads = case["n"], case["heads"]
    lens, cu, _ = lengths_of(case, g)
    total = int(cu[-1])
    indices = torch.randperm(2 * n, device="cuda", generator=g)[:n].to(torch.int32)
    padded = int(case["pad"] * n)
    if padded:
        indices[torch.randperm(n, device="cuda", generator=g)[:padded]] = -1
    kept = (torch.rand(n, device="cuda", generator=g) * lens).to(torch.int32).clamp_(max=lens - 1) + 1
    inter = torch.randn(total, heads, HEAD, HEAD, device="cuda", generator=g) * 0.1
    pool = torch.randn(2 * n, heads, HEAD, HEAD, device="cuda", generator=g) * 0.1
    return dict(inter=inter, pool=pool, kept=kept, indices=indices, cu=cu)


def make_maps(case, seed):
    g = generator(seed)
    n, block = case["n"], case["block"]
    ints = lambda lo, hi: torch.randint(lo, hi + 1, (n,), device="cuda", generator=g, dtype=torch.int32)  # noqa: E731
    lengths = ints(1, case["longest"])
    lengths[torch.rand(n, device="cuda", generator=g) < 0.05] = 0         # requests that wait
    context = ints(0, case["cached"])
    held = (context + block - 1) // block + ints(0, 1)
    slots = torch.randperm(2 * n, device="cuda", generator=g)[:n].to(torch.int32)
    slots[torch.rand(n, device="cuda", generator=g) < 0.03] = -1          # rows of the batch without a request
    wide = (case["cached"] + case["longest"]) // block + 2
    blocks = torch.randperm(n * wide + 64, device="cuda", generator=g).to(torch.int32)
    table = torch.where(torch.arange(wide, device="cuda") < held[:, None], blocks[: n * wide].view(n, wide), -1).to(torch.int32)
    free = blocks.flip(0).clone()                                         # ids of its own: only their use is measured
    capacity = -(-max(1, n * (case["longest"] + 1) // 2 + 3 * case["longest"] + 8) // 64) * 64
    capacity = max(capacity, -(-int(lengths.sum()) // 64) * 64)
    new = lambda *shape, dtype=torch.int32: torch.empty(*shape, device="cuda", dtype=dtype)  # noqa: E731
    return dict(lengths=lengths, context=context, slots=slots, table=table, held=held.to(torch.int32), free=free,
                head=torch.full((1,), 7, device="cuda", dtype=torch.int32), block=block, cu=new(n + 1), indices=new(n), row_seq=new(capacity),
                positions=new(capacity), slot_map=new(capacity, dtype=torch.int64), held_out=new(n), head_out=new(1), capacity=capacity)


MAKE = {"probs": make_probs, "verify": make_verify, "commit": make_commit, "maps": make_maps}


def prepare(case, seed):
    s = MAKE[case["op"]](case, seed)
    s["op"] = case["op"]
    if own:
        from gated_deltanet_recurrent_sigmoid_b200 import speculative
        s["call"] = {"probs": own_probs, "verify": own_verify, "commit": own_commit, "maps": own_maps}[case["op"]](speculative, s)
    return s


# ---------------------------------------------------------------- the framework's calls

def own_probs(spec, s):
    return spec.PreparedTokenProbs(s["logits"], s["probs"], temperature=s["temperature"], row_seq=s["row_seq"])


def own_verify(spec, s):
    return spec.PreparedVerifyDrafts(s["target"], s["tokens"], s["draft"], s["uniforms"], s["out"], s["num"], cu_seqlens=s["cu"])


def own_commit(spec, s):
    return spec.PreparedCommitStates(s["inter"], s["kept"], s["pool"], s["indices"], cu_seqlens=s["cu"])


def own_maps(spec, s):
    return spec.PreparedStepMaps(s["lengths"], s["context"], s["slots"], s["cu"], s["indices"], s["row_seq"], s["positions"],
                                 block_tables=s["table"], blocks_held=s["held"], free_blocks=s["free"], free_head=s["head"],
                                 blocks_held_out=s["held_out"], free_head_out=s["head_out"], slot_map=s["slot_map"], block_size=s["block"])


# ---------------------------------------------------------------- plain forms

def plain_probs(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    x = torch.where(torch.isnan(x), -math.inf, x)
    top = x.amax(-1, keepdim=True)
    t = s["temperature"][s["row_seq"].clamp(min=0).long()][:, None]
    e = torch.where(x == top, 1.0, torch.exp((x - top) / torch.where(t > 0, t, 1.0)))
    e = torch.where(x == -math.inf, 0.0, e)                               # rows with nothing left: zeros
    p = e / e.sum(-1, keepdim=True).clamp(min=1)
    column = torch.arange(vocab, device=x.device)
    first = torch.where((x == top) & (x > -math.inf), column, vocab).amin(-1, keepdim=True)
    p = torch.where(t > 0, p, (column == first).float())
    if s["skipped"]:
        s["probs"][: rows - s["skipped"]] = p[: rows - s["skipped"]].to(s["probs"].dtype)
        return s["probs"]
    return p.to(s["probs"].dtype)


def plain_verify(s):
    target, draft, cu, u = s["target"], s["draft"], s["cu"].long(), s["uniforms"].double()
    n, d = s["tokens"].shape
    vocab = target.shape[1]
    lens = cu[1:] - cu[:-1] - 1                                           # drafts of each sequence
    j = torch.arange(d, device=target.device)
    x = s["tokens"].long()
    row = (cu[:-1, None] + j).clamp(max=target.shape[0] - 1)
    p = target[row, x].double()
    q = torch.ones_like(p) if draft is None else draft.gather(2, x[..., None])[..., 0].double()
    accept = (u[:, :d] * q < p) & (j < lens[:, None])
    kept = accept.long().cumprod(1).sum(1)                                # accepted before the first rejection
    w = target[cu[:-1] + kept].double()
    rejected = (kept < lens)[:, None]
    if d:
        i = torch.arange(n, device=target.device)
        at = kept.clamp(max=d - 1)
        if draft is None:
            less = torch.where(torch.arange(vocab, device=target.device) == x[i, at][:, None], 0.0, w)
        else:
            less = (w - draft[i, at].double()).clamp(min=0)
        less = torch.where(less.sum(1, keepdim=True) > 0, less, w)
        w = torch.where(rejected, less, w)
    below = w.cumsum(1)
    drawn = (below > u[:, d:] * below[:, -1:]).to(torch.int32).argmax(1)
    slot = torch.arange(d + 1, device=target.device)
    padded = torch.cat((x, torch.full((n, 1), -1, device=x.device)), 1)
    out = torch.where(slot < kept[:, None], padded, torch.where(slot == kept[:, None], drawn[:, None], -1))
    return out.to(torch.int32), (kept + 1).to(torch.int32)


def plain_commit(s):
    row = s["cu"][:-1].long() + s["kept"].long() - 1
    slot = s["indices"].long()
    slots = s["pool"].shape[0]
    # a padded row (-1) must write nothing: its state goes to the place of a
    # live row, with that row's own state
    live = slot >= 0
    some = live.to(torch.int32).argmax()
    s["pool"][torch.where(live, slot, slot[some]).clamp(0, slots - 1)] = s["inter"][torch.where(live, row, row[some])]
    return s["pool"]


def plain_maps(s):
    dev, block = s["lengths"].device, s["block"]
    runs = torch.where(s["slots"] >= 0, s["lengths"], 0).long()
    cu = torch.zeros(runs.numel() + 1, device=dev, dtype=torch.int64)
    cu[1:] = runs.cumsum(0)
    context, held = s["context"].long(), s["held"].long()
    needed = torch.where(runs > 0, (context + runs + block - 1) // block, 0)
    fresh = (needed - held).clamp(min=0)
    offset = s["head"].long() + fresh.cumsum(0) - fresh
    column = torch.arange(s["table"].shape[1], device=dev)
    ids = s["free"][(offset[:, None] + column - held[:, None]).clamp(0, s["free"].numel() - 1)]
    new = (column >= held[:, None]) & (column < (held + fresh)[:, None])
    s["table"].copy_(torch.where(new, ids, s["table"]))
    t = torch.arange(s["capacity"], device=dev)
    inside = t < cu[-1]
    seq = torch.searchsorted(cu[1:], t, right=True).clamp(max=runs.numel() - 1)
    position = context[seq] + t - cu[seq]
    slot = s["table"][seq, (position // block).clamp(0, s["table"].shape[1] - 1)].long() * block + position % block
    mark = lambda v: torch.where(inside, v, -1)                           # noqa: E731
    return dict(cu_seqlens=cu.to(torch.int32), state_indices=torch.where(runs > 0, s["slots"], -1).to(torch.int32), row_seq=mark(seq).to(torch.int32),
                positions=mark(position).to(torch.int32), slot_map=mark(slot), block_tables=s["table"], blocks_held=(held + fresh).to(torch.int32),
                free_head=(s["head"].long() + fresh.sum()).to(torch.int32))


PLAIN = {"probs": plain_probs, "verify": plain_verify, "commit": plain_commit, "maps": plain_maps}


def run(state):
    op = state["op"]
    if not own:
        return PLAIN[op](state)
    state["call"]()
    if op == "probs":
        return state["probs"]
    if op == "verify":
        return state["out"], state["num"]
    if op == "commit":
        return state["pool"]
    return dict(cu_seqlens=state["cu"], state_indices=state["indices"], row_seq=state["row_seq"], positions=state["positions"],
                slot_map=state["slot_map"], block_tables=state["table"], blocks_held=state["held_out"], free_head=state["head_out"])


# ---------------------------------------------------------------- floors

def work(case):
    size = lambda name: 2 if name == "bf16" else 4                        # noqa: E731
    if case["op"] == "probs":
        n = (case["rows"] - int(case["skip"] * case["rows"])) * case["vocab"]
        return dict(bytes=n * (size(case["dtype"]) + size(case["out"])), flops=5 * n)
    if case["op"] == "verify":
        rows = case["n"] * (1 if case["onehot"] or not case["drafts"] else 1 + REJECTED)
        return dict(bytes=rows * case["vocab"] * size(case["dtype"]) + 16 * case["n"] * (case["drafts"] + 1), flops=2 * rows * case["vocab"])
    if case["op"] == "commit":
        live = case["n"] - int(case["pad"] * case["n"])
        return dict(bytes=2 * live * case["heads"] * HEAD * HEAD * 4 + 16 * case["n"], flops=0)
    rows = 0.95 * 0.97 * case["n"] * (case["longest"] + 1) / 2
    return dict(bytes=16 * rows + 8 * rows / case["block"] + 28 * case["n"], flops=10 * rows)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = MAKE[case["op"]](case, seed)
    return {"probs": exact_probs, "verify": exact_verify, "commit": exact_commit, "maps": exact_maps}[case["op"]](s)


def exact_probs(s):
    x = s["logits"].double()
    seq = s["row_seq"].cpu().tolist()
    temp = s["temperature"].double().cpu().tolist()
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for r, i in enumerate(seq):
        if i < 0 or not bool((x[r] > -math.inf).any()):
            continue
        if temp[i] == 0:
            out[r, int(np.argmax(x[r].cpu().numpy()))] = 1
        else:
            out[r] = torch.softmax(x[r] / temp[i], 0)
    return out


def exact_verify(s):
    cu = s["cu"].cpu().numpy()
    x, u = s["tokens"].cpu().numpy(), s["uniforms"].double().cpu().numpy()
    n, d = x.shape
    out, num = np.full((n, d + 1), -1, np.int32), np.zeros(n, np.int32)
    for i in range(n):
        a, last = 0, int(cu[i + 1] - cu[i]) - 1
        while True:
            p = s["target"][int(cu[i]) + a].double().cpu().numpy()
            if a == last:
                w = p
                break
            v = int(x[i, a])
            q = np.eye(1, len(p), v)[0] if s["draft"] is None else s["draft"][i, a].double().cpu().numpy()
            if not u[i, a] * q[v] < p[v]:
                w = np.maximum(p - q, 0)
                if s["draft"] is None:
                    w[v] = 0
                w = w if w.sum() > 0 else p
                break
            out[i, a] = v
            a += 1
        below = np.cumsum(w)
        out[i, a] = int(np.argmax(below > u[i, d] * below[-1]))
        num[i] = a + 1
    return torch.from_numpy(out), torch.from_numpy(num)


def exact_commit(s):
    pool, cu = s["pool"].double(), s["cu"].cpu().tolist()
    for i, (slot, kept) in enumerate(zip(s["indices"].cpu().tolist(), s["kept"].cpu().tolist())):
        if slot >= 0 and kept > 0:
            pool[slot] = s["inter"][cu[i] + kept - 1].double()
    return pool


def exact_maps(s):
    table, free, block, cap = s["table"].cpu().clone(), s["free"].cpu().tolist(), s["block"], s["capacity"]
    head = int(s["head"])
    cu, indices, held_out = [0], [], []
    row_seq, positions, slot_map = [-1] * cap, [-1] * cap, [-1] * cap
    at = 0
    for i, (length, context, slot, held) in enumerate(zip(*(s[k].cpu().tolist() for k in ("lengths", "context", "slots", "held")))):
        length = length if slot >= 0 else 0
        indices.append(slot if length else -1)
        if length:
            while held * block < context + length:
                table[i, held] = free[head]
                held, head = held + 1, head + 1
            line = table[i].tolist()
            for k in range(length):
                row_seq[at], positions[at] = i, context + k
                slot_map[at] = line[(context + k) // block] * block + (context + k) % block
                at += 1
        held_out.append(held)
        cu.append(at)
    ints = lambda v: torch.tensor(v, dtype=torch.int32)                   # noqa: E731
    return dict(cu_seqlens=ints(cu), state_indices=ints(indices), row_seq=ints(row_seq), positions=ints(positions),
                slot_map=torch.tensor(slot_map, dtype=torch.int64), block_tables=table, blocks_held=ints(held_out), free_head=ints([head]))
