"""The operators of a speculative step from their definitions, in 64 bits on
the host (TEST INFRASTRUCTURE): plain loops, no code of the package."""
import numpy as np

DEV_BAD_SLOT, DEV_BAD_SEQLENS = 1, 2
DEV_BAD_SEQ, DEV_BAD_TEMPERATURE, DEV_BAD_TOKEN, DEV_BAD_PROBS = 8, 16, 32, 64
DEV_BAD_COUNT, DEV_BAD_LENGTH, DEV_BAD_BLOCKS, DEV_NO_ROOM = 128, 256, 512, 1024


def probs(logits, temperature, row_seq, before):
    """(probabilities [R, V] in fp64 over ``before``, status).  logits fp64."""
    out, status = np.array(before, dtype=np.float64), 0
    for r, x in enumerate(logits):
        t = 1.0
        if temperature is not None:
            i = r if row_seq is None else int(row_seq[r])
            if i < 0 or i >= len(temperature):
                status |= DEV_BAD_SEQ if i != -1 else 0
                continue
            t = float(temperature[i])
        out[r] = 0
        if not 0 <= t < np.inf:
            status |= DEV_BAD_TEMPERATURE
            continue
        x = np.where(np.isnan(x), -np.inf, x)
        top = x.max()
        if top == -np.inf:
            continue
        if t == 0:
            out[r, int(np.flatnonzero(x == top)[0])] = 1
            continue
        if top == np.inf:
            e = (x == top).astype(np.float64)
        else:
            e = np.exp((x - top) / t)
        out[r] = e / e.sum()
    return out, status


def weights(p, q):
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(p) & np.isfinite(q) & (p > q), p - q, 0.0)


def verify(target, tokens, draft, uniforms, cu, indices=None):
    """(out_tokens, num_tokens, status).  target [T_tot, V], draft [N, D, V]
    or None, uniforms: fp64 values of the inputs."""
    n, d_max = tokens.shape
    rows, vocab = target.shape
    out, num, status = np.full((n, d_max + 1), -1, np.int32), np.zeros(n, np.int32), 0
    for i in range(n):
        a, b = int(cu[i]), int(cu[i + 1])
        if a < 0 or b < a or b > rows or b - a > d_max + 1:
            status |= DEV_BAD_SEQLENS
            continue
        if b == a or (indices is not None and indices[i] < 0):
            continue
        kept, w = 0, None
        while w is None:
            p = target[a + kept].astype(np.float64)
            if kept == b - a - 1:
                w = weights(p, np.zeros(vocab))
                break
            x = int(tokens[i, kept])
            if not 0 <= x < vocab:
                status |= DEV_BAD_TOKEN if x != -1 else 0
                w = weights(p, np.zeros(vocab))
                break
            q = draft[i, kept].astype(np.float64) if draft is not None else None
            if uniforms[i, kept] * (q[x] if q is not None else 1.0) < p[x]:
                out[i, kept] = x
                kept += 1
                continue
            w = weights(p, q if q is not None else np.zeros(vocab))
            if q is None:
                w[x] = 0
            if not w.sum() > 0:
                w = weights(p, np.zeros(vocab))
        num[i] = kept + 1
        below = np.cumsum(w)
        if not below[-1] > 0:
            status |= DEV_BAD_PROBS
            continue
        u = uniforms[i, d_max]
        u = 0.0 if np.isnan(u) else max(u, 0.0)
        over = np.flatnonzero(below > u * below[-1])
        out[i, kept] = over[0] if len(over) else np.flatnonzero(w > 0)[-1]
    return out, num, status


def commit(inter, num, pool, indices, cu):
    pool, status = pool.copy(), 0
    for i, (slot, n) in enumerate(zip(indices, num)):
        if slot == -1:
            continue
        bad = 0
        if slot < -1 or slot >= len(pool):
            bad |= DEV_BAD_SLOT
        if cu[i] < 0 or cu[i + 1] < cu[i] or cu[i + 1] > len(inter):
            bad |= DEV_BAD_SEQLENS
        elif n < 0 or n > cu[i + 1] - cu[i]:
            bad |= DEV_BAD_COUNT
        status |= bad
        if not bad and n:
            pool[slot] = inter[cu[i] + n - 1]
    return pool, status


def maps(lengths, context, slots, capacity, tables=None, held=None, free=None, head=0, block=0):
    """dict of every output array, and the status."""
    n, status = len(lengths), 0
    tables = None if tables is None else tables.copy()
    taken, at, full = head, 0, False
    if tables is not None and not 0 <= head <= len(free):
        status |= DEV_BAD_BLOCKS
        full = True
    cu, indices, held_out = [0], [], []
    row_seq, positions, slot_map = [-1] * capacity, [-1] * capacity, [-1] * capacity
    for i in range(n):
        length, have, slot = int(lengths[i]), int(context[i]), int(slots[i])
        wrong = 0
        if slot < -1:
            wrong |= DEV_BAD_SLOT
        if length < 0 or have < 0 or length + have > 2**31 - 1:
            wrong |= DEV_BAD_LENGTH
        lacks = 0
        if slot != -1 and not wrong and length > 0 and tables is not None:
            need = -(-(have + length) // block)
            if held[i] < 0 or held[i] > tables.shape[1] or int(held[i]) * block < have or need > tables.shape[1]:
                wrong |= DEV_BAD_BLOCKS
            else:
                lacks = max(0, need - int(held[i]))
        if slot != -1:
            status |= wrong
        runs = slot != -1 and not wrong and length > 0
        if runs and (full or at + length > capacity or (tables is not None and taken + lacks > len(free))):
            status |= DEV_NO_ROOM
            full, runs = True, False
        if runs:
            for k in range(lacks):
                tables[i, held[i] + k] = free[taken + k]
            taken += lacks
            for k in range(length):
                pos = have + k
                row_seq[at], positions[at] = i, pos
                if tables is not None:
                    slot_map[at] = int(tables[i, pos // block]) * block + pos % block
                at += 1
        cu.append(at)
        indices.append(slot if runs else -1)
        if tables is not None:
            held_out.append(int(held[i]) + (lacks if runs else 0))
    got = dict(cu_seqlens=np.array(cu, np.int32), state_indices=np.array(indices, np.int32),
               row_seq=np.array(row_seq, np.int32), positions=np.array(positions, np.int32))
    if tables is not None:
        got.update(block_tables=tables, blocks_held_out=np.array(held_out, np.int32),
                   free_head_out=np.array([taken], np.int32), slot_map=np.array(slot_map, np.int64))
    return got, status
