"""fp64 statement of the cache calls: rotary append, chunk attention over a paged cache, path compaction.

Plain numpy over one layer's pages as arrays [pages, page_size, heads, dim]; sequences one after the other,
from the definitions ("All About Transformer Inference", the KV cache and its pages, lines 25-38 and 240-245).
"""
from __future__ import annotations

import numpy as np


def rows_of(seq_offsets, b):
    """First row and tokens of sequence b's chunk."""
    return int(seq_offsets[b]) + b, int(seq_offsets[b + 1]) - int(seq_offsets[b]) + 1


def depths(parents):
    """Depth of every node of one tree (node 0 is the root; parents of nodes 1, 2, ...)."""
    dep = [0]
    for p in parents:
        dep.append(dep[p] + 1)
    return np.array(dep, dtype=np.int64)


def lineage(parents):
    """[T, T] booleans: node i is j itself or an ancestor of j."""
    T = len(parents) + 1
    m = np.zeros((T, T), dtype=bool)
    for j in range(T):
        if j:
            m[j] = m[parents[j - 1]]
        m[j, j] = True
    return m


def _parents(parents, seq_offsets, b, T):
    if parents is None:
        return list(range(T - 1))
    o = int(seq_offsets[b])
    return [int(p) for p in parents[o:o + T - 1]]


def rotate(x, angles, interleaved):
    """x [..., dim] by angles [..., n]: the first 2 n elements are rotated pairwise."""
    y = np.array(x, dtype=np.float64)
    n = angles.shape[-1]
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    u, w = y[..., a].copy(), y[..., b].copy()
    y[..., a] = u * np.cos(angles) - w * np.sin(angles)
    y[..., b] = w * np.cos(angles) + u * np.sin(angles)
    return y


def append(q, k, v, seq_offsets, parents, cached, freq=None, interleaved=False):
    """(rotated q, rotated k, slots, sequence of each row). freq: [n] radians per position, None: no rotation."""
    B = len(cached)
    q, k = np.array(q, dtype=np.float64), np.array(k, dtype=np.float64)
    slots = np.full(len(k), -1, dtype=np.int64)
    seq = np.full(len(k), -1, dtype=np.int64)
    for b in range(B):
        r, T = rows_of(seq_offsets, b)
        dep = depths(_parents(parents, seq_offsets, b, T))
        if freq is not None:
            ang = (int(cached[b]) + dep)[:, None, None] * np.asarray(freq, dtype=np.float64)
            q[r:r + T] = rotate(q[r:r + T], ang, interleaved)
            k[r:r + T] = rotate(k[r:r + T], ang, interleaved)
        slots[r:r + T] = int(cached[b]) + np.arange(T)
        seq[r:r + T] = b
    return q, k, slots, seq


def attend(q, k_pages, v_pages, table, seq_offsets, parents, cached, scale, window=0):
    """(out [rows, hq, D], lse [rows, hq], mean |v| under the weights, score magnitude, weight floor).

    The last three bound what rounding may do: sum w |v| / sum w; the largest sum_d |scale q_d k_d| of a row and
    head; sum |v| / sum w' with w' relative to the largest weight. Pages outside the pool hold nothing.
    """
    q = np.asarray(q, dtype=np.float64)
    R, hq, D = q.shape
    pages, ps, hkv, _ = k_pages.shape
    G = hq // hkv
    out, mean = np.zeros((R, hq, D)), np.zeros((R, hq, D))
    lse, big, floor = np.full((R, hq), -np.inf), np.zeros((R, hq)), np.zeros((R, hq, D))
    for b in range(len(cached)):
        r, T = rows_of(seq_offsets, b)
        past = int(cached[b])
        par = _parents(parents, seq_offsets, b, T)
        dep = depths(par)
        seen = np.concatenate([np.ones((T, past), dtype=bool), lineage(par)], axis=1)
        pos = np.concatenate([np.arange(past), past + dep])
        if window:
            seen &= (past + dep)[:, None] - pos < window
        slot = np.arange(past + T)
        page = table[b][slot // ps].astype(np.int64)
        held = (page >= 0) & (page < pages)
        seen &= held
        need = seen.any(axis=0)  # only what some token sees is ever read
        s = slot[need]
        seen = seen[:, need]
        for h in range(hkv):
            K = np.asarray(k_pages[page[need], s % ps, h], dtype=np.float64)
            V = np.asarray(v_pages[page[need], s % ps, h], dtype=np.float64)
            for g in range(h * G, h * G + G):
                z = scale * (q[r:r + T, g] @ K.T)
                mag = abs(scale) * (np.abs(q[r:r + T, g]) @ np.abs(K).T)
                for j in range(T):
                    m = seen[j]
                    if not m.any():
                        continue
                    top = z[j, m].max()
                    e = np.exp(z[j, m] - top)
                    out[r + j, g] = e @ V[m] / e.sum()
                    mean[r + j, g] = e @ np.abs(V[m]) / e.sum()
                    floor[r + j, g] = np.abs(V[m]).sum(axis=0) / e.sum()
                    lse[r + j, g] = top + np.log(e.sum())
                    big[r + j, g] = mag[j, m].max()
    return out, lse, mean, big, floor


def compact(pages_kv, table, seq_offsets, cached, accepted, path):
    """Pages [..., pages, page_size, heads, dim] after the accepted paths moved, and the new lengths."""
    x = np.array(pages_kv)
    ps = x.shape[-3]
    now = np.array(cached).copy()
    for b, n in enumerate(int(a) for a in accepted):
        if n < 0:
            continue
        past, o = int(cached[b]), int(seq_offsets[b])
        old = x.copy() if path is not None else x
        for j in range(n if path is not None else 0):
            a, z = past + int(path[o + j]), past + 1 + j
            x[..., table[b][z // ps], z % ps, :, :] = old[..., table[b][a // ps], a % ps, :, :]
        now[b] = past + n + 1
    return x, now


def reserve(table, queue, held, state, want, page_size):
    """Pages for sequences that are to hold `want` slots each (None: a sequence with a finding): (table, queue, held,
    state, sequences that went without). Plain lists, one page after the other. Entries that a sequence wants and does
    not get are -1 in the table."""
    table, queue = np.array(table), np.array(queue)
    pages, width = len(queue), table.shape[1]
    head, count = int(state[0]), int(state[1])
    need = []

    def none(b):
        if want[b] is not None and want[b] >= 0 and held[b] >= 0:
            table[b, int(held[b]):-(-want[b] // page_size)] = -1
    for b, n in enumerate(want):
        ok = n is not None and n >= 0 and 0 <= held[b] <= width and -(-n // page_size) <= width
        need.append(-(-n // page_size) if ok else None)
    give = sum(int(held[b]) - n for b, n in enumerate(need) if n is not None and n < held[b])
    if not 0 <= head < pages or count < 0 or count + give > pages:
        for b in range(len(want)):
            none(b)
        return table, queue, np.array(held), np.array(state), set(range(len(want)))
    for b, n in enumerate(need):
        for i in range(n if n is not None else width, int(held[b]) if n is not None else 0):
            queue[(head + count) % pages] = table[b, i]
            count += 1
    now, without, dry = np.array(held), set(), False
    for b, n in enumerate(need):
        if n is None:
            without.add(b)
            none(b)
            continue
        lack = n - int(held[b])
        if lack > 0:
            dry = dry or lack > count
            if dry:
                without.add(b)
                none(b)
                continue
            for i in range(int(held[b]), n):
                table[b, i] = queue[head]
                head, count = (head + 1) % pages, count - 1
        now[b] = n
    return table, queue, now, np.array([head, count]), without


def attend_scored(q, k_pages, v_pages, table, seq_offsets, parents, cached, scale, window=0, cap=0.0, slopes=None,
                  prefix=None):
    """attend on scores capped by a tanh, less slopes[head] |distance|, slots before prefix[b] seen by every token.

    (out, lse, mean |v|, score magnitude before the cap, weight floor, largest bias of a slot whose weight is not below
    2^-30 of the row's largest).
    """
    q = np.asarray(q, dtype=np.float64)
    R, hq, D = q.shape
    pages, ps, hkv, _ = k_pages.shape
    G = hq // hkv
    out, mean, floor = (np.zeros((R, hq, D)) for _ in range(3))
    lse, big, bias = np.full((R, hq), -np.inf), np.zeros((R, hq)), np.zeros((R, hq))
    for b in range(len(cached)):
        r, T = rows_of(seq_offsets, b)
        past = int(cached[b])
        par = _parents(parents, seq_offsets, b, T)
        slot = np.arange(past + T)
        pos = np.concatenate([slot[:past], past + depths(par)])
        seen = np.concatenate([np.ones((T, past), dtype=bool), lineage(par)], axis=1)
        if prefix is not None:
            seen |= slot < int(prefix[b])
        apart = pos[past:, None] - pos
        if window:
            seen &= apart < window
        page = table[b][slot // ps].astype(np.int64)
        seen &= (page >= 0) & (page < pages)
        need = seen.any(axis=0)
        s, seen, apart = slot[need], seen[:, need], np.abs(apart[:, need]).astype(np.float64)
        for h in range(hkv):
            K = np.asarray(k_pages[page[need], s % ps, h], dtype=np.float64)
            V = np.asarray(v_pages[page[need], s % ps, h], dtype=np.float64)
            for g in range(h * G, h * G + G):
                z = scale * (q[r:r + T, g] @ K.T)
                mag = abs(scale) * (np.abs(q[r:r + T, g]) @ np.abs(K).T)
                if cap:
                    z = cap * np.tanh(z / cap)
                d = np.zeros_like(apart) if slopes is None else float(slopes[g]) * apart
                z = np.where(seen, z - d, -np.inf)
                for j in range(T):
                    if not seen[j].any():
                        continue
                    top = z[j].max()
                    e = np.exp(z[j] - top)
                    m = seen[j]
                    out[r + j, g] = e[m] @ V[m] / e.sum()
                    mean[r + j, g] = e[m] @ np.abs(V[m]) / e.sum()
                    floor[r + j, g] = np.abs(V[m]).sum(axis=0) / e.sum()
                    lse[r + j, g] = top + np.log(e.sum())
                    big[r + j, g] = mag[j, m].max()
                    bias[r + j, g] = np.abs(d[j, e > 2.0 ** -30]).max()
    return out, lse, mean, big, floor, bias
