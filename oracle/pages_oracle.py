"""CPU oracle for the cache-page operators (include/pa_pages.h).

TEST INFRASTRUCTURE ONLY: plain loops over numpy arrays, one sequence and one
page at a time, in the order the definitions state. Every function changes
the arrays it is given and returns the error bits. ``caches`` is a list of
arrays ``[num_blocks, block_size, ...]``."""
from __future__ import annotations

import numpy as np

POOL, PAGE, CONTEXT, CUMSEQ = 0x100, 0x200, 0x20, 0x08


def copy(caches, src, dst, rows, bs):
    nb, err = caches[0].shape[0], 0
    n = len(src)
    rows = [bs] * n if rows is None else list(rows)
    fine = [0 <= src[i] < nb and 0 <= dst[i] < nb and 0 <= rows[i] <= bs for i in range(n)]
    moves = [i for i in range(n) if fine[i] and src[i] != dst[i]]
    if not all(fine):
        err |= PAGE
    targets = {}
    for i in moves:
        targets.setdefault(int(dst[i]), i)
    old = [c.copy() for c in caches]
    for i in moves:
        if targets[int(dst[i])] != i or int(src[i]) in targets:
            err |= PAGE
            continue
        for c, o in zip(caches, old):
            c[dst[i], :rows[i]] = o[src[i], :rows[i]]
    return err


def free(table, past, ref, seqs):
    err = 0
    for s in seqs:
        if not 0 <= s < len(past):
            err |= PAGE
            continue
        for j in range(table.shape[1]):
            page = table[s, j]
            table[s, j] = -1
            if page == -1:
                continue
            if not 0 <= page < len(ref) or ref[page] <= 0:
                err |= PAGE
            else:
                ref[page] -= 1
        past[s] = 0
    return err


def fork(caches, table, past, ref, parents, children, bs):
    err = 0
    ns, mb = table.shape
    nb = len(ref)
    named = [0 <= p < ns and 0 <= c < ns for p, c in zip(parents, children)]
    first = {}
    for i, ok in enumerate(named):
        if ok:
            first.setdefault(int(children[i]), i)
    start = table.copy(), ref.copy(), past.copy()
    pages = [p for p in range(nb) if ref[p] == 0]
    old = [c.copy() for c in caches]
    for i, ok in enumerate(named):
        p, c = int(parents[i]), int(children[i])
        if not ok or first[c] != i or p in first:
            err |= PAGE
            continue
        ctx = int(start[2][p])
        if ctx < 0 or ctx > mb * bs:
            err |= CONTEXT
            continue
        held = -(-ctx // bs)
        mine = start[0][p, :held]
        if (start[0][c] >= 0).any() or any(not 0 <= q < nb or start[1][q] <= 0 for q in mine):
            err |= PAGE
            continue
        tail = ctx % bs
        if tail and not pages:
            err |= POOL
            continue
        full = ctx // bs
        for j in range(full):
            table[c, j] = start[0][p, j]
            ref[start[0][p, j]] += 1
        past[c] = ctx
        if tail:
            new = pages.pop(0)
            table[c, full] = new
            ref[new] = 1
            for arr, o in zip(caches, old):
                arr[new, :tail] = o[start[0][p, full], :tail]
    return err


def reserve(table, past, ref, cumseq, num_tokens, bs):
    """Returns (error bits, slot_mapping)."""
    err = 0
    ns, mb = table.shape
    nb = len(ref)
    ref0 = ref.copy()
    pages = [p for p in range(nb) if ref[p] == 0]
    total, wanted = len(pages), 0
    slots = np.full(num_tokens, -1, dtype=np.int32)
    for b in range(ns):
        q0, q1, p0 = int(cumseq[b]), int(cumseq[b + 1]), int(past[b])
        if q0 < 0 or q1 < q0 or q1 > num_tokens:
            err |= CUMSEQ
            continue
        if q1 == q0:
            continue
        if p0 < 0 or p0 + q1 - q0 > mb * bs:
            err |= CONTEXT
            continue
        span = range(p0 // bs, (p0 + q1 - q0 - 1) // bs + 1)
        held = [int(table[b, j]) for j in span if table[b, j] != -1]
        if any(not 0 <= p < nb or ref0[p] != 1 for p in held) or \
                (p0 % bs and table[b, p0 // bs] == -1):
            err |= PAGE
            continue
        lack = [j for j in span if table[b, j] == -1]
        wanted += len(lack)
        if lack and wanted > total:
            err |= POOL
            continue
        for j in lack:
            table[b, j] = pages.pop(0)
            ref[table[b, j]] = 1
        for t in range(q0, q1):
            pos = p0 + t - q0
            slots[t] = table[b, pos // bs] * bs + pos % bs
    return err, slots


def compact(caches, table, ref):
    """Returns (error bits, number of held pages)."""
    err = 0
    nb = len(ref)
    live = int((ref != 0).sum())
    to = {p: p for p in range(live) if ref[p] != 0}
    holes = [p for p in range(live) if ref[p] == 0]
    for p in range(live, nb):
        if ref[p] != 0:
            q = holes.pop(0)
            to[p] = q
            for c in caches:
                c[q] = c[p]
            ref[q], ref[p] = ref[p], 0
    for b in range(table.shape[0]):
        for j in range(table.shape[1]):
            if table[b, j] == -1:
                continue
            new = to.get(int(table[b, j]), -1)
            if new < 0:
                err |= PAGE
            table[b, j] = new
    return err, live
