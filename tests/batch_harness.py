"""Plain forms of nexus_plan, nexus_verify and nexus_attend_shared for the tests: whole numbers
by Python's own, attention in 64 bits."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np
import torch

BAD_LEN, BAD_PAGE, BAD_TOKENS, FULL, NO_PAGES, BAD_PROBS = 2, 8, 16, 32, 128, 256


def plan_plain(lens, new_tokens, capacity, *, tokens, max_tokens, page=0, num_pages=0, table=None,
               free=None, count=0, held=None, first_pos=None):
    """lens [layers][seqs][kv_heads], table [seqs][entries], free [num_pages]: numpy, changed in
    place, as held [seqs] is. Returns (cu, token_seq, token_pos, free count, status)."""
    S = lens.shape[1]
    status, n, need, ok = 0, [0] * S, [0] * S, [True] * S
    for s in range(S):
        ends = new_tokens[s] < 0
        n[s] = 0 if ends else int(new_tokens[s])
        flag, rows = 0, 0
        if page and not 0 <= held[s] <= table.shape[1]:
            flag = BAD_PAGE
        elif not ends and (lens[:, s].min() < 0 or lens[:, s].max() > capacity):
            flag = BAD_LEN
        else:
            rows = 0 if ends else int(lens[:, s].max())
            if n[s] > max_tokens:
                flag = BAD_TOKENS
            elif rows + n[s] > capacity:
                flag = FULL
        status |= flag
        ok[s] = not flag
        if page:
            need[s] = -(-(rows + n[s]) // page)
    at = 0                                  # those that the per-token arrays have no room for
    for s in range(S):
        if ok[s] and n[s]:
            at += n[s]
            if at > tokens:
                ok[s], status = False, status | BAD_TOKENS
    if page:
        if not 0 <= count <= num_pages:
            count, status = 0, status | BAD_PAGE
        top = count
        for s in range(S):
            if ok[s]:
                for e in range(need[s], int(held[s])):
                    if top < num_pages:
                        free[top] = table[s, e]
                        top += 1
                    else:
                        status |= BAD_PAGE
        asked, left = 0, top
        for s in range(S):
            more = need[s] - int(held[s])
            if not ok[s] or more <= 0:
                continue
            asked += more
            if asked > top:
                ok[s], status = False, status | NO_PAGES
                continue
            for e in range(int(held[s]), need[s]):
                left -= 1
                table[s, e] = free[left]
        for s in range(S):
            if ok[s]:
                held[s] = need[s]
        count = left
    cu, seq, pos = [0], [], []
    for s in range(S):
        if ok[s]:
            if new_tokens[s] < 0:
                lens[:, s] = 0
            seq += [s] * n[s]
            if first_pos is not None:
                pos += [int(first_pos[s]) + j for j in range(n[s])]
        cu.append(len(seq))
    return cu, seq, pos, count, status


def _unit(x):
    return np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(0), np.float32(1)))


def draw_plain(w, u):
    """The column drawn from float32 weights in [0, 1]; -1 where all of them are 0."""
    whole = (w.astype(np.float64) * 2.0 ** 42).astype(np.int64)      # exact, then cut off
    sums = np.cumsum(whole)
    if not sums[-1]:
        return -1
    u = float(u)
    U = min((1 << 31) - 1, int(u * 2.0 ** 31)) if u > 0 else 0
    return int(np.searchsorted(sums, U * int(sums[-1]) >> 31, side="right"))


def verify_plain(token, p, q, u, u_draw, cu):
    """token [N] ints, p and q [N, V] float32 arrays (q may be None), u, u_draw float32. Returns
    (out, emitted, drafts that went, status)."""
    V = p.shape[1]
    out, emitted, gone, status = [], [], [], 0
    for s in range(len(cu) - 1):
        a, b = cu[s], cu[s + 1]
        if a == b:
            emitted.append(0)
            gone.append(0)
            continue
        for i in range(a, b - 1):
            if not 0 <= token[i + 1] < V:
                status |= BAD_TOKENS
        i = a
        while i + 1 < b:
            x = int(token[i + 1])
            if not 0 <= x < V:
                break
            had = 1 if q is None else Fraction(float(_unit(q[i, x])))
            ui = float(u[i])
            if math.isnan(ui) or not Fraction(ui) * had < Fraction(float(_unit(p[i, x]))):
                break
            i += 1
        w = _unit(p[i])
        if i + 1 < b:
            if q is not None:
                w = np.maximum(w - _unit(q[i]), np.float32(0))
            elif 0 <= token[i + 1] < V:
                w = w.copy()
                w[token[i + 1]] = 0
        x = draw_plain(w, u_draw[s])
        if x < 0:
            x = draw_plain(_unit(p[i]), u_draw[s])
        if x < 0:
            x, status = 0, status | BAD_PROBS
        out += [int(t) for t in token[a + 1:i + 1]] + [x] + [-1] * (b - 1 - i)
        emitted.append(i - a + 1)
        gone.append(b - 1 - i)
    return out, emitted, gone, status


def prefix_of(cu_seqs, s):
    """The prefix that sequence s shares, or -1."""
    for p in range(len(cu_seqs) - 1):
        if cu_seqs[p] <= s < cu_seqs[p + 1]:
            return p
    return -1


def shared64(q, parts, scale):
    """Softmax attention of q [m, d] over several runs of rows. parts: (k, v, M), k and v [T, d],
    M [m] rows that each query sees of the run. Returns out, lse, sum p |v| / sum p and the largest
    sum |q_i k_i| of each row, in float64."""
    q = q.double()
    out = torch.zeros_like(q)
    A = torch.zeros_like(q)
    lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
    big = torch.zeros(q.shape[0], dtype=torch.float64)
    for i in range(q.shape[0]):
        k = torch.cat([k[:max(0, int(M[i]))] for k, _, M in parts]).double()
        v = torch.cat([v[:max(0, int(M[i]))] for _, v, M in parts]).double()
        if not k.shape[0]:
            continue
        x = (k @ q[i]) * scale
        x = torch.where(x == -math.inf, x, x)
        top = x.max()
        w = torch.exp(x - top)
        out[i], A[i] = w @ v / w.sum(), w @ v.abs() / w.sum()
        lse[i] = top + torch.log(w.sum())
        big[i] = (k.abs() @ q[i].abs()).max()
    return out, lse, A, big
