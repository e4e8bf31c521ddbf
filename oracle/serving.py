"""CPU float64 oracle of the operators around a verification step: plain loops over requests, tokens
and heads from the definitions, sharing no code with the library."""
from __future__ import annotations

import numpy as np

ERR_TOKEN, ERR_ROW, ERR_TREE, ERR_PAGE, ERR_LENGTH = 1, 4, 8, 16, 64
ERR_REQUEST, ERR_PENALTY = 128, 256


def rows_of(start, b, T, most=None):
    """(lo, hi) of request b's packed rows, or None where `start` says nothing of the kind."""
    lo, hi = int(start[b]), int(start[b + 1])
    return (lo, hi) if 0 <= lo <= hi <= T and (most is None or hi - lo <= most) else None


def resize(prefix_len, pages, block_table, free_pages, free_head, *, page_size, num_pages,
           chunk_start=None, rows=0, shares=None):
    """dict of pages, free_head, shares, position, slots, block_table, free_pages and error."""
    B, table = len(prefix_len), np.array(block_table, dtype=np.int64)
    free = np.array(free_pages, dtype=np.int64)
    owned = [int(x) for x in pages]
    left = None if shares is None else [int(x) for x in shares]
    position, slots = np.full(rows, -1, np.int64), np.full(rows, -1, np.int64)
    err, max_pages = 0, table.shape[1]
    head = int(free_head)
    if not 0 <= head <= len(free):
        err |= ERR_PAGE
        head = len(free)
    span, need = [], []
    for b in range(B):
        got = (0, 0) if chunk_start is None else rows_of(chunk_start, b, rows)
        bad = 0 if got is not None else ERR_TREE
        n = 0 if got is None else got[1] - got[0]
        length = int(prefix_len[b])
        want = -(-(length + n) // page_size)
        if length < 0 or not 0 <= owned[b] <= max_pages or owned[b] * page_size < length or want > max_pages:
            bad |= ERR_LENGTH
        err |= bad
        span.append(None if bad else got)
        need.append(owned[b] if bad else want)
    times = {}
    for b in range(B):
        for j in range(need[b], owned[b]):
            p = int(table[b, j])
            if 0 <= p < num_pages:
                times[p] = times.get(p, 0) + 1
            else:
                err |= ERR_PAGE
    back = sorted(p for p, k in times.items() if k > (left[p] if left else 0))
    if left is not None:
        for p, k in times.items():
            left[p] = max(left[p] - k, 0)
    if len(back) > head:
        err |= ERR_PAGE
        back = back[:head]
    free[head - len(back):head] = back
    head -= len(back)
    short = False
    for b in range(B):
        fits = True
        if need[b] > owned[b]:
            more = need[b] - owned[b]
            if short or head + more > len(free):
                short, fits = True, False
                err |= ERR_PAGE
            else:
                for j in range(more):
                    p = int(free[head + j])
                    if not 0 <= p < num_pages:
                        p = -1
                        err |= ERR_PAGE
                    table[b, owned[b] + j] = p
                head += more
                owned[b] = need[b]
        else:
            owned[b] = need[b]
        if span[b] is not None:
            for i in range(span[b][0], span[b][1]):
                at = int(prefix_len[b]) + i - span[b][0]
                position[i] = at
                if fits:
                    p = int(table[b, at // page_size])
                    if 0 <= p < num_pages:
                        slots[i] = p * page_size + at % page_size
                    else:
                        err |= ERR_PAGE
    return dict(pages=np.array(owned), free_head=head, shares=None if left is None else np.array(left),
                position=position, slots=slots, block_table=table, free_pages=free, error=err)


def fork(source, target, prefix_len, pages, block_table, free_pages, free_head, shares, k_cache,
         v_cache, *, num_pages):
    """dict of prefix_len, pages, free_head, shares, block_table, k_cache, v_cache and error."""
    table, length = np.array(block_table, dtype=np.int64), np.array(prefix_len, dtype=np.int64)
    owned, held = np.array(pages, dtype=np.int64), np.array(shares, dtype=np.int64)
    kc, vc = np.array(k_cache), np.array(v_cache)
    B, page_size, max_pages = len(length), kc.shape[2], table.shape[1]
    head, err = int(free_head), 0
    good_head = 0 <= head <= len(free_pages)
    room = len(free_pages) - head if good_head else 0
    if not good_head and len(source):
        err |= ERR_PAGE
    named, short, taken = set(), False, 0
    for s, t in zip(source, target):
        s, t = int(s), int(t)
        again = t in named
        named.add(t)
        if not 0 <= s < B or not 0 <= t < B or s == t or pages[t] != 0 or prefix_len[t] != 0 or again:
            err |= ERR_REQUEST
            continue
        n = int(prefix_len[s])
        if n < 0 or not 0 <= pages[s] <= max_pages or pages[s] * page_size < n:
            err |= ERR_LENGTH
            continue
        full, part = divmod(n, page_size)
        if part and (short or taken + 1 > room):
            short = True
            err |= ERR_PAGE
            continue
        for i in range(full):
            p = int(table[s, i])
            if 0 <= p < num_pages:
                held[p] += 1
            else:
                p = -1
                err |= ERR_PAGE
            table[t, i] = p
        if part:
            old, new = int(table[s, full]), int(free_pages[head + taken])
            taken += 1
            if not 0 <= new < num_pages:
                new = -1
                err |= ERR_PAGE
            table[t, full] = new
            if 0 <= old < num_pages and new >= 0:
                kc[:, new, :part] = kc[:, old, :part]
                vc[:, new, :part] = vc[:, old, :part]
            else:
                err |= ERR_PAGE
        length[t], owned[t] = n, full + (part > 0)
    return dict(prefix_len=length, pages=owned, free_head=head + taken, shares=held, block_table=table,
                k_cache=kc, v_cache=vc, error=err)


def rotate(x, weight, position, inv_freq, *, eps, interleaved):
    """(y, size) of heads x [T, H, D] in float64: size [T, H, D] is |a| + |b| of the pair that each
    element came of, for tolerances. Rows of negative positions come back as NaN."""
    y = np.array(x, dtype=np.float64)
    T, H, D = y.shape
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    size = np.abs(y)
    out = y.copy()
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = np.asarray(position, np.float64) * np.float64(inv_freq[i])
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        out[:, :, a] = y[:, :, a] * c - y[:, :, b] * s
        out[:, :, b] = y[:, :, b] * c + y[:, :, a] * s
        size[:, :, a] = size[:, :, b] = np.abs(y[:, :, a]) + np.abs(y[:, :, b])
    out[np.asarray(position) < 0] = np.nan
    return out, size


def attention(q, k_cache, v_cache, block_table, prefix_len, chunk_start, *, max_chunk, scale):
    """out [T, Hq, D], lse [T, Hq], and for tolerances: weight [T, Hq, D] = sum_j p_j |v_j| and
    spread [T, Hq] = max_j sum_d |q_d k_jd| scale over the keys a row sees. Inputs float64; NaN in
    out and lse where a row was not written."""
    T, Hq, D = q.shape
    num_pages, page_size, Hkv = k_cache.shape[:3]
    G, most = Hq // Hkv, block_table.shape[1] * page_size
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    weight, spread = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(prefix_len)):
        got = rows_of(chunk_start, b, T, max_chunk)
        if got is None or got[1] - got[0] > most:
            continue
        n = got[1] - got[0]
        length = min(max(int(prefix_len[b]), 0), most - n)
        k, v = np.zeros((2, length + n, Hkv, D))
        for j in range(length + n):
            p = int(block_table[b, j // page_size])
            if 0 <= p < num_pages:
                k[j], v[j] = k_cache[p, j % page_size], v_cache[p, j % page_size]
        for i in range(n):
            seen = length + i + 1
            for h in range(Hq):
                row, kv = q[got[0] + i, h], h // G
                z = scale * (k[:seen, kv] @ row)
                top = z.max()
                w = np.exp(z - top)
                total = w.sum()
                w /= total
                at = (got[0] + i, h)
                out[at], lse[at] = w @ v[:seen, kv], top + np.log(total)
                weight[at] = w @ np.abs(v[:seen, kv])
                spread[at] = scale * (np.abs(k[:seen, kv]) @ np.abs(row)).max()
    return out, lse, weight, spread


def penalize(logits, tokens, node_start, history, prefix_len, prompt_len, repetition, presence,
             frequency, *, paths, max_nodes, bias_start=None, bias_token=None, bias=None, mask=None):
    """(out, size, error): the logits [T, V] in float64, size [T, V] the sum of what was added up in
    absolute values. paths[i] are the nodes of row i's path, indices within its request. NaN in out
    where a row was not written as well as where the rule asks for it (see `written`)."""
    T, V = logits.shape
    out, size = np.full((T, V), np.nan), np.zeros((T, V))
    written, err, most = np.zeros(T, bool), 0, history.shape[1]
    for b in range(len(prefix_len)):
        got = rows_of(node_start, b, T, max_nodes)
        if got is None:
            err |= ERR_TREE
            continue
        lo, hi = got
        if lo == hi:
            continue
        written[lo:hi] = True
        bad = 0
        if not repetition[b] > 0:
            bad |= ERR_PENALTY
        if bias_start is not None and not 0 <= bias_start[b] <= bias_start[b + 1] <= len(bias):
            bad |= ERR_LENGTH
        if bad:
            err |= bad
            continue
        length, prompt = (min(max(int(x[b]), 0), most) for x in (prefix_len, prompt_len))
        if length != prefix_len[b] or prompt != prompt_len[b]:
            err |= ERR_LENGTH
        told, said = np.zeros(V, np.int64), np.zeros(V, np.int64)
        for j in range(length):
            x = int(history[b, j])
            if not 0 <= x < V:
                err |= ERR_TOKEN
            elif j < prompt:
                told[x] += 1
            else:
                said[x] += 1
        for x in tokens[lo:hi]:
            if not 0 <= x < V:
                err |= ERR_TOKEN
        add, much = np.zeros(V), np.zeros(V)
        if bias_start is not None:
            for j in range(int(bias_start[b]), int(bias_start[b + 1])):
                x = int(bias_token[j])
                if 0 <= x < V:
                    add[x] += float(bias[j])
                    much[x] += abs(float(bias[j]))
                else:
                    err |= ERR_TOKEN
        rep, pres, freq = float(repetition[b]), float(presence[b]), float(frequency[b])
        for i in range(lo, hi):
            times = said.copy()
            for m in paths[i]:
                x = int(tokens[lo + m])
                if m < hi - lo and 0 <= x < V:
                    times[x] += 1
            x = logits[i].astype(np.float64)
            hit = (told + times) > 0
            x[hit] = np.where(x[hit] > 0, x[hit] / rep, x[hit] * rep)
            size[i] = np.abs(x) + much
            often = times > 0
            x[often] -= freq * times[often] + pres
            size[i][often] += abs(freq) * times[often] + abs(pres)
            x = x + add
            if mask is not None:
                bits = (mask[i][np.arange(V) // 32].astype(np.int64) >> (np.arange(V) % 32)) & 1
                x[bits == 0] = -np.inf
            out[i] = x
    return out, size, written, err
