"""CPU float64 oracle of the operators on drafted token trees: plain loops over requests and
nodes from the definitions, sharing no code with the library."""
from __future__ import annotations

import numpy as np

FIXED, IID, DISTINCT = 0, 1, 2
ERR_TOKEN, ERR_ROW, ERR_TREE, ERR_PAGE, ERR_UNIFORM, ERR_LENGTH = 1, 4, 8, 16, 32, 64


def is_tree(parents) -> bool:
    return all((p == -1) if i == 0 else (0 <= p < i) for i, p in enumerate(parents))


def line_of(parents, node: int) -> list:
    """The nodes from the root to `node`."""
    line = []
    while node >= 0:
        line.insert(0, node)
        node = int(parents[node])
    return line


def ancestor_words(parents, max_nodes: int) -> np.ndarray:
    words = (max_nodes + 63) // 64
    out = np.zeros((len(parents), words), dtype=np.uint64)
    for i in range(len(parents)):
        for m in line_of(parents, i):
            out[i, m // 64] |= np.uint64(1) << np.uint64(m % 64)
    return out


def node_range(node_start, b, T, max_nodes):
    lo, hi = int(node_start[b]), int(node_start[b + 1])
    return (lo, hi) if 0 <= lo <= hi <= T and hi - lo <= max_nodes else None


def plan(parents, node_start, prefix_len, pages, block_table, free_pages, free_head, *, page_size,
         num_pages, max_nodes, max_path):
    """dict of ancestors, depth, position, slots, pages, free_head, block_table and error. Rows of
    [T, ...] outputs that belong to no request hold None's place: 0 / -1 (see `written`)."""
    T, B = len(parents), len(prefix_len)
    words = (max_nodes + 63) // 64
    table = np.array(block_table, dtype=np.int64)
    max_pages = table.shape[1]
    anc = np.zeros((T, words), dtype=np.uint64)
    depth = np.full(T, -1, dtype=np.int64)
    position = np.full(T, -1, dtype=np.int64)
    written = np.zeros(T, dtype=bool)
    slots = np.full((B, max_path), -1, dtype=np.int64)
    owned = np.array(pages, dtype=np.int64)
    err = 0
    head = int(free_head)
    good_head = 0 <= head <= len(free_pages)
    if not good_head:
        err |= ERR_PAGE
    left = len(free_pages) - head if good_head else 0
    at = head
    starved = False
    for b in range(B):
        rng = node_range(node_start, b, T, max_nodes)
        n = 0 if rng is None else rng[1] - rng[0]
        if rng is None:
            err |= ERR_TREE
        tokens = min(n, max_path)
        length, have = int(prefix_len[b]), int(owned[b])
        want = -(-(length + tokens) // page_size)
        ok = length >= 0 and 0 <= have <= max_pages and have * page_size >= length and want <= max_pages
        if not ok:
            err |= ERR_LENGTH
        more = max(0, want - have) if ok else 0
        fits = True
        if more and (starved or more > left):
            fits, starved = False, True
            err |= ERR_PAGE
        elif more:
            for j in range(more):
                page = int(free_pages[at])
                if not 0 <= page < num_pages:
                    err |= ERR_PAGE
                    page = -1
                table[b, have + j] = page
                at += 1
            left -= more
            owned[b] = have + more
        par = [] if rng is None else [int(p) for p in parents[rng[0]:rng[1]]]
        tree = rng is not None and is_tree(par)
        if tree:
            depths = [len(line_of(par, i)) - 1 for i in range(n)]
            tree = all(d < max_path for d in depths)
        if not tree:
            err |= ERR_TREE
        if rng is not None:
            written[rng[0]:rng[1]] = True
            if tree and n:
                anc[rng[0]:rng[1]] = ancestor_words(par, max_nodes)
                depth[rng[0]:rng[1]] = depths
                if ok:
                    position[rng[0]:rng[1]] = length + np.array(depths)
        if tree and ok and fits:
            for i in range(tokens):
                page = int(table[b, (length + i) // page_size])
                if 0 <= page < num_pages:
                    slots[b, i] = page * page_size + (length + i) % page_size
                else:
                    err |= ERR_PAGE
    return dict(ancestors=anc, depth=depth, position=position, slots=slots, pages=owned,
                free_head=at, block_table=table, error=err, written=written)


def attention(q, k_tree, v_tree, k_cache, v_cache, block_table, prefix_len, node_start, ancestors,
              *, max_nodes, scale):
    """out [T, Hq, D], lse [T, Hq], and for tolerances: weight [T, Hq, D] = sum_j p_j |v_j| and
    spread [T, Hq] = max_j sum_d |q_d k_jd| scale over the keys a row sees. Inputs float64; NaN in
    out and lse where a row was not written."""
    T, Hq, D = q.shape
    num_pages, page_size, Hkv = k_cache.shape[:3]
    B, G = len(prefix_len), Hq // Hkv
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    weight = np.zeros((T, Hq, D))
    spread = np.zeros((T, Hq))
    capacity = block_table.shape[1] * page_size
    for b in range(B):
        rng = node_range(node_start, b, T, max_nodes)
        if rng is None:
            continue
        lo, hi = rng
        length = min(max(int(prefix_len[b]), 0), capacity)
        keys = np.zeros((length, Hkv, D))
        vals = np.zeros((length, Hkv, D))
        for j in range(length):
            page = int(block_table[b, j // page_size])
            if 0 <= page < num_pages:
                keys[j], vals[j] = k_cache[page, j % page_size], v_cache[page, j % page_size]
        for i in range(lo, hi):
            if ancestors is None:
                seen = list(range(i - lo + 1))
            else:
                seen = [m for m in range(hi - lo)
                        if (int(ancestors[i, m // 64]) >> (m % 64)) & 1]
            rows = [lo + m for m in seen]
            for h in range(Hkv):
                kk = np.concatenate([keys[:, h], k_tree[rows, h]])
                vv = np.concatenate([vals[:, h], v_tree[rows, h]])
                for g in range(h * G, (h + 1) * G):
                    if not len(kk):
                        out[i, g], lse[i, g] = 0.0, -np.inf
                        continue
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = kk @ q[i, g] * scale
                        top = s.max()
                        p = np.exp(s - top)
                        total = p.sum()
                        out[i, g] = (p @ vv) / total
                        lse[i, g] = top + np.log(total)
                        weight[i, g] = (p @ np.abs(vv)) / total
                        spread[i, g] = (np.abs(kk) @ np.abs(q[i, g])).max() * scale
    return out, lse, weight, spread


def verify(target, draft, tokens, parents, node_start, u, r, *, mode, max_nodes, max_path):
    """dict of accept_len, path, emitted, out_token, error: the residuals are kept as whole rows,
    normalised after each rejection."""
    T, V = target.shape
    B = len(r)
    accept = np.full(B, -1, dtype=np.int64)
    path = np.full((B, max_path), -1, dtype=np.int64)
    emitted = np.full((B, max_path), -1, dtype=np.int64)
    token = np.full(B, -1, dtype=np.int64)
    error = 0

    def proper(x):
        return bool(np.all(np.isfinite(x)) and np.all(np.asarray(x) >= 0))

    for b in range(B):
        rng = node_range(node_start, b, T, max_nodes)
        if rng is None:
            error |= ERR_TREE
            continue
        lo, hi = rng
        if hi == lo:
            continue
        par = [int(x) for x in parents[lo:hi]]
        bad = 0 if is_tree(par) else ERR_TREE
        if not bad and not 0.0 <= r[b] < 1.0:
            bad = ERR_UNIFORM
        cur, line, words = 0, [0], []
        while not bad:
            p = np.asarray(target[lo + cur], dtype=np.float64)
            q = None if mode == FIXED else np.asarray(draft[lo + cur], dtype=np.float64)
            res, mass, left, passes = p.copy(), 1.0, 1.0, 0
            nxt = -1
            for i in range(cur + 1, hi - lo):
                if par[i] != cur:
                    continue
                x = int(tokens[lo + i])
                bad |= 0 if 0 <= x < V else ERR_TOKEN
                bad |= 0 if 0.0 <= u[lo + i] < 1.0 else ERR_UNIFORM
                if not bad & ERR_TOKEN and not (proper(p[x]) and (q is None or proper(q[x]))):
                    bad |= ERR_ROW
                if bad:
                    break
                qx = 1.0 if q is None else q[x] / left if left > 0 else 0.0
                if u[lo + i] * qx * mass < res[x]:
                    nxt = i
                    break
                if q is None:
                    mass -= res[x]
                    res[x] = 0.0
                elif mass > 0.0:
                    if not (proper(p) and proper(q)):
                        bad |= ERR_ROW
                        break
                    res = np.maximum(res - (mass / left if left > 0 else 0.0) * q, 0.0)
                    mass = float(res.sum())
                    if mode == DISTINCT:
                        left -= q[x]
            if bad:
                break
            if nxt < 0:
                if not proper(p):
                    bad = ERR_ROW
                    break
                if not res.sum() > 0:
                    res = p
                if not res.sum() > 0:
                    bad = ERR_ROW
                    break
                sums = np.cumsum(res)
                y = int(np.searchsorted(sums, r[b] * sums[-1], side="right"))
                if y >= V:
                    y = int(np.nonzero(res)[0][-1])
                break
            if len(line) >= max_path:
                bad = ERR_TREE
                break
            cur = nxt
            line.append(cur)
            words.append(int(tokens[lo + cur]))
        if bad:
            error |= bad
            continue
        accept[b], token[b] = len(words), y
        path[b, :len(line)] = line
        emitted[b, :len(words) + 1] = words + [y]
    return dict(accept_len=accept, path=path, emitted=emitted, out_token=token, error=error)


def commit(k_tree, v_tree, k_cache, v_cache, node_start, path, accept_len, slots, prefix_len, *,
           max_nodes):
    """New caches (copies), new lengths and the error word; arrays of any type."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    length = np.array(prefix_len, dtype=np.int64)
    T = k_tree.shape[1]
    num_pages, page_size = k_cache.shape[1:3]
    error = 0
    for b in range(len(length)):
        taken = int(accept_len[b])
        if taken < 0:
            continue
        rng = node_range(node_start, b, T, max_nodes)
        if rng is None or rng[1] == rng[0] or taken >= path.shape[1]:
            error |= ERR_TREE
            continue
        nodes = [int(x) for x in path[b, :taken + 1]]
        to = [int(x) for x in slots[b, :taken + 1]]
        bad = 0
        if not all(0 <= x < rng[1] - rng[0] for x in nodes):
            bad |= ERR_TREE
        if not all(0 <= x < num_pages * page_size for x in to):
            bad |= ERR_PAGE
        if bad:
            error |= bad
            continue
        for x, s in zip(nodes, to):
            k_cache[:, s // page_size, s % page_size] = k_tree[:, rng[0] + x]
            v_cache[:, s // page_size, s % page_size] = v_tree[:, rng[0] + x]
        length[b] += taken + 1
    return k_cache, v_cache, length, error
