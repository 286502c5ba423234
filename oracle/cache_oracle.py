"""Float64 restatement of the paged key-value cache's operators (test infrastructure; shares no code with the library).

Written from the formulas: plain loops over requests and heads, numpy float64, Python integers for the plan."""
import numpy as np


def plan(lengths, new_tokens, tables, free_pages, free_state, n_rows, page, n_pages):
    """One step's page plan over copies of the inputs: (slots, positions, starts, lengths, free_state, tables, ring)."""
    tables, ring, width = tables.copy(), list(map(int, free_pages)), tables.shape[1]
    head, count = int(free_state[0]), int(free_state[1])
    free = [ring[(head + i) % n_pages] for i in range(count)]
    slots, positions = [-1] * n_rows, [0] * n_rows
    starts, out_len, back, used, want_total, refused = [0], [], [], 0, 0, 0
    for b, length in enumerate(map(int, lengths)):
        new = 1 if new_tokens is None else int(new_tokens[b])
        row = starts[-1]
        starts.append(row + max(new, 0))
        held = -(-length // page)
        if new < 0:
            back += [int(x) for x in tables[b, :held]]
            out_len.append(0)
            continue
        need = -(-(length + new) // page) - held
        if held + need > width or row + new > n_rows:
            refused += 1
            out_len.append(length)
            continue
        want_total += need
        if need and want_total > count:
            refused += 1
            out_len.append(length)
            continue
        tables[b, held:held + need] = free[used:used + need]
        used += need
        out_len.append(length + new)
        for j in range(new):
            pos = length + j
            positions[row + j] = pos
            p = int(tables[b, pos // page])
            slots[row + j] = p * page + pos % page if 0 <= p < n_pages else -1
    for i, p in enumerate(back):
        ring[(head + count + i) % n_pages] = p
    state = [(head + used) % n_pages, count - used + len(back), refused]
    i32 = np.int32
    return (np.array(slots, i32), np.array(positions, i32), np.array(starts, i32), np.array(out_len, i32),
            np.array(state, i32), tables.astype(i32), np.array(ring, i32))


def norm_rope(x, gamma, positions, rope, theta, offset, eps):
    """x [T, heads, D] float64. Also returns the size |a| + |b| of what each output element is made of."""
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (offset + gamma)
    out, size = x.copy(), np.abs(x)
    half = rope // 2
    for i in range(half):
        a = positions.astype(np.float64) * theta ** (-2.0 * i / rope)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        lo, hi = x[..., i], x[..., i + half]
        out[..., i], out[..., i + half] = lo * c - hi * s, hi * c + lo * s
        size[..., i] = size[..., i + half] = np.abs(lo) + np.abs(hi)
    return out, size


def attend(q, tables, lengths, k_pool, v_pool, scale, gate=None):
    """q [B, Hq, D], pools [pages, Hkv, page, D], all float64 (scales of the cache already applied). Returns the output
    [B, Hq, D], the weighted size sum_j p_j |v_j| it is made of, and the largest sum |q_i k_i| * scale of a score."""
    B, Hq, D = q.shape
    n_pages, Hkv, page, _ = k_pool.shape
    out, size, mag = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, Hq, 1))
    for b in range(B):
        n = int(lengths[b])
        if n == 0:
            continue
        ids = tables[b, :-(-n // page)]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k = np.concatenate([k_pool[p, g] if 0 <= p < n_pages else np.zeros((page, D)) for p in ids])[:n]
            v = np.concatenate([v_pool[p, g] if 0 <= p < n_pages else np.zeros((page, D)) for p in ids])[:n]
            with np.errstate(invalid="ignore", over="ignore"):
                s = k @ q[b, h] * scale
                e = np.exp(s - s.max())
                p = e / e.sum()
                out[b, h], size[b, h] = p @ v, p @ np.abs(v)
                mag[b, h] = (np.abs(k) @ np.abs(q[b, h])).max() * abs(scale)
    if gate is not None:
        sg = 1.0 / (1.0 + np.exp(-gate))
        out, size = out * sg, size * sg
    return out, size, mag


def _ring(free_pages, free_state, n_pages):
    head, count = int(free_state[0]), int(free_state[1])
    return [int(free_pages[(head + i) % n_pages]) for i in range(count)], head, count


def tree(parents, starts, lengths, refused, n_rows, words):
    """Masks (uint64 [n_rows, words]) and positions of drafted trees: each token's ancestors by walking up. refused: the
    requests whose tokens are not in the cache."""
    masks, positions = np.zeros((n_rows, words), np.uint64), np.zeros(n_rows, np.int32)
    for b, length in enumerate(map(int, lengths)):
        lo, n = int(starts[b]), int(starts[b + 1]) - int(starts[b])
        if refused[b]:
            continue
        for i in range(n):
            depth, j = -1, i
            while j >= 0:
                masks[lo + i, j // 64] |= np.uint64(1 << (j % 64))
                depth += 1
                j = int(parents[lo + j])
            positions[lo + i] = length - n + depth
    return masks, positions


def attend_tree(q, starts, refused, masks, tables, lengths, k_pool, v_pool, scale, gate=None):
    """As attend, for rows starts[b] .. starts[b + 1] - 1 of request b, its last tokens: each sees the older tokens and the
    new ones in its mask (None: those up to itself). Rows of refused requests are 0, rows past the last token NaN (not
    given). Also returns each row's number of tokens seen."""
    rows, Hq, D = q.shape
    n_pages, Hkv, page, _ = k_pool.shape
    out, size, mag, seen = np.zeros(q.shape), np.zeros(q.shape), np.zeros((rows, Hq, 1)), np.zeros((rows, 1, 1))
    out[int(starts[-1]):] = np.nan
    for b in range(len(lengths)):
        lo, hi, length = int(starts[b]), int(starts[b + 1]), int(lengths[b])
        m = hi - lo
        if m == 0 or refused[b]:
            continue
        sees = np.ones((m, length), bool)
        for i in range(m):
            for j in range(m):
                sees[i, length - m + j] = j <= i if masks is None else int(masks[lo + i, j // 64]) >> (j % 64) & 1
        seen[lo:hi, 0, 0] = sees.sum(1)
        ids = tables[b, :-(-length // page)]
        for g in range(Hkv):
            k = np.concatenate([k_pool[p, g] if 0 <= p < n_pages else np.zeros((page, D)) for p in ids])[:length]
            v = np.concatenate([v_pool[p, g] if 0 <= p < n_pages else np.zeros((page, D)) for p in ids])[:length]
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                for i in range(m):
                    kk, vv, x = k[sees[i]], v[sees[i]], q[lo + i, h]
                    if len(kk) == 0:
                        continue
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = kk @ x * scale
                        e = np.exp(s - s.max())
                        p = e / e.sum()
                        out[lo + i, h], size[lo + i, h] = p @ vv, p @ np.abs(vv)
                        mag[lo + i, h] = (np.abs(kk) @ np.abs(x)).max() * abs(scale)
    if gate is not None:
        sg = 1.0 / (1.0 + np.exp(-gate))
        out, size = out * sg, size * sg
    return out, size, mag, seen


def keep(counts, lengths, starts, refused, path, tables, free_pages, free_state, refs, pools, page, n_pages):
    """What of the new tokens stays, over copies: (lengths, free_state, tables, ring, refs, pools). starts None: every token
    is new. pools: arrays [n_pages, heads, page, ...]."""
    tables, ring, pools = tables.copy(), free_pages.copy(), [p.copy() for p in pools]
    before = [p.copy() for p in pools]
    holders = None if refs is None else [int(r) + 1 for r in refs]
    free, head, count = _ring(free_pages, free_state, n_pages)
    out_len, back, moves, used, wanted, stayed = [], [], [], 0, 0, 0
    for b, (k, length) in enumerate(zip(map(int, counts), map(int, lengths))):
        n = length if starts is None else 0 if refused[b] else int(starts[b + 1]) - int(starts[b])
        older = length - n
        new = 0 if k < 0 else older + k
        steps = [] if k < 0 else [i if path is None else int(path[b][i]) for i in range(k)]
        held, stay = -(-length // page), -(-new // page)
        changed = {(older + i) // page for i, j in enumerate(steps) if i != j}
        if new % page:
            changed.add(stay - 1)
        swap = [i for i in sorted(changed) if refs is not None and refs[tables[b, i]] > 0]
        wanted += len(swap)
        if swap and wanted > count:
            stayed += 1
            out_len.append(length)
            continue
        old = tables[b].copy()
        for i in swap:
            tables[b, i] = free[used]
            used += 1
        back += [int(old[i]) for i in swap] + [int(old[i]) for i in range(stay, held)]
        out_len.append(new)
        for p in range(new):
            s = p if p < older else older + steps[p - older]
            if s != p or p // page in swap:
                moves.append((old[s // page], s % page, tables[b, p // page], p % page))
    for src, so, dst, do in moves:
        for a, z in zip(before, pools):
            z[dst, :, do] = a[src, :, so]
    gone = []
    if holders is None:
        gone = back
    else:
        for p in back:
            holders[p] -= 1
        for p in back:
            if holders[p] <= 0 and p not in gone:
                gone.append(p)
        refs = np.array([max(0, h - 1) for h in holders], np.int32)
    for i, p in enumerate(gone[:n_pages - count]):
        ring[(head + count + i) % n_pages] = p
    state = [(head + used) % n_pages, count - used + min(len(gone), n_pages - count), stayed]
    i32 = np.int32
    return np.array(out_len, i32), np.array(state, i32), tables, ring, refs, pools


def fork(src, dst, lengths, tables, free_pages, free_state, refs, pools, page, n_pages):
    """Requests dst over the tokens of src, over copies: (lengths, free_state, tables, ring, refs, pools)."""
    tables, refs, pools, out_len = tables.copy(), refs.copy(), [p.copy() for p in pools], lengths.copy()
    free, head, count = _ring(free_pages, free_state, n_pages)
    used, wanted, refused, named = 0, 0, 0, set()
    for s, d in zip(map(int, src), map(int, dst)):
        if s < 0:
            continue
        if not (s < len(lengths) and 0 <= d < len(lengths)):
            continue
        twice = d in named
        named.add(d)
        if twice or lengths[d] != 0:
            continue
        n = int(lengths[s])
        full, part = n // page, n % page
        wanted += part > 0
        if part and wanted > count:
            refused += 1
            continue
        tables[d, :full] = tables[s, :full]
        for p in tables[s, :full]:
            refs[p] += 1
        if part:
            tables[d, full] = free[used]
            used += 1
            for z in pools:
                z[tables[d, full], :, :part] = z[tables[s, full], :, :part]
        out_len[d] = n
    i32 = np.int32
    return out_len, np.array([(head + used) % n_pages, count - used, refused], i32), tables, free_pages.copy(), refs, pools
