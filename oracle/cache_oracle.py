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
