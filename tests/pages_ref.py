"""Plain sequential code for the page calls, on numpy arrays: what include/kvq.h says, row by row."""
import numpy as np

BLOCK, TABLE, SEQ, ROW, NO_PAGES, CONFLICT = 1, 2, 4, 32, 64, 128


def _pages(tokens, bs):
    return -(-tokens // bs)


def fork(table, lens, parents, nb, bs, width, spaces, keep=None, new=None, pins=None):
    """table [old rows, spaces, width].  Returns (table, lens, refs [spaces, nb], copies [(space, src, dst)], error bits)."""
    n, cap, err = len(parents), width * bs, 0
    out = np.full((n, spaces, width), -1, np.int64)
    kept, total = np.zeros(n, np.int64), np.zeros(n, np.int64)
    for i, p in enumerate(parents):
        if p >= len(lens):
            err |= ROW
            continue
        L = int(lens[p]) if p >= 0 else 0
        err |= (SEQ if L < 0 else 0) | (TABLE if L > cap else 0)
        L = max(0, min(L, cap))
        if keep is not None:
            err |= SEQ if keep[i] < 0 else 0
            L = min(L, max(0, int(keep[i])))
        a = 0 if new is None else int(new[i])
        err |= SEQ if a < 0 else 0
        t = L + max(0, a)
        err |= TABLE if t > cap else 0
        kept[i], total[i] = L, min(t, cap)
        for s in range(spaces):
            for e in range(_pages(L, bs)):
                v = int(table[p, s, e])
                if v >= nb:
                    err |= BLOCK
                out[i, s, e] = v if 0 <= v < nb else -1
    refs = np.zeros((spaces, nb), np.int64) if pins is None else np.maximum(pins.astype(np.int64), 0)
    tails = {}
    for i in range(n):
        for s in range(spaces):
            for e in range(_pages(kept[i], bs)):
                v = out[i, s, e]
                if v < 0:
                    continue
                if kept[i] % bs and e == kept[i] // bs:
                    tails.setdefault((s, v), []).append(i)
                else:
                    refs[s, v] += 1
    copies = []
    for s in range(spaces):
        keepers = {(s2, v): min(r) for (s2, v), r in tails.items() if s2 == s and refs[s, v] == 0}
        held = {v for (s2, v) in tails if s2 == s}
        free = [u for u in range(nb) if refs[s, u] == 0 and u not in held][::-1]
        for i in range(n):
            want = []
            if kept[i] % bs and out[i, s, kept[i] // bs] >= 0:
                e = kept[i] // bs
                v = int(out[i, s, e])
                if keepers.get((s, v)) == i:
                    refs[s, v] = 1
                else:
                    want.append((e, v))
            want += [(e, None) for e in range(_pages(kept[i], bs), _pages(total[i], bs))]
            for e, v in want:
                u = free.pop() if free else -1
                err |= NO_PAGES if u < 0 else 0
                out[i, s, e] = u
                if u >= 0:
                    refs[s, u] = 1
                    if v is not None:
                        copies.append((s, v, u))
    return out, total, refs, copies, err


def compact(table, lens, nb, bs, spaces, pins=None):
    """Returns (table, page_map, refs, num_used, copies, error bits)."""
    width, err = table.shape[2], 0
    refs = np.zeros((spaces, nb), np.int64) if pins is None else np.maximum(pins.astype(np.int64), 0)
    fixed = refs > 0
    out = np.full(table.shape, -1, np.int64)
    for b, L in enumerate(lens):
        err |= (SEQ if L < 0 else 0) | (TABLE if L > width * bs else 0)
        for s in range(spaces):
            for e in range(min(width, _pages(max(0, int(L)), bs))):
                v = int(table[b, s, e])
                err |= BLOCK if v >= nb else 0
                if 0 <= v < nb:
                    out[b, s, e] = v
                    refs[s, v] += 1
    page_map, moved, copies = np.full((spaces, nb), -1, np.int64), np.zeros((spaces, nb), np.int64), []
    used = refs > 0
    for s in range(spaces):
        n = int(used[s].sum())
        holes = iter([u for u in range(n) if not used[s, u]])
        for u in range(nb):
            if used[s, u]:
                to = next(holes) if u >= n and not fixed[s, u] else u
                page_map[s, u] = to
                moved[s, to] = refs[s, u]
                if to != u:
                    copies.append((s, u, to))
        sel = out[:, s] >= 0
        out[:, s][sel] = page_map[s][out[:, s][sel]]
    return out, page_map, moved, used.sum(1), copies, err


def copy_pairs(src, dst, units):
    """(pairs that are done, error bits)."""
    err, todo = 0, []
    for i, (a, b) in enumerate(zip(src, dst)):
        if a < 0 or b < 0:
            continue
        if a >= units or b >= units:
            err |= BLOCK if a != b else 0
            continue
        todo.append((i, int(a), int(b)))
    read = {a for _, a, _ in todo}
    done, written = [], set()
    for i, a, b in todo:
        if a == b:
            continue
        if b in read or b in written:
            err |= CONFLICT
            continue
        written.add(b)
        done.append((a, b))
    return done, err
