"""Plain forms of the calls on shared pages, told request by request on the host."""
import numpy as np


def shared_tables(lens, new, parents, table, free, count, refs, page, room):
    """kv_shared_tables: (table, free, refs, slots, positions, starts, lens_out,
    count_out, refused, copies)."""
    n, was, before = len(lens), table.copy(), refs.copy()
    table, free, refs = table.copy(), free.copy(), refs.copy()
    most, pool = table.shape[1] * page, refs.size
    slots, positions = np.full(room, -1, np.int64), np.zeros(room, np.int32)
    starts, out, copies, gone, asked, refused, given = [0], [], [], [], 0, 0, 0
    for b in range(n):
        a, z, p = int(lens[b]), int(new[b]), int(parents[b])
        bad = not (0 <= a <= most and 0 <= z <= most)
        if p >= 0:
            bad = bad or a != 0 or p >= n or p == b or not 0 <= lens[p] <= most or parents[p] >= 0
            if not bad:
                a = min(int(lens[p]), z)
        row = was[p if p >= 0 and not bad else b]
        have, want = (0, 0) if bad else (-(-a // page), -(-z // page))
        last = int(row[have - 1]) if have else -1
        cut = not bad and z > a and a % page != 0 and (p >= 0 or (0 <= last < pool and before[last] > 1))
        ask = max(0, want - have) + cut if not bad and z > a else 0
        rows = 0 if bad else max(0, z - a)
        asked += ask
        ok = not bad and (not ask or asked <= count) and (not rows or starts[-1] + rows <= room)
        if ok:
            at = asked - ask
            if p >= 0:
                table[b, :have - cut] = row[:have - cut]
                np.add.at(refs, row[:have - cut], 1)
            if cut:
                copies.append((last, int(free[count - 1 - at])))
                if p < 0:
                    refs[last] -= 1
                    gone.append(last)
            for j in range(have - cut, want if z > a else 0):
                table[b, j] = free[count - 1 - at]
                refs[table[b, j]] = 1
                at += 1
            given = max(given, at) if ask else given
            for j in range(want, have):
                refs[row[j]] -= 1
                gone.append(int(row[j]))
            for t in range(rows):
                slots[starts[-1] + t] = int(table[b, (a + t) // page]) * page + (a + t) % page
                positions[starts[-1] + t] = a + t
        refused += not ok
        out.append(z if ok else int(lens[b]))
        starts.append(starts[-1] + rows)
    top = count - given
    for q in dict.fromkeys(gone):
        if refs[q] == 0:
            free[top] = q
            top += 1
    return (table, free, refs, slots, positions, np.array(starts, np.int32), np.array(out, np.int32), top, refused, copies)


def compact(lens, table, free, refs, page, room):
    """kv_compact: (table, free, refs, count, copies, moved)."""
    table, free, refs = table.copy(), free.copy(), refs.copy()
    used = np.flatnonzero(refs > 0)
    P = used.size
    high, low = used[used >= P][::-1], np.setdiff1d(np.arange(P), used)
    moved = np.arange(refs.size, dtype=np.int32)
    copies = list(zip(high[:room].tolist(), low[:room].tolist()))
    for a, b in copies:
        moved[a], refs[b], refs[a] = b, refs[a], 0
    for b, n in enumerate(lens):
        held = -(-int(n) // page)
        table[b, :held] = moved[table[b, :held]]
    rest = np.flatnonzero(refs <= 0)[::-1]
    free[:rest.size] = rest
    return table, free, refs, rest.size, copies, moved
