"""Plain models of the calls on shared pages: holders counted one by one, and a stack."""


def pages_of(n):
    return (n + 63) // 64


def fork_model(source, lens, keep, table, shares, free, n_free, kv_slots):
    """tpk_kv_pages_fork.  Lists; returns (rows, shares, free, n_free, len, granted, copy_src, copy_dst, bad), rows being each
    request's pages afterwards."""
    n, cap, bad = len(source), 64 * len(table[0]), False
    clamped = [min(max(x, 0), cap) for x in lens]
    bad |= clamped != list(lens)
    n_free = min(max(n_free, 0), len(free))
    src, want, refused = [], [], []
    for b in range(n):
        s, k, ok = source[b], 0, True
        if s == -1:
            s = b
        elif not 0 <= s < n:
            ok = False
        else:
            k = clamped[s] if keep is None else keep[b]
            ok = 0 <= k <= clamped[s]
        src.append(s if ok else b)
        want.append(k if ok else clamped[b])
        refused.append(not ok)
    changed = [b for b in range(n) if not refused[b] and (src[b] != b or want[b] != clamped[b])]
    inside = lambda x: 0 <= x < kv_slots  # noqa: E731
    holders = [x + 1 for x in shares]
    for b in changed:
        for j in range(max(pages_of(clamped[b]), want[b] // 64)):
            old = table[b][j] if j < pages_of(clamped[b]) else None
            new = table[src[b]][j] if j < want[b] // 64 else None
            if old is not None and old == new:
                continue
            for x, d in ((old, -1), (new, 1)):
                if x is not None and inside(x):
                    holders[x] += d
                bad |= x is not None and not inside(x)
    asking = {}
    for b in changed:
        if want[b] % 64:
            x = table[src[b]][want[b] // 64]
            bad |= not inside(x)
            if inside(x):
                asking.setdefault(x, []).append(b)
    bad |= any(h < 0 for h in holders)
    stack = list(free[:n_free])
    copies = []
    for x in range(kv_slots - 1, -1, -1):
        if holders[x] <= 0:
            if x not in asking:
                stack.append(x)
            else:
                copies += asking[x][1:]
        elif x in asking:
            copies += asking[x]
    shares_out = [max(0, h - 1) for h in holders]
    bad |= len(stack) > len(free)
    stack = stack[:len(free)]
    length, granted = list(want), [int(not r) for r in refused]
    rows = [list(table[src[b]][:pages_of(want[b])]) for b in range(n)]
    copy_src, copy_dst = [-1] * n, [-1] * n
    for b in changed:
        if want[b] % 64 and not inside(rows[b][-1]):
            granted[b], length[b] = 0, want[b] // 64 * 64
            rows[b].pop()
    for b in sorted(copies):
        if stack:
            copy_src[b], copy_dst[b] = rows[b][-1], stack.pop()
            rows[b][-1] = copy_dst[b]
        else:
            granted[b], length[b] = 0, want[b] // 64 * 64
            rows[b].pop()
    free_out = list(free)
    free_out[n_free:len(stack)] = stack[n_free:]
    return rows, shares_out, free_out, len(stack), length, granted, copy_src, copy_dst, bad


def compact_model(lens, table, shares, free, n_free, kv_slots, max_copies):
    """tpk_kv_pages_compact.  Returns (rows, shares, free, n_free, new_slot, copy_src, copy_dst, n_copies, bad)."""
    cap, bad = 64 * len(table[0]), False
    n_free = min(max(n_free, 0), len(free))
    on_stack = {x for x in free[:n_free] if 0 <= x < kv_slots}
    bad |= any(not 0 <= x < kv_slots for x in free[:n_free])
    low = sorted(on_stack)
    top = [x for x in range(kv_slots - 1, -1, -1) if x not in on_stack]
    moves = [(s, d) for s, d in list(zip(top, low))[:max_copies] if d < s]
    new = [-1 if x in on_stack else x for x in range(kv_slots)]
    for s, d in moves:
        new[s] = d
    shares_out = [0] * kv_slots
    for x in top:
        shares_out[new[x]] = shares[x]
    used = {new[x] for x in top}
    stack = [x for x in range(kv_slots - 1, -1, -1) if x not in used]
    bad |= len(stack) > len(free)
    free_out = list(free)
    stack = stack[:len(free)]
    free_out[:len(stack)] = stack
    rows = []
    for b, n in enumerate(lens):
        c = min(max(n, 0), cap)
        bad |= c != n
        row = []
        for x in table[b][:pages_of(c)]:
            ok = 0 <= x < kv_slots and new[x] >= 0
            bad |= not ok
            row.append(new[x] if ok else x)
        rows.append(row)
    pad = [-1] * (max_copies - len(moves))
    return rows, shares_out, free_out, len(stack), new, [s for s, _ in moves] + pad, [d for _, d in moves] + pad, len(moves), bad
