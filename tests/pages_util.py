"""Plain forms of the operators for sequences that share pages, step by step."""
import numpy as np


class Pages:
    """The state of a paged cache's bookkeeping, as numpy arrays."""

    def __init__(self, table, lens, n_pages, shares, free, head, page):
        self.table, self.lens, self.n_pages = np.array(table), np.array(lens), np.array(n_pages)
        self.shares, self.free, self.head, self.page = np.array(shares), np.array(free), int(head), page

    def copy(self):
        return Pages(self.table, self.lens, self.n_pages, self.shares, self.free, self.head, self.page)

    def check(self):
        """Every page has as many holders as the table says, or is free, once."""
        held = np.zeros(len(self.shares), int)
        for b in range(len(self.lens)):
            row = self.table[b, :self.n_pages[b]]
            assert self.n_pages[b] * self.page >= self.lens[b]
            assert len(set(row)) == len(row)
            held[row] += 1
        free = self.free[self.head:]
        assert len(set(free)) == len(free)
        assert not held[free].any()
        assert np.array_equal(np.maximum(held - 1, 0), self.shares)


def _give_back(s, gone, added, taken):
    """gone: (row, block, page) released, in order; added: pages joined."""
    for p in added:
        s.shares[p] += 1
    for _, _, p in gone:
        s.shares[p] -= 1
    back, seen = [], set()
    for _, _, p in gone:
        if s.shares[p] < 0 and p not in seen:
            seen.add(p)
            back.append(p)
    head = s.head + taken - len(back)
    if head < 0:
        return False
    for p in back:
        s.shares[p] = 0
    s.free[head:head + len(back)] = back
    s.head = head
    return True


def fork_ref(s, parent):
    """(state, src, dst) after the fork; None where it is refused."""
    n, page, B = s.copy(), s.page, len(s.lens)
    src, dst = np.full((B, page), -1), np.full((B, page), -1)
    gone, added, taken, heirs = [], [], 0, set()
    for b in range(B):
        if parent[b] < -1 or parent[b] >= B:
            return None
    for b in range(B):
        p = parent[b]
        if p == b:
            continue
        gone += [(b, j, s.table[b, j]) for j in range(s.n_pages[b])]
        n.table[b, :s.n_pages[b]] = -1
        n.n_pages[b] = n.lens[b] = 0
        if p < 0:
            continue
        t = s.lens[p]
        whole, rest = t // page, t % page
        n.lens[b], n.n_pages[b] = t, whole + (rest > 0)
        n.table[b, :whole] = s.table[p, :whole]
        added += list(s.table[p, :whole])
        if rest:
            last = s.table[p, whole]
            if parent[p] != p and p not in heirs and s.shares[last] == 0:
                n.table[b, whole] = last
                added.append(last)
            else:
                if s.head + taken >= len(s.free):
                    return None
                new = s.free[s.head + taken]
                taken += 1
                n.table[b, whole] = new
                src[b, :rest] = last * page + np.arange(rest)
                dst[b, :rest] = new * page + np.arange(rest)
            heirs.add(p)
    return (n, src, dst) if _give_back(n, gone, added, taken) else None


def compact_ref(s, keep, m):
    """(state, src, dst) after sequences keep the positions keep[b][:m[b]] (m < 0: all)."""
    n, page, B, cap = s.copy(), s.page, len(s.lens), keep.shape[1]
    src, dst = np.full((B, cap), -1), np.full((B, cap), -1)
    gone, taken = [], 0
    for b in range(B):
        if m[b] < 0:
            continue
        k = keep[b, :m[b]]
        if m[b] > s.lens[b] or (len(k) and (k[0] < 0 or k[-1] >= s.lens[b] or (np.diff(k) <= 0).any())):
            return None
        same = 0
        while same < m[b] and k[same] == same:
            same += 1
        stay = same // page
        if same == m[b] and same % page and s.shares[s.table[b, stay]] == 0:
            stay += 1
        blocks = -(-m[b] // page)
        if s.head + taken + blocks - stay > len(s.free):
            return None
        gone += [(b, j, s.table[b, j]) for j in range(stay, s.n_pages[b])]
        n.table[b, stay:s.n_pages[b]] = -1
        for j in range(stay, blocks):
            n.table[b, j] = s.free[s.head + taken]
            taken += 1
        for i in range(stay * page, m[b]):
            src[b, i] = s.table[b, k[i] // page] * page + k[i] % page
            dst[b, i] = n.table[b, i // page] * page + i % page
        n.lens[b], n.n_pages[b] = m[b], blocks
    return (n, src, dst) if _give_back(n, gone, [], taken) else None


def find_ref(table, lens, n, page, group, min_keys):
    """(first row, rows, shared keys, 0) of every row."""
    B = len(lens)
    out = np.array([[b, 1, 0, 0] for b in range(B)])
    family, common, prev = [], 0, None

    def close():
        if len(family) > 1:
            for b in family:
                out[b] = [family[0], family[-1] - family[0] + 1, common * page, 0]

    for b in range(B):
        if n[b] <= 0:
            continue
        pages = 0
        if prev is not None:
            for j in range(min(lens[prev], lens[b]) // page):
                if table[prev, j] != table[b, j]:
                    break
                pages += 1
        prev = b
        new = min(common, pages) if len(family) > 1 else pages
        k = len(family)
        if (k and n[b] * group < 256 and new > 0 and new * page >= min_keys
                and (k == 1 or k * new >= (k - 1) * common)):
            family, common = family + [b], new
            continue
        close()
        family, common = ([] if n[b] * group >= 256 else [b]), 0
    close()
    return out
