"""Plain sequence extension with pages that a sequence holds beyond its length, for the tests:
lists and loops, no code shared with the library."""
from __future__ import annotations

PAGE = 16


def pages_of(L):
    return -(-L // PAGE)


class Held:
    """B sequences over a pool. tables: lists of `width` entries, -1 where there is no block."""

    def __init__(self, lens, width, free, nb, extra=()):
        """Blocks of the lengths' pages, and of extra[b] pages behind them, from a list of ids."""
        ids = list(range(nb))
        self.nb, self.width, self.lens = nb, width, list(lens)
        self.held = [pages_of(L) for L in lens]
        for b, n in enumerate(extra):
            self.held[b] += n
        self.tables = [[ids.pop() if q < h else -1 for q in range(width)] for h in self.held]
        self.stack = ids[:free]
        self.lost = set(ids[free:])  # ids that this pool's user has put elsewhere

    def step(self, news, T, window=0, sinks=0):
        """Returns (offsets, slots, positions, errors)."""
        B, errors, offsets, slots, positions = len(news), set(), [0], [], []
        bad = []
        for L, n, h in zip(self.lens, news, self.held):
            bad.append(L < 0 or h < pages_of(L) or h > self.width or
                       (n >= 0 and L + n > self.width * PAGE))
            if bad[-1]:
                errors.add(3)
        for b in range(B):
            if bad[b]:
                continue
            if news[b] < 0:
                back = range(self.held[b])
            elif window > 0:  # wholly behind the window of the next token, and behind the sinks
                back = [q for q in range(self.width) if q * PAGE >= sinks and
                        (q + 1) * PAGE <= self.lens[b] - window + 1]
                gone = [q for q in back if self.tables[b][q] < 0]
                back = [q for q in back if not gone or q > max(gone)]
            else:
                back = []
            for q in sorted(back, reverse=True):
                if self.tables[b][q] >= 0:
                    self.stack.append(self.tables[b][q])
                    self.tables[b][q] = -1
            if news[b] < 0:
                self.lens[b] = self.held[b] = 0
        asked = wanted = 0
        there = len(self.stack)
        for b in range(B):
            n = 0 if bad[b] else max(news[b], 0)
            need = max(pages_of(self.lens[b] + n) - self.held[b], 0) if n else 0
            asked, wanted = asked + n, wanted + need
            if n and asked > T:
                errors.add(3)
                n = 0
            elif need and wanted > there:
                errors.add(7)
                n = 0
            elif need:
                for q in range(self.held[b], self.held[b] + need):
                    self.tables[b][q] = self.stack.pop()
                self.held[b] += need
            for at in range(self.lens[b], self.lens[b] + n):
                slots.append(self.tables[b][at // PAGE] * PAGE + at % PAGE)
                positions.append(at)
            if not bad[b]:
                self.lens[b] += n
            offsets.append(len(slots))
        pad = T - len(slots)
        return offsets, slots + [-1] * pad, positions + [0] * pad, errors

    def shorten(self, by):
        for b, n in enumerate(by):
            self.lens[b] -= n

    def check_blocks(self):
        """Every block is in one table or on the stack."""
        held = [e for row in self.tables for e in row if e >= 0]
        assert sorted(held + self.stack) == sorted(set(range(self.nb)) - self.lost)
        for row, h in zip(self.tables, self.held):
            assert all(e < 0 for e in row[h:])
