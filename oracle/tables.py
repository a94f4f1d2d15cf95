"""Block tables of a batch over a ring of free slots, written plainly (lists and loops)."""
from __future__ import annotations

from collections import deque

__all__ = ["TableOracle"]


class TableOracle:
    """rows: the slots each request owns, in order; free: the ring from its front."""

    def __init__(self, n_slots, n_req, block_size, free=None, rows=None):
        self.bs = block_size
        self.free = deque(range(n_slots) if free is None else free)
        self.rows = [list(r) for r in rows] if rows is not None else [[] for _ in range(n_req)]
        self.short = 0

    def reserve(self, ctx):
        """True if every row got its blocks; else nothing changed and `short` blocks were lacking."""
        need = [-(-n // self.bs) for n in ctx]
        back = sum(max(0, len(r) - m) for r, m in zip(self.rows, need))
        want = sum(max(0, m - len(r)) for r, m in zip(self.rows, need))
        self.short = max(0, want - back - len(self.free))
        if self.short:
            return False
        for r, m in zip(self.rows, need):
            self.free.extend(r[m:])
            del r[m:]
        for r, m in zip(self.rows, need):
            while len(r) < m:
                r.append(self.free.popleft())
        return True

    def places(self, ctx, cu, n_tok, delta=None):
        """(place, pos) of each token."""
        place, pos = [-1] * n_tok, [0] * n_tok
        for r, n in enumerate(ctx):
            for t in range(cu[r], cu[r + 1]):
                p = n - (cu[r + 1] - t)
                pos[t] = p + (delta[r] if delta is not None else 0)
                if p >= 0 and p // self.bs < len(self.rows[r]):
                    place[t] = self.rows[r][p // self.bs] * self.bs + p % self.bs
        return place, pos
