"""A paged memory with its pages' accounting: sequences that begin, draft, fork and end apart.

"Transformer-XL: Attentive Language Models Beyond a Fixed-Length Context", §3.2
keeps one memory of M states per layer for a batch that advances in step.  A
:class:`PagedMemory` keeps the projected keys and values of M rows for every sequence
on its own, in pages of a common pool: a sequence's table of pages is a ring
that its memory slides through (so a running stream reuses its own pages and needs
no allocation), a fork shares the pages of its parent until either writes one,
and a sequence that ends gives its pages back.

The host keeps a copy of every sequence's table, begin and fill; what a call
changes goes to the device with it.  The rows themselves never leave the device.
"""

from __future__ import annotations

import numpy as np
import torch

from . import _lib as txl


class PagedMemory:
    """Memories of M rows for B sequences and ``layers`` layers, in a pool of
    ``n_pages`` pages (by default enough for all of them).  ``max_new``: the most
    rows appended at once.  ``kv`` is the :class:`PagedKV` for the attention."""

    def __init__(self, layers: int, B: int, H: int, M: int, max_new: int, *, device,
                 dtype=torch.bfloat16, page_rows: int = 64, n_pages: int | None = None, dh: int = 64):
        if M < 0 or max_new < 1:
            raise ValueError("PagedMemory: M >= 0 and max_new >= 1")
        self.M, self.max_new, self.B, self.layers = M, max_new, B, layers
        slots = -(-(M + max_new) // page_rows) + 1
        n = B * slots if n_pages is None else n_pages
        self.device = torch.device(device)
        pool = torch.zeros(2 * layers, n, H, page_rows, dh, dtype=dtype, device=self.device)
        table = torch.full((B, slots), -1, dtype=torch.int32, device=self.device)
        self.kv = txl.PagedKV(pool, table)
        self.pages = txl.PagePool(n)
        self._table = np.full((B, slots), -1, dtype=np.int32)
        self.begin = [0] * B
        self.fill = [0] * B

    # ---- host accounting --------------------------------------------------------

    def _ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.device)

    def _counts(self, n) -> list[int]:
        counts = [n] * self.B if isinstance(n, int) else [int(x) for x in n]
        if len(counts) != self.B or min(counts) < 0:
            raise ValueError("one count of rows per sequence, none negative")
        if max(counts) > self.max_new:
            raise ValueError(f"at most {self.max_new} rows at once")
        return counts

    def _sequence(self, b: int) -> int:
        if not 0 <= b < self.B:
            raise IndexError(f"no sequence {b} of {self.B}")
        return b

    def _upload(self):
        self.kv.table.copy_(torch.from_numpy(self._table))

    def _live(self, b: int, slot: int) -> bool:
        """Whether a memory row of sequence b lies in the page of this slot."""
        P, R = self.kv.page_rows, self.kv.rows
        first = (slot * P - self.begin[b]) % R     # ring distance from the oldest row
        return first < self.fill[b] or first + P > R and self.fill[b] > 0

    def reserve(self, n):
        """Make the pages of the next n rows (an int, or one count per sequence) the
        sequence's own: missing ones are allocated, ones shared with another sequence
        replaced, by a copy where they hold rows of the memory.  All or nothing: raises
        TxlError when the pool has too few free pages."""
        counts = self._counts(n)
        P, slots = self.kv.page_rows, self.kv.slots
        want, users = [], {}
        for b, c in enumerate(counts):
            if c == 0:
                continue
            x = self.begin[b] + self.fill[b]
            for s in range(x // P, (x + c - 1) // P + 1):
                page = int(self._table[b, s % slots])
                if page >= 0:
                    # (of the sequences that write a page they share, the last keeps it)
                    left = users.get(page, self.pages.users(page))
                    if left == 1:
                        continue
                    users[page] = left - 1
                want.append((b, s % slots))
        if not want:
            return
        src, dst = [], []
        for (b, s), new in zip(want, self.pages.alloc(len(want))):
            old = int(self._table[b, s])
            if old >= 0:
                if self._live(b, s):
                    src.append(old)
                    dst.append(new)
                self.pages.release([old])
            self._table[b, s] = new
        if src:
            txl.paged_copy(self.kv, self._ints(src), self._ints(dst))
        self._upload()

    def append(self, k, v, n=None, rows=None):
        """Append rows of k and v ([layers, B, H, N, dh]; with one layer also
        [B, H, N, dh]) and advance to the newest M.  n: rows per sequence (all N when
        omitted); rows: per sequence the source rows (e.g. the accepted nodes of a
        drafted tree), n then being their numbers."""
        idx = None
        if (k.shape[0] if k.dim() == 5 else 1) != self.layers:
            raise ValueError(f"k and v must hold the rows of all {self.layers} layers")
        if rows is not None:
            if n is None:
                n = [len(r) for r in rows]
            counts = self._counts(n)
            if len(rows) != self.B or any(len(r) < c for r, c in zip(rows, counts)):
                raise ValueError("rows: one list per sequence, of at least its count")
            width = max(counts)
            idx = np.zeros((self.B, width), dtype=np.int32)
            for b, c in enumerate(counts):
                idx[b, :c] = rows[b][:c]
                if c and not (0 <= idx[b, :c].min() and idx[b, :c].max() < k.shape[-2]):
                    raise ValueError(f"rows of sequence {b} are not rows of k and v")
            idx = torch.from_numpy(idx).to(self.device)
        else:
            counts = self._counts(k.shape[-2] if n is None else n)
            if max(counts) > k.shape[-2]:
                raise ValueError("more rows than k and v hold")
        self.reserve(counts)
        same = idx is None and min(counts) == k.shape[-2]
        txl.paged_append(self.kv, k, v, rows=idx,
                         n_new=None if same else self._ints(counts), keep=self.M)
        R = self.kv.rows
        for b, c in enumerate(counts):
            total = self.fill[b] + c
            self.fill[b] = min(total, self.M)
            self.begin[b] = (self.begin[b] + total - self.fill[b]) % R

    def rows(self, layer: int, b: int):
        """Copies of layer ``layer``'s keys and values of sequence b, each [H, fill, dh], oldest
        row first."""
        if not 0 <= layer < self.layers:
            raise IndexError(f"no layer {layer} of {self.layers}")
        x = (self.begin[self._sequence(b)] + np.arange(self.fill[b])) % self.kv.rows
        page, row = (torch.from_numpy(i.astype(np.int64)).to(self.device)
                     for i in (self._table[b, x // self.kv.page_rows], x % self.kv.page_rows))
        k, v = (self.kv.pool[2 * layer + i][page, :, row].transpose(0, 1).contiguous() for i in (0, 1))
        return k, v

    def free(self, b: int):
        """End sequence b: its memory is empty and its pages have one user less."""
        held = [int(p) for p in self._table[self._sequence(b)] if p >= 0]
        self.pages.release(held)
        self._table[b] = -1
        self.begin[b] = self.fill[b] = 0
        self.kv.begin[b:b + 1].zero_()
        self.kv.fill[b:b + 1].zero_()
        self._upload()

    def fork(self, src: int, dst: int):
        """Sequence dst becomes a copy of src, sharing its pages (dst's own are freed)."""
        if self._sequence(src) == self._sequence(dst):
            return
        self.free(dst)
        self.pages.retain([int(p) for p in self._table[src] if p >= 0])
        self._table[dst] = self._table[src]
        self.begin[dst], self.fill[dst] = self.begin[src], self.fill[src]
        self.kv.begin[dst:dst + 1].copy_(self.kv.begin[src:src + 1])
        self.kv.fill[dst:dst + 1].copy_(self.kv.fill[src:src + 1])
        self._upload()

    def trim(self) -> int:
        """Give back the pages without a row of any memory; returns how many became free."""
        freed = 0
        for b in range(self.B):
            for s in range(self.kv.slots):
                if self._table[b, s] >= 0 and not self._live(b, s):
                    freed += self.pages.release([int(self._table[b, s])])
                    self._table[b, s] = -1
        self._upload()
        return freed

    def compact(self) -> int:
        """Move the pages in use to the lowest ids (copying those that lie behind
        them); returns how many are in use."""
        used = sorted({int(p) for p in self._table.ravel() if p >= 0})
        users = {p: self.pages.users(p) for p in used}
        n = len(used)
        holes = sorted(set(range(n)) - set(used))
        moves = dict(zip([p for p in used if p >= n], holes))
        if moves:
            txl.paged_copy(self.kv, self._ints(list(moves)), self._ints(list(moves.values())))
        place = np.vectorize(lambda p: moves.get(p, p), otypes=[np.int32])
        self._table = place(self._table)
        self._recount({moves.get(p, p): c for p, c in users.items()})
        self._upload()
        return n

    def _recount(self, users: dict):
        """A fresh accounting: pages 0 .. len(users) - 1, each with its number of users."""
        self.pages = txl.PagePool(self.kv.n_pages)
        for p in self.pages.alloc(len(users)):
            for _ in range(users[p] - 1):
                self.pages.retain([p])

    # ---- checkpoint -------------------------------------------------------------

    def checkpoint(self) -> dict:
        """Host copy of the memory (compacted first)."""
        n = self.compact()
        return {"pool": self.kv.pool[:, :n].to("cpu", copy=True), "table": self._table.copy(),
                "begin": list(self.begin), "fill": list(self.fill), "M": self.M, "max_new": self.max_new,
                "users": [self.pages.users(p) for p in range(n)]}

    def restore(self, ck: dict):
        """Load a checkpoint (same shapes and options)."""
        pool = self.kv.pool[:, :len(ck["users"])]
        if (ck["table"].shape != self._table.shape or ck["pool"].shape != pool.shape or
                ck["pool"].dtype != pool.dtype):
            raise ValueError("restore: a memory of other shapes")
        # (slots are rounded up to pages: memories of other lengths can have tables of one shape)
        if ((ck.get("M", self.M), ck.get("max_new", self.max_new)) != (self.M, self.max_new) or
                max(ck["fill"]) > self.M):
            raise ValueError("restore: a memory of another length or of other appends")
        self._table = ck["table"].copy()
        self.begin, self.fill = list(ck["begin"]), list(ck["fill"])
        self._recount(dict(enumerate(ck["users"])))
        pool.copy_(ck["pool"])
        self.kv.begin.copy_(self._ints(self.begin))
        self.kv.fill.copy_(self._ints(self.fill))
        self._upload()
