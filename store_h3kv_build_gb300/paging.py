"""Which sequence owns which pages of a PagedStore: bookkeeping on the host.

A ``PagePool`` hands out pages, lets sequences share them (a fork), takes them
back, and says which pages the device has to copy before a shared one is
written.  It holds no tensor data and launches nothing: the rows, page tables
and page pairs that it returns go to ``binding.paged_append``,
``binding.attend_tree``, ``binding.paged_keep`` and ``binding.paged_copy``.

Pages are handed out lowest first, so the same calls give the same pages.  A
call that cannot be met raises and leaves the pool as it was.
"""
from __future__ import annotations

import heapq

import torch


class PoolFull(RuntimeError):
    """Not enough free pages for the call; nothing was changed."""


class PagePool:
    def __init__(self, pages: int, page_size: int = 64):
        if page_size not in (16, 32, 64, 128):
            raise ValueError(f"page_size {page_size}, expected 16, 32, 64 or 128")
        if pages < 0 or pages * page_size > 2 ** 31 - 256:
            raise ValueError(f"{pages} pages of {page_size} rows: rows are numbered in 31 bits")
        self.pages, self.page_size = int(pages), int(page_size)
        self._free = list(range(self.pages))  # a heap
        self._refs = [0] * self.pages
        self._table: dict[int, list[int]] = {}
        self._length: dict[int, int] = {}
        self._next = 0

    # ------------------------------------------------------------- reading --
    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, seq: int) -> int:
        return self._length[seq]

    def pages_of(self, seq: int) -> tuple[int, ...]:
        return tuple(self._table[seq])

    def sequences(self) -> tuple[int, ...]:
        return tuple(self._table)

    def rows(self, seq: int, start: int = 0, stop: int | None = None) -> torch.Tensor:
        """Pool rows of the sequence's tokens start .. stop-1 (int32, CPU)."""
        stop = self._length[seq] if stop is None else stop
        if not 0 <= start <= stop <= self._length[seq]:
            raise ValueError(f"tokens {start} .. {stop} of a sequence of {self._length[seq]}")
        pos = torch.arange(start, stop)
        table = torch.tensor(self._table[seq] or [0])
        return (table[pos // self.page_size] * self.page_size + pos % self.page_size).to(torch.int32)

    def table(self, seqs, max_pages: int | None = None) -> torch.Tensor:
        """Page table [len(seqs), max_pages] (int32, CPU); entries behind a
        sequence's last page are -1."""
        need = max((len(self._table[s]) for s in seqs), default=0)
        max_pages = max(need, 1) if max_pages is None else int(max_pages)
        if max_pages < need:
            raise ValueError(f"max_pages {max_pages}, a sequence has {need}")
        out = torch.full((len(seqs), max_pages), -1, dtype=torch.int32)
        for i, s in enumerate(seqs):
            t = self._table[s]
            out[i, :len(t)] = torch.tensor(t, dtype=torch.int32)
        return out

    def lengths(self, seqs) -> torch.Tensor:
        return torch.tensor([self._length[s] for s in seqs], dtype=torch.int32)

    # ------------------------------------------------------------ changing --
    def new(self) -> int:
        """An empty sequence."""
        seq, self._next = self._next, self._next + 1
        self._table[seq], self._length[seq] = [], 0
        return seq

    def _take(self) -> int:
        page = heapq.heappop(self._free)
        self._refs[page] = 1
        return page

    def _drop(self, page: int) -> None:
        self._refs[page] -= 1
        if self._refs[page] == 0:
            heapq.heappush(self._free, page)

    def own(self, seq: int, start: int) -> list[tuple[int, int]]:
        """Make the pages of tokens start and on belong to this sequence alone:
        (from, to) pages for paged_copy, to be copied before they are written
        (before paged_keep moves rows of a forked sequence, say)."""
        table = self._table[seq]
        if not 0 <= start <= self._length[seq]:
            raise ValueError(f"token {start} of a sequence of {self._length[seq]}")
        shared = [i for i in range(start // self.page_size, len(table)) if self._refs[table[i]] > 1]
        if len(shared) > len(self._free):
            raise PoolFull(f"{len(shared)} pages to copy, {len(self._free)} free")
        pairs = []
        for i in shared:
            page = self._take()
            pairs.append((table[i], page))
            self._drop(table[i])
            table[i] = page
        return pairs

    def extend(self, seq: int, tokens: int) -> tuple[torch.Tensor, list[tuple[int, int]]]:
        """Room for `tokens` more tokens: (their pool rows for paged_append,
        pages to be copied before).  A last page that is shared and not full
        is copied, since its free rows are written."""
        if tokens < 0:
            raise ValueError(f"{tokens} tokens")
        table, n = self._table[seq], self._length[seq]
        tail_shared = tokens > 0 and n % self.page_size != 0 and self._refs[table[-1]] > 1
        more = -(-(n + tokens) // self.page_size) - len(table)
        if more + tail_shared > len(self._free):
            raise PoolFull(f"{more + tail_shared} pages needed, {len(self._free)} free")
        pairs = self.own(seq, n) if tail_shared else []
        table.extend(self._take() for _ in range(more))
        self._length[seq] = n + tokens
        return self.rows(seq, n), pairs

    def truncate(self, seq: int, length: int) -> None:
        """Drop the tokens from `length` on (after paged_keep, say) and the
        pages that hold none any more."""
        if not 0 <= length <= self._length[seq]:
            raise ValueError(f"length {length} of a sequence of {self._length[seq]}")
        table = self._table[seq]
        keep = -(-length // self.page_size)
        for page in table[keep:]:
            self._drop(page)
        del table[keep:]
        self._length[seq] = length

    def fork(self, seq: int) -> int:
        """A new sequence with the same tokens, sharing every page."""
        table, length = list(self._table[seq]), self._length[seq]
        child = self.new()
        for page in table:
            self._refs[page] += 1
        self._table[child], self._length[child] = table, length
        return child

    def free(self, seq: int) -> None:
        for page in self._table.pop(seq):
            self._drop(page)
        del self._length[seq]

    def compact(self) -> list[tuple[int, int]]:
        """Move the highest used pages into the lowest free ones until the used
        pages are the first ones of the pool: (from, to) pages for paged_copy,
        to be copied before the next write; tables change to the new places."""
        used = self.pages - len(self._free)
        to = sorted(p for p in self._free if p < used)
        old = [p for p in range(used, self.pages) if self._refs[p]]
        move = dict(zip(old, to))
        for a, b in move.items():
            self._refs[b], self._refs[a] = self._refs[a], 0
        for table in self._table.values():
            table[:] = [move.get(p, p) for p in table]
        self._free = list(range(used, self.pages))
        return list(move.items())
