"""Windowed and tree attention over a paged cache in fp64, and a pool of pages in plain Python.

Used by the tests only; shares nothing with the library."""
from __future__ import annotations

import torch


def window_rule(window: int, sinks: int):
    """seen(length, R) -> bool [R, length]: the tokens each of a request's rows sees."""
    def seen(length, R, request):
        p = torch.arange(length - R, length)[:, None]
        j = torch.arange(length)[None, :]
        return (j <= p) & ((j < sinks) | (j > p - window))
    return seen


def tree_rule(mask: torch.Tensor):
    """The same for a tree's mask words int32 [N, R, ceil(R / 32)]."""
    def seen(length, R, request):
        base = length - R
        got = torch.zeros(R, length, dtype=torch.bool)
        got[:, :max(base, 0)] = True
        for i in range(R):
            for b in range(R):
                if (int(mask[request, i, b // 32]) >> (b % 32)) & 1 and 0 <= base + b < length:
                    got[i, base + b] = True
        return got
    return seen


def attention(cache, q, tables, lens, R, scale, rule):
    """out, and the magnitudes a tolerance is made of: sum_j w_j |v_j|, the largest |v_j| seen,
    sm_scale max_j sum_d |q_d k_jd| and sm_scale max_d |q_d| max_j sum_d |k_jd|.  cache: dict of CPU tensors (codes float8 e4m3 or uint8,
    scales); q [N R, Hq, 128]; all fp64 [N R, Hq, 128] (the last three [N R, Hq, 1])."""
    f8 = torch.float8_e4m3fn
    bs = cache["block_size"]
    H = cache["k_codes"].shape[1]
    rows, Hq, D = q.shape
    G = Hq // H
    out = torch.zeros(rows, Hq, D, dtype=torch.float64)
    mag, big = torch.zeros_like(out), torch.zeros(rows, Hq, 1, dtype=torch.float64)
    dot, peak = torch.zeros_like(big), torch.zeros_like(big)
    for r, length in enumerate(lens):
        if length == 0:
            continue
        j = torch.arange(length)
        page = tables[r, j // bs].long()
        sees = rule(length, R, r)
        any_row = sees.any(dim=0)
        slot = torch.where(any_row, page * bs + j % bs, torch.zeros_like(j))
        for h in range(H):
            k = cache["k_codes"][slot, h].view(f8).double() * cache["k_scales"][slot, h].double()[:, None]
            v = cache["v_codes"][slot, h].view(f8).double() * cache["v_scales"][slot, h].double()[:, None]
            k[~any_row] = 0
            v[~any_row] = 0
            for i in range(R):
                if not bool(sees[i].any()):
                    continue
                at = sees[i].nonzero()[:, 0]
                x = q[r * R + i, h * G:(h + 1) * G].double()
                s = (x @ k[at].T) * scale
                w = torch.exp(s - s.amax(dim=-1, keepdim=True))
                w = w / w.sum(dim=-1, keepdim=True)
                out[r * R + i, h * G:(h + 1) * G] = w @ v[at]
                mag[r * R + i, h * G:(h + 1) * G] = w @ v[at].abs()
                big[r * R + i, h * G:(h + 1) * G] = v[at].abs().max()
                dot[r * R + i, h * G:(h + 1) * G, 0] = \
                    abs(scale) * (x.abs() @ k[at].abs().T).amax(dim=-1)
                peak[r * R + i, h * G:(h + 1) * G, 0] = \
                    abs(scale) * x.abs().amax(dim=-1) * k[at].abs().sum(dim=-1).max()
    return out, mag, big, dot, peak


class Pool:
    """References and the stack of free pages, one entry at a time."""

    def __init__(self, num_pages: int):
        self.refs = [0] * num_pages
        self.free = list(range(num_pages))           # the top is the last

    def take(self) -> int:
        page = self.free.pop()
        self.refs[page] = 1
        return page

    def alloc(self, tables, begin, end):
        """Entries of the tables (lists) that get a page; requests that do not fit get -1."""
        want = 0
        room = len(self.free)
        for row, b, e in zip(tables, begin, end):
            want += e - b
            for i in range(b, e):
                row[i] = self.take() if want <= room else -1

    def release(self, tables, begin, end):
        back = set()
        for row, b, e in zip(tables, begin, end):
            for page in row[b:e]:
                if page >= 0 and self.refs[page] > 0:
                    self.refs[page] -= 1
                    if self.refs[page] == 0:
                        back.add(page)
        self.free += sorted(back)

    def fork(self, parents, tables, lens, child_tables, bs):
        """The children's lengths and the copies (source slot, target slot, rows)."""
        out, copies = [], []
        for i, p in enumerate(parents):
            if p < 0 or (lens[p] % bs and not self.free):
                out.append(0)
                continue
            full, rest = divmod(lens[p], bs)
            for k in range(full):
                child_tables[i][k] = tables[p][k]
                self.refs[tables[p][k]] += 1
            if rest:
                page = self.take()
                child_tables[i][full] = page
                copies.append((tables[p][full] * bs, page * bs, rest))
            out.append(lens[p])
        return out, copies
