"""The full-rank serving operators from their definitions (``include/lrkv_serve.h``):
attention with score modifiers in fp64, the 8-bit pages' quantisation step by step in
fp32 as specified, and the page operations on host lists.  Torch tensors in, any device.
"""
import math

import torch

QMAX = {"int8": 127.0, "e4m3": 448.0}
KIND = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TINY = 2.0 ** -100


def attend(q, k, v, pos, lo, hi, scale=0.0, softcap=0.0, slope=None):
    """One sequence and head: rows q [n,d] at positions pos [n] see keys lo..hi of k, v [T,d].
    Returns fp64 (out [n,d], mean |v| under the same weights [n,d], sum |v| over seen keys
    relative to the sum of weights (largest weight 1) [n,d], largest seen |score| [n],
    largest seen sum |q k| scale [n])."""
    q, k, v = q.double(), k.double(), v.double()
    n, d = q.shape
    T = k.shape[0]
    if T == 0 or n == 0:
        z = torch.zeros(n, d, dtype=torch.float64, device=q.device)
        return z, z, z, z[:, 0], z[:, 0]
    scale = scale or 1.0 / math.sqrt(d)
    key = torch.arange(T, device=q.device)
    seen = (key >= lo[:, None]) & (key <= hi[:, None])
    some = seen.any(0)                       # what no row sees may be anything
    k = torch.where(some[:, None], k, torch.zeros_like(k))
    v = torch.where(some[:, None], v, torch.zeros_like(v))
    s = q @ k.T * scale
    size = q.abs() @ k.abs().T * scale
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    if slope is not None:
        s = s - float(slope) * (pos[:, None] - key).abs()
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.max(1, keepdim=True).values
    p = torch.exp(s - top.clamp_min(-1e300))
    p = torch.where(seen, p, torch.zeros_like(p))
    total = p.sum(1, keepdim=True)
    safe = total.clamp_min(1e-300)
    zero = torch.zeros_like(s)
    return (p @ v / safe, p @ v.abs() / safe, seen.double() @ v.abs() / safe.clamp_min(1.0),
            torch.where(seen, s, zero).abs().max(1).values, torch.where(seen, size, zero).max(1).values)


def rows_seen(pos, total, window=0, first_key=None, prefix_end=None):
    """First and last key that rows at positions pos see (lo > hi: none)."""
    lo = torch.zeros_like(pos) if first_key is None else first_key.to(pos).clamp_min(0)
    if window:
        lo = torch.maximum(lo, pos - window + 1)
    hi = pos if prefix_end is None else torch.maximum(pos, prefix_end.to(pos) - 1)
    return lo, hi.clamp_max(total - 1)


def round_codes(x, code):
    """fp32 values in units of their scale as codes (nearest, ties to even), fp32."""
    x = x.clamp(-QMAX[code], QMAX[code])
    return x.round() if code == "int8" else x.to(torch.float8_e4m3fn).float()


def append_page(codes, scale, rows, held, code):
    """One page and head: `held` rows of codes [page,d] (fp32) under `scale` (fp32 scalar
    tensor), then the new rows [n,d] (bf16).  Returns (codes, scale), every step in fp32."""
    f32 = torch.float32
    x = rows.to(f32)
    big = torch.tensor(3.3895313892515355e38, dtype=f32, device=x.device)
    x = torch.where(x.isnan(), torch.zeros_like(x), x)
    x = torch.where(x.isinf(), torch.copysign(big, x), x)
    before = scale if held else torch.zeros_like(scale)
    # a tensor divisor: a scalar one may be multiplied by its reciprocal
    s = torch.maximum(before, x.abs().max() / torch.full_like(scale, QMAX[code]))
    if float(s) < TINY:
        s = torch.zeros_like(s)
    inv = torch.ones_like(s) / s if float(s) > 0 else torch.zeros_like(s)
    out = codes.clone()
    if held and bool(s > before):
        out[:held] = round_codes(codes[:held] * (before * inv), code)
    out[held:held + len(x)] = round_codes(x * inv, code)
    return out, s


class Pool:
    """Reference counts, page table and lengths on the host, with the rules of lrkv_pages_*."""

    def __init__(self, table, refs, seq_len, page):
        self.table = [list(r) for r in table]
        self.refs, self.len, self.page = list(refs), list(seq_len), page
        self.moves = []          # (source, target) of copied pages, in any order
        self.status = 0

    def free_ids(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def reserve(self, counts):
        ended = False
        for b, n in enumerate(counts):
            if n == 0:
                continue
            if self.len[b] + n > len(self.table[b]) * self.page:
                self.status |= 0x2
                continue
            stop = -(-(self.len[b] + n) // self.page)
            slot = self.len[b] // self.page
            while slot < stop and self.table[b][slot] >= 0:
                slot += 1
            need = stop - slot
            if need <= 0:
                continue
            free = self.free_ids()
            if ended or need > len(free):
                ended = True
                self.status |= 0x20
                continue
            for i in range(need):
                self.table[b][slot + i] = free[i]
                self.refs[free[i]] = 1

    def page_ok(self, b, slot):
        return 0 <= self.table[b][slot] < len(self.refs)

    def advance(self, counts):
        for b, n in enumerate(counts):
            if self.len[b] + n > len(self.table[b]) * self.page:
                self.status |= 0x2
            for _ in range(n):                   # token by token, to the first that has no page
                slot = self.len[b] // self.page
                if slot >= len(self.table[b]):
                    break
                if not self.page_ok(b, slot):
                    self.status |= 0x10
                    break
                self.len[b] += 1

    def fork(self, src, dst):
        B = len(self.table)
        was = list(self.len)
        named, plan = set(), []
        for s, d in zip(src, dst):
            fresh = 0 <= d < B and d not in named
            if 0 <= d < B:
                named.add(d)
            if not (0 <= s < B and fresh and s != d and was[d] == 0 and self.table[d][0] < 0):
                self.status |= 0x40
                continue
            if was[s] % self.page and not self.page_ok(s, was[s] // self.page):
                self.status |= 0x10
                continue
            plan.append((s, d))
        old = [list(r) for r in self.table]
        free = self.free_ids()
        for s, d in plan:
            full, part = divmod(was[s], self.page)
            if part and not free:
                self.status |= 0x20
                break
            for i in range(full):
                self.table[d][i] = old[s][i]
                self.refs[old[s][i]] += 1
            if part:
                own = free.pop(0)
                self.refs[own] = 1
                self.table[d][full] = own
                self.moves.append((old[s][full], own))
            self.len[d] = was[s]

    def free(self, seqs):
        done = set()
        for b in seqs:
            if not 0 <= b < len(self.table) or b in done:
                self.status |= 0x40
                continue
            done.add(b)
            for i, page in enumerate(self.table[b]):
                if page >= 0:
                    self.refs[page] -= 1
                self.table[b][i] = -1
            self.len[b] = 0

    def copy(self, src, dst):
        n = len(self.refs)
        named = {d for d in dst if 0 <= d < n}
        done = set()
        for s, d in zip(src, dst):
            ok = 0 <= d < n and d not in done
            done.add(d)
            if not ok or not 0 <= s < n or s in named:
                self.status |= 0x10
                continue
            self.moves.append((s, d))

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        src = [i for i, r in enumerate(self.refs) if r > 0 and i >= live]
        dst = [i for i, r in enumerate(self.refs) if r <= 0 and i < live]
        to = dict(zip(src, dst))
        self.moves += list(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
