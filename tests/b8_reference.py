"""Plain forms of the rotary positions and of the block-scaled 8-bit cache for
the tests: element by element from the definitions in include/kvq.h, in fp64
(attention, mass, rotation) or in the fp32 operations that the header pins
(codes and scales), on the CPU."""
import math

import numpy as np
import torch


def rotate(x, pos, inv_freq, factor, interleaved, inverse=False):
    """x [tokens, heads, D] -> fp64, pos [tokens]."""
    x = x.double().cpu().clone()
    ang = torch.outer(pos.double().cpu(), inv_freq.double().cpu()) * (-1 if inverse else 1)
    c, s = ang.cos()[:, None] * factor, ang.sin()[:, None] * factor
    r = 2 * inv_freq.numel()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    u, v = x[..., a].clone(), x[..., b].clone()
    x[..., a], x[..., b] = u * c - v * s, v * c + u * s
    return x


class Cache:
    """CPU copy of a B8Cache's planes with the header's append, read and evict."""

    def __init__(self, c):
        self.codes = {"k": c.k_codes.cpu().clone(), "v": c.v_codes.cpu().clone()}
        self.scales = {"k": c.k_scales.cpu().clone(), "v": c.v_scales.cpu().clone()}
        self.table = c.block_table.cpu().long()
        self.bs, self.dim, self.hkv = c.block_size, c.head_dim, c.num_kv_heads
        self.nb = c.num_blocks

    def page(self, b, t):
        """block of token t, -1 if it has none"""
        if t < 0 or t // self.bs >= self.table.shape[1]:
            return -1
        p = int(self.table[b, t // self.bs])
        return p if 0 <= p < self.nb else -1

    def put(self, w, page, h, row0, x, old_rows):
        """fp32 rows x [n, D] at row0 of a block that holds old_rows rows."""
        amax = x.abs().max()
        if amax < 2.0 ** -100:
            amax = amax * 0
        need = amax / torch.tensor(127.0)
        old = self.scales[w][page, h] if old_rows else torch.tensor(0.0)
        scale = torch.maximum(need, old)
        inv = torch.tensor(1.0) / scale if scale > 0 else torch.tensor(0.0)
        if old_rows and old > 0 and scale > old:
            c = self.codes[w][page, h, :old_rows].float()
            self.codes[w][page, h, :old_rows] = torch.round(c * (old / scale)).to(torch.int8)
        q = torch.round(x * inv).clamp(-127, 127).to(torch.int8)
        self.codes[w][page, h, row0:row0 + x.shape[0]] = q
        self.scales[w][page, h] = scale

    def append(self, b, start, k, v):
        """k, v [n, hkv, D] fp32 (already rotated) at tokens start ..."""
        n, first = k.shape[0], max(start, 0)
        t, end = first, start + n
        while t < end:
            stop = min(end, (t // self.bs + 1) * self.bs)
            p = self.page(b, t)
            if p >= 0:
                for w, x in (("k", k), ("v", v)):
                    for h in range(self.hkv):
                        self.put(w, p, h, t % self.bs, x[t - start:stop - start, h],
                                 t % self.bs if start > t // self.bs * self.bs else 0)
            t = stop

    def values(self, w, b, n):
        """fp64 [hkv, n, D] and a mask of the mapped tokens."""
        x = torch.zeros((self.hkv, n, self.dim), dtype=torch.float64)
        ok = torch.zeros(n, dtype=torch.bool)
        for t0 in range(0, n, self.bs):
            p, m = self.page(b, t0), min(self.bs, n - t0)
            if p >= 0:
                x[:, t0:t0 + m] = (self.codes[w][p, :, :m].double()
                                   * self.scales[w][p].double()[:, None, None])
                ok[t0:t0 + m] = True
        return x, ok

    def evict(self, into, b, n, mass, keep, recent, sinks):
        """mass [hkv, >= n] -> kept [hkv, m] per head; writes into `into`."""
        m = min(n, keep)
        kept = []
        for h in range(self.hkv):
            if n <= keep:
                ids = list(range(n))
            else:
                w = mass[h].tolist()
                key = [(-math.inf if x != x else -x) for x in w]  # NaN counts as largest
                nan = [x == x for x in w]
                mid = sorted(range(sinks, n - recent), key=lambda t: (nan[t], key[t], t))
                ids = sorted(list(range(sinks)) + mid[:m - sinks - recent]
                             + list(range(n - recent, n)))
            kept.append(ids)
        for c0 in range(0, m, into.bs):
            p = into.page(b, c0)
            if p < 0:
                continue
            for h in range(self.hkv):
                for w in ("k", "v"):
                    rows = []
                    for t in kept[h][c0:c0 + into.bs]:
                        q = self.page(b, t)
                        rows.append(self.codes[w][q, h, t % self.bs].float() * self.scales[w][q, h]
                                    if q >= 0 else torch.zeros(self.dim))
                    into.put(w, p, h, 0, torch.stack(rows), 0)
        return kept


def attention(ref, q, lens, cu, scale):
    """fp64 (out, lse, a) per query row; a: the largest |scale| * sum |q| |k| of
    the row, which bounds the rounding of its scores."""
    hq = q.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    a = torch.zeros(q.shape[:2], dtype=torch.float64)
    qd = q.double().cpu()
    for b, n in enumerate(lens):
        nq = cu[b + 1] - cu[b]
        k, ok = ref.values("k", b, n)
        v, _ = ref.values("v", b, n)
        see = ok[None] & (torch.arange(n)[None] <= n - nq + torch.arange(nq)[:, None])
        for h in range(hq):
            kh = h // (hq // ref.hkv)
            x = qd[cu[b]:cu[b + 1], h]
            s = (x @ k[kh].T * scale).masked_fill(~see, -math.inf)
            live = see.any(1)
            t = torch.logsumexp(s, 1)
            p = torch.where(live[:, None], torch.exp(s - t[:, None]), 0.0)
            out[cu[b]:cu[b + 1], h] = p @ v[kh]
            lse[cu[b]:cu[b + 1], h] = t
            if n:
                a[cu[b]:cu[b + 1], h] = (x.abs() @ k[kh].abs().T).amax(1) * abs(scale)
    return out, lse, a


def mass(ref, q, lse, lens, cu, scale, into):
    """fp64 into [batch, hkv, T] plus the weights of each token."""
    into = into.double().cpu().clone()
    qd, ld = q.double().cpu(), lse.double().cpu()
    for b, n in enumerate(lens):
        nq = cu[b + 1] - cu[b]
        k, ok = ref.values("k", b, n)
        see = ok[None] & (torch.arange(n)[None] <= n - nq + torch.arange(nq)[:, None])
        for h in range(q.shape[1]):
            kh = h // (q.shape[1] // ref.hkv)
            s = qd[cu[b]:cu[b + 1], h] @ k[kh].T * scale
            t = ld[cu[b]:cu[b + 1], h, None]
            p = torch.where(see & torch.isfinite(t), torch.exp(s - t), 0.0)
            into[b, kh, :n] += p.sum(0)
    return into
