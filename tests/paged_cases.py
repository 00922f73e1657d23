"""Plain float64 forms of the paged serving operators (numpy and torch on the CPU) for the tests:
the 8-bit elements, a cache in pages, chunk attention, draft verification. They share nothing with
the library but the layouts."""
import math
from decimal import Decimal, getcontext

import numpy as np
import torch

BF16, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def e4m3_grid():
    """The 127 magnitudes of e4m3, ascending: four exponent bits of bias 7, three of fraction."""
    v = []
    for code in range(127):
        e, f = code >> 3, code & 7
        v.append(f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return np.array(v)


def quantised(x):
    """float64 x [..., dh] -> (values as stored, scale bytes), block by block."""
    grid = e4m3_grid()
    shape = x.shape
    B = min(32, shape[-1])
    x = x.reshape(-1, B)
    out, byte = np.zeros_like(x), np.zeros(len(x), np.uint8)
    for i, row in enumerate(x):
        if not np.all(np.isfinite(row)):
            out[i], byte[i] = np.nan, 255
            continue
        a, e = np.abs(row).max(), -110
        while a > 448.0 * 2.0 ** e:
            e += 1
        y = np.abs(row) * 2.0 ** -e
        hi = np.clip(np.searchsorted(grid, y), 1, 126)
        dlo, dhi = y - grid[hi - 1], grid[hi] - y
        up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
        out[i] = np.where(up, grid[hi], grid[hi - 1]) * np.sign(row) * 2.0 ** e
        byte[i] = e + 127
    return out.reshape(shape), byte.reshape(shape[:-1] + (shape[-1] // B,))


class Case:
    """A cache with random contents, its page table, and a chunk of rows per sequence."""

    def __init__(self, rows, lens, H=2, dh=64, page=16, dtype=BF16, e4=False, seed=0, stale=None,
                 pad=0, value_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.rows, self.lens = g, list(rows), list(lens)
        self.H, self.dh, self.page, self.dtype, self.e4 = H, dh, page, dtype, e4
        n = len(rows)
        need = [-(-L // page) for L in lens]
        self.n_pages = sum(need) + 2
        order = torch.randperm(self.n_pages, generator=g)
        self.table = torch.full((n, max(need + [1]) + 1), -1, dtype=torch.int32)
        at = 0
        for b in range(n):
            self.table[b, :need[b]] = order[at:at + need[b]].int()
            at += need[b]
        self.cu = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
        self.total = int(self.cu[-1]) + pad
        # what each position of each sequence holds, float64 [len][H][2][dh]
        self.kv = []
        pages = torch.full((self.n_pages, H, 2, page, dh), 0.0 if stale is None else stale,
                           dtype=torch.float64)
        scales = None
        B = min(32, dh)
        if e4:
            scales = torch.full((self.n_pages, H, 2, page, dh // B), 255 if stale is not None
                                else 127, dtype=torch.uint8)
        codes = torch.zeros(pages.shape, dtype=torch.uint8)
        for b, L in enumerate(lens):
            x = torch.randn((L, H, 2, dh), generator=g, dtype=torch.float64)
            x[:, :, 0] *= 1.5
            x[::2, :, 1] *= value_scale  # every other position
            x = x.to(dtype).double()
            if e4:
                v, s = quantised(x.numpy())
                held = torch.from_numpy(v)
                for p in range(L):
                    pg, sl = int(self.table[b, p // page]), p % page
                    sc = torch.from_numpy(s[p])
                    scales[pg, :, :, sl] = sc
                    y = (v[p].reshape(H, 2, -1, B) * 2.0 ** -(s[p].astype(float) - 127)[..., None])
                    codes[pg, :, :, sl] = torch.from_numpy(y.reshape(H, 2, dh)).float().to(
                        E4).view(torch.uint8)
            else:
                held = x
                for p in range(L):
                    pages[int(self.table[b, p // page]), :, :, p % page] = x[p]
            self.kv.append(held)
        self.pages = codes.view(E4) if e4 else pages.to(dtype)
        self.scales = scales

    def device(self):
        from token_recurrent_decoding_b200 import rlt
        self.d_pages = self.pages.cuda()
        self.d_scales = None if self.scales is None else self.scales.cuda()
        self.cache = rlt.PagedKV(self.d_pages, self.d_scales, dtype=self.dtype)
        self.d_table, self.d_cu = self.table.cuda(), self.cu.cuda()
        self.d_len = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return self

    def queries(self, heads, scale=1.0):
        """[total][heads][dh] as a part of wider rows."""
        wide = torch.randn((self.total, heads + 3, self.dh), generator=self.g) * scale
        return wide.to(self.dtype)[:, 1:heads + 1]


def attend64(q, kv, len_, window):
    """One sequence: q [m][Hq][dh], kv [len][H][2][dh], all float64 -> (out, lse, mass, size): mass
    the weighted |v| of each output, size the largest |q| . |k| / sqrt(dh) of the row."""
    m, Hq, dh = q.shape
    out, mass = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((m, Hq), -math.inf, dtype=torch.float64)
    size = torch.zeros((m, Hq), dtype=torch.float64)
    group = Hq // kv.shape[1]
    for i in range(m):
        pos = len_ - m + i
        lo = max(0, pos - window + 1) if window else 0
        if pos < lo or pos < 0:
            continue
        for h in range(Hq):
            k, v = kv[lo:pos + 1, h // group, 0], kv[lo:pos + 1, h // group, 1]
            s = k @ q[i, h] / math.sqrt(dh)
            p = torch.softmax(s, 0)
            out[i, h], mass[i, h] = p @ v, p @ v.abs()
            lse[i, h] = torch.logsumexp(s, 0)
            size[i, h] = (k.abs() @ q[i, h].abs()).max() / math.sqrt(dh)
    return out, lse, mass, size


def attend_bound(ref, mass, size, dh, dtype):
    """Largest error of an output, from the arithmetic: a score is a sum of dh products in fp32
    (each addition at most 2^-23 of the sum of magnitudes where the tensor cores cut instead of
    rounding, and the scale's and exponent's roundings: dh + 8 of them), which moves a weight by
    that factor; the weighted sum in fp32 over any length, added in parts of at most a few hundred
    (2^-23 * 512); a bf16 result adds the weights' and its own rounding to bf16, 2^-8 each."""
    ds = size.unsqueeze(-1) * (dh + 8) * 2.0 ** -23
    b = mass * (2 * ds + 512 * 2.0 ** -23) + 2.0 ** -22 * ref.abs()
    if dtype == BF16:
        b = b + 2.0 ** -8 * 1.01 * (mass + ref.abs())
    return b + 1e-30


def verify64(target, draft, tokens, lens, u, tau, digits=0):
    """float64 numpy arrays; tokens [n][k]. Returns (tokens, counts, margin): margin the least
    relative distance of a comparison from its border. digits: of decimal arithmetic instead of
    float64, where 1 - 1e-38 and 1 have to differ."""
    n, k1, V = target.shape
    k = k1 - 1
    out, counts, margin = np.full((n, k1), -1, np.int64), np.zeros(n, np.int64), math.inf

    def weights(x):
        x = np.where(np.isnan(x), -np.inf, x)
        top = x.max()
        if top == -np.inf:
            return np.zeros(V)
        if top == np.inf:
            w = (x == np.inf).astype(np.float64)
        elif digits:
            t = Decimal(float(tau))
            w = np.array([Decimal(0) if v == -np.inf else ((Decimal(float(v)) - Decimal(float(top)))
                                                           / t).exp() for v in x])
        else:
            w = np.exp((x - top) / tau)
        w[w < 2.0 ** -1000] *= 0
        return w / w.sum()

    if digits:
        getcontext().prec = digits
        u = np.array([[Decimal(float(v)) for v in row] for row in u])

    for b in range(n):
        L = min(max(int(lens[b]), 0), k)
        for i in range(L):
            if not 0 <= tokens[b, i] < V:
                L = i
                break
        j = 0
        while True:
            row = target[b, j]
            clean = np.where(np.isnan(row), -np.inf, row)
            if tau == 0:
                best = int(np.argmax(clean)) if clean.max() > -np.inf else -1
                if j < L and tokens[b, j] == best:
                    out[b, j] = best
                    j += 1
                    continue
                out[b, j] = best
                counts[b] = j + (best >= 0)
                break
            p = weights(row)
            q = None
            if j < L:
                x = tokens[b, j]
                if draft is not None:
                    q = weights(draft[b, j])
                else:
                    q = np.zeros(V) * p[0]
                    q[x] += 1
                a, c = u[b, j] * q[x], p[x]
                if max(a, c) > 0:
                    margin = min(margin, float(abs(a - c) / max(a, c)) if a != c else margin)
                if a < c:
                    out[b, j] = x
                    j += 1
                    continue
                r = np.maximum(p - q, 0)
                if r.sum() > 0:
                    p = r
            if p.sum() == 0:
                counts[b] = j
                break
            cum = np.cumsum(p)
            t = u[b, k] * cum[-1]
            margin = min(margin, float(np.abs(cum - t).min() / cum[-1]))
            v = int(np.searchsorted(cum, t, side="right"))
            out[b, j] = min(v, int(np.flatnonzero(p).max()))
            counts[b] = j + 1
            break
    return out, counts, margin
