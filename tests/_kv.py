"""Plain forms of the KV-cache calls for the tests: the step's plan by a loop,
q4_0 encoding in numpy fp32, attention in float64 over the oracle's decode."""
import numpy as np
import torch

import oracle

Q4_0 = 2


def pages(x, page):
    return -(-int(x) // page)


def plan(cached, new, table, free, taken, page, cap):
    """(seq_lens, cu_new, slots, positions, table, taken) of inputs that fit."""
    table = table.copy()
    cu, slots, pos = [0], [], []
    for b, (c, m) in enumerate(zip(cached, new)):
        for p in range(c, c + m):
            if p % page == 0:
                table[b, p // page] = free[taken]
                taken += 1
            slots.append(table[b, p // page] * page + p % page)
            pos.append(p)
        cu.append(cu[-1] + m)
    pad = [-1] * (cap - len(slots))
    return np.add(cached, new), np.array(cu), np.array(slots + pad), np.array(pos + pad), table, taken


def encode(x):
    """q4_0 wire bytes uint8 [..., n / 32 * 18] of fp32 values [..., n]."""
    x = np.asarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = np.take_along_axis(b, np.abs(b).argmax(-1)[..., None], -1)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        d = (top / np.float32(-8)).astype(np.float32)
        h = d.astype(np.float16)
        inv = np.where(h == 0, np.float32(0), (np.float32(1) / d).astype(np.float32))
        code = np.clip(np.trunc((b * inv).astype(np.float32) + np.float32(8.5)), 0, 15).astype(np.uint8)
    return np.concatenate([h.view(np.uint8).reshape(*h.shape[:-1], 2), code[..., :16] | (code[..., 16:] << 4)],
                          -1).reshape(*x.shape[:-1], -1)


def random_rows(rng, shape, d, lo=-4.0, hi=0.0):
    """Random q4_0 rows [*shape, d / 32 * 18]: scales of both signs, 2^lo .. 2^hi."""
    s = (2.0 ** rng.uniform(lo, hi, (*shape, d // 32)) * rng.choice([-1, 1], (*shape, d // 32))).astype(np.float16)
    code = rng.integers(0, 256, (*shape, d // 32, 16), dtype=np.uint8)
    return np.concatenate([s[..., None].view(np.uint8), code], -1).reshape(*shape, -1)


class Case:
    """Sequences [(keys, new tokens)] over shuffled pages; every byte that
    belongs to no visible token is 0xff (a scale that is not a number)."""

    def __init__(self, seqs, hq, hkv, d, page, seed=0, k_exp=(-4.0, -1.0), v_exp=(-4.0, 0.0), q_scale=1.0, pad=0, spare=2):
        rng = np.random.default_rng(seed)
        self.seqs, self.hq, self.hkv, self.d, self.page = seqs, hq, hkv, d, page
        need = [pages(n, page) for n, _ in seqs]
        self.n_pages = sum(need) + 3
        row = d // 32 * 18
        perm = rng.permutation(self.n_pages)
        most = max(need + [0]) + spare
        self.table = np.full((len(seqs), most), -1, np.int32)
        self.k = np.full((self.n_pages, hkv, page, row), 255, np.uint8)
        self.v = self.k.copy()
        at = 0
        for b, (n, _) in enumerate(seqs):
            self.table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            for j in range(need[b]):
                m = min(page, n - j * page)
                self.k[self.table[b, j], :, :m] = random_rows(rng, (hkv, m), d, *k_exp)
                self.v[self.table[b, j], :, :m] = random_rows(rng, (hkv, m), d, *v_exp)
        self.lens = np.array([n for n, _ in seqs], np.int32)
        self.cu = np.concatenate([[0], np.cumsum([m for _, m in seqs])]).astype(np.int32)
        t = int(self.cu[-1]) + pad
        self.q = (torch.from_numpy(rng.standard_normal((t, hq, d)).astype(np.float32)) * q_scale).to(torch.bfloat16)
        self.max_new = max([m for _, m in seqs] + [1])

    def rows(self, pool, b, h):
        n = int(self.lens[b])
        ids = self.table[b, :pages(n, self.page)]
        raw = pool[ids, h].reshape(-1, pool.shape[-1])[:n]
        if n == 0:
            return np.zeros((0, self.d))
        return oracle.dequantize(Q4_0, np.ascontiguousarray(raw), self.d).astype(np.float64)

    def steps(self, b, h):
        """8 |d| of every cached value: the largest magnitude that its block holds."""
        n = int(self.lens[b])
        raw = self.v[self.table[b, :pages(n, self.page)], h].reshape(-1, self.d // 32, 18)[:n]
        d = np.ascontiguousarray(raw[..., :2]).view(np.float16).astype(np.float64)
        return np.repeat(8 * np.abs(np.where(np.isfinite(d), d, 0)), 32, -1).reshape(n, self.d)

    def expected(self, scale, causal=True, window=0, hidden=()):
        """(output, sum of p |v|, largest scale * sum |q k|, sum of p 8 |d|) in
        float64; `hidden`: (sequence, block) pairs whose keys do not count."""
        t = int(self.cu[-1])
        out, mag = np.zeros((t, self.hq, self.d)), np.zeros((t, self.hq, self.d))
        big, step = np.zeros((t, self.hq, 1)), np.zeros((t, self.hq, self.d))
        q = self.q.double().numpy()
        grp = self.hq // self.hkv
        for b, (n, m) in enumerate(self.seqs):
            if m == 0:
                continue
            n = int(self.lens[b])
            pos = n - m + np.arange(m)
            key = np.arange(n)
            see = np.ones((m, n), bool)
            if causal:
                see &= key <= pos[:, None]
            if window:
                see &= key > pos[:, None] - window
            for hb, j in hidden:
                if hb == b:
                    see &= (key // self.page != j)[None]
            for h in range(self.hkv):
                k, v = self.rows(self.k, b, h), self.rows(self.v, b, h)
                for a in range(h * grp, (h + 1) * grp):
                    qi = q[self.cu[b]:self.cu[b] + m, a]
                    s = np.where(see, qi @ k.T * scale, -np.inf)
                    if n == 0:
                        continue
                    top = s.max(-1, keepdims=True)
                    e = np.exp(s - np.where(np.isfinite(top), top, 0))
                    z = e.sum(-1, keepdims=True)
                    p = np.divide(e, z, out=np.zeros_like(e), where=z > 0)
                    rows = slice(self.cu[b], self.cu[b] + m)
                    out[rows, a] = p @ np.where(np.isfinite(v), v, 0)
                    mag[rows, a] = p @ np.abs(np.where(np.isfinite(v), v, 0))
                    step[rows, a] = p @ self.steps(b, h)
                    big[rows, a, 0] = (np.where(see, np.abs(qi) @ np.abs(k).T, 0)).max(-1) * abs(scale)
        return out, mag, big, step
