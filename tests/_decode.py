"""Plain 64-bit forms of the speculative-decoding operators, for the tests."""
import math

import numpy as np
import torch

EPS = 1e-6


def angles(n_pos, rot):
    half = rot // 2
    f = 1e4 ** (-torch.arange(half, dtype=torch.float64) / half)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def split(x, rot, style):
    """Index pairs (a, b) the rotation mixes."""
    i = torch.arange(rot // 2)
    return (i, i + rot // 2) if style == "rotate_half" else (2 * i, 2 * i + 1)


def rotate(x, cs, pos, style, sign=1.0):
    """x [B, S, H, D] float64, cs fp32 table, pos [B, S]; NaN rows for positions outside."""
    rot = cs.shape[1]
    bad = (pos < 0) | (pos >= cs.shape[0])
    row = cs.double()[pos.clamp(0, cs.shape[0] - 1).long()][:, :, None]
    c, s = row[..., :rot // 2], sign * row[..., rot // 2:]
    a, b = split(x, rot, style)
    out = x.clone()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    out[bad] = math.nan
    return out


def norm_rope(x, w, cs, pos, style):
    x = x.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return rotate(x * r * w.double(), cs, pos, style)


def pair_size(x, w, cs, style):
    """|n_a| + |n_b| of every channel's pair before rotation: what its rounding errors scale with."""
    x = x.double()
    n = (x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()).abs()
    a, b = split(n, cs.shape[1], style)
    out = n.clone()
    out[..., a] = out[..., b] = n[..., a] + n[..., b]
    return out


def norm_rope_grad(g, x, w, cs, pos, style):
    """dx, dw and the sizes their fp32 errors scale with."""
    x, g, w = x.double(), g.double(), w.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    h = x * r
    t = rotate(g, cs, pos, style, sign=-1.0)
    tw = t * w
    dx = r * (tw - h * (tw * h).mean(-1, keepdim=True))
    ga = g.abs()
    a, b = split(ga, cs.shape[1], style)
    size_t = ga.clone()
    size_t[..., a] = size_t[..., b] = ga[..., a] + ga[..., b]
    size = r * (size_t * w.abs() + h.abs() * (size_t * w.abs() * h.abs()).mean(-1, keepdim=True))
    return dx, (t * h).sum((0, 1, 2)), size, (size_t * h.abs()).sum((0, 1, 2))


class Pages:
    """A paged cache on lists: one row, one block, one token at a time."""

    def __init__(self, k, v, table, lens, refs):
        self.k, self.v = k, v  # CPU tensors [layers, pages, heads, page, D]
        self.table, self.lens, self.refs = table, lens, refs
        self.page = k.shape[3]

    def truncate(self, rows, lens):
        for r, n in zip(rows, lens):
            self.lens[r] = min(self.lens[r], n)
            for j, e in enumerate(self.table[r]):
                if e >= 0 and j * self.page >= self.lens[r]:
                    self.refs[e] -= 1
                    self.table[r][j] = -1

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            for j in range(-(-self.lens[s] // self.page)):
                self.table[d][j] = self.table[s][j]
                self.refs[self.table[s][j]] += 1
            self.lens[d] = self.lens[s]

    def reserve(self, rows, counts):
        """False (and nothing changed) when the free pages do not suffice."""
        before = list(self.refs)
        wanted = []
        for r, n in zip(rows, counts):
            if n <= 0:
                continue
            for j in range(self.lens[r] // self.page, -(-(self.lens[r] + n) // self.page)):
                if j >= len(self.table[r]):
                    return False
                e = self.table[r][j]
                if e < 0 or before[e] > 1:
                    wanted.append((r, j, e))
        free = [p for p, c in enumerate(before) if c == 0]
        if len(wanted) > len(free):
            return False
        for (r, j, e), p in zip(wanted, free):
            if e >= 0:
                self.refs[e] -= 1
                if j * self.page < self.lens[r]:
                    self.k[:, p] = self.k[:, e]
                    self.v[:, p] = self.v[:, e]
            self.table[r][j] = p
            self.refs[p] = 1
        return True

    def slot(self, r, pos):
        return self.table[r][pos // self.page], pos % self.page

    def compact(self, rows, paths, counts):
        for r, path, n in zip(rows, paths, counts):
            moved = [[pool[:, self.slot(r, self.lens[r] + x)[0], :, self.slot(r, self.lens[r] + x)[1]].clone()
                      for x in path[:n]] for pool in (self.k, self.v)]
            for pool, vals in zip((self.k, self.v), moved):
                for j, val in enumerate(vals):
                    p, s = self.slot(r, self.lens[r] + j)
                    pool[:, p, :, s] = val
            self.lens[r] += n
            self.truncate([r], [self.lens[r]])


def random_tree(rng, nodes, branch):
    parents = [-1]
    for i in range(1, nodes):
        open_nodes = [p for p in range(i) if parents[1:].count(p) < branch] or [i - 1]
        parents.append(int(rng.choice(open_nodes)))
    return parents


def ancestors(parents):
    masks, depths = [], []
    for i, p in enumerate(parents):
        ok = 0 <= p < i
        masks.append((masks[p] if ok else 0) | (1 << i))
        depths.append(depths[p] + 1 if ok else 0)
    return masks, depths


def signed(masks):
    return torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in masks], dtype=torch.int64)


def attention(q, keys, values, visible, scale):
    """q [N, Hq, D], keys / values [T, Hk, D], visible [N, T] bool -> out float64, lse (0, -inf on empty rows).
    Also returns sum p |v|, what the rounding of p scales with."""
    N, Hq, D = q.shape
    G = Hq // keys.shape[1]
    out, lse = torch.zeros(N, Hq, D, dtype=torch.float64), torch.full((N, Hq), -math.inf, dtype=torch.float64)
    size = torch.zeros_like(out)
    for t in range(N):
        see = visible[t].nonzero()[:, 0]
        if not len(see):
            continue
        k, v = keys[see].double(), values[see].double()
        for h in range(Hq):
            s = k[:, h // G] @ q[t, h].double() * scale
            lse[t, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[t, h])
            out[t, h] = p @ v[:, h // G]
            size[t, h] = p @ v[:, h // G].abs()
    return out, lse, size


def verify(p, q, tokens, parents, accept, sample):
    """One request, one number at a time (float64 numpy rows)."""
    N, V = p.shape
    node, path = 0, [0]
    while True:
        a, R = 0.0, 1.0
        dist = p[node].astype(np.float64)
        reached = None
        for i in range(1, N):
            if parents[i] != node or not 0 <= parents[i] < i or not 0 <= tokens[i] < V:
                continue
            x = tokens[i]
            qx = float(q[node, x]) if q is not None else 1.0
            if float(accept[i]) * qx * R < dist[x]:
                reached = i
                break
            if q is not None:
                a += R
                dist = np.maximum(p[node].astype(np.float64) - a * q[node].astype(np.float64), 0)
                R = dist.sum()
            else:
                R -= dist[x]
                dist[x] = 0
        if reached is None:
            break
        node = reached
        path.append(node)
    if not dist.sum() > 0:
        dist = p[node].astype(np.float64)
    if not dist.sum() > 0:
        return path, -1
    c = np.cumsum(dist)
    t = float(sample) * c[-1]
    over = np.nonzero(c > t)[0]
    return path, int(over[0]) if len(over) else int(np.nonzero(dist)[0].max())
