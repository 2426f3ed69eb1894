"""Plain 64-bit forms of the tree-verification operators, and seeded inputs for
their GPU tests.  Nothing here uses the CUDA library."""
from __future__ import annotations

import math

import numpy as np
import torch

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype) -> float:
    """Largest relative error of rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def tiny_step(dtype) -> float:
    """Half a step of `dtype`'s subnormal numbers: the absolute error of rounding near 0."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def gen(seed: int) -> torch.Generator:
    return torch.Generator().manual_seed(seed)


def random_tree(n: int, g: torch.Generator) -> list[int]:
    return [int(torch.randint(-1, i, (), generator=g)) if i else -1 for i in range(n)]


def lineage(parent: list[int], i: int) -> list[int] | None:
    """Token i and its ancestors; None for a padded token or a descendant of one."""
    line = []
    while i >= 0:
        line.append(i)
        i = parent[i]
    return line if i == -1 else None


# ----------------------------------------------------------------- attention

class Trees:
    """A batch of trees over a paged cache, on the CPU.

    ctx, parents: cached rows and tree of each batch entry; pages are taken from a
    shuffled pool, what no sequence may read (rows beyond a length, free pages)
    holds NaN."""

    def __init__(self, ctx, parents, heads, kv_heads, dim, page, dtype, seed=0, extra_rows=0, extra_pages=3, poison=float("nan")):
        g = gen(seed)
        self.ctx, self.parents, self.page = list(ctx), [list(p) for p in parents], page
        self.heads, self.kv_heads, self.dim, self.dtype = heads, kv_heads, dim, dtype
        counts = [-(-c // page) for c in ctx]
        n_pages = sum(counts) + extra_pages
        b = len(ctx)
        order = torch.randperm(n_pages, generator=g).tolist()
        # sequences sit in the table in reverse order of the batch
        self.seqs = torch.tensor(list(range(b))[::-1], dtype=torch.int32)
        self.table = torch.full((b, max(1, max(counts)) + 1), -7, dtype=torch.int32)
        self.lens = torch.zeros(b, dtype=torch.int32)
        self.held = torch.zeros(b, dtype=torch.int32)
        self.refs = torch.zeros(n_pages, dtype=torch.int32)
        shape = (1, n_pages, kv_heads, page, dim)
        self.k = torch.full(shape, poison).to(dtype)
        self.v = torch.full(shape, poison).to(dtype)
        self.K, self.V = [], []
        for i, c in enumerate(ctx):
            s = int(self.seqs[i])
            mine = [order.pop() for _ in range(counts[i])]
            self.table[s, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            self.lens[s], self.held[s] = c, len(mine)
            K = torch.randn(c, kv_heads, dim, generator=g).to(dtype)
            V = torch.randn(c, kv_heads, dim, generator=g).to(dtype)
            for j, p in enumerate(mine):
                self.refs[p] = 1
                m = min(page, c - j * page)
                self.k[0, p, :, :m] = K[j * page:j * page + m].transpose(0, 1)
                self.v[0, p, :, :m] = V[j * page:j * page + m].transpose(0, 1)
            self.K.append(K)
            self.V.append(V)
        starts = [0]
        for p in self.parents:
            starts.append(starts[-1] + len(p))
        self.rows = starts[-1] + extra_rows
        self.q_start = torch.tensor(starts, dtype=torch.int32)
        self.parent = torch.tensor(sum(self.parents, []) + [-1] * extra_rows, dtype=torch.int32)
        self.max_nodes = max(1, max(len(p) for p in self.parents))
        self.q = torch.randn(self.rows, heads, dim, generator=g).to(dtype)
        self.k_new = torch.randn(self.rows, kv_heads, dim, generator=g).to(dtype)
        self.v_new = torch.randn(self.rows, kv_heads, dim, generator=g).to(dtype)
        self.scale = 1 / math.sqrt(dim)

    def reference(self, subnormal=2.0 ** -25):
        """(out, lse, tolerance of out, tolerance of lse) in 64 bits, for the rows of the trees.

        The kernel's errors, in units of u = half a step of the 16-bit type and of f32's 2^-24:
        a score is a sum of `dim` exact products in f32 (each addition off by at most 2^-23 of the
        sum of magnitudes: the tensor core may truncate), so ds = dim 2^-23 scale sum |q k| + the
        rounding of the exponent's product, 2^-23 |s| log2 e; a weight is off by a factor within
        e^(2 ds) and, rounded for the product with v, by u (or, for f16, by half a subnormal step,
        2^-25, where weights are at least 1 in sum); the sum over n keys adds n 2^-23; the result is
        rounded by u.

        subnormal: that half step, in units of the largest weight.  The kernel's weights are 2^6
        larger than their softmax numerators, so it keeps to 2^-31 as well."""
        G, D = self.heads // self.kv_heads, self.dim
        u = half_step(self.dtype)
        out = torch.zeros(self.rows, self.heads, D, dtype=torch.float64)
        lse = torch.full((self.rows, self.heads), -math.inf, dtype=torch.float64)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        for b, parent in enumerate(self.parents):
            a, c = int(self.q_start[b]), self.ctx[b]
            for i in range(len(parent)):
                line = lineage(parent, i)
                if line is None:
                    continue
                idx = [a + x for x in line]
                K = torch.cat([self.K[b], self.k_new[idx]]).double()
                V = torch.cat([self.V[b], self.v_new[idx]]).double()
                n = K.shape[0]
                for j in range(self.heads):
                    q, kk, vv = self.q[a + i, j].double(), K[:, j // G], V[:, j // G]
                    s = kk @ q * self.scale
                    mag = float((kk.abs() @ q.abs()).max()) * self.scale
                    ds = D * 2.0 ** -23 * mag + 2.0 ** -23 * 1.5 * float(s.abs().max())
                    w = torch.softmax(s, 0)
                    out[a + i, j] = w @ vv
                    lse[a + i, j] = torch.logsumexp(s, 0)
                    A = w @ vv.abs()
                    sub = n * subnormal * float(vv.abs().max()) if self.dtype == torch.float16 else 0.0
                    tol[a + i, j] = u * out[a + i, j].abs() + A * (1.01 * u + 2.5 * ds + (n + 16) * 2.0 ** -23) + sub + tiny_step(self.dtype)
                    ltol[a + i, j] = 1.5 * ds + (n + 16) * 2.0 ** -23 + float(lse[a + i, j].abs()) * 2.0 ** -21
        return out, lse, tol, ltol


# ------------------------------------------------------------------ norm, rope

def norm_rope(x, gamma, pos, rope, theta, eps):
    """x [n, heads, dim] -> 64-bit result and the magnitudes |z| the rotation mixes."""
    x = x.double()
    z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double()
    mag = z.abs().clone()
    if rope:
        i = torch.arange(rope // 2, dtype=torch.float64)
        ang = pos.double()[:, None] * theta ** (-2 * i / rope)
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        a, b = z[..., :rope // 2].clone(), z[..., rope // 2:rope].clone()
        z[..., :rope // 2] = a * c - b * s
        z[..., rope // 2:rope] = b * c + a * s
        m = a.abs() + b.abs()
        mag[..., :rope // 2] = m
        mag[..., rope // 2:rope] = m
    return z, mag


# -------------------------------------------------------------------- DeltaNet

def deltanet_tree(y, starts, parent, states, index, Hk, Hv):
    """64-bit outputs and states of every token (numpy); NaN states for padded tokens."""
    y, states = np.asarray(y, np.float64), np.asarray(states, np.float64)
    n = y.shape[0]
    o, snaps = np.zeros((n, Hv * 128)), np.full((n, Hv, 128, 128), np.nan)
    head = np.arange(Hv) // (Hv // Hk)
    for b in range(len(starts) - 1):
        par = list(parent[starts[b]:starts[b + 1]])
        for i in range(len(par)):
            row = starts[b] + i
            if lineage(par, i) is None:
                continue
            S = snaps[starts[b] + par[i]] if par[i] >= 0 else states[index[b]] if index[b] >= 0 else np.zeros((Hv, 128, 128))
            q, k, v, bb, aa = np.split(y[row], np.cumsum([Hk * 128, Hk * 128, Hv * 128, Hv]))
            q, k, v = q.reshape(Hk, 128)[head], k.reshape(Hk, 128)[head], v.reshape(Hv, 128)
            q = q / np.sqrt((q * q).sum(1, keepdims=True) + 1e-6)
            k = k / np.sqrt((k * k).sum(1, keepdims=True) + 1e-6)
            beta, alpha = 1 / (1 + np.exp(-bb)), 1 / (1 + np.exp(aa))
            Sk = np.einsum("hij,hj->hi", S, k)
            S = alpha[:, None, None] * (S - beta[:, None, None] * Sk[:, :, None] * k[:, None, :]) + (beta[:, None] * v)[:, :, None] * k[:, None, :]
            snaps[row] = S
            o[row] = np.einsum("hij,hj->hi", S, q).reshape(-1)
    return o, snaps


# ----------------------------------------------------------------------- pages

OK, E_ARG, E_STATE, E_OOM = 0, -1, -2, -3


class Pages:
    """The page operations, one request after another, on plain lists."""

    def __init__(self, n_pages, page_rows, n_seqs, max_pages):
        self.P, self.max_pages = page_rows, max_pages
        self.refs = [0] * n_pages
        self.rows = [[] for _ in range(n_seqs)]      # pages held
        self.lens = [0] * n_seqs
        self.copies = []                             # (from, to, rows) of the last extend

    def _named(self, seqs, i):
        return not 0 <= seqs[i] < len(self.rows) or seqs[i] in seqs[:i]

    def free(self, seqs):
        out = []
        for i, s in enumerate(seqs):
            if self._named(seqs, i):
                out.append(E_ARG)
                continue
            for p in self.rows[s]:
                self.refs[p] -= 1
            self.rows[s], self.lens[s] = [], 0
            out.append(OK)
        return out

    def fork(self, src, dst):
        out = []
        for i, (s, d) in enumerate(zip(src, dst)):
            if not 0 <= s < len(self.rows) or self._named(dst, i) or s in dst:
                out.append(E_ARG)
            elif self.rows[d] or self.lens[d]:
                out.append(E_STATE)
            else:
                self.rows[d] = self.rows[s][:-(-self.lens[s] // self.P)]
                self.lens[d] = self.lens[s]
                for p in self.rows[d]:
                    self.refs[p] += 1
                out.append(OK)
        return out

    def extend(self, seqs, add):
        """Requests that do not fail for their own reasons take pages in order; the first that the
        pool cannot serve and every later one that needs a page or shares its last one fail."""
        self.copies, out, plans = [], [], []
        total, refs = 0, list(self.refs)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        for i, (s, m) in enumerate(zip(seqs, add)):
            if self._named(seqs, i) or m < 0:
                out.append(E_ARG)
                continue
            n, held = self.lens[s], len(self.rows[s])
            want = -(-(n + m) // self.P)
            if want > self.max_pages:
                out.append(E_ARG)
                continue
            at = n // self.P
            span = self.rows[s][at:want] if m else []
            if any(self.refs[p] > 1 for p in span[1:]):
                out.append(E_STATE)
                continue
            copied = bool(span) and refs[span[0]] > 1
            shared = bool(span) and self.refs[span[0]] > 1
            need = int(copied) + (max(0, want - held) if m else 0)
            if copied:
                refs[span[0]] -= 1
            begin, total = total, total + need
            if total > len(free) and (need or shared):
                out.append(E_OOM)
                continue
            plans.append((s, at, copied, free[begin:total], n % self.P))
            out.append(OK)
        for s, at, copied, pages, rows in plans:
            if copied:
                old, new = self.rows[s][at], pages[0]
                self.refs[old] -= 1
                self.rows[s][at] = new
                self.copies.append((old, new, rows))
                pages_left = pages[1:]
            else:
                pages_left = pages
            self.rows[s] += pages_left
            for p in pages:
                self.refs[p] = 1
        return out
