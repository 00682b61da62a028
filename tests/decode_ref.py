"""Plain models of the decode-step operators for the tests: 4-bit packing and products, the paged
cache's bookkeeping written as loops over Python lists, and attention in 64 bits."""
import numpy as np
import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2  # relative error of one rounding to bf16
F32_STEP = 2.0 ** -23  # one binary32 operation, also where a sum is cut off instead of rounded


def bf16(a):
    """Nearest bf16 of an array, as a CPU tensor."""
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


# --------------------------------------------------------------------------- 4-bit weights
def w4_pack_codes(t):
    """t (N, K) in [-8, 7] -> bytes, straight from the format's bit positions."""
    N, K = t.shape
    blocks = -(-K // 128)
    words = np.zeros((N, blocks * 16), np.uint32)
    for k in range(blocks * 128):
        code = (t[:, k] + 8 if k < K else np.full(N, 8)).astype(np.uint32)
        r = k % 128
        j, c, i = r // 32, r % 32 // 8, r % 8
        shift = 2 * i if i % 2 == 0 else 2 * i + 14
        words[:, k // 128 * 16 + 4 * c + j] |= code << np.uint32(shift)
    return words.view(np.uint8).reshape(N, -1)


def w4_quantise(W, group):
    """Codes t and bf16 scales of W, in binary32 as the format defines them."""
    N, K = W.shape
    groups = -(-K // group)
    t = np.zeros((N, K), np.int64)
    scales = torch.zeros(N, groups, dtype=torch.bfloat16)
    for g in range(groups):
        part = W[:, g * group:(g + 1) * group]
        amax = np.maximum(np.abs(part).max(1), np.float32(1e-5)).astype(np.float32)
        s = bf16(amax / np.float32(7))
        scales[:, g] = s
        t[:, g * group:(g + 1) * group] = np.clip(np.rint(part / s.float().numpy()[:, None]), -8, 7)
    return t, scales


def w4_linear(x, t, scales, group):
    """(y, sum of |terms|) in 64 bits; x a bf16 tensor."""
    s = scales.double().numpy().repeat(group, 1)[:, :t.shape[1]]
    w = t * s
    xd = x.double().numpy()
    return xd @ w.T, np.abs(xd) @ np.abs(w).T


# --------------------------------------------------------------------------- cache
class Model:
    """The cache's tables as Python lists, every rule of bitnet.h as a loop."""

    def __init__(self, num_pages, max_seqs, max_pages, page):
        self.P, self.S, self.W, self.page = num_pages, max_seqs, max_pages, page
        self.table = [[-1] * max_pages for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.refs = [0] * num_pages

    def pages(self, n):
        return -(-n // self.page)

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            if s < 0 or d < 0:
                continue
            for j in range(self.pages(self.lens[s])):
                self.table[d][j] = self.table[s][j]
                self.refs[self.table[s][j]] += 1
            self.lens[d] = self.lens[s]

    def extend(self, seqs, add):
        """The pairs to copy, or None if the pages do not suffice."""
        shared = {}
        for i, (s, a) in enumerate(zip(seqs, add)):
            if s >= 0 and a > 0 and self.lens[s] % self.page:
                p = self.table[s][self.pages(self.lens[s]) - 1]
                if self.refs[p] > 1:
                    shared.setdefault(p, []).append(i)
        cow = {i: p for p, holders in shared.items()
               for i in (holders[:-1] if len(holders) == self.refs[p] else holders)}
        need = sum(self.pages(self.lens[s] + a) - self.pages(self.lens[s]) + (i in cow)
                   for i, (s, a) in enumerate(zip(seqs, add)) if s >= 0)
        free = [p for p in range(self.P) if self.refs[p] == 0]
        if need > len(free):
            return None
        pairs = []
        for i, (s, a) in enumerate(zip(seqs, add)):
            if s < 0:
                continue
            had = self.pages(self.lens[s])
            if i in cow:
                p = free.pop(0)
                self.refs[p] = 1
                self.refs[cow[i]] -= 1
                self.table[s][had - 1] = p
                pairs.append((cow[i], p))
            for j in range(had, self.pages(self.lens[s] + a)):
                p = free.pop(0)
                self.refs[p] = 1
                self.table[s][j] = p
            self.lens[s] += a
        return pairs

    def free(self, seqs):
        for s in seqs:
            if s >= 0:
                for j in range(self.pages(self.lens[s])):
                    self.refs[self.table[s][j]] -= 1
                self.lens[s] = 0

    def compact(self):
        used = [p for p in range(self.P) if self.refs[p]]
        moves = list(zip([p for p in used if p >= len(used)],
                         [p for p in range(len(used)) if not self.refs[p]]))
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s in range(self.S):
            for j in range(self.pages(self.lens[s])):
                self.table[s][j] = to.get(self.table[s][j], self.table[s][j])
        return moves

    def check(self, cache):
        """The device's tables equal the model's, where they say anything."""
        assert cache.lens.tolist() == self.lens
        assert cache.refs.tolist() == self.refs
        table = cache.table.tolist()
        for s in range(self.S):
            n = self.pages(self.lens[s])
            assert table[s][:n] == self.table[s][:n], s


def pairs(copies):
    c = copies.tolist()
    assert c[1] == 0
    return list(zip(c[2:2 + 2 * c[0]:2], c[3:3 + 2 * c[0]:2]))


def quantise(x):
    """(q, scale) of bf16 rows in binary32, one scale per row."""
    a = np.maximum(np.abs(x.float().numpy()).max(-1), np.float32(1e-5)).astype(np.float32)
    s = np.float32(127) / a
    return np.rint(x.float().numpy() * s[..., None]).astype(np.int8), s


# --------------------------------------------------------------------------- attention
def attention(q, k, v, scale):
    """One query row set q (heads, D) over k, v (n, kv_heads, D), 64-bit arrays: out, lse, and the
    bounds that binary32 arithmetic implies for them (before out's rounding to bf16)."""
    H, D = q.shape
    n, kv, _ = k.shape
    G = H // kv
    out, lse = np.zeros((H, D)), np.full(H, -np.inf)
    tol_out, tol_lse = np.zeros((H, D)), np.zeros(H)
    if n == 0:
        return out, lse, tol_out, tol_lse
    for h in range(H):
        kk, vv = k[:, h // G], v[:, h // G]
        z = scale * (kk @ q[h])
        w = np.exp(z - z.max())
        p = w / w.sum()
        out[h], lse[h] = p @ vv, z.max() + np.log(w.sum())
        # a score: D products and sums, one step each at worst, relative to the sum of |terms|, its
        # scaling to base 2 and the exponential (2 steps of |z| and 4 more)
        dz = ((D + 4) * abs(scale) * (np.abs(kk) @ np.abs(q[h])).max()
              + 4 * np.abs(z).max() + 4) * F32_STEP
        # sums over n terms, cut up to n / 16 + 32 times on the way, and the join of their parts
        ds = (n / 16 + 64) * F32_STEP
        tol_lse[h] = dz + ds + 4 * F32_STEP * abs(lse[h])
        # weights enter the second product within 2^-16; each error acts on the weighted |v|
        tol_out[h] = (2 * dz + 2 * ds + 2.0 ** -16) * (p @ np.abs(vv)) + 2.0 ** -126
    return out, lse, tol_out, tol_lse
