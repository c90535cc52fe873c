"""Which keys the paged attention's tcgen05 kernel weighs, and how closely.

Two checks that a lost or repeated tile, a lost partial of a split block, a mask off by one row or
a wrong head cannot pass (the last tests plant such mistakes in the 64-bit reference):

* Weights that are powers of two. Queries are unit vectors, keys whole numbers and the scale ln 2,
  so that every probability is a power of two times the row's largest, exact in bf16, and V marks
  keys by the dimension they add to. All terms are positive: what is left is fp32 (the tensor
  cores may drop 2^-22 of a running sum every 16 keys, 2^-13.7 over 5,229 keys, and 2^-20 for the
  exponential and the scale) and the output's rounding, half a step 2^-8 of the value.
* Random values, row by row, in the mean square. A bf16 rounding is off by at most 2^-8 of the
  value, in the mean square over a step by no more than u = 2^-8 / sqrt(3). Independent roundings
  of the probabilities (p_i v_i each), of the query (a score's terms) and of the output add up to
    u^2 (sum_i p_i^2 |v_i|^2 + sum_i p_i^2 |v_i - o|^2 sum_j (scale q_j k_ij)^2 + |o|^2),
  the middle term only for blocks of more than 128 query rows. The v_i of d = 64 or 128 random
  elements are orthogonal to within a tenth, so a row's error passes the first and last term's
  square root by at most sqrt(3), with every rounding at its worst; the bound is twice the root.
"""
import math

import numpy as np
import pytest
import torch

from test_paged import Case, gpu_test, msa, rotate64  # noqa: F401

LN2 = math.log(2.0)


# ------------------------------------------------------------------ powers of two
def exponent(i, h, j, rise):
    """log2 of key i's weight for the unit vector j, KV head h: 0 to -3; with ``rise`` some keys
    above that, within what the running maximum lets pass (8) and beyond it."""
    e = -((7 * i + 3 * j + h) % 4)
    if rise:
        e = np.where(i % 97 == 5, 6, e)
        e = np.where(i % 1501 == 700, 10, e)
    return e


def mark(i, h, d, shift):
    """The dimension of V that key i adds to."""
    return ((i >> shift) + h) % d


def weigh(vis, unit, h, d, shift, rise):
    """O of one KV head: row t with unit vector unit[t] sees keys < vis[t] (0: nothing)."""
    n = int(max(vis.max(initial=0), 0))
    i = np.arange(n)
    w = 2.0 ** exponent(i[None, :], h, unit[:, None], rise)
    w *= i[None, :] < vis[:, None]
    v = np.zeros((n, d))
    v[i, mark(i, h, d, shift)] = 1.0
    o = w @ v
    s = w.sum(1, keepdims=True)
    return np.divide(o, s, out=np.zeros_like(o), where=s > 0)


def off(got, o):
    return np.abs(got - o) > (2.0 ** -8 + 2.0 ** -13) * o


class Marked(Case):
    """A Case whose queries, keys and values are those above; memory rows come first."""

    def __init__(self, gpu, lens, new, page, h_q, h_kv, d, mem, shift, rise):
        super().__init__(gpu, 7, "bf16", lens, new, page, h_q, h_kv, d, mem, base=0.0)
        self.shift, self.rise = shift, rise
        K, V = self.K.cpu(), self.V.cpu()
        table = self.table.cpu().numpy()
        j = np.arange(d)
        for r, L in enumerate(lens):
            m = mem[r] if mem else 0
            i = np.arange(m + L)
            for h in range(h_kv):
                k = exponent(i[:, None], h, j[None, :], rise).astype(np.float32)
                v = np.zeros((m + L, d), np.float32)
                v[i, mark(i, h, d, shift)] = 1.0
                k, v = torch.from_numpy(k), torch.from_numpy(v)
                if m:
                    self.ctx["ctxK"][r, :m, h] = k[:m].bfloat16().to(gpu)
                    self.ctx["ctxV"][r, :m, h] = v[:m].bfloat16().to(gpu)
                for c in range(-(-L // page)):
                    n = min(page, L - c * page)
                    K[table[r, c], :n, h] = k[m + c * page:m + c * page + n].bfloat16()
                    V[table[r, c], :n, h] = v[m + c * page:m + c * page + n].bfloat16()
        self.K, self.V = K.to(gpu), V.to(gpu)
        # token t's query head hq is the unit vector of dimension (5 t + hq) mod d
        t, hq = np.arange(self.total)[:, None], np.arange(h_q)[None, :]
        self.unit = (5 * t + hq) % d
        q = torch.zeros(self.total, h_q, d)
        q[t, hq, self.unit] = 1.0
        self.Q = q.bfloat16().to(gpu)

    def bad(self, O):
        got = O[:self.rows].double().cpu().numpy()
        g, a, out = self.h_q // self.h_kv, 0, []
        for r, (L, T) in enumerate(zip(self.lens, self.new)):
            m = self.mem[r] if self.mem else 0
            vis = m + np.maximum(L - T + np.arange(T) + 1, 0)
            for hq in range(self.h_q):
                o = weigh(vis, self.unit[a:a + T, hq], hq // g, self.d, self.shift, self.rise)
                out += [(r, hq, *x) for x in np.argwhere(off(got[a:a + T, hq], o)).tolist()]
            a += T
        return out


KEYS = {
    # lens, new, page, h_q, h_kv, d, mem: more than eight query rows per KV head each
    "five_tokens": ([90, 1500, 5, 17, 4096], [5] * 5, 32, 32, 8, 128, [8, 16, 0, 24, 129]),
    "long_chunk": ([5000], [700], 64, 8, 2, 128, [100]),
    "long_chunk_d64": ([5000], [700], 16, 8, 2, 64, [128]),
    "one_head_each": ([1200, 31], [300, 31], 16, 5, 5, 128, None),
    "three_heads_each": ([700, 450], [130, 90], 16, 9, 3, 64, [5, 0]),
    "five_heads_each": ([333, 900], [200, 52], 32, 10, 2, 128, [7, 0]),
    "seven_heads_each": ([600], [111], 64, 7, 1, 128, [33]),
    "hundred_heads": ([1500, 40], [5, 2], 16, 200, 2, 64, [0, 9]),
    "prompts": ([130, 257, 64, 1029], [130, 257, 64, 1029], 16, 4, 1, 64, None),
    "halves_alternate": ([900 + 37 * i for i in range(24)], [6 if i % 2 else 45 for i in range(24)],
                         64, 16, 4, 128, [i % 5 * 8 for i in range(24)]),
    "mixed": ([700, 33, 400, 1, 2129], [1, 33, 100, 1, 60], 128, 16, 4, 128, [8, 0, 40, 3, 1]),
    "big_page": ([3000, 300], [100, 300], 1024, 8, 2, 128, None),
    "chunk_longer_than_context": ([100, 0], [300, 40], 16, 8, 2, 128, [9, 0]),
    "256_heads_each": ([400, 70], [3, 1], 16, 256, 1, 128, [5, 0]),
    "129_heads_each": ([400, 70], [3, 1], 16, 258, 2, 64, [0, 130]),
    "85_heads_each": ([400, 700], [7, 30], 32, 85, 1, 128, [5, 0]),
    "1024_kv_heads": ([200, 33], [12, 9], 16, 1024, 1024, 64, [3, 0]),
    "one_token_of_17_heads": ([3000, 129, 1], [1, 1, 1], 16, 34, 2, 128, [64, 0, 0]),
    "long": ([70000], [5], 64, 8, 1, 128, [128]),
    "a_key_past_a_tile": ([129, 257, 128, 256], [3, 65, 3, 65], 16, 16, 4, 128, [129, 128, 0, 1]),
}


@gpu_test
@pytest.mark.parametrize("shift,rise", [(0, False), (0, True), (4, False), (7, True)])
@pytest.mark.parametrize("name", KEYS)
def test_every_key_has_its_weight(msa, gpu, name, shift, rise):
    c = Marked(gpu, *KEYS[name], shift, rise)
    bad = c.bad(c.run(msa, scale=LN2))
    assert not bad, (len(bad), bad[:6])


# ------------------------------------------------------------------ random values
def rounded(q, K, V, vis, scale, two):
    """(o, bound) of one head: rotated q [T, d]; bound on a row's |error| as above."""
    u = 2.0 ** -8 / math.sqrt(3)
    s = q @ K.T * scale
    s[np.arange(K.shape[0])[None, :] >= vis[:, None]] = -np.inf
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    o = p @ V
    oo, vv = (o * o).sum(1), (V * V).sum(1)
    e2 = (p * p) @ vv + oo
    if two:
        away = vv[None, :] - 2 * o @ V.T + oo[:, None]
        e2 += (p * p * away * ((q * q) @ (K * K).T * scale * scale)).sum(1)
    return o, 2 * u * np.sqrt(e2)


CLOSE = {
    # lens, new, page, h_q, h_kv, d, mem
    "one_half": ([3000, 700], [6, 25], 64, 32, 8, 128, [64, 0]),
    "one_half_d64": ([2000, 900], [17, 30], 16, 8, 2, 64, [16, 0]),
    "two_halves": ([3000], [320], 64, 8, 2, 128, [100]),
    "two_halves_d64": ([2000, 1100], [256, 100], 16, 8, 2, 64, None),
}


@gpu_test
@pytest.mark.parametrize("name", CLOSE)
def test_rows_in_the_mean_square(msa, gpu, name):
    lens, new, page, h_q, h_kv, d, mem = CLOSE[name]
    c = Case(gpu, 23, "bf16", lens, new, page, h_q, h_kv, d, mem)
    got = c.run(msa)[:c.rows].double().cpu().numpy()
    g, a = h_q // h_kv, 0
    for r, (L, T) in enumerate(zip(lens, new)):
        m = mem[r] if mem else 0
        local = L - T + np.arange(T)
        q = rotate64(c.q64[a:a + T], c.pos0 + local)
        # blocks of 256 / g tokens; the last may be one half
        tb = 256 // g
        two = np.array([min(tb, T - t // tb * tb) * g > 128 for t in range(T)])
        for h in range(h_q):
            k, v = c.k64[r][:, h // g], c.v64[r][:, h // g]
            if m:
                k = np.concatenate([c.ck64[r, :m, h // g], k])
                v = np.concatenate([c.cv64[r, :m, h // g], v])
            for which in (False, True):
                rows = np.flatnonzero(two == which)
                if not len(rows):
                    continue
                o, bound = rounded(q[rows, h], k, v, m + local[rows] + 1, d ** -0.5, which)
                err = np.linalg.norm(got[a + rows, h] - o, axis=1)
                assert (err <= bound).all(), (r, h, which, (err / bound).max())
        a += T


# ------------------------------------------------------------------ what the checks reject (CPU)
MISTAKES = {
    "a lost tile": lambda vis, i: (i // 128 == 3),
    "the token's own key lost": lambda vis, i: i == vis - 1,
    "one key lost": lambda vis, i: i == 777,
}


@pytest.mark.parametrize("rise", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_powers_of_two_reject_mistakes(d, rise):
    T, L = 40, 5000
    vis = L - T + np.arange(T) + 1
    unit = (5 * np.arange(T)) % d
    shifts = (0, 4, 7)
    right = [weigh(vis, unit, 1, d, s, rise) for s in shifts]
    assert not any(off(o * (1 + 2.0 ** -8), o).any() for o in right)  # a rounding passes
    i = np.arange(L)
    for what, lost in MISTAKES.items():
        w = 2.0 ** exponent(i[None, :], 1, unit[:, None], rise) * (i[None, :] < vis[:, None])
        w *= ~lost(vis[:, None], i[None, :])
        seen = []
        for s, o in zip(shifts, right):
            v = np.zeros((L, d))
            v[i, mark(i, 1, d, s)] = 1.0
            seen.append(off(w @ v / w.sum(1, keepdims=True), o).any())
        assert any(seen), what
    # a future key, another head's keys, a tile of other keys
    assert any(off(weigh(vis + 1, unit, 1, d, s, rise), o).any() for s, o in zip(shifts, right))
    assert any(off(weigh(vis, unit, 2, d, s, rise), o).any() for s, o in zip(shifts, right))
    assert any(off(weigh(vis, (unit + 1) % d, 1, d, s, rise), o).any()
               for s, o in zip(shifts, right))
    w = 2.0 ** exponent(i[None, :], 1, unit[:, None], rise) * (i[None, :] < vis[:, None])
    swapped = np.where(i // 128 == 3, i + 128, i)  # tile 4 read twice, tile 3 not
    seen = []
    for s, o in zip(shifts, right):
        v = np.zeros((L, d))
        v[i, mark(swapped, 1, d, s)] = 1.0
        seen.append(off(w @ v / w.sum(1, keepdims=True), o).any())
    assert any(seen)


@pytest.mark.parametrize("two", [False, True])
def test_mean_square_rejects_mistakes(two):
    rs = np.random.RandomState(0)
    T, L, d = 64, 3000, 128
    q, K, V = rs.standard_normal((T, d)), rs.standard_normal((L, d)), rs.standard_normal((L, d))
    vis = L - T + np.arange(T) + 1
    o, bound = rounded(q, K, V, vis, d ** -0.5, two)
    rejects = lambda x: (np.linalg.norm(x - o, axis=1) > bound).any()
    # the documented roundings pass
    bf = lambda x: torch.from_numpy(np.ascontiguousarray(x)).bfloat16().double().numpy()
    s = (bf(q) if two else q) @ K.T * d ** -0.5
    s[np.arange(L)[None, :] >= vis[:, None]] = -np.inf
    p = np.exp(s - s.max(1, keepdims=True))
    assert not rejects(bf(bf(p) @ V / p.sum(1, keepdims=True)))
    i = np.arange(L)
    s = q @ K.T * d ** -0.5
    for what, lost in MISTAKES.items():
        x = np.where((i[None, :] >= vis[:, None]) | lost(vis[:, None], i[None, :]), -np.inf, s)
        p = np.exp(x - x.max(1, keepdims=True))
        assert rejects(p @ V / p.sum(1, keepdims=True)), what
    ahead, _ = rounded(q, K, V, vis + 1, d ** -0.5, two)
    assert rejects(ahead)
    assert rejects(np.zeros_like(o)) and rejects(o * 1.01)
