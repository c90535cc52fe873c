"""The paged local context (page_plan, paged_append, paged_attend) against plain 64-bit forms.

Tolerances follow from the roundings, element by element. bf16 (half a step 2^-8): the rotated
query may be rounded, so a score moves by at most 2^-8 scale sum|q k| = ds and a probability by a
factor within exp(2 ds); the probabilities may be rounded (2^-8) and the output is (2^-8 |o|).
Where both enter the products with their low parts (eight query rows per KV head or fewer),
test_decode_keeps_the_low_parts holds them to 2^-16 instead.
fp32: products of tf32 high and low parts leave out 2^-22 of each product (the low parts'
rounding twice, and low x low), the tensor core's accumulation may drop 2^-22 of the running sum a
step; the score, the probabilities' exponential (2^-22) and the product with V err accordingly.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

gpu_test = pytest.mark.gpu
BASE = 1e6


@pytest.fixture(scope="module")
def msa():
    import long_context_doc_b200 as m
    return m


# ------------------------------------------------------------------ plain 64-bit forms
def rotate64(x, pos, base=BASE):
    """x [n, heads, d], positions [n]; base <= 0: as given."""
    if base <= 0:
        return x.copy()
    d = x.shape[-1]
    ang = np.asarray(pos, np.float64)[:, None] * base ** (-np.arange(0, d, 2) / d)
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
    a, b = x[..., :d // 2], x[..., d // 2:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def plan64(target, length, table, free, n_free, page, max_rows):
    """The stack as a list, request by request."""
    table, stack, free = table.copy(), list(free[:n_free]), free.copy()
    held = lambda x: -(-x // page)
    for r, (o, t) in enumerate(zip(length, target)):
        stack += list(table[r, held(t):held(o)])
    slot, pos, start = [], [], [0]
    for r, (o, t) in enumerate(zip(length, target)):
        for c in range(held(o), held(t)):
            table[r, c] = stack.pop()
        for p in range(o, t):
            slot.append(table[r, p // page] * page + p % page)
            pos.append(p)
        start.append(len(slot))
    free[n_free:len(stack)] = stack[n_free:]
    pad = [-1] * (max_rows - len(slot))
    return dict(length=list(target), n_free=[len(stack)], row_start=start, slot_map=slot + pad,
                row_pos=pos + pad), table, free


def attend64(q, K, V, vis, scale, dtype):
    """One head: rotated q [T, d], keys K, V [n, d]; token t sees keys < vis[t]. Returns
    (o, tol)."""
    T, d = q.shape
    o, tol = np.zeros((T, d)), np.zeros((T, d))
    if K.shape[0] == 0:
        return o, tol
    if dtype == "bf16":
        u_s, u_p, u_o = 2.0 ** -8 + 2.0 ** -20, 2.0 ** -8 + 2.0 ** -20, 2.0 ** -8
    else:
        u_s = (3 + 3 * d / 8 + 4) * 2.0 ** -22
        u_p = (4 + 3 * K.shape[0] / 8 + 8) * 2.0 ** -22
        u_o = 2.0 ** -23
    s = q @ K.T * scale
    mag = np.abs(q) @ np.abs(K).T * abs(scale)
    for t in range(T):
        n = vis[t]
        if n <= 0:
            continue
        p = np.exp(s[t, :n] - s[t, :n].max())
        p /= p.sum()
        o[t] = p @ V[:n]
        spread = p @ np.abs(V[:n])
        ds = u_s * mag[t, :n].max()
        tol[t] = (math.expm1(2 * ds) + 2 * u_p) * spread + u_o * np.abs(o[t])
    return o, tol


TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


class Case:
    """A pool with held pages scattered over it, every row nobody holds NaN, the table's unused
    entries out of range, and the dense K/V of each request beside it."""

    def __init__(self, gpu, seed, dtype, lens, new, page, h_q, h_kv, d, mem=None, pos0=3, base=BASE,
                 spare=2, width_extra=2, pad=3, q_extra=0):
        rs = np.random.RandomState(seed)
        self.dtype, self.tt = dtype, TYPES[dtype]
        self.lens, self.new, self.page = lens, new, page
        self.h_q, self.h_kv, self.d, self.pos0, self.base = h_q, h_kv, d, pos0, base
        n = len(lens)
        held = [-(-x // page) for x in lens]
        n_pages = sum(held) + spare
        perm = rs.permutation(n_pages)
        width = max(held + [1]) + width_extra
        table = np.full((n, width), 1 << 30, np.int64)
        at = 0
        for r, h in enumerate(held):
            table[r, :h] = perm[at:at + h]
            at += h

        def rnd(*shape):
            return torch.from_numpy(rs.standard_normal(shape).astype(np.float32)).to(self.tt)
        self.table = torch.from_numpy(table.astype(np.int32)).to(gpu)
        K = torch.full((n_pages, page, h_kv, d), float("nan"), dtype=self.tt)
        V = K.clone()
        self.k64, self.v64 = [], []
        for r, L in enumerate(lens):
            k, v = rnd(L, h_kv, d), rnd(L, h_kv, d)
            for c in range(held[r]):
                m = min(page, L - c * page)
                K[table[r, c], :m] = k[c * page:c * page + m]
                V[table[r, c], :m] = v[c * page:c * page + m]
            self.k64.append(k.double().numpy())
            self.v64.append(v.double().numpy())
        self.K, self.V = K.to(gpu), V.to(gpu)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows, self.total = int(start[-1]), int(start[-1]) + pad
        self.row_start = torch.from_numpy(start).to(gpu)
        self.length = torch.tensor(lens, dtype=torch.int32, device=gpu)
        q = rnd(self.total, h_q, d)
        q[self.rows:] = float("nan")
        self.q64 = q.double().numpy()
        wide = torch.full((self.total, h_q * d + q_extra), float("nan"), dtype=self.tt)
        wide[:, :h_q * d] = q.reshape(self.total, h_q * d)
        self.Q = wide.to(gpu)[:, :h_q * d].unflatten(1, (h_q, d))
        self.mem = mem
        self.ctx = dict(ctxK=None, ctxV=None, ctx_len=None)
        if mem is not None:
            w = max(mem + [1]) + 1
            ck, cv = rnd(n, w, h_kv, d), rnd(n, w, h_kv, d)
            for r, m in enumerate(mem):
                ck[r, m:] = float("nan")
                cv[r, m:] = float("nan")
            self.ck64, self.cv64 = ck.double().numpy(), cv.double().numpy()
            self.ctx = dict(ctxK=ck.to(gpu), ctxV=cv.to(gpu),
                            ctx_len=torch.tensor(mem, dtype=torch.int32, device=gpu))

    def reference(self, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        g = self.h_q // self.h_kv
        o = np.zeros((self.rows, self.h_q, self.d))
        tol = np.zeros_like(o)
        a = 0
        for r, (L, T) in enumerate(zip(self.lens, self.new)):
            m = 0 if self.mem is None else self.mem[r]
            local = L - T + np.arange(T)
            q = rotate64(self.q64[a:a + T], self.pos0 + local, self.base)
            for h in range(self.h_q):
                k, v = self.k64[r][:, h // g], self.v64[r][:, h // g]
                if m:
                    k = np.concatenate([self.ck64[r, :m, h // g], k])
                    v = np.concatenate([self.cv64[r, :m, h // g], v])
                vis = m + np.maximum(local + 1, 0)
                o[a:a + T, h], tol[a:a + T, h] = attend64(q[:, h], k, v, vis, scale, self.dtype)
            a += T
        return o, tol

    def workspace(self, msa, fill=0xFF):
        ck = self.ctx["ctxK"]
        n = msa.msa_paged_attend_workspace(self.total, len(self.lens), self.h_q, self.h_kv, self.d,
                                           msa.dtype_code(self.Q), 0 if ck is None else
                                           ck.shape[1], self.table.shape[1], self.page)
        return torch.full((n,), fill, dtype=torch.uint8, device=self.Q.device)

    def run(self, msa, **kw):
        return msa.paged_attend(self.Q, self.row_start, self.length, self.K, self.V, self.table,
                                self.pos0, self.base, **self.ctx, **kw)

    def check(self, O, scale=None):
        o, tol = self.reference(scale)
        got = O[:self.rows].double().cpu().numpy()
        assert np.isfinite(got).all()
        bad = np.abs(got - o) > tol
        assert not bad.any(), (bad.sum(), np.abs(got - o).max(), np.argwhere(bad)[:4].tolist())


# ------------------------------------------------------------------ refusals (CPU)
def _plan_call(msa, n_req=2, page=16, width=4, n_pages=8, rows=5, ws=512, ws_bytes=256, null=()):
    f = {k: (None if k in null else ctypes.c_void_p(1024)) for k in
         ("target", "len", "nfree", "table", "free", "len_out", "nfree_out", "start", "slot",
          "pos")}
    return msa.lib.msa_page_plan(f["target"], f["len"], f["nfree"], n_req, page, width, n_pages,
                                 rows, f["table"], f["free"], f["len_out"], f["nfree_out"],
                                 f["start"], f["slot"], f["pos"],
                                 ctypes.c_void_p(ws) if ws else None, ws_bytes, None)


def test_plan_refuses_on_the_host(msa):
    for page in (0, 8, 24, 48, -16, 1 << 21):
        assert _plan_call(msa, page=page) == 2, page
    assert _plan_call(msa, n_req=4097) == 2
    assert _plan_call(msa, n_req=-1) == 1
    assert _plan_call(msa, n_pages=0) == 1
    assert _plan_call(msa, n_pages=1 << 27) == 1     # 2^31 rows
    assert _plan_call(msa, width=1 << 27) == 1
    assert _plan_call(msa, rows=-1) == 1
    assert _plan_call(msa, ws=None) == 3
    assert _plan_call(msa, ws=520) == 3
    assert _plan_call(msa, ws_bytes=255) == 3
    need = msa.msa_page_plan_workspace(2, 5000)
    assert need > 256 and _plan_call(msa, rows=5000, ws_bytes=need - 1) == 3
    for name in ("target", "len", "nfree", "table", "free", "len_out", "nfree_out", "start",
                 "slot", "pos"):
        assert _plan_call(msa, null=(name,)) == 1, name


def _append_call(msa, n_pages=8, page=16, rows=3, h_kv=2, d=64, dtype=1, pos0=0, stride=None,
                 ptr=1024, ws=512, ws_bytes=256, maps=1024):
    f = ctypes.c_void_p(ptr) if ptr else None
    m = ctypes.c_void_p(maps) if maps else None
    stride = h_kv * d if stride is None else stride
    return msa.lib.msa_paged_append(f, f, n_pages, page, m, m, f, f, stride, stride, rows, h_kv, d,
                                    dtype, pos0, 0.0, ctypes.c_void_p(ws) if ws else None,
                                    ws_bytes, None)


def test_append_refuses_on_the_host(msa):
    assert _append_call(msa, dtype=2) == 2
    assert _append_call(msa, d=96) == 2
    assert _append_call(msa, h_kv=0) == 1
    assert _append_call(msa, h_kv=1025) == 2
    assert _append_call(msa, page=12) == 2
    assert _append_call(msa, n_pages=0) == 1
    assert _append_call(msa, rows=-1) == 1
    assert _append_call(msa, pos0=-1) == 1
    assert _append_call(msa, stride=127) == 1        # shorter than a row
    assert _append_call(msa, stride=132) == 1        # not a multiple of 16 bytes
    assert _append_call(msa, dtype=0, stride=130) == 1
    assert _append_call(msa, ptr=1032) == 1
    assert _append_call(msa, ptr=None) == 1
    assert _append_call(msa, maps=None) == 1
    assert _append_call(msa, ws=None) == 3
    assert _append_call(msa, ws_bytes=128) == 3
    assert _append_call(msa, rows=0, ptr=None, maps=None) == 0  # nothing to write


def _attend_call(msa, rows=4, h_q=8, h_kv=2, d=64, dtype=1, n_req=2, n_pages=8, page=16, width=4,
                 max_ctx=5, pos0=0, scale=0.0, q_stride=None, ptr=1024, ctx=1024, ws=512,
                 ws_short=0):
    f = ctypes.c_void_p(ptr) if ptr else None
    c = ctypes.c_void_p(ctx) if ctx else None
    need = msa.msa_paged_attend_workspace(max(rows, 1), max(n_req, 1), 8, 2, 64, 1, 5, 4, 16)
    return msa.lib.msa_paged_attend(f, h_q * d if q_stride is None else q_stride, rows, h_q, f, f,
                                    n_req, f, f, n_pages, page, f, width, c, c, c, max_ctx, h_kv,
                                    d, dtype, pos0, 0.0, scale, f,
                                    ctypes.c_void_p(ws) if ws else None, need - ws_short, None)


def test_attend_refuses_on_the_host(msa):
    assert _attend_call(msa, dtype=3) == 2
    assert _attend_call(msa, d=32) == 2
    assert _attend_call(msa, h_kv=0) == 1
    assert _attend_call(msa, h_q=7) == 1
    assert _attend_call(msa, h_q=1) == 1
    assert _attend_call(msa, page=17) == 2
    assert _attend_call(msa, n_pages=1 << 27) == 1
    assert _attend_call(msa, width=0) == 1
    assert _attend_call(msa, n_req=4097) == 2
    assert _attend_call(msa, rows=-1) == 1
    assert _attend_call(msa, rows=1 << 29) == 1      # n_rows * h_q past 2^31
    assert _attend_call(msa, max_ctx=-1) == 1
    assert _attend_call(msa, pos0=-2) == 1
    assert _attend_call(msa, scale=float("nan")) == 1
    assert _attend_call(msa, scale=float("inf")) == 1
    assert _attend_call(msa, q_stride=508) == 1
    assert _attend_call(msa, q_stride=513) == 1
    assert _attend_call(msa, ptr=None) == 1
    assert _attend_call(msa, ptr=1032) == 1
    assert _attend_call(msa, ctx=None) == 1          # memory rows without a memory
    assert _attend_call(msa, ctx=1032) == 1
    assert _attend_call(msa, ws=None) == 3
    assert _attend_call(msa, ws=528) == 3
    assert _attend_call(msa, ws_short=1) == 3


def test_helpers_refuse_what_pointers_cannot_show(msa):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    pool = torch.zeros(4, 16, 2, 64)
    with pytest.raises(msa.MSAError, match="target is torch.int64"):
        msa.page_plan(torch.zeros(2, dtype=torch.int64), i32(2), i32(1), i32(2, 3), i32(4), 16, 8)
    with pytest.raises(msa.MSAError, match="target has 3"):
        msa.page_plan(i32(3), i32(2), i32(1), i32(2, 3), i32(4), 16, 8)
    with pytest.raises(msa.MSAError, match="not contiguous"):
        msa.page_plan(i32(4)[::2], i32(2), i32(1), i32(2, 3), i32(4), 16, 8)
    with pytest.raises(msa.MSAError, match="V_new is"):
        msa.paged_append(pool, pool, i32(3), i32(3), torch.zeros(3, 2, 64),
                         torch.zeros(2, 2, 64), 0, 0.0)
    with pytest.raises(msa.MSAError, match="K_new is torch.bfloat16"):
        msa.paged_append(pool, pool, i32(3), i32(3), torch.zeros(3, 2, 64, dtype=torch.bfloat16),
                         torch.zeros(3, 2, 64), 0, 0.0)
    with pytest.raises(msa.MSAError, match="not dense"):
        msa.paged_append(pool, pool, i32(3), i32(3), torch.zeros(3, 64, 2).transpose(1, 2),
                         torch.zeros(3, 2, 64), 0, 0.0)
    with pytest.raises(msa.MSAError, match="cover 2 of 3"):
        msa.paged_append(pool, pool, i32(2), i32(3), torch.zeros(3, 2, 64),
                         torch.zeros(3, 2, 64), 0, 0.0)
    Q = torch.zeros(5, 4, 64)
    with pytest.raises(msa.MSAError, match="row_start has 2"):
        msa.paged_attend(Q, i32(2), i32(2), pool, pool, i32(2, 3), 0, 0.0)
    with pytest.raises(msa.MSAError, match="the memory is"):
        msa.paged_attend(Q, i32(3), i32(2), pool, pool, i32(2, 3), 0, 0.0,
                         ctxK=torch.zeros(2, 5, 2, 64))
    with pytest.raises(msa.MSAError, match="Q is"):
        msa.paged_attend(torch.zeros(5, 4, 128), i32(3), i32(2), pool, pool, i32(2, 3), 0, 0.0)
    with pytest.raises(msa.MSAError, match="O is not like Q"):
        msa.paged_attend(Q, i32(3), i32(2), pool, pool, i32(2, 3), 0, 0.0, O=torch.zeros(4, 4, 64))
    # nothing wrong but where they are
    with pytest.raises(msa.MSAError, match="device memory"):
        msa.page_plan(i32(2), i32(2), i32(1), i32(2, 3), i32(4), 16, 8)
    with pytest.raises(msa.MSAError, match="device memory"):
        msa.paged_append(pool, pool, i32(3), i32(3), torch.zeros(3, 2, 64),
                         torch.zeros(3, 2, 64), 0, 0.0)
    with pytest.raises(msa.MSAError, match="device memory"):
        msa.paged_attend(Q, i32(3), i32(2), pool, pool, i32(2, 3), 0, 0.0)


# ------------------------------------------------------------------ plan
def _i32(x, gpu):
    return torch.tensor(x, dtype=torch.int32, device=gpu)


def _plan_state(rs, lens, page, width, n_pages):
    held = [-(-x // page) for x in lens]
    perm = rs.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), width), -9, np.int32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = perm[at:at + h]
        at += h
    free = np.full(n_pages, -7, np.int32)
    free[:n_pages - at] = perm[at:]
    return table, free, n_pages - at


def _run_plan(msa, gpu, target, lens, table, free, n_free, page, max_rows, alias):
    t, f = torch.from_numpy(table.copy()).to(gpu), torch.from_numpy(free.copy()).to(gpu)
    length, nf = _i32(lens, gpu), _i32([n_free], gpu)
    out = msa.page_plan_buffers(len(lens), max_rows, gpu)
    for v in out.values():
        v.fill_(-5)
    if alias:
        out["length"], out["n_free"] = length, nf
    ws = torch.full((msa.msa_page_plan_workspace(len(lens), max_rows),), 0x5A, dtype=torch.uint8,
                    device=gpu)
    msa.page_plan(_i32(target, gpu), length, nf, t, f, page, max_rows, out=out, ws=ws)
    got = {k: v.cpu().tolist() for k, v in out.items()}
    return got, t.cpu().numpy(), f.cpu().numpy(), msa.msa_workspace_status(ws)


PLANS = {
    "one_token": ([37], [38], 16, 64),
    "new_page": ([32], [33], 16, 1),
    "first_token": ([0], [1], 16, 3),
    "nothing": ([5, 0, 16], [5, 0, 16], 16, 7),
    "ends_and_begins": ([100, 0, 33, 16, 1], [0, 77, 33, 48, 2], 16, 200),
    "shrinks_only": ([100, 50, 64], [3, 0, 33], 32, 10),
    "rows_fill_the_map": ([0, 0, 0], [17, 0, 15], 16, 32),
    "more_back_than_needed": ([200, 3, 90], [10, 70, 0], 16, 80),
    "more_needed_than_back": ([20, 3, 90], [0, 200, 120], 16, 300),
    "cut_inside_a_page": ([40, 40], [33, 45], 32, 9),
    "no_requests": ([], [], 16, 5),
    "no_rows": ([3], [0], 16, 0),
}


@gpu_test
@pytest.mark.parametrize("alias", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("name", PLANS)
def test_plan_small(msa, gpu, name, alias):
    lens, target, page, max_rows = PLANS[name]
    width = max([1] + [-(-x // page) for x in lens + target]) + 1
    table, free, n_free = _plan_state(np.random.RandomState(1), lens, page, width, 40)
    ref, rt, rf = plan64(target, lens, table, free, n_free, page, max_rows)
    got, t, f, status = _run_plan(msa, gpu, target, lens, table, free, n_free, page, max_rows,
                                  alias)
    assert status == 0 and got == ref
    np.testing.assert_array_equal(t, rt)
    np.testing.assert_array_equal(f, rf)


@gpu_test
@pytest.mark.parametrize("n,page,hi,new,max_rows", [
    (300, 64, 3000, 1, 300), (1025, 16, 70, 40, 40000), (4096, 16, 40, 3, 8195),
    (37, 128, 9000, 3000, 70001), (2500, 32, 400, 1, 4096)])
@pytest.mark.parametrize("alias", [False, True], ids=["apart", "in_place"])
def test_plan_large(msa, gpu, n, page, hi, new, max_rows, alias):
    rs = np.random.RandomState(n)
    lens = rs.randint(0, hi, n).tolist()
    kind = rs.rand(n)
    target = [0 if k < 0.2 else int(rs.randint(0, x + 1)) if k < 0.3 else x + int(rs.randint(0, new + 1))
              for x, k in zip(lens, kind)]
    budget = max_rows
    for r in range(n):  # the map holds every new row
        target[r] = min(target[r], lens[r] + budget)
        budget -= max(0, target[r] - lens[r])
    width = max(-(-x // page) for x in lens + target) + 1
    need = sum(-(-x // page) for x in lens) + sum(-(-x // page) for x in target)
    table, free, n_free = _plan_state(rs, lens, page, width, need + 1)
    ref, rt, rf = plan64(target, lens, table, free, n_free, page, max_rows)
    got, t, f, status = _run_plan(msa, gpu, target, lens, table, free, n_free, page, max_rows,
                                  alias)
    assert status == 0
    for k in ref:
        assert got[k] == ref[k], k
    np.testing.assert_array_equal(t, rt)
    np.testing.assert_array_equal(f, rf)


@gpu_test
@pytest.mark.parametrize("what,code", [("pages", 2), ("rows", 2), ("negative", 3), ("long", 3),
                                       ("count", 3), ("held_too_much", 3)])
@pytest.mark.parametrize("max_rows", [30, 9000], ids=["one_cta", "cluster"])
@pytest.mark.parametrize("alias", [False, True], ids=["apart", "in_place"])
def test_plan_refuses_on_the_device(msa, gpu, what, code, max_rows, alias):
    lens, target = [20, 5, 30], [25, 0, 31]
    table, free, n_free = _plan_state(np.random.RandomState(2), lens, 16, 600, 9)
    if what == "pages":
        target = [20, 5, 30 + 16 * 7]
        max_rows = max(max_rows, 200)
    elif what == "rows":
        lens, target = [0, 0, 0], [0, max_rows + 1, 0]
        table, free, n_free = _plan_state(np.random.RandomState(2), lens, 16, 600, 600)
    elif what == "negative":
        target = [25, -1, 31]
    elif what == "long":
        target = [25, 0, 600 * 16 + 1]
    elif what == "count":
        n_free = 10
    elif what == "held_too_much":  # more returned than the pool can hold free
        n_free, target = 9, [0, 0, 0]
    got, t, f, status = _run_plan(msa, gpu, target, lens, table, free, n_free, 16, max_rows, alias)
    assert status == code
    assert got == dict(length=lens, n_free=[n_free], row_start=[0] * 4, slot_map=[-1] * max_rows,
                       row_pos=[-1] * max_rows)
    np.testing.assert_array_equal(t, table)
    np.testing.assert_array_equal(f, free)


@gpu_test
def test_plan_bad_page_ids(msa, gpu):
    """A page id outside the pool, in the table or on the stack: its rows get slot -1, the others
    their slots, and the status says so."""
    lens, target = [3, 3, 16], [5, 17, 18]
    table, free, n_free = _plan_state(np.random.RandomState(3), lens, 16, 4, 8)
    table[0, 0] = 8
    free[n_free - 2] = -4  # the second page popped: request 2's second page
    ref, rt, rf = plan64(target, lens, table, free, n_free, 16, 20)
    got, t, f, status = _run_plan(msa, gpu, target, lens, table, free, n_free, 16, 20, False)
    assert status == 3
    want = [-1 if i < 2 or i >= 16 else s for i, s in enumerate(ref["slot_map"])]
    assert got["slot_map"] == want and got["row_pos"] == ref["row_pos"]
    np.testing.assert_array_equal(t, rt)


# ------------------------------------------------------------------ append
@gpu_test
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h_kv,rows,page,base,extra", [
    (8, 1, 16, BASE, 0), (2, 37, 64, BASE, 64), (1, 129, 16, 0.0, 0), (3, 1000, 32, 1e4, 8),
    (5, 7000, 128, BASE, 0)])
def test_append(msa, gpu, dtype, d, h_kv, rows, page, base, extra):
    rs = np.random.RandomState(rows + d)
    n_pages = -(-rows // page) + 3
    pos0 = 16
    slots = rs.permutation(n_pages * page)[:rows].astype(np.int32)
    pos = rs.randint(0, 1 << 20, rows).astype(np.int32)
    skip = rs.rand(rows) < 0.1
    slots[skip] = -1
    tt = TYPES[dtype]
    K = torch.randn(n_pages, page, h_kv, d).to(tt)
    V = torch.randn(n_pages, page, h_kv, d).to(tt)
    new = torch.randn(rows, 2 * h_kv * d + extra).to(tt)
    k_new = new[:, :h_kv * d].unflatten(1, (h_kv, d))
    v_new = new[:, h_kv * d:2 * h_kv * d].unflatten(1, (h_kv, d))
    ref_k, ref_v = K.double().numpy().copy(), V.double().numpy().copy()
    rot = rotate64(k_new.double().numpy(), pos.astype(np.int64) + pos0, base)
    keep = ~skip
    ref_k.reshape(-1, h_kv, d)[slots[keep]] = rot[keep]
    ref_v.reshape(-1, h_kv, d)[slots[keep]] = v_new.double().numpy()[keep]
    Kd, Vd, nd = K.to(gpu), V.to(gpu), new.to(gpu)
    ws = msa.paged_append(Kd, Vd, torch.from_numpy(slots).to(gpu), torch.from_numpy(pos).to(gpu),
                          nd[:, :h_kv * d].unflatten(1, (h_kv, d)),
                          nd[:, h_kv * d:2 * h_kv * d].unflatten(1, (h_kv, d)), pos0, base)
    assert msa.msa_workspace_status(ws) == 0
    # V and the rows not named: bit for bit. K: half a step of the type, and the rotation's
    # error: the angle is off by less than 2^-24 half turns (2e-7 rad) and sin, cos, the two
    # products and their sum by 2^-22 of the pair's size
    np.testing.assert_array_equal(Vd.double().cpu().numpy(), ref_v)
    got = Kd.double().cpu().numpy().reshape(-1, h_kv, d)
    want = ref_k.reshape(-1, h_kv, d)
    half = torch.finfo(tt).eps / 2
    pair = np.abs(want) + np.abs(np.roll(want, d // 2, axis=-1))
    touched = np.zeros(n_pages * page, bool)
    touched[slots[keep]] = True
    np.testing.assert_array_equal(got[~touched], want[~touched])
    tol = half * np.abs(want) + (half * 2.0 ** -10 + 2.0 ** -22 + 4e-7) * pair if base > 0 else 0.0 * pair
    assert (np.abs(got - want) <= tol)[touched].all(), np.abs(got - want)[touched].max()


@gpu_test
def test_append_past_the_pool(msa, gpu):
    """A slot past the pool is skipped and recorded; the status is kept until a plan starts it."""
    K = torch.zeros(2, 16, 2, 64, device=gpu)
    V = torch.zeros_like(K)
    new = torch.ones(3, 2, 64, device=gpu)
    ws = torch.zeros(256, dtype=torch.uint8, device=gpu)
    msa.paged_append(K, V, _i32([5, 32, 31], gpu), _i32([0, 1, 2], gpu), new, new, 0, 0.0, ws=ws)
    assert msa.msa_workspace_status(ws) == 3
    msa.paged_append(K, V, _i32([5], gpu), _i32([0], gpu), new[:1], new[:1], 0, 0.0, ws=ws)
    assert msa.msa_workspace_status(ws) == 3
    rows = V.sum((2, 3)).flatten().nonzero().flatten().tolist()
    assert rows == [5, 31]
    table, free, nf = _plan_state(np.random.RandomState(0), [0], 16, 2, 2)
    msa.page_plan(_i32([4], gpu), _i32([0], gpu), _i32([nf], gpu),
                  torch.from_numpy(table).to(gpu), torch.from_numpy(free).to(gpu), 16, 8, ws=ws)
    assert msa.msa_workspace_status(ws) == 0


# ------------------------------------------------------------------ attend
ATTEND = {
    # lens, new, page, h_q, h_kv, d, mem
    "one_token_one_row": ([1], [1], 16, 4, 1, 128, None),
    "one_token": ([77], [1], 16, 32, 8, 128, [9]),
    "one_token_long": ([5000], [1], 64, 8, 2, 128, [128]),
    "ragged_tokens": ([1, 15, 16, 17, 300, 2047, 64, 33], [1] * 8, 16, 8, 2, 64, None),
    "page_ends_in_tile": ([130, 127, 129, 255], [1, 3, 2, 1], 32, 16, 4, 128, [16, 17, 0, 1]),
    "no_new_tokens": ([40, 25, 3], [0, 2, 0], 16, 4, 2, 64, [0, 3, 7]),
    "nothing_at_all": ([0, 0], [0, 0], 16, 4, 2, 64, [2, 0]),
    "sees_nothing": ([0, 2], [3, 5], 16, 4, 2, 128, None),
    "memory_only": ([0, 2], [3, 5], 16, 4, 2, 128, [33, 1]),
    "five_tokens": ([90, 500, 5, 17], [5, 5, 5, 5], 32, 32, 8, 128, [8, 16, 0, 24]),
    "three_heads_each": ([70, 45], [7, 1], 16, 9, 3, 64, [5, 0]),
    "one_head_each": ([200, 31], [40, 31], 16, 5, 5, 128, None),
    "sixteen_heads_each": ([129, 64], [3, 1], 64, 32, 2, 128, [40, 0]),
    "forty_heads_each": ([129, 64], [3, 1], 64, 40, 1, 64, [0, 40]),
    "chunk": ([300], [150], 64, 8, 2, 128, [20]),
    "prompts": ([130, 1, 257, 64], [130, 1, 257, 64], 16, 4, 1, 64, None),
    "mixed": ([700, 33, 400, 1, 129], [1, 33, 100, 1, 60], 32, 16, 4, 128, [8, 0, 40, 3, 1]),
    "big_page": ([1000, 5], [1, 2], 1024, 4, 2, 128, None),
    # blocks of one half and of two follow one another within a CTA's share
    "halves_alternate": ([900 + 37 * i for i in range(24)], [6 if i % 2 else 45 for i in range(24)],
                         64, 32, 8, 128, [i % 5 * 8 for i in range(24)]),
    "halves_alternate_d64": ([700 + 61 * i for i in range(20)],
                             [(3, 70, 5, 40)[i % 4] for i in range(20)], 16, 32, 4, 64, None),
    "five_heads_chunk": ([333, 12], [200, 12], 32, 10, 2, 128, [7, 0]),
    "hundred_heads": ([150, 40], [5, 1], 16, 200, 2, 64, [0, 9]),
    "past_a_block_of_heads": ([70, 33], [2, 1], 16, 300, 1, 64, [3, 0]),
    "sixteen_heads_decode": ([700, 90, 1], [1, 1, 1], 16, 32, 2, 128, [5, 0, 0]),
    "long_chunk": ([5000], [700], 64, 8, 2, 128, [100]),
    "chunk_longer_than_context": ([100, 0], [300, 40], 16, 8, 2, 128, [9, 0]),
    "many_kv_heads": ([40, 9], [2, 1], 16, 24, 12, 64, [3, 0]),
}


@gpu_test
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", ATTEND)
def test_attend(msa, gpu, name, dtype):
    lens, new, page, h_q, h_kv, d, mem = ATTEND[name]
    c = Case(gpu, 11, dtype, lens, new, page, h_q, h_kv, d, mem)
    ws = c.workspace(msa)
    O = torch.full((c.total, h_q, d), 7.0, dtype=c.tt, device=gpu)
    c.run(msa, O=O, ws=ws)
    assert msa.msa_workspace_status(ws) == 0
    c.check(O)
    assert (O[c.rows:] == 7.0).all()  # rows behind the last request


@gpu_test
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kw", [dict(base=0.0), dict(pos0=0), dict(pos0=1 << 20), dict(q_extra=64),
                                dict(scale=0.5), dict(pad=0)],
                         ids=["no_rope", "pos0_0", "far_positions", "strided_q", "scale", "no_pad"])
def test_attend_arguments(msa, gpu, dtype, kw):
    kw = dict(kw)
    scale = kw.pop("scale", None)
    c = Case(gpu, 5, dtype, [100, 37, 260], [1, 9, 40], 16, 8, 2, 128, [4, 0, 30], **kw)
    c.check(c.run(msa, scale=scale or 0.0), scale)


@gpu_test
@pytest.mark.parametrize("n", [200, 1000, 4096])
def test_attend_many_requests(msa, gpu, n):
    rs = np.random.RandomState(n)
    lens = rs.randint(0, 60, n).tolist()
    new = [min(x, int(rs.randint(0, 3))) for x in lens]
    c = Case(gpu, n, "bf16", lens, new, 16, 4, 2, 64, rs.randint(0, 5, n).tolist())
    c.check(c.run(msa))


@gpu_test
def test_attend_equal_and_extreme_scores(msa, gpu):
    """Equal keys give the mean of V; one key far above the others gives its V."""
    for T in (1, 40):
        c = Case(gpu, 8, "bf16", [90], [T], 16, 4, 1, 128, None, base=0.0)
        c.K.copy_(torch.where(torch.isnan(c.K), c.K, torch.zeros_like(c.K)))
        c.k64 = [np.zeros_like(c.k64[0])]
        c.check(c.run(msa))
        page, row = int(c.table[0, 1]), 3                   # local row 19
        c.K[page, row] = 100.0 * torch.sign(c.Q[0, 0])
        c.k64[0][19] = 100.0 * np.sign(c.q64[0, 0])
        c.check(c.run(msa))


@gpu_test
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,T,h_q,h_kv", [([3000, 17, 900], 1, 8, 2), ([65], 4, 4, 2),
                                             ([40, 2500], 1, 5, 5)])
def test_decode_keeps_the_low_parts(msa, gpu, lens, T, h_q, h_kv, d):
    """Eight query rows per KV head or fewer: queries and probabilities are high and low bf16
    parts, which leave 2^-16 of a value (two half steps); the output's rounding is the rest."""
    c = Case(gpu, 17, "bf16", lens, [T] * len(lens), 16, h_q, h_kv, d, [5] * len(lens))
    got = c.run(msa)[:c.rows].double().cpu().numpy()
    g = h_q // h_kv
    a = 0
    for r, L in enumerate(lens):
        local = L - T + np.arange(T)
        q = rotate64(c.q64[a:a + T], c.pos0 + local)
        for h in range(h_q):
            k = np.concatenate([c.ck64[r, :5, h // g], c.k64[r][:, h // g]])
            v = np.concatenate([c.cv64[r, :5, h // g], c.v64[r][:, h // g]])
            for t in range(T):
                n = 5 + local[t] + 1
                s = k[:n] @ q[t, h] * d ** -0.5
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ v[:n]
                # 2^-16 of the score's terms for the query's parts, as much for the angles'
                # and the fp32 sums' errors (2^-18 and n d 2^-24 at most), 2^-16 of the
                # probabilities twice (their parts; exponential and sums)
                ds = 2.0 ** -15 * (np.abs(k[:n]) @ np.abs(q[t, h])).max() * d ** -0.5
                tol = (math.expm1(2 * ds) + 2 * 2.0 ** -16) * (p @ np.abs(v[:n])) + \
                    2.0 ** -8 * np.abs(o)
                assert (np.abs(got[a + t, h] - o) <= tol).all(), (r, h, t)
        a += T


@gpu_test
def test_attend_is_repeatable(msa, gpu):
    c = Case(gpu, 21, "bf16", [3000, 20, 900], [1, 1, 64], 64, 32, 8, 128, [64, 3, 0])
    first = c.run(msa)
    for _ in range(5):
        assert torch.equal(c.run(msa)[:c.rows], first[:c.rows])


@gpu_test
@pytest.mark.parametrize("T", [1, 40])
def test_attend_bad_requests(msa, gpu, T):
    """A page outside the pool, a length past the table, a negative one and row starts past the
    rows: recorded, and the other requests are right."""
    def case():
        return Case(gpu, 31, "bf16", [200, 150, 90], [T, T, T], 16, 8, 2, 128, [4, 5, 6])

    def others(c, O, bad):
        o, tol = c.reference()
        got = O[:c.rows].double().cpu().numpy()
        a = 0
        for r, t in enumerate(c.new):
            if r not in bad:
                assert (np.abs(got - o) <= tol)[a:a + t].all(), r
            a += t

    for what in ("page", "negative_page", "long", "negative", "starts"):
        c = case()
        bad = {1}
        if what == "page":
            c.table[1, 2] = c.K.shape[0]
        elif what == "negative_page":
            c.table[1, 0] = -1
        elif what == "long":
            c.length[1] = c.table.shape[1] * 16 + 1
        elif what == "negative":
            c.length[1] = -3
        else:
            c.row_start[2:] = 1 << 30
            bad = {1, 2}
        ws = c.workspace(msa)
        O = c.run(msa, ws=ws)
        assert msa.msa_workspace_status(ws) == 3, what
        others(c, O, bad)
    c = case()
    assert msa.msa_workspace_status(ws) == 3
    others(c, c.run(msa, ws=ws), set())
    assert msa.msa_workspace_status(ws) == 0  # each call starts the word


@gpu_test
def test_attend_rows_of_a_long_pool(msa, gpu):
    """Pages whose element offsets pass 2^31 (a pool of 4.6 GB)."""
    page, h_kv, d = 64, 8, 128
    n_pages = (1 << 31) // (page * h_kv * d) + 40
    K = torch.zeros(n_pages, page, h_kv, d, dtype=torch.bfloat16, device=gpu)
    V = torch.zeros_like(K)
    for T in (1, 40):
        c = Case(gpu, 41, "bf16", [100, 70], [T, T], page, 16, h_kv, d, None)
        used = torch.unique(c.table[c.table < c.K.shape[0]]).long()
        shift = n_pages - c.K.shape[0]
        K[used + shift], V[used + shift] = c.K[used], c.V[used]
        O = msa.paged_attend(c.Q, c.row_start, c.length, K, V,
                             torch.where(c.table < c.K.shape[0], c.table + shift, c.table),
                             c.pos0, c.base)
        c.check(O)
    slot = _i32([n_pages * page - 1], gpu)
    new = torch.ones(1, h_kv, d, dtype=torch.bfloat16, device=gpu)
    msa.paged_append(K, V, slot, _i32([0], gpu), new, new, 0, 0.0)
    assert (V[-1, -1] == 1).all() and (K[-1, -1] == 1).all()
    assert int((V[:10].float() != 0).sum()) == 0


@gpu_test
def test_one_row_of_any_stride(msa, gpu):
    """A single row's stride means nothing (torch leaves it as it was)."""
    c = Case(gpu, 61, "bf16", [50], [1], 16, 8, 2, 128, None, pad=0)
    for stride in (1, 7):
        q = torch.as_strided(c.Q.contiguous(), c.Q.shape, (stride, 128, 1))
        O = msa.paged_attend(q, c.row_start, c.length, c.K, c.V, c.table, c.pos0, c.base)
        c.check(O)
        new = torch.as_strided(torch.ones(1, 2, 128, dtype=torch.bfloat16, device=gpu), (1, 2, 128),
                               (stride, 128, 1))
        K = torch.zeros(1, 16, 2, 128, dtype=torch.bfloat16, device=gpu)
        V = torch.zeros_like(K)
        msa.paged_append(K, V, _i32([3], gpu), _i32([0], gpu), new, new, 0, 0.0)
        assert (V[0, 3] == 1).all() and float(V.float().sum()) == 256


@gpu_test
def test_cache_keeps_a_captured_workspace(msa, gpu):
    """A later, larger call of the cache's own workspace leaves a captured step's alone."""
    rs = np.random.RandomState(3)
    f = lambda *s: torch.from_numpy(rs.standard_normal(s).astype(np.float32)).bfloat16().to(gpu)
    cache = msa.PagedCache(2, 40, 16, 20, 256, 2, 128, rope_base=BASE, device=gpu)
    cache.plan(_i32([200, 30], gpu))
    cache.append(0, f(230, 2, 128), f(230, 2, 128))
    cache.plan(_i32([201, 31], gpu))
    cache.append(0, f(2, 2, 128), f(2, 2, 128))
    q = f(2, 4, 128)
    want = cache.attend(0, q).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cache.attend(0, q)
    wide = cache.attend(0, f(200, 32, 128), O=torch.zeros(200, 32, 128, dtype=torch.bfloat16,
                                                          device=gpu))  # a larger workspace
    junk = [torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device=gpu) for _ in range(8)]
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(int(j.min()) == 0xFF for j in junk)
    assert wide.shape == (200, 32, 128)


# ------------------------------------------------------------------ the three together
class Life:
    """Requests that begin, grow, are cut back and end, step by step, against dense K/V kept on
    the host."""

    def __init__(self, msa, gpu, n_req=6, layers=2, seed=0):
        self.rs = np.random.RandomState(seed)
        self.h_q, self.h_kv, self.d, self.layers, self.n = 8, 2, 128, layers, n_req
        self.cache = msa.PagedCache(n_req, 60, 16, 20, 160, self.h_kv, self.d, n_layers=layers,
                                    pos0=4, rope_base=BASE, device=gpu)
        self.gpu, self.lens = gpu, [0] * n_req
        e = np.zeros((0, self.h_kv, self.d))
        self.k = [[e] * n_req for _ in range(layers)]
        self.v = [[e] * n_req for _ in range(layers)]
        self.mem = self.rs.randint(0, 9, n_req).tolist()
        f = lambda: torch.from_numpy(self.rs.standard_normal(
            (n_req, 8, self.h_kv, self.d)).astype(np.float32)).bfloat16()
        self.ctx = [(f(), f()) for _ in range(layers)]
        self.ctx_dev = [(a.to(gpu), b.to(gpu)) for a, b in self.ctx]
        self.ctx_len = _i32(self.mem, gpu)

    def targets(self):
        out = []
        for x in self.lens:
            u = self.rs.rand()
            out.append(0 if u < 0.15 else int(self.rs.randint(0, x + 1)) if u < 0.3 else
                       min(150, x + int(self.rs.randint(0, 26))))
        return out

    def inputs(self, rows=160):
        f = lambda h: torch.from_numpy(self.rs.standard_normal(
            (rows, h, self.d)).astype(np.float32)).bfloat16()
        return [(f(self.h_q), f(self.h_kv), f(self.h_kv)) for _ in range(self.layers)]

    def step(self, layer, q, k, v):
        c = self.cache
        c.append(layer, k, v)
        return c.attend(layer, q, *self.ctx_dev[layer], self.ctx_len)

    def check(self, target, inputs, outs):
        new = [max(0, t - x) for x, t in zip(self.lens, target)]
        start = np.concatenate([[0], np.cumsum(new)])
        assert self.cache.out["row_start"].cpu().tolist() == start.tolist()
        g = self.h_q // self.h_kv
        for layer in range(self.layers):
            q64, k64, v64 = (t.double().numpy() for t in inputs[layer])
            got = outs[layer].double().cpu().numpy()
            for r in range(self.n):
                a, b, x, t = start[r], start[r + 1], self.lens[r], target[r]
                pos = 4 + x + np.arange(b - a)
                kr = rotate64(k64[a:b], pos)
                kr = torch.from_numpy(kr).float().bfloat16().double().numpy()
                keep = min(x, t)
                K = self.k[layer][r] = np.concatenate([self.k[layer][r][:keep], kr])
                V = self.v[layer][r] = np.concatenate([self.v[layer][r][:keep], v64[a:b]])
                assert K.shape[0] == t
                m = self.mem[r]
                q = rotate64(q64[a:b], pos)
                for h in range(self.h_q):
                    ck, cv = (z[r, :m, h // g].double().numpy() for z in self.ctx[layer])
                    o, tol = attend64(q[:, h], np.concatenate([ck, K[:, h // g]]),
                                      np.concatenate([cv, V[:, h // g]]),
                                      m + x + 1 + np.arange(b - a), self.d ** -0.5, "bf16")
                    # a stored key may fall on the other side of a rounding than the 64-bit
                    # rotation's: twice the query's share
                    assert (np.abs(got[a:b, h] - o) <= 2 * tol).all(), (layer, r, h)
        self.lens = list(target)


@gpu_test
def test_requests_live_and_die(msa, gpu):
    life = Life(msa, gpu)
    for _ in range(12):
        target, inputs = life.targets(), life.inputs()
        life.cache.plan(_i32(target, gpu))
        outs = [life.step(i, *(t.to(gpu) for t in inputs[i])) for i in range(life.layers)]
        assert life.cache.status() == 0
        life.check(target, inputs, outs)
    table, n_free = life.cache.block_table.cpu().numpy(), int(life.cache.n_free.item())
    held = [table[r, c] for r, x in enumerate(life.lens) for c in range(-(-x // 16))]
    free = life.cache.free_list[:n_free].cpu().tolist()
    assert sorted(held + free) == list(range(60))  # every page once


@gpu_test
def test_captured_step_replays(msa, gpu):
    """One captured step (plan, two layers) replayed as the requests live and die."""
    life = Life(msa, gpu, seed=4)
    target_dev = _i32([0] * life.n, gpu)
    bufs = [tuple(t.to(gpu) for t in x) for x in life.inputs()]

    def whole():
        life.cache.plan(target_dev)
        return [life.step(i, *bufs[i]) for i in range(life.layers)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        whole()  # warm-up: nothing is asked for
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = whole()
    for _ in range(8):
        target, inputs = life.targets(), life.inputs()
        target_dev.copy_(_i32(target, gpu))
        for b, x in zip(bufs, inputs):
            for dst, src in zip(b, x):
                dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert life.cache.status() == 0
        life.check(target, inputs, outs)


@gpu_test
def test_two_streams_at_once(msa, gpu):
    """Two calls in flight on two streams, each with its own workspace."""
    cases = [Case(gpu, 50 + i, "bf16", [2000 + 300 * i, 40], [1, 30], 32, 16, 4, 128, [64, 2])
             for i in range(2)]
    wss = [c.workspace(msa) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(4):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                outs[i].append(c.run(msa, ws=wss[i]))
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        for x in o:
            c.check(x)
