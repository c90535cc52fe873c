"""What the paged local context promises beside its numbers: streams, errors, limits."""
import ctypes
import glob
import os

import numpy as np
import pytest
import torch

from test_paged import BASE, Case, _i32, _plan_state, gpu_test, msa, plan64  # noqa: F401

SLEEP = 60_000_000  # SM clocks, some 30 ms


# ------------------------------------------------------------------ streams
@gpu_test
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_plan_on_another_stream(msa, gpu, raw):
    """The outputs that page_plan makes are filled on its stream, before its kernel, however
    late the current stream runs."""
    lens, target = [37, 0, 16], [38, 5, 16]
    table, free, n_free = _plan_state(np.random.RandomState(1), lens, 16, 5, 20)
    ref, _, _ = plan64(target, lens, table, free, n_free, 16, 12)
    t, f = torch.from_numpy(table).to(gpu), torch.from_numpy(free).to(gpu)
    args = _i32(target, gpu), _i32(lens, gpu), _i32([n_free], gpu)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)  # the current stream
    out = msa.page_plan(*args, t, f, 16, 12, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert {k: v.cpu().tolist() for k, v in out.items()} == ref


@gpu_test
def test_append_status_on_another_stream(msa, gpu):
    K = torch.zeros(2, 16, 2, 64, device=gpu)
    V, new = torch.zeros_like(K), torch.ones(1, 2, 64, device=gpu)
    slot, pos = _i32([32], gpu), _i32([0], gpu)  # past the pool
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    ws = msa.paged_append(K, V, slot, pos, new, new, 0, 0.0, stream=side)
    torch.cuda.synchronize()
    assert msa.msa_workspace_status(ws, side) == 3


@gpu_test
@pytest.mark.parametrize("cached", [False, True], ids=["helper", "cache"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attend_on_another_stream(msa, gpu, dtype, cached):
    """The workspace that paged_attend makes is not handed to the current stream while the
    call's kernels have yet to run."""
    c = Case(gpu, 71, dtype, [2000, 300], [1, 40], 32, 16, 4, 128, [64, 2])
    size = c.workspace(msa).numel()
    side = torch.cuda.Stream()
    cache = None
    if cached:
        cache = msa.PagedCache(2, c.K.shape[0], 32, c.table.shape[1], c.total, 4, 128,
                               pos0=c.pos0, rope_base=c.base, dtype=c.tt, device=gpu)
        cache.K[0].copy_(c.K)
        cache.V[0].copy_(c.V)
        cache.block_table.copy_(c.table)
        cache.length.copy_(c.length)
        cache.out["row_start"].copy_(c.row_start)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    if cached:
        O = cache.attend(0, c.Q, **c.ctx, stream=side)
    else:
        O = c.run(msa, stream=side)
    junk = [torch.full((size,), 0x7F, dtype=torch.uint8, device=gpu) for _ in range(4)]
    junk += [torch.full(tuple(O.shape), 9.0, dtype=O.dtype, device=gpu) for _ in range(4)]
    torch.cuda.synchronize()
    c.check(O)
    assert all(bool((j == (0x7F if j.dtype == torch.uint8 else 9.0)).all()) for j in junk)


@gpu_test
def test_cache_has_a_workspace_a_stream(msa, gpu):
    """Calls of one cache on two streams may overlap."""
    cache = msa.PagedCache(2, 200, 16, 100, 400, 2, 128, rope_base=BASE, device=gpu)
    f = lambda *s: torch.randn(*s, device=gpu).bfloat16()
    cache.plan(_i32([300, 100], gpu))
    cache.append(0, f(400, 2, 128), f(400, 2, 128))
    q = [f(400, 8, 128), f(400, 8, 128)]
    want = [cache.attend(0, x)[:400].clone() for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            got[i].append(cache.attend(0, q[i], stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for g, w in zip(got, want) for x in g)


# ------------------------------------------------------------------ errors of a step
def _two_request_step(msa, gpu, T, dtype=torch.bfloat16):
    cache = msa.PagedCache(2, 40, 16, 12, 2 * T, 2, 64, rope_base=BASE, dtype=dtype, device=gpu)
    f = lambda n, h: torch.randn(n, h, 64, device=gpu).to(dtype)
    cache.plan(_i32([T, T], gpu))
    cache.append(0, f(2 * T, 2), f(2 * T, 2))
    assert cache.status() == 0
    cache.plan(_i32([2 * T, 2 * T], gpu))
    return cache, f


@gpu_test
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 40])
def test_cache_status_covers_attention(msa, gpu, T, dtype):
    """A bad page and queries for fewer rows than planned reach status(), and stay there until
    the next plan."""
    cache, f = _two_request_step(msa, gpu, T, dtype)
    cache.append(0, f(2 * T, 2), f(2 * T, 2))
    cache.attend(0, f(2 * T, 8))
    assert cache.status() == 0
    page = int(cache.block_table[1, 0])
    cache.block_table[1, 0] = 40  # past the pool
    cache.attend(0, f(2 * T, 8))
    cache.block_table[1, 0] = page
    cache.attend(0, f(2 * T, 8))  # a later layer that finds nothing wrong
    assert cache.status() == 3
    cache.plan(cache.length + 0)
    assert cache.status() == 0
    cache.plan(_i32([3 * T, 3 * T], gpu))
    cache.append(0, f(2 * T, 2), f(2 * T, 2))
    assert cache.status() == 0
    cache.attend(0, f(2 * T - 1, 8))  # a planned row without its query
    assert cache.status() == 3


@gpu_test
@pytest.mark.parametrize("rows", [0, 1, 39])
def test_cache_append_of_fewer_rows_than_planned(msa, gpu, rows):
    """Rows that the plan has a place for and that append is not given are told of: attention
    would read what their pages held before."""
    cache, f = _two_request_step(msa, gpu, 20)
    cache.append(0, f(rows, 2), f(rows, 2))
    assert cache.status() == 3
    cache.plan(_i32([50, 50], gpu))
    cache.append(0, f(40, 2), f(40, 2))  # 20 planned rows, padded
    assert cache.status() == 0


@gpu_test
@pytest.mark.parametrize("T,d", [(40, 128), (5, 128), (40, 64)])
def test_attend_wait_timeout_is_reported_and_the_stream_recovers(msa, gpu, T, d):
    """A limit of a few dozen cycles, which no scores meet: the wait runs out, the status says so,
    copies and MMAs land, and the next call is right."""
    c = Case(gpu, 91, "bf16", [900, 250, 40], [T] * 3, 32, 16, 4, d, [9, 0, 3])
    ws, O = c.workspace(msa), torch.zeros(c.total, 16, d, dtype=c.tt, device=gpu)
    step_ws = torch.zeros(256, dtype=torch.uint8, device=gpu)
    prev = msa.msa_set_device_wait_limit(64)
    try:
        c.run(msa, O=O, ws=ws, step_ws=step_ws)
        code = msa.msa_workspace_status(ws)  # synchronises the stream
    finally:
        assert msa.msa_set_device_wait_limit(prev) == 64
    assert code == 1 and msa.msa_workspace_status(step_ws) == 1
    c.check(c.run(msa, O=O, ws=ws))
    assert msa.msa_workspace_status(ws) == 0


def test_attend_step_refuses_a_misaligned_word(msa):
    ws = ctypes.c_void_p(512)
    f = ctypes.c_void_p(1024)
    need = msa.msa_paged_attend_workspace(4, 2, 8, 2, 64, 1, 5, 4, 16)
    call = lambda step: msa.lib.msa_paged_attend_step(
        f, 512, 4, 8, f, f, 2, f, f, 8, 16, f, 4, f, f, f, 5, 2, 64, 1, 0, 0.0, 0.0, f, ws, need,
        ctypes.c_void_p(step), None)
    assert call(520) == 3
    pool, i32 = torch.zeros(4, 16, 2, 64), lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(msa.MSAError, match="step_ws"):
        msa.paged_attend(torch.zeros(5, 4, 64), i32(3), i32(2), pool, pool, i32(2, 3), 0, 0.0,
                         step_ws=torch.zeros(8, dtype=torch.uint8))


def test_append_refuses_a_bad_row_start(msa):
    pool, i32 = torch.zeros(4, 16, 2, 64), lambda *s: torch.zeros(s, dtype=torch.int32)
    new = torch.zeros(3, 2, 64)
    for bad, text in ((torch.zeros(2, dtype=torch.int64), "row_start is torch.int64"),
                      (i32(0), "row_start is empty"), (i32(4)[::2], "not contiguous")):
        with pytest.raises(msa.MSAError, match=text):
            msa.paged_append(pool, pool, i32(3), i32(3), new, new, 0, 0.0, row_start=bad)


# ------------------------------------------------------------------ values
@gpu_test
@pytest.mark.parametrize("dtype,bits", [(torch.bfloat16, torch.int16), (torch.float32, torch.int32)],
                         ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
def test_append_without_rope_copies(msa, gpu, dtype, bits, d):
    """Without RoPE the keys are stored as given, bit for bit: infinities, NaN, signed zeros."""
    new = torch.randn(5, 3, d, device=gpu).to(dtype)
    new[0, 0, 3] = float("inf")
    new[1, 1, d // 2 + 7] = -float("inf")
    new[2, 2, 1] = float("nan")
    new[3] = -0.0
    new[3, 0, d // 2:] = -2.0
    K = torch.zeros(1, 16, 3, d, dtype=dtype, device=gpu)
    V = torch.zeros_like(K)
    msa.paged_append(K, V, _i32([4, 0, 9, 15, 2], gpu), _i32([0, 1, 2, 3, 4], gpu), new, new, 7,
                     0.0)
    for got in (K, V):
        assert torch.equal(got[0, [4, 0, 9, 15, 2]].view(bits), new.view(bits))


def _tolerance(dtype, rows, mag, n, spread, o, d):
    """As in test_paged: of the low parts for up to eight rows per KV head, else of the type."""
    if dtype == "bf16" and rows <= 8:
        return (np.expm1(2 * 2.0 ** -15 * mag) + 2 * 2.0 ** -16) * spread + 2.0 ** -8 * np.abs(o)
    u_s, u_p, u_o = ((2.0 ** -8 + 2.0 ** -20, 2.0 ** -8 + 2.0 ** -20, 2.0 ** -8) if dtype == "bf16"
                     else ((3 + 3 * d / 8 + 4) * 2.0 ** -22, (4 + 3 * n / 8 + 8) * 2.0 ** -22,
                           2.0 ** -23))
    return (np.expm1(2 * u_s * mag) + 2 * u_p) * spread + u_o * np.abs(o)


@gpu_test
@pytest.mark.parametrize("dtype,T,what", [
    *((dt, T, w) for dt, T in (("bf16", 1), ("bf16", 2), ("fp32", 1), ("fp32", 40), ("bf16", 40))
      for w in "vkq"), ("bf16", 9, "v")])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_infinities(msa, gpu, dtype, T, d, what):
    """Infinite elements that a token sees: one of V makes its dimension infinite; one of a key
    makes its score infinite, so that it has weight 0 or makes the row NaN; one of the query does
    so for every key."""
    c = Case(gpu, 81, dtype, [300, 45], [T, T], 16, 8, 2, d, None, base=0.0)
    inf = float("inf")
    for r, i, j, sign in ((0, 3, 5, 1), (0, 200, d - 1, -1), (1, 2, 0, 1)):
        if what != "q":
            (c.K if what == "k" else c.V)[int(c.table[r, i // 16]), i % 16, :, j] = sign * inf
            (c.k64 if what == "k" else c.v64)[r][i, :, j] = sign * inf
    if what == "q":  # rows of request 1
        c.Q[T:2 * T, :, 6] = -inf
        c.q64[T:2 * T, :, 6] = -inf
    O = c.run(msa)[:c.rows].double().cpu().numpy()
    seen = {"nan": 0, "inf": 0, "finite": 0}
    with np.errstate(invalid="ignore"):
        for r in range(2):
            for h in range(8):
                k, v = c.k64[r][:, h // 4], c.v64[r][:, h // 4]
                for t in range(T):
                    n, q = c.lens[r] - T + t + 1, c.q64[r * T + t, h]
                    s = k[:n] @ q * d ** -0.5
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    o = p @ v[:n]
                    got, good = O[r * T + t, h], np.isfinite(o)
                    np.testing.assert_array_equal(got[~good], o[~good])
                    mag = np.abs(k[:n]) @ np.abs(q) * d ** -0.5
                    mag = mag[np.isfinite(mag)].max(initial=0)
                    tol = _tolerance(dtype, T * 4, mag, n, p @ np.abs(v[:n]), o, d)
                    assert (np.abs(got - o) <= tol)[good].all(), (r, h, t)
                    seen["nan"] += int(np.isnan(o).any())
                    seen["inf"] += int(np.isinf(o).any())
                    seen["finite"] += int(good.any())
    assert seen["finite"] and (seen["inf"] if what == "v" else seen["nan"])


@gpu_test
@pytest.mark.parametrize("d", [64, 128])
def test_attend_into_rows_aligned_to_16_bytes(msa, gpu, d):
    c = Case(gpu, 33, "bf16", [300, 700, 45], [40, 5, 45], 16, 8, 2, d, [4, 0, 9])
    n = c.total * 8 * d
    buf = torch.full((n + 16,), 7.0, dtype=c.tt, device=gpu)
    O = buf[8:8 + n].view(c.total, 8, d)
    assert O.data_ptr() % 32 == 16
    c.check(c.run(msa, O=O))
    assert (O[c.rows:] == 7.0).all() and (buf[:8] == 7.0).all() and (buf[8 + n:] == 7.0).all()


# ------------------------------------------------------------------ limits
def test_attend_refuses_more_query_heads_than_it_indexes(msa):
    """One row of 2^24 heads of 128 (4 GB of bf16) passes the kernels' 32-bit offsets in a row."""
    f, ws = ctypes.c_void_p(1024), ctypes.c_void_p(512)
    for h_q in ((1 << 20) + 1, 1 << 24, 1 << 25):
        for d, dtype in ((64, 0), (128, 0), (128, 1)):
            need = msa.msa_paged_attend_workspace(1, 1, h_q, 1, d, dtype, 0, 4, 16)
            got = msa.lib.msa_paged_attend(f, h_q * d, 1, h_q, f, f, 1, f, f, 8, 16, f, 4, None,
                                           None, None, 0, 1, d, dtype, 0, 0.0, 0.0, f, ws,
                                           max(need, 256), None)
            assert got == 2, (h_q, d, dtype)


def test_kernels_that_start_early_use_ordinary_loads(msa):
    """The paged kernels are launched while the one before them may still write their inputs. A
    load through the non-coherent path is only defined for memory that nothing writes while the
    kernel lives, and the compiler may move it ahead of the wait."""
    files = glob.glob(os.path.join(os.path.dirname(msa.LIB_PATH), "csrc", "paged*.cu*"))
    assert len(files) >= 4
    for name in files:
        with open(name) as f:
            text = f.read()
        assert "__ldg(" not in text and "global.nc" not in text, name


@gpu_test
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attend_at_the_most_kv_heads(msa, gpu, dtype):
    c = Case(gpu, 44, dtype, [50, 3], [1, 1], 16, 1024, 1024, 64, [2, 0])
    c.check(c.run(msa))


@gpu_test
def test_a_cache_without_requests_and_calls_without_rows(msa, gpu):
    cache = msa.PagedCache(0, 4, 16, 1, 8, 2, 64, device=gpu)
    f = lambda n, h: torch.randn(n, h, 64, device=gpu).bfloat16()
    plan = cache.plan(torch.zeros(0, dtype=torch.int32, device=gpu))
    cache.append(0, f(8, 2), f(8, 2))
    O = torch.full((8, 8, 64), 5.0, dtype=torch.bfloat16, device=gpu)
    cache.attend(0, f(8, 8), O=O)
    assert cache.status() == 0 and (O == 5.0).all()
    assert plan["row_start"].tolist() == [0] and plan["slot_map"].tolist() == [-1] * 8
    cache = msa.PagedCache(2, 4, 16, 1, 8, 2, 64, device=gpu)
    cache.plan(_i32([0, 0], gpu))
    cache.append(0, f(0, 2), f(0, 2))
    assert cache.attend(0, f(0, 8)).shape == (0, 8, 64)
    assert cache.status() == 0
    cache.plan(_i32([2, 1], gpu))
    cache.append(0, f(3, 2), f(3, 2))
    assert cache.attend(0, f(3, 8)).isfinite().all()
    assert cache.status() == 0


@pytest.mark.parametrize("stream", [None, 0, 1234])
def test_a_cache_on_the_host_is_refused(msa, stream):
    cache = msa.PagedCache(1, 4, 16, 2, 8, 2, 64, device="cpu")
    rows = lambda h: torch.zeros(2, h, 64, dtype=torch.bfloat16)
    for call in (lambda: cache.plan(torch.ones(1, dtype=torch.int32), stream=stream),
                 lambda: cache.append(0, rows(2), rows(2), stream=stream),
                 lambda: cache.attend(0, rows(4), stream=stream)):
        with pytest.raises(msa.MSAError, match="device memory"):
            call()
