"""Workloads of the paged local context of sparse generation.

Three operators that serve a batch of requests of different lengths together:

* ``plan``: the block tables and slot maps of a step, built on the GPU from the requests' lengths;
* ``append``: the step's new K/V rows, keys rotated at their positions, written into pages;
* ``attend``: attention of every request's new tokens over [routed memory ; paged local context].

``listed()`` names fixed cases, ``draw`` makes more of the same ranges, ``prepare`` builds a
case's inputs on the GPU, ``run`` is one call (``own`` chooses between the library's kernels and
the plain torch form of the same operation), ``work`` counts the bytes and operations the
operation cannot do without, and ``exact`` evaluates the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

ROPE_BASE = 1e6
CHUNKS_PER_DOC = 8
# the costliest case that ``draw`` may return: as the largest listed ones
MAX_FLOPS = 1.1e12
MAX_FP32_FLOPS = 3.0e10  # fp32 has no wide tensor-core path
MAX_BYTES = 2.2e9
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    bf = dict(op="attend", dtype="bf16", h_q=32, h_kv=8, d=128)
    return [
        # one token for each of a serving batch's requests: the plan every decode step begins with
        dict(name="plan_decode_256", op="plan", n_req=256, page=64, old_lo=100, old_hi=8192,
             new_lo=1, new_hi=1, finished=0.03),
        # admission of a large batch of prompts into small pages while one request in eight ends
        dict(name="plan_prompts_512", op="plan", n_req=512, page=16, old_lo=0, old_hi=2500,
             new_lo=1, new_hi=1000, finished=0.125),
        # the rows of a decode step of 64 requests
        dict(name="append_decode_64", op="append", dtype="bf16", h_kv=8, d=128, page=64, rows=64,
             n_req=64, longest=16384, pad=0),
        # prompts of a prefill step, padded to the step's row capacity
        dict(name="append_prompts_16k", op="append", dtype="bf16", h_kv=8, d=128, page=64,
             rows=15873, n_req=9, longest=20000, pad=511),
        # an fp32 layer with small heads and small pages
        dict(name="append_fp32_1000", op="append", dtype="fp32", h_kv=2, d=64, page=16, rows=1000,
             n_req=7, longest=2048, pad=24),
        # one user, one token: latency (the 2,048-row local context of the decode workloads)
        dict(bf, name="attend_one_2k", n_req=1, longest=2048, shortest=2048, new_lo=1, new_hi=1,
             ones=1.0, page=64, k=8),
        # a serving batch's decode step, ragged lengths: bound by the cache's bytes
        dict(bf, name="attend_decode_64x16k", n_req=64, longest=16384, shortest=256, new_lo=1,
             new_hi=1, ones=1.0, page=64, k=16),
        # many short conversations, eight query heads per KV head, small heads, small pages
        dict(name="attend_decode_256_d64", op="attend", dtype="bf16", h_q=16, h_kv=2, d=64,
             n_req=256, longest=2000, shortest=33, new_lo=1, new_hi=1, ones=1.0, page=16, k=0),
        # checking five drafted tokens of each of 16 requests
        dict(bf, name="attend_verify_16x5", n_req=16, longest=8000, shortest=1000, new_lo=5,
             new_hi=5, ones=0.0, page=32, k=16),
        # one chunk of a long prompt over what is cached of it: bound by the tensor cores
        dict(bf, name="attend_chunk_2k_of_32k", n_req=1, longest=32768, shortest=32768,
             new_lo=2048, new_hi=2048, ones=0.0, page=64, k=16),
        # a mixed step: most requests decode while a few prompts are read in odd chunks
        dict(bf, name="attend_mixed_24", n_req=24, longest=8256, shortest=1025, new_lo=65,
             new_hi=1000, ones=0.8, page=16, k=4),
        # fp32, small: the tiny-layer configuration's type
        dict(name="attend_fp32_5x40", op="attend", dtype="fp32", h_q=8, h_kv=2, d=64, n_req=5,
             longest=1500, shortest=40, new_lo=1, new_hi=40, ones=0.2, page=16, k=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        hi = _log_int(rng, 100, 8192)
        new_hi = rng.choice([1, 1, _log_int(rng, 2, 1000)])
        return dict(op=op, n_req=_log_int(rng, 1, 512), page=page, old_lo=rng.choice([0, 1, 100]),
                    old_hi=hi, new_lo=rng.choice([0, 1]), new_hi=new_hi,
                    finished=rng.choice([0.0, 0.05, 0.125]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128, 128])
    if op == "append":
        rows = _log_int(rng, 1, 15000)
        n_req = min(rows, _log_int(rng, 1, 128))
        return dict(op=op, dtype=dtype, h_kv=rng.choice([1, 2, 4, 8]), d=d, page=page, rows=rows,
                    n_req=n_req, longest=max(256, _log_int(rng, rows // n_req + 1, 20000)),
                    pad=rng.choice([0, rng.randint(0, 512)]))
    while True:
        h_kv = rng.choice([1, 2, 4, 8, 8])
        kind = rng.choice(["decode", "decode", "verify", "chunk", "mixed"])
        n_req = _log_int(rng, 1, 256) if kind == "decode" else _log_int(rng, 1, 32)
        new_hi = {"decode": 1, "verify": rng.randint(2, 8), "chunk": _log_int(rng, 9, 2048),
                  "mixed": _log_int(rng, 9, 1000)}[kind]
        longest = _log_int(rng, max(64, new_hi), 32768)
        case = dict(op=op, dtype=dtype, h_q=h_kv * rng.choice([1, 2, 4, 4, 8]), h_kv=h_kv, d=d,
                    n_req=n_req, longest=longest, shortest=rng.randint(1, longest),
                    new_lo=rng.randint(1, new_hi), new_hi=new_hi,
                    ones={"mixed": rng.uniform(0.3, 0.9)}.get(kind, 0.0), page=page,
                    k=rng.choice([0, 4, 8, 16]))
        w = work(case)
        if (w["bytes"] <= MAX_BYTES and
                w["flops"] <= (MAX_FP32_FLOPS if dtype == "fp32" else MAX_FLOPS)):
            return case


# ------------------------------------------------------------------ lengths (from the case alone)
def _lengths(case):
    """(old, new, end) of every request: cached rows, new rows, target length (0: finished)."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["n_req"]
    if case["op"] == "plan":
        old = [rng.randint(case["old_lo"], case["old_hi"]) for _ in range(n)]
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
        gone = [rng.random() < case["finished"] for _ in range(n)]
        new = [0 if g else x for x, g in zip(new, gone)]
        return old, new, [0 if g else o + x for o, x, g in zip(old, new, gone)]
    if case["op"] == "append":
        cuts = sorted(rng.sample(range(1, case["rows"]), n - 1)) if n > 1 else []
        new = [b - a for a, b in zip([0] + cuts, cuts + [case["rows"]])]
        end = [rng.randint(x, max(x, case["longest"])) for x in new]
    else:
        end = [rng.randint(case["shortest"], case["longest"]) for _ in range(n)]
        end[rng.randrange(n)] = case["longest"]
        new = [min(e, 1 if rng.random() < case["ones"] else
                   rng.randint(case["new_lo"], case["new_hi"])) for e in end]
    return [e - x for e, x in zip(end, new)], new, end


def _memory_lengths(case):
    """Routed memory rows of every request: k documents of up to CHUNKS_PER_DOC chunks."""
    rng = random.Random(f"memory {case['n_req']} {case['longest']} {case['k']}")
    return [sum(rng.randint(5, CHUNKS_PER_DOC) for _ in range(case["k"]))
            for _ in range(case["n_req"])]


def _pages(rows, page):
    return -(-rows // page)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    old, new, end = _lengths(case)
    n, page = case["n_req"], case["page"]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    # a pool with some pages to spare; held pages are scattered over it
    held_rows = old if case["op"] == "plan" else end
    counts = [_pages(x, page) for x in held_rows]
    grow = sum(max(0, _pages(e, page) - _pages(o, page)) for o, e in zip(old, end))
    n_pages = sum(counts) + (grow if case["op"] == "plan" else 0) + 3
    width = max(1, max(_pages(max(o, e), page) for o, e in zip(old, end))) + 1
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    first = np.concatenate([[0], np.cumsum(counts)])
    slot = torch.arange(width, device=dev)[None, :]
    cnt = torch.tensor(counts, device=dev)[:, None]
    where = torch.tensor(first[:-1], device=dev)[:, None] + slot
    table = torch.where(slot < cnt, perm[where.clamp(max=n_pages - 1)], table).contiguous()
    st = dict(op=case["op"], case=case, page=page, old=old, new=new, end=end, table=table,
              n_pages=n_pages)
    rows = sum(new)
    starts = [0] + np.cumsum(new).tolist()
    if case["op"] == "plan":
        free = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        n_free = n_pages - int(first[-1])
        free[:n_free] = perm[int(first[-1]):]
        cap = -(-max(rows, 1) // 64) * 64
        st.update(length=ints(old), target=ints(end), free=free, n_free=ints([n_free]), cap=cap)
        if own:
            import long_context_doc_b200 as msa
            st["ws"] = torch.zeros(msa.msa_page_plan_workspace(n, cap), dtype=torch.uint8,
                                   device=dev)
            st["out"] = msa.page_plan_buffers(n, cap, dev)
        return st
    dt, h_kv, d = DTYPES[case["dtype"]], case["h_kv"], case["d"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=dt)

    st.update(K_pages=normal(n_pages, page, h_kv, d), V_pages=normal(n_pages, page, h_kv, d))
    if case["op"] == "append":
        total = rows + case["pad"]
        pos = np.concatenate([np.arange(o, e) for o, e in zip(old, end)])
        req = np.repeat(np.arange(n), new)
        tab = table.cpu().numpy().astype(np.int64)
        slots = tab[req, pos // page] * page + pos % page
        pad = [-1] * case["pad"]
        st.update(slot_map=ints(slots.tolist() + pad), row_pos=ints(pos.tolist() + pad),
                  K_new=normal(total, h_kv, d), V_new=normal(total, h_kv, d), pos0=16)
        if own:
            st["ws"] = torch.zeros(256, dtype=torch.uint8, device=dev)
        return st
    st.update(Q=normal(rows, case["h_q"], d), row_start=ints(starts), length=ints(end),
              pos0=case["k"], ctxK=None, ctxV=None, ctx_len=None)
    if case["k"]:
        mem = _memory_lengths(case)
        width = case["k"] * CHUNKS_PER_DOC
        st.update(ctxK=normal(n, width, h_kv, d), ctxV=normal(n, width, h_kv, d),
                  ctx_len=ints(mem), mem=mem)
    else:
        st["mem"] = [0] * n
    if own:
        import long_context_doc_b200 as msa
        st["ws"] = torch.zeros(
            msa.msa_paged_attend_workspace(rows, n, case["h_q"], h_kv, d, msa.dtype_code(st["Q"]),
                                           case["k"] * CHUNKS_PER_DOC, table.shape[1], page),
            dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------------ one call
def run(st):
    if own:
        return _run_own(st)
    return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}[st["op"]](st)


def _run_own(st):
    import long_context_doc_b200 as msa
    if st["op"] == "plan":
        out = msa.page_plan(st["target"], st["length"], st["n_free"], st["table"], st["free"],
                            st["page"], st["cap"], out=st["out"], ws=st["ws"])
        return dict(length=out["length"], n_free=out["n_free"], row_start=out["row_start"],
                    slot_map=out["slot_map"], row_pos=out["row_pos"], table=st["table"],
                    free=st["free"])
    if st["op"] == "append":
        msa.paged_append(st["K_pages"], st["V_pages"], st["slot_map"], st["row_pos"], st["K_new"],
                         st["V_new"], st["pos0"], ROPE_BASE, ws=st["ws"])
        return st["K_pages"], st["V_pages"]
    return msa.paged_attend(st["Q"], st["row_start"], st["length"], st["K_pages"], st["V_pages"],
                            st["table"], st["pos0"], ROPE_BASE, ctxK=st["ctxK"], ctxV=st["ctxV"],
                            ctx_len=st["ctx_len"], ws=st["ws"])


def _plain_plan(st):
    """Pages that requests give up go back on the stack of free pages in request order, then the
    pages they need come off its top in request order; the slots follow from the tables."""
    page, n_pages = st["page"], st["n_pages"]
    old, tgt, table, free = st["length"].long(), st["target"].long(), st["table"], st["free"]
    n, width = table.shape
    dev = table.device
    have, want = (old + page - 1) // page, (tgt + page - 1) // page
    col = torch.arange(width, device=dev)[None, :]
    back = (col >= want[:, None]) & (col < have[:, None])
    need = (col >= have[:, None]) & (col < want[:, None])
    back_rank = (torch.cumsum(back.flatten().long(), 0) - 1).view(n, width)
    need_rank = (torch.cumsum(need.flatten().long(), 0) - 1).view(n, width)
    n_back, n_need = back.sum(), need.sum()
    n_free = st["n_free"][0].long()
    stack = torch.zeros(2 * n_pages + 1, dtype=torch.int32, device=dev)
    stack[:n_pages] = free
    at = torch.where(back, n_free + back_rank, 2 * n_pages)
    stack[at.flatten()] = table.flatten()
    top = n_free + n_back
    took = stack[(top - 1 - need_rank).clamp(0, 2 * n_pages)]
    table.copy_(torch.where(need, took, table))
    i = torch.arange(n_pages, device=dev)
    free.copy_(torch.where((i >= n_free) & (i < top - n_need), stack[:n_pages], free))
    new = (tgt - old).clamp(min=0)
    row_start = torch.zeros(n + 1, dtype=torch.int64, device=dev)
    row_start[1:] = torch.cumsum(new, 0)
    r = torch.arange(st["cap"], device=dev)
    req = torch.searchsorted(row_start, r, right=True) - 1
    ok = r < row_start[-1]
    req = req.clamp(max=n - 1)
    pos = old[req] + r - row_start[req]
    slot = table[req, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    return dict(length=tgt.int(), n_free=(top - n_need).int().view(1), row_start=row_start.int(),
                slot_map=torch.where(ok, slot, -1).int(), row_pos=torch.where(ok, pos, -1).int(),
                table=table, free=free)


def _rotate(x, pos):
    """Rotate-half RoPE of x [rows, heads, d] (fp32) at integer positions, angles in 64 bits."""
    d = x.shape[-1]
    inv = ROPE_BASE ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / d)
    ang = pos.double()[:, None] * inv
    c, s = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
    a, b = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], dim=-1)


def _plain_append(st):
    n = sum(st["new"])
    slot = st["slot_map"][:n].long()
    pos = st["row_pos"][:n].long() + st["pos0"]
    K, V = st["K_pages"], st["V_pages"]
    K.view(-1, *K.shape[2:])[slot] = _rotate(st["K_new"][:n].float(), pos).to(K.dtype)
    V.view(-1, *V.shape[2:])[slot] = st["V_new"][:n]
    return K, V


def _plain_attend(st):
    Q, page = st["Q"], st["page"]
    h_q, d = Q.shape[1], Q.shape[2]
    h_kv = st["K_pages"].shape[2]
    g = h_q // h_kv
    out = torch.empty_like(Q)
    r0 = 0
    for r, (old, new, end, mem) in enumerate(zip(st["old"], st["new"], st["end"], st["mem"])):
        ids = st["table"][r, :_pages(end, page)].long()
        K = st["K_pages"][ids].reshape(-1, h_kv, d)[:end]
        V = st["V_pages"][ids].reshape(-1, h_kv, d)[:end]
        if mem:
            K = torch.cat([st["ctxK"][r, :mem], K])
            V = torch.cat([st["ctxV"][r, :mem], V])
        K, V = K.float().permute(1, 2, 0), V.float().permute(1, 0, 2)
        block = max(1, (1 << 28) // (h_q * (mem + end)))  # query tokens whose scores are held
        for t0 in range(0, new, block):
            t1 = min(new, t0 + block)
            local = old + torch.arange(t0, t1, device=Q.device)
            q = _rotate(Q[r0 + t0:r0 + t1].float(), local + st["pos0"])
            q = q.view(t1 - t0, h_kv, g, d).permute(1, 2, 0, 3).reshape(h_kv, g * (t1 - t0), d)
            s = torch.matmul(q, K) / math.sqrt(d)
            key = torch.arange(mem + end, device=Q.device)
            hidden = key[None, :] > mem + local[:, None]
            s = s.view(h_kv, g, t1 - t0, mem + end).masked_fill(hidden, float("-inf"))
            s = torch.exp(s - s.amax(-1, keepdim=True))
            s = (s / s.sum(-1, keepdim=True)).view(h_kv, g * (t1 - t0), mem + end)
            o = torch.matmul(s, V).view(h_kv, g, t1 - t0, d).permute(2, 0, 1, 3)
            out[r0 + t0:r0 + t1] = o.reshape(t1 - t0, h_q, d).to(Q.dtype)
        r0 += new
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    old, new, end = _lengths(case)
    rows, page = sum(new), case["page"]
    if case["op"] == "plan":
        back = sum(max(0, _pages(o, page) - _pages(e, page)) for o, e in zip(old, end))
        need = sum(max(0, _pages(e, page) - _pages(o, page)) for o, e in zip(old, end))
        cap = -(-max(rows, 1) // 64) * 64
        # lengths in, targets in, lengths out, row starts; pages moved; a slot and a position a row
        return {"bytes": 16 * case["n_req"] + 12 + 8 * (back + need) + 8 * cap, "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    row = case["h_kv"] * case["d"] * size
    if case["op"] == "append":
        return {"bytes": 4 * rows * row + 8 * (rows + case["pad"]),
                "flops": 3 * rows * case["h_kv"] * case["d"]}
    mem = _memory_lengths(case)
    seen = sum(x * (m + o) + x * (x + 1) // 2 for o, x, m in zip(old, new, mem))
    pages = sum(_pages(e, page) for e in end)
    return {"bytes": 2 * rows * case["h_q"] * case["d"] * size + 2 * row * (sum(end) + sum(mem)) +
            4 * pages + 12 * case["n_req"],
            "flops": 4 * case["d"] * case["h_q"] * seen}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attend": _exact_attend}[st["op"]](st)


def _exact_plan(st):
    """Request by request with a list as the stack."""
    page = st["page"]
    table, free = st["table"].tolist(), st["free"].tolist()
    n0 = st["n_free"].item()
    stack = free[:n0]
    held = [table[r][:_pages(o, page)] for r, o in enumerate(st["old"])]
    for r, e in enumerate(st["end"]):
        stack.extend(held[r][_pages(e, page):])
        del held[r][_pages(e, page):]
    starts, slots, pos = [0], [], []
    for r, (o, e) in enumerate(zip(st["old"], st["end"])):
        while len(held[r]) < _pages(e, page):
            held[r].append(stack.pop())
            table[r][len(held[r]) - 1] = held[r][-1]
        for p in range(o, e):
            slots.append(held[r][p // page] * page + p % page)
            pos.append(p)
        starts.append(len(pos))
    free[n0:len(stack)] = stack[n0:]
    pad = [-1] * (st["cap"] - len(pos))

    def ints(x):
        return torch.tensor(x, dtype=torch.int32)

    return dict(length=ints(st["end"]), n_free=ints([len(stack)]), row_start=ints(starts),
                slot_map=ints(slots + pad), row_pos=ints(pos + pad), table=ints(table),
                free=ints(free))


def _turn64(x, first):
    """x [rows, heads, d] float64, row i rotated by the angles of position first + i, as complex
    numbers (pair: element j with element j + d/2)."""
    n, _, d = x.shape
    half = d // 2
    theta = torch.exp(-math.log(ROPE_BASE) * torch.arange(half, device=x.device,
                                                           dtype=torch.float64) / half)
    p = torch.arange(first, first + n, device=x.device, dtype=torch.float64)
    z = torch.complex(x[..., :half], x[..., half:])
    z = z * torch.polar(torch.ones_like(p)[:, None] * torch.ones_like(theta),
                        p[:, None] * theta)[:, None, :]
    return torch.cat([z.real, z.imag], dim=-1)


def _exact_append(st):
    K, V, page = st["K_pages"].double(), st["V_pages"].double(), st["page"]
    table = st["table"].tolist()
    at = 0
    for r, (o, e) in enumerate(zip(st["old"], st["end"])):
        k = _turn64(st["K_new"][at:at + e - o].double(), st["pos0"] + o)
        v = st["V_new"][at:at + e - o].double()
        p = o
        while p < e:
            q = min(e, (p // page + 1) * page)
            dst = table[r][p // page]
            K[dst, p % page:p % page + q - p] = k[p - o:q - o]
            V[dst, p % page:p % page + q - p] = v[p - o:q - o]
            p = q
        at += e - o
    return K, V


def _exact_attend(st):
    Q, page = st["Q"].double(), st["page"]
    rows, h_q, d = Q.shape
    g = h_q // st["K_pages"].shape[2]
    out = torch.zeros_like(Q)
    table = st["table"].tolist()
    at = 0
    for r, (o, x, e, m) in enumerate(zip(st["old"], st["new"], st["end"], st["mem"])):
        K = torch.cat([st["K_pages"][p] for p in table[r][:_pages(e, page)]])[:e].double()
        V = torch.cat([st["V_pages"][p] for p in table[r][:_pages(e, page)]])[:e].double()
        q = _turn64(Q[at:at + x], st["pos0"] + o)
        for h in range(h_q):
            k, v = K[:, h // g], V[:, h // g]
            if m:
                k = torch.cat([st["ctxK"][r, :m, h // g].double(), k])
                v = torch.cat([st["ctxV"][r, :m, h // g].double(), v])
            s = torch.einsum("td,nd->tn", q[:, h], k) * d ** -0.5
            last = m + o + torch.arange(x, device=s.device)
            ahead = torch.arange(m + e, device=s.device)[None, :] > last[:, None]
            s[ahead] = float("-inf")
            out[at:at + x, h] = torch.softmax(s, dim=-1) @ v
        at += x
    return out
