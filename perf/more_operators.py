"""A paged key/value cache: its tables, its rows, its attention, and the prompts that fill it.

Four operators, each with the plain form that defines it (elementary torch
operations, in 32 bits) and, where `own` is set, the library's call:

  pages      target_model_verify_gb300.plan_pages: block tables and slot maps
             built on the GPU from the requests' lengths.
  append     target_model_verify_gb300.append_paged: new positions' keys and
             values into the pages that a slot map names.
  paged      target_model_verify_gb300.verify_attention_paged: attention of
             one new token, or of a verify step's few, over a paged bf16 cache.
  prompt     target_model_verify_gb300.prompt_attention: causal attention over
             packed prompts of different lengths.

Both attention operators have grouped heads and take a tanh cap on the scores,
a bias that falls with distance and a sliding window.
"""
import math
import random

import torch

own = False

# 26 nodes, depth 5 (4, 7, 7, 5, 2 per level): the token tree of this repository's workloads.
TREE26 = (-1, 0, 0, 0, 0, 1, 1, 1, 2, 2, 3, 4, 5, 5, 6, 7, 8, 10, 11, 12, 12, 13, 14, 16, 19, 21)


def _pages(name, B, L, n, page, prompts=False):
    return {"name": name, "op": "pages", "B": B, "L": L, "n": n, "page": page, "prompts": prompts}


def _append(name, B, n, Hkv, D, page, prompts=False):
    return {"name": name, "op": "append", "B": B, "n": n, "Hkv": Hkv, "D": D, "page": page, "prompts": prompts}


def _paged(name, B, L, n, Hq, Hkv, D, page, ragged=False, cap=0.0, window=0, slopes=False, tree=False):
    return {"name": name, "op": "paged", "B": B, "L": L, "n": n, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
            "ragged": ragged, "cap": cap, "window": window, "slopes": slopes, "tree": tree}


def _prompt(name, B, L, Hq, Hkv, D, ragged=False, cap=0.0, window=0, slopes=False):
    return {"name": name, "op": "prompt", "B": B, "L": L, "Hq": Hq, "Hkv": Hkv, "D": D, "ragged": ragged,
            "cap": cap, "window": window, "slopes": slopes}


def listed():
    return [
        # a small batch's step: room for gamma = 4 guesses and the bonus position, and what is left given back
        _pages("pages_step_b8", 8, 2000, 5, 16),
        # many requests admitted at once, and their pages given back
        _pages("pages_prompts_b256", 256, 4096, 0, 16, prompts=True),
        # a full serving batch's step
        _append("append_step_b256", 256, 5, 8, 128, 16),
        # packed prompts of unequal lengths
        _append("append_prompts", 16, 4096, 8, 128, 64, prompts=True),
        # one short conversation's drafter: latency
        _paged("paged_b1_short", 1, 517, 1, 32, 8, 128, 16),
        # a full serving batch, a token each
        _paged("paged_b64_4k", 64, 4096, 1, 32, 8, 128, 16),
        # one long document
        _paged("paged_b1_long", 1, 131072, 1, 32, 8, 128, 64),
        # a verify step with wide heads, capped scores and a local window
        _paged("paged_verify_wide", 16, 8192, 5, 8, 4, 256, 32, ragged=True, cap=50.0, window=1024),
        # one long prompt
        _prompt("prompt_b1_8k", 1, 8192, 32, 8, 128),
        # a batch of unequal prompts
        _prompt("prompt_ragged", 24, 2500, 32, 8, 128, ragged=True),
        # short questions with narrow heads, biased by distance
        _prompt("prompt_short_bias", 33, 101, 16, 4, 64, ragged=True, slopes=True),
        # wide heads, capped scores, a local window
        _prompt("prompt_wide_window", 2, 4001, 8, 4, 256, cap=50.0, window=1024),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def draw(rng):
    op = rng.choice(("pages", "append", "paged", "paged", "prompt", "prompt"))
    page = rng.choice((16, 16, 32, 64, 128, 256))
    if op == "pages":
        if rng.random() < 0.5:
            return _unnamed(_pages("", _log_int(rng, 1, 256), _log_int(rng, 1, 4096), 0, page, True))
        n = rng.randint(1, 32)
        return _unnamed(_pages("", _log_int(rng, 1, 512), n + _log_int(rng, 1, 8192), n, page))
    D, Hkv = rng.choice((64, 128, 128, 256)), rng.choice((1, 2, 4, 8, 16))
    if op == "append":
        prompts = rng.random() < 0.5
        B = _log_int(rng, 1, 16 if prompts else 256)
        most = (1 << 26) // (B * Hkv * D)                # rows of one sequence
        n = _log_int(rng, 1, max(1, min(4096, most))) if prompts else rng.randint(1, 26)
        return _unnamed(_append("", B, n, Hkv, D, page, prompts))
    G = rng.choice((1, 2, 4, 5, 8))
    cap, slopes = rng.choice((0.0, 0.0, 20.0, 50.0)), rng.random() < 0.3
    if op == "paged":
        B = _log_int(rng, 1, 64)
        tree = rng.random() < 0.15
        n = 26 if tree else rng.choice((1, 1, 1, rng.randint(2, 9)))
        # the cache's size, and the products, stay below those of the largest listed case
        most = min((1 << 28) // (B * Hkv * D), (1 << 32) // (B * Hkv * G * n * D), 131072)
        L = n + _log_int(rng, 1, max(2, most))
        return _unnamed(_paged("", B, L, n, G * Hkv, Hkv, D, page, rng.random() < 0.6, cap,
                               rng.choice((0, 0, _log_int(rng, 1, L))), slopes, tree))
    B = _log_int(rng, 1, 48)
    most = min(int(math.sqrt((1 << 38) // (B * Hkv * G * D))), (1 << 28) // (B * Hkv * (G + 1) * D), 8192)
    L = _log_int(rng, 1, max(2, most))
    return _unnamed(_prompt("", B, L, G * Hkv, Hkv, D, rng.random() < 0.7, cap,
                            rng.choice((0, 0, _log_int(rng, 1, L))), slopes))


# ----------------------------------------------------- what a case fixes --

def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lens(case):
    """Rows of every sequence: cached ones with the new positions (paged), or the prompt's."""
    r, n, L = _rng(case), case.get("n", 1), case["L"]
    if not case["ragged"]:
        return [L] * case["B"]
    return [L if b == 0 else _log_int(r, n, L) for b in range(case["B"])]


def _steps(case):
    """Of a pages or append case, per sequence: rows held before, rows to write, rows kept of them."""
    r, n = _rng(case), case["n"]
    got = []
    for b in range(case["B"]):
        if case["prompts"]:
            count = case.get("L", n) if b == 0 else _log_int(r, 1, case.get("L", n))
            got.append((0, count, 0))
        else:
            got.append((r.randint(0, case.get("L", 1000) - 1) if case["op"] == "append" else
                        r.randint(0, case["L"] - n), n, r.randint(1, n)))
    return got


def _pages_of(rows, page):
    return -(-rows // page)


def _pairs(L, n, window):
    """(query, key) pairs of the last n of L positions."""
    full = lambda m: m * (m + 1) // 2                                  # noqa: E731
    if not window or window >= L:
        return full(L) - full(L - n)
    seen = lambda m: full(m) if m <= window else full(window) + (m - window) * window   # noqa: E731
    return seen(L) - seen(L - n)


def work(case):
    B, page = case["B"], case.get("page", 1)
    if case["op"] == "pages":
        st = _steps(case)
        rows = sum(c for _, c, _ in st)
        slots = rows if case["prompts"] else 2 * rows
        moved = sum(_pages_of(s + c, page) - _pages_of(s + k, page) for s, c, k in st)
        # per call the lengths and the pages held, the pages that change hands, and the map
        return {"bytes": 4 * (2 * 4 * B + 2 * 2 * moved + slots + rows), "flops": 2 * slots}
    if case["op"] == "append":
        rows = sum(c for _, c, _ in _steps(case))
        return {"bytes": rows * (2 * 2 * 2 * case["Hkv"] * case["D"] + 4), "flops": 0}
    Hq, Hkv, D, w, lens = case["Hq"], case["Hkv"], case["D"], case["window"], _lens(case)
    if case["op"] == "paged":
        n = case["n"]
        seen = sum(min(L, w + n - 1) if w else L for L in lens)        # rows that some position sees
        pairs = sum(min(L, w) if w else L for L in lens) * n * Hq if case["tree"] else \
            sum(_pairs(L, n, w) for L in lens) * Hq
        return {"bytes": 2 * 2 * (B * n * Hq * D + seen * Hkv * D) + 4 * (seen // page + B), "flops": 4 * pairs * D}
    T = sum(lens)
    return {"bytes": 2 * 2 * T * (Hq + Hkv) * D + 4 * B, "flops": 4 * D * Hq * sum(_pairs(L, L, w) for L in lens)}


# ---------------------------------------------------------------- inputs --

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _keys(g, *shape):
    """Keys as models have them: some channels far larger than the rest."""
    k = torch.randn(*shape, generator=g, device="cuda")
    return k.mul_(torch.randn(*shape[-2:], generator=g, device="cuda").mul_(0.6).exp_())


def _slopes(case):
    if not case["slopes"]:
        return None
    h = torch.arange(1, case["Hq"] + 1, device="cuda", dtype=torch.float32)
    return torch.exp2(-8.0 * h / case["Hq"])


def _tables(g, rows, page, max_pages, spare):
    """(table [B, max_pages], held [B], free [all], n_free [1]): pages in any order, a few more than in use."""
    held = [_pages_of(r, page) for r in rows]
    total = sum(held) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(rows), max_pages), -1, dtype=torch.int32, device="cuda")
    held_t = _ints(held)
    at = torch.arange(max_pages, device="cuda")[None, :] < held_t[:, None]
    table[at] = order[:sum(held)]
    free = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    free[:spare] = order[sum(held):]
    return table, held_t, free, _ints([spare])


@torch.no_grad()
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, st = case["B"], {"case": case}
    if case["op"] in ("pages", "append"):
        page, steps = case["page"], _steps(case)
        st["start"], st["counts"] = _ints([s for s, _, _ in steps]), _ints([c for _, c, _ in steps])
        ends = [s + c for s, c, _ in steps]
        st["cu"] = None
        st["rows"] = (B, case["n"])
        if case["prompts"]:
            cu = [0]
            for _, c, _ in steps:
                cu.append(cu[-1] + c)
            st["cu"], st["rows"] = _ints(cu), (cu[-1],)
    if case["op"] == "pages":
        need = sum(_pages_of(e, page) for e in ends)
        st["kept"] = _ints([k for _, _, k in steps])
        before = [s for s, _, _ in steps]
        used = sum(_pages_of(s, page) for s in before)
        st["tables"] = _tables(g, before, page, _pages_of(max(ends), page) + 3, need - used + 7)
        st["slots"] = torch.empty(*st["rows"], dtype=torch.int32, device="cuda")
        return st
    if case["op"] == "append":
        Hkv, D = case["Hkv"], case["D"]
        table, _, _, _ = _tables(g, ends, page, _pages_of(max(ends), page), 5)
        pool = sum(_pages_of(e, page) for e in ends) + 5
        slots = []
        host = table.cpu().tolist()
        for b, (s, c, _) in enumerate(steps):
            slots.append([host[b][r // page] * page + r % page for r in range(s, s + c)])
        flat = [x for row in slots for x in row]
        st["slots"] = _ints(flat).view(*st["rows"])
        # the projection's output: keys and values side by side
        kv = torch.randn(*st["rows"], 2, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
        st["k_new"], st["v_new"] = kv.unbind(-3)
        st["k"], st["v"] = (torch.randn(pool, page, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
                            for _ in range(2))
        return st
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    st["slopes"] = _slopes(case)
    if case["op"] == "paged":
        page, lens = case["page"], _lens(case)
        st["table"], _, _, _ = _tables(g, lens, page, _pages_of(max(lens), page) + 1, 3)
        pool = sum(_pages_of(L, page) for L in lens) + 3
        st["q"] = torch.randn(B, case["n"], Hq, D, generator=g, device="cuda").mul_(1.3).to(torch.bfloat16)
        st["k"] = _keys(g, pool, page, Hkv, D).to(torch.bfloat16)
        st["v"] = torch.randn(pool, page, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
        st["lens"], st["parent"] = _ints(lens), TREE26 if case["tree"] else None
        return st
    lens = _lens(case)
    T = sum(lens)
    # the projection's output: queries, keys and values side by side
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda")
    qkv[:, :Hq] *= 1.3
    qkv[:, Hq:Hq + Hkv] *= torch.randn(Hkv, D, generator=g, device="cuda").mul_(0.6).exp_()
    qkv = qkv.to(torch.bfloat16)
    st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cu = [0]
    for L in lens:
        cu.append(cu[-1] + L)
    st["cu"] = _ints(cu)
    return st


# ------------------------------------------------------------ plain forms --

def _plain_plan(tables, start, counts, page, slots, cu):
    """The tables after the sequences have gone to start + counts rows, and the map of the rows from start on."""
    table, held, free, n_free = tables
    B, max_pages = table.shape
    total, dev = free.numel(), table.device
    want = ((start + counts + page - 1) // page)[:, None]
    have, at = held[:, None], torch.arange(max_pages, device=dev)[None, :]
    give, take = (at >= want) & (at < have), (at >= have) & (at < want)
    rank = lambda m: (m.view(-1).cumsum(0) - 1).view(B, max_pages)      # noqa: E731
    top = n_free.long() + give.sum()
    ok = take.sum() <= top
    give, take = give & ok, take & ok
    stack = torch.cat([free, free[:1]])                                 # a last entry for what is not moved
    stack.scatter_(0, torch.where(give, n_free + rank(give), total).view(-1), table.view(-1))
    taken = stack[torch.where(take, top - 1 - rank(take), total)]
    table.copy_(torch.where(take, taken, torch.where(give, -1, table)))
    free.copy_(stack[:total])
    n_free.add_(give.sum() - take.sum())
    held.copy_(torch.where(ok, want[:, 0], held))
    if slots is None:
        return
    t = torch.arange(slots.numel(), device=dev)
    if cu is None:
        b = t // slots.shape[1]
        i = t - b * slots.shape[1]
    else:
        b = torch.searchsorted(cu, t, right=True) - 1
        i = t - cu[b]
    row = (start[b] + i).clamp_max(max_pages * page - 1)
    s = table[b, row // page] * page + row % page
    slots.copy_(torch.where((i < counts[b]) & ok, s, -1).view(slots.shape))


def _plain_append(st):
    at = st["slots"].view(-1).long()
    Hkv, D = st["k"].shape[2:]
    st["k"].view(-1, Hkv, D)[at] = st["k_new"].reshape(-1, Hkv, D)
    st["v"].view(-1, Hkv, D)[at] = st["v_new"].reshape(-1, Hkv, D)
    return {"k": st["k"], "v": st["v"]}


def _tree(parent, device):
    """(depth [n], ancestor-or-self [n, n]) of a tree given by its parents."""
    n = len(parent)
    up = torch.eye(n, dtype=torch.bool)
    depth = [0] * n
    for i in range(1, n):
        up[i] |= up[parent[i]]
        depth[i] = depth[parent[i]] + 1
    return torch.tensor(depth).to(device), up.to(device)


def _plain_paged(st):
    case, q, lens, table = st["case"], st["q"].float(), st["lens"].long(), st["table"].long()
    B, n, Hq, D = q.shape
    page, L = case["page"], max(_lens(case))
    dev, Hkv = q.device, case["Hkv"]
    j = torch.arange(L, device=dev)[None, :]
    row = table[:, :_pages_of(L, page)].clamp_min(0).repeat_interleave(page, 1)[:, :L] * page + j % page
    k = st["k"].view(-1, Hkv, D)[row].float()
    v = st["v"].view(-1, Hkv, D)[row].float()
    G = Hq // Hkv
    qg = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    s = torch.matmul(qg, k.permute(0, 2, 3, 1)).view(B, Hkv, G, n, L) / math.sqrt(D)
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    # positions: row j of the prefix at j, new position i at lens - n + depth[i]
    depth, up = _tree(st["parent"] or tuple(range(-1, n - 1)), dev)
    first = (lens - n)[:, None]
    new = (j - first).clamp(0, n - 1)                                      # [B, L]
    pos_k = torch.where(j < first, j, first + depth[new])
    pos_q = first + depth[None, :]                                         # [B, n]
    away = pos_q[:, :, None] - pos_k[:, None, :]                           # [B, n, L]
    seen = (j < first)[:, None, :] | ((j < lens[:, None])[:, None, :] & (j >= first)[:, None, :]
                                      & up[:, new].permute(1, 0, 2))
    if case["window"]:
        seen = seen & (away < case["window"])
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, Hkv, G, 1, 1) * away[:, None, None].float()
    s = torch.where(seen[:, None, None], s, -math.inf)
    p = torch.softmax(s, -1).view(B, Hkv, G * n, L)
    o = torch.matmul(p, v.permute(0, 2, 1, 3))                             # [B, Hkv, G n, D]
    return o.view(B, Hkv, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).to(torch.bfloat16)


def _plain_prompt(st):
    case, w = st["case"], st["case"]["window"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    out = torch.empty_like(st["q"], memory_format=torch.contiguous_format)
    t0 = 0
    for L in _lens(case):
        of = slice(t0, t0 + L)
        t0 += L
        q = st["q"][of].float().view(L, Hkv, G, D).permute(1, 2, 0, 3)      # [Hkv, G, L, D]
        k, v = st["k"][of].float().transpose(0, 1), st["v"][of].float().transpose(0, 1)
        s = torch.matmul(q, k.transpose(1, 2)[:, None]).mul_(1 / math.sqrt(D))
        if case["cap"]:
            s = case["cap"] * torch.tanh(s / case["cap"])
        i = torch.arange(L, device=q.device)
        away = i[:, None] - i[None, :]
        seen = away >= 0
        if w:
            seen = seen & (away < w)
        if st["slopes"] is not None:
            s = s - st["slopes"].view(Hkv, G, 1, 1) * away.float()
        p = torch.softmax(s.masked_fill_(~seen, -math.inf), -1)
        out[of] = torch.matmul(p, v[:, None]).permute(2, 0, 1, 3).reshape(L, Hq, D).to(torch.bfloat16)
    return out


def _plan(st, start, counts, slots):
    page, cu = st["case"]["page"], st["cu"]
    if own:
        import target_model_verify_gb300 as tv
        tv.plan_pages(*st["tables"], start, counts, page, slots=slots, cu_rows=cu if slots is not None else None)
    else:
        _plain_plan(st["tables"], start, counts, page, slots, cu)


@torch.no_grad()
def run(st):
    case = st["case"]
    if case["op"] == "pages":
        # room for the new rows, then what the step did not keep is given back (of a prompt: all of it)
        _plan(st, st["start"], st["counts"], st["slots"])
        if case["prompts"]:
            _plan(st, st["start"], st["kept"], None)
            return dict(zip(("table", "held", "free", "n_free"), st["tables"]), slots=st["slots"])
        kept = torch.empty_like(st["slots"])
        _plan(st, st["start"], st["kept"], kept)
        return dict(zip(("table", "held", "free", "n_free"), st["tables"]), slots=st["slots"], kept=kept)
    if case["op"] == "append":
        if own:
            import target_model_verify_gb300 as tv
            tv.append_paged(st["k_new"], st["v_new"], st["k"], st["v"], st["slots"])
            return {"k": st["k"], "v": st["v"]}
        return _plain_append(st)
    if own:
        import target_model_verify_gb300 as tv
        how = {"softcap": case["cap"], "window": case["window"], "slopes": st["slopes"]}
        if case["op"] == "paged":
            return tv.verify_attention_paged(st["q"], st["k"], st["v"], st["table"], st["lens"],
                                             parent=st["parent"], **how)
        return tv.prompt_attention(st["q"], st["k"], st["v"], st["cu"], **how)
    return _plain_paged(st) if case["op"] == "paged" else _plain_prompt(st)


# ------------------------------------------------- from the definition, fp64 --

def _exact_pages(case, st):
    table, held, free = (st["tables"][x].tolist() for x in range(3))
    n_free, page = int(st["tables"][3]), case["page"]

    def go(counts):
        nonlocal n_free
        steps = _steps(case)
        for b, (s, _, _) in enumerate(steps):
            for x in range(_pages_of(s + counts[b], page), held[b]):
                free[n_free], table[b][x] = table[b][x], -1
                n_free += 1
        for b, (s, _, _) in enumerate(steps):
            for x in range(held[b], _pages_of(s + counts[b], page)):
                n_free -= 1
                table[b][x] = free[n_free]
            held[b] = _pages_of(s + counts[b], page)
        most = [c for _, c, _ in steps]
        return [table[b][r // page] * page + r % page if r - s < counts[b] else -1
                for b, (s, _, _) in enumerate(steps) for r in range(s, s + most[b])]

    out = {"slots": go([c for _, c, _ in _steps(case)])}
    kept = go([k for _, _, k in _steps(case)])
    if not case["prompts"]:
        out["kept"] = kept
    out.update(table=table, held=held, free=free, n_free=[n_free])
    like = dict(zip(("table", "held", "free", "n_free"), st["tables"]), slots=st["slots"], kept=st["slots"])
    return {k: _ints(v).view(like[k].shape) for k, v in out.items()}


def _weights(s, see):
    w = torch.exp(s - s.masked_fill(~see, -math.inf).amax(-1, keepdim=True)) * see
    return w / w.sum(-1, keepdim=True)


@torch.no_grad()
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "pages":
        out = _exact_pages(case, st)
        return {k: out[k] for k in ("table", "held", "free", "n_free", "slots", "kept") if k in out}
    if case["op"] == "append":
        out = {}
        for x in ("k", "v"):
            pages = st[x].double()
            new = st[x + "_new"].double().reshape(-1, case["Hkv"], case["D"])
            for i, s in enumerate(st["slots"].view(-1).tolist()):
                pages[s // case["page"], s % case["page"]] = new[i]
            out[x] = pages
        return out
    Hq, Hkv, D, cap, w = case["Hq"], case["Hkv"], case["D"], case["cap"], case["window"]
    G = Hq // Hkv
    if case["op"] == "prompt":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        t0 = 0
        for L in _lens(case):
            for h in range(Hkv):
                k, v = st["k"][t0:t0 + L, h].double(), st["v"][t0:t0 + L, h].double()
                for i0 in range(0, L, 2048):                   # queries i0 .. i1 - 1 see keys j0 .. i1 - 1
                    i1 = min(L, i0 + 2048)
                    j0 = max(0, i0 - w + 1) if w else 0
                    q = st["q"][t0 + i0:t0 + i1, h * G:(h + 1) * G].double()
                    s = torch.einsum("igd,jd->gij", q, k[j0:i1]) * D ** -0.5
                    if cap:
                        s = torch.tanh(s / cap) * cap
                    away = torch.arange(i0, i1, device="cuda")[:, None] - torch.arange(j0, i1, device="cuda")[None]
                    see = (away >= 0) & (away < w) if w else away >= 0
                    if st["slopes"] is not None:
                        s -= st["slopes"][h * G:(h + 1) * G].double()[:, None, None] * away
                    out[t0 + i0:t0 + i1, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", _weights(s, see), v[j0:i1])
            t0 += L
        return out
    q, parent, n, page = st["q"].double(), st["parent"], case["n"], case["page"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    chains = [{i} for i in range(n)]
    for i in range(1, n):
        chains[i] |= chains[i - 1 if parent is None else parent[i]]
    depth = torch.tensor([len(c) - 1 for c in chains], device="cuda")
    for b, L in enumerate(_lens(case)):
        ids = st["table"][b, :_pages_of(L, page)].long()
        k, v = st["k"][ids].double().flatten(0, 1)[:L], st["v"][ids].double().flatten(0, 1)[:L]
        first = L - n
        pos = torch.cat([torch.arange(first, device="cuda"), first + depth])
        see = torch.zeros(n, L, dtype=torch.bool, device="cuda")
        see[:, :first] = True
        for i, c in enumerate(chains):
            see[i, [first + a for a in c]] = True
        away = (first + depth)[:, None] - pos[None, :]
        if w:
            see &= away < w
        for h in range(Hkv):
            of = slice(h * G, (h + 1) * G)
            s = torch.einsum("igd,ld->gil", q[b, :, of], k[:, h]) * D ** -0.5
            if cap:
                s = torch.tanh(s / cap) * cap
            if st["slopes"] is not None:
                s -= st["slopes"][of].double()[:, None, None] * away
            out[b, :, of] = torch.einsum("gil,ld->igd", _weights(s, see), v[:, h])
    return out
