"""The operators around the cached attention calls, as measurable cases: rotary
positions (forward and gradient), rotary positions written into a KV cache,
attention of a chunk of new tokens over a paged cache, and the management of
cache pages.

``run`` computes them in plain torch (``own`` false) or through the calls of
global_soft_capped_b200 (``own`` true).
"""
import math

import numpy as np
import torch

own = False

# Head layouts of the repository's workloads: (H, Hkv, d)
SHAPES = ((8, 4, 256), (16, 8, 256), (32, 16, 128), (4, 2, 64))


def listed():
    return [
        # one new token of one sequence: the latency of a rotation in a decode step
        dict(name="rope one token", op="rope", tokens=1, H=8, Hkv=4, d=256, rot=256,
             interleaved=False, scaling="none", far=8192, grad=False),
        # a training batch of the 9B head layout, q and k cut out of one projection
        dict(name="rope 8192 tokens 9B", op="rope", tokens=8192, H=16, Hkv=8, d=256, rot=256,
             interleaved=False, scaling="none", far=8192, grad=False),
        # gradients of an odd batch, interleaved pairs on half of the head, long-context scaling
        dict(name="rope gradient 4095 tokens", op="rope", tokens=4095, H=32, Hkv=16, d=128,
             rot=64, interleaved=True, scaling="yarn", far=1 << 20, grad=True),
        # decode step of 64 sequences: one token each into pages of 16 rows
        dict(name="append 64 tokens paged", op="append", layout="paged", seqs=64, t_lo=1, t_hi=1,
             len_lo=1024, len_hi=8192, page=16, H=32, Hkv=16, d=128, rot=128, interleaved=False,
             scaling="none"),
        # prompt chunks of 16 sequences into pages of 64 rows
        dict(name="append prompt chunks paged", op="append", layout="paged", seqs=16, t_lo=200,
             t_hi=900, len_lo=1000, len_hi=4000, page=64, H=16, Hkv=8, d=256, rot=256,
             interleaved=False, scaling="linear"),
        # prompts into the rings of a local layer, wrapping round
        dict(name="append prompts ring", op="append", layout="ring", seqs=5, t_lo=900, t_hi=4096,
             len_lo=4096, len_hi=20000, page=4096, H=8, Hkv=4, d=256, rot=256, interleaved=False,
             scaling="none"),
        # five proposed tokens checked against one long context, pages of 16 rows
        dict(name="extend one long sequence", op="extend", seqs=1, t_lo=5, t_hi=5, len_lo=30001,
             len_hi=30001, page=16, H=8, Hkv=4, d=256, cap=50.0, window=0),
        # a batch of ragged proposals on a local layer
        dict(name="extend ragged batch local", op="extend", seqs=32, t_lo=1, t_hi=8, len_lo=500,
             len_hi=8192, page=64, H=16, Hkv=8, d=256, cap=50.0, window=4096),
        # longer chunks without the cap over long caches
        dict(name="extend chunks 27B uncapped", op="extend", seqs=24, t_lo=17, t_hi=32,
             len_lo=1000, len_hi=16000, page=128, H=32, Hkv=16, d=128, cap=0.0, window=0),
        # the page bookkeeping of a decode step: reserve new rows, give back rejected ones
        dict(name="pages grow and truncate", op="pages", what="step", seqs=256, len_hi=4096,
             page=16, pages=70001, row_bytes=0, caches=0),
        # beam search: 64 beams take new parents, partly filled pages are copied
        dict(name="pages fork beams", op="pages", what="fork", seqs=64, len_hi=1500, page=64,
             pages=2048, row_bytes=2048, caches=4),
        # live pages packed to the front of the cache
        dict(name="pages compact", op="pages", what="compact", seqs=96, len_hi=2048, page=64,
             pages=4096, row_bytes=2048, caches=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "extend", "pages"))
    H, Hkv, d = rng.choice(SHAPES)
    rot = rng.choice((d, d, d // 2, d // 4))
    common = dict(op=op, H=H, Hkv=Hkv, d=d)
    turn = dict(rot=rot, interleaved=rng.random() < 0.5,
                scaling=rng.choice(("none", "linear", "yarn")))
    if op == "rope":
        most = 8192 * 24 * 256 // ((H + Hkv) * d)
        return dict(common, **turn, tokens=_log(rng, 1, most), far=_log(rng, 1000, 1 << 20),
                    grad=rng.random() < 0.5)
    if op == "append":
        layout = rng.choice(("paged", "paged", "ring", "linear"))
        seqs = _log(rng, 1, 64)
        most = max(1, min(4096, 12000 * 12 * 256 // ((H + Hkv) * d) // seqs))
        t_hi = _log(rng, 1, most)
        page = 4096 if layout == "ring" else rng.choice((1, 8, 16, 64, 128, 256))
        return dict(common, **turn, layout=layout, seqs=seqs, t_lo=rng.randint(1, t_hi),
                    t_hi=t_hi, len_lo=t_hi, len_hi=t_hi + _log(rng, 1, 4096), page=page)
    if op == "extend":
        seqs = _log(rng, 1, 32)
        t_hi = _log(rng, 1, 64 if seqs <= 12 else 32)
        most = min(32768, 24 * 8500 * 16 * 128 * 32 // (seqs * Hkv * d * max(t_hi, 32)))
        len_hi = t_hi + _log(rng, 1, most)
        return dict(common, seqs=seqs, t_lo=rng.randint(1, t_hi), t_hi=t_hi,
                    len_lo=t_hi + _log(rng, 1, len_hi - t_hi) // 2, len_hi=len_hi,
                    page=rng.choice((1, 8, 16, 64, 128, 256)), cap=rng.choice((50.0, 50.0, 0.0)),
                    window=rng.choice((0, 0, 100, 1024, 4096)))
    what = rng.choice(("step", "fork", "compact"))
    page = rng.choice((8, 16, 64))
    seqs = _log(rng, 1, 256)
    len_hi = _log(rng, 1, 2048)
    pages = seqs * (-(-len_hi // page) + 2) + rng.randint(1, 500)
    bytes_hi = 2048
    while bytes_hi > 256 and pages * page * bytes_hi > 1 << 29:
        bytes_hi //= 2
    fits = pages * page * bytes_hi <= 1 << 29
    return dict(op=op, what=what, seqs=seqs, len_hi=len_hi, page=page, pages=pages,
                row_bytes=bytes_hi if fits and what != "step" else 0,
                caches=2 if fits and what != "step" else 0)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _inv_freq(rot, scaling):
    """Radians a position of each pair, and the factor on cos and sin."""
    base, inv, m = 10000.0, [], 1.0
    if scaling == "yarn":  # factor 16 over 8192 trained positions, bands of 32 and 1 turns
        factor, trained = 16.0, 8192.0
        edge = [rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
                for turns in (32.0, 1.0)]
        low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
        m = 0.1 * math.log(factor) + 1.0
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= 8.0
        elif scaling == "yarn":
            ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            w = w / factor * ramp + w * (1.0 - ramp)
        inv.append(w)
    return inv, m


def _turn_state(case):
    inv, m = _inv_freq(case["rot"], case["scaling"])
    # the same angles as turns in 64-bit fixed point, the table that a program keeps
    whole = [round(w / (2 * math.pi) * 2 ** 64) % 2 ** 64 for w in inv]
    turns = torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in whole], dtype=torch.int64,
                         device="cuda")
    return dict(inv=torch.tensor(inv, dtype=torch.float64, device="cuda"), turns=turns,
                mscale=m, rot=case["rot"], interleaved=case["interleaved"])


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).bfloat16()


def _ragged(case):
    """Lengths of the new chunks and of the sequences with them, as lists: the case's own."""
    r = np.random.RandomState(case["seqs"] + 64 * case["t_hi"] + case["len_lo"] + case["len_hi"])
    T = [r.randint(case["t_lo"], case["t_hi"] + 1) for _ in range(case["seqs"])]
    L = [max(t, r.randint(case["len_lo"], case["len_hi"] + 1)) for t in T]
    return T, L


def _ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


def _tables(r, L, page, spare):
    """A block table of scattered pages for these lengths, and the pages of the cache."""
    n = [-(-x // page) for x in L]
    perm = r.permutation(sum(n) + spare)
    table = np.full((len(L), max(n) + 1), -1, dtype=np.int32)
    at = 0
    for s, c in enumerate(n):
        table[s, :c] = perm[at:at + c]
        at += c
    return _ints(table), len(perm)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (2 ** 32))
    st = dict(case)
    if case["op"] == "rope":
        st.update(_turn_state(case))
        n, H, Hkv, d = case["tokens"], case["H"], case["Hkv"], case["d"]
        qkv = _randn(g, n, H + 2 * Hkv, d)  # one projection: q, k and v of a token side by side
        st["q"], st["k"] = qkv[:, :H], qkv[:, H:H + Hkv]
        first = r.randint(0, max(1, case["far"] - n))
        st["positions"] = _ints(first + np.arange(n))
    elif case["op"] == "append":
        st.update(_turn_state(case))
        H, Hkv, d = case["H"], case["Hkv"], case["d"]
        T, L = _ragged(case)
        qkv = _randn(g, sum(T), H + 2 * Hkv, d)
        st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        st["cu_q"] = _ints(np.concatenate([[0], np.cumsum(T)]))
        st["one_each"] = case["t_hi"] == 1
        st["lens"] = _ints(L)
        if case["layout"] == "paged":
            st["table"], pages = _tables(r, L, case["page"], 7)
            shape = (pages, case["page"], Hkv, d)
        elif case["layout"] == "ring":
            shape = (case["seqs"], case["page"], Hkv, d)
        else:
            st["cu_k"] = _ints(np.concatenate([[0], np.cumsum(L)]))
            shape = (sum(L), Hkv, d)
        st["kc"], st["vc"] = _randn(g, *shape), _randn(g, *shape)
    elif case["op"] == "extend":
        H, Hkv, d = case["H"], case["Hkv"], case["d"]
        T, L = _ragged(case)
        st["T"], st["L"] = T, L
        st["table"], pages = _tables(r, L, case["page"], 7)
        st["q"] = _randn(g, sum(T), H, d)
        st["kc"] = _randn(g, pages, case["page"], Hkv, d)
        st["vc"] = _randn(g, pages, case["page"], Hkv, d)
        st["cu_q"] = _ints(np.concatenate([[0], np.cumsum(T)]))
        st["lens"] = _ints(L)
        st["max_t"], st["max_len"] = max(T), max(L)
        st["scale"] = d ** -0.5
    else:
        n, page, pages = case["seqs"], case["page"], case["pages"]
        L = r.randint(1, case["len_hi"] + 1, n)
        table, _ = _tables(r, [int(x) for x in L], page, 0)
        wide = -(-case["len_hi"] // page) + 2
        used = int((-(-L // page)).sum())
        at = np.sort(r.permutation(pages)[:used])  # where in the cache the used pages lie
        host = np.full((n, wide), -1, dtype=np.int32)
        t = table.cpu().numpy()[:, :wide]
        host[:, :t.shape[1]] = np.where(t >= 0, at[np.maximum(t, 0)], -1)
        refs = np.zeros(pages, dtype=np.int32)
        refs[host[host >= 0]] = 1
        st["table"], st["refs"], st["lens"] = _ints(host), _ints(refs), _ints(L)
        if case["what"] == "step":
            st["add"] = _ints(r.randint(0, min(page, 8) + 1, n))
            st["back"] = _ints(r.randint(0, 4, n))
        elif case["what"] == "fork":
            parent = np.arange(n)
            moved = r.rand(n) < 0.6
            parent[moved] = r.randint(0, n, int(moved.sum()))
            st["parent"] = _ints(parent)
        st["all"] = _randn(g, case["caches"], pages, page, case["row_bytes"] // 2)
        st["caches"] = list(st["all"].unbind(0))  # a layer's cache each, as the calls take them
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _turned(x, pos, st, sign):
    """x (tokens, heads, d) turned by the angles of its positions, in fp32."""
    rot, half = st["rot"], st["rot"] // 2
    a = pos.double()[:, None] * st["inv"][None, :]
    c = (a.cos() * st["mscale"]).float()[:, None, :]
    s = (a.sin() * (sign * st["mscale"])).float()[:, None, :]
    x = x.float()
    part, rest = x[..., :rot], x[..., rot:]
    if st["interleaved"]:
        one, two = part[..., 0::2], part[..., 1::2]
        y = torch.stack((one * c - two * s, two * c + one * s), dim=-1).flatten(-2)
    else:
        one, two = part[..., :half], part[..., half:]
        y = torch.cat((one * c - two * s, two * c + one * s), dim=-1)
    return torch.cat((y, rest), dim=-1).to(torch.bfloat16)


def _plain_rope(st):
    sign = -1.0 if st["grad"] else 1.0
    return [_turned(st["q"], st["positions"], st, sign),
            _turned(st["k"], st["positions"], st, sign)]


def _plain_append(st):
    t = torch.arange(st["q"].shape[0], device="cuda", dtype=torch.int32)
    s = (torch.searchsorted(st["cu_q"], t, right=True) - 1).long()
    cu, lens = st["cu_q"].long(), st["lens"].long()
    pos = lens[s] - (cu[s + 1] - cu[s]) + (t - cu[s])
    q, k = _turned(st["q"], pos, st, 1.0), _turned(st["k"], pos, st, 1.0)
    page = st["page"]
    if st["layout"] == "paged":
        row = st["table"].long()[s, pos // page] * page + pos % page
    elif st["layout"] == "ring":
        row = s * page + pos % page
    else:
        row = st["cu_k"].long()[s] + pos
    st["kc"].view(-1, *st["k"].shape[1:]).index_copy_(0, row, k)
    st["vc"].view(-1, *st["k"].shape[1:]).index_copy_(0, row, st["v"].contiguous())
    return [q, st["kc"], st["vc"]]


def _plain_extend(st):
    q, table, page = st["q"], st["table"].long(), st["page"]
    Hkv, d = st["kc"].shape[2], st["kc"].shape[3]
    cu, lens = st["cu_q"].long(), st["lens"].long()
    T = cu[1:] - cu[:-1]
    j = torch.arange(st["max_len"], device="cuda")
    i = torch.arange(st["max_t"], device="cuda")
    row = table[:, j // page].clamp_min(0) * page + j % page                    # (n, S)
    there = (j[None, :] < lens[:, None])[:, :, None, None]
    k = st["kc"].view(-1, Hkv, d)[row].float().where(there, 0.0)
    v = st["vc"].view(-1, Hkv, d)[row].float().where(there, 0.0)
    at = (cu[:-1, None] + torch.minimum(i[None, :], T[:, None] - 1))            # (n, T)
    x = torch.einsum("ntghd,nsgd->nghts", q.view(-1, Hkv, 2, d)[at].float(), k) * st["scale"]
    if st["cap"] > 0:
        x = torch.tanh(x / st["cap"]) * st["cap"]
    p = (lens - T)[:, None] + i[None, :]                                        # (n, T)
    seen = j[None, None, :] <= p[:, :, None]
    if st["window"] > 0:
        seen &= p[:, :, None] - j[None, None, :] < st["window"]
    x = x.where(seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - top)
    total = w.sum(-1, keepdim=True)
    o = torch.einsum("nghts,nsgd->ntghd", w / total, v)
    lse = (top + torch.log(total))[..., 0]                                      # (n, g, h, T)
    rows = torch.arange(q.shape[0], device="cuda", dtype=torch.int32)
    s = (torch.searchsorted(st["cu_q"], rows, right=True) - 1).long()
    t = rows - cu[s]
    return [o[s, t].flatten(1, 2).to(torch.bfloat16),
            lse[s, :, :, t].flatten(1, 2).t().contiguous()]


def _pages_of(n, page):
    return (n + (page - 1)) // page


def _free_pages(refs):
    """Page numbers, the free ones first, each part ascending; and how many are free."""
    used = (refs != 0).int()
    return torch.argsort(used, stable=True), (1 - used).sum()


def _plain_step(st):
    table, lens, refs, page = st["table"].clone(), st["lens"].long(), st["refs"].clone(), st["page"]
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    # grow
    have, want = _pages_of(lens, page), _pages_of(lens + st["add"], page)
    fits = want <= table.shape[1]
    need = torch.where(fits, want - have, 0)
    end = need.cumsum(0)
    order, free = _free_pages(refs)
    granted = fits & ((end <= free) | (need == 0))
    new = granted[:, None] & (col >= have[:, None]) & (col < want[:, None])
    rank = (end - need)[:, None] + col - have[:, None]
    page_no = order[rank.clamp(0, refs.numel() - 1)]
    table = torch.where(new, page_no.int(), table)
    refs.index_add_(0, page_no.flatten(), new.flatten().int())
    lens = torch.where(granted, lens + st["add"], lens)
    grown, grown_refs = table.clone(), refs.clone()
    # truncate
    keep = (lens - st["back"]).clamp_min(0)
    gone = (col >= _pages_of(keep, page)[:, None]) & (table >= 0)
    refs.index_add_(0, table.clamp_min(0).flatten().long(), -gone.flatten().int())
    table = torch.where(gone, -1, table)
    return [grown, grown_refs, granted.int(), table, keep.int(), refs]


def _plain_fork(st):
    table, lens, refs, page = st["table"], st["lens"].long(), st["refs"].clone(), st["page"]
    parent = st["parent"].long()
    n = lens.numel()
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    moves = parent != torch.arange(n, device="cuda")
    full, part = lens[parent] // page, lens[parent] % page > 0
    need = (moves & part).long()
    end = need.cumsum(0)
    order, free = _free_pages(refs)
    granted = ~moves | (end <= free) | (need == 0)
    moves = moves & granted
    fresh = order[(end - 1).clamp(0, refs.numel() - 1)].int()
    share = moves[:, None] & (col < full[:, None])
    tail = (moves & part)[:, None] & (col == full[:, None])
    old = table[parent]
    out = torch.where(share, old, torch.where(tail, fresh[:, None], -1))
    out = torch.where(moves[:, None], out, table)
    src = torch.where(moves & part, old.gather(1, full.clamp_max(table.shape[1] - 1)[:, None])[:, 0], -1)
    dst = torch.where(moves & part, fresh, -1)
    gone = moves[:, None] & (table >= 0)
    refs.index_add_(0, table.clamp_min(0).flatten().long(), -gone.flatten().int())
    refs.index_add_(0, out.clamp_min(0).flatten().long(), (share | tail).flatten().int())
    lens = torch.where(moves, lens[parent], lens).int()
    return [out, lens, refs, src, dst, granted.int()]


def _plain_compact(st):
    table, refs = st["table"], st["refs"]
    n = refs.numel()
    used = refs != 0
    live = used.sum()
    at = torch.arange(n, device="cuda")
    hole, mover = ~used & (at < live), used & (at >= live)
    to = torch.argsort((~hole).int(), stable=True)       # holes ascending, then the rest
    of = torch.argsort((~mover).int(), stable=True)      # movers ascending, then the rest
    rank = torch.arange(n // 2, device="cuda")
    real = rank < mover.sum()
    src = torch.where(real, of[:n // 2], -1).int()
    dst = torch.where(real, to[:n // 2], -1).int()
    new = at.clone()
    new[of] = torch.where(at < mover.sum(), to, of)
    table = torch.where(table >= 0, new[table.clamp_min(0).long()].int(), -1)
    refs = torch.where(at < live, torch.where(hole, refs[of[(hole.cumsum(0) - 1).clamp_min(0)]], refs), 0)
    return [table, refs, src, dst, live.int().reshape(1)]


def _plain_copy(caches, src, dst):
    """Pages src to pages dst of every cache, where src is not -1."""
    real = src >= 0
    caches[:, dst[real].long()] = caches[:, src[real].long()]


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _own(st):
    import global_soft_capped_b200 as g2
    if st["op"] in ("rope", "append"):
        plan = g2.RopePlan(st["turns"], st["rot"], st["interleaved"], st["mscale"])
    if st["op"] == "rope":
        turn = g2.rope_backward if st["grad"] else g2.rope
        return list(turn(st["q"], st["k"], st["positions"], plan))
    if st["op"] == "append":
        cu = None if st["one_each"] else st["cu_q"]
        if st["layout"] == "paged":
            q = g2.rope_append_paged(st["q"], st["k"], st["v"], st["kc"], st["vc"], cu,
                                     st["table"], st["lens"], plan)
        elif st["layout"] == "ring":
            q = g2.rope_append_ring(st["q"], st["k"], st["v"], st["kc"], st["vc"], cu,
                                    st["lens"], plan)
        else:
            q = g2.rope_append(st["q"], st["k"], st["v"], st["kc"], st["vc"], cu, st["cu_k"],
                               plan)
        return [q, st["kc"], st["vc"]]
    if st["op"] == "extend":
        return list(g2.extend_paged(st["q"], st["kc"], st["vc"], st["cu_q"], st["table"],
                                    st["lens"], st["max_t"], query_scale=st["scale"],
                                    softcap=st["cap"], window=st["window"]))
    page, refs = st["page"], st["refs"].clone()
    if st["what"] == "step":
        table, lens = st["table"].clone(), st["lens"].clone()
        granted = g2.pages_grow(table, lens, refs, st["add"], page)
        grown, grown_refs = table.clone(), refs.clone()
        keep = (lens - st["back"]).clamp_min_(0)
        g2.pages_truncate(table, lens, refs, keep, page)
        return [grown, grown_refs, granted, table, lens, refs]
    if st["what"] == "fork":
        table, lens, src, dst, granted = g2.pages_fork(st["table"], st["lens"], refs,
                                                       st["parent"], page)
        if st["caches"]:
            g2.pages_copy(st["caches"], src, dst)
        return [table, lens, refs, src, dst, granted] + st["caches"]
    table = st["table"].clone()
    src, dst, live = g2.pages_compact(table, refs)
    if st["caches"]:
        g2.pages_copy(st["caches"], src, dst)
    return [table, refs, src, dst, live] + st["caches"]


def run(st):
    if own:
        return _own(st)
    if st["op"] == "rope":
        return _plain_rope(st)
    if st["op"] == "append":
        return _plain_append(st)
    if st["op"] == "extend":
        return _plain_extend(st)
    if st["what"] == "step":
        return _plain_step(st)
    out = _plain_fork(st) if st["what"] == "fork" else _plain_compact(st)
    if st["caches"]:
        _plain_copy(st["all"], *(out[3:5] if st["what"] == "fork" else out[2:4]))
    return out + st["caches"]


# ---------------------------------------------------------------------------
# Work and definition
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * (case["H"] + case["Hkv"])
        return dict(bytes=4.0 * n * case["d"], flops=3.0 * n * case["rot"])
    if case["op"] == "append":
        t = sum(_ragged(case)[0])
        return dict(bytes=4.0 * t * (case["H"] + 2 * case["Hkv"]) * case["d"],
                    flops=3.0 * t * (case["H"] + case["Hkv"]) * case["rot"])
    if case["op"] == "extend":
        T, L = (np.array(x, dtype=np.int64) for x in _ragged(case))
        window, H, Hkv, d = case["window"] or 1 << 30, case["H"], case["Hkv"], case["d"]
        rows = np.minimum(L, window + T - 1).sum()
        seen = sum(np.minimum(np.arange(a - t, a) + 1, window).sum() for t, a in zip(T, L))
        return dict(bytes=4.0 * d * (rows * Hkv + T.sum() * H), flops=4.0 * H * seen * d)
    n, page = case["seqs"], case["page"]
    used = n * ((case["len_hi"] + 1) / 2 / page + 0.5)
    whole = case["caches"] * page * case["row_bytes"]
    if case["what"] == "step":
        moved, ints = 0, case["pages"] + 8 * n
    elif case["what"] == "fork":  # 0.6 of the sequences move, nearly all with a part-filled page
        moved, ints = 0.6 * n * (1 - 1 / page), case["pages"] + 2 * used + 8 * n
    else:
        moved, ints = used * max(0.0, 1 - used / case["pages"]), 2 * case["pages"] + 2 * used
    return dict(bytes=4.0 * ints + 2.0 * moved * whole, flops=0.0)


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "extend": _exact_extend,
            "pages": _exact_pages}[case["op"]](st)


def _exact_turn(x, pos, st, sign=1):
    """Every pair as a complex number, times m e^(i sign p w)."""
    y, half = x.double().clone(), st["rot"] // 2
    first = torch.arange(half, device="cuda")
    first, second = (2 * first, 2 * first + 1) if st["interleaved"] else (first, first + half)
    angle = sign * torch.outer(pos.double(), st["inv"])
    by = torch.polar(torch.full_like(angle, st["mscale"]), angle)
    z = torch.complex(y[:, :, first], y[:, :, second]) * by[:, None]
    y[:, :, first], y[:, :, second] = z.real, z.imag
    return y


def _exact_rope(st):
    sign = -1 if st["grad"] else 1
    return [_exact_turn(st[x], st["positions"], st, sign) for x in "qk"]


def _exact_append(st):
    cu, lens = st["cu_q"].tolist(), st["lens"].tolist()
    kc, vc = st["kc"].double(), st["vc"].double()
    q = []
    for s, length in enumerate(lens):
        a, b = cu[s], cu[s + 1]
        pos = torch.arange(length - (b - a), length, device="cuda")
        q.append(_exact_turn(st["q"][a:b], pos, st))
        k, v = _exact_turn(st["k"][a:b], pos, st), st["v"][a:b].double()
        if st["layout"] == "paged":
            at = (st["table"][s, pos // st["page"]].long(), pos % st["page"])
        elif st["layout"] == "ring":
            at = (s, pos % st["page"])
        else:
            at = (int(st["cu_k"][s]) + pos,)
        kc[at], vc[at] = k, v
    return [torch.cat(q), kc, vc]


def _exact_extend(st):
    page, cap, window = st["page"], st["cap"], st["window"]
    cu, outs, lses = st["cu_q"].tolist(), [], []
    for s, (t, length) in enumerate(zip(st["T"], st["L"])):
        pages = st["table"][s, :-(-length // page)].long()
        k = st["kc"][pages].flatten(0, 1)[:length].double().repeat_interleave(2, 1)
        v = st["vc"][pages].flatten(0, 1)[:length].double().repeat_interleave(2, 1)
        q = st["q"][cu[s]:cu[s + 1]].double()
        x = torch.bmm(q.transpose(0, 1), k.permute(1, 2, 0)) * st["scale"]
        if cap > 0:
            x = cap * torch.tanh(x / cap)
        p = torch.arange(length - t, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None, :]
        hidden = j > p
        if window > 0:
            hidden |= j <= p - window
        x.masked_fill_(hidden, -math.inf)
        lse = torch.logsumexp(x, -1)
        outs.append(torch.bmm(torch.exp(x - lse[..., None]), v.transpose(0, 1)).transpose(0, 1))
        lses.append(lse)
    return [torch.cat(outs), torch.cat(lses, 1)]


def _exact_pages(st):
    page = st["page"]
    table, refs = st["table"].cpu().numpy().copy(), st["refs"].cpu().numpy().copy()
    lens = st["lens"].cpu().numpy().copy()
    n, wide = table.shape
    free = [int(x) for x in np.flatnonzero(refs == 0)]
    if st["what"] == "step":
        granted, asked = np.ones(n, dtype=np.int32), 0
        for s in range(n):
            have, want = -(-int(lens[s]) // page), -(-int(lens[s] + st["add"][s]) // page)
            asked += want - have if want <= wide else 0
            if want > wide or (asked > len(free) and want > have):
                granted[s] = 0
                continue
            for c in range(have, want):
                table[s, c] = free[asked - want + c]
                refs[table[s, c]] += 1
            lens[s] += int(st["add"][s])
        grown = [table.copy(), refs.copy(), granted]
        for s in range(n):
            lens[s] = max(0, lens[s] - int(st["back"][s]))
            for c in range(-(-int(lens[s]) // page), wide):
                if table[s, c] >= 0:
                    refs[table[s, c]] -= 1
                    table[s, c] = -1
        return grown + [table, lens, refs]
    if st["what"] == "fork":
        old, was, parent = table.copy(), lens.copy(), st["parent"].tolist()
        src, dst = np.full(n, -1, dtype=np.int32), np.full(n, -1, dtype=np.int32)
        granted, asked = np.ones(n, dtype=np.int32), 0
        for s, p in enumerate(parent):
            if p == s:
                continue
            full, part = int(was[p]) // page, int(was[p]) % page > 0
            asked += part
            if part and asked > len(free):
                granted[s] = 0
                continue
            refs[old[s][old[s] >= 0]] -= 1
            table[s] = -1
            table[s, :full] = old[p, :full]
            if part:
                src[s], dst[s] = old[p, full], free[asked - 1]
                table[s, full] = dst[s]
            refs[table[s][table[s] >= 0]] += 1
            lens[s] = was[p]
        return [table, lens, refs, src, dst, granted] + _exact_copy(st, src, dst)
    live = int((refs != 0).sum())
    movers = [int(x) for x in np.flatnonzero(refs) if x >= live]
    src, dst = (np.full(len(refs) // 2, -1, dtype=np.int32) for _ in range(2))
    for i, x in enumerate(movers):
        src[i], dst[i] = x, free[i]
        table[table == x] = free[i]
        refs[free[i]], refs[x] = refs[x], 0
    return [table, refs, src, dst, np.array([live], dtype=np.int32)] + _exact_copy(st, src, dst)


def _exact_copy(st, src, dst):
    out = [c.double() for c in st["caches"]]
    for a, b in zip(src.tolist(), dst.tolist()):
        for c in out:
            if a >= 0:
                c[b] = c[a]
    return out
