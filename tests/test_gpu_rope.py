"""Rotary positions, their gradients, and the appends into linear, ring and
paged caches, against 64-bit rotations (rope_model.py). Cache rows that a call
must not write keep their contents bit for bit."""
import numpy as np
import pytest
import torch

import global_soft_capped_b200 as g2
from rope_model import check, turn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g2.load_library()
    yield
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK


def randn(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


CASES = [
    # tokens, H, Hkv, d, rotary_dim, interleaved, scaling
    (1, 1, 1, 64, 64, False, {}),
    (1, 8, 4, 256, 256, True, {}),
    (3, 2, 1, 64, 16, False, {}),
    (5, 4, 2, 64, 48, True, {}),
    (7, 8, 4, 128, 32, False, dict(scaling="ntk", factor=8.0)),
    (129, 3, 5, 128, 128, False, {}),
    (1000, 16, 8, 256, 256, False, {}),
    (517, 32, 16, 128, 64, True, dict(scaling="yarn", factor=16.0)),
    (33, 5, 1, 256, 112, False, dict(scaling="linear", factor=4.0)),
    (4099, 4, 2, 64, 64, False, {}),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_rope_and_gradient(case):
    n, H, Hkv, d, rot, inter, scaling = case
    inv, m = g2.rope_frequencies(rot, **scaling)
    plan = g2.rope_plan(rot, interleaved=inter, **scaling)
    q, k = randn(n, H, d, seed=1), randn(n, Hkv, d, seed=2)
    rng = np.random.default_rng(n)
    pos = rng.integers(0, 1 << 20, n)
    pos[0] = 0
    pd = torch.tensor(pos, dtype=torch.int32).cuda()
    for fn, sign in ((g2.rope, 1), (g2.rope_backward, -1)):
        qo, ko = fn(q.cuda(), k.cuda(), pd, plan)
        for x, y in ((q, qo), (k, ko)):
            check(y, f64(x), turn(f64(x), pos, inv, rot, inter, m, sign), m, f"{fn.__name__} {case}")
            assert torch.equal(y.cpu()[..., rot:], x[..., rot:])  # passes through unrounded


def test_extreme_positions():
    """Every int32 position, negative ones too, is as exact as position 1."""
    pos = np.array([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 1 << 30, 123456789])
    inv, _ = g2.rope_frequencies(128)
    # positions times frequencies need more than 64 bits of angle: take the
    # phase from the fixed-point table's own definition, in Python integers
    plan = g2.rope_plan(128)
    bits = [b % 2 ** 64 for b in plan.freqs.tolist()]
    x = randn(len(pos), 2, 128, seed=5)
    qo, _ = g2.rope(x.cuda(), x.cuda(), torch.tensor(pos, dtype=torch.int32).cuda(), plan)
    want = f64(x).copy()
    for t, p in enumerate(pos):
        for i, b in enumerate(bits):
            ph = (int(p) * b) % 2 ** 64 / 2.0 ** 64 * 2 * np.pi
            one, two = f64(x)[t, :, i], f64(x)[t, :, i + 64]
            want[t, :, i] = one * np.cos(ph) - two * np.sin(ph)
            want[t, :, i + 64] = two * np.cos(ph) + one * np.sin(ph)
    check(qo, f64(x), want, 1.0, "extreme positions")


def test_strided_inputs_and_in_place():
    """q and k cut out of one projection, dense batches, results in place and
    into other strided tensors."""
    B, T, H, Hkv, d = 2, 37, 8, 4, 128
    plan = g2.rope_plan(d)
    qkv = randn(B, T, H + 2 * Hkv, d, seed=3).cuda()
    pos = torch.arange(B * T, dtype=torch.int32, device="cuda")
    q, k = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
    want = g2.rope(q.contiguous(), k.contiguous(), pos, plan)
    got = g2.rope(q, k, pos, plan)
    assert got[0].shape == q.shape and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    v = qkv[:, :, H + Hkv:].clone()
    back = g2.rope(q, k, pos, plan, out=(q, k))
    assert back[0].data_ptr() == qkv.data_ptr()
    assert torch.equal(qkv[:, :, :H], want[0]) and torch.equal(qkv[:, :, H:H + Hkv], want[1])
    assert torch.equal(qkv[:, :, H + Hkv:], v)
    big = torch.zeros(B * T, H + Hkv + 1, d, dtype=torch.bfloat16, device="cuda")
    g2.rope(randn(B * T, H, d, seed=4).cuda(), randn(B * T, Hkv, d, seed=4).cuda(), pos, plan,
            out=(big[:, :H], big[:, H:H + Hkv]))
    assert torch.count_nonzero(big[:, -1]) == 0 and torch.count_nonzero(big[:, :-1]) > 0


def test_helper_checks():
    plan = g2.rope_plan(64)
    x = randn(4, 2, 64).cuda()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    for bad in [lambda: g2.rope(x, x[:3], pos, plan), lambda: g2.rope(x, x, pos[:3], plan),
                lambda: g2.rope(x, x, pos.long(), plan), lambda: g2.rope(x.float(), x, pos, plan),
                lambda: g2.rope(x.transpose(0, 1), x, pos, plan),
                lambda: g2.rope(x, x, pos, g2.RopePlan(plan.freqs[:5], 64)),
                lambda: g2.rope(randn(2, 2, 4, 2, 64).cuda(), x, pos, plan),
                lambda: g2.rope_append_ring(x, x, x, x[:, None], x[:, None], None, pos[:3], plan),
                lambda: g2.rope_append_paged(x, x, x, x[None], x[None].float(), None, pos[None],
                                             pos, plan)]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(g2.G2AttnError):
        g2.rope(x[:, :, :63].contiguous()[..., :48].contiguous(), x[..., :48].contiguous(), pos,
                g2.rope_plan(48))


def reference_append(cache_rows, q, k, v, Ts, Ls, inv, rot, inter, m):
    """What the appends compute, in 64 bits: (q, [(row, k, v)]), rows from
    cache_rows(s, position) (None: not stored)."""
    pos = np.concatenate([np.arange(L - T, L) for T, L in zip(Ts, Ls)] or [[]])
    seq = np.repeat(np.arange(len(Ts)), Ts)
    qr, kr = turn(f64(q), pos, inv, rot, inter, m), turn(f64(k), pos, inv, rot, inter, m)
    at = [cache_rows(int(s), int(p)) for s, p in zip(seq, pos)]
    return pos, qr, kr, at


APPEND = [
    # layout, T_s, L_s, H, Hkv, d, rot, interleaved, page or ring
    ("linear", [3, 0, 1, 70], [3, 9, 100, 80], 4, 2, 64, 64, False, 0),
    ("ring", [1, 1, 1], [1, 64, 1000], 8, 4, 256, 256, False, 64),
    ("ring", [100, 5, 64, 0], [130, 5, 64, 7], 2, 1, 128, 64, True, 64),
    ("paged", [1, 1, 1, 1, 1], [1, 16, 17, 300, 33], 32, 16, 128, 128, False, 16),
    ("paged", [7, 0, 40, 1], [7, 3, 100, 64], 8, 4, 256, 128, True, 1),
    ("paged", [129, 300], [129, 1000], 16, 8, 256, 256, False, 128),
    ("paged", [5], [5], 2, 1, 64, 16, False, 1024),
]


@pytest.mark.parametrize("case", APPEND, ids=str)
@pytest.mark.parametrize("one_each", [False, True], ids=["chunks", "tokens"])
def test_append(case, one_each):
    layout, Ts, Ls, H, Hkv, d, rot, inter, size = case
    if one_each:
        Ls = [L for L in Ls if L > 0]
        Ts = [1] * len(Ls)
    n, total = len(Ts), sum(Ts)
    inv, m = g2.rope_frequencies(rot, scaling="yarn", factor=2.0)
    plan = g2.rope_plan(rot, interleaved=inter, scaling="yarn", factor=2.0)
    pad = 0 if one_each else 3           # rows behind the last sequence
    qkv = randn(total + pad, H + 2 * Hkv, d, seed=11).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    cu = None if one_each else torch.tensor(np.concatenate([[0], np.cumsum(Ts)]),
                                            dtype=torch.int32).cuda()
    lens = torch.tensor(Ls, dtype=torch.int32).cuda()
    q_out = torch.full((total + pad, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    if layout == "linear":
        ck = np.concatenate([[0], np.cumsum(Ls)])
        kc = randn(int(ck[-1]) + 2, Hkv, d, seed=12).cuda()
        rows = lambda s, p: int(ck[s]) + p
        run = lambda kc, vc: g2.rope_append(q, k, v, kc, vc, cu, torch.tensor(
            ck, dtype=torch.int32).cuda(), plan, q_out=q_out)
    elif layout == "ring":
        kc = randn(n, size, Hkv, d, seed=12).cuda()
        rows = lambda s, p: None if p < Ls[s] - size else s * size + p % size
        run = lambda kc, vc: g2.rope_append_ring(q, k, v, kc, vc, cu, lens, plan, q_out=q_out)
    else:
        need = [-(-L // size) for L in Ls]
        perm = np.random.default_rng(5).permutation(sum(need) + 3)
        table = -np.ones((n, max(need) + 2), dtype=np.int32)
        at = 0
        for s, c in enumerate(need):
            table[s, :c] = perm[at:at + c]
            at += c
        kc = randn(len(perm), size, Hkv, d, seed=12).cuda()
        td = torch.tensor(table).cuda()
        rows = lambda s, p: int(table[s, p // size]) * size + p % size
        run = lambda kc, vc: g2.rope_append_paged(q, k, v, kc, vc, cu, td, lens, plan, q_out=q_out)
    vc = randn(*kc.shape, seed=13).cuda()
    k0, v0 = kc.clone().view(-1, Hkv, d).cpu(), vc.clone().view(-1, Hkv, d).cpu()
    run(kc, vc)
    torch.cuda.synchronize()
    pos, qr, kr, at = reference_append(rows, q[:total], k[:total], v, Ts, Ls, inv, rot, inter, m)
    check(q_out[:total], f64(q[:total]), qr, m, "q")
    assert torch.isnan(q_out[total:].float()).all()
    kf, vf = kc.view(-1, Hkv, d), vc.view(-1, Hkv, d)
    stored = [i for i, r in enumerate(at) if r is not None]
    rs = torch.tensor([at[i] for i in stored], dtype=torch.long)
    check(kf[rs.cuda()], f64(k[stored]), kr[stored], m, "k rows")
    assert torch.equal(vf.cpu()[rs], v.cpu()[stored])
    others = torch.ones(len(kf), dtype=torch.bool)
    others[rs] = False
    assert torch.equal(kf.cpu()[others], k0[others]) and torch.equal(vf.cpu()[others], v0[others])


def test_append_in_place_and_same_as_rope():
    """q rotated in place; the same bits as the plain rotation."""
    n, H, Hkv, d = 50, 8, 4, 128
    plan = g2.rope_plan(d)
    q, k, v = (randn(n, h, d, seed=s).cuda() for s, h in ((1, H), (2, Hkv), (3, Hkv)))
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    kc, vc = torch.zeros(n, Hkv, d, dtype=torch.bfloat16).cuda(), torch.zeros(
        n, Hkv, d, dtype=torch.bfloat16).cuda()
    want = g2.rope(q, k, torch.arange(n, dtype=torch.int32).cuda(), plan)
    got = g2.rope_append(q, k, v, kc, vc, cu, cu, plan, q_out=q)
    assert got.data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(kc, want[1]) and torch.equal(vc, v)


def test_tokens_without_a_row_are_dropped_and_reported():
    H, Hkv, d = 2, 1, 64
    plan = g2.rope_plan(d)
    q, k = randn(6, H, d).cuda(), randn(6, Hkv, d).cuda()
    cu = torch.tensor([0, 3, 6], dtype=torch.int32).cuda()
    kc = torch.zeros(4, 4, Hkv, d, dtype=torch.bfloat16).cuda()
    vc = kc.clone()
    # sequence 0: positions 3, 4, 5 (page column 1 has no page); sequence 1: a
    # page outside the cache, and a column past the table
    table = torch.tensor([[2, -1], [0, 9]], dtype=torch.int32).cuda()
    g2.rope_append_paged(q, k, k, kc, vc, cu, table, torch.tensor([6, 9], dtype=torch.int32).cuda(),
                         plan)
    assert g2.g2attn_get_device_error() == g2.G2ATTN_ERR_CACHE_ROW
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK
    assert torch.equal(vc[2, 3], k[0])
    vc[2, 3] = 0
    assert torch.count_nonzero(vc) == 0
    # more new tokens than the sequence is long
    kr = torch.zeros(2, 8, Hkv, d, dtype=torch.bfloat16).cuda()
    vr = kr.clone()
    g2.rope_append_ring(q, k, k, kr, vr, cu, torch.tensor([2, 3], dtype=torch.int32).cuda(), plan)
    assert g2.g2attn_get_device_error() == g2.G2ATTN_ERR_CACHE_ROW
    assert torch.equal(vr[0, :2], k[1:3]) and torch.equal(vr[1, :3], k[3:])
    assert torch.count_nonzero(vr[0, 2:]) == 0 and torch.count_nonzero(vr[1, 3:]) == 0
    # rows past the end of a packed cache
    kl = torch.zeros(4, Hkv, d, dtype=torch.bfloat16).cuda()
    g2.rope_append(q, k, k, kl, kl.clone(), cu, torch.tensor([0, 3, 6], dtype=torch.int32).cuda(),
                   plan)
    assert g2.g2attn_get_device_error() == g2.G2ATTN_ERR_CACHE_ROW
    # a ring that a chunk overruns is no error
    g2.rope_append_ring(q, k, k, kr[:, :2].contiguous(), vr[:, :2].contiguous(), cu,
                        torch.tensor([3, 3], dtype=torch.int32).cuda(), plan)
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK


def test_empty_slots_of_a_decode_batch():
    """One token each, sequences of length 0 among them: no row, no error."""
    n, H, Hkv, d = 5, 4, 2, 128
    plan = g2.rope_plan(d)
    q, k, v = (randn(n, h, d, seed=s).cuda() for s, h in ((1, H), (2, Hkv), (3, Hkv)))
    lens = torch.tensor([3, 0, 8, 0, 1], dtype=torch.int32).cuda()
    out = torch.full_like(q, 7.0)
    kr = torch.zeros(n, 8, Hkv, d, dtype=torch.bfloat16).cuda()
    vr = kr.clone()
    g2.rope_append_ring(q, k, v, kr, vr, None, lens, plan, q_out=out)
    assert (out[[1, 3]] == 7.0).all() and torch.count_nonzero(vr[[1, 3]]) == 0
    for s, p in ((0, 2), (2, 7), (4, 0)):
        assert torch.equal(vr[s, p], v[s])
    want = g2.rope(q, k, (lens - 1).clamp_min(0), plan)
    assert torch.equal(out[[0, 2, 4]], want[0][[0, 2, 4]])
    table = torch.tensor([[0, -1], [-1, -1], [1, 2], [-1, -1], [3, -1]], dtype=torch.int32).cuda()
    kb, vb = torch.zeros(4, 4, Hkv, d, dtype=torch.bfloat16).cuda(), torch.zeros(
        4, 4, Hkv, d, dtype=torch.bfloat16).cuda()
    out.fill_(7.0)
    g2.rope_append_paged(q, k, v, kb, vb, None, table, lens, plan, q_out=out)
    assert (out[[1, 3]] == 7.0).all() and torch.equal(vb[0, 2], v[0]) and torch.equal(vb[2, 3], v[2])
    assert torch.equal(kb[3, 0], k[4]) and torch.count_nonzero(vb.abs().amax((-1, -2))) == 3
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK


def test_single_steps_of_a_dense_batch():
    """(B, 1, H, d) slices of one projection, as a decode loop has them."""
    B, H, Hkv, d = 6, 8, 4, 64
    plan = g2.rope_plan(d, interleaved=True)
    qkv = randn(B, 1, H + 2 * Hkv, d, seed=8).cuda()
    pos = torch.tensor([5, 0, 99, 7, 7, 1 << 20], dtype=torch.int32).cuda()
    got = g2.rope(qkv[:, :, :H], qkv[:, :, H:H + Hkv], pos, plan)
    want = g2.rope(qkv[:, 0, :H].contiguous(), qkv[:, 0, H:H + Hkv].contiguous(), pos, plan)
    assert torch.equal(got[0][:, 0], want[0]) and torch.equal(got[1][:, 0], want[1])
    one = g2.rope(qkv[:1, :, :H], qkv[:1, :, H:H + Hkv], pos[:1], plan)
    assert torch.equal(one[0], got[0][:1])


def test_many_sequences():
    """More sequences than a warp or a CTA has tokens, empty ones among them."""
    n, H, Hkv, d, bs = 3001, 2, 1, 64, 8
    rng = np.random.default_rng(9)
    Ts = rng.integers(0, 3, n)
    Ls = Ts + rng.integers(0, 9, n)
    plan = g2.rope_plan(d)
    inv, _ = g2.rope_frequencies(d)
    total = int(Ts.sum())
    q, k = randn(total, H, d, seed=1).cuda(), randn(total, Hkv, d, seed=2).cuda()
    table = torch.arange(2 * n, dtype=torch.int32).view(n, 2).cuda()
    kc = torch.zeros(2 * n, bs, Hkv, d, dtype=torch.bfloat16).cuda()
    vc = kc.clone()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(Ts)]), dtype=torch.int32).cuda()
    g2.rope_append_paged(q, k, k, kc, vc, cu, table, torch.tensor(Ls, dtype=torch.int32).cuda(),
                         plan)
    pos = np.concatenate([np.arange(L - T, L) for T, L in zip(Ts, Ls)])
    rows = np.repeat(np.arange(n), Ts) * 2 * bs + pos
    assert torch.equal(vc.view(-1, Hkv, d)[torch.tensor(rows).cuda()], k)
    check(kc.view(-1, Hkv, d)[torch.tensor(rows).cuda()], f64(k), turn(f64(k), pos, inv, d, False),
          1.0, "k")
    assert torch.count_nonzero(vc.abs().amax(-1)) <= total


def test_graph_replay_and_other_stream():
    """Captured and replayed on new inputs; run on a stream of the caller's."""
    n, H, Hkv, d = 9, 8, 4, 256
    plan = g2.rope_plan(d)
    q, k = randn(n, H, d, seed=1).cuda(), randn(n, Hkv, d, seed=2).cuda()
    pos = torch.arange(n, dtype=torch.int32).cuda()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g2.rope(q, k, pos, plan, out=(qo, ko), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    first = qo.clone()
    assert torch.equal(first, g2.rope(q, k, pos, plan)[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2.rope(q, k, pos, plan, out=(qo, ko))
    q.copy_(randn(n, H, d, seed=7))
    pos.add_(1000)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, g2.rope(q, k, pos, plan)[0]) and not torch.equal(qo, first)
