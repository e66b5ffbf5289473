"""The calls together, as a model uses them: serving over a paged cache
(reserve, append, attend, fork, roll back, compact) and training (rotate,
attend, gradients)."""
import numpy as np
import pytest
import torch

import global_soft_capped_b200 as g2
import oracle
from parity import check
from rope_model import turn

pytestmark = pytest.mark.gpu

H, HKV, D, BS = 8, 4, 128, 16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g2.load_library()
    yield
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK


class Layer:
    """One layer's caches and, on the side, every sequence's plain history."""

    def __init__(self, pages, n, window):
        self.k = torch.full((pages, BS, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.window = window
        self.hist = [(torch.empty(0, HKV, D, dtype=torch.bfloat16),
                      torch.empty(0, HKV, D, dtype=torch.bfloat16)) for _ in range(n)]

    def step(self, rng_seed, Ts, table, lens, plan):
        """Appends T_s random tokens per sequence and attends; checks both."""
        g = torch.Generator().manual_seed(rng_seed)
        total = sum(Ts)
        qkv = torch.randn(total, H + 2 * HKV, D, generator=g).bfloat16()
        x = qkv.cuda()
        cu = torch.tensor(np.concatenate([[0], np.cumsum(Ts)]), dtype=torch.int32).cuda()
        q = g2.rope_append_paged(x[:, :H], x[:, H:H + HKV], x[:, H + HKV:], self.k, self.v, cu,
                                 table, lens, plan)
        out, lse = g2.extend_paged(q, self.k, self.v, cu, table, lens, max(Ts),
                                   query_scale=D ** -0.5, window=self.window)
        pos = np.concatenate([np.arange(len(h[0]), len(h[0]) + T) for h, T in zip(self.hist, Ts)])
        kr = g2.rope(x[:, :H], x[:, H:H + HKV], torch.tensor(pos, dtype=torch.int32).cuda(),
                     plan)[1].cpu()
        at = 0
        for s, T in enumerate(Ts):
            k, v = self.hist[s]
            k, v = torch.cat([k, kr[at:at + T]]), torch.cat([v, qkv[at:at + T, H + HKV:]])
            self.hist[s] = k, v
            if T:
                ro, rl = oracle.attn(q[at:at + T].cpu()[None], k[None], v[None],
                                     q_offset=len(k) - T, query_scale=D ** -0.5,
                                     window=self.window)
                check(out[at:at + T], ro[0], lse[:, at:at + T], rl[0], f"sequence {s}")
            at += T
        return out, lse


def test_serving():
    n, cols, pages = 5, 24, 70
    plan = g2.rope_plan(D)
    table = torch.full((n, cols), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    layers = [Layer(pages, n, 0), Layer(pages, n, 40)]
    caches = [c for l in layers for c in (l.k, l.v)]

    def grow(Ts):
        granted = g2.pages_grow(table, lens, refs, torch.tensor(Ts, dtype=torch.int32).cuda(), BS)
        assert (granted == 1).all()

    def step(seed, Ts):
        grow(Ts)
        return [l.step(seed + i, Ts, table, lens, plan) for i, l in enumerate(layers)]

    step(1, [100, 33, 1, 0, 0])                  # prompts
    step(10, [1, 1, 1, 0, 0])                    # a token each
    # beams: 3 and 4 fork 0 and 1, 2 becomes a fork of 0 too
    parents = torch.tensor([0, 1, 0, 0, 1], dtype=torch.int32).cuda()
    table, lens, src, dst, granted = g2.pages_fork(table, lens, refs, parents, BS)
    assert (granted == 1).all()
    g2.pages_copy(caches, src, dst)
    for l in layers:
        l.hist = [l.hist[p] for p in parents.tolist()]
    step(20, [1, 1, 1, 1, 1])                    # each beam goes its own way
    step(30, [4, 7, 2, 5, 3])                    # proposed tokens
    before = lens.tolist()
    back = [2, 7, 0, 1, 3]                       # some are rejected
    keep = [a - b for a, b in zip(before, back)]
    g2.pages_truncate(table, lens, refs, torch.tensor(keep, dtype=torch.int32).cuda(), BS)
    assert lens.tolist() == keep
    for l in layers:
        l.hist = [(k[:m], v[:m]) for (k, v), m in zip(l.hist, keep)]
    step(40, [3, 1, 1, 20, 2])
    # one sequence ends, the rest moves to the front of the cache
    end = lens.clone()
    end[0] = 0
    g2.pages_truncate(table, lens, refs, end, BS)
    for l in layers:
        l.hist[0] = (l.hist[0][0][:0], l.hist[0][1][:0])
    src, dst, live = g2.pages_compact(table, refs)
    assert int((src >= 0).sum()) > 0 and not refs[int(live):].any()
    g2.pages_copy(caches, src, dst)
    for l in layers:
        l.k[int(live):] = float("nan")           # nothing looks behind the live pages
        l.v[int(live):] = float("nan")
    step(50, [9, 1, 1, 1, 1])                    # a new prompt in the free slot
    # the same state through the existing single-token call
    q = torch.randn(n, H, D, device="cuda").bfloat16()
    out, lse = g2.decode_paged(q, layers[0].k, layers[0].v, table, lens, int(lens.max()),
                               query_scale=D ** -0.5)
    for s in range(n):
        k, v = layers[0].hist[s]
        ro, rl = oracle.attn(q[s].cpu()[None, None], k[None], v[None], q_offset=len(k) - 1,
                             query_scale=D ** -0.5)
        check(out[s], ro[0, 0], lse[s], rl[0, :, 0], f"decode {s}")
    g2.pages_truncate(table, lens, refs, torch.zeros(n, dtype=torch.int32, device="cuda"), BS)
    assert not refs.any()


def test_ring_serving():
    """A local layer's ring: prompt longer than the ring, then single tokens."""
    R, W, n = 64, 64, 2
    plan = g2.rope_plan(D, interleaved=True)
    kr = torch.zeros(n, R, HKV, D, dtype=torch.bfloat16, device="cuda")
    vr = torch.zeros_like(kr)
    hist = [[], []]
    lens = [0, 0]
    for step, Ts in enumerate([[150, 30], [1, 1], [1, 1], [1, 1]]):
        x = torch.randn(sum(Ts), H + 2 * HKV, D, generator=torch.Generator().manual_seed(step)
                        ).bfloat16().cuda()
        lens = [a + t for a, t in zip(lens, Ts)]
        ld = torch.tensor(lens, dtype=torch.int32).cuda()
        cu = None if step else torch.tensor([0, 150, 180], dtype=torch.int32).cuda()
        q = g2.rope_append_ring(x[:, :H], x[:, H:H + HKV], x[:, H + HKV:], kr, vr, cu, ld, plan)
        pos = np.concatenate([np.arange(a - t, a) for a, t in zip(lens, Ts)])
        k = g2.rope(x[:, :H], x[:, H:H + HKV], torch.tensor(pos, dtype=torch.int32).cuda(), plan)[1]
        at = 0
        for s, T in enumerate(Ts):
            hist[s].append((k[at:at + T].cpu(), x[at:at + T, H + HKV:].cpu()))
            at += T
        if step:
            out, lse = g2.decode_ring(q, kr, vr, ld, W, query_scale=D ** -0.5)
            for s in range(n):
                kk, vv = (torch.cat(t) for t in zip(*hist[s]))
                ro, rl = oracle.attn(q[s].cpu()[None, None], kk[None], vv[None],
                                     q_offset=len(kk) - 1, query_scale=D ** -0.5, window=W)
                check(out[s], ro[0, 0], lse[s], rl[0, :, 0], f"ring {s}")


def test_training():
    """Rotation, attention and both gradients: dq and dk of the unrotated
    inputs, against the chain rule in 64 bits."""
    B, T, h, g, d = 1, 150, 4, 2, 64
    plan = g2.rope_plan(d)
    inv, _ = g2.rope_frequencies(d)
    gen = torch.Generator().manual_seed(2)
    q, k, v, dout = (torch.randn(B, T, n, d, generator=gen).bfloat16() for n in (h, g, g, h))
    pos = np.arange(T)
    pd = torch.tensor(pos, dtype=torch.int32).cuda()
    qr, kr = g2.rope(q.cuda(), k.cuda(), pd, plan)
    out, lse = g2.prefill(qr, kr, v.cuda(), query_scale=d ** -0.5, window=70)
    dqr, dkr, dv = g2.prefill_backward(qr, kr, v.cuda(), out, lse, dout.cuda(),
                                       query_scale=d ** -0.5, window=70)
    dq, dk = g2.rope_backward(dqr, dkr, pd, plan)
    rq, rk, rv = oracle.attn_bwd(qr.cpu(), kr.cpu(), v, dout, query_scale=d ** -0.5, window=70)
    for got, ref in ((dq, turn(rq[0], pos, inv, d, False, 1.0, -1)),
                     (dk, turn(rk[0], pos, inv, d, False, 1.0, -1)), (dv, rv[0])):
        # the gradients' bound (1e-2 relative) plus one more rounding (2^-8)
        err = np.linalg.norm(got[0].double().cpu().numpy() - ref)
        assert err <= (1e-2 + 2.0 ** -8) * np.linalg.norm(ref)
