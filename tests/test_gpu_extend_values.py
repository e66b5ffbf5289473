"""Chunk attention over paged caches on values that a test of random ones does
not meet: NaN and infinities that queries see, scores that overflow."""
import math

import numpy as np
import pytest
import torch

import global_soft_capped_b200 as g2
import oracle
from global_soft_capped_b200.inputs import varlen_inputs
from parity import check
from test_gpu_extend import paged

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g2.load_library()
    yield
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK


# whole units, units cut over a few CTAs, one unit cut over every CTA; chunks
# for each row count of the kernel
LENS = [
    [(3, 70), (8, 8), (1, 300), (5, 129)],
    [(16, 40), (9, 500), (12, 12)],
    [(32, 32), (17, 700), (20, 21)],
    [(3, 20001)],
    [(30, 9000)],
]


class Chunks:
    """One set of inputs, its call and the oracle on the values as they are now."""

    def __init__(self, lens, d, cap, window=0, H=4, Hkv=2, bs=16, seed=0):
        self.H, self.d, self.bs, self.seed = H, d, bs, seed
        self.kw = dict(query_scale=d ** -0.5, softcap=cap, window=window)
        (self.Ts, self.Ss, self.cq, self.ck, self.q, self.k,
         self.v) = varlen_inputs(0, 0, 0, H, Hkv, d, 1.0, seed, seq_lens=lens)

    def run(self):
        kb, vb, table = paged(self.Ts, self.Ss, self.ck, self.k, self.v, self.bs,
                              self.kw["window"], self.seed)
        out, lse = g2.extend_paged(self.q.cuda(), kb, vb, self.cq.cuda(), table,
                                   torch.tensor(self.Ss, dtype=torch.int32).cuda(), max(self.Ts),
                                   **self.kw)
        torch.cuda.synchronize()
        return out.float().cpu(), lse.cpu()

    def oracle(self):
        out, lse = oracle.varlen(self.q, self.k, self.v, self.cq, self.ck, **self.kw)
        return np.array(out), np.array(lse)

    def sees(self, s, j):
        """(rows, ) whether each packed query row sees key j of sequence s."""
        m = np.zeros(self.q.shape[0], dtype=bool)
        pos = self.Ss[s] - self.Ts[s] + np.arange(self.Ts[s])
        w = self.kw["window"] or 1 << 40
        m[int(self.cq[s]):int(self.cq[s + 1])] = (pos >= j) & (pos - j < w)
        return m


def held(out, lse, ro, rl, bad, what):
    """Rows marked in bad (rows, heads) are NaN throughout, the others right."""
    bad = torch.from_numpy(bad)
    assert torch.isnan(out[bad]).all() and torch.isnan(lse.t()[bad]).all(), what
    good = ~bad.numpy()
    check(out[~bad], ro[good], lse.t()[~bad], rl.T[good], what)


@pytest.mark.parametrize("cap", [50.0, 0.0, 100.0])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_nan_in_a_query(lens, d, cap):
    """One element of one head of a query: that row is NaN, no other one is."""
    c = Chunks(lens, d, cap, seed=d)
    ro, rl = c.oracle()
    bad = np.zeros((c.q.shape[0], c.H), dtype=bool)
    for s in range(len(lens)):
        row, h = int(c.cq[s + 1]) - 1 - s % c.Ts[s], s % c.H
        c.q[row, h, (7 * s) % d] = NAN
        bad[row, h] = True
    held(*c.run(), ro, rl, bad, f"{lens} {d} {cap}")


@pytest.mark.parametrize("cap,window", [(50.0, 0), (0.0, 0), (100.0, 0), (50.0, 150), (0.0, 150)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_nan_in_a_visible_key(lens, d, cap, window):
    """A key's NaN reaches every query that sees it, for its KV head only, and
    none of those before it or past its window."""
    c = Chunks(lens, d, cap, window, seed=d + 1)
    ro, rl = c.oracle()
    bad = np.zeros((c.q.shape[0], c.H), dtype=bool)
    for s, (T, S) in enumerate(lens):
        # a key inside the chunk, the first, or one in the middle of what is seen
        lo = max(0, S - T - window + 1) if window else 0
        j, g = (S - (T + 1) // 2, lo, (lo + S) // 2)[s % 3], s % 2
        c.k[int(c.ck[s]) + j, g, (5 * s) % d] = NAN
        bad[:, 2 * g:2 * g + 2] |= c.sees(s, j)[:, None]
    held(*c.run(), ro, rl, bad, f"{lens} {d} {cap} {window}")


@pytest.mark.parametrize("lens", LENS, ids=str)
def test_scores_that_overflow(lens):
    """Without the cap: a score of +inf makes the row NaN (inf - inf), one of
    -inf is a key of weight 0."""
    for sign in (1.0, -1.0):
        c = Chunks(lens, 128, 0.0, seed=3)
        bad = np.zeros((c.q.shape[0], c.H), dtype=bool)
        for s, (T, S) in enumerate(lens):
            c.q[int(c.cq[s]):int(c.cq[s + 1]), 0] = c.q[int(c.cq[s]):int(c.cq[s + 1]), 0].abs() + 1
            at = int(c.ck[s]) + S - (T + 1) // 2
            c.k[at, 0] = -1000.0   # for the oracle: weight 0 for head 0
            bad[:, 0] |= c.sees(s, S - (T + 1) // 2)
        ro, rl = c.oracle()
        for s, (T, S) in enumerate(lens):
            c.k[int(c.ck[s]) + S - (T + 1) // 2, 0] = sign * 3e38
        out, lse = c.run()
        head = torch.from_numpy(bad[:, 0])
        if sign > 0:
            assert torch.isnan(out[head, 0]).all() and not (lse[0, head] == -INF).any()
        else:
            check(out[head, 0], ro[bad[:, 0], 0], lse[0, head], rl[0, bad[:, 0]], f"-inf {lens}")
        check(out[~head, 0], ro[~bad[:, 0], 0], lse[0, ~head], rl[0, ~bad[:, 0]], f"{sign} {lens}")
        check(out[:, 2:], ro[:, 2:], lse[2:], rl[2:], f"other KV head {sign} {lens}")


def test_capped_infinite_scores_are_the_cap():
    """With the cap an infinite score is the cap itself, not a NaN."""
    for lens in LENS:
        c = Chunks(lens, 64, 50.0, seed=5)
        c.q[:, 0] = c.q[:, 0].abs() + 1
        for s, (T, S) in enumerate(lens):
            c.k[int(c.ck[s]) + S - T, 0] = 2000.0     # past the cap: tanh is 1
        ro, rl = c.oracle()
        for s, (T, S) in enumerate(lens):
            c.k[int(c.ck[s]) + S - T, 0] = 3e38
        out, lse = c.run()
        check(out[:, 0], ro[:, 0], lse[0], rl[0], f"{lens}")


def test_as_the_other_calls():
    """The single-token call and the prefill give NaN for the same rows."""
    c = Chunks([(1, 700), (1, 129), (1, 3)], 128, 50.0, bs=128, seed=9)
    c.q[0, 1, 5] = NAN
    c.k[int(c.ck[1]) + 100, 1, 0] = NAN
    kb, vb, table = paged(c.Ts, c.Ss, c.ck, c.k, c.v, c.bs)
    vb = torch.nan_to_num(vb)
    unseen = torch.ones(kb.shape[:2], dtype=torch.bool)
    for s, S in enumerate(c.Ss):
        j = torch.arange(S)
        unseen[table.cpu()[s, j // c.bs].long(), j % c.bs] = False
    kb[unseen.cuda()] = 0
    lens = torch.tensor(c.Ss, dtype=torch.int32).cuda()
    kw = c.kw
    out, lse = g2.extend_paged(c.q.cuda(), kb, vb, c.cq.cuda(), table, lens, 1, **kw)
    do, dl = g2.decode_paged(c.q.cuda(), kb, vb, table, lens, 700, **kw)
    po, pl = g2.prefill_paged(c.q.cuda(), kb, vb, c.cq.cuda(), table, lens, 1, 700, **kw)
    want = torch.zeros(3, 4, dtype=torch.bool)
    want[0, 1] = want[1, 2] = want[1, 3] = True
    for o, l in ((out, lse.t()), (do, dl), (po, pl.t())):
        assert torch.equal(torch.isnan(o.float()).all(-1).cpu(), want)
        assert torch.equal(torch.isnan(o.float()).any(-1).cpu(), want)
        assert torch.equal(torch.isnan(l).cpu(), want)


def test_queries_before_the_first_key_beside_nan():
    """Rows that see no key stay 0 and -inf in a chunk whose others are NaN."""
    for cap in (50.0, 0.0):
        c = Chunks([(6, 6), (2, 300)], 64, cap, seed=2)
        c.k[0] = NAN
        kb, vb, table = paged(c.Ts, c.Ss, c.ck, c.k, c.v, c.bs)
        lens = torch.tensor([2, 300], dtype=torch.int32).cuda()
        out, lse = g2.extend_paged(c.q.cuda(), kb, vb, c.cq.cuda(), table, lens, 6, **c.kw)
        assert torch.count_nonzero(out[:4]) == 0 and (lse[:, :4] == -INF).all()
        assert torch.isnan(out[4:6].float()).all() and torch.isnan(lse[:, 4:6]).all()
        assert torch.isfinite(out[6:].float()).all() and math.isfinite(float(lse[:, 6:].sum()))


@pytest.mark.parametrize("cap", [0.0, 100.0])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(4, 700), (8, 600)] * 8, [(13, 900)] * 12, [(30, 1500)] * 8],
                         ids=["4-8", "13", "30"])
def test_values_of_any_size(lens, d, cap):
    """Scores that rise by 2^40 along the cache with values 2^100 and 2^-100 of
    the usual ones: as a weighted mean the result scales alike. (Weights that
    were allowed to grow that far before they are rescaled would overflow. Many
    units, so that a CTA meets a unit's tiles one after the other.)"""
    c = Chunks(lens, d, cap, H=32, Hkv=16, seed=d + 2)
    way = torch.sign(torch.randn(d, generator=torch.Generator().manual_seed(3)))
    c.q.copy_((0.1 * c.q.float() + way).bfloat16())
    for s, (T, S) in enumerate(lens):
        rise = 28.0 / d ** 0.5 * torch.linspace(0.0, 1.0, S).clamp_min(0.2)[:, None, None]
        rows = slice(int(c.ck[s]), int(c.ck[s]) + S)
        c.k[rows] = (0.1 * c.k[rows].float() + rise * way).bfloat16()
    ro, rl = c.oracle()
    v = c.v.clone()
    for power in (0, 100, -100):
        c.v.copy_(v.float() * 2.0 ** power)
        out, lse = c.run()
        check(out * 2.0 ** -power, ro, lse, rl, f"{d} {cap} 2^{power}")


@pytest.mark.parametrize("d,T", [(64, 3), (128, 12), (256, 30)])
def test_lowest_scores(d, T):
    """Without the cap, rows whose every score is near the lowest finite number
    still are weighted means: equal scores, equal weights."""
    c = Chunks([(T, 400), (1, 130)], d, 0.0, seed=4)
    c.q.fill_(1.0)
    # products of -2^127: -3.2e38 in log2 units, the lowest number is -3.4e38
    c.k.fill_(-2.0 ** 127 / d)
    c.kw["query_scale"] = 1.3
    out, lse = c.run()
    for s, (t, S) in enumerate([(T, 400), (1, 130)]):
        for i in range(t):
            j = slice(int(c.ck[s]), int(c.ck[s]) + S - t + i + 1)
            want = c.v[j].double().mean(0).repeat_interleave(2, 0).numpy()
            row = int(c.cq[s]) + i
            check(out[row], want, what=f"{s} {i}")
            assert torch.allclose(lse[:, row].double(),
                                  torch.full((4,), -1.3 * 2.0 ** 127, dtype=torch.float64), rtol=1e-5)


@pytest.mark.parametrize("d,lens", [(64, [(4, 700), (8, 600)] * 8), (128, [(13, 900)] * 12),
                                    (256, [(30, 1500)] * 8)], ids=["64", "128", "256"])
def test_nan_where_scores_rise(d, lens):
    """A NaN row, and one before a NaN key, in units whose references are raised
    tile by tile."""
    c = Chunks(lens, d, 0.0, H=32, Hkv=16, seed=d + 5)
    way = torch.sign(torch.randn(d, generator=torch.Generator().manual_seed(3)))
    c.q.copy_((0.1 * c.q.float() + way).bfloat16())
    for s, (T, S) in enumerate(lens):
        rise = 60.0 / d ** 0.5 * torch.linspace(0.0, 1.0, S)[:, None, None]
        rows = slice(int(c.ck[s]), int(c.ck[s]) + S)
        c.k[rows] = (0.1 * c.k[rows].float() + rise * way).bfloat16()
    ro, rl = c.oracle()
    bad = np.zeros((c.q.shape[0], c.H), dtype=bool)
    for s, (T, S) in enumerate(lens):
        row, h, g = int(c.cq[s]) + s % T, (5 * s) % c.H, (3 * s) % 16
        c.q[row, h, s] = NAN
        bad[row, h] = True
        c.k[int(c.ck[s]) + S - 2, g, s] = NAN
        bad[:, 2 * g:2 * g + 2] |= c.sees(s, S - 2)[:, None]
    held(*c.run(), ro, rl, bad, f"{d}")
