"""Attention of short chunks over a paged cache, against the fp64 oracle's
packed layer on the same keys and values. Every cache row that no query may see
(unused pages, rows behind a sequence's end, keys that left the window) holds
NaN, so a stray read shows up as a non-finite output."""
import numpy as np
import pytest
import torch

import global_soft_capped_b200 as g2
import oracle
from global_soft_capped_b200.inputs import varlen_inputs
from parity import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g2.load_library()
    yield
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK


def paged(Ts, Ss, ck, k, v, bs, window=0, seed=0, spare=2):
    """Scattered pages; NaN wherever no query of the call may look."""
    need = [-(-S // bs) for S in Ss]
    perm = np.random.default_rng(seed).permutation(sum(need) + spare)
    Hkv, d = k.shape[1], k.shape[2]
    kb = torch.full((len(perm) * bs, Hkv, d), float("nan"), dtype=torch.bfloat16)
    vb = kb.clone()
    table = -np.ones((len(Ss), max(need) + 2), dtype=np.int32)
    at = 0
    for s, S in enumerate(Ss):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
        lo = max(0, S - Ts[s] - window + 1) if window else 0
        j = np.arange(lo, S)
        if len(j) and Ts[s]:
            rows = torch.from_numpy(table[s, j // bs].astype(np.int64) * bs + j % bs)
            kb[rows], vb[rows] = k[int(ck[s]) + lo:int(ck[s]) + S], v[int(ck[s]) + lo:int(ck[s]) + S]
    shape = (len(perm), bs, Hkv, d)
    return kb.view(shape).cuda(), vb.view(shape).cuda(), torch.from_numpy(table).cuda()


def run(lens, H, Hkv, d, bs, window=0, cap=50.0, alpha=None, max_T=None, seed=0, std=1.0, edit=None):
    alpha = d ** -0.5 if alpha is None else alpha
    Ts, Ss, cq, ck, q, k, v = varlen_inputs(0, 0, 0, H, Hkv, d, std, seed, seq_lens=lens)
    if edit is not None:
        edit(q, k, v, cq, ck)
    kb, vb, table = paged(Ts, Ss, ck, k, v, bs, window, seed)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, q.shape[0]), float("nan"), device="cuda")
    g2.extend_paged(q.cuda(), kb, vb, cq.cuda(), table, torch.tensor(Ss, dtype=torch.int32).cuda(),
                    max(Ts) if max_T is None else max_T, query_scale=alpha, softcap=cap,
                    window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK
    ro, rl = oracle.varlen(q, k, v, cq, ck, query_scale=alpha, softcap=cap, window=window)
    return out, lse, ro, rl


CASES = [
    # (T_s, S_s), H, Hkv, d, block_size, window, cap
    ([(1, 1)], 2, 1, 64, 1, 0, 50.0),
    ([(1, 1), (1, 2), (1, 127), (1, 128), (1, 129), (1, 1000)], 4, 2, 64, 16, 0, 50.0),
    ([(1, 1), (1, 2), (1, 127), (1, 128), (1, 129), (1, 1000)], 4, 2, 128, 2, 0, 0.0),
    ([(1, 1), (1, 2), (1, 127), (1, 128), (1, 129), (1, 1000)], 4, 2, 256, 128, 0, 50.0),
    ([(2, 3), (8, 8), (5, 900), (0, 40), (7, 256)], 8, 4, 256, 16, 0, 50.0),
    ([(2, 3), (8, 8), (5, 900), (0, 40), (7, 256)], 8, 4, 128, 64, 0, 0.0),
    ([(2, 3), (8, 8), (5, 900), (0, 40), (7, 256)], 6, 3, 64, 8, 0, 50.0),
    ([(9, 9), (16, 17), (3, 700), (13, 333)], 4, 2, 256, 32, 0, 50.0),
    ([(9, 9), (16, 17), (3, 700), (13, 333)], 4, 2, 128, 256, 0, 50.0),
    ([(9, 9), (16, 17), (3, 700), (13, 333)], 4, 2, 64, 1, 0, 0.0),
    ([(17, 17), (32, 500), (31, 129), (1, 5)], 4, 2, 256, 16, 0, 50.0),
    ([(17, 17), (32, 500), (31, 129), (1, 5)], 4, 2, 128, 16, 0, 0.0),
    ([(17, 17), (32, 500), (31, 129), (1, 5)], 4, 2, 64, 16, 0, 50.0),
    ([(70, 70), (200, 333), (33, 1200)], 2, 1, 256, 64, 0, 50.0),
    ([(70, 70), (200, 333), (33, 1200)], 2, 1, 256, 64, 0, 0.0),
    # windows: smaller than the chunk, across tile edges, one key
    ([(8, 900), (3, 3), (1, 500)], 4, 2, 128, 16, 1, 50.0),
    ([(8, 900), (3, 3), (1, 500)], 4, 2, 256, 16, 5, 0.0),
    ([(16, 900), (9, 9), (1, 500)], 4, 2, 64, 32, 100, 50.0),
    ([(40, 900), (64, 64), (5, 500)], 4, 2, 256, 128, 130, 50.0),
    ([(40, 900), (64, 64), (5, 500)], 4, 2, 128, 8, 257, 0.0),
    # caps whose fixed shift would not fit (running max with the cap), tight caps
    ([(4, 700), (8, 50)], 4, 2, 128, 16, 0, 100.0),
    ([(20, 700), (8, 50)], 4, 2, 256, 16, 300, 100.0),
    ([(4, 700), (8, 50)], 4, 2, 256, 16, 0, 5.0),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_chunks(case):
    lens, H, Hkv, d, bs, window, cap = case
    out, lse, ro, rl = run(lens, H, Hkv, d, bs, window, cap, seed=CASES.index(case))
    check(out, ro, lse, rl, str(case))


@pytest.mark.parametrize("d,cap", [(256, 50.0), (128, 0.0), (64, 50.0)])
def test_one_long_sequence(d, cap):
    """A single long cache is split over every CTA and joined."""
    out, lse, ro, rl = run([(3, 20001)], 4, 2, d, 16, 0, cap, seed=d)
    check(out, ro, lse, rl, f"long {d}")


@pytest.mark.parametrize("d,T", [(256, 3), (128, 12), (64, 30), (256, 30)])
def test_growing_scores(d, T):
    """Scores that rise along the cache make the running max rise tile by tile
    (O and the sums are rescaled), then fall; also between split parts."""
    def edit(q, k, v, cq, ck):
        S = k.shape[0]
        ramp = torch.sin(torch.linspace(0.0, 9.0, S))[:, None, None] + 0.1
        direction = torch.randn(k.shape[2], generator=torch.Generator().manual_seed(1))
        k.copy_((k.float() * 0.3 + ramp * direction).bfloat16())
        q.copy_((q.float() * 0.3 + direction).bfloat16())
    out, lse, ro, rl = run([(T, 3000), (T, 400)], 2, 1, d, 16, 0, 0.0, alpha=0.5, seed=d + T,
                           edit=edit)
    check(out, ro, lse, rl, f"growing {d}")


@pytest.mark.parametrize("cap", [50.0, 0.0, 1e-3])
@pytest.mark.parametrize("alpha", [-0.1, 0.0])
def test_odd_scales(alpha, cap):
    """Negative and zero query scales, a cap that flattens every score."""
    out, lse, ro, rl = run([(4, 300), (9, 9)], 4, 2, 128, 16, 0, cap, alpha=alpha, seed=12)
    check(out, ro, lse, rl, f"{alpha} {cap}")


def test_zero_keys_and_queries():
    """Products of exactly 0 (with any cap), rows of equal weights."""
    def edit(q, k, v, cq, ck):
        k[::3] = 0
        q[::2] = 0
    for cap in (50.0, 0.0, 1e-30, 100.0):
        out, lse, ro, rl = run([(8, 200), (3, 130)], 4, 2, 64, 16, 0, cap, seed=13, edit=edit)
        check(out, ro, lse, rl, f"zeros {cap}")


def test_peaked_scores_with_the_cap():
    out, lse, ro, rl = run([(4, 1000), (16, 130)], 4, 2, 128, 16, 0, 50.0, alpha=3.0, seed=2)
    check(out, ro, lse, rl, "peaked")


def test_chunks_longer_than_max_T():
    """max_T only picks the variant: longer chunks are right with any."""
    for max_T in (1, 9, 500):
        out, lse, ro, rl = run([(20, 300), (1, 40), (33, 77)], 4, 2, 128, 16, 50, 50.0,
                               max_T=max_T, seed=4)
        check(out, ro, lse, rl, f"max_T {max_T}")


def test_prompt_sized_chunks():
    """Many units per sequence: prompts of hundreds of tokens in small pages."""
    out, lse, ro, rl = run([(700, 700), (300, 1500), (1, 900)], 4, 2, 64, 8, 0, 50.0, max_T=700,
                           seed=21)
    check(out, ro, lse, rl, "prompts")
    out, lse, ro, rl = run([(500, 900)], 2, 1, 128, 16, 300, 0.0, seed=22)
    check(out, ro, lse, rl, "windowed prompt")


def test_many_sequences():
    rng = np.random.default_rng(8)
    lens = [(int(t), int(t) + int(s)) for t, s in zip(rng.integers(0, 4, 1024),
                                                      rng.integers(0, 60, 1024))]
    lens = [(t, max(1, s)) for t, s in lens]
    out, lse, ro, rl = run(lens, 2, 1, 64, 16, 0, 50.0, seed=6)
    check(out, ro, lse, rl, "1024 sequences")


def _random_cases(n, seed):
    rng = np.random.default_rng(seed)
    cases = []
    for _ in range(n):
        d = int(rng.choice([64, 128, 256]))
        Hkv = int(rng.integers(1, 4))
        top = int(rng.choice([1, 8, 16, 40]))
        lens = []
        for _ in range(int(rng.integers(1, 9))):
            T = int(rng.integers(1, top + 1))
            lens.append((T, T + int(rng.integers(0, 700))))
        window = 0 if rng.random() < 0.5 else int(rng.integers(1, 400))
        cases.append((lens, 2 * Hkv, Hkv, d, int(2 ** rng.integers(0, 9)), window,
                      float(rng.choice([50.0, 50.0, 0.0, 100.0])), int(rng.integers(1 << 30))))
    return cases


RANDOM = _random_cases(24, 20270101)


@pytest.mark.parametrize("case", RANDOM, ids=[str(i) for i in range(len(RANDOM))])
def test_random(case):
    lens, H, Hkv, d, bs, window, cap, seed = case
    out, lse, ro, rl = run(lens, H, Hkv, d, bs, window, cap, seed=seed)
    check(out, ro, lse, rl, str(case))


def _inputs(lens, H, Hkv, d, bs, seed=0):
    Ts, Ss, cq, ck, q, k, v = varlen_inputs(0, 0, 0, H, Hkv, d, 1.0, seed, seq_lens=lens)
    kb, vb, table = paged(Ts, Ss, ck, k, v, bs)
    return (q.cuda(), kb, vb, cq.cuda(), table, torch.tensor(Ss, dtype=torch.int32).cuda(),
            max(Ts)), (q, k, v, cq, ck)


def test_rows_behind_the_last_sequence_stay():
    args, host = _inputs([(3, 50), (2, 9)], 4, 2, 128, 16)
    q = torch.cat([args[0], torch.full((4, 4, 128), float("nan"), dtype=torch.bfloat16,
                                       device="cuda")])
    out = torch.full_like(q, 7.0)
    lse = torch.full((4, 9), 7.0, device="cuda")
    g2.extend_paged(q, *args[1:], query_scale=0.1, out=out, lse=lse)
    ro, rl = oracle.varlen(*host, query_scale=0.1)
    check(out[:5], ro, lse[:, :5], rl, "padded")
    assert (out[5:] == 7.0).all() and (lse[:, 5:] == 7.0).all()


def test_rows_without_keys():
    """More queries than keys (T_s > L_s): the first ones see nothing."""
    args, host = _inputs([(5, 5), (1, 300)], 4, 2, 64, 16)
    lens = torch.tensor([3, 300], dtype=torch.int32).cuda()
    for cap in (50.0, 0.0):
        out, lse = g2.extend_paged(*args[:5], lens, 5, query_scale=0.1, softcap=cap)
        assert torch.count_nonzero(out[:2]) == 0 and (lse[:, :2] == float("-inf")).all()
        q, k, v, cq, ck = host
        ro, rl = oracle.attn(q[None, 2:5], k[None, :3], v[None, :3], query_scale=0.1, softcap=cap)
        check(out[2:5], ro[0], lse[:, 2:5], rl[0], "rows with keys")
    # a sequence without any key
    out, lse = g2.extend_paged(*args[:5], lens * 0, 5, query_scale=0.1)
    assert torch.count_nonzero(out) == 0 and (lse == float("-inf")).all()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 9])
def test_largest_windows(window):
    """A window past every position changes nothing, also where the first
    queries sit before the first key and their position less the window wraps round."""
    args, _ = _inputs([(12, 12), (3, 300)], 4, 2, 64, 8)
    lens = torch.tensor([2, 300], dtype=torch.int32).cuda()
    for cap in (50.0, 0.0):
        out, lse = g2.extend_paged(*args[:5], lens, 12, query_scale=0.1, softcap=cap, window=window)
        ro, rl = g2.extend_paged(*args[:5], lens, 12, query_scale=0.1, softcap=cap)
        assert torch.isfinite(rl[:, 10:]).all() and (rl[:, :10] == float("-inf")).all()
        assert torch.equal(out, ro) and torch.equal(lse, rl)


@pytest.mark.parametrize("bs", [4, 8, 16, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_pages_seen_in_part(bs, d):
    """What is seen starts and ends inside pages, one and the same among them,
    and ends at their borders: whole, partly seen and unseen pages side by side."""
    lens = [(3, 70), (1, 64), (2, 129), (1, 7), (4, 260), (2, 384), (20, 140)]
    for window, cap in ((0, 50.0), (5, 50.0), (70, 0.0)):
        out, lse, ro, rl = run(lens, 4, 2, d, bs, window, cap, seed=bs + d)
        check(out, ro, lse, rl, f"pages of {bs}, d {d}, window {window}")


def test_malformed_tables_stay_in_bounds():
    """Entries outside the cache, lengths past the table, offsets past the
    tensors: undefined results, but finite ones, as every row read is a row of
    the cache (all finite here)."""
    n, H, Hkv, d, bs = 3, 4, 2, 128, 16
    q = torch.randn(12, H, d, device="cuda").bfloat16()
    kb = torch.randn(5, bs, Hkv, d, device="cuda").bfloat16()
    table = torch.tensor([[7, -3, 1 << 30], [0, 1, 2], [4, 4, 4]], dtype=torch.int32).cuda()
    lens = torch.tensor([1 << 30, -5, 40], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 4, 9, 100], dtype=torch.int32).cuda()
    out, lse = g2.extend_paged(q, kb, kb, cu, table, lens, 8, query_scale=0.1)
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK


def test_deterministic_and_streams_and_graphs():
    """Same bits every time: repeated, on two streams at once with workspaces
    of their own, and from captured graphs replayed on new inputs."""
    args, _ = _inputs([(5, 3000), (2, 64), (8, 777)], 8, 4, 256, 16)
    kw = dict(query_scale=1 / 16)
    want, wl = g2.extend_paged(*args, **kw)
    other, _ = _inputs([(1, 900), (7, 1500)], 8, 4, 256, 16, seed=3)
    want2, _ = g2.extend_paged(*other, **kw)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        ws1, ws2 = g2.extend_workspace(8, 256), g2.extend_workspace(8, 256)
        torch.cuda.synchronize()
        o1, l1 = g2.extend_paged(*args, workspace=ws1, stream=s1, **kw)
        o2, _ = g2.extend_paged(*other, workspace=ws2, stream=s2, **kw)
        torch.cuda.synchronize()
        assert torch.equal(o1, want) and torch.equal(l1, wl) and torch.equal(o2, want2)
    out, lse, ws = torch.empty_like(want), torch.empty_like(wl), g2.extend_workspace(8, 256)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2.extend_paged(*args, out=out, lse=lse, workspace=ws, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    args[0].copy_(args[0].flip(0))
    args[5].copy_(torch.tensor([2500, 60, 700], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, g2.extend_paged(*args, **kw)[0]) and not torch.equal(out, want)


def test_no_lse():
    args, _ = _inputs([(5, 300), (1, 64)], 4, 2, 128, 16)
    a, l = g2.extend_paged(*args, query_scale=0.1)
    b, none = g2.extend_paged(*args, query_scale=0.1, want_lse=False)
    assert none is None and torch.equal(a, b)


def test_far_rows_of_a_large_cache():
    """Rows past 2^31 elements of the cache, written by the append and read here."""
    H, Hkv, d, bs = 16, 8, 256, 64
    pages = (2 ** 31 // (Hkv * d * bs)) + 40
    L, T = 500, 4
    need = -(-L // bs)
    kb = torch.empty(pages, bs, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vb = torch.empty_like(kb)
    table = torch.tensor([[pages - 1 - 3 * i for i in range(need)]], dtype=torch.int32).cuda()
    plan = g2.rope_plan(d)
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(L, h, d, generator=g).bfloat16() for h in (H, Hkv, Hkv))
    cu = torch.tensor([0, L], dtype=torch.int32).cuda()
    lens = torch.tensor([L], dtype=torch.int32).cuda()
    qr = g2.rope_append_paged(q.cuda(), k.cuda(), v.cuda(), kb, vb, cu, table, lens, plan)
    pos = torch.arange(L, dtype=torch.int32).cuda()
    kr = g2.rope(q.cuda(), k.cuda(), pos, plan)[1].cpu()
    out, lse = g2.extend_paged(qr[-T:].contiguous(), kb, vb, torch.tensor([0, T], dtype=torch.int32)
                               .cuda(), table, lens, T, query_scale=1 / 16)
    ro, rl = oracle.attn(qr[-T:].cpu()[None], kr[None], v[None], q_offset=L - T,
                         query_scale=1 / 16)
    check(out, ro[0], lse, rl[0], "far rows")


def test_agrees_with_decode_and_prefill():
    """One token: the decode's operation; larger pages: the prefill's."""
    args, (q, k, v, cq, ck) = _inputs([(1, 700), (1, 129), (1, 3)], 8, 4, 128, 128)
    kb, vb = torch.nan_to_num(args[1]), torch.nan_to_num(args[2])
    out, lse = g2.extend_paged(args[0], kb, vb, *args[3:], query_scale=0.1)
    do, dl = g2.decode_paged(args[0], kb, vb, args[4], args[5], 700, query_scale=0.1)
    po, pl = g2.prefill_paged(args[0], kb, vb, args[3], args[4], args[5], 1, 700, query_scale=0.1)
    for o, l in ((do, dl.t()), (po, pl)):
        # each is within 5e-3 relative (and 1e-3 for the log-sum) of the exact one
        assert (out.float() - o.float()).norm() <= 1e-2 * o.float().norm()
        assert (lse - l).abs().max() <= 2e-3


def test_helper_checks():
    args, _ = _inputs([(2, 30)], 4, 2, 128, 16)
    q, kb, vb, cu, table, lens, T = args
    for bad in [lambda: g2.extend_paged(q.float(), kb, vb, cu, table, lens, T),
                lambda: g2.extend_paged(q, kb, vb[:-1], cu, table, lens, T),
                lambda: g2.extend_paged(q, kb, vb, cu.long(), table, lens, T),
                lambda: g2.extend_paged(q, kb, vb, cu[:1], table, lens, T),
                lambda: g2.extend_paged(q, kb, vb, cu, table[0], lens, T),
                lambda: g2.extend_paged(q, kb, vb, cu, table, lens, T, out=q[:1]),
                lambda: g2.extend_paged(q, kb, vb, cu, table, lens, T, lse=torch.empty(
                    2, 4, device="cuda")),
                lambda: g2.extend_paged(q.transpose(1, 2).contiguous().transpose(1, 2), kb, vb, cu,
                                        table, lens, T)]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(g2.G2AttnError):
        g2.extend_paged(q, kb, vb, cu, table, lens, T, workspace=torch.empty(16, dtype=torch.uint8,
                                                                            device="cuda"))


def test_results_for_another_stream_are_not_memory_still_in_use():
    """A block that the current stream freed, and that its queued work still
    writes, must not become the result of a call on another stream."""
    args, _ = _inputs([(5, 300), (2, 64)], 8, 4, 256, 16)
    plan = g2.rope_plan(256)
    pos = torch.arange(7, dtype=torch.int32).cuda()
    k = torch.randn(7, 4, 256).bfloat16().cuda()
    parents = torch.tensor([1, 0], dtype=torch.int32).cuda()
    refs = torch.zeros(args[1].shape[0], dtype=torch.int32).cuda()
    refs[args[4][args[4] >= 0].long()] = 1
    calls = [lambda st: g2.extend_paged(*args, query_scale=0.1, stream=st),
             lambda st: g2.rope(args[0], k, pos, plan, stream=st),
             lambda st: g2.pages_fork(args[4], args[5], counts.pop(), parents, 16, stream=st)]
    counts = [refs.clone(), refs.clone()]  # (a fork changes them)
    side = torch.cuda.Stream()
    for call in calls:
        want = [t.clone() for t in call(None)]
        held = [torch.empty_like(t) for t in want for _ in range(3)]
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        for t in held:
            t.fill_(7)
        del held, t
        got = call(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_workspaces_elsewhere_are_refused():
    args, _ = _inputs([(2, 30)], 4, 2, 128, 16)
    n = g2.g2attn_extend_workspace_size(8, 128)
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(n, 2, dtype=torch.uint8).cuda()[:, 0]):
        with pytest.raises(ValueError):
            g2.extend_paged(*args, workspace=ws)
    table = torch.full((2, 4), -1, dtype=torch.int32).cuda()
    zero = torch.zeros(8, dtype=torch.int32).cuda()
    with pytest.raises(ValueError):
        g2.pages_grow(table, zero[:2], zero, zero[:2], 16, workspace=torch.empty(4096))
