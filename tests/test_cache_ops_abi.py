"""Host-side behaviour of the rotary, append, chunk-attention and page calls:
arguments refused before any launch, workspace sizes, frequency tables, the
tensor helpers' checks. No GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import global_soft_capped_b200 as g2
from global_soft_capped_b200 import build as g2build

FAKE = ctypes.c_void_p(1 << 20)   # aligned, never dereferenced: calls fail before launch
ODD8 = ctypes.c_void_p((1 << 20) + 8)
ODD2 = ctypes.c_void_p((1 << 20) + 2)
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = (
    g2.G2ATTN_ERR_INVALID_ARG, g2.G2ATTN_ERR_UNSUPPORTED, g2.G2ATTN_ERR_MISALIGNED,
    g2.G2ATTN_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def lib():
    g2build.build()
    return g2.load_library()


def call(fn, base, kw):
    assert set(kw) <= set(base), set(kw) - set(base)
    return fn(*{**base, **kw}.values())


ROPE = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, positions=FAKE, freqs=FAKE, num_tokens=4, H=8,
            Hkv=4, d=128, rotary_dim=128, interleaved=0, mscale=1.0, inverse=0, q_stride=1024,
            k_stride=512, q_out_stride=1024, k_out_stride=512, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k_out=None), INVALID), (dict(positions=None), INVALID),
    (dict(freqs=None), INVALID), (dict(num_tokens=0), INVALID), (dict(H=0), INVALID),
    (dict(Hkv=-1), INVALID), (dict(rotary_dim=0), INVALID), (dict(rotary_dim=256), INVALID),
    (dict(mscale=float("nan")), INVALID), (dict(mscale=float("inf")), INVALID),
    (dict(q_stride=1000), INVALID), (dict(k_stride=8), INVALID), (dict(k_out_stride=8), INVALID),
    (dict(q_stride=2048), INVALID),                     # in place with another stride
    (dict(d=96, rotary_dim=96), UNSUPPORTED), (dict(rotary_dim=24), UNSUPPORTED),
    (dict(q=ODD8), MISALIGNED), (dict(freqs=ctypes.c_void_p((1 << 20) + 4)), MISALIGNED),
    (dict(positions=ODD2), MISALIGNED), (dict(q_stride=1028, q_out_stride=1028), MISALIGNED),
    (dict(k_out=ODD8), MISALIGNED),
])
def test_rope_refuses(kw, status):
    assert call(g2.g2attn_rope, ROPE, kw) == status


SEQ = dict(freqs=FAKE, num_seqs=2, total_q=4)
HEAD = dict(H=8, Hkv=4, d=128, rotary_dim=128, interleaved=0, mscale=1.0, q_stride=1024,
            k_stride=512, v_stride=512, stream=None)
TENSORS = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, k_cache=FAKE, v_cache=FAKE, cu_seqlens_q=FAKE)
LINEAR = {**TENSORS, "cu_seqlens_k": FAKE, **SEQ, "total_k": 100, **HEAD}
RING = {**TENSORS, "seq_lens": FAKE, **SEQ, "ring_size": 64, **HEAD}
PAGED = {**TENSORS, "block_table": FAKE, "seq_lens": FAKE, **SEQ, "num_blocks": 10,
         "block_size": 16, "max_blocks_per_seq": 4, **HEAD}
APPENDS = [(g2.g2attn_rope_append, LINEAR), (g2.g2attn_rope_append_ring, RING),
           (g2.g2attn_rope_append_paged, PAGED)]


@pytest.mark.parametrize("fn,base", APPENDS, ids=["linear", "ring", "paged"])
@pytest.mark.parametrize("kw,status", [
    (dict(v=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(num_seqs=0), INVALID), (dict(total_q=0), INVALID), (dict(freqs=None), INVALID),
    (dict(cu_seqlens_q=None), INVALID),                 # 4 tokens of 2 sequences, one each
    (dict(v_stride=8), INVALID), (dict(q_stride=4096), INVALID),  # in place, not packed
    (dict(d=32, rotary_dim=32), UNSUPPORTED), (dict(rotary_dim=8), UNSUPPORTED),
    (dict(v=ODD8), MISALIGNED), (dict(v_cache=ODD8), MISALIGNED), (dict(cu_seqlens_q=ODD2), MISALIGNED),
    (dict(v_stride=516), MISALIGNED),
])
def test_appends_refuse(fn, base, kw, status):
    assert call(fn, base, kw) == status


@pytest.mark.parametrize("fn,base,kw,status", [
    (g2.g2attn_rope_append, LINEAR, dict(cu_seqlens_k=None), INVALID),
    (g2.g2attn_rope_append, LINEAR, dict(total_k=0), INVALID),
    (g2.g2attn_rope_append, LINEAR, dict(cu_seqlens_k=ODD2), MISALIGNED),
    (g2.g2attn_rope_append_ring, RING, dict(ring_size=48), INVALID),
    (g2.g2attn_rope_append_ring, RING, dict(seq_lens=None), INVALID),
    (g2.g2attn_rope_append_ring, RING, dict(ring_size=1 << 30), UNSUPPORTED),
    (g2.g2attn_rope_append_ring, RING, dict(seq_lens=ODD2), MISALIGNED),
    (g2.g2attn_rope_append_paged, PAGED, dict(block_size=24), INVALID),
    (g2.g2attn_rope_append_paged, PAGED, dict(block_table=None), INVALID),
    (g2.g2attn_rope_append_paged, PAGED, dict(num_blocks=0), INVALID),
    (g2.g2attn_rope_append_paged, PAGED, dict(max_blocks_per_seq=0), INVALID),
    (g2.g2attn_rope_append_paged, PAGED, dict(num_blocks=1 << 28), UNSUPPORTED),
    (g2.g2attn_rope_append_paged, PAGED, dict(block_table=ODD2), MISALIGNED),
])
def test_append_layouts_refuse(fn, base, kw, status):
    assert call(fn, base, kw) == status


EXTEND = dict(q=FAKE, k_blocks=FAKE, v_blocks=FAKE, out=FAKE, lse=None, cu_seqlens_q=FAKE,
              block_table=FAKE, seq_lens=FAKE, num_seqs=2, total_q=8, num_blocks=10, block_size=16,
              max_blocks_per_seq=4, max_T=4, H=8, Hkv=4, d=128, query_scale=0.1, softcap=50.0,
              window=0, workspace=FAKE, workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(cu_seqlens_q=None), INVALID), (dict(block_table=None), INVALID),
    (dict(seq_lens=None), INVALID), (dict(num_seqs=0), INVALID), (dict(total_q=0), INVALID),
    (dict(max_T=0), INVALID), (dict(block_size=12), INVALID), (dict(block_size=0), INVALID),
    (dict(num_blocks=0), INVALID), (dict(window=-1), INVALID), (dict(softcap=-1.0), INVALID),
    (dict(query_scale=float("inf")), INVALID),
    (dict(H=4), UNSUPPORTED), (dict(d=80), UNSUPPORTED), (dict(num_seqs=1025), UNSUPPORTED),
    (dict(num_blocks=1 << 28), UNSUPPORTED), (dict(max_blocks_per_seq=1 << 28), UNSUPPORTED),
    (dict(max_blocks_per_seq=(1 << 27) - 1), UNSUPPORTED),  # a tile's end would pass 32 bits
    (dict(out=ODD8), MISALIGNED), (dict(lse=ODD8), MISALIGNED), (dict(seq_lens=ODD2), MISALIGNED),
    (dict(workspace=ODD8), MISALIGNED),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=64), WORKSPACE),
])
def test_extend_refuses(kw, status):
    assert call(g2.g2attn_extend_paged, EXTEND, kw) == status


def test_extend_workspace_size():
    sizes = [g2.g2attn_extend_workspace_size(t, 256) for t in (1, 8, 9, 16, 17, 1000)]
    assert sizes[0] == sizes[1] < sizes[2] == sizes[3] < sizes[4] == sizes[5]
    assert g2.g2attn_extend_workspace_size(0, 256) == 0
    assert g2.g2attn_extend_workspace_size(1, 96) == 0
    need = g2.g2attn_extend_workspace_size(4, 128)
    assert call(g2.g2attn_extend_paged, EXTEND, dict(workspace_bytes=need - 1)) == WORKSPACE


STATE = dict(num_seqs=4, num_blocks=100, block_size=16, max_blocks_per_seq=8)
WS = dict(workspace=FAKE, workspace_bytes=1 << 20, stream=None)
GROW = {**dict(block_table=FAKE, seq_lens=FAKE, ref_counts=FAKE, add=FAKE, granted=FAKE,
               copy_src=FAKE, copy_dst=FAKE), **STATE, **WS}
CUT = {**dict(block_table=FAKE, seq_lens=FAKE, ref_counts=FAKE, keep=FAKE), **STATE, "stream": None}
OTHER = ctypes.c_void_p(1 << 21)
FORK = {**dict(block_table=FAKE, seq_lens=FAKE, parents=FAKE, new_table=OTHER, new_lens=OTHER,
               ref_counts=FAKE, copy_src=FAKE, copy_dst=FAKE, granted=FAKE), **STATE, **WS}
COMPACT = {**dict(block_table=FAKE, ref_counts=FAKE, copy_src=FAKE, copy_dst=FAKE, num_live=FAKE,
                  num_seqs=4, num_blocks=100, max_blocks_per_seq=8), **WS}


@pytest.mark.parametrize("fn,base", [(g2.g2attn_pages_grow, GROW), (g2.g2attn_pages_truncate, CUT),
                                     (g2.g2attn_pages_fork, FORK),
                                     (g2.g2attn_pages_compact, COMPACT)],
                         ids=["grow", "truncate", "fork", "compact"])
@pytest.mark.parametrize("kw,status", [
    (dict(block_table=None), INVALID), (dict(ref_counts=None), INVALID), (dict(num_seqs=0), INVALID),
    (dict(num_blocks=0), INVALID), (dict(max_blocks_per_seq=0), INVALID),
    (dict(block_size=10), INVALID), (dict(block_size=1 << 26), UNSUPPORTED),
    (dict(ref_counts=ODD8), MISALIGNED), (dict(block_table=ODD2), MISALIGNED),
    (dict(seq_lens=None), INVALID), (dict(seq_lens=ODD2), MISALIGNED),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=16), WORKSPACE),
    (dict(workspace=ODD8), MISALIGNED), (dict(granted=None), INVALID), (dict(add=None), INVALID),
    (dict(keep=None), INVALID), (dict(parents=None), INVALID), (dict(num_live=None), INVALID),
    (dict(copy_src=None), INVALID), (dict(new_table=FAKE), INVALID), (dict(new_lens=FAKE), INVALID),
])
def test_pages_refuse(fn, base, kw, status):
    if set(kw) <= set(base):
        assert call(fn, base, kw) == status


def test_pages_copy_refuses():
    ptrs = (ctypes.c_void_p * 2)(1 << 20, 1 << 21)
    base = dict(caches=ptrs, num_caches=2, src=FAKE, dst=FAKE, num_pairs=3, num_blocks=10,
                page_bytes=4096, stream=None)
    for kw, status in [(dict(caches=None), INVALID), (dict(src=None), INVALID),
                       (dict(num_pairs=0), INVALID), (dict(num_caches=0), INVALID),
                       (dict(page_bytes=0), INVALID), (dict(page_bytes=4100), UNSUPPORTED),
                       (dict(num_pairs=1 << 30, page_bytes=1 << 20), UNSUPPORTED),
                       (dict(dst=ODD2), MISALIGNED),
                       (dict(caches=(ctypes.c_void_p * 2)(1 << 20, (1 << 20) + 8)), MISALIGNED),
                       (dict(caches=(ctypes.c_void_p * 2)(1 << 20, None)), INVALID)]:
        assert call(g2.g2attn_pages_copy, base, kw) == status, kw


def test_new_status_has_a_name():
    assert "row" in g2.g2attn_status_string(g2.G2ATTN_ERR_CACHE_ROW)


def test_frequencies():
    inv, m = g2.rope_frequencies(64)
    assert m == 1.0 and len(inv) == 32 and inv[0] == 1.0
    assert inv[16] == pytest.approx(10000.0 ** -0.5, rel=1e-15)
    lin, _ = g2.rope_frequencies(64, scaling="linear", factor=4.0)
    assert lin == [w / 4.0 for w in inv]
    ntk, _ = g2.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(inv[-1] / 4.0, rel=1e-12)
    yarn, m = g2.rope_frequencies(64, scaling="yarn", factor=4.0, trained_len=4096)
    assert m == pytest.approx(0.1 * math.log(4.0) + 1.0)
    turns = [4096 * w / (2 * math.pi) for w in inv]
    for w, y, t in zip(inv, yarn, turns):
        assert w / 4.0 * (1 - 1e-12) <= y <= w
        if t > 45.0:
            assert y == w
        if t < 0.7:
            assert y == pytest.approx(w / 4.0, rel=1e-12)
    for bad in (dict(rotary_dim=63), dict(rotary_dim=0), dict(rotary_dim=64, scaling="cubic"),
                dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, scaling="linear", factor=0.5)):
        with pytest.raises(ValueError):
            g2.rope_frequencies(**bad)


def test_plan_table_holds_turns():
    plan = g2.rope_plan(128, device="cpu")
    inv, _ = g2.rope_frequencies(128)
    for bits, w in zip(plan.freqs.tolist(), inv):
        assert (bits % 2 ** 64) / 2.0 ** 64 == pytest.approx(w / (2 * math.pi), rel=1e-15)
    # the phase of a far position, whole turns dropped, against 64-bit arithmetic
    p = 2 ** 31 - 1
    w = inv[40]
    got = (p * (plan.freqs[40].item() % 2 ** 64)) % 2 ** 64 / 2.0 ** 64
    want = math.fmod(p * w / (2 * math.pi), 1.0)
    assert abs(got - want) < 2.0 ** -33
    # more than half a turn per position (and a negative frequency) wrap
    plan = g2.rope_plan(4, device="cpu", frequencies=[4.0, -1.0])
    assert (plan.freqs[0].item() % 2 ** 64) / 2.0 ** 64 == pytest.approx(4.0 / (2 * math.pi))
    assert plan.freqs[1].item() / 2.0 ** 64 == pytest.approx(-1.0 / (2 * math.pi))
    with pytest.raises(ValueError):
        g2.rope_plan(4, device="cpu", frequencies=[1.0])
    with pytest.raises(ValueError):
        g2.rope_plan(4, device="cpu", frequencies=[1.0, 2.0], base=100.0)


def test_rotation_formula_against_differences():
    """The transposed rotation is the gradient: numeric differences of the
    formula that the GPU tests compare with."""
    from rope_model import turn
    rng = np.random.default_rng(3)
    inv, _ = g2.rope_frequencies(16)
    pos = np.array([0, 5, 100000])
    for inter in (False, True):
        x = rng.standard_normal((3, 2, 32))
        dy = rng.standard_normal((3, 2, 32))
        dx = turn(dy, pos, inv, 16, inter, 1.3, -1)
        for at in [(0, 0, 0), (1, 1, 9), (2, 0, 15), (2, 1, 31), (1, 0, 8)]:
            h = 1e-4
            up, down = x.copy(), x.copy()
            up[at] += h
            down[at] -= h
            diff = (dy * (turn(up, pos, inv, 16, inter, 1.3) -
                          turn(down, pos, inv, 16, inter, 1.3))).sum() / (2 * h)
            assert diff == pytest.approx(dx[at], abs=1e-8)


def test_helpers_refuse_host_tensors():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    plan = g2.rope_plan(64, device="cpu")
    with pytest.raises(ValueError):
        g2.rope(x, x, torch.zeros(2, dtype=torch.int32), plan)
    with pytest.raises(ValueError):
        g2.extend_paged(x, x, x, None, None, None, 1)
    with pytest.raises(ValueError):
        g2.pages_copy([x], torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        g2.pages_truncate(torch.zeros(2, 2, dtype=torch.int32), None,
                          torch.zeros(2, dtype=torch.int32), None, 16)


def test_extend_refuses_more_tiles_than_it_can_number():
    """A million tokens over as many keys in units of 8 positions (max_T 4) would be
    4 * 131,073 * 8,200 tiles; in units of 32 they fit, and the next check speaks."""
    big = dict(total_q=1 << 20, num_seqs=1, max_blocks_per_seq=1 << 16, workspace=None)
    assert call(g2.g2attn_extend_paged, EXTEND, big) == UNSUPPORTED
    assert call(g2.g2attn_extend_paged, EXTEND, {**big, "max_T": 1 << 20}) == WORKSPACE
    assert call(g2.g2attn_extend_paged, EXTEND, {**big, "window": 4096}) == WORKSPACE
    wide = dict(total_q=8192, num_seqs=1024, Hkv=16, H=32, max_blocks_per_seq=1 << 20)
    assert call(g2.g2attn_extend_paged, EXTEND, {**wide, "workspace": None}) == UNSUPPORTED
    wide["max_blocks_per_seq"] = 500_000  # 8,000,000 keys
    assert call(g2.g2attn_extend_paged, EXTEND, {**wide, "workspace": None}) == WORKSPACE
