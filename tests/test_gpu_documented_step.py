"""The decode step over a paged cache that users are shown first, run as it stands
there: sequences that are refused rows, or share a page they were cut in."""
import os
import re

import numpy as np
import pytest
import torch

import global_soft_capped_b200 as g2
import oracle
from parity import check

pytestmark = pytest.mark.gpu

H, HKV, D, BS = 8, 4, 128, 16
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def documented_step():
    with open(README) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "pages_grow" in b)


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g2.load_library()
    yield
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class State:
    """A cache, its tables and what every sequence's rows should hold."""

    def __init__(self, n, cols, pages):
        self.table = torch.full((n, cols), -1, dtype=torch.int32, device="cuda")
        self.lens, self.refs = ints([0] * n), ints([0] * pages)
        self.k_blocks = torch.zeros(pages, BS, HKV, D, dtype=torch.bfloat16, device="cuda")
        self.v_blocks = torch.zeros_like(self.k_blocks)
        self.keys = [torch.empty(0, HKV, D, dtype=torch.bfloat16) for _ in range(n)]
        self.values = [k.clone() for k in self.keys]

    def step(self, seed, new_rows, accepted=None):
        """Runs the documented step; checks results and caches. Returns granted."""
        g = torch.Generator().manual_seed(seed)
        qkv = torch.randn(sum(new_rows), H + 2 * HKV, D, generator=g).bfloat16()
        x, before = qkv.cuda(), self.lens.tolist()
        env = dict(g2=g2, torch=torch, q=x[:, :H], k=x[:, H:H + HKV], v=x[:, H + HKV:],
                   table=self.table, lens=self.lens, refs=self.refs, k_blocks=self.k_blocks,
                   v_blocks=self.v_blocks, caches=[self.k_blocks, self.v_blocks],
                   new_rows=ints(new_rows), block_size=BS, max_T=max(new_rows),
                   accepted_lens=ints(accepted or [1 << 20] * len(new_rows)))
        env["cu_q"] = ints(np.concatenate([[0], np.cumsum(new_rows)]))
        exec(documented_step(), env)
        torch.cuda.synchronize()
        granted, plan = env["granted"].tolist(), env["plan"]
        at = row = 0
        for s, t in enumerate(new_rows):
            if granted[s] and t:
                pos = ints(np.arange(before[s], before[s] + t))
                kr = g2.rope(x[at:at + t, :H], x[at:at + t, H:H + HKV], pos, plan)
                self.keys[s] = torch.cat([self.keys[s], kr[1].cpu()])
                self.values[s] = torch.cat([self.values[s], qkv[at:at + t, H + HKV:]])
                ro, rl = oracle.attn(kr[0].cpu()[None], self.keys[s][None], self.values[s][None],
                                     q_offset=before[s], query_scale=D ** -0.5)
                check(env["out"][row:row + t], ro[0], env["lse"][:, row:row + t], rl[0], f"{s}")
                row += t
            at += t
            m = min(len(self.keys[s]), accepted[s] if accepted else 1 << 20)
            self.keys[s], self.values[s] = self.keys[s][:m], self.values[s][:m]
        assert env["out"].shape[0] == row
        self.holds()
        return granted

    def holds(self):
        table, lens = self.table.cpu().long(), self.lens.tolist()
        for s, (k, v) in enumerate(zip(self.keys, self.values)):
            assert lens[s] == len(k), s
            j = torch.arange(lens[s])
            rows = (table[s, j // BS], j % BS)
            assert torch.equal(self.k_blocks.cpu()[rows], k), f"keys of sequence {s}"
            assert torch.equal(self.v_blocks.cpu()[rows], v), f"values of sequence {s}"


def test_step_with_refused_sequences():
    """Pages run out for one sequence, another's table row is too short: both
    keep every row, the others go on."""
    st = State(4, 3, 8)
    assert st.step(1, [40, 20, 15, 0]) == [1, 1, 1, 1]     # 3 + 2 + 1 pages of 8
    # the first has no column left, the second's rows fit the pages it has, the third
    # takes the last two pages, and the fourth finds none
    assert st.step(2, [9, 12, 20, 5]) == [0, 1, 1, 0]
    assert st.step(3, [1, 0, 1, 1]) == [1, 1, 1, 0]
    assert st.step(4, [3, 3, 2, 0], accepted=[42, 33, 38, 0]) == [1, 0, 1, 1]


def test_step_after_a_cut_inside_a_shared_page():
    """Beams that share a page and were cut inside it go their own ways."""
    st = State(3, 4, 12)
    assert st.step(1, [30, 5, 1]) == [1, 1, 1]
    caches = [st.k_blocks, st.v_blocks]
    st.table, st.lens, src, dst, granted = g2.pages_fork(st.table, st.lens, st.refs,
                                                         ints([0, 0, 0]), BS)
    g2.pages_copy(caches, src, dst)
    st.keys, st.values = [st.keys[0]] * 3, [st.values[0]] * 3
    g2.pages_truncate(st.table, st.lens, st.refs, ints([10, 12, 30]), BS)
    st.keys = [k[:m] for k, m in zip(st.keys, (10, 12, 30))]
    st.values = [v[:m] for v, m in zip(st.values, (10, 12, 30))]
    st.holds()
    assert st.step(2, [4, 7, 1]) == [1, 1, 1]
    assert st.step(3, [1, 1, 1]) == [1, 1, 1]
