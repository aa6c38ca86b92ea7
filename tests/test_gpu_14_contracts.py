"""GPU tests of what the rotary, tree, weight and eviction calls promise beside their formulas: which outputs may be
which inputs, whose memory a call may touch when, and what a workspace may hold."""
import os
import sys

import pytest
import torch

import masked_attention_paged_gb300 as lib

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_12_evict import _evict_inputs  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("B,Hkv,longest", [(40, 8, 3000), (12, 8, 20000), (4, 8, 65000)])
def test_evict_updates_the_lengths_in_place(B, Hkv, longest):
    """new_lens is ctx_lens: every head and every CTA of a cluster has to select by the old lengths, also those that
    begin after others of the sequence are done (several waves of CTAs, clusters of one, four and eight)."""
    keep = 96
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(keep // 2, longest, (B,), generator=g).tolist()
    lens[0], lens[1], lens[2] = -1, keep, longest
    kc, vc, acc, bt, lens, dt = _evict_inputs(lens, Hkv, 64, keep, seed=B)
    ws = lib.Workspace(256)

    def call(into):
        n = lens.clone()
        k, v, a = kc.clone(), vc.clone(), acc.clone()
        nl, kept = lib.kv_evict(k, v, a, bt, n, dt, keep, sink=3, recent=20, new_lens=n if into else None, workspace=ws)
        assert not into or nl is n
        assert into or torch.equal(n, lens)
        return nl, kept, k, v, a

    want = call(False)
    assert torch.equal(want[0], torch.where(lens < 0, lens, lens.clamp(max=keep)))
    for _ in range(5):
        for x, y in zip(call(True), want):
            assert torch.equal(x, y)
    assert ws.status() == 0
