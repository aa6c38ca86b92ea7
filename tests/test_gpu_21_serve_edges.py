"""Draft verification, pools and the e4m3 cache at the ends of what their calls take: nothing at
all, rows far past 32 bits, calls at the same time and captured in two graphs."""
import numpy as np
import pytest
import torch

import masked_attention_paged_gb300 as lib
from _serve_ref import verify
from test_gpu_15_verify import _equal, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("given", [False, True])
def test_calls_with_nothing_to_do(given):
    """No sequences, no queries, no children, no tensors: results of that size, and no memory touched."""
    ws = lib.Workspace(1 << 24) if given else None
    p = torch.zeros((0, 4, 100), device=DEV)
    path, n, nxt = lib.draft_verify(p, _i(0, 4), _i(0, 4), torch.zeros((0, 4), device=DEV), workspace=ws)
    assert path.shape == (0, 4) and n.shape == (0,) and nxt.shape == (0,)
    refs, table = torch.ones(5, dtype=torch.int32, device=DEV), torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    cache = torch.arange(10, device=DEV, dtype=torch.float32).reshape(5, 2)
    lib.kv_free(refs, table[:0], _i(0), workspace=ws)
    lib.kv_reserve(refs, table[:0], _i(0), _i(0), workspace=ws)
    lib.kv_fork([cache], refs, table, _i(2) - 1, _i(0), _i(0, 3), _i(0), workspace=ws)
    child, sizes = _i(2, 3), _i(2)
    lib.kv_fork([], refs, table[:0], _i(0), _i(2) - 1, child, sizes, workspace=ws)
    assert (child == -1).all() and (sizes == -1).all()
    refs[1:3] = 0
    table[0] = torch.tensor([4, 0, 3], device=DEV)
    assert lib.kv_compact([], refs, table, workspace=ws).item() == 3
    assert table[0].tolist() == [2, 0, 1] and refs.tolist() == [1, 1, 1, 0, 0]
    refs.zero_()
    assert lib.kv_compact([cache], refs, table[1:], workspace=ws).item() == 0
    assert cache.reshape(-1).tolist() == list(range(10))
    codes = [torch.full((5, 2, 16, 64), 0x38, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)]
    scales = [torch.ones((5, 2), device=DEV) for _ in range(2)]
    for B, T in ((0, 1), (0, 40), (2, 0)):
        new = torch.zeros((B, 2, T, 64), device=DEV, dtype=torch.bfloat16)
        q = torch.zeros((B, 4, T, 64), device=DEV, dtype=torch.bfloat16)
        lib.kv_append_f8(*codes, *scales, table[:B], _i(B), new, new, workspace=ws)
        out, lse = lib.paged_attn_f8(q, *codes, *scales, table[:B], _i(B), return_lse=True, workspace=ws)
        assert out.shape == q.shape and lse.shape == q.shape[:3]
    assert all((c.view(torch.uint8) == 0x38).all() for c in codes) and all((s == 1).all() for s in scales)
    torch.cuda.synchronize()


@pytest.mark.parametrize("mode", ["distinct", "certain"])
def test_rows_whose_offsets_pass_32_bits(mode):
    """Probabilities of 4.8 GB, almost all of them zero; the reference sees the others, in order."""
    B, T, V = 3, 2, 400_000_003
    rng = np.random.default_rng(7)
    at = np.sort(rng.choice(V, 40, replace=False))
    at[0], at[-1] = 0, V - 1
    p = (rng.integers(1, 16, (B, T, 40)) / 256.0).astype(np.float32)  # exact in bf16
    q = (rng.integers(1, 16, (B, T, 40)) / 256.0).astype(np.float32)
    tok = rng.integers(0, 40, (B, T)).astype(np.int32)
    q[0, 0, tok[0, 1]] = 1.0  # refused with u = 0.999
    par = np.tile(np.array([-1, 0], np.int32), (B, 1))
    cols = torch.from_numpy(at).to(DEV)

    def wide(x):
        big = torch.zeros((B, T, V), device=DEV, dtype=torch.bfloat16)
        big[:, :, cols] = torch.from_numpy(x).to(DEV, torch.bfloat16)
        return big

    P, Q = wide(p), None if mode == "certain" else wide(q)
    taken = 0
    for seed in range(8):
        u = np.random.default_rng(seed).random((B, T)).astype(np.float32)
        u[:, 1] = [0.999, 0.01, 0.5]
        got = lib.draft_verify(P, torch.from_numpy(at[tok].astype(np.int32)).to(DEV), torch.from_numpy(par).to(DEV),
                               torch.from_numpy(u).to(DEV), draft_probs=Q)
        want = verify(p, None if Q is None else q, tok, par, u, False)
        taken += int((want[1] == 2).sum())
        want[2] = at[want[2]].astype(np.int32)
        _equal([x.cpu().numpy() for x in got], want)
    assert 0 < taken < 8 * B


def test_verification_at_the_same_time_and_in_two_graphs():
    """Two streams with a workspace each, and two graphs that share one, replayed in turns."""
    sets = []
    for seed in (1, 2):
        p, q, tok, par, u = _inputs(6, 9, 33000, seed=seed)
        args = [torch.from_numpy(x).to(DEV) for x in (p, tok, par, u, q)]
        sets.append((args, verify(p, q, tok, par, u, False)))
    call = lambda a, ws, **kw: lib.draft_verify(*a[:4], draft_probs=a[4], workspace=ws, **kw)  # noqa: E731
    streams, own = [torch.cuda.Stream() for _ in range(2)], [lib.Workspace(256) for _ in range(2)]
    torch.cuda.synchronize()
    got = [[call(a, own[i], stream=streams[i]) for i, (a, _) in enumerate(sets)] for _ in range(30)]
    torch.cuda.synchronize()
    for pair in got:
        for x, (_, want) in zip(pair, sets):
            _equal([y.cpu().numpy() for y in x], want)
    ws, graphs = lib.Workspace(256), []
    for a, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(a, ws)
        graphs.append((g, out))
    for i in (0, 1, 1, 0, 1):
        for y in graphs[i][1]:
            y.fill_(-7)
        graphs[i][0].replay()
        torch.cuda.synchronize()
        _equal([y.cpu().numpy() for y in graphs[i][1]], sets[i][1])
    assert ws.status() == 0
