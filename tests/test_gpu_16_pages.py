"""Pools of blocks with owner counts on the GPU, against books kept in Python: all bit for bit."""
import numpy as np
import pytest
import torch

import masked_attention_paged_gb300 as lib
from _serve_ref import BS, Pool

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _ints(x):
    return torch.tensor(np.asarray(x, np.int32).copy(), device=DEV)


def _pool(N, lens, width, rng, shapes=(((2, BS, 8), torch.bfloat16),)):
    """A shuffled pool with a sequence per length (-1: idle), and cache tensors of random bytes."""
    order, at = rng.permutation(N), 0
    table = np.full((len(lens), width), -1, np.int32)
    refs = np.zeros(N, np.int32)
    for b, n in enumerate(lens):
        k = -(-max(n, 0) // BS)
        table[b, :k] = order[at:at + k]
        refs[order[at:at + k]] = 1
        at += k
    caches = []
    for shape, dtype in shapes:
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        caches.append(torch.from_numpy(rng.integers(0, 256, (N, n), np.uint8)).to(DEV).view(dtype).view(N, *shape))
    return table, refs, caches


def _bytes(c):
    return c.reshape(c.shape[0], -1).view(torch.uint8).cpu().numpy()


def _same(ref, refs, caches):
    assert refs.cpu().tolist() == ref.refs
    for a, b in zip(caches, ref.caches):
        assert np.array_equal(_bytes(a), b)


SHAPES = [((2, BS, 64), torch.bfloat16), ((2, BS, 64), torch.float8_e4m3fn), ((3,), torch.float32),
          ((5,), torch.uint8), ((2, BS), torch.float32), ((8, BS, 128), torch.bfloat16)]


@pytest.mark.parametrize("N,lens,src,width,cw", [
    (40, [33, 16, 0, -1, 100], [0, 0, 1, 4, 2, 3, -1, 4], 8, 9),
    (9, [1], [0, 0, 0], 1, 1),
    (12, [17, 31], [1, 0, 1, 0, 1, 0, 1, 0, 1, 0], 2, 3),  # the free blocks run out
    (600, [160, 161, 4000], [2] * 40 + [0, 1] * 5, 260, 251),
])
def test_fork(N, lens, src, width, cw):
    rng = np.random.default_rng(N)
    table, refs, caches = _pool(N, lens, width, rng, SHAPES)
    ref = Pool(refs, [_bytes(c) for c in caches])
    rows, sizes = ref.fork(table.tolist(), lens, src, cw)
    g_refs, g_table, ws = _ints(refs), _ints(table), lib.Workspace(lib.kv_pool_workspace_size(N, len(src)))
    child, cl = _ints(np.full((len(src), cw), 77)), _ints([5] * len(src))
    lib.kv_fork(caches, g_refs, g_table, _ints(lens), _ints(src), child, cl, workspace=ws)
    assert child.cpu().tolist() == rows and cl.cpu().tolist() == sizes
    assert np.array_equal(g_table.cpu().numpy(), table)
    _same(ref, g_refs, caches)
    assert ws.status() == (5 if ref.flag else 0)
    # given back, the pool is as it was
    lib.kv_free(g_refs, child, cl, workspace=ws)
    assert g_refs.cpu().tolist() == refs.tolist() and (child == -1).all() and (cl == -1).all()


def test_fork_refuses_what_does_not_fit():
    """Each bad child is idle and reported; the others are served."""
    rng = np.random.default_rng(1)
    table, refs, caches = _pool(30, [40, 35, 50, 20], 4, rng)
    lens = [40, 35, 200, 20]  # sequence 2 claims more than its row holds
    table[1, 2] = 30  # its partial block lies outside the pool
    table[0, 0] = -5  # a full block of sequence 0 does
    src = [1, 2, 4, 3, 0]
    ref = Pool(refs, [_bytes(c) for c in caches])
    rows, sizes = ref.fork(table.tolist(), lens, src, 4)
    g_refs, child, cl, ws = _ints(refs), _ints(np.zeros((5, 4))), _ints([0] * 5), lib.Workspace(1 << 16)
    lib.kv_fork(caches, g_refs, _ints(table), _ints(lens), _ints(src), child, cl, workspace=ws)
    assert child.cpu().tolist() == rows and cl.cpu().tolist() == sizes and sizes == [-1, -1, -1, 20, 40]
    _same(ref, g_refs, caches)
    assert ws.status() == 5
    ws.reset()
    narrow, cl = _ints(np.zeros((1, 2))), _ints([0])
    lib.kv_fork(caches, _ints(refs), _ints(table), _ints(lens), _ints([0]), narrow, cl, workspace=ws)
    assert cl.item() == -1 and (narrow == -1).all() and ws.status() == 5


@pytest.mark.parametrize("N,lens,new,width,have", [
    (50, [0, 1, 15, 16, 17, -1, 30], [1, 15, 1, 1, 16, 5, 0], 4, 0),
    (50, [0, 33, 40], [48, 16, -3], 4, 1),
    (4, [3, 5, 7], [40, 30, 30], 3, 0),       # runs out in the middle of a row
    (40000, [16 * 5] * 70, [700] * 70, 64, 0),
    (2000, [7], [16000], 1024, 0),
    (60, [10], [1000], 3, 0),                 # past the table
])
def test_reserve(N, lens, new, width, have):
    rng = np.random.default_rng(N + width)
    table, refs, _ = _pool(N, [n + BS * have if n >= 0 else n for n in lens], width, rng)
    ref, want = Pool(refs), table.tolist()
    ref.reserve(want, lens, new)
    g_refs, g_table, ws = _ints(refs), _ints(table), lib.Workspace(lib.kv_pool_workspace_size(N, len(lens)))
    lib.kv_reserve(g_refs, g_table, _ints(lens), _ints(new), workspace=ws)
    assert g_table.cpu().tolist() == want
    assert g_refs.cpu().tolist() == ref.refs
    assert ws.status() == (5 if ref.flag else 0)


def test_reserve_finds_the_last_free_blocks_of_a_large_pool():
    N = (1 << 20) - 3
    refs = torch.ones(N, dtype=torch.int32, device=DEV)
    refs[[5, 16384, N - 1]] = 0
    table = _ints(np.full((2, 2), -1))
    ws = lib.Workspace(lib.kv_pool_workspace_size(N, 2))
    lib.kv_reserve(refs, table, _ints([0, 3]), _ints([32, 1]), workspace=ws)
    assert table.cpu().tolist() == [[5, 16384], [N - 1, -1]] and ws.status() == 0 and (refs == 1).all()


def test_free():
    rng = np.random.default_rng(8)
    lens = [100, 5, 64, -1, 30]
    table, refs, _ = _pool(40, lens, 7, rng)
    table[1, 3], refs[table[0, 0]] = table[0, 0], 2  # shared
    table[2, 6] = 40   # outside
    table[4, 5] = next(i for i in range(40) if refs[i] == 0)  # nobody's
    done = [1, 1, 7, 0, -2]
    ref, want, wl = Pool(refs), table.tolist(), list(lens)
    ref.free(want, wl, done)
    g_refs, g_table, gl, ws = _ints(refs), _ints(table), _ints(lens), lib.Workspace(256)
    lib.kv_free(g_refs, g_table, gl, _ints(done), workspace=ws)
    assert g_table.cpu().tolist() == want and gl.cpu().tolist() == wl and g_refs.cpu().tolist() == ref.refs
    assert ws.status() == 5 and ref.flag


def test_free_rows_of_a_wider_table():
    table = _ints(np.arange(60).reshape(4, 15))
    refs = torch.ones(60, dtype=torch.int32, device=DEV)
    lens = _ints([3, 3, 3])
    lib.kv_free(refs, table[:3, 2:9], lens)
    t = table.cpu().numpy()
    assert (t[:3, 2:9] == -1).all() and (t[3] >= 0).all() and (t[:, :2] >= 0).all() and (t[:, 9:] >= 0).all()
    assert refs.sum() == 60 - 21


@pytest.mark.parametrize("N,keep", [(1, 1.0), (7, 0.5), (1021, 0.6), (1021, 0.0), (1021, 1.0), (16384, 0.5),
                                    (40003, 0.3)])
def test_compact(N, keep):
    rng = np.random.default_rng(N)
    shapes = SHAPES if N < 2000 else SHAPES[2:5]
    width = 10
    rows = N // width + 1
    refs = (rng.random(N) < keep) * rng.integers(1, 4, N)
    used = rng.permutation(np.nonzero(refs)[0])
    table = np.full((rows, width), -1, np.int32)
    table.reshape(-1)[rng.permutation(rows * width)[:len(used)]] = used
    _, _, caches = _pool(N, [], 1, rng, shapes)
    ref, want = Pool(refs, [_bytes(c) for c in caches]), table.tolist()
    n = ref.compact(want)
    g_refs, g_table, ws = _ints(refs), _ints(table), lib.Workspace(lib.kv_pool_workspace_size(N, 0))
    ws.tensor[256:].random_(0, 256)  # whatever another call left
    got = lib.kv_compact(caches, g_refs, g_table, workspace=ws)
    assert got.item() == n and g_table.cpu().tolist() == want
    _same(ref, g_refs, caches)
    assert ws.status() == 0 and not (g_refs[n:] != 0).any() and (g_refs[:n] != 0).all()


def test_compact_reports_entries_that_name_no_block_in_use():
    refs, table, ws = _ints([1, 0, 0, 1, 0, 0]), _ints([[0, 3, 5, 6]]), lib.Workspace(lib.kv_pool_workspace_size(6, 0))
    cache = torch.arange(6, device=DEV, dtype=torch.float32).reshape(6, 1)
    lib.kv_compact([cache], refs, table, workspace=ws)
    assert table.cpu().tolist() == [[0, 1, 5, 6]] and refs.cpu().tolist() == [1, 1, 0, 0, 0, 0] and ws.status() == 5
    assert cache.cpu().reshape(-1).tolist() == [0, 3, 2, 3, 4, 5]


def test_large_blocks_and_many_tensors():
    """Blocks of more than a piece, and more tensors than one byte counts."""
    rng = np.random.default_rng(2)
    shapes = [((40001,), torch.uint8), ((12, BS, 128), torch.bfloat16)] + [((3, 5), torch.float32)] * 253
    table, refs, caches = _pool(6, [20, 3], 3, rng, shapes)
    ref = Pool(refs, [_bytes(c) for c in caches])
    rows, sizes = ref.fork(table.tolist(), [20, 3], [0, 1], 3)
    g_refs, child, cl = _ints(refs), _ints(np.zeros((2, 3))), _ints([0, 0])
    lib.kv_fork(caches, g_refs, _ints(table), _ints([20, 3]), _ints([0, 1]), child, cl)
    assert child.cpu().tolist() == rows
    _same(ref, g_refs, caches)
    with pytest.raises(lib.LibAttnError, match="UNSUPPORTED"):
        lib.kv_fork(caches + caches[:2], g_refs, _ints(table), _ints([20, 3]), _ints([0, 1]), child, cl)


def test_pool_of_more_than_four_gigabytes():
    """Byte offsets past 32 bits: a copy from the end of the pool to its front."""
    N, row = 70000, 65536
    big = torch.zeros((N, row), dtype=torch.uint8, device=DEV)
    big[N - 1] = torch.arange(row, device=DEV).to(torch.uint8)
    refs = torch.zeros(N, dtype=torch.int32, device=DEV)
    refs[N - 1] = 1
    table = _ints([[N - 1]])
    child, cl = _ints([[0]]), _ints([0])
    lib.kv_fork([big], refs, table, _ints([5]), _ints([0]), child, cl)
    assert child.item() == 0 and torch.equal(big[0], big[N - 1])
    lib.kv_free(refs, child, cl)
    big[0].zero_()
    assert lib.kv_compact([big], refs, table).item() == 1
    assert table.item() == 0 and torch.equal(big[0], big[N - 1]) and refs[0] == 1 and refs[N - 1] == 0


def test_a_captured_loop_allocates():
    """Free, fork, reserve and compact in one graph, replayed on other contents."""
    N, width, C = 300, 12, 10
    rng = np.random.default_rng(5)
    ws = lib.Workspace(lib.kv_pool_workspace_size(N, C))
    _, refs, caches = _pool(N, [], width, rng, SHAPES[:3])
    bufs = dict(refs=_ints(refs), table=_ints(np.full((3, width), -1)), lens=_ints([-1] * 3), src=_ints([0] * C),
                child=_ints(np.full((C, width), -1)), cl=_ints([-1] * C), new=_ints([0] * C), used=_ints([0]))

    def step():
        b = bufs
        lib.kv_free(b["refs"], b["child"], b["cl"], workspace=ws)
        lib.kv_fork(caches, b["refs"], b["table"], b["lens"], b["src"], b["child"], b["cl"], workspace=ws)
        lib.kv_reserve(b["refs"], b["child"], b["cl"], b["new"], workspace=ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for turn in range(4):
        lens = [int(x) for x in rng.integers(1, 150, 3)]
        table, refs, new_caches = _pool(N, lens, width, rng, SHAPES[:3])
        src, new = rng.integers(-1, 3, C).tolist(), rng.integers(0, 40, C).tolist()
        ref = Pool(refs, [_bytes(c) for c in new_caches])
        for c, x in zip(caches, new_caches):
            c.copy_(x)
        for k, x in (("refs", refs), ("table", table), ("lens", lens), ("src", src), ("new", new)):
            bufs[k].copy_(_ints(x))
        bufs["child"].fill_(-1)
        rows, sizes = ref.fork(table.tolist(), lens, src, width)
        ref.reserve(rows, sizes, new)
        g.replay()
        assert bufs["child"].cpu().tolist() == rows and bufs["cl"].cpu().tolist() == sizes
        _same(ref, bufs["refs"], caches)
        g.replay()  # frees what it gave out, and gives out the same
        assert bufs["child"].cpu().tolist() == rows
        _same(ref, bufs["refs"], caches)


def test_on_another_stream():
    s = torch.cuda.Stream()
    refs, table, lens = torch.zeros(20, dtype=torch.int32, device=DEV), _ints(np.full((2, 4), -1)), _ints([0, 5])
    new = _ints([17, 1])
    s.wait_stream(torch.cuda.current_stream())
    lib.kv_reserve(refs, table, lens, new, stream=s)
    s.synchronize()
    assert table.cpu().tolist() == [[0, 1, -1, -1], [2, -1, -1, -1]]
