"""GPU tests of what the rotary, tree, weight and eviction calls promise beside their formulas: which outputs may be
which inputs, whose memory a call may touch when, and what a workspace may hold."""
import os
import sys

import pytest
import torch

import masked_attention_paged_gb300 as lib

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_11_tree import _make as _tree_inputs, _run as _tree_run  # noqa: E402
from test_gpu_12_evict import _evict_inputs, _make as _weight_inputs, _run as _weight_run  # noqa: E402

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


@pytest.mark.parametrize("raw", [False, True])
def test_a_default_workspace_is_zeroed_before_another_stream_uses_it(monkeypatch, raw):
    monkeypatch.setattr(lib, "_default_ws", {})
    kc, vc, acc, bt, lens, dt = _evict_inputs([100, 60], 2, 64, 32, seed=30)
    bad = dt.clone()
    bad[0, 0] = -9  # noted in the workspace's status
    side = torch.cuda.Stream()
    lib.kv_evict(kc, vc, acc, bt, lens, dt, 32, workspace=lib.Workspace(256))  # the code is loaded
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # the current stream has a tenth of a second to go
    lib.kv_evict(kc, vc, acc, bt, lens, bad, 32, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert lib._small_ws(kc.device).status() == 5


def test_a_default_attention_workspace_is_zeroed_before_another_stream_uses_it(monkeypatch):
    """The word that a call leaves stays: a timed-out wait of the self-test stands for any."""
    monkeypatch.setattr(lib, "_default_ws", {})
    q = torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16, device=DEV)
    out, lse, side = torch.empty_like(q), torch.empty(1, 1, 64, device=DEV), torch.cuda.Stream()
    first = lib.Workspace(lib.attn_fwd_workspace_size_for(1, 1, 64, 64))  # the code is loaded
    lib.attn_fwd(q, q, q, out=out, lse=lse, workspace=first)
    lib._check("selftest", lib.load().attn_selftest_wait_timeout(first.ptr, first.nbytes, 100, side.cuda_stream))
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    lib.attn_fwd(q, q, q, out=out, lse=lse, stream=side)
    ws = lib._attn_ws(q, q)
    lib._check("selftest", lib.load().attn_selftest_wait_timeout(ws.ptr, ws.nbytes, 100, side.cuda_stream))
    torch.cuda.synchronize()
    assert ws.status() == 4


def test_a_replayed_graph_leaves_the_status_of_other_calls(monkeypatch):
    """The first call on a device captured without a workspace: its clearing is no part of a word that others share."""
    monkeypatch.setattr(lib, "_default_ws", {})
    kc, vc, acc, bt, lens, dt = _evict_inputs([100, 60], 2, 64, 32, seed=31)
    nl, kept = torch.empty_like(lens), torch.empty(2, 2, 32, dtype=torch.int32, device=DEV)
    want = lib.kv_evict(kc.clone(), vc.clone(), acc.clone(), bt, lens, dt, 32, sink=1, recent=4,
                        workspace=lib.Workspace(256))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.kv_evict(kc, vc, acc, bt, lens, dt, 32, sink=1, recent=4, new_lens=nl, kept=kept)
    bad = dt.clone()
    bad[0, 0] = -9  # noted in the workspace's status
    lib.kv_evict(kc.clone(), vc.clone(), acc.clone(), bt, lens, bad, 32)
    assert lib._small_ws(kc.device).status() == 5
    for _ in range(2):
        graph.replay()
        assert torch.equal(nl, want[0]) and torch.equal(kept, want[1])
        assert lib._small_ws(kc.device).status() == 5


_STALE_COUNTS = """
import math, torch
import masked_attention_paged_gb300 as lib
DEV = "cuda"
g = torch.Generator().manual_seed(1)
mb, Hkv, D = 700, 2, 64
bt = torch.randperm(mb, generator=g).to(torch.int32).view(1, mb).to(DEV)
kc, vc = (torch.randn(mb, Hkv, 16, D, generator=g).bfloat16().to(DEV) for _ in range(2))
q = torch.randn(1, 8, D, generator=g).bfloat16().to(DEV)
lens = torch.tensor([mb * 16], dtype=torch.int32, device=DEV)
lse = torch.full((1, 8), 9.0, device=DEV)
size = max(lib.paged_decode_workspace_size(1, 8, mb, 16, D), lib.paged_attn_weights_workspace_size(1, Hkv, mb))
ws = lib.Workspace(size)

def decode():
    out = torch.zeros_like(q)
    lib.paged_decode_attn(q, kc, vc, bt, lens, out=out, workspace=ws)
    return out

def weights():
    acc = torch.zeros(mb, Hkv, 16, device=DEV)
    lib.paged_attn_weights(q, lse, kc, bt, lens - 1, acc, workspace=ws)
    return acc

want = {f: f() for f in (decode, weights)}
number = 2  # calls so far that count
for _ in range(4):
    for f, ref in want.items():
        number += 1
        words = ws.tensor[256:].view(torch.int32).view(-1, 2)
        words[:, 0], words[:, 1] = 1000, number
        got = f()
        assert torch.equal(got, ref), (f.__name__, number, float((got - ref).abs().max()))
assert ws.status() == 0
print("counted")
"""


def test_small_integers_in_a_workspace_are_no_counts():
    """What a call finds where its counts go are other calls' tables of small integers; the calls of a fresh process are
    numbered from one, so that some of these words hold the very number of the call."""
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _STALE_COUNTS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "counted" in r.stdout, r.stderr[-2000:]


BAD = (-1, -7, "past")  # ids that name no block; -1 is what tables are often filled with


def _with(s, b, i, bad):
    """The inputs with entry i of sequence b's table set to an id that names no block."""
    bt = s["bt"].clone()
    bt[b, i] = s["kc"].shape[0] if bad == "past" else bad
    return dict(s, bt=bt)


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("T", [6, 40, 70])  # drafts aside, in ring stages, two row tiles
def test_tree_reports_every_id_that_names_no_block(T, bad):
    s = _tree_inputs([300, 300, 20], T, 4, 2, 64, seed=40 + T)
    good = _tree_run(s)
    # a block in the middle of the context, its last, and one of the drafts alone
    for i in (3, 18, (300 + T - 1) // 16):
        o, l, _, _, st = _tree_run(_with(s, 0, i, bad))
        assert st == 5, (i, st)
        assert torch.equal(o[1:], good[0][1:]) and torch.equal(l[1:], good[1][1:])
    assert good[4] == 0


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("T", [20, 40, 70])
def test_blocks_of_absent_drafts_alone_need_not_be_there(T, bad):
    """Shorter trees of a batch: what the table holds past their drafts is no matter, also when the drafts are cached
    already; the block of a draft that is there is."""
    s = _tree_inputs([300, 305, 20], T, 4, 2, 64, seed=50 + T)
    n = int((s["parents"][1] >= -1).sum())
    assert n == T // 2
    fresh = _tree_run(s)
    cached = dict(s, kc=fresh[2], vc=fresh[3])
    none = dict(k_new=None, v_new=None)
    want = _tree_run(cached, **none)
    assert fresh[4] == want[4] == 0
    last, first_free = (305 + n - 1) // 16, (305 + n + 15) // 16
    assert first_free <= (305 + T - 1) // 16
    for inputs, ref, kw in ((s, fresh, {}), (cached, want, none)):
        o, l, _, _, st = _tree_run(_with(inputs, 1, first_free, bad), **kw)
        assert st == 0 and torch.equal(o, ref[0]) and torch.equal(l, ref[1])
        o, l, _, _, st = _tree_run(_with(inputs, 1, last, bad), **kw)
        assert st == 5
        for b in (0, 2):
            assert torch.equal(o[b], ref[0][b]) and torch.equal(l[b], ref[1][b])


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("T", [1, 50])
def test_weights_report_every_id_that_names_no_block(T, bad):
    s = _weight_inputs([400, 20], T, 4, 2, 64, seed=60 + T)
    good, st = _weight_run(s)
    assert st == 0
    for i in (4, (400 + T - 1) // 16):
        lost = int(s["bt"][0, i])
        out, st = _weight_run(_with(s, 0, i, bad))
        keep = torch.arange(good.shape[0], device=DEV) != lost
        assert st == 5 and torch.equal(out[keep].view(torch.int32), good[keep].view(torch.int32))
        assert torch.equal(out[lost].view(torch.int32), s["acc"][lost].view(torch.int32))


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_reports_every_id_that_names_no_block(D, causal, bad):
    g = torch.Generator().manual_seed(70)
    nb, mb, T = 60, 25, 40
    kc, vc = (torch.randn(nb, 2, 16, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    s = dict(kc=kc, bt=torch.randperm(nb, generator=g)[:2 * mb].to(torch.int32).view(2, mb).to(DEV))
    q = torch.randn(2, 4, T, D, generator=g).bfloat16().to(DEV)
    start = torch.tensor([330, 31], dtype=torch.int32, device=DEV)
    ws = lib.Workspace(256)

    def run(x):
        ws.reset()
        out, lse = lib.paged_prefill_attn(q, kc, vc, x["bt"], start, causal=causal, return_lse=True, workspace=ws)
        return out, lse, ws.status()

    good = run(s)
    assert good[2] == 0
    for i in (3, 20, (330 + T - 1) // 16):  # in the context, at its end, in the chunk
        out, lse, st = run(_with(s, 0, i, bad))
        assert st == 5, i
        assert torch.equal(out[1], good[0][1]) and torch.equal(lse[1], good[1][1])
    assert run(_with(s, 0, 24, bad))[2] == 0  # past the chunk


def _step(q, k, v, kc, vc, acc, bt, dt, lens, parents, path, n, freqs, ws):
    """One step of a server over its cache: every call of the three groups."""
    pos = lens[:, None] + torch.arange(q.shape[2], device=DEV, dtype=torch.int32)
    rq = lib.rope_kv_append(q, k, v, pos, freqs, kc, vc, bt, lens, workspace=ws)
    cached, _ = lib.paged_tree_attn(rq, kc, vc, bt, lens, parents, return_lse=True, workspace=ws)
    out, lse = lib.paged_tree_attn(rq, kc, vc, bt, lens, parents, k_new=k, v_new=v, return_lse=True, workspace=ws)
    lib.kv_tree_accept(kc, vc, bt, lens, path, n, workspace=ws)
    few = path.shape[1]
    lib.paged_attn_weights(rq[:, :, :few], lse[:, :, :few].contiguous(), kc, bt, lens, acc, q_lens=n, workspace=ws)
    new_lens, kept = lib.kv_evict(kc, vc, acc, bt, lens + n, dt, 100, sink=4, recent=20, workspace=ws)
    return rq, cached, out, lse, new_lens, kept


def _step_inputs(seed, blocks, B, Hq, Hkv, T, D, longest):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    mb = (longest + T + 15) // 16
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    lens = torch.randint(1, longest, (B,), generator=g, device=DEV).to(torch.int32)
    lens[0] = longest
    size = max(lib.paged_tree_workspace_size(B, Hq, Hkv, T, mb, 16, D),
               lib.paged_attn_weights_workspace_size(B, Hkv, mb))
    return dict(q=r(B, Hq, T, D), k=r(B, Hkv, T, D), v=r(B, Hkv, T, D), kc=r(blocks, Hkv, 16, D),
                vc=r(blocks, Hkv, 16, D), acc=torch.rand(blocks, Hkv, 16, generator=g, device=DEV),
                bt=perm[:B * mb].view(B, mb), dt=perm[B * mb:B * mb + 7 * B].view(B, 7), lens=lens,
                parents=torch.tensor([[max(-1, t - 1 - t % 2) for t in range(T)]] * B, dtype=torch.int32, device=DEV),
                path=torch.tensor([[0, 2, 5, 8]] * B, dtype=torch.int32, device=DEV),
                n=torch.arange(B, device=DEV, dtype=torch.int32) % 5, freqs=lib.rope_frequencies(D)[0],
                ws=lib.Workspace(size))


def _same(x, y):
    return torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


def test_two_steps_at_once():
    """Two threads, two streams, workspaces and caches of their own: the results of each alone."""
    import threading
    inputs = [_step_inputs(seed, 500, 4, 8, 4, T, 64, 900) for seed, T in ((1, 9), (2, 40))]
    streams = [torch.cuda.Stream() for _ in inputs]
    want, wrong = [None, None], []

    def go(i, times):
        try:
            s = inputs[i]
            with torch.cuda.stream(streams[i]):
                for _ in range(times):
                    x = {k: v.clone() if k in ("kc", "vc", "acc") else v for k, v in s.items()}
                    got = [t.clone() for t in (*_step(**x), x["kc"], x["vc"], x["acc"])]
                    if want[i] is None:
                        want[i] = got
                    assert all(_same(a, b) for a, b in zip(got, want[i]))
                assert s["ws"].status() == 0
        except BaseException as e:
            wrong.append(e)

    torch.cuda.synchronize()
    go(0, 1), go(1, 1)
    threads = [threading.Thread(target=go, args=(i, 40)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_offsets_past_32_bits():
    """A cache of 2.3e9 elements, the step in its first blocks and in its last: the same bits."""
    s = _step_inputs(3, 200, 3, 32, 8, 11, 128, 600)
    n, few = 140000, 200
    ends = []
    big = {c: torch.zeros(n, *s[c].shape[1:], dtype=s[c].dtype, device=DEV) for c in ("kc", "vc", "acc")}
    assert big["kc"].numel() > 1 << 31
    for flip in (False, True):
        for c in big:
            (big[c][n - few:] if flip else big[c][:few]).copy_(s[c].flip(0) if flip else s[c])
        at = lambda t: (n - 1 - t).to(torch.int32) if flip else t  # noqa: E731
        x = dict(s, **big, bt=at(s["bt"]).contiguous(), dt=at(s["dt"]).contiguous())
        got = [t.clone() for t in _step(**x)]
        ends.append(got + [(big[c][n - few:].flip(0) if flip else big[c][:few]).clone() for c in big])
    assert s["ws"].status() == 0
    assert all(_same(a, b) for a, b in zip(*ends))
    # a rotation of rows 2^29 elements apart, in place
    far = torch.zeros(9, (1 << 29) + 64, dtype=torch.bfloat16, device=DEV)[:, -64:][None, None]
    far.copy_(torch.randn(9, 64, device=DEV))
    pos, (freqs, _) = torch.arange(9, dtype=torch.int32, device=DEV)[None], lib.rope_frequencies(64)
    want = lib.rope_apply(far.contiguous(), pos, freqs)
    assert torch.equal(lib.rope_apply(far, pos, freqs, out=far), want)


def test_the_handle_of_the_default_stream_is_the_default_stream():
    """What a call allocates and zeroes is ordered before its kernels also when the stream comes as its handle, 0."""
    here = torch.device(DEV, torch.cuda.current_device())
    side = torch.cuda.Stream()
    for stream in (0, torch.cuda.default_stream(), side, side.cuda_stream):
        handle = getattr(stream, "cuda_stream", stream)
        with torch.cuda.stream(torch.cuda.Stream()):  # whichever is current
            assert lib._fresh(lambda: torch.cuda.current_stream().cuda_stream, stream, here) == handle
    # the zeroes of a workspace would reach it from a stream that nothing orders before the call's
    s = _weight_inputs([700, 90, 400], 60, 8, 2, 128, seed=80)
    want, _ = _weight_run(s)
    for _ in range(50):
        acc = s["acc"].clone()
        lib.paged_attn_weights(s["q"], s["lse"], s["kc"], s["bt"], s["start"], acc, scale=s["scale"], stream=0)
        assert torch.equal(acc.view(torch.int32), want.view(torch.int32))


def test_what_the_older_calls_allocate_belongs_to_their_stream():
    """The zeroes of a workspace or of the gather's rows, queued on a busy current stream, would land on the results."""
    g = torch.Generator().manual_seed(90)
    kc, vc = (torch.randn(200, 2, 16, 128, generator=g).bfloat16().to(DEV) for _ in range(2))
    bt = torch.randperm(200, generator=g)[:180].to(torch.int32).view(2, 90).to(DEV)
    lens = torch.tensor([1400, 700], dtype=torch.int32, device=DEV)
    q = torch.randn(2, 8, 128, generator=g).bfloat16().to(DEV)
    qp = torch.randn(2, 8, 33, 128, generator=g).bfloat16().to(DEV)
    kq, sc = torch.randint(-127, 128, kc.shape, generator=g, dtype=torch.int8).to(DEV), torch.rand(200, 2, 16).to(DEV)
    side = torch.cuda.Stream()

    def chain(stream):
        kw = dict(stream=stream)
        out, lse = lib.attn_fwd(qp, qp, qp, **kw)
        return [out, lse, lib.attn_fwd_varlen(qp, qp, qp, short, **kw)[0],
                *lib.attn_lse_merge([out, out], [lse, lse], **kw),
                lib.paged_decode_attn(q, kc, vc, bt, lens, **kw),
                lib.paged_decode_attn_append(q, q[:, :2], q[:, 2:4], kc, vc, bt, lens, **kw),
                lib.paged_prefill_attn(qp, kc, vc, bt, lens, **kw),
                lib.paged_decode_attn_q8(q, kq, kq, sc, sc, bt, lens, **kw),
                lib.paged_kv_gather(kc, bt, lens, 1400, **kw)]

    short = lens.clamp(max=20)
    want = [x.clone() for x in chain(None)]
    chain(side)  # the default workspaces are there
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(100_000_000)
        got = chain(stream)
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(got, want))
