"""GPU tests of the attention weights and of the eviction against their definitions.

Weights, in 64 bits: a score (natural-log units) is off by at most D 2^-23 of
the sum of its terms' sizes; the log2 LSE and the fused subtraction round to
2^-24 of |lse| and of |x| each, and ex2.approx to 2^-22: e = D 2^-23 size + 2^-22
|lse| + 2^-21 relative for each weight.  A sum of n float32 terms in eight
chains adds (n / 8 + 8) 2^-24 relative (every term is positive), and joining it
to the old sum 2^-24 of the result.  The eviction copies and selects: exact."""
import math

import pytest
import torch

import masked_attention_paged_gb300 as lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _make(starts, T, Hq, Hkv, D, seed, lens=None, causal=True, gain=1.0):
    """K caches whose free slots are NaN, sums whose chunk slots are NaN, and the LSE of the same rows."""
    g = _gen(seed)
    B = len(starts)
    mb = max(1, (max(starts) + T + 15) // 16)
    nb = B * mb + 2
    bt = torch.randperm(nb, generator=g)[:B * mb].to(torch.int32).view(B, mb)
    kc = torch.full((nb, Hkv, 16, D), float("nan"), dtype=torch.bfloat16)
    acc = torch.rand(nb, Hkv, 16, generator=g)
    q = (torch.randn(B, T, Hq, D, generator=g) * gain).bfloat16().transpose(1, 2)
    lse = torch.full((B, Hq, T), float("nan"))  # rows past q_lens may hold anything
    scale = 1.0 / math.sqrt(D)
    for b, s in enumerate(starts):
        n = T if lens is None else max(0, min(lens[b], T))
        if s < 0 or n == 0:
            continue
        keys = torch.randn(Hkv, s + n, D, generator=g).bfloat16()
        for i in range((s + n + 15) // 16):
            m = min(16, s + n - 16 * i)
            kc[bt[b, i], :, :m] = keys[:, 16 * i:16 * i + m]
        for i in range(s, s + n):
            acc[bt[b, i // 16], :, i % 16] = float("nan")
        x = q[b, :, :n].double() @ keys.double().repeat_interleave(Hq // Hkv, 0).transpose(1, 2) * scale
        if causal:
            x.masked_fill_(torch.arange(s + n) > s + torch.arange(n)[:, None], -math.inf)
        lse[b, :, :n] = torch.logsumexp(x, -1).float()
    return dict(q=q.to(DEV), lse=lse.to(DEV), kc=kc.to(DEV), bt=bt.to(DEV), acc=acc.to(DEV), scale=scale, causal=causal,
                start=torch.tensor(starts, dtype=torch.int32, device=DEV),
                q_lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV))


def _define(s):
    """(sums, bounds) in 64 bits; NaN bounds where nothing is promised."""
    B, Hq, T, D = s["q"].shape
    Hkv = s["kc"].shape[1]
    G = Hq // Hkv
    acc, tol = s["acc"].double(), torch.zeros_like(s["acc"], dtype=torch.float64)
    for b in range(B):
        st = int(s["start"][b])
        n = T if s["q_lens"] is None else max(0, min(int(s["q_lens"][b]), T))
        if st < 0 or n == 0 or st + n > s["bt"].shape[1] * 16:
            continue
        at = torch.arange(st + n, device=DEV)
        blk = s["bt"][b, at // 16].long()
        for h in range(Hkv):
            k = s["kc"][blk, h, at % 16].double()
            q = s["q"][b, h * G:(h + 1) * G, :n].double()
            lse = s["lse"][b, h * G:(h + 1) * G, :n].double()[..., None]
            w = torch.exp(q @ k.t() * s["scale"] - lse)
            if s["causal"]:
                w = torch.tril(w, diagonal=st)
            w = torch.where(torch.isneginf(lse), 0.0, w)
            size = float((q.abs() @ k.abs().t()).max()) * abs(s["scale"])
            fin = lse[torch.isfinite(lse)]
            e = D * 2.0 ** -23 * size + 2.0 ** -22 * float(fin.abs().max() if fin.numel() else 0) + 2.0 ** -21
            got = w.sum((0, 1))
            old = torch.where(at < st, acc[blk, h, at % 16], 0.0)
            acc[blk, h, at % 16] = old + got
            tol[blk, h, at % 16] = got * (e + (G * n / 8 + 8) * 2.0 ** -24) + (old + got) * 2.0 ** -24
    return acc, tol


def _run(s, acc=None, ws=None):
    acc = s["acc"].clone() if acc is None else acc
    B, Hkv, mb = s["q"].shape[0], s["kc"].shape[1], s["bt"].shape[1]
    ws = ws or lib.Workspace(lib.paged_attn_weights_workspace_size(B, Hkv, mb))
    lib.paged_attn_weights(s["q"], s["lse"], s["kc"], s["bt"], s["start"], acc, q_lens=s["q_lens"], causal=s["causal"],
                           scale=s["scale"], workspace=ws)
    return acc, ws.status()


def _check(s, status=0):
    got, st = _run(s)
    assert st == status
    ref, tol = _define(s)
    touched = tol > 0
    err = (got.double() - ref).abs()
    assert bool((err[touched] <= tol[touched]).all()), float((err - tol)[touched].max())
    # everything else is as it was, bit for bit
    assert torch.equal(got[~touched].view(torch.int32), s["acc"][~touched].view(torch.int32))
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 2, 2), (1, 8, 1), (5, 6, 2), (40, 8, 2), (128, 2, 2), (129, 7, 1), (300, 4, 2)])
def test_weights(T, Hq, Hkv, D):
    """Chunks of one token to several row chunks, after no context and contexts around block, tile and pair ends."""
    _check(_make([0, 1, 15, 130, 255, 256, 600], T, Hq, Hkv, D, seed=T + D))
    _check(_make([0, 3, 260], T, Hq, Hkv, D, seed=T + D + 1, causal=False))


@pytest.mark.parametrize("D", [64, 128])
def test_long_chunks_and_long_contexts_are_cut_between_sms(D):
    _check(_make([0], 3001, 4, 1, D, seed=2))       # a whole prompt, causal
    _check(_make([40007], 1, 4, 2, D, seed=3))      # one token over a long context
    _check(_make([9000, 100], 200, 8, 1, D, seed=4))


def test_many_sequences_and_ragged_chunks():
    starts = [(53 * b * b + 7 * b) % 700 for b in range(45)]
    _check(_make(starts, 3, 8, 2, 128, seed=5))
    lens = [b % 5 - 1 for b in range(45)]  # -1, 0, 1, 2, 3: none, one, all
    _check(_make(starts, 3, 8, 2, 64, seed=6, lens=lens))


def test_peaked_scores():
    _check(_make([300, 40], 30, 8, 2, 128, seed=7, gain=6.0))


def test_every_row_sums_to_one():
    """A causal prompt: the sums of all tokens add up to the number of rows."""
    s = _make([0, 0], 500, 6, 2, 128, seed=8)
    s["acc"].zero_()
    got, _ = _run(s)
    for b in range(2):
        at = torch.arange(500, device=DEV)
        total = got[s["bt"][b, at // 16].long(), :, at % 16].double().sum(0)
        assert bool(((total - 3 * 500).abs() <= 3 * 500 * 2.0 ** -14).all())  # e of each weight is below 2^-14 here


def test_rows_that_saw_nothing_and_nan_in_keys_that_are_not_seen():
    """lse = -inf adds nothing, whatever the row's query holds; a NaN key takes only its own sum with it."""
    s = _make([100], 20, 4, 2, 64, seed=9)
    s["lse"][0, 1, 7] = -math.inf
    s["q"][0, 1, 7] = float("inf")
    got = _check_no_inf(s)
    z = dict(s, kc=s["kc"].clone())
    z["kc"][z["bt"][0, 110 // 16].long(), 0, 110 % 16, 3] = float("nan")
    bad, st = _run(z)
    assert st == 0
    assert math.isnan(float(bad[z["bt"][0, 6].long(), 0, 14]))
    keep = torch.ones_like(bad, dtype=torch.bool)
    keep[z["bt"][0, 6].long(), 0, 14] = False
    assert torch.equal(bad[keep].view(torch.int32), got[keep].view(torch.int32))


def _check_no_inf(s):
    clean = dict(s, q=torch.where(torch.isinf(s["q"]), 0.0, s["q"]))
    got, st = _run(s)
    ref, _ = _run(clean)
    assert st == 0 and torch.equal(got.view(torch.int32), ref.view(torch.int32))
    _check(clean)
    return got


def test_idle_and_refused_sequences():
    s = _make([40, 5, 33, 60], 4, 4, 2, 128, seed=10)
    s["start"][1] = -1
    s["start"][2] = s["bt"].shape[1] * 16 - 3
    _check(s, status=5)
    s = _make([400, 20], 1, 4, 2, 64, seed=11)
    got, _ = _run(s)
    z = dict(s, bt=s["bt"].clone())
    lost = int(z["bt"][0, 4])
    z["bt"][0, 4] = -3
    out, st = _run(z)
    keep = torch.arange(s["acc"].shape[0], device=DEV) != lost
    assert st == 5 and torch.equal(out[keep].view(torch.int32), got[keep].view(torch.int32))
    assert torch.equal(out[lost].view(torch.int32), s["acc"][lost].view(torch.int32))


def test_weights_workspace_reuse_streams_and_graphs():
    a, b = _make([700, 90, 400], 60, 8, 2, 128, seed=12), _make([2000], 300, 4, 1, 128, seed=13)
    ws = lib.Workspace(max(lib.paged_attn_weights_workspace_size(x["q"].shape[0], x["kc"].shape[1], x["bt"].shape[1])
                           for x in (a, b)))
    ws.tensor[256:].random_(0, 256)
    eq = lambda x, y: torch.equal(x.view(torch.int32), y.view(torch.int32))  # noqa: E731
    ref = [_run(x)[0] for x in (a, b)]
    for x, r in ((a, ref[0]), (b, ref[1]), (a, ref[0])):
        got, st = _run(x, ws=ws)
        assert st == 0 and eq(got, r)
    calls = []
    for x in (a, b):
        acc = x["acc"].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _cap(x, acc, ws)
        calls.append((g, acc))
    for i in (0, 1, 1, 0):
        calls[i][1].copy_((a, b)[i]["acc"])
        calls[i][0].replay()
        assert eq(calls[i][1], ref[i])
    a["start"].sub_(torch.tensor([300, 60, 17], dtype=torch.int32, device=DEV))  # other cuts
    want, _ = _run(a)
    calls[0][1].copy_(a["acc"])
    calls[0][0].replay()
    assert eq(calls[0][1], want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = _run(a, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert eq(got, want)


def _cap(s, acc, ws):
    lib.paged_attn_weights(s["q"], s["lse"], s["kc"], s["bt"], s["start"], acc, scale=s["scale"], workspace=ws)


# --------------------------------------------------------------------------
def _evict_inputs(lens, Hkv, D, keep, seed, values="plain"):
    g = _gen(seed)
    B = len(lens)
    mb = max(1, (max(max(lens), 1) + 15) // 16)
    db = (keep + 15) // 16
    n = B * (mb + db) + 1
    perm = torch.randperm(n, generator=g).to(torch.int32)
    bt, dt = perm[:B * mb].view(B, mb), perm[B * mb:B * (mb + db)].view(B, db)
    kc, vc = (torch.randn(n, Hkv, 16, D, generator=g).bfloat16() for _ in range(2))
    acc = torch.rand(n, Hkv, 16, generator=g)
    if values == "ties":
        acc = (acc * 4).floor()
    elif values == "equal":
        acc.zero_()
    elif values == "wild":
        acc = torch.randn(n, Hkv, 16, generator=g) * 1e30
        pick = torch.randint(0, 12, acc.shape, generator=g)
        for i, v in enumerate((math.inf, -math.inf, math.nan, -0.0, 0.0, 1e-42, -1e-42)):
            acc[pick == i] = v
    return [x.to(DEV) for x in (kc, vc, acc, bt, torch.tensor(lens, dtype=torch.int32), dt)]


def _evict_define(kc, vc, acc, bt, lens, dt, keep, sink, recent):
    """Lists, sorted in Python: (new_lens, kept, K, V, acc)."""
    B, Hkv = lens.shape[0], kc.shape[1]
    ek, ev, ea = kc.clone(), vc.clone(), acc.clone()
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32)
    a, t = acc.cpu(), bt.cpu().tolist()
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            x = [float(a[t[b][i // 16], h, i % 16]) for i in range(n)]
            held = [i for i in range(n) if i < sink or i >= n - recent]
            free = [i for i in range(n) if not (i < sink or i >= n - recent)]
            free.sort(key=lambda i: (math.isnan(x[i]), -x[i] if not math.isnan(x[i]) else 0.0, i))
            best = sorted((held + free)[:keep]) if n > keep else list(range(max(n, 0)))
            kept[b, h, :len(best)] = torch.tensor(best, dtype=torch.int32)
            for i, j in enumerate(best):
                d, s = int(dt[b, i // 16]), t[b][j // 16]
                ek[d, h, i % 16], ev[d, h, i % 16] = kc[s, h, j % 16], vc[s, h, j % 16]
                ea[d, h, i % 16] = acc[s, h, j % 16]
    return torch.where(lens < 0, lens, lens.clamp(max=keep)), kept.to(DEV), ek, ev, ea


def _evict_check(args, keep, sink, recent, status=0):
    want = _evict_define(*args, keep, sink, recent)
    kc, vc, acc, bt, lens, dt = args
    kc, vc, acc = kc.clone(), vc.clone(), acc.clone()
    ws = lib.Workspace(256)
    nl, kept = lib.kv_evict(kc, vc, acc, bt, lens, dt, keep, sink=sink, recent=recent, workspace=ws)
    assert ws.status() == status
    assert torch.equal(nl, want[0]) and torch.equal(kept, want[1])
    assert torch.equal(kc, want[2]) and torch.equal(vc, want[3])
    assert torch.equal(acc.view(torch.int32), want[4].view(torch.int32))


@pytest.mark.parametrize("values", ["plain", "ties", "equal", "wild"])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (16, 4, 8), (37, 0, 37), (100, 3, 20), (100, 50, 50)])
def test_evict(keep, sink, recent, values):
    """Idle, empty, shorter than, equal to and just past the budget, and longer sequences."""
    args = _evict_inputs([-1, 0, 1, keep, keep + 1, 333, 90], 3, 64, keep, seed=keep, values=values)
    _evict_check(args, keep, sink, recent)


@pytest.mark.parametrize("L,keep", [(5000, 4096), (20000, 700), (70001, 512), (140000, 64)])
def test_evict_long(L, keep):
    """One CTA a head, clusters of two to eight, and a context longer than a cluster's registers hold."""
    _evict_check(_evict_inputs([L, L // 3], 1, 128, keep, seed=L, values="ties" if L == 20000 else "plain"), keep, 4, 16)


def test_evict_reports_bad_tables():
    args = _evict_inputs([200, 100, 60], 2, 64, 48, seed=20)
    kc, vc, acc, bt, lens, dt = args
    good = _evict_define(*args, 48, 2, 10)
    ws = lib.Workspace(256)
    d2 = dt.clone()
    d2[1, 1] = kc.shape[0] + 5
    k2, v2, a2 = kc.clone(), vc.clone(), acc.clone()
    nl, kept = lib.kv_evict(k2, v2, a2, bt, lens, d2, 48, sink=2, recent=10, workspace=ws)
    assert ws.status() == 5 and torch.equal(nl, good[0]) and torch.equal(kept, good[1])
    lost = int(dt[1, 1])
    rest = torch.arange(kc.shape[0], device=DEV) != lost
    assert torch.equal(k2[rest], good[2][rest]) and torch.equal(v2[rest], good[3][rest])
    assert torch.equal(k2[lost], kc[lost]) and torch.equal(a2[lost], acc[lost])
    # a table that is too short for what is kept
    ws.reset()
    k3, v3, a3 = kc.clone(), vc.clone(), acc.clone()
    lib.kv_evict(k3, v3, a3, bt, lens, dt[:, :2], 48, sink=2, recent=10, workspace=ws)
    assert ws.status() == 5
    third = torch.isin(torch.arange(kc.shape[0], device=DEV), dt[:, 2].long())
    assert torch.equal(k3[third], kc[third]) and torch.equal(k3[~third], good[2][~third])
    # a length past the table is cut to it
    ws.reset()
    big = lens.clone()
    big[0] = bt.shape[1] * 16 + 9
    nl, kept = lib.kv_evict(kc.clone(), vc.clone(), acc.clone(), bt, big, dt, 48, workspace=ws)
    assert ws.status() == 5 and int(nl[0]) == 48 and int(kept.max()) < bt.shape[1] * 16


def test_evict_in_a_graph():
    args = _evict_inputs([500, 300], 2, 128, 64, seed=21)
    kc, vc, acc, bt, lens, dt = args
    nl, kept = torch.empty(2, dtype=torch.int32, device=DEV), torch.empty(2, 2, 64, dtype=torch.int32, device=DEV)
    ws = lib.Workspace(256)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.kv_evict(kc, vc, acc, bt, lens, dt, 64, sink=1, recent=9, new_lens=nl, kept=kept, workspace=ws)
    acc.neg_()
    lens.copy_(torch.tensor([60, 299], dtype=torch.int32))
    want = _evict_define(*args, 64, 1, 9)
    g.replay()
    assert torch.equal(nl, want[0]) and torch.equal(kept, want[1])
    assert torch.equal(kc, want[2]) and torch.equal(vc, want[3]) and torch.equal(acc, want[4])
