"""Draft verification, pools of blocks and the e4m3 cache without a GPU: sizes, refusals,
marshalling, devices."""
import ctypes

import pytest
import torch

import masked_attention_paged_gb300 as lib
from masked_attention_paged_gb300 import AttnKVCacheF8, AttnPoolTensor
from test_binding_marshalling import rec  # noqa: F401  (fixture)
from test_boundary import FAKE, INVALID, L, OK, UNSUPPORTED, WORKSPACE, _t  # noqa: F401

BIG = 1 << 33
F8 = torch.float8_e4m3fn
FAR = [FAKE + (i << 30) for i in range(1, 9)]


# --------------------------------------------------------------------------
# draft verification
# --------------------------------------------------------------------------
def _verify(L, p=None, q=None, tok=FAR[0], ts=6, par=FAR[1], ps=6, u=FAR[2], us=6, path=FAR[3], n=FAR[4],  # noqa: F811
            nxt=FAR[5], ws=FAKE, ws_bytes=256):
    p = p or _t([2, 6, 100], 0)
    return L.draft_verify(ctypes.byref(p), None if q is None else ctypes.byref(q), tok, ts, par, ps, u, us, 0, path, n,
                          nxt, ws, ws_bytes, None)


def test_draft_verify_rejects(L):  # noqa: F811
    assert L.draft_verify_workspace_size(4, 8, 1000) == 256 and L.draft_verify_workspace_size(-1, 8, 9) == 0
    assert _verify(L, p=_t([2, 600], 0)) == INVALID
    assert _verify(L, p=_t([2, 6, 100], 3)) == INVALID
    assert _verify(L, p=_t([2, 0, 100], 0)) == INVALID and _verify(L, p=_t([2, 6, 0], 0)) == INVALID
    assert _verify(L, p=_t([2, 257, 100], 0), ts=257, ps=257, us=257) == UNSUPPORTED
    assert _verify(L, p=_t([2, 6, (1 << 30) + 1], 0)) == UNSUPPORTED
    assert _verify(L, p=_t([65536, 6, 100], 0)) == UNSUPPORTED
    assert _verify(L, q=_t([2, 6, 101], 0)) == INVALID
    assert _verify(L, q=_t([2, 6, 100], 1)) == INVALID  # another type
    assert _verify(L, p=_t([2, 6, 100], 0, data=FAKE + 2)) == INVALID
    assert _verify(L, p=_t([2, 6, 100], 0, stride=(1200, 200, 2))) == INVALID
    for kw in (dict(tok=None), dict(par=None), dict(u=None), dict(path=None), dict(n=None), dict(nxt=None)):
        assert _verify(L, **kw) == INVALID, kw
    assert _verify(L, ts=5) == INVALID and _verify(L, ps=5) == INVALID and _verify(L, us=5) == INVALID
    assert _verify(L, path=FAR[4] - 44) == INVALID  # over the lengths
    assert _verify(L, n=FAR[5] + 4) == INVALID
    assert _verify(L, path=FAR[0] + 4) == INVALID and _verify(L, nxt=FAR[2]) == INVALID
    assert _verify(L, ws=None) == WORKSPACE and _verify(L, ws_bytes=255) == WORKSPACE
    assert _verify(L, p=_t([0, 6, 100], 0)) == OK


# --------------------------------------------------------------------------
# pools
# --------------------------------------------------------------------------
def _tensors(*blocks):
    arr = (AttnPoolTensor * max(1, len(blocks)))()
    for i, n in enumerate(blocks):
        arr[i].data, arr[i].block_bytes = FAKE, n
    return arr


def test_pool_sizes(L):  # noqa: F811
    size = L.kv_pool_workspace_size
    assert size(1000, 64) >= 256 + 4 * (2 * 1000 + 64) and size(1000, 64) % 256 == 0
    assert size(-1, 3) == 0 and size(10, -1) == 0 and size((1 << 20) + 1, 1) == 0 and size(1 << 20, 1) > 0


def test_kv_free_and_reserve_reject(L):  # noqa: F811
    def free(refs=FAKE, N=10, bt=FAR[0], st=4, mb=4, cl=FAR[1], done=FAR[2], b=2, ws=FAKE, n=256):
        return L.kv_free(refs, N, bt, st, mb, cl, done, b, ws, n, None)

    def reserve(refs=FAKE, N=10, bt=FAR[0], st=4, mb=4, cl=FAR[1], new=FAR[2], b=2, ws=FAKE, n=1 << 20):
        return L.kv_reserve(refs, N, bt, st, mb, cl, new, b, ws, n, None)
    for call in (free, reserve):
        assert call(refs=None) == INVALID and call(bt=None) == INVALID and call(cl=None) == INVALID
        assert call(N=0) == INVALID and call(b=-1) == INVALID and call(mb=0) == INVALID and call(st=3) == INVALID
        assert call(N=(1 << 20) + 1) == UNSUPPORTED and call(b=65536) == UNSUPPORTED
        assert call(mb=(1 << 24) + 1, st=1 << 25) == INVALID
        assert call(ws=None) == WORKSPACE and call(n=255) == WORKSPACE
        assert call(b=0, bt=None) == OK
    assert free(done=FAR[1] + 4) == INVALID
    assert reserve(new=None) == INVALID
    assert reserve(N=100000, n=100000) == WORKSPACE


def test_kv_fork_and_compact_reject(L):  # noqa: F811
    def fork(t=_tensors(64, 64), n=2, refs=FAKE, N=10, bt=FAR[0], st=4, mb=4, cl=FAR[1], b=2, src=FAR[2], ct=FAR[3],
             cs=5, cb=5, chl=FAR[4], c=3, ws=FAKE, wn=1 << 20):
        return L.kv_fork(n, t, refs, N, bt, st, mb, cl, b, src, ct, cs, cb, chl, c, ws, wn, None)

    def compact(t=_tensors(64, 64), n=2, refs=FAKE, N=10, bt=FAR[0], st=4, mb=4, b=2, used=FAR[1], ws=FAKE, wn=1 << 20):
        return L.kv_compact(n, t, refs, N, bt, st, mb, b, used, ws, wn, None)
    for call in (fork, compact):
        assert call(t=None) == INVALID and call(n=-1) == INVALID and call(n=257) == UNSUPPORTED
        assert call(t=_tensors(64, 0)) == INVALID
        assert call(t=_tensors(64, 1 << 40)) == UNSUPPORTED
        null = _tensors(64, 64)
        null[1].data = None
        assert call(t=null) == INVALID
        assert call(refs=None) == INVALID and call(bt=None) == INVALID and call(N=0) == INVALID
        assert call(N=(1 << 20) + 1) == UNSUPPORTED and call(st=3) == INVALID
        assert call(ws=None) == WORKSPACE and call(N=100000, wn=100000) == WORKSPACE
    assert compact(used=None) == INVALID
    assert fork(cl=None) == INVALID and fork(src=None) == INVALID and fork(ct=None) == INVALID
    assert fork(chl=None) == INVALID and fork(cs=4) == INVALID and fork(cb=0) == INVALID and fork(c=-1) == INVALID
    assert fork(c=65536) == UNSUPPORTED
    assert fork(c=0) == OK
    # outputs over what is read
    assert fork(ct=FAR[0] + 16) == INVALID and fork(ct=FAR[0] - 56) == INVALID
    assert fork(chl=FAR[1] + 4) == INVALID and fork(chl=FAR[2] + 8) == INVALID and fork(ct=FAR[2] + 8) == INVALID
    assert fork(chl=FAR[3]) == INVALID and fork(chl=FAR[0]) == INVALID and fork(ct=FAR[1]) == INVALID


# --------------------------------------------------------------------------
# e4m3 cache
# --------------------------------------------------------------------------
def _f8(N=100, H=4, bs=16, D=128, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE):
    c = AttnKVCacheF8()
    c.k, c.v, c.k_scale, c.v_scale, c.num_blocks = k, v, ks, vs, N
    c.num_kv_heads, c.block_size, c.head_dim = H, bs, D
    return c


BAD_CACHES = [(dict(k=None), INVALID), (dict(vs=None), INVALID), (dict(N=0), INVALID), (dict(bs=32), UNSUPPORTED),
              (dict(D=96), UNSUPPORTED), (dict(k=FAKE + 8), INVALID), (dict(ks=FAKE + 2), INVALID), (dict(H=0), INVALID)]


def test_kv_append_f8_rejects(L):  # noqa: F811
    def call(c=None, k=None, v=None, bt=FAKE, st=10, mb=10, pos=FAKE, lens=None, ws=FAKE, n=256):
        c, k, v = c or _f8(), k or _t([2, 4, 5, 128]), v or _t([2, 4, 5, 128])
        return L.kv_append_f8(ctypes.byref(c), bt, st, mb, pos, lens, ctypes.byref(k), ctypes.byref(v), ws, n, None)
    for kw, want in BAD_CACHES:
        assert call(c=_f8(**kw)) == want, kw
    assert call(k=_t([2, 4, 6, 128])) == INVALID and call(k=_t([2, 3, 5, 128])) == INVALID
    assert call(k=_t([2, 4, 5, 64]), v=_t([2, 4, 5, 64])) == INVALID
    assert call(k=_t([2, 4, 5, 128], 0)) == UNSUPPORTED
    assert call(k=_t([2, 4, 128])) == INVALID
    assert call(v=_t([2, 4, 5, 128], data=FAKE + 2)) == INVALID
    assert call(k=_t([2, 4, 5, 128], stride=(2564, 641, 128, 1))) == INVALID
    assert call(bt=None) == INVALID and call(pos=None) == INVALID and call(st=9) == INVALID and call(mb=0) == INVALID
    assert call(ws=None) == WORKSPACE and call(n=0) == WORKSPACE
    assert call(k=_t([2, 4, 0, 128]), v=_t([2, 4, 0, 128])) == OK


def test_paged_attn_f8_rejects(L):  # noqa: F811
    def call(q=None, c=None, out=None, bt=FAKE, st=10, mb=10, pos=FAKE, scale=0.1, ws=FAKE, n=BIG):
        q, c = q or _t([2, 12, 6, 128]), c or _f8()
        out = out or _t(list(q.shape[:4]), data=FAR[0])
        return L.paged_attn_f8(ctypes.byref(q), ctypes.byref(c), bt, st, mb, pos, None, 1, scale, ctypes.byref(out),
                               None, ws, n, None)
    for kw, want in BAD_CACHES:
        assert call(c=_f8(**kw)) == want, kw
    assert call(q=_t([2, 12, 6, 128], 0)) == UNSUPPORTED
    assert call(q=_t([2, 12, 6, 64])) == INVALID and call(q=_t([2, 10, 6, 128])) == INVALID
    assert call(q=_t([2, 12, 128])) == INVALID
    assert call(out=_t([2, 12, 7, 128])) == INVALID
    assert call(q=_t([1, 129, 2, 128]), c=_f8(H=1)) == UNSUPPORTED
    assert call(c=_f8(N=1 << 30)) == UNSUPPORTED
    assert call(q=_t([65535, 65535, 1, 128]), c=_f8(H=65535)) == UNSUPPORTED  # more items than a grid has CTAs
    assert call(q=_t([2, 12, 6, 128], data=FAKE + 8)) == INVALID
    assert call(out=_t([2, 12, 6, 128], data=FAKE + 8)) == INVALID
    flat = _t([2, 12, 6, 128])
    flat.stride[1] = 0
    assert call(q=flat) == INVALID and call(out=flat) == INVALID
    assert call(scale=float("inf")) == INVALID
    assert call(bt=None) == INVALID and call(pos=None) == INVALID and call(st=9) == INVALID and call(mb=0) == INVALID
    assert call(ws=None) == WORKSPACE and call(n=255) == WORKSPACE
    assert call(q=_t([2, 12, 0, 128])) == OK and call(q=_t([0, 12, 6, 128])) == OK


def test_paged_attn_f8_sizes(L):  # noqa: F811
    size = L.paged_attn_f8_workspace_size
    assert size(0, 8, 8, 1, 10, 16, 128) == 256 and size(2, 8, 8, 0, 10, 16, 128) == 256
    assert size(2, 8, 3, 1, 10, 16, 128) == 0 and size(2, 8, 8, 1, 10, 32, 128) == 0 and size(-1, 8, 8, 1, 9, 16, 64) == 0
    assert size(64, 32, 8, 1, 513, 16, 128) % 256 == 0
    assert size(64, 32, 8, 1, 513, 16, 128) < 64 * 32 * 16 * 130 * 4 * 2  # a few partial rows a query row


# --------------------------------------------------------------------------
# the binding
# --------------------------------------------------------------------------
def _calls(ws):
    """Each call with the tensors that its kernels touch."""
    i32 = lambda *s: torch.ones(*s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    p, q, tok, par, u = torch.zeros(2, 3, 9), torch.zeros(2, 3, 9), i32(2, 3), i32(2, 3), torch.zeros(2, 3)
    refs, bt, n, ct, cl, src, done = i32(9), i32(2, 4), i32(2), i32(3, 4), i32(3), i32(3), i32(2)
    k, v = bf(9, 2, 16, 128), bf(9, 2, 16, 128)
    kq, vq, ks, vs = k.to(F8), v.to(F8), torch.zeros(9, 2), torch.zeros(9, 2)
    kn, qq = bf(2, 2, 3, 128), bf(2, 8, 3, 128)
    kw = dict(workspace=ws, stream=0)
    return [
        ("draft_verify", lambda: lib.draft_verify(p, tok, par, u, draft_probs=q, **kw), (p, q, tok, par, u)),
        ("kv_free", lambda: lib.kv_free(refs, bt, n, done, **kw), (refs, bt, n, done)),
        ("kv_reserve", lambda: lib.kv_reserve(refs, bt, n, done, **kw), (refs, bt, n, done)),
        ("kv_fork", lambda: lib.kv_fork([k, v, ks], refs, bt, n, src, ct, cl, **kw), (k, v, ks, refs, bt, n, src, ct, cl)),
        ("kv_compact", lambda: lib.kv_compact([k, kq], refs, bt, **kw), (k, kq, refs, bt)),
        ("kv_append_f8", lambda: lib.kv_append_f8(kq, vq, ks, vs, bt, n, kn, kn, lens=done, **kw),
         (kq, vq, ks, vs, bt, n, kn, done)),
        ("paged_attn_f8", lambda: lib.paged_attn_f8(qq, kq, vq, ks, vs, bt, n, lens=done, return_lse=True, **kw),
         (qq, kq, vq, ks, vs, bt, n, done)),
    ]


def test_every_call_is_marshalled(rec):  # noqa: F811
    for ws in (lib.Workspace(1 << 20, device="cpu"), None):
        for name, call, _ in _calls(ws):
            call()
            assert name in rec.calls
    kq, sc, bt, n = torch.zeros(9, 2, 16, 64).to(F8), torch.zeros(9, 2), torch.ones(2, 4, dtype=torch.int32), \
        torch.ones(2, dtype=torch.int32)
    one = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    lib.kv_append_f8(kq, kq, sc, sc, bt, n, one, one, stream=0)
    out, lse = lib.paged_attn_f8(torch.zeros(2, 4, 64, dtype=torch.bfloat16), kq, kq, sc, sc, bt, n, return_lse=True,
                                 stream=0)
    assert out.shape == (2, 4, 64) and lse.shape == (2, 4)
    path, acc, nxt = lib.draft_verify(torch.zeros(2, 3, 9), torch.ones(2, 3, dtype=torch.int32),
                                      torch.ones(2, 3, dtype=torch.int32), torch.zeros(2, 3), stream=0)
    assert path.shape == (2, 3) and acc.shape == nxt.shape == (2,)


def test_devices_are_checked(rec, monkeypatch):  # noqa: F811
    seen = {}
    monkeypatch.setattr(lib, "_check_devices", lambda name, *t: seen.setdefault(name, []).extend(t))
    ws = lib.Workspace(1 << 20, device="cpu")
    for name, call, tensors in _calls(ws):
        call()
        for t in (*tensors, ws.tensor):
            assert any(t is x or (isinstance(x, torch.Tensor) and x.data_ptr() == t.data_ptr()) for x in seen[name]), name


def test_a_workspace_off_the_gpu_is_refused(rec, monkeypatch):  # noqa: F811
    ws = lib.Workspace(1 << 20, device="cpu")
    monkeypatch.setattr(lib, "_on_device", lambda t: t is not ws.tensor)
    for name, call, _ in _calls(ws):
        with pytest.raises(ValueError, match="workspace must be on a CUDA device"):
            call()
    assert not [c for c in rec.calls if not c.endswith("size")]


def test_the_binding_refuses(rec):  # noqa: F811
    i32 = lambda *s: torch.ones(*s, dtype=torch.int32)  # noqa: E731
    p, tok, u = torch.zeros(2, 3, 9), i32(2, 3), torch.zeros(2, 3)

    def refused(match, f, *a, **k):
        with pytest.raises(ValueError, match=match):
            f(*a, **k, stream=0)

    refused("target_probs must be float32 or bfloat16", lib.draft_verify, p.half(), tok, tok, u)
    refused(r"tokens must be \[2, 3\]", lib.draft_verify, p, i32(2, 4), tok, u)
    refused("parents must be int32", lib.draft_verify, p, tok, tok.long(), u)
    refused("uniforms must be float32", lib.draft_verify, p, tok, tok, u.double())
    refused("uniforms must be float32", lib.draft_verify, p, tok, tok, u[:1])
    refused("draft_probs must be", lib.draft_verify, p, tok, tok, u, draft_probs=p[0])
    refused("path must be contiguous", lib.draft_verify, p, tok, tok, u, path=i32(2, 4))
    refused("next_token must be", lib.draft_verify, p, tok, tok, u, next_token=i32(3))
    refs, bt, n = i32(9), i32(2, 4), i32(2)
    refused("refs must be", lib.kv_free, refs.long(), bt, n)
    refused("block_table must be int32", lib.kv_free, refs, bt.t(), n)
    refused("done must be", lib.kv_free, refs, bt, n, i32(3))
    refused("n_new must be", lib.kv_reserve, refs, bt, n, i32(1))
    refused(r"block_table must be int32 \[rows", lib.kv_reserve, refs, bt[:1].expand(2, 4), n, n)
    cache = torch.zeros(9, 4)
    refused("with 9 blocks", lib.kv_fork, [cache[:8]], refs, bt, n, n, i32(2, 4), i32(2))
    refused("must be contiguous", lib.kv_fork, [torch.zeros(9, 8)[:, ::2]], refs, bt, n, n, i32(2, 4), i32(2))
    refused("src must be", lib.kv_fork, [cache], refs, bt, n, i32(3), i32(2, 4), i32(2))
    refused("child_lens must be", lib.kv_fork, [cache], refs, bt, n, n, i32(2, 4), i32(1))
    refused("used must be", lib.kv_compact, [cache], refs, bt, i32(2))
    kq, sc = torch.zeros(9, 2, 16, 64).to(F8), torch.zeros(9, 2)
    rows = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16)
    refused("must be float8_e4m3fn", lib.kv_append_f8, kq.view(torch.uint8), kq, sc, sc, bt, n, rows, rows)
    refused("block scales must be", lib.kv_append_f8, kq, kq, sc, torch.zeros(9, 2, 16), bt, n, rows, rows)
    refused("block scales must be", lib.kv_append_f8, kq, kq, sc.double(), sc, bt, n, rows, rows)
    refused("contiguous CUDA", lib.kv_append_f8, kq, kq, torch.zeros(2, 9).t(), sc, bt, n, rows, rows)
    refused("lens must be", lib.kv_append_f8, kq, kq, sc, sc, bt, n, rows, rows, lens=i32(3))
    refused("q must be", lib.paged_attn_f8, rows[0, 0], kq, kq, sc, sc, bt, n)
    refused("out must be", lib.paged_attn_f8, rows, kq, kq, sc, sc, bt, n, out=rows[:1])
    refused("lse must hold", lib.paged_attn_f8, rows, kq, kq, sc, sc, bt, n, lse=torch.zeros(5))
    refused("start_pos must be", lib.paged_attn_f8, rows, kq, kq, sc, sc, bt, n.long())
    assert not [c for c in rec.calls if not c.endswith("size")]
