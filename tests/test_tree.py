"""Tree attention and path acceptance without a GPU: sizes, refusals, marshalling."""
import ctypes

import pytest
import torch

import masked_attention_paged_gb300 as lib
from test_binding_marshalling import rec  # noqa: F401  (fixture)
from test_boundary import FAKE, INVALID, L, OK, UNSUPPORTED, WORKSPACE, _cache, _t  # noqa: F401

BIG = 1 << 30


def test_workspace_size(L):
    size = lambda *a: L.paged_tree_workspace_size(*a, 64, 16, 128)  # noqa: E731  (batch, Hq, Hkv, T)
    assert size(4, 32, 8, 0) >= 256 and size(4, 32, 8, 8) % 256 == 0
    assert size(64, 32, 8, 25) == size(4, 32, 8, 25) >= size(4, 32, 8, 8)
    assert size(4, 30, 8, 8) == 0 and size(-1, 32, 8, 8) == 0 and size(4, 32, 0, 8) == 0
    # the context's length does not matter: what is cut is bounded by the SMs
    a = L.paged_tree_workspace_size(4, 32, 8, 8, 100, 16, 128)
    assert a == L.paged_tree_workspace_size(4, 32, 8, 8, 100000, 16, 128)


def test_paged_tree_rejects(L):
    def call(q=None, k=None, v=None, c=None, cl=FAKE, par=FAKE, ps=6, out=None, ws=FAKE, ws_bytes=BIG, scale=0.1,
             bt=FAKE, bts=10, mb=10):
        q = q or _t([2, 12, 6, 128])
        out = out or _t([2, 12, 6, 128])
        c = c or _cache(H=4)
        return L.paged_tree_attn(ctypes.byref(q), None if k is None else ctypes.byref(k),
                                 None if v is None else ctypes.byref(v), ctypes.byref(c), bt, bts, mb, cl, par, ps,
                                 scale, ctypes.byref(out), None, ws, ws_bytes, None)
    kn = _t([2, 4, 6, 128])
    assert call(k=kn) == INVALID  # k_new without v_new
    assert call(k=_t([2, 4, 5, 128]), v=_t([2, 4, 5, 128])) == INVALID
    assert call(k=_t([2, 8, 6, 128]), v=_t([2, 8, 6, 128])) == INVALID
    assert call(k=kn, v=_t([2, 4, 6, 128], 0)) == INVALID
    assert call(k=kn, v=_t([2, 4, 6, 128], data=FAKE + 2)) == INVALID
    assert call(q=_t([2, 12, 6, 128], 0), out=_t([2, 12, 6, 128], 0)) == UNSUPPORTED
    assert call(q=_t([2, 12, 6, 64]), out=_t([2, 12, 6, 64])) == INVALID
    assert call(q=_t([2, 10, 6, 128]), out=_t([2, 10, 6, 128])) == INVALID  # 10 % 4
    assert call(q=_t([2, 12, 257, 128]), out=_t([2, 12, 257, 128]), ps=257) == UNSUPPORTED
    # 128 x 4 (sequence, KV head)s of 2^21 tiles are counted in 31 bits, three row groups of each are not
    wide = lambda t: _t([128, 12, t, 128])  # noqa: E731
    assert call(q=wide(6), out=wide(6), bts=1 << 24, mb=1 << 24) != UNSUPPORTED
    assert call(q=wide(256), out=wide(256), ps=256, bts=1 << 24, mb=1 << 24) == UNSUPPORTED
    assert call(out=_t([2, 12, 7, 128])) == INVALID
    assert call(q=_t([2, 12, 6, 128], data=FAKE + 8)) == INVALID
    assert call(out=_t([2, 12, 6, 128], data=FAKE + 8)) == INVALID
    flat = _t([2, 12, 6, 128])
    flat.stride[1] = 0  # one row for all heads
    assert call(q=flat) == INVALID
    assert call(k=kn, v=kn) != INVALID
    one = _t([2, 4, 6, 128])
    one.stride[0] = 0
    assert call(k=kn, v=one) == INVALID
    assert call(scale=float("nan")) == INVALID
    assert call(cl=None) == INVALID
    assert call(par=None) == INVALID
    assert call(ps=5) == INVALID
    assert call(ps=-6) == INVALID
    assert call(bt=None) == INVALID
    assert call(bts=9) == INVALID
    assert call(mb=0) == INVALID
    assert call(c=_cache(H=4, bs=32)) == UNSUPPORTED
    assert call(c=_cache(H=4, D=96)) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE
    assert call(ws=FAKE + 16) == WORKSPACE
    assert call(ws_bytes=128) == WORKSPACE  # without a GPU there are no SMs to size partials for
    assert call(q=_t([2, 12, 0, 128]), out=_t([2, 12, 0, 128])) == OK  # no drafts: nothing launched


def test_tree_accept_rejects(L):
    def call(c=None, bt=FAKE, bts=10, mb=10, cl=FAKE, path=FAKE, ps=8, mp=8, n=FAKE, b=2, ws=FAKE):
        c = c or _cache()
        return L.kv_tree_accept(ctypes.byref(c), bt, bts, mb, cl, path, ps, mp, n, b, ws, 256, None)
    assert call(c=_cache(dtype=0)) == UNSUPPORTED
    assert call(bt=None) == INVALID
    assert call(cl=None) == INVALID
    assert call(path=None) == INVALID
    assert call(n=None) == INVALID
    assert call(bts=9) == INVALID
    assert call(ps=7) == INVALID
    assert call(mb=0) == INVALID
    assert call(mp=-1) == INVALID
    assert call(b=-1) == INVALID
    assert call(b=65536) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE
    assert call(mp=0) == OK and call(b=0) == OK


def test_binding_checks():
    q = torch.zeros(2, 8, 3, 128, dtype=torch.bfloat16)
    kc = torch.zeros(10, 2, 16, 128, dtype=torch.bfloat16)
    bt, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    par = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="parents must be int32"):
        lib.paged_tree_attn(q, kc, kc, bt, lens, par.long())
    with pytest.raises(ValueError, match=r"parents must be \[2, 3\]"):
        lib.paged_tree_attn(q, kc, kc, bt, lens, par[:, :2].contiguous())
    with pytest.raises(ValueError, match=r"parents must be \[2, n\]"):
        lib.paged_tree_attn(q, kc, kc, bt, lens, par[:1])
    with pytest.raises(ValueError, match=r"ctx_lens must be contiguous \[2\]"):
        lib.paged_tree_attn(q, kc, kc, bt, lens[:1], par)
    with pytest.raises(ValueError, match="lse must hold 48 elements"):
        lib.paged_tree_attn(q, kc, kc, bt, lens, par, lse=torch.zeros(2, 8))
    with pytest.raises(ValueError, match="path must be int32"):
        lib.kv_tree_accept(kc, kc, bt, lens, par.float(), lens)
    with pytest.raises(ValueError, match=r"n_accept must be contiguous \[2\]"):
        lib.kv_tree_accept(kc, kc, bt, lens, par, lens[:1])


def test_marshalling(rec):  # noqa: F811
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    q, kc, kn = bf(2, 8, 3, 128), bf(10, 2, 16, 128), bf(2, 2, 3, 128)
    bt, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    par = torch.zeros(2, 3, dtype=torch.int32)
    ws = lib.Workspace(4096, device="cpu")
    out, lse = lib.paged_tree_attn(q, kc, kc, bt, lens, par, k_new=kn, v_new=kn, return_lse=True, workspace=ws, stream=0)
    assert out.shape == q.shape and lse.shape == (2, 8, 3)
    lib.paged_tree_attn(q, kc, kc, bt, lens, par, out=out, workspace=ws, stream=0)
    lib.kv_tree_accept(kc, kc, bt, lens, par, lens, stream=0)
    assert rec.calls == ["paged_tree_attn", "paged_tree_attn", "kv_tree_accept"]
