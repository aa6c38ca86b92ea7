"""Attention weights and eviction without a GPU: sizes, refusals, marshalling."""
import ctypes

import pytest
import torch

import masked_attention_paged_gb300 as lib
from test_binding_marshalling import rec  # noqa: F401  (fixture)
from test_boundary import FAKE, INVALID, L, OK, UNSUPPORTED, WORKSPACE, _cache, _t  # noqa: F401


def test_workspace_size(L):
    a, b, c = (L.paged_attn_weights_workspace_size(8, 8, m, 16) for m in (1600, 3200, 4800))
    assert a % 256 == 0 and b - a == c - b == 8 * 8 * 100 * 8  # an 8-byte count per 256 tokens and KV head
    assert L.paged_attn_weights_workspace_size(-1, 8, 10, 16) == 0
    assert L.paged_attn_weights_workspace_size(1, 8, 10, 32) == 0


def test_paged_attn_weights_rejects(L):
    def call(q=None, lse=FAKE, c=None, bt=FAKE, bts=10, mb=10, sp=FAKE, ql=None, causal=1, scale=0.1, acc=FAKE,
             ws=FAKE, ws_bytes=1 << 30):
        q = q or _t([2, 12, 6, 128])
        c = c or _cache(H=4)
        return L.paged_attn_weights(ctypes.byref(q), lse, ctypes.byref(c), bt, bts, mb, sp, ql, causal, scale, acc, ws,
                                    ws_bytes, None)
    assert call(q=_t([2, 12, 6, 128], 0)) == UNSUPPORTED
    assert call(q=_t([2, 12, 128])) == INVALID
    assert call(q=_t([2, 12, 6, 64])) == INVALID
    assert call(q=_t([2, 10, 6, 128])) == INVALID  # 10 % 4
    assert call(q=_t([2, 12, 6, 128], data=FAKE + 8)) == INVALID
    assert call(q=_t([2, 12, 1 << 25, 128])) == UNSUPPORTED
    assert call(lse=None) == INVALID and call(lse=FAKE + 2) == INVALID
    assert call(acc=None) == INVALID and call(acc=FAKE + 2) == INVALID
    assert call(sp=None) == INVALID
    assert call(bt=None) == INVALID
    assert call(bts=9) == INVALID
    assert call(mb=0) == INVALID
    assert call(causal=2) == INVALID
    assert call(scale=float("inf")) == INVALID
    assert call(c=_cache(H=4, D=96)) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(ws_bytes=256) == WORKSPACE
    assert call(q=_t([2, 12, 0, 128])) == OK  # no queries: nothing launched


def test_kv_evict_rejects(L):
    def call(c=None, acc=FAKE, bt=FAKE, bts=10, mb=10, cl=FAKE, dt=FAKE, dts=4, db=4, b=2, keep=60, sink=4, recent=8,
             nl=FAKE, kept=FAKE, ws=FAKE):
        c = c or _cache()
        return L.kv_evict(ctypes.byref(c), acc, bt, bts, mb, cl, dt, dts, db, b, keep, sink, recent, nl, kept, ws, 256,
                          None)
    for bad in (dict(acc=None), dict(acc=FAKE + 2), dict(bt=None), dict(cl=None), dict(dt=None), dict(nl=None),
                dict(kept=None), dict(bts=9), dict(dts=3), dict(mb=0), dict(db=0), dict(b=-1), dict(keep=0),
                dict(sink=-1), dict(recent=-1), dict(sink=50, recent=11)):
        assert call(**bad) == INVALID, bad
    assert call(b=65536) == UNSUPPORTED
    assert call(c=_cache(bs=32)) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE
    assert call(b=0) == OK


def _args():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    return (bf(2, 8, 3, 128), torch.zeros(2, 8, 3), bf(10, 2, 16, 128), torch.zeros(2, 4, dtype=torch.int32),
            torch.ones(2, dtype=torch.int32), torch.zeros(10, 2, 16))


def test_binding_checks():
    q, lse, kc, bt, one, acc = _args()
    with pytest.raises(ValueError, match="lse must hold 48 elements"):
        lib.paged_attn_weights(q, lse[:, :4].contiguous(), kc, bt, one, acc)
    with pytest.raises(ValueError, match="start_pos must be int32"):
        lib.paged_attn_weights(q, lse, kc, bt, one.long(), acc)
    with pytest.raises(ValueError, match=r"q_lens must be contiguous \[2\]"):
        lib.paged_attn_weights(q, lse, kc, bt, one, acc, q_lens=one[:1])
    with pytest.raises(ValueError, match="K and V caches must be on a CUDA device"):
        lib.paged_attn_weights(q, lse, kc, bt, one, acc)
    with pytest.raises(ValueError, match="dst_block_table must be int32"):
        lib.kv_evict(kc, kc, acc, bt, one, bt.long(), 10)


def test_marshalling(rec):  # noqa: F811
    q, lse, kc, bt, one, acc = _args()
    ws = lib.Workspace(4096, device="cpu")
    assert lib.paged_attn_weights(q, lse, kc, bt, one, acc, workspace=ws, stream=0) is acc
    lib.paged_attn_weights(q[:, :, 0], lse[:, :, 0].contiguous(), kc, bt, one, acc, q_lens=one, causal=False,
                           workspace=ws, stream=0)
    nl, kept = lib.kv_evict(kc, kc, acc, bt, one, bt, 10, sink=1, recent=2, stream=0)
    assert nl.shape == (2,) and kept.shape == (2, 2, 10)
    with pytest.raises(ValueError, match="acc must be contiguous float32"):
        lib.kv_evict(kc, kc, acc[:5], bt, one, bt, 10, stream=0)
    with pytest.raises(ValueError, match="kept must be contiguous int32"):
        lib.kv_evict(kc, kc, acc, bt, one, bt, 10, kept=kept[:, :, :9], stream=0)
    assert rec.calls == ["paged_attn_weights", "paged_attn_weights", "kv_evict"]
