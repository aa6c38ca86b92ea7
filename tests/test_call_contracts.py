"""What the rotary, tree, weight and eviction calls promise about their arguments
beside shapes and types, without a GPU: which outputs may be which inputs."""
import ctypes
import sysconfig

import pytest
import torch

import masked_attention_paged_gb300 as lib
from masked_attention_paged_gb300 import build
from test_binding_marshalling import rec  # noqa: F401  (fixture)
from test_boundary import FAKE, INVALID, L, _cache, _t  # noqa: F401


def test_evict_refuses_lengths_that_overlap_in_part(L):  # noqa: F811
    """new_lens may be ctx_lens, or lie beside it; shifted by an entry, sequence b would write b + 1's length."""
    def call(cl, nl, kept, b=4):
        c = _cache()
        return L.kv_evict(ctypes.byref(c), FAKE, FAKE, 10, 10, cl, FAKE, 4, 4, b, 60, 4, 8, nl, kept, FAKE, 256, None)
    far = FAKE + (1 << 30)
    for shift in (-12, -4, 4, 12):
        assert call(FAKE, FAKE + shift, far) == INVALID, shift
    # the kept slots over either of the lengths: 4 x 4 x 60 of them begin up to 3840 bytes ahead
    kept_bytes = 4 * 4 * _cache().num_kv_heads * 60
    for at in (FAKE, FAKE + 12, FAKE - kept_bytes + 4):
        assert call(FAKE, FAKE + 16, at) == INVALID
        assert call(FAKE + 16, FAKE, at) == INVALID
        assert call(FAKE, FAKE, at) == INVALID


def test_the_compiled_caller_is_told_apart_by_interpreter(monkeypatch):
    """Compiled against one Python's object layouts, it is not what another one loads from the same tree."""
    here, var = build.marshal_path(), sysconfig.get_config_var
    assert sysconfig.get_config_var("SOABI") in here
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-399-other" if n == "SOABI" else var(n))
    assert build.marshal_path() != here
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: None if n == "SOABI" else var(n))
    assert build.marshal_path().endswith(".so") and "None" not in build.marshal_path()


@pytest.mark.parametrize("scaling,high", [("banded", 4.0), ("ramp", 32.0)])
def test_rope_frequencies_blend_as_models_of_each_kind_do_unless_told(scaling, high):
    kw = dict(scaling=scaling, factor=8.0, original_len=8192, device="cpu")
    got, m = lib.rope_frequencies(128, **kw)
    want, n = lib.rope_frequencies(128, high=high, **kw)
    assert torch.equal(got, want) and m == n
    other, _ = lib.rope_frequencies(128, high=36.0 - high, **kw)
    assert not torch.equal(got, other)


FAR = FAKE + (1 << 30)  # another buffer


def _rope(L, x, out):  # noqa: F811
    return L.rope_apply(ctypes.byref(x), FAKE, 5, FAKE, 64, 0, 0, 1.0, ctypes.byref(out), None)


def test_rows_of_an_output_must_be_apart(L):  # noqa: F811
    """A broadcast output has rows that several threads write; in place they would be rotated several times."""
    shape, row = (2, 4, 5, 128), (2560, 640, 128, 1)
    for i in range(3):
        flat = _t(shape, stride=[0 if j == i else v for j, v in enumerate(row)], data=FAR)
        assert _rope(L, _t(shape), flat) == INVALID, i
        assert _rope(L, flat, flat) == INVALID, i
        c = _cache(H=4)
        assert L.rope_kv_append(*(ctypes.byref(_t(shape)) for _ in range(3)), FAKE, 5, FAKE,
                                64, 0, 1.0, ctypes.byref(flat), ctypes.byref(c), FAKE, 10, 10, FAKE, FAKE, 256,
                                None) == INVALID, i
        assert L.paged_tree_attn(ctypes.byref(_t(shape)), None, None, ctypes.byref(c), FAKE, 10, 10, FAKE,
                                 FAKE, 5, 0.1, ctypes.byref(flat), None, FAKE, 1 << 30, None) == INVALID, i


def test_a_rotation_in_place_has_the_same_rows(L):  # noqa: F811
    shape = (2, 4, 5, 128)
    assert _rope(L, _t(shape), _t(shape, stride=(2560, 128, 512, 1))) == INVALID


def _calls(ws):
    """Each call that checks devices, with its caches: (name, the call, tensors that its kernels touch)."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.ones(*s, dtype=torch.int32)  # noqa: E731
    q, kn, k, v, acc = bf(2, 8, 3, 128), bf(2, 2, 3, 128), bf(9, 2, 16, 128), bf(9, 2, 16, 128), torch.zeros(9, 2, 16)
    kq, vq, ks, vs = k.to(torch.int8), v.to(torch.int8), torch.zeros(9, 2, 16), torch.zeros(9, 2, 16)
    bt, dt, n, pos, fr = i32(2, 4), i32(2, 4), i32(2), i32(2, 3), torch.ones(64, dtype=torch.int64)
    lse = torch.zeros(2, 8, 3)
    kw = dict(workspace=ws, stream=0)
    return [
        ("rope_kv_append", lambda: lib.rope_kv_append(q, kn, kn, pos, fr, k, v, bt, n, **kw), (k, v, bt, pos, fr)),
        ("rope_kv_append_q8", lambda: lib.rope_kv_append_q8(q, kn, kn, pos, fr, kq, vq, ks, vs, bt, n, **kw),
         (kq, vq, ks, vs, bt)),
        ("paged_tree_attn", lambda: lib.paged_tree_attn(q, k, v, bt, n, pos, k_new=kn, v_new=kn, **kw), (k, v, pos)),
        ("kv_tree_accept", lambda: lib.kv_tree_accept(k, v, bt, n, pos, n, **kw), (k, v, bt, pos)),
        ("paged_attn_weights", lambda: lib.paged_attn_weights(q, lse, k, bt, n, acc, **kw), (k, lse, acc)),
        ("kv_evict", lambda: lib.kv_evict(k, v, acc, bt, n, dt, 5, **kw), (k, v, acc, bt, dt)),
    ]


def test_caches_and_workspaces_are_held_to_the_current_device(rec, monkeypatch):  # noqa: F811
    """A kernel of one device that reads a cache or writes a workspace of another faults."""
    seen = {}
    monkeypatch.setattr(lib, "_check_devices", lambda name, *t: seen.setdefault(name, []).extend(t))
    ws = lib.Workspace(1 << 20, device="cpu")
    for name, call, tensors in _calls(ws):
        call()
        for t in (*tensors, ws.tensor):
            assert any(t is x for x in seen[name]), (name, tuple(t.shape))


def test_a_workspace_off_the_gpu_is_refused(rec, monkeypatch):  # noqa: F811
    ws = lib.Workspace(1 << 20, device="cpu")
    monkeypatch.setattr(lib, "_on_device", lambda t: t is not ws.tensor)
    for name, call, _ in _calls(ws):
        with pytest.raises(ValueError, match="workspace must be on a CUDA device"):
            call()
    assert not set(rec.calls) - {"paged_tree_workspace_size", "paged_attn_weights_workspace_size"}


@pytest.mark.parametrize("kw", [dict(sink=1 << 32), dict(recent=(1 << 32) + 2), dict(sink=-(1 << 40)),
                                dict(keep=1 << 31)])
def test_evict_counts_past_32_bits_are_refused(rec, kw):  # noqa: F811
    """Their low 32 bits are counts like any other: no sinks, two recent tokens."""
    k, acc = torch.zeros(9, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(9, 2, 16)
    bt, n = torch.ones(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be 32-bit integers"):
        lib.kv_evict(k, k, acc, bt, n, bt, **{"keep": 5, **kw}, stream=0)
    assert not rec.calls


def test_two_first_calls_at_once_share_one_default_workspace(rec, monkeypatch):  # noqa: F811
    """What either notes in the status word is noted for all: neither's workspace is lost."""
    import threading
    made, both = lib.Workspace, threading.Barrier(2)

    def slowly(*a, **k):
        both.wait(20)  # neither is kept before both are made
        return made(*a, **k)

    monkeypatch.setattr(lib, "Workspace", slowly)
    got = [None, None]

    def go(i):
        got[i] = lib._small_ws("cpu")

    threads = [threading.Thread(target=go, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert got[0] is got[1] is lib._small_ws("cpu")
