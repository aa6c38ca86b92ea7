"""What the rotary, tree, weight and eviction calls promise about their arguments
beside shapes and types, without a GPU: which outputs may be which inputs."""
import ctypes
import sysconfig

import pytest
import torch

import masked_attention_paged_gb300 as lib
from masked_attention_paged_gb300 import build
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
