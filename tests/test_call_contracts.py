"""What the rotary, tree, weight and eviction calls promise about their arguments
beside shapes and types, without a GPU: which outputs may be which inputs."""
import ctypes

from test_boundary import FAKE, INVALID, L, _cache  # noqa: F401


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
