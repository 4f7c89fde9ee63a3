"""Host side of the token-mixing calls without a GPU: angular speeds, and the
refusals that need no handle."""
import ctypes
import math

import pytest

import q4_quantized_decode_b200 as q4


def test_rope_freqs_plain_and_linear():
    st, f = q4.q4gemv_rope_freqs(q4.ROPE_PLAIN, 16, 10000.0)
    assert st == q4.Q4_OK and len(f) == 8
    for i, w in enumerate(f):
        assert w == pytest.approx(10000.0 ** (-i / 8), rel=1e-15)
    st, g = q4.q4gemv_rope_freqs(q4.ROPE_LINEAR, 16, 10000.0, 4.0)
    assert st == q4.Q4_OK and g == [w / 4 for w in f]


def test_rope_freqs_by_parts():
    """Pairs that turn more than `hi` times in the trained length keep their
    speed, pairs under `lo` turns are slowed by the factor, between them the
    mix is linear in the turns."""
    rot, base, factor, trained, lo, hi = 64, 1e6, 8.0, 32768.0, 1.0, 32.0
    _, plain = q4.q4gemv_rope_freqs(q4.ROPE_PLAIN, rot, base)
    st, f = q4.q4gemv_rope_freqs(q4.ROPE_BY_PARTS, rot, base, factor, trained, lo, hi)
    assert st == q4.Q4_OK
    kinds = set()
    for w, x in zip(plain, f):
        turns = trained * w / (2 * math.pi)
        if turns >= hi:
            kinds.add("kept")
            assert x == w
        elif turns <= lo:
            kinds.add("slowed")
            assert x == pytest.approx(w / factor, rel=1e-15)
        else:
            kinds.add("mixed")
            keep = (turns - lo) / (hi - lo)
            assert x == pytest.approx(w * (keep + (1 - keep) / factor), rel=1e-13)
    assert kinds == {"kept", "slowed", "mixed"}


@pytest.mark.parametrize("args,status", [
    ((3, 16, 1e4), q4.Q4_EINVAL), ((-1, 16, 1e4), q4.Q4_EINVAL),
    ((0, 15, 1e4), q4.Q4_ESHAPE), ((0, -2, 1e4), q4.Q4_ESHAPE), ((0, 258, 1e4), q4.Q4_ESHAPE),
    ((0, 16, 0.0), q4.Q4_EINVAL), ((0, 16, math.inf), q4.Q4_EINVAL), ((0, 16, math.nan), q4.Q4_EINVAL),
    ((1, 16, 1e4, 0.5), q4.Q4_EINVAL), ((1, 16, 1e4, math.nan), q4.Q4_EINVAL),
    ((2, 16, 1e4, 2.0, 0.0, 1.0, 32.0), q4.Q4_EINVAL), ((2, 16, 1e4, 2.0, 4096.0, 32.0, 32.0), q4.Q4_EINVAL),
    ((2, 16, 1e4, 2.0, math.inf, 1.0, 32.0), q4.Q4_EINVAL),
])
def test_rope_freqs_refusals(args, status):
    assert q4.q4gemv_rope_freqs(*args)[0] == status


def test_rope_freqs_edges():
    assert q4.q4gemv_rope_freqs(0, 0, 1e4) == (q4.Q4_OK, [])
    assert q4.q4gemv_rope_freqs(0, 2, 1e4) == (q4.Q4_OK, [1.0])
    assert q4.lib.q4gemv_rope_freqs(0, 16, 1e4, 1.0, 0.0, 0.0, 0.0, None) == q4.Q4_EINVAL


def test_null_handles_are_refused():
    A = 1 << 20
    kv = q4.q4gemv_kv(A, A, A, 1, 16, 1, 64, 1024, 64, 64, 1, 1, q4.F16)
    r = ctypes.byref(kv)
    assert q4.q4gemv_kv_append(None, r, 1, 1, A, A, None, None, None, 0, 0, A, 64, A, 64, None, 0, None) == q4.Q4_EINVAL
    assert q4.q4gemv_attn_paged(None, r, 1, 1, A, A, 1, A, 64, 1, A, 64, 1.0, 1, 0, None) == q4.Q4_EINVAL
    assert q4.q4gemv_linattn(None, q4.q4gemv_linattn_args(), 1, 1, A, 1, None) == q4.Q4_EINVAL


def test_status_text():
    assert q4.Q4_EINDEX == -10 and q4.q4gemv_strerror(q4.Q4_EINDEX) != "unknown status"
