"""What the rotated append takes and refuses on the host, beyond single arguments (no GPU needed)."""

from paged_kv_attention_32_gb300 import _lib as L
from tests.test_pages_binding import rope


def test_no_tokens_need_no_positions():
    """The address of an empty tensor is NULL."""
    none = dict(T=0, k=None, v=None, slots=None, pos=None, kp=None, vp=None)
    assert rope(**none) == L.PKA_OK
    assert rope(**none, Hq=0, q=None, q_out=None) == L.PKA_OK
    # what the call would rotate by is looked at all the same
    for kw in (dict(freq=None), dict(sections=None), dict(axes=0), dict(pairs=2)):
        assert rope(**(none | kw)) == L.PKA_ERR_INVALID_ARG
