"""Limits of the packed-batch entry points (nothing is launched: CPU only)."""
from test_packed_host import APPEND, CHUNK, INVALID, OK, PROMPT, UNSUPPORTED, _call, _i64  # noqa: F401


def test_append_refuses_pages_that_32_bits_cannot_index():
    # rows x features of a page; 2^25 x 128 is 0 in 32 bits (a division on the host)
    for P, D in ((1 << 25, 128), (1 << 24, 128), (1 << 27, 16), (1 << 23, 256), (1 << 28, 8)):
        assert _call("sa_append_kv_rope", APPEND, P=P, D=D, rot=0, max_pages=1) == UNSUPPORTED
