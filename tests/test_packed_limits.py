"""Limits of the packed-batch entry points (nothing is launched: CPU only)."""
import ctypes

from test_packed_host import APPEND, CHUNK, INVALID, PROMPT, UNSUPPORTED, _call

OTHER = ctypes.c_void_p(0x2000)


def test_append_refuses_pages_that_32_bits_cannot_index():
    # rows x features of a page; 2^25 x 128 is 0 in 32 bits (a division on the host)
    for P, D in ((1 << 25, 128), (1 << 24, 128), (1 << 27, 16), (1 << 23, 256), (1 << 28, 8)):
        assert _call("sa_append_kv_rope", APPEND, P=P, D=D, rot=0, max_pages=1) == UNSUPPORTED


def test_dense_attention_refuses_an_output_that_is_an_input():
    # (the other pointers are fakes too: the refusal comes before anything is launched)
    assert _call("sa_chunk_attention", CHUNK) == INVALID           # o is q
    for kw in (dict(q=OTHER), dict(q=OTHER, k=OTHER), dict(q=OTHER, v=OTHER)):   # o is k and v, v, k
        assert _call("sa_chunk_attention", CHUNK, **kw) == INVALID
        assert _call("sa_prompt_attention", PROMPT, **kw) == INVALID
    assert _call("sa_prompt_attention", PROMPT) == INVALID


def test_dense_attention_refuses_a_scale_whose_base_2_form_is_infinite():
    for name, base in (("sa_chunk_attention", CHUNK), ("sa_prompt_attention", PROMPT)):
        for scale in (2.4e38, 3.4e38):
            assert _call(name, base, scale=scale, q=OTHER, k=OTHER, v=OTHER, total=1 << 28) == INVALID
        assert _call(name, base, scale=2.3e38, total=1 << 28) == UNSUPPORTED   # the next check's
