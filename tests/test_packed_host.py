"""The packed-batch entry points' refusals (nothing is launched: CPU only) and pins of
the oracle's rotation and dense attention to other statements of the same definitions."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O
import paged_sparse_kv_sa_b200 as sa

FAKE = ctypes.c_void_p(0x1000)      # never dereferenced: validation fails first
BIG = 1 << 40
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def _i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


QS, KS = _i64(1024, 128, 1), _i64(4096, 2048, 128, 1)
CHUNK = dict(q=FAKE, qs=QS, cu=FAKE, total=4, k=FAKE, ks=KS, v=FAKE, vs=KS, pt=FAKE, max_pages=8, sl=FAKE, B=2, Hq=8,
             Hkv=2, D=128, P=16, pool=64, scale=0.1, window=0, o=FAKE, lse=None, ws=FAKE, ws_bytes=BIG, err=None,
             stream=None)
PROMPT = dict(q=FAKE, qs=QS, cu=FAKE, total=4, k=FAKE, ks=_i64(256, 128, 1), v=FAKE, vs=_i64(256, 128, 1), cu_k=FAKE,
              total_k=9, B=2, Hq=8, Hkv=2, D=128, scale=0.1, window=0, o=FAKE, lse=None, ws=FAKE, ws_bytes=BIG,
              err=None, stream=None)
APPEND = dict(q=FAKE, qs=QS, k=FAKE, kn=_i64(256, 128, 1), v=FAKE, vn=_i64(256, 128, 1), cu=FAKE, total=4, table=FAKE,
              n_pos=100, rot=128, inter=0, q_out=FAKE, k_out=None, kc=FAKE, ks=KS, vc=FAKE, vs=KS, pt=FAKE,
              max_pages=8, sl=FAKE, out_sl=None, B=2, Hq=8, Hkv=2, D=128, P=16, pool=64, sig=FAKE, err=None,
              stream=None)
ODD = ctypes.c_void_p(0x1008)


def _call(name, base, **kw):
    assert set(kw) <= set(base)
    return getattr(sa.load(), name)(*{**base, **kw}.values())


@pytest.mark.parametrize("kw,want", [
    (dict(Hq=6, Hkv=4), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-0.1), INVALID), (dict(window=-1), INVALID), (dict(total=-1), INVALID), (dict(B=-1), INVALID),
    (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(cu=None), INVALID), (dict(o=None), INVALID),
    (dict(o=ODD), INVALID), (dict(qs=_i64(1024, 128, 2)), INVALID), (dict(qs=_i64(1020, 128, 1)), INVALID),
    (dict(k=None), INVALID), (dict(v=ODD), INVALID), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(Hq=258, Hkv=2), UNSUPPORTED), (dict(B=4097), UNSUPPORTED), (dict(total=1 << 28), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=ODD), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE),
])
@pytest.mark.parametrize("name,base", [("sa_chunk_attention", CHUNK), ("sa_prompt_attention", PROMPT)])
def test_dense_refusals(name, base, kw, want):
    assert _call(name, base, **kw) == want


def test_chunk_and_prompt_own_refusals():
    for kw, want in ((dict(P=24), UNSUPPORTED), (dict(P=0), INVALID), (dict(pool=0), INVALID), (dict(pt=None), INVALID),
                     (dict(sl=None), INVALID), (dict(max_pages=1 << 27), UNSUPPORTED),
                     (dict(ks=_i64(4096, 0, 128, 1)), INVALID), (dict(ks=_i64(1 << 40, 2048, 128, 1)), UNSUPPORTED)):
        assert _call("sa_chunk_attention", CHUNK, **kw) == want, kw
    for kw, want in ((dict(cu_k=None), INVALID), (dict(total_k=-1), INVALID), (dict(total_k=1 << 30), UNSUPPORTED),
                     (dict(ks=_i64(0, 128, 1)), UNSUPPORTED)):
        assert _call("sa_prompt_attention", PROMPT, **kw) == want, kw
    # nothing to do
    assert _call("sa_chunk_attention", CHUNK, B=0) == OK and _call("sa_prompt_attention", PROMPT, total=0) == OK


@pytest.mark.parametrize("kw,want", [
    (dict(D=100), INVALID), (dict(rot=24), INVALID), (dict(rot=144), INVALID), (dict(rot=-16), INVALID),
    (dict(table=None), INVALID), (dict(table=ODD), INVALID), (dict(cu=None), INVALID), (dict(k=None), INVALID),
    (dict(v=ODD), INVALID), (dict(q_out=None), INVALID), (dict(q_out=ODD), INVALID), (dict(k_out=ODD), INVALID),
    (dict(kc=None), INVALID), (dict(vs=_i64(4096, 2048, 100, 1)), INVALID), (dict(pt=None), INVALID),
    (dict(sl=None), INVALID), (dict(out_sl=FAKE), INVALID), (dict(P=0), INVALID), (dict(pool=0), INVALID),
    (dict(qs=_i64(1024, 127, 1)), INVALID), (dict(Hq=0), INVALID), (dict(total=-1), INVALID),
    (dict(D=264, rot=64), UNSUPPORTED), (dict(max_pages=1 << 28), UNSUPPORTED), (dict(B=0), OK),
])
def test_append_refusals(kw, want):
    assert _call("sa_append_kv_rope", APPEND, **kw) == want


def test_two_level_refusals():
    lib = sa.load()
    for i, bad in ((1, -1), (4, 17), (4, -1)):
        d = [FAKE, 4, FAKE, 8, 3]
        d[i] = bad
        c = list(CHUNK.values())
        assert lib.sa_chunk_attention_dir(*c[:8], *d, *c[10:]) == INVALID
        a = list(APPEND.values())
        assert lib.sa_append_kv_rope_dir(*a[:18], *d, *a[20:]) == INVALID


def test_workspace_size_covers_the_parts():
    lib = sa.load()
    size = lib.sa_dense_attention_workspace_size
    assert size(0, 8, 2, 128) == 0 and size(4, 6, 4, 128) == 0
    # two parts per CTA (at most 160) of min(256, tokens x group heads) rows
    assert size(1, 8, 2, 128) == 160 * 32 + 320 * 4 * 4 + 320 * 4 * 128 * 4
    assert size(10 ** 5, 8, 2, 64) == 160 * 32 + 320 * 256 * 4 + 320 * 256 * 64 * 4
    assert all(size(n, 8, 2, 128) <= size(n + 1, 8, 2, 128) for n in range(1, 80))


def test_python_refusals():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):   # not on a GPU
        sa.sa_chunk_attention(bf(2, 8, 64), bf(4, 2, 16, 64), bf(4, 2, 16, 64), i(1, 4), i(1), i(2), 0.1)
    with pytest.raises(ValueError):
        sa.sa_prompt_attention(bf(2, 8, 64), bf(2, 2, 64), bf(2, 2, 64), i(2), i(2), 0.1)
    with pytest.raises(ValueError):
        sa.sa_append_kv_rope(None, bf(2, 2, 64), bf(2, 2, 64), i(2), None, bf(4, 2, 16, 64), bf(4, 2, 16, 64), i(1, 4),
                             i(1))
    with pytest.raises(TypeError):
        sa.sa_chunk_attention(bf(2, 8, 64).float(), bf(4, 2, 16, 64), bf(4, 2, 16, 64), i(1, 4), i(1), i(2), 0.1)
    with pytest.raises(TypeError):
        sa.sa_prompt_attention(bf(2, 8, 64), bf(2, 128), bf(2, 2, 64), i(2), i(2), 0.1)


# ------------------------------------------------------------------ oracle pins
def _bits(x):
    return O.f64_to_bf16_rne(np.asarray(x, dtype=np.float64))


@pytest.mark.parametrize("inter", [False, True])
def test_oracle_rotation_is_a_complex_product(inter):
    rng = np.random.default_rng(0)
    x = _bits(rng.standard_normal((5, 3, 32)))
    ang = rng.uniform(0, 6, (9, 8))
    table = np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)
    pos = np.array([0, 8, 3, 3, 1])
    got = O.bf16_to_f64(O.rotate_bf16(x, table, pos, inter))
    f = O.bf16_to_f64(x)
    i = np.arange(0, 16, 2) if inter else np.arange(8)
    j = i + (1 if inter else 8)
    w = (f[..., i] + 1j * f[..., j]) * np.exp(1j * ang[pos])[:, None, :]
    # two products and a sum in float32, one rounding to bf16
    tol = 2.0 ** -8 * np.abs(w) + 2.0 ** -20
    assert np.all(np.abs(got[..., i] - w.real) <= tol) and np.all(np.abs(got[..., j] - w.imag) <= tol)
    assert np.array_equal(got[..., 16:], f[..., 16:])


def test_oracle_rotated_scores_depend_on_distance_alone():
    rng = np.random.default_rng(1)
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    ang = np.arange(50)[:, None] * f
    table = np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)
    q, k = (np.repeat(_bits(rng.standard_normal((1, 1, 64))), 50, 0) for _ in range(2))
    rq, rk = (O.bf16_to_f64(O.rotate_bf16(x, table, np.arange(50)))[:, 0] for x in (q, k))
    s = rq @ rk.T
    # each rotated feature is off by at most 2^-8 of itself (its rounding to bf16; the
    # table's and the float32 steps' 2^-21 lie inside the 2.1), a pair's products sum to
    # at most |q pair| |k pair| in magnitude at every position, and two scores differ
    pair = lambda x: np.hypot(*np.split(O.bf16_to_f64(x[0, 0]), 2))
    tol = 2 * 2.1 * 2.0 ** -8 * pair(q) @ pair(k)
    for d in range(0, 40, 7):
        assert np.ptp(np.diagonal(s, d)) <= tol


@pytest.mark.parametrize("n,L,window", [(1, 7, 0), (5, 5, 0), (4, 30, 9), (6, 3, 0), (3, 20, 1)])
def test_oracle_dense_attention_is_masked_softmax(n, L, window):
    g = torch.Generator().manual_seed(n * 100 + L)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((n, 4, 16), (L, 2, 16), (L, 2, 16)))
    o, lse, A, reach = O.dense_attention(q.numpy(), k.numpy(), v.numpy(), 0.3, window)
    s = 0.3 * torch.einsum("nhd,lhd->hnl", q, k.repeat_interleave(2, 1))
    p, j = L - n + torch.arange(n)[:, None], torch.arange(L)[None, :]
    s = s.masked_fill(~((j <= p) & (j > p - (window or L + n + 1))), -math.inf)
    z = torch.logsumexp(s, -1)
    w = torch.where(z[..., None] > -math.inf, torch.exp(s - z[..., None]), torch.zeros_like(s))
    want = torch.einsum("hnl,lhd->nhd", w, v.repeat_interleave(2, 1)).numpy()
    assert np.allclose(o, want, atol=1e-12) and np.array_equal(lse, np.where(np.isfinite(z.T.numpy()), lse, -np.inf))
    fin = np.isfinite(lse)
    assert np.allclose(lse[fin], z.T.numpy()[fin], atol=1e-12) and np.all(A >= np.abs(o) - 1e-12)
