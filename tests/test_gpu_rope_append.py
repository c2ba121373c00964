"""sa_append_kv_rope against the oracle, bit for bit (marked gpu): the rotation
is float32 arithmetic with one rounding per product and sum, so queries, cache
rows, summaries and lengths all have exactly one right value.  Then the run of
the packed operators as a serving loop uses them."""
import math

import numpy as np
import pytest
import torch

import oracle as O
import paged_sparse_kv_sa_b200 as sa
from test_gpu_dense import check

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _case(seed, ns, ctx, Hq, Hkv, D, P, rot, spare=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: _bits(torch.randn(s, generator=g).to(torch.bfloat16))  # noqa: E731
    B, n = len(ns), sum(ns)
    npg = [-(-(a + b) // P) for a, b in zip(ns, ctx)]
    pool = sum(npg) + 2
    perm = torch.randperm(pool, generator=g).numpy()
    pt = np.full((B, max(max(npg), 1) + spare), -1, dtype=np.int32)
    off = 0
    for b, m in enumerate(npg):
        pt[b, :m] = perm[off:off + m]
        off += m
    k, v = r(pool, Hkv, P, D), r(pool, Hkv, P, D)
    sl = np.array(ctx, dtype=np.int32)
    c = dict(q=r(n, Hq, D), k=r(n, Hkv, D), v=r(n, Hkv, D), kc=k, vc=v, pt=pt, sl=sl, P=P,
             sig=O.page_summaries(k, pt, sl, P), cu=np.array([0] + list(np.cumsum(ns)), dtype=np.int32))
    n_pos = max([a + b for a, b in zip(ns, ctx)] + [1])
    f = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.arange(n_pos)[:, None] * f[None, :]
    c["table"] = np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32) if rot else None
    return c


def _gpu(c):
    return dict(q=_dev(c["q"]), k=_dev(c["k"]), v=_dev(c["v"]), kc=_dev(c["kc"]), vc=_dev(c["vc"]), sig=_dev(c["sig"]),
                pt=_i32(c["pt"]), sl=_i32(c["sl"]), cu=_i32(c["cu"]),
                table=None if c["table"] is None else torch.from_numpy(c["table"]).to(DEV))


def _run(d, interleaved=False, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    new = torch.full((d["sl"].shape[0],), -1, dtype=torch.int32, device=DEV)
    qo, _ = sa.sa_append_kv_rope(d["q"], d["k"], d["v"], d["cu"], d["table"], d["kc"], d["vc"], d["pt"], d["sl"],
                                 d["sig"], interleaved=interleaved, out_seq_lens=new, dev_error=err, **kw)
    torch.cuda.synchronize()
    return qo, new, int(err.item())


def _want(c, interleaved=False):
    return O.append_kv_rope(c["q"], c["k"], c["v"], c["cu"], c["table"], c["kc"], c["vc"], c["sig"], c["pt"], c["sl"],
                            c["P"], interleaved)


CASES = [
    # ns, ctx, Hq, Hkv, D, P, rot, interleaved
    ([1], [0], 8, 2, 64, 16, 64, False),
    ([1, 1, 1], [15, 16, 700], 32, 8, 128, 16, 128, False),
    ([3, 0, 40, 17], [100, 5, 0, 31], 8, 4, 128, 16, 128, True),
    ([200, 1], [63, 4000], 6, 2, 64, 64, 32, False),
    ([77, 5], [10, 0], 5, 5, 128, 48, 64, True),
    ([130], [1], 3, 1, 256, 128, 256, False),
    ([9, 9], [3, 60], 4, 2, 64, 16, 0, False),        # no table: a plain append
    ([50], [20], 4, 2, 72, 16, 16, False),            # most of the head unrotated, an odd width
    ([1] * 70, list(range(70)), 2, 1, 64, 16, 64, False),
    ([600], [13], 1, 1, 128, 512, 128, False),        # a page of many rows
    ([900, 3, 700, 0, 650], [5, 60, 0, 9, 31], 8, 8, 128, 16, 128, False),   # pages enough for several heads a CTA
    ([700, 1200], [3, 40], 5, 5, 64, 16, 32, True),
    ([900, 2000], [70, 1], 2, 16, 128, 64, 64, False),
]


@pytest.mark.parametrize("ns,ctx,Hq,Hkv,D,P,rot,inter", CASES)
def test_rope_append_matches_oracle(ns, ctx, Hq, Hkv, D, P, rot, inter):
    c = _case(21 + sum(ns) + D, ns, ctx, Hq, Hkv, D, P, rot)
    d = _gpu(c)
    k_out = torch.empty_like(d["k"])
    qo, new, err = _run(d, inter, k_out=k_out)
    q, k, kc, vc, sig, lens = _want(c, inter)
    assert err == 0
    assert np.array_equal(_bits(qo), q) and np.array_equal(_bits(k_out), k)
    assert np.array_equal(_bits(d["kc"]), kc) and np.array_equal(_bits(d["vc"]), vc)
    assert np.array_equal(_bits(d["sig"]), sig) and np.array_equal(new.cpu().numpy(), lens)


def test_in_place_strided_and_without_optional_parts():
    # q, k, v as views of one fused projection, rotated in place where contiguous
    c = _case(31, [30, 2], [7, 90], 8, 2, 128, 16, 128)
    q, k, kc, vc, sig, lens = _want(c)
    d = _gpu(c)
    fused = torch.cat((d["q"], d["k"], d["v"]), 1)
    v = dict(d, q=fused[:, :8], k=fused[:, 8:10], v=fused[:, 10:])
    qo, _, err = _run(v)
    assert err == 0 and np.array_equal(_bits(qo), q) and np.array_equal(_bits(d["kc"]), kc)
    assert np.array_equal(_bits(d["vc"]), vc) and np.array_equal(_bits(d["sig"]), sig)
    d = _gpu(c)
    qo, _, err = _run(d, q_out=d["q"], k_out=d["k"])
    assert qo is d["q"] and err == 0
    assert np.array_equal(_bits(d["q"]), q) and np.array_equal(_bits(d["k"]), k)
    assert np.array_equal(_bits(d["kc"]), kc) and np.array_equal(_bits(d["sig"]), sig)
    d = _gpu(c)
    keep = _bits(d["sig"])
    d2 = dict(d, q=None)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo, _ = sa.sa_append_kv_rope(None, d2["k"], d2["v"], d2["cu"], d2["table"], d2["kc"], d2["vc"], d2["pt"], d2["sl"],
                                 dev_error=err)
    torch.cuda.synchronize()
    assert qo is None and int(err.item()) == 0
    assert np.array_equal(_bits(d["kc"]), kc) and np.array_equal(_bits(d["sig"]), keep)


def test_summaries_where_float64_is_not_enough():
    # columns whose exponents span more than a float64 sum holds
    c = _case(32, [20], [12], 2, 2, 64, 32, 0)
    rng = np.random.default_rng(0)
    e = rng.integers(60, 200, c["k"].shape).astype(np.uint16)
    c["k"] = ((e << 7) | rng.integers(0, 128, e.shape).astype(np.uint16)
              | (rng.integers(0, 2, e.shape).astype(np.uint16) << 15)).astype(np.uint16)
    d = _gpu(c)
    _, _, err = _run(d)
    assert err == 0 and np.array_equal(_bits(d["sig"]), _want(c)[4])


def test_tokens_behind_the_batch_and_past_the_ends():
    c = _case(33, [4, 6], [30, 10], 4, 2, 64, 16, 64)
    d = _gpu(c)
    # offsets that start past zero and end before the tensor does
    c2 = dict(c, cu=np.array([2, 4, 9], dtype=np.int32))
    d["cu"] = _i32(c2["cu"])
    qo = torch.full_like(d["q"], 7.0)
    qo, new, err = _run(d, q_out=qo)
    q, k, kc, vc, sig, lens = _want(c2)
    assert err == 0
    assert np.array_equal(_bits(qo)[2:9], q) and bool((qo[:2] == 7).all()) and bool((qo[9:] == 7).all())
    assert np.array_equal(_bits(d["kc"]), kc) and np.array_equal(_bits(d["sig"]), sig)
    # a table that ends at position 31: sequence 0's tokens 32, 33 are dropped and flagged
    d = _gpu(c)
    d["table"] = d["table"][:32].contiguous()
    qo = torch.full_like(d["q"], 7.0)
    qo, new, err = _run(d, q_out=qo)
    assert err == 1 and np.array_equal(new.cpu().numpy(), [34, 16])
    keep = np.r_[0:2, 4:10]
    cut = dict(c, q=c["q"][keep], k=c["k"][keep], v=c["v"][keep], cu=np.array([0, 2, 8], dtype=np.int32))
    q, k, kc, vc, sig, _ = _want(cut)
    assert np.array_equal(_bits(qo)[keep], q) and bool((qo[2:4] == 7).all())
    assert np.array_equal(_bits(d["kc"]), kc) and np.array_equal(_bits(d["vc"]), vc)
    assert np.array_equal(_bits(d["sig"]), sig)


def test_bad_pages_lengths_and_offsets_are_flagged_and_skipped():
    c = _case(34, [20, 3], [0, 5], 4, 2, 64, 16, 64)
    d = _gpu(c)
    d["pt"][0, 1] = 99999
    _, _, err = _run(d)
    assert err == 2
    cut = dict(c, k=np.r_[c["k"][:16], c["k"][20:]], v=np.r_[c["v"][:16], c["v"][20:]],
               q=np.r_[c["q"][:16], c["q"][20:]], cu=np.array([0, 16, 19], dtype=np.int32))
    _, _, kc, vc, sig, _ = _want(cut)
    assert np.array_equal(_bits(d["kc"]), kc) and np.array_equal(_bits(d["sig"]), sig)
    for bad, flag in ((dict(sl=_i32([-4, 5])), 1), (dict(cu=_i32([0, 20, 5000])), 4)):
        d = dict(_gpu(c), **bad)
        _, _, err = _run(d)
        assert err & flag


@pytest.mark.parametrize("cu,skipped", [([-5, 20, 23], (0, 20)), ([0, 20, 5000], (20, 23)), ([0, -1, 23], None)])
def test_a_sequence_with_bad_offsets_is_skipped(cu, skipped):
    c = _case(35, [20, 3], [0, 5], 4, 2, 64, 16, 64)
    d = dict(_gpu(c), cu=_i32(cu))
    before = {k: d[k].clone() for k in ("kc", "vc", "sig")}
    qo = torch.full_like(d["q"], 7.0)
    qo, _, err = _run(d, q_out=qo)
    assert err & 4
    if skipped is None:   # offsets that turn back: neither sequence holds
        assert all(torch.equal(d[k], x) for k, x in before.items())
        return
    x, y = skipped
    assert bool((qo[x:y] == 7).all())
    other = 1 if x == 0 else 0
    rest = slice(20, 23) if other else slice(0, 20)
    q, _, kc, vc, sig, _ = _want(c)
    assert np.array_equal(_bits(qo)[rest], q[rest])
    mine = c["pt"][other][:-(-(len(range(*rest.indices(23))) + int(c["sl"][other])) // 16)]
    pages = np.setdiff1d(np.arange(kc.shape[0]), mine)
    assert np.array_equal(_bits(d["kc"])[mine], kc[mine]) and np.array_equal(_bits(d["sig"])[mine], sig[mine])
    assert all(np.array_equal(_bits(d[k])[pages], _bits(b)[pages]) for k, b in before.items())


def test_two_level_map_is_the_flat_call():
    c = _case(35, [40, 3], [100, 250], 8, 2, 128, 16, 128, spare=3)
    d, e = _gpu(c), _gpu(c)
    qo, new, err = _run(d)
    w, shift = d["pt"].shape[1], 2
    nd = -(-w // 4)
    pad = torch.full((2, nd * 4), -1, dtype=torch.int32, device=DEV)
    pad[:, :w] = d["pt"]
    blocks = pad.view(-1, 4).contiguous()
    direc = torch.arange(2 * nd, dtype=torch.int32, device=DEV).view(2, nd)
    q2, _ = sa.sa_append_kv_rope_dir(e["q"], e["k"], e["v"], e["cu"], e["table"], e["kc"], e["vc"], direc, blocks,
                                     shift, e["sl"], e["sig"])
    torch.cuda.synchronize()
    assert err == 0
    for a, b in ((qo, q2), (d["kc"], e["kc"]), (d["vc"], e["vc"]), (d["sig"], e["sig"])):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_a_serving_loop():
    """Prompts through the append and the prompt attention, then chunks and single tokens
    through the append and the chunk attention, then a sparse step over the same cache:
    every step against the oracle on the cache the oracle's appends give."""
    Hq, Hkv, D, P = 8, 2, 128, 16
    g = torch.Generator().manual_seed(77)
    steps = [[50, 1, 130], [1, 20, 0], [1, 1, 1], [3, 0, 60]]
    total = [sum(x) for x in zip(*steps)]
    c = _case(41, total, [0, 0, 0], Hq, Hkv, D, P, 128)
    d = _gpu(c)
    scale = 1.0 / math.sqrt(D)
    r = lambda n, h: _bits(torch.randn((n, h, D), generator=g).to(torch.bfloat16))  # noqa: E731
    kc, vc, sig, sl = c["kc"], c["vc"], c["sig"], np.zeros(3, dtype=np.int32)
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    for i, ns in enumerate(steps):
        n = sum(ns)
        q, k, v = r(n, Hq), r(n, Hkv), r(n, Hkv)
        cu = np.array([0] + list(np.cumsum(ns)), dtype=np.int32)
        qr, kr, kc, vc, sig, sl2 = O.append_kv_rope(q, k, v, cu, c["table"], kc, vc, sig, c["pt"], sl, P)
        new = torch.empty_like(lens)
        k_out = torch.empty((n, Hkv, D), dtype=torch.bfloat16, device=DEV)
        vd = _dev(v)
        qo, _ = sa.sa_append_kv_rope(_dev(q), _dev(k), vd, _i32(cu), d["table"], d["kc"], d["vc"], d["pt"], lens,
                                     d["sig"], k_out=k_out, out_seq_lens=new)
        ks, vs = [], []
        for b in range(3):
            pg = c["pt"][b, :-(-int(sl2[b]) // P)]
            for dst, src in ((ks, kc), (vs, vc)):
                dst.append(_dev(src[pg].transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:sl2[b]]))
        if i == 0:
            o, lse = sa.sa_prompt_attention(qo, k_out, vd, _i32(cu), _i32(cu), scale)
            check(o, lse, qo, ks, vs, ns, scale, 0)
        o, lse = sa.sa_chunk_attention(qo, d["kc"], d["vc"], d["pt"], new, _i32(cu), scale)
        torch.cuda.synchronize()
        assert np.array_equal(_bits(qo), qr) and np.array_equal(new.cpu().numpy(), sl2)
        check(o, lse, qo, ks, vs, ns, scale, 0)
        lens, sl = new, sl2
    assert np.array_equal(_bits(d["kc"]), kc) and np.array_equal(_bits(d["sig"]), sig)
    # a sparse step whose budget holds every page is the dense answer
    q = _dev(r(3, Hq))
    pages = d["pt"].shape[1]
    out = sa.sa_sparse_step(q.view(3, 1, Hq, D), d["sig"], d["kc"], d["vc"], d["pt"], lens, P, P, P, pages * P, scale)
    o, lse = sa.sa_chunk_attention(q, d["kc"], d["vc"], d["pt"], lens, _i32([0, 1, 2, 3]), scale)
    torch.cuda.synchronize()
    assert float((out[4].view(3, Hq) - lse).abs().max()) < 1e-4
    check(o, lse, q, ks, vs, [1, 1, 1], scale, 0)


def test_append_of_nothing_reports_the_lengths():
    c = _case(36, [0, 0], [5, 20], 4, 2, 64, 16, 64)
    d = _gpu(c)
    before = [d[x].clone() for x in ("kc", "vc", "sig")]
    _, new, err = _run(d)
    assert err == 0 and np.array_equal(new.cpu().numpy(), [5, 20])
    for a, b in zip(before, (d["kc"], d["vc"], d["sig"])):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_a_captured_serving_step():
    # append, attend and move the lengths on, captured once and replayed token by token:
    # the cache, the lengths and the last answer are those of the same calls made one by one
    Hq, Hkv, D, P, B, n = 8, 2, 128, 16, 3, 20
    c = _case(42, [n] * B, [3, 30, 700], Hq, Hkv, D, P, 128)
    g = torch.Generator().manual_seed(5)
    feed = [[torch.randn((B, h, D), generator=g).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv)] for _ in range(n)]
    cu = _i32([0, 1, 2, 3])
    ws = sa.dense_attention_workspace(B, Hq, Hkv, D, DEV)

    def step(d, x, lens, new, qo, o, lse):
        sa.sa_append_kv_rope(x[0], x[1], x[2], cu, d["table"], d["kc"], d["vc"], d["pt"], lens, d["sig"], q_out=qo,
                             out_seq_lens=new)
        sa.sa_chunk_attention(qo, d["kc"], d["vc"], d["pt"], new, cu, 0.09, o_out=o, lse_out=lse, workspace=ws)
        lens.copy_(new)

    ends = []
    for captured in (False, True):
        d = _gpu(c)
        x = [t.clone() for t in feed[0]]
        lens, new = d["sl"].clone(), torch.empty_like(d["sl"])
        qo, o, lse = torch.empty_like(x[0]), torch.empty_like(x[0]), torch.empty((B, Hq), device=DEV)
        if captured:
            step(d, x, lens, new, qo, o, lse)     # warm-up, on a copy of the state
            d, lens = _gpu(c), lens
            lens.copy_(d["sl"])
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(d, x, lens, new, qo, o, lse)
        for y in feed:
            for a, b in zip(x, y):
                a.copy_(b)
            if captured:
                graph.replay()
            else:
                step(d, x, lens, new, qo, o, lse)
        torch.cuda.synchronize()
        ends.append([t.clone() for t in (d["kc"], d["vc"], d["sig"], lens, o, lse)])
    for a, b in zip(*ends):
        assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                           b.view(torch.int16) if b.dtype == torch.bfloat16 else b)
