"""Dense attention of packed tokens (sa_chunk_attention, sa_prompt_attention)
against the oracle in float64 (marked gpu).

Tolerances, from the arithmetic (u = 2^-8, one bf16 rounding):
  each probability is rounded once to bf16 before the value product and the
  output once after it: u (A + |O|), A = sum_j softmax_j |v_j|;
  a score is a float32 sum of D products, each of whose D steps may be off by
  2^-23 of the terms' absolute sum `reach` (the tensor core may truncate), a
  multiplication by the scale and 2^x (2^-22 relative): every probability is
  off by a factor within exp(+-eta), eta = (D + 4) 2^-23 reach + 2^-21;
  normalising doubles it, and the value product's own float32 steps add less
  than eta again: 4 eta A.
  lse: eta + the sum's float32 steps (2^-24 each over the chain of 20 adds per
  tile and one per tile) + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
import paged_sparse_kv_sa_b200 as sa

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _randn(g, *shape, mul=1.0):
    return (torch.randn(shape, generator=g) * mul).to(torch.bfloat16).to(DEV)


def _cu(ns):
    return torch.tensor([0] + list(np.cumsum(ns)), dtype=torch.int32, device=DEV)


def check(o, lse, q, ks, vs, ns, scale, window, cu0=0):
    """o, lse, q packed; ks, vs: each sequence's keys and values [L, Hkv, D]"""
    o, lse, q = _f64(o), _f64(lse), _f64(q)
    at = cu0
    for n, k, v in zip(ns, ks, vs):
        if n == 0:
            continue
        D = q.shape[2]
        ro, rl, A, reach = O.dense_attention(q[at:at + n], _f64(k), _f64(v), scale, window)
        eta = (D + 4) * 2.0 ** -23 * reach + 2.0 ** -21
        tol = U * (A + np.abs(ro)) * (1 + U) + 4 * eta[..., None] * A
        err = np.abs(o[at:at + n] - ro)
        assert np.all(err <= tol), (float((err - tol).max()), n, k.shape)
        seen = np.isfinite(rl)
        assert np.array_equal(np.isfinite(lse[at:at + n]), seen)
        assert np.all(lse[at:at + n][~seen] == -np.inf)
        steps = (20 + k.shape[0] / 128) * 2.0 ** -24
        tl = eta + steps + 2.0 ** -22 * np.abs(np.where(seen, rl, 0.0))
        assert np.all(np.abs(lse[at:at + n][seen] - rl[seen]) <= tl[seen])
        at += n


def make_pages(g, ks, vs, P, Hkv, D, spare=3, layout="hpd", fill=float("nan")):
    """Paged caches holding the sequences; every other row of the pool is `fill`."""
    B = len(ks)
    npg = [-(-k.shape[0] // P) for k in ks]
    pool = sum(npg) + spare
    perm = torch.randperm(pool, generator=g)
    width = max(max(npg), 1)
    pt = torch.full((B, width), -1, dtype=torch.int32)
    shape = (pool, Hkv, P, D) if layout == "hpd" else (pool, P, Hkv, D)
    kc, vc = (torch.full(shape, fill, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    if layout != "hpd":
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    off = 0
    for b in range(B):
        pt[b, :npg[b]] = perm[off:off + npg[b]].to(torch.int32)
        off += npg[b]
        for p in range(npg[b]):
            m = min(P, ks[b].shape[0] - p * P)
            ph = int(pt[b, p])
            kc[ph, :, :m] = ks[b][p * P:p * P + m].transpose(0, 1)
            vc[ph, :, :m] = vs[b][p * P:p * P + m].transpose(0, 1)
    return kc, vc, pt.to(DEV)


def chunk_case(seed, ns, Ls, G, Hkv, D, P, window=0, layout="hpd", mul=1.0, tail=0, fill=float("nan")):
    g = torch.Generator().manual_seed(seed)
    ks = [_randn(g, L, Hkv, D, mul=mul) for L in Ls]
    vs = [_randn(g, L, Hkv, D) for L in Ls]
    q = _randn(g, sum(ns) + tail, G * Hkv, D)
    kc, vc, pt = make_pages(g, ks, vs, P, Hkv, D, layout=layout, fill=fill)
    sl = torch.tensor(Ls, dtype=torch.int32, device=DEV)
    return dict(q=q, ks=ks, vs=vs, kc=kc, vc=vc, pt=pt, sl=sl, cu=_cu(ns), scale=1.0 / math.sqrt(D))


def run_chunk(c, window=0, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = sa.sa_chunk_attention(c["q"], c["kc"], c["vc"], c["pt"], c["sl"], c["cu"], c["scale"],
                                   window=window, dev_error=err, **kw)
    torch.cuda.synchronize()
    return o, lse, int(err.item())


CHUNKS = [
    # ns, Ls, G, Hkv, D, P, window
    ([1], [1], 4, 2, 64, 16, 0),
    ([1], [129], 4, 2, 128, 16, 0),
    ([1, 1, 1], [5, 1000, 300], 4, 2, 128, 16, 0),
    ([1], [9000], 8, 1, 128, 64, 0),                       # one item over many CTAs
    ([1, 1], [6000, 17], 1, 3, 64, 16, 0),
    ([3, 8, 1, 5], [3, 700, 1, 129], 8, 2, 128, 64, 0),
    ([33], [33], 4, 2, 64, 16, 0),                         # 132 rows: two tiles, the second nearly empty
    ([64, 65], [64, 500], 4, 1, 128, 48, 0),
    ([200], [1111], 4, 2, 128, 16, 0),
    ([37, 1, 100], [300, 2000, 100], 3, 2, 128, 128, 0),   # 3 heads a group: tokens straddle tiles
    ([50], [400], 7, 1, 64, 256, 0),                       # pages larger than a tile
    ([3], [500], 128, 1, 128, 16, 0),
    ([0, 5, 0, 1, 0], [7, 40, 0, 90, 0], 4, 2, 128, 16, 0),   # sequences without new tokens
    ([6, 2], [2, 0], 4, 2, 128, 16, 0),                    # more queries than keys: rows that see none
    ([1, 40, 300], [700, 800, 900], 4, 2, 128, 16, 100),
    ([1, 90], [5000, 600], 4, 1, 64, 64, 1),               # only its own key
    ([150], [150], 2, 2, 128, 32, 128),
    ([1], [300], 4, 2, 128, 16, 1000),                     # a window longer than the sequence
]


@pytest.mark.parametrize("ns,Ls,G,Hkv,D,P,window", CHUNKS)
def test_chunk_matches_oracle(ns, Ls, G, Hkv, D, P, window):
    # every row of the pool that is no key is NaN: none of it may reach an output
    c = chunk_case(11 + sum(ns) + sum(Ls), ns, Ls, G, Hkv, D, P)
    o, lse, err = run_chunk(c, window)
    assert err == 0
    check(o, lse, c["q"], c["ks"], c["vs"], ns, c["scale"], window)


def test_chunk_vllm_layout_strided_queries_and_sharp_scores():
    ns, Ls, G, Hkv, D = [20, 1, 70], [333, 1200, 70], 4, 2, 128
    c = chunk_case(5, ns, Ls, G, Hkv, D, 16, layout="phd", mul=3.0)
    # queries as a view into a fused [tokens, (Hq + 2 Hkv), D] projection
    qkv = torch.zeros((sum(ns), (G + 2) * Hkv, D), dtype=torch.bfloat16, device=DEV)
    qkv[:, :G * Hkv] = c["q"]
    c["q"] = qkv[:, :G * Hkv]
    assert not c["q"].is_contiguous() and not c["kc"].is_contiguous()
    o, lse, err = run_chunk(c)
    assert err == 0
    check(o, lse, c["q"], c["ks"], c["vs"], ns, c["scale"], 0)


def test_chunk_leaves_tokens_behind_the_batch_alone_and_starts_past_zero():
    ns, Ls = [4, 9], [100, 260]
    c = chunk_case(6, ns, Ls, 4, 2, 64, 16, tail=7)
    c["cu"] = c["cu"] + 3      # tokens 0-2 and the last 4 belong to nobody
    o = torch.full_like(c["q"], 7.0)
    lse = torch.full(c["q"].shape[:2], 7.0, device=DEV)
    o, lse, err = run_chunk(c, o_out=o, lse_out=lse)
    assert err == 0
    for t in (o, lse):
        assert bool((t[:3] == 7.0).all()) and bool((t[16:] == 7.0).all())
    check(o, lse, c["q"], c["ks"], c["vs"], ns, c["scale"], 0, cu0=3)


def test_chunk_over_a_two_level_map_is_bitwise_the_flat_call():
    ns, Ls, P, shift = [1, 30], [2000, 500], 16, 3
    c = chunk_case(7, ns, Ls, 4, 2, 128, P)
    o, lse, err = run_chunk(c)
    w = c["pt"].shape[1]
    nd = -(-w // (1 << shift))
    pad = torch.full((2, nd << shift), -1, dtype=torch.int32, device=DEV)
    pad[:, :w] = c["pt"]
    blocks = pad.view(-1, 1 << shift).flip(0).contiguous()
    direc = (2 * nd - 1 - torch.arange(2 * nd, dtype=torch.int32, device=DEV)).view(2, nd).contiguous()
    o2, lse2 = sa.sa_chunk_attention_dir(c["q"], c["kc"], c["vc"], direc, blocks, shift, c["sl"],
                                         c["cu"], c["scale"])
    torch.cuda.synchronize()
    assert err == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


def test_chunk_bad_pages_are_left_out_and_flagged():
    # a page id outside the pool inside the sequence: its keys are not there
    P, G, Hkv, D = 16, 4, 2, 128
    c = chunk_case(8, [5], [500], G, Hkv, D, P)
    c["pt"][0, 3] = 10 ** 6
    c["pt"][0, 20] = -1
    o, lse, err = run_chunk(c)
    assert err == 2   # SA_DEVERR_POOL_RANGE
    keep = torch.ones(500, dtype=torch.bool)
    keep[48:64] = False
    keep[320:336] = False
    k, v = c["ks"][0][keep.to(DEV)], c["vs"][0][keep.to(DEV)]
    check(o, lse, c["q"], [k], [v], [5], c["scale"], 0)


def test_chunk_length_past_the_page_map_is_flagged():
    c = chunk_case(9, [1, 1], [64, 32], 4, 2, 64, 16)
    c["sl"] = torch.tensor([64, 1000], dtype=torch.int32, device=DEV)
    o, lse, err = run_chunk(c)
    assert err & 1
    check(o[:1], lse[:1], c["q"][:1], c["ks"][:1], c["vs"][:1], [1], c["scale"], 0)


def test_offsets_outside_the_tokens_are_flagged():
    c = chunk_case(10, [2, 2], [40, 50], 4, 2, 64, 16)
    c["cu"] = torch.tensor([0, 2, 900], dtype=torch.int32, device=DEV)
    o, lse, err = run_chunk(c)
    assert err & 4
    check(o[:2], lse[:2], c["q"][:2], c["ks"][:1], c["vs"][:1], [2], c["scale"], 0)


def test_many_sequences():
    rng = np.random.default_rng(1)
    B = 600
    Ls = [int(x) for x in rng.integers(0, 40, B)]
    ns = [int(min(x, L)) for x, L in zip(rng.integers(0, 4, B), Ls)]
    c = chunk_case(12, ns, Ls, 2, 1, 64, 16)
    o, lse, err = run_chunk(c)
    assert err == 0
    check(o, lse, c["q"], c["ks"], c["vs"], ns, c["scale"], 0)


PROMPTS = [
    ([1], 4, 2, 64, 0),
    ([128], 1, 1, 128, 0),
    ([300, 1, 0, 77], 4, 2, 128, 0),
    ([257, 511], 1, 3, 64, 0),
    ([700], 8, 1, 128, 0),
    ([130] * 40, 5, 1, 64, 0),          # more items than a planning batch holds per CTA
    ([400, 90], 4, 2, 128, 64),
    ([1000], 2, 1, 64, 333),
]


@pytest.mark.parametrize("ns,G,Hkv,D,window", PROMPTS)
def test_prompt_matches_oracle(ns, G, Hkv, D, window):
    g = torch.Generator().manual_seed(100 + sum(ns))
    q, k, v = (_randn(g, sum(ns), h, D) for h in (G * Hkv, Hkv, Hkv))
    cu = _cu(ns)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    scale = 1.0 / math.sqrt(D)
    o, lse = sa.sa_prompt_attention(q, k, v, cu, cu, scale, window=window, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ks, vs = torch.split(k, ns), torch.split(v, ns)
    check(o, lse, q, ks, vs, ns, scale, window)


def test_prompt_other_key_offsets_and_foreign_nan():
    # keys packed with gaps: NaN rows between the sequences belong to nobody
    g = torch.Generator().manual_seed(3)
    ns, Ls, G, Hkv, D = [10, 40, 3], [50, 40, 0], 4, 2, 128
    q = _randn(g, sum(ns), G * Hkv, D)
    k = torch.full((200, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    # sequence 0: keys 20..69, 1: 100..139, 2: none.  Offsets must not decrease, so
    # the gaps are sequences of their own without queries.
    k[20:70], v[20:70] = _randn(g, 50, Hkv, D), _randn(g, 50, Hkv, D)
    k[100:140], v[100:140] = _randn(g, 40, Hkv, D), _randn(g, 40, Hkv, D)
    cu_k = torch.tensor([20, 70, 100, 140, 140], dtype=torch.int32, device=DEV)
    cu_q = torch.tensor([0, 10, 10, 50, 53], dtype=torch.int32, device=DEV)
    o, lse = sa.sa_prompt_attention(q, k, v, cu_q, cu_k, 0.1)
    torch.cuda.synchronize()
    check(o, lse, q, [k[20:70], k[100:140], k[:0]], [v[20:70], v[100:140], v[:0]], ns, 0.1, 0)


def test_prompt_without_keys():
    q = torch.randn((3, 4, 64), device=DEV).to(torch.bfloat16)
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    cu_q = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    cu_k = torch.zeros(2, dtype=torch.int32, device=DEV)
    o, lse = sa.sa_prompt_attention(q, k, k.clone(), cu_q, cu_k, 0.125)
    torch.cuda.synchronize()
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


def test_empty_batches_touch_nothing():
    c = chunk_case(13, [2], [40], 4, 2, 64, 16)
    o = torch.full_like(c["q"], 7.0)
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    sa.sa_chunk_attention(c["q"], c["kc"], c["vc"], c["pt"][:0].contiguous(), c["sl"][:0], cu, 0.1, o_out=o)
    c["cu"] = torch.zeros(2, dtype=torch.int32, device=DEV)
    o, _, err = run_chunk(c, o_out=o)
    assert err == 0 and bool((o == 7.0).all())


def test_repeats_give_the_same_bits():
    c = chunk_case(14, [1, 60, 7], [5000, 900, 2500], 4, 2, 128, 16)
    o, lse, _ = run_chunk(c)
    for _ in range(5):
        o2, lse2, _ = run_chunk(c)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_captured_graph_follows_new_lengths():
    # one capture, replayed while the sequences grow: lengths are read on the device
    ns, P = [1, 1, 3], 16
    Ls = [700, 40, 1500]
    c = chunk_case(15, ns, Ls, 4, 2, 128, P)
    ws = sa.dense_attention_workspace(5, 8, 2, 128, DEV)
    o, lse = torch.empty_like(c["q"]), torch.empty((5, 8), device=DEV)
    sl = c["sl"].clone()
    call = lambda: sa.sa_chunk_attention(c["q"], c["kc"], c["vc"], c["pt"], sl, c["cu"], c["scale"],  # noqa: E731
                                         o_out=o, lse_out=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for cut in ([0, 0, 0], [13, 39, 700], [600, 2, 1497]):
        cur = [L - x for L, x in zip(Ls, cut)]
        sl.copy_(torch.tensor(cur, dtype=torch.int32))
        o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(o, lse, c["q"], [k[:L] for k, L in zip(c["ks"], cur)],
              [v[:L] for v, L in zip(c["vs"], cur)], ns, c["scale"], 0)


def test_two_streams_with_their_own_workspaces():
    cs = [chunk_case(16 + i, [1, 20], [3000, 800], 4, 2, 128, 16) for i in range(2)]
    want = [run_chunk(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    wss = [sa.dense_attention_workspace(21, 8, 2, 128, DEV) for _ in cs]
    outs = [(torch.empty_like(c["q"]), torch.empty((21, 8), device=DEV)) for c in cs]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s, ws, (o, lse) in zip(cs, streams, wss, outs):
            sa.sa_chunk_attention(c["q"], c["kc"], c["vc"], c["pt"], c["sl"], c["cu"], c["scale"],
                                  o_out=o, lse_out=lse, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for (o, lse), (wo, wl, _) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_tensors_made_by_the_call_belong_to_its_stream():
    c = chunk_case(19, [1, 20], [3000, 800], 4, 2, 128, 16)
    want = run_chunk(c)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)   # some 25 ms: the call waits behind it
    o, lse = sa.sa_chunk_attention(c["q"], c["kc"], c["vc"], c["pt"], c["sl"], c["cu"], c["scale"], stream=s)
    n = sa.dense_attention_workspace(21, 8, 2, 128, DEV).numel()
    for x in [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(4)]:   # the workspace's memory, were it free
        x.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------ loads that fill the GPU
def dense64(q, k, v, scale, window):
    """O.dense_attention for one sequence, in float64 torch operations on the GPU."""
    (n, Hq, D), (L, Hkv, _) = q.shape, k.shape
    if L == 0:
        z = torch.zeros((n, Hq, D), dtype=torch.float64, device=q.device)
        return z, torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device), z, z[..., 0]
    qd = q.double().view(n, Hkv, Hq // Hkv, D)
    kd, vd = k.double(), v.double()
    s = scale * torch.einsum("nhgd,lhd->nhgl", qd, kd)
    p, j = L - n + torch.arange(n, device=q.device)[:, None], torch.arange(L, device=q.device)[None, :]
    seen = (j <= p) & (j > p - (window or L + n + 1))
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.where(lse[..., None] > -math.inf, torch.exp(s - lse[..., None]), torch.zeros_like(s))
    reach = scale * torch.einsum("nhgd,lhd->nhgl", qd.abs(), kd.abs()).masked_fill(~seen[:, None, None], 0.0).amax(-1)
    return (torch.einsum("nhgl,lhd->nhgd", w, vd).reshape(n, Hq, D), lse.view(n, Hq),
            torch.einsum("nhgl,lhd->nhgd", w, vd.abs()).reshape(n, Hq, D), reach.view(n, Hq))


def check64(o, lse, q, ks, vs, ns, scale, window):
    """check() on the GPU: the same tolerances."""
    at = 0
    for n, k, v in zip(ns, ks, vs):
        if n == 0:
            continue
        D = q.shape[2]
        ro, rl, A, reach = dense64(q[at:at + n], k, v, scale, window)
        eta = (D + 4) * 2.0 ** -23 * reach + 2.0 ** -21
        tol = U * (A + ro.abs()) * (1 + U) + 4 * eta[..., None] * A
        off = (o[at:at + n].double() - ro).abs() - tol
        assert bool((off <= 0).all()), (float(off.max()), n, k.shape)
        seen = rl > -math.inf
        assert bool((lse[at:at + n][~seen] == -math.inf).all())
        tl = eta + (20 + k.shape[0] / 128) * 2.0 ** -24 + 2.0 ** -22 * torch.where(seen, rl, torch.zeros_like(rl)).abs()
        assert bool(((lse[at:at + n].double() - rl).abs()[seen] <= tl[seen]).all())
        at += n


LOADS = [
    # B, n_lo, n_hi, L_lo, L_hi, G, Hkv, D, P, window: many ragged tiles in every CTA's share
    (64, 1, 1, 500, 3000, 2, 8, 128, 16, 0),          # single tokens
    (24, 2, 8, 900, 6000, 8, 8, 128, 64, 0),          # drafts
    (16, 1, 400, 1000, 4000, 4, 8, 128, 16, 0),       # chunks between single tokens
    (64, 1, 1, 500, 3000, 4, 8, 64, 48, 0),
    (20, 1, 300, 300, 2500, 3, 8, 64, 128, 700),
]


@pytest.mark.parametrize("B,n_lo,n_hi,L_lo,L_hi,G,Hkv,D,P,window", LOADS)
def test_chunk_under_load(B, n_lo, n_hi, L_lo, L_hi, G, Hkv, D, P, window):
    rng = np.random.default_rng(B * D + n_hi)
    ns = [int(x) for x in rng.integers(n_lo, n_hi + 1, B)]
    Ls = [int(x) for x in rng.integers(L_lo, L_hi + 1, B)]
    Ls = [max(n, L) for n, L in zip(ns, Ls)]
    c = chunk_case(50 + B + D, ns, Ls, G, Hkv, D, P)
    for _ in range(3):
        o, lse, err = run_chunk(c, window)
        assert err == 0
        check64(o, lse, c["q"], c["ks"], c["vs"], ns, c["scale"], window)


@pytest.mark.parametrize("B,lo,hi,G,Hkv,D,window", [(12, 150, 2048, 4, 8, 128, 0), (30, 1, 700, 4, 8, 64, 0),
                                                  (3, 2000, 3001, 4, 8, 64, 1024), (9, 100, 900, 5, 6, 128, 333)])
def test_prompt_under_load(B, lo, hi, G, Hkv, D, window):
    rng = np.random.default_rng(B * D + hi)
    ns = [int(x) for x in rng.integers(lo, hi + 1, B)]
    g = torch.Generator().manual_seed(B)
    q, k, v = (_randn(g, sum(ns), h, D) for h in (G * Hkv, Hkv, Hkv))
    cu = _cu(ns)
    ks, vs = torch.split(k, ns), torch.split(v, ns)
    for _ in range(3):
        o, lse = sa.sa_prompt_attention(q, k, v, cu, cu, 1.0 / math.sqrt(D), window=window)
        check64(o, lse, q, ks, vs, ns, 1.0 / math.sqrt(D), window)


def test_prompt_over_views_of_one_projection():
    # q, k, v as slices of a fused [tokens, (Hq + 2 Hkv), D] projection: no copies
    g = torch.Generator().manual_seed(4)
    ns, G, Hkv, D = [300, 45], 4, 2, 128
    qkv = _randn(g, sum(ns), (G + 2) * Hkv, D)
    q, k, v = qkv[:, :G * Hkv], qkv[:, G * Hkv:(G + 1) * Hkv], qkv[:, (G + 1) * Hkv:]
    cu = _cu(ns)
    o, lse = sa.sa_prompt_attention(q, k, v, cu, cu, 0.08)
    check64(o, lse, q, torch.split(k, ns), torch.split(v, ns), ns, 0.08, 0)


def test_non_finite_scores_stay_in_their_rows():
    # a query of inf and one of NaN give NaN rows; every other row is as without them
    c = chunk_case(21, [3, 40], [300, 700], 4, 2, 128, 16)
    o, lse, _ = run_chunk(c)
    c["q"][1, 2] = float("inf")
    c["q"][20, 5] = float("nan")
    o2, lse2, err = run_chunk(c)
    assert err == 0
    keep = torch.ones(o.shape[:2], dtype=torch.bool, device=DEV)
    keep[1, 2] = keep[20, 5] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert bool(o2[1, 2].isnan().all()) and bool(o2[20, 5].isnan().all()) and bool(lse2[20, 5].isnan())


def test_recorded_call_is_the_call():
    c = chunk_case(22, [1, 9], [400, 90], 4, 2, 64, 16)
    want, want_lse, _ = run_chunk(c)
    ws = sa.dense_attention_workspace(10, 8, 2, 64, DEV)
    o, lse = torch.empty_like(want), torch.empty_like(want_lse)
    run = sa.bind(lambda: sa.sa_chunk_attention(c["q"], c["kc"], c["vc"], c["pt"], c["sl"], c["cu"], c["scale"],
                                                o_out=o, lse_out=lse, workspace=ws))
    assert run.n_calls == 1
    run()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_python_refuses_what_the_call_would_misread():
    c = chunk_case(23, [2], [40], 4, 2, 64, 16)
    args = lambda **kw: {**dict(q=c["q"], k_cache=c["kc"], v_cache=c["vc"], page_table=c["pt"], seq_lens=c["sl"],  # noqa: E731
                                cu_q=c["cu"], scale=0.1), **kw}
    for bad in (dict(seq_lens=c["sl"].long()), dict(cu_q=c["cu"].float()), dict(v_cache=c["vc"][:, :1]),
                dict(page_table=c["pt"].repeat(2, 1)), dict(o_out=torch.empty_like(c["q"])[:, :4]),
                dict(lse_out=torch.empty((2, 7), device=DEV)), dict(k_cache=c["kc"].float()),
                dict(workspace=torch.empty(100, device=DEV)), dict(seq_lens=c["sl"].repeat(2))):
        with pytest.raises((TypeError, ValueError)):
            sa.sa_chunk_attention(**args(**bad))
    for bad in (dict(seq_lens=c["sl"].cpu()), dict(k_cache=c["kc"].cpu(), v_cache=c["vc"].cpu())):
        with pytest.raises(ValueError):
            sa.sa_chunk_attention(**args(**bad))
    with pytest.raises(sa.SAError):
        sa.sa_chunk_attention(**args(scale=-1.0))
    with pytest.raises(sa.SAError):
        sa.sa_chunk_attention(**args(workspace=torch.empty(100, dtype=torch.uint8, device=DEV)))
