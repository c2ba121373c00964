"""Edges of the packed-batch operators (marked gpu)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_sparse_kv_sa_b200 as sa
from paged_sparse_kv_sa_b200 import workloads as W
from test_gpu_dense import U, _cu, _randn, check, chunk_case, run_chunk
from test_gpu_rope_append import _bits, _case, _gpu, _i32, _run, _want

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def test_offsets_that_turn_back_do_not_pass_the_counters():
    # every other sequence holds all tokens: 1985 x 8 kv heads x 270,464 key tiles are
    # 2^32 + 1024 in all, which 32 bits take for 1024
    B, T, pages, D = 3969, 63114, 1338, 64
    q = torch.zeros((T, 8, D), dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros((1, 8, 128, D), dtype=torch.bfloat16, device=DEV)
    pt = torch.zeros((B, pages), dtype=torch.int32, device=DEV)
    sl = torch.full((B,), pages * 128, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T] * ((B + 1) // 2), dtype=torch.int32, device=DEV)
    ws = sa.dense_attention_workspace(T, 8, 8, D, DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sa.sa_chunk_attention(q, kv, kv, pt, sl, cu, 0.125, workspace=ws, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) & 4
    c = chunk_case(80, [1, 30], [2000, 500], 4, 2, 128, 16)
    o, lse, err = run_chunk(c, workspace=ws)
    assert err == 0
    check(o, lse, c["q"], c["ks"], c["vs"], [1, 30], c["scale"], 0)


@pytest.mark.parametrize("ns,Ls,G,D", [([35], [3000], 7, 128), ([3], [2500], 8, 128), ([60, 2], [900, 700], 4, 64)])
def test_queries_that_are_nobodys_change_no_bit(ns, Ls, G, D):
    # the boxes of queries bring the tokens behind a batch along: whatever they hold, the
    # rows that are kept are the same bits
    c = chunk_case(81, ns, Ls, G, 2, D, 16, tail=40)
    want = run_chunk(c)
    for x in (float("nan"), float("inf"), 3e38):
        c["q"][sum(ns):] = x
        o, lse, err = run_chunk(c)
        assert err == 0 and torch.equal(o[:sum(ns)], want[0][:sum(ns)])
        assert torch.equal(lse[:sum(ns)], want[1][:sum(ns)])


# ------------------------------------------------------------------ behind the window
BEHIND = [
    # ns, Ls, G, Hkv, D, P, window
    ([1], [700], 4, 2, 128, 16, 100),
    ([1, 90], [5000, 600], 4, 1, 64, 64, 1),
    ([40, 300], [800, 900], 4, 2, 128, 16, 100),       # items of two full row tiles
    ([20, 20], [900, 500], 8, 2, 64, 48, 130),
    ([5, 1], [3000, 290], 4, 2, 128, 256, 333),        # pages larger than a tile
    ([1] * 40, [1000 + 37 * i for i in range(40)], 4, 2, 64, 16, 129),
    ([130, 1], [130, 400], 2, 3, 128, 32, 17),         # nothing behind the first one's window
]


def _release(c, ns, P, window, ids):
    """The keys behind each sequence's window become NaN; ids: the pages that hold nothing
    else leave the map."""
    for b, (n, k) in enumerate(zip(ns, c["ks"])):
        first = max(0, k.shape[0] - n - window + 1)    # the first key that any token sees
        for p in range(-(-first // P)):
            ph, m = int(c["pt"][b, p]), min(P, first - p * P)
            c["kc"][ph, :, :m] = NAN
            c["vc"][ph, :, :m] = NAN
            if ids and m == P:
                c["pt"][b, p] = -1 if p % 2 else 10 ** 7


@pytest.mark.parametrize("ids", [False, True])
@pytest.mark.parametrize("ns,Ls,G,Hkv,D,P,window", BEHIND)
def test_what_lies_behind_the_window_is_not_looked_at(ns, Ls, G, Hkv, D, P, window, ids):
    c = chunk_case(60 + sum(Ls), ns, Ls, G, Hkv, D, P)
    _release(c, ns, P, window, ids)
    o, lse, err = run_chunk(c, window)
    assert err == 0
    check(o, lse, c["q"], c["ks"], c["vs"], ns, c["scale"], window)
    direc, blocks = W.page_directory(c["pt"], c["sl"], P, 2)
    e = torch.zeros(1, dtype=torch.int32, device=DEV)
    o2, lse2 = sa.sa_chunk_attention_dir(c["q"], c["kc"], c["vc"], direc, blocks, 2, c["sl"], c["cu"], c["scale"],
                                         window=window, dev_error=e)
    torch.cuda.synchronize()
    assert int(e.item()) == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_missing_page_inside_the_window_is_still_flagged():
    ns, Ls, P, window = [4], [900], 16, 200
    c = chunk_case(61, ns, Ls, 4, 2, 128, P)
    _release(c, ns, P, window, True)
    c["pt"][0, 50] = -1                                # keys 800 .. 815
    o, lse, err = run_chunk(c, window)
    assert err == 2
    # the keys of that page are left out: the visible ones around it are the same for a
    # sequence that never had them, positions and window shortened by a page
    keep = torch.cat((torch.arange(800), torch.arange(816, 900))).to(DEV)
    check(o, lse, c["q"], [c["ks"][0][keep]], [c["vs"][0][keep]], ns, c["scale"], window - 16)


@pytest.mark.parametrize("n,L,window,D", [(1, 500, 70, 128), (40, 700, 129, 64), (100, 900, 33, 128)])
def test_packed_keys_behind_the_window_are_not_looked_at(n, L, window, D):
    g = torch.Generator().manual_seed(L)
    q, k, v = _randn(g, n, 8, D), _randn(g, L, 2, D), _randn(g, L, 2, D)
    k2, v2 = k.clone(), v.clone()
    k2[:L - n - window + 1] = NAN
    v2[:L - n - window + 1] = NAN
    o, lse = sa.sa_prompt_attention(q, k2, v2, _cu([n]), _cu([L]), 0.1, window=window)
    torch.cuda.synchronize()
    check(o, lse, q, [k], [v], [n], 0.1, window)


# ------------------------------------------------------------------ windows past 32 bits
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 1, 2 ** 40 + 7])
def test_windows_past_32_bits_are_no_limit(window):
    c = chunk_case(62, [3], [300], 4, 2, 64, 16)
    want, want_lse, _ = run_chunk(c)
    o, lse, _ = run_chunk(c, window)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    q, k, v = c["q"], c["ks"][0], c["vs"][0]
    a = sa.sa_prompt_attention(q, k, v, _cu([3]), _cu([300]), 0.1)
    b = sa.sa_prompt_attention(q, k, v, _cu([3]), _cu([300]), 0.1, window=window)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("window", [-1, -2 ** 32 + 5, -2 ** 40])
def test_negative_windows_are_refused(window):
    c = chunk_case(62, [3], [300], 4, 2, 64, 16)
    with pytest.raises(sa.SAError):
        run_chunk(c, window)


# ------------------------------------------------------------------ appends that skip
def _long_table(n):
    f = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    return torch.from_numpy(np.concatenate((np.cos(f), np.sin(f)), 1).astype(np.float32)).to(DEV)


def test_a_length_past_the_page_map_skips_the_sequence_and_its_queries():
    c = _case(70, [6, 3], [0, 5], 4, 2, 64, 16, 64)
    cap = c["pt"].shape[1] * 16
    for bad in (cap + 1, cap + 40, 2 ** 30):
        d = dict(_gpu(c), sl=_i32([bad, 5]), table=_long_table(500))
        before = {k: d[k].clone() for k in ("kc", "vc", "sig")}
        qo = torch.full_like(d["q"], 7.0)
        qo, new, err = _run(d, q_out=qo)
        assert err & 1 and bool((qo[:6] == 7).all())
        q, _, kc, vc, sig, _ = _want(dict(c, q=c["q"][6:], k=c["k"][6:], v=c["v"][6:], cu=np.array([0, 3]),
                                          pt=c["pt"][1:], sl=c["sl"][1:]))
        assert np.array_equal(_bits(qo)[6:], q)
        mine = int(c["pt"][1, 0])
        for k, x in (("kc", kc), ("vc", vc), ("sig", sig)):
            assert np.array_equal(_bits(d[k])[mine], x[mine])
            rest = torch.arange(d[k].shape[0], device=DEV) != mine
            assert torch.equal(d[k][rest].view(torch.int16), before[k][rest].view(torch.int16))


@pytest.mark.parametrize("lens,cu,want", [
    ([-4, 5], [0, 20, 23], [-4, 8]),            # a negative length
    ([5000, 5], [0, 20, 23], [5000, 8]),        # one past the page map
    ([0, 5], [-5, 20, 23], [0, 8]),             # offsets outside the tokens
    ([0, 5], [0, 20, 5000], [20, 5]),
    ([0, 5], [0, -1, 23], [0, 5]),              # offsets that turn back
    ([30, 5], [0, 20, 23], [50, 8]),            # tokens past the page map: counted, flagged
])
def test_every_sequence_reports_its_length(lens, cu, want):
    c = _case(71, [20, 3], [0, 5], 4, 2, 64, 16, 64)
    d = dict(_gpu(c), sl=_i32(lens), cu=_i32(cu))
    _, new, err = _run(d)
    assert err != 0 and new.tolist() == want


def test_lengths_of_many_sequences():
    # more sequences than one block reports, good and bad ones mixed
    B = 700
    rng = np.random.default_rng(2)
    ns = [int(x) for x in rng.integers(0, 3, B)]
    c = _case(72, ns, [int(x) for x in rng.integers(0, 20, B)], 2, 1, 64, 16, 64)
    d = _gpu(c)
    _, new, err = _run(d)
    assert err == 0 and np.array_equal(new.cpu().numpy(), _want(c)[5])
    sl = c["sl"].copy()
    sl[::97] = -1
    want = np.where(sl < 0, sl, sl + np.array(ns))
    _, new, err = _run(dict(_gpu(c), sl=_i32(sl)))
    assert err & 1 and np.array_equal(new.cpu().numpy(), want)


def test_offsets_that_turn_back_are_flagged_wherever_they_do():
    # the tokens of the sequence between do not exist, and its page slots are another's
    c = _case(73, [100, 10, 90], [0, 0, 0], 2, 1, 64, 16, 64)
    _, new, err = _run(dict(_gpu(c), cu=_i32([0, 100, 50, 200])))
    assert err & 4 and int(new[1]) == 0


# ------------------------------------------------------------------ the optional LSE, the largest batch
def test_without_an_lse():
    c = chunk_case(63, [1, 30, 300], [2000, 500, 700], 4, 2, 128, 16)
    want, _, _ = run_chunk(c)
    q, o = c["q"], torch.empty_like(c["q"])
    ws = sa.dense_attention_workspace(q.shape[0], 8, 2, 128, DEV)
    s3, s4 = (lambda t: (ctypes.c_int64 * 3)(*t.stride())), (lambda t: (ctypes.c_int64 * 4)(*t.stride()))
    lib, st = sa.load(), torch.cuda.current_stream().cuda_stream
    assert lib.sa_chunk_attention(q.data_ptr(), s3(q), c["cu"].data_ptr(), q.shape[0], c["kc"].data_ptr(), s4(c["kc"]),
                                  c["vc"].data_ptr(), s4(c["vc"]), c["pt"].data_ptr(), c["pt"].shape[1],
                                  c["sl"].data_ptr(), 3, 8, 2, 128, 16, c["kc"].shape[0], c["scale"], 0, o.data_ptr(),
                                  None, ws.data_ptr(), ws.numel(), None, st) == 0
    torch.cuda.synchronize()
    assert torch.equal(o, want)


def test_the_largest_batch():
    B, L, D, P = 4096, 20, 64, 32
    g = torch.Generator().manual_seed(9)
    rng = np.random.default_rng(3)
    ns = [int(x) for x in rng.integers(0, 2, B)]
    q, kc, vc = _randn(g, sum(ns), 2, D), _randn(g, B, 1, P, D), _randn(g, B, 1, P, D)
    pt = torch.randperm(B, generator=g).to(torch.int32).to(DEV).view(B, 1)
    sl = torch.from_numpy(rng.integers(1, L + 1, B).astype(np.int32)).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = sa.sa_chunk_attention(q, kc, vc, pt, sl, _cu(ns), 0.125, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    b = torch.tensor([i for i, n in enumerate(ns) if n], device=DEV)
    k, v = (x[pt[b, 0].long(), 0].double() for x in (kc, vc))
    hide = torch.arange(P, device=DEV)[None, :] >= sl[b][:, None]
    s = 0.125 * torch.einsum("bhd,bld->bhl", q.double(), k)
    reach = 0.125 * torch.einsum("bhd,bld->bhl", q.double().abs(), k.abs()).masked_fill(hide[:, None], 0.0).amax(-1)
    s = s.masked_fill(hide[:, None], -math.inf)
    w = torch.softmax(s, -1)
    A, ref = torch.einsum("bhl,bld->bhd", w, v.abs()), torch.einsum("bhl,bld->bhd", w, v)
    eta = (D + 4) * 2.0 ** -23 * reach + 2.0 ** -21        # the bounds of test_gpu_dense.py
    assert bool(((o.double() - ref).abs() <= U * (A + ref.abs()) * (1 + U) + 4 * eta[..., None] * A).all())
    z = torch.logsumexp(s, -1)
    assert bool(((lse.double() - z).abs() <= eta + 21 * 2.0 ** -24 + 2.0 ** -22 * z.abs()).all())


def test_pages_past_32_bits_of_elements():
    # the last pages of a pool of more than 2^31 elements: appended to, then attended over
    Hq, Hkv, P, D, n = 16, 8, 16, 128, 100
    pool = (1 << 31) // (Hkv * P * D) + 10
    kc, vc = (torch.empty((pool, Hkv, P, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sig = torch.empty((pool, Hkv, D), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(6)
    q, k, v = (_randn(g, n, h, D) for h in (Hq, Hkv, Hkv))
    pt = (pool - 1 - torch.arange(7, dtype=torch.int32, device=DEV)).view(1, 7).contiguous()
    table, k_out, lens = _long_table(n), torch.empty_like(k), torch.empty(1, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo, _ = sa.sa_append_kv_rope(q, k, v, _cu([n]), table, kc, vc, pt, _i32([0]), sig, k_out=k_out, out_seq_lens=lens,
                                 dev_error=err)
    o, lse = sa.sa_chunk_attention(qo, kc, vc, pt, lens, _cu([n]), 0.09, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and lens.tolist() == [n]
    rows = kc[pt[0].long()].transpose(1, 2).reshape(-1, Hkv, D)[:n]
    assert torch.equal(rows, k_out) and torch.equal(vc[pt[0].long()].transpose(1, 2).reshape(-1, Hkv, D)[:n], v)
    assert torch.equal(sig[pt[0, 0].long()], k_out[:P].double().mean(0).to(torch.bfloat16))
    check(o, lse, qo, [k_out], [v], [n], 0.09, 0)
