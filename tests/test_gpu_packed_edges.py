"""Edges of the packed-batch operators (marked gpu)."""
import pytest
import torch

import paged_sparse_kv_sa_b200 as sa
from test_gpu_dense import check, chunk_case, run_chunk

pytestmark = pytest.mark.gpu
DEV = "cuda"


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
