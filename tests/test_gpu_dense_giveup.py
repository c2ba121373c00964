"""The dense attention's way out of a wait that runs out (marked gpu): a build of the
library whose waits give up after a few polls, which every call reaches, has to report
SA_DEVERR_TIMEOUT, end by itself and leave the GPU to the next call."""
import math
import os

import pytest
import torch

import paged_sparse_kv_sa_b200 as sa
from paged_sparse_kv_sa_b200 import _lib, build
from test_gpu_dense import _cu, _randn, check, chunk_case, run_chunk

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    """The library with dense.cu rebuilt for waits of 8 polls that do not suspend."""
    d = str(tmp_path_factory.mktemp("hasty"))
    os.makedirs(build.OBJ, exist_ok=True)
    objs = [build._compile(s, False) for s in build.SOURCES if s != "dense.cu"]
    objs.append(build._compile("dense.cu", True, d, ("SA_DENSE_POLLS=8",)))
    out = os.path.join(d, "libsa_hasty.so")
    build.subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-o", out, *objs, "-lcudart"], check=True)
    return out


CASES = [
    # ns, Ls, G, Hkv, D, P, window
    ([1], [3000], 4, 2, 128, 16, 0),                 # few rows, one tile a CTA
    ([1] * 24, [4000] * 24, 8, 8, 128, 16, 0),       # full rings
    ([300, 1, 700], [2000, 900, 700], 4, 8, 128, 16, 0),
    ([500, 40], [500, 2100], 3, 8, 64, 48, 700),     # rows that are no key, several planning batches
    ([20] * 300, [60] * 300, 2, 8, 64, 16, 0),
]


def test_waits_that_run_out_are_reported_and_leave_the_gpu_usable(hasty, monkeypatch):
    cases = [(chunk_case(90 + i, *c[:6]), c) for i, c in enumerate(CASES)]
    monkeypatch.setattr(_lib, "_lib", None)
    _lib.load(hasty)
    for c, (ns, Ls, G, Hkv, D, P, window) in cases:
        for _ in range(5):
            o, lse, err = run_chunk(c, window)
            assert err == 8
    q, k, v = (_randn(torch.Generator().manual_seed(1), 2000, h, 128) for h in (32, 8, 8))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sa.sa_prompt_attention(q, k, v, _cu([2000]), _cu([2000]), 0.1, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 8
    monkeypatch.undo()
    for c, (ns, Ls, G, Hkv, D, P, window) in cases:
        o, lse, err = run_chunk(c, window)
        assert err == 0
        if sum(ns) < 2000:
            check(o, lse, c["q"], c["ks"], c["vs"], ns, 1.0 / math.sqrt(D), window)
