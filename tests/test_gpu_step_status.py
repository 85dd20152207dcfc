"""One status word for the calls of a speculative step: the first of the tree attention's workspace."""
import pytest
import torch

from paged_kv_cache_95_gb300 import pagedkv as P
from test_gpu_tree import Problem, i32, status_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    P.load_library()


@pytest.mark.parametrize("fp8", [False, True])
def test_one_word_for_a_step(fp8):
    p = Problem([4, 3], [40, 30], 4, 2, fp8, seed=1)
    _, ws = p.call()
    word = ws[:4].view(torch.int32)
    tables, ctx, cu = i32(p.tables), i32(p.ctx), i32(p.cu)
    target = torch.softmax(torch.randn(7, 50, device="cuda"), -1)
    out, path = (torch.zeros(2, 4, dtype=torch.int32, device="cuda") for _ in "ab")
    counts = torch.zeros(2, dtype=torch.int32, device="cuda")

    def verify(cu):
        P.speculative_verify(out, path, counts, target, i32([1] * 7), cu, 4, torch.full((7,), 0.5, device="cuda"), status=word)

    def compact(path, counts, tables):
        P.kv_compact_path(p.k, p.v, tables, ctx, cu, i32(path), i32(counts), status=word, **p.scales)

    verify(cu)
    compact([[0, 2, 3, -1], [0, 2, -1, -1]], [3, 2], tables)
    assert status_of(ws) == 0
    verify(i32([0, 4, 99]))
    assert status_of(ws) == P.PKV_STATUS_BAD_Q_LEN
    bad = i32(p.tables)
    bad[1, 1] = 10 ** 6  # position 29
    compact([[0, -1, -1, -1], [0, 2, -1, -1]], [1, 2], bad)
    assert status_of(ws) == P.PKV_STATUS_BAD_Q_LEN | P.PKV_STATUS_BAD_BLOCK_ID
    p.call(workspace=ws)  # (sticky: the word is the caller's to clear)
    assert status_of(ws) == P.PKV_STATUS_BAD_Q_LEN | P.PKV_STATUS_BAD_BLOCK_ID
