"""Absorbed attention over an FP8 latent pool: what its codes, scales and factors could get wrong."""
import pytest
import torch

import latent_reference as R
from paged_kv_cache_95_gb300 import pagedkv as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    P.load_library()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def status_of(ws):
    return int(ws[:4].view(torch.int32).cpu().item()) & 0xFFFFFFFF


@pytest.mark.parametrize("heads", [16, 32, 64])
def test_sequences_of_one_tile_keep_their_own_query_factors(heads):
    """Hundreds of sequences of up to 64 tokens, whose queries differ in size by 2^8 from one to the next: a query's
    factor taken for its neighbour's would make its scores 256 times too large or too small."""
    lens = [1 + (i * 29) % 64 for i in range(400)]
    pool = R.Pool(heads, lens, True)
    g = R.gen(heads + 1)
    size = torch.tensor([1.0 if i % 2 else 2.0 ** -8 for i in range(len(lens))]).bfloat16()[:, None, None]
    ql, qr = R.normal(g, len(lens), heads, 512) * size, R.normal(g, len(lens), heads, 64)
    ref, tol = R.decode(ql, qr, pool, 1)
    d, q, tables, ctx = pool.device(), (ql.cuda(), qr.cuda()), pool.tables.cuda(), i32(lens)
    first = None
    for _ in range(30):
        out = torch.full((len(lens), heads, 512), R.NAN, device="cuda")
        ws = P.latent_attention_decode(out, *q, block_tables=tables, context_lens=ctx, scale=R.SCALE, **d)
        if first is None:
            first = out
            R.assert_within(out, ref, tol, "one tile a sequence")
        assert torch.equal(out, first)
        assert status_of(ws) == 0
