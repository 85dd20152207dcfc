"""A workspace that the binding allocates belongs to the stream of the call: another, busy stream neither delays the call
nor clears its status word behind it."""
import pytest
import torch

from paged_kv_cache_95_gb300 import pagedkv as P

pytestmark = pytest.mark.gpu

B, N_Q, N_KV, BLOCKS, SCALE = 3, 8, 2, 64, 128.0 ** -0.5
LENS = [300, 40, 17]


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    P.load_library()


def status_of(ws):
    return int(ws[:4].view(torch.int32).cpu().item()) & 0xFFFFFFFF


def _calls():
    """name -> (out, call(stream) -> workspace); the last sequence names a block that does not exist."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = normal(BLOCKS, N_KV, 16, 128), normal(BLOCKS, N_KV, 16, 128)
    tables = torch.arange(B * 20, device="cuda").int().view(B, 20).contiguous()
    tables[2, 0] = BLOCKS + 3
    lens = i32(LENS)
    pool = (k, v, tables, lens, SCALE)
    q, qv, key, value = normal(B, N_Q, 128), normal(2 * B, N_Q, 128), normal(B, N_KV, 128), normal(B, N_KV, 128)
    out = {name: torch.zeros((2 if name in ("verify", "prefill") else 1) * B, N_Q, 128, device="cuda")
           for name in ("decode", "append", "verify", "prefill")}
    return {
        "decode": (out["decode"], lambda s: P.paged_attention_decode(out["decode"], q, *pool, stream=s)),
        "append": (out["append"], lambda s: P.paged_attention_decode_append(out["append"], q, key, value, *pool, stream=s)),
        "verify": (out["verify"], lambda s: P.paged_attention_verify(out["verify"], qv, 2, *pool, stream=s)),
        "prefill": (out["prefill"], lambda s, cu=i32([0, 2, 4, 6]): P.paged_attention_prefill_chunk(
            out["prefill"], qv, cu, 2, *pool, stream=s)),
    }


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["decode", "append", "verify", "prefill"])
def test_workspace_of_another_stream(name, handle):
    out, call = _calls()[name]
    ws = call(None)
    want, status = out.clone(), status_of(ws)
    assert status == P.PKV_STATUS_BAD_BLOCK_ID
    out.zero_()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second on the current stream
    ws = call(s.cuda_stream if handle else s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert status_of(ws) == status
