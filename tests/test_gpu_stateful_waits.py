"""The bounded waits of the calls that keep state: with a lowered limit their
kernels give up, report it and return, and the next call is right. Nothing here
faults or hangs the GPU: every wait ends by itself, and what is in flight is
waited for on the way out."""
import pytest
import torch

from test_gpu_cache import Cache, offsets
from test_gpu_decay import _inputs
from test_gpu_diag import _status_code

pytestmark = pytest.mark.gpu

DEV = "cuda"
NONE, ONE = 100, 8000      # cycles: below one try, and one try (about 4 us)


def _gives_up(sa, call, limit, always=True):
    ref = call()
    torch.cuda.synchronize()
    assert _status_code(sa) == "SA_OK"
    try:
        sa.sa_diag_set_wait_limit(limit)
        call()
        torch.cuda.synchronize()
    finally:
        sa.sa_diag_set_wait_limit(0)
    code = _status_code(sa)
    assert code == "SA_ERR_DEVICE_TIMEOUT" or (code == "SA_OK" and not always)
    assert _status_code(sa) == "SA_OK"                      # the read cleared it
    for _ in range(2):
        got = call()
        torch.cuda.synchronize()
        assert _status_code(sa) == "SA_OK"
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("kv,new,d", [([3000, 1500], [1, 1], 128), ([700, 90], [300, 90], 64)])
def test_attention_gives_up(cuda_lib, kind, kv, new, d):
    sa = cuda_lib
    c = Cache(kind, kv, 2, d, 64, seed=1)
    c.fill(sa, 2)
    q = torch.randn(sum(new), 8, d, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).to(torch.bfloat16)
    call = lambda: sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets(new), c.lens(), max(new), want_lse=True, **c.args())
    _gives_up(sa, call, NONE)
    _gives_up(sa, call, ONE, always=False)


@pytest.mark.parametrize("B,H,N,d", [(1, 2, 3000, 64), (1, 2, 3000, 128), (1, 148, 600, 64), (1, 148, 2000, 128)])
def test_decayed_attention_gives_up(cuda_lib, B, H, N, d):
    """Cut heads and whole ones (of d = 128, a chunk of which takes longer than the one
    try: those stop in the middle, with loads, products and stores in flight)."""
    sa = cuda_lib
    x = _inputs(B, H, N, d, 4)
    fwd = lambda: sa.sa_decay_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"], want_state=True)
    bwd = lambda: sa.sa_decay_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dout"], state=x["state"], dstate=x["dstate"])
    for call in (fwd, bwd):
        _gives_up(sa, call, NONE)
        _gives_up(sa, call, ONE, always=False)
