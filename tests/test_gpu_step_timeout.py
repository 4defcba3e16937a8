"""Window attention after waits that ran out: what CTA 0 had to do is left as it was, everything else is right, and so is
the next call."""
import time

import pytest
import torch

from deepseek_v4_sparse_c128_gb300 import binding
from test_gpu_step_window import Case, consecutive

pytestmark = pytest.mark.gpu
TIMEOUT = 32


@pytest.mark.parametrize("window,H", [(30, 1), (300, 1), (300, 20)], ids=["short", "long", "long_many_heads"])
def test_a_cta_that_gives_up(window, H):
    # 400 tokens: in order over the CTAs, so CTA 0 has the first of them
    c = Case(50, consecutive(0, 0, 200) + consecutive(1, 5, 200), [200, 205], H, window, 2, 16)
    dev = [torch.from_numpy(a).cuda() for a in (c.cache, c.table, c.req, c.pos, c.slots)]
    out = torch.full((400, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((400, H), 7.0, device="cuda")
    q = c.q.cuda()
    args = (q, dev[0], c.block, *dev[1:], c.window, c.scale, out)
    torch.cuda.synchronize()
    start = time.monotonic()
    binding.debug_stall_window_attention(*args, first=c.first, lse=lse)
    assert binding.device_errors() == TIMEOUT
    assert time.monotonic() - start < 30
    left = ((out == 3).all(-1) & (lse == 7)).any(-1).cpu().tolist()  # (of some heads at least)
    assert left[0] and not all(left)
    first = left.index(False)
    assert all(left[:first]) and not any(left[first + 4:])  # (a run of tokens behind may be shared with CTA 0)
    c.check(out, lse, tokens=[t for t in range(0, 400, 7) if not left[t]])
    binding.window_attention(*args, first=c.first, lse=lse)
    assert binding.device_errors() == 0
    c.check(out, lse, tokens=range(0, 400, 13))
