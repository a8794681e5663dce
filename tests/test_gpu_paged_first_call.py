"""A process whose first call of the library is a captured attention or append:
what a kernel needs before its first launch is set up inside the capture."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import long_context_exact_ring_gb300 as ra
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
new = NEW
lens, cu, table = i([new + 3]), i([0, new]), i([list(range(8))])
pools = [torch.ones(8, 8, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
q = torch.ones(new, 4, 64, dtype=torch.bfloat16, device="cuda")
o, lse = torch.zeros_like(q), torch.zeros(4, new, device="cuda")
rows, slots = torch.full((1, 1, 64), 2.0, dtype=torch.bfloat16, device="cuda"), i([63])
ws = torch.empty(ra.paged_attn_workspace_size(1, new, 4, 1, 64), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    if APPEND:
        ra.paged_kv_append(rows, rows, *pools, slots)
    ra.paged_attn_fwd(q, *pools, table, lens, cu, True, o=o, lse=lse, workspace=ws)
g.replay()
torch.cuda.synchronize()
assert (o == 1).all(), o                         # every key has the same V
want = torch.log(torch.arange(4, 4 + new, device="cuda").double()) + 8
assert float((lse.double() - want).abs().max()) < 1e-4, lse
assert not APPEND or float(pools[0][7, 7].sum()) == 128
assert ra.check_status() == ra.RA_OK
"""


@pytest.mark.parametrize("new,append", [(1, False), (40, False), (1, True)])
def test_first_call_is_captured(new, append):
    from long_context_exact_ring_gb300 import build
    build.build()
    subprocess.run([sys.executable, "-c", PROGRAM.replace("NEW", str(new)).replace("APPEND", str(append))], check=True,
                   timeout=300)
