"""The gated product's bounded waits, without a GPU fault: with MOE_TEST_STALL_PRODUCER=1 no stage is ever filled, the
waits expire after MOE_WAIT_TIMEOUT_NS, the status words report it and the context stays usable.  A child
process, because both variables are read once per process."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, sys, time
sys.path.insert(0, sys.argv[1])
import torch
import block_scaled_moe_topk_gb300 as moe
E, M, I, K = (int(v) for v in sys.argv[2:6])
dev = torch.device("cuda", 0)
z = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device=dev)
x, xs = z(M, K, dtype=torch.uint8), z(M, -(-K // 128), dtype=torch.float32)
w, ws = z(E, 2 * I, K, dtype=torch.uint8), z(E, -(-2 * I // 128), -(-K // 128), dtype=torch.float32)
off = torch.arange(E + 1, device=dev) * (M // E)
off[-1] = M
codes, scales = z(M, I, dtype=torch.uint8), z(M, -(-I // 128), dtype=torch.float32)
space = z(moe.moe_gemm_fp8_block_workspace_bytes(M, 2 * I, K, E), dtype=torch.uint8)
t0 = time.time()
moe.moe_gemm_fp8_block_swiglu(x, xs, w, ws, space, codes=codes, scales=scales, offsets=off)
torch.cuda.synchronize()
dt = time.time() - t0
status = moe.moe_read_device_status(space)
words = space.view(torch.int32)[:8].cpu().tolist()
alive = float((torch.arange(1000, device=dev, dtype=torch.float32) * 2).sum().item())
print(json.dumps({"status": status, "words": words, "alive": alive, "seconds": dt}))
"""

# (E, M, I, K), and the form that runs
CASES = {"split": ((1, 16, 128, 4096), 4), "single": ((2, 200, 2048, 512), 2), "pair": ((1, 8192, 512, 2048), 3)}


@pytest.mark.parametrize("case", list(CASES))
def test_expired_wait_is_reported_and_the_context_survives(case):
    import __graft_entry__
    __graft_entry__.build()
    args, form = CASES[case]
    env = dict(os.environ, MOE_TEST_STALL_PRODUCER="1", MOE_WAIT_TIMEOUT_NS="50000000")  # 50 ms
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, *map(str, args)], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    d = json.loads(r.stdout.strip().splitlines()[-1])
    words = d["words"]
    assert d["status"] == 6 and words[1] == 1 and words[7] == form
    assert words[6] >= 25000                   # it waited the limit (50 ms or more at 2 GHz or less), in us
    assert d["alive"] == 999000.0 and d["seconds"] < 60
