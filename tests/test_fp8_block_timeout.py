"""The FP8 product's bounded waits, without a GPU fault: with MOE_TEST_STALL_PRODUCER=1 no stage is
ever filled, the waits expire after MOE_WAIT_TIMEOUT_NS, the status words report it and the context
stays usable.  A child process, because both variables are read once per process."""
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
E, M, N, K, dgrad = (int(v) for v in sys.argv[2:7])
dev = torch.device("cuda", 0)
red, cols = (N, K) if dgrad else (K, N)
z = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device=dev)
x, xs = z(M, red, dtype=torch.uint8), z(M, -(-red // 128), dtype=torch.float32)
w, ws = z(E, N, K, dtype=torch.uint8), z(E, -(-N // 128), -(-K // 128), dtype=torch.float32)
off = torch.arange(E + 1, device=dev) * (M // E)
off[-1] = M
out = z(M, cols, dtype=torch.float32)
space = z(moe.moe_gemm_fp8_block_workspace_bytes(M, N, K, E), dtype=torch.uint8)
call = moe.moe_gemm_fp8_block_dgrad if dgrad else moe.moe_gemm_fp8_block
t0 = time.time()
call(x, xs, w, ws, out, space, offsets=off)
torch.cuda.synchronize()
dt = time.time() - t0
status = moe.moe_read_device_status(space)
words = space.view(torch.int32)[:8].cpu().tolist()
alive = float((torch.arange(1000, device=dev, dtype=torch.float32) * 2).sum().item())
print(json.dumps({"status": status, "words": words, "alive": alive, "seconds": dt}))
"""


# (E, M, N, K, dgrad), and the index of the first accumulator-ready barrier: 2 x 4 stages on single
# CTAs, 2 x 6 on pairs (one for each half of the columns: 12 and 13)
CASES = {"split": ((1, 16, 256, 4096, 0), 8), "single": ((2, 200, 4096, 512, 0), 8),
         "single_dgrad": ((2, 200, 512, 4096, 1), 8), "pair": ((1, 8192, 1024, 256, 0), 12)}


@pytest.mark.parametrize("case", list(CASES))
def test_expired_wait_is_reported_and_the_context_survives(case):
    import __graft_entry__
    __graft_entry__.build()
    args, acc_ready = CASES[case]
    env = dict(os.environ, MOE_TEST_STALL_PRODUCER="1", MOE_WAIT_TIMEOUT_NS="50000000")  # 50 ms
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, *map(str, args)], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    d = json.loads(r.stdout.strip().splitlines()[-1])
    words = d["words"]
    assert d["status"] == 6 and words[1] == 1  # MOE_ERR_DEVICE_TIMEOUT, an expiry was recorded
    # the first expiry: stage 0 in an MMA warp (1; 3 too on pairs), or the accumulator in a summing warp
    assert (words[2] == 0 and words[5] in (1, 3)) or (words[2] - acc_ready in (0, acc_ready // 12) and 4 <= words[5] <= 11), words
    assert words[6] >= 25000                   # it waited the limit (50 ms or more at 2 GHz or less), in us
    assert d["alive"] == 999000.0 and d["seconds"] < 60
