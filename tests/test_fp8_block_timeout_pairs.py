"""An expired wait of the FP8 product on CTA pairs: the record in the status words, by the pair kernel's own barriers.

Barriers of a pair: 4 stage-filled (0-3), 4 stage-free (4-7), then the accumulators' ready ones, two buffers of two
column halves: half h of the first buffer is 8 + h.  With no stage ever filled the first wait to expire is that of an
issuing warp (1 or 3, one for each half) on stage 0, or that of a summing warp (4-7 half 0, 8-11 half 1) on the
first buffer of its half."""
import json
import os
import subprocess
import sys

import pytest

from test_fp8_block_timeout import CHILD, ROOT

PAIR = 3


@pytest.mark.gpu
@pytest.mark.parametrize("dgrad", [0, 1])
def test_expired_wait_on_pairs_names_the_barrier(dgrad):
    import __graft_entry__
    __graft_entry__.build()
    env = dict(os.environ, MOE_TEST_STALL_PRODUCER="1", MOE_WAIT_TIMEOUT_NS="50000000")  # 50 ms
    for M in (8192, 16384, 32768):
        r = subprocess.run([sys.executable, "-c", CHILD, ROOT, *map(str, (1, M, 2048, 2048, dgrad))], env=env,
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        d = json.loads(r.stdout.strip().splitlines()[-1])
        words = d["words"]
        if words[7] == PAIR:
            break
    assert words[7] == PAIR, "no size ran on pairs"
    assert d["status"] == 6 and words[1] == 1
    bar, warp = words[2], words[5]
    assert (bar == 0 and warp in (1, 3)) or (4 <= warp <= 11 and bar == 8 + (warp - 4) // 4), words
    assert words[6] >= 25000
    assert d["alive"] == 999000.0 and d["seconds"] < 60
