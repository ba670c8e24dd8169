"""A wait of the attention over 8-bit pages that runs out: the call ends, the status says so, every row that the waiting CTA had a part
in is NaN, the others are right, and so is the next call (the hook is described in test_gpu_paged_timeout.py)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_rows_of_a_wait_that_ran_out_are_nan():
    env = dict(os.environ, TKV_FAULT_INJECT="wait:-1", PYTHONPATH=os.path.dirname(HERE) + os.pathsep + HERE)
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "8 shapes" in r.stdout, r.stdout


def child():
    import numpy as np
    import torch

    import tiered_kv_cache_gqa_gb300 as tkv
    from test_gpu_paged import BF16, close, ints, queries
    from test_gpu_paged8 import Pool8

    shapes = 0
    for d in (64, 128):
        for lengths, n, G, max_len, max_new in (([2500, 700, 0, 90, 300], [1, 1, 1, 0, 1], 4, 2500, 1),      # items cut by CTAs
                                                ([200, 30, 0, 250, 256] * 40, [1, 2, 1, 0, 1] * 40, 2, 256, 2),   # whole items
                                                ([1500, 700, 90], [7, 3, 20], 4, 1500, 20),                  # tiles of 16 rows
                                                ([1500, 700, 90], [7, 3, 20], 4, 1 << 30, 20)):              # and of 32
            p = Pool8(lengths, n, d=d).fill()
            q = queries(p, G)
            want = p.oracle(q)
            seen = 0
            for warp in list(range(0, 70, 3)) + list(range(70, 304 * 7, 97)):
                os.environ["TKV_FAULT_INJECT"] = "wait:%d" % warp
                out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
                status = ints([0])
                p.cache.attend(q, p.cu_t, max_new=max_new, max_len=max_len, out=out, lse=lse, status=status)
                bad = out.isnan().all(-1)
                assert status.item() == (tkv.TKV_ETIMEOUT if bad.any() else 0), (d, lengths, warp)
                assert torch.equal(bad, lse.isnan()) and torch.equal(bad, out.isnan().any(-1))
                o64 = want[0].copy()
                o64[bad.cpu().numpy()] = np.nan
                close(p, out, lse, (o64,) + want[1:], BF16)          # what is not NaN is right
                seen += bool(bad.any())
            assert seen >= 3, (d, lengths, seen)
            os.environ["TKV_FAULT_INJECT"] = "wait:-1"
            close(p, *p.cache.attend(q, p.cu_t, max_new=max_new, max_len=max_len, return_lse=True), want, BF16)
            shapes += 1
    print(shapes, "shapes")


if __name__ == "__main__":
    child()
