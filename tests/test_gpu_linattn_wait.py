"""The bounded waits of linear attention on the tensor cores, run out on purpose.

In libgdn_waittest.so every wait gives up after 5 ms, and one warp of the first
block (sequence 0, head 0, first 64 columns of v) does not signal that the state
before chunk 1 is written, so that the product with it is waited for in vain.
Nothing asynchronous is left in flight by that.  The kernel raises
GDN_DEV_WAIT_TIMEOUT and returns, the states of that block are not written, every
other block's results are right, and an ordinary call afterwards is too.
"""
import ctypes
import time

import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from linattn_exact import agrees, walk
from test_gpu_linattn import make, on_tensor_cores
from test_gpu_wait_timeout import waittest_lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("odd", [False, True])
def test_a_wait_that_runs_out(monkeypatch, odd):
    from gated_delta_rule_09_gb300 import _lib
    H, d, T = 2, 128, 640                                        # five chunks, eight blocks
    x = {n: t.clone() for n, t in make((2, T), H, H, d, d, "bf16", seed=43).items()}
    if odd:                                                      # in the first block, behind the chunk that stalls
        x["v"][0, 300, 0, 3] = float("inf")
    assert on_tensor_cores(x) and gdn.gdn_get_device_status() == 0
    ro, bo, rS, bS = walk(**{**x, "v": torch.nan_to_num(x["v"], posinf=0.0)}, parts=True)
    lib = waittest_lib()
    out = torch.full((2, H, d, d), 7.0, device="cuda")
    with monkeypatch.context() as m:
        m.setattr(_lib, "load", lambda *a, **k: lib)
        w = make((1, 128), 1, 1, d, d, "bf16")                   # one chunk: nothing is withheld
        gdn.gdn_linattn_fwd(**w)
        assert gdn.gdn_get_device_status() == 0
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        o, S = gdn.gdn_linattn_fwd(**x, state_out=out)
        flags = ctypes.c_uint(0)
        st = lib.gdn_get_device_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), ctypes.byref(flags))
        elapsed = time.perf_counter() - t0
    assert st == _lib.GDN_ERR_TIMEOUT and flags.value == _lib.GDN_DEV_WAIT_TIMEOUT, (st, flags.value)
    assert elapsed < 1.0, elapsed
    assert bool((S[0, 0, :64] == 7.0).all())                     # the first block's state
    for n in range(2):
        for h in range(H):
            for v0 in (0, 64):
                if (n, h, v0) != (0, 0, 0):
                    cut = (n, slice(None), h, slice(v0, v0 + 64))
                    assert agrees(o[cut], ro[cut], bo[cut]) <= 1
                    assert agrees(S[n, h, v0:v0 + 64], rS[n][h, v0:v0 + 64], bS[n][h, v0:v0 + 64]) <= 1
    x["v"] = torch.nan_to_num(x["v"], posinf=0.0)
    o, S = gdn.gdn_linattn_fwd(**x)
    assert gdn.gdn_get_device_status() == 0 and agrees(o, ro, bo) <= 1
    assert all(agrees(S[n], rS[n], bS[n]) <= 1 for n in range(2))
