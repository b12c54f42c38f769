"""fp32 calls whose token codes fill the shared memory that a kernel has without
asking (48 KB, a few bytes of which the kernel uses itself), and calls of two
lengths from several host threads.  Padding throughout: only the launches matter.
"""

import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _b():
    from vla_prefix_lm_b200 import binding
    return binding


def _padding(S):
    x = torch.zeros(1, S, 1, 32, device="cuda")
    ar = torch.ones(S, dtype=torch.uint8, device="cuda")
    return x, ar, torch.full((S,), -1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("S", [12255, 12256, 12288])
def test_codes_that_fill_the_default_limit(S):
    b = _b()
    x, ar, seg = _padding(S)
    out = b.pi_attn_prefill(x, x, x, ar, seg, out=torch.full_like(x, 3.0))
    assert (out == 0).all()
    out = b.pi_attn_suffix(x, x, x, x[:, :5].contiguous(), x[:, :5].contiguous(), ar,
                           segment_ids=seg, out=torch.full_like(x, 3.0))
    assert (out == 0).all()
    assert int(b.pi_attn_debug_mask(ar, seg).sum()) == 0
    assert b.pi_attn_read_status() == b.PI_OK


def test_two_lengths_from_several_threads():
    b = _b()
    L = b.lib()
    jobs, bad = [], []
    for S in (16383, 12400):
        x, ar, seg = _padding(S)
        out = torch.full_like(x, 3.0)
        d = b.PiAttnDesc(1, S, 0, 1, 1, 32, b.PI_F32, 1.0, 0)
        p = [t.data_ptr() for t in (x, x, x, ar, seg, out)]
        jobs.append(((x, ar, seg, out), (ctypes.byref(d), *p, None, None)))

    def run(i):
        args = jobs[i % 2][-1]
        for _ in range(150):
            rc = L.pi_attn_prefill(*args)
            if rc != b.PI_OK:
                bad.append((i % 2, rc))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, (len(bad), bad[:3])
    for tensors, _ in jobs:
        assert (tensors[-1] == 0).all()
