"""A wait of a bulk-copy ring that gives up: the ring of the RMS norm's gradient
and of the many-tensor AdamW, in a kernel whose one copy does not come in time.
No thread may leave before the others (they would wait at the next barrier),
no later copy may be requested, and what is under way lands before the end.
Every wait in it is bounded by the limit that the test gives."""

import pytest
import torch

pytestmark = pytest.mark.gpu
TIMEOUT, BIT_SELFTEST = 7, 0x10
LIMIT_US = 20000


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_06_b200 as q
    return q


# rounds 0 to 2 land; round 3 does not come in time; round 4, requested before anyone gave up, lands; nothing
# is requested after that
@pytest.mark.parametrize("mode,drained", [("NEVER", 0), ("LATE", 1)])
def test_a_copy_that_does_not_come_in_time(q, mode, drained):
    assert q.qlora_device_status() == (0, 0)
    out = torch.full((129,), -1, dtype=torch.int32, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    q.qlora_selftest_ring_timeout(LIMIT_US, getattr(q, "SELFTEST_RING_" + mode), out)
    end.record()
    assert q.qlora_device_status() == (TIMEOUT, BIT_SELFTEST)
    assert torch.all(out[:128] == 4) and int(out[128]) == drained
    # one limit for the wait (later ones end at once) and one for the drain; 10 ms for hardware waits and launch
    assert start.elapsed_time(end) <= 2 * LIMIT_US / 1000 + 10
    assert q.qlora_device_status() == (0, 0)


def test_one_thread_gives_up_while_the_copy_lands_for_the_others(q):
    out = torch.full((129,), -1, dtype=torch.int32, device="cuda")
    q.qlora_selftest_ring_timeout(LIMIT_US, q.SELFTEST_RING_ONE, out)
    assert q.qlora_device_status() == (TIMEOUT, BIT_SELFTEST)
    # rounds 0 to 3 for the others; thread 5 passes over round 2 and sees its copy in round 4's place
    assert torch.all(out[:128] == 4) and int(out[128]) == 1
    # the rings of the kernels in earnest work afterwards
    h = torch.randn(300, 512, device="cuda").bfloat16()
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    rstd = q.qlora_rmsnorm_fwd(h, gamma)[2]
    dx, dgamma = q.qlora_rmsnorm_bwd(h, h, gamma, rstd)
    assert torch.isfinite(dx.float()).all() and torch.isfinite(dgamma).all()
    assert q.qlora_device_status() == (0, 0)
