"""Failure handling of the bounded kernel waits, made to happen on purpose without any
fault: with a short wait limit set, the next attention launch leaves one of its loads
undone (moba_debug_fault_next_launch), so the wait for it runs out.  The launch must
end (its roles stop, drain their copies, free TMEM), moba_device_status() must report
MOBA_ERR_DEVICE, and the next normal call in the same process must give the right
answer."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from tests.parity import check_out

pytestmark = pytest.mark.gpu

MOBA_ERR_DEVICE = -7


def test_a_wait_that_runs_out_reports_an_error_and_the_context_stays_usable():
    import block_sparse_long_prefill_b200 as moba
    w = workloads.small_swa(batch=1, hq=2, hkv=2, seqlen=1024, d=64, window=256)
    q, k, v = workloads.make_inputs(w, 17)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    ref, ref_lse = moba.swa_attn_fwd(qd, kd, vd, w.window)
    torch.cuda.synchronize()
    assert moba.device_status() == 0
    try:
        moba.debug_set_wait_limit_us(2000)           # 2 ms
        moba.debug_fault_next_launch(1)
        out, lse = moba.swa_attn_fwd(qd, kd, vd, w.window)
        assert moba.device_status() == MOBA_ERR_DEVICE
    finally:
        moba.debug_fault_next_launch(0)
        moba.debug_set_wait_limit_us(0)
    assert moba.device_status() == 0                  # read and cleared
    out2, lse2 = moba.swa_attn_fwd(qd, kd, vd, w.window)
    torch.cuda.synchronize()
    assert moba.device_status() == 0
    assert torch.equal(out2, ref) and torch.equal(lse2, ref_lse)
    rows = np.arange(w.seqlen, dtype=np.int32)
    out_o, lse_o = oracle.swa(q, k, v, window=w.window, rows=rows)
    check_out(out2.float().cpu().numpy(), lse2.cpu().numpy(), out_o, lse_o)


def _bad_index(moba):
    """A rotation whose one row has no angles: MOBA_ERR_INDEX."""
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(1, 8, device="cuda")
    moba.qk_norm_rope_fwd(x, x, t, t, torch.full((1, 1), -1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("index_first", [True, False])
def test_a_wait_that_runs_out_is_not_hidden_by_a_bad_index(index_first):
    """Both errors between two reads of the status, in either order: the one that left a
    launch unfinished is reported."""
    import block_sparse_long_prefill_b200 as moba
    w = workloads.small_swa(batch=1, hq=2, hkv=2, seqlen=1024, d=64, window=256)
    q, k, v = (t.cuda() for t in workloads.make_inputs(w, 18))
    assert moba.device_status() == 0
    try:
        moba.debug_set_wait_limit_us(2000)
        if index_first:
            _bad_index(moba)
        moba.debug_fault_next_launch(1)
        moba.swa_attn_fwd(q, k, v, w.window)
        if not index_first:
            _bad_index(moba)
        assert moba.device_status() == MOBA_ERR_DEVICE
    finally:
        moba.debug_fault_next_launch(0)
        moba.debug_set_wait_limit_us(0)
    assert moba.device_status() == 0
    _bad_index(moba)
    assert moba.device_status() == -10 and moba.device_status() == 0


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("which", ["forward", "dq", "dkdv"])
def test_the_sliding_window_kernels_give_up_in_one_wait(which, d):
    """A product of the first CTA that is never announced: the launch ends after one wait limit
    (a loader that gives up between two copies must not wait for the one it has not issued),
    says so, and the next call is right to the bit."""
    import block_sparse_long_prefill_b200 as moba
    g = torch.Generator("cuda").manual_seed(d)
    q, k, v, do = (torch.randn(1, h, 2000, d, generator=g, device="cuda").bfloat16() for h in (2, 1, 1, 2))

    def fwd():
        return moba.swa_attn_fwd(q, k, v, 1500, sink=4)

    out, lse = fwd()
    call = fwd if which == "forward" else lambda: moba.swa_attn_bwd(q, k, v, out, lse, do, 1500, 4)
    want = call()
    assert moba.device_status() == 0
    limit = 0.05
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    try:
        moba.debug_set_wait_limit_us(int(limit * 1e6))
        moba.debug_fault_next_launch(2 if which == "dkdv" else 1)
        start.record()
        call()
        end.record()
        assert moba.device_status() == MOBA_ERR_DEVICE
    finally:
        moba.debug_fault_next_launch(0)
        moba.debug_set_wait_limit_us(0)
    # One limit, and the launches themselves (well below a millisecond).
    assert limit <= start.elapsed_time(end) * 1e-3 < 1.5 * limit
    assert all(torch.equal(a, b) for a, b in zip(want, call()))
    assert moba.device_status() == 0
