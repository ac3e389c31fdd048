"""What the calls around the prefill refuse, on the host and before any launch (CPU only):
the C ABI's codes, and the binding's checks of its tensors."""
import ctypes

import pytest
import torch

import block_sparse_long_prefill_b200 as moba

T, W = moba.MobaTensor, moba.MobaWeight
OK = T(1 << 20, 8 * 1024, 8 * 1024, 128)
NULL, MIS, ODD = T(None, 0, 0, 0), T((1 << 20) + 2, 8 * 1024, 8 * 1024, 128), T(1 << 20, 8 * 1024, 8 * 1024, 100)
ZERO = T(1 << 20, 8 * 1024, 8 * 1024, 0)
P, NO = 1 << 20, W(None, 0)
SHAPE, DIM, ALIGN, ARG, WORKSPACE, NODEVICE = -1, -2, -3, -4, -5, -8
NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")


def test_the_index_status_has_a_text():
    assert moba.status_string(-10) != "unknown status"


def _fwd(q=OK, out=OK, lse=P, batch=1, hq=2, hkv=1, N=100, Nk=200, d=128, window=10, sink=4):
    return moba.library().swa_sink_attn_fwd(q, OK, OK, batch, hq, hkv, N, Nk, d, window, sink, 0.0, out, lse, None)


def test_rows_beyond_32_bits_are_refused():
    size = ctypes.c_size_t(0)
    lib = moba.library()
    assert lib.qk_norm_rope_bwd_workspace_size(1 << 20, 32, 32, 1 << 20, 128, ctypes.byref(size)) == SHAPE
    assert _append(T_=1 << 30, hkv=8) == SHAPE
    assert _fwd(Nk=(1 << 31) - 1) == SHAPE


@pytest.mark.parametrize("scale", [1e-31, 1e-45])
def test_backward_of_a_vanishing_scale(scale):
    """The kernels hold lse / scale in float32."""
    args = (OK, OK, OK, OK, OK, P, 1, 2, 1, 300, 128, 10, 4)
    assert moba.library().swa_attn_bwd(*args, scale, OK, OK, OK, P, 1 << 40, None) == ARG


@pytest.mark.parametrize("kw,code", [
    (dict(sink=-1), ARG), (dict(window=0), ARG), (dict(d=96), DIM), (dict(hq=3, hkv=2), SHAPE), (dict(Nk=99), SHAPE),
    (dict(N=0), SHAPE), (dict(q=NULL), ARG), (dict(q=MIS), ALIGN), (dict(out=ODD), ALIGN), (dict(lse=None), ARG),
    (dict(lse=P + 2), ALIGN)])
def test_sink_forward(kw, code):
    assert _fwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(out=ZERO), ARG), (dict(out=T(1 << 20, 8 * 1024, 0, 128)), ARG), (dict(out=T(1 << 20, 0, 8 * 1024, 128), batch=2), ARG),
    (dict(out=ZERO, sink=0), ARG)])
def test_sink_forward_into_an_output_whose_rows_share_an_address(kw, code):
    assert _fwd(**kw) == code


@NO_GPU
def test_a_stride_of_zero_over_one_element_is_fine():
    assert _fwd(out=T(1 << 20, 0, 8 * 1024, 128)) == _fwd(out=ZERO, N=1) == NODEVICE


def _bwd(q=OK, dq=OK, dk=OK, lse=P, ws=P, nbytes=1 << 40, batch=1, hq=2, hkv=1, N=300, d=128, window=10, sink=4):
    return moba.library().swa_attn_bwd(q, OK, OK, OK, OK, lse, batch, hq, hkv, N, d, window, sink, 0.0, dq, dk, OK, ws,
                                       nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(sink=-1), ARG), (dict(window=0), ARG), (dict(d=72), DIM), (dict(hq=3, hkv=2), SHAPE), (dict(N=1 << 30), SHAPE),
    (dict(q=NULL), ARG), (dict(dq=MIS), ALIGN), (dict(dk=ZERO), ARG), (dict(lse=None), ARG), (dict(ws=None), WORKSPACE),
    (dict(nbytes=1000), WORKSPACE), (dict(ws=P + 8), ALIGN)])
def test_sliding_window_backward(kw, code):
    assert _bwd(**kw) == code


def test_backward_workspace_holds_the_statistics_and_the_parts_of_the_sinks():
    size = moba.swa_bwd_workspace_size
    band, sinks = size(1, 8, 2, 20000, 128, 256), size(1, 8, 2, 20000, 128, 256, 4)
    rows = 8 * 157 * 128
    assert band >= rows * (8 + 32) and sinks > band
    # Nothing behind the band: no parts.
    assert size(1, 8, 2, 20000, 128, 20000, 4) == band
    # Parts stay bounded where the far walks are very long, and where there are many sinks.
    assert size(1, 4, 1, 1 << 20, 128, 128, 4) < (1 << 30) and size(1, 8, 8, 65536, 128, 128, 8192) < (1 << 31)
    with pytest.raises(moba.MobaError):
        size(1, 8, 3, 100, 128, 10)


def _rope(bwd=False, q=OK, qo=OK, cos=P, sin=P, pos=None, wq=NO, wk=NO, batch=1, hq=2, hkv=3, N=10, d=128, rot=64, max_pos=10,
          inter=0, eps=1e-6, dqw=None, dkw=None, ws=P, nbytes=1 << 30):
    if bwd:
        return moba.library().qk_norm_rope_bwd(OK, OK, q, OK, cos, sin, pos, wq, wk, batch, hq, hkv, N, d, rot, max_pos,
                                               inter, eps, qo, OK, dqw, dkw, ws, nbytes, None)
    return moba.library().qk_norm_rope_fwd(q, OK, cos, sin, pos, wq, wk, batch, hq, hkv, N, d, rot, max_pos, inter, eps, qo,
                                           OK, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(rot=0), DIM), (dict(rot=24), DIM), (dict(rot=144), DIM), (dict(d=96), DIM), (dict(max_pos=9), SHAPE),
    (dict(max_pos=0, pos=P), SHAPE), (dict(cos=None), ARG), (dict(sin=P + 4), ALIGN), (dict(pos=P + 2), ALIGN),
    (dict(inter=2), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(wq=W(P + 1, 0), dqw=P), ALIGN),
    (dict(wk=W(P + 2, 1), dkw=P), ALIGN), (dict(wk=W(P, 2), dkw=P), ARG), (dict(N=0), SHAPE), (dict(qo=MIS), ALIGN),
    (dict(qo=ZERO), ARG), (dict(qo=NULL), ARG)])
def test_norm_rope(bwd, kw, code):
    if not bwd:
        kw = {k: v for k, v in kw.items() if k not in ("dqw", "dkw")}
    assert _rope(bwd, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(wq=W(P, 0)), ARG), (dict(dqw=P), ARG), (dict(wq=W(P, 0), dqw=P + 2), ALIGN),
    (dict(wq=W(P, 0), dqw=P, ws=None), WORKSPACE), (dict(wq=W(P, 0), dqw=P, nbytes=64), WORKSPACE),
    (dict(wq=W(P, 0), dqw=P, q=NULL), ARG)])
def test_norm_rope_backward_weights(kw, code):
    assert _rope(True, **kw) == code


def _append(k=OK, kp=OK, q=NULL, qo=NULL, cu=P, lens=P, table=P, cos=P, sin=P, wq=NO, wk=NO, batch=2, T_=5, hq=0, hkv=1, d=64,
            rot=64, max_pos=9, eps=1e-6, page=16, pages=4, width=2):
    return moba.library().kv_append(k, OK, q, cu, lens, table, cos, sin, wq, wk, batch, T_, hq, hkv, d, rot, max_pos, 0, eps,
                                    page, pages, width, kp, OK, qo, None)


@pytest.mark.parametrize("kw,code", [
    (dict(cu=None), SHAPE), (dict(T_=-1), SHAPE), (dict(page=0), SHAPE), (dict(pages=0), SHAPE), (dict(width=0), SHAPE),
    (dict(batch=0), SHAPE), (dict(table=None), ARG), (dict(lens=None), ARG), (dict(lens=P + 1), ALIGN), (dict(cu=P + 2), ALIGN),
    (dict(cos=None), ARG), (dict(cos=None, sin=None), ARG), (dict(cos=None, sin=None, rot=0, d=60), DIM), (dict(rot=8), DIM),
    (dict(wq=W(P, 0)), ARG), (dict(q=OK, hq=2), ARG), (dict(q=OK, qo=OK), SHAPE), (dict(k=MIS), ALIGN), (dict(kp=ODD), ALIGN),
    (dict(kp=ZERO), ARG), (dict(T_=0), 0)])
def test_append(kw, code):
    assert _append(**kw) == code


def _decode(q=OK, out=OK, kp=OK, table=P, lens=P, lse=P, ws=P, nbytes=1 << 40, batch=2, hq=4, hkv=2, d=64, page=16, pages=9,
            width=3, window=0, sink=0):
    return moba.library().paged_decode_attn(q, kp, OK, table, lens, batch, hq, hkv, d, page, pages, width, window, sink, 0.0,
                                            out, lse, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(hq=5), SHAPE), (dict(batch=0), SHAPE), (dict(d=256), DIM), (dict(window=-1), ARG), (dict(sink=-1), ARG),
    (dict(page=0), SHAPE), (dict(width=1 << 30, page=64), SHAPE), (dict(batch=1 << 20, width=1 << 16), SHAPE),
    (dict(table=None), ARG), (dict(lse=None), ARG), (dict(q=NULL), ARG), (dict(out=MIS), ALIGN), (dict(kp=ODD), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(nbytes=100), WORKSPACE), (dict(ws=P + 4), ALIGN)])
def test_decode(kw, code):
    assert _decode(**kw) == code


def test_decode_counts_its_work_and_the_run_of_the_last_block_in_32_bits():
    """The work is dealt out in runs of ceil(work / blocks): the sum of both has to fit too.
    8 sequences of 2 KV heads; an item of w pages of 16 costs up to w + 8 tiles."""
    w = (1 << 27) - 17
    assert 16 * (w + 8) + 443 >= 1 << 31            # (work + blocks - 1)
    assert _decode(batch=8, page=16, width=w) == SHAPE


@NO_GPU
def test_valid_calls_without_a_device_report_no_device():
    assert _fwd() == _bwd() == _rope() == _rope(True) == _append() == _decode() == NODEVICE


def test_workspace_sizes_are_host_only():
    out = ctypes.c_size_t(0)
    lib = moba.library()
    assert lib.paged_decode_workspace_size(4, 8, 2, 128, ctypes.byref(out)) == 0 and out.value > 0
    assert lib.paged_decode_workspace_size(4, 8, 3, 128, ctypes.byref(out)) == SHAPE
    assert lib.qk_norm_rope_bwd_workspace_size(1, 8, 2, 100, 96, ctypes.byref(out)) == DIM
    assert lib.qk_norm_rope_bwd_workspace_size(1, 8, 2, 100, 64, None) == ARG
    assert lib.swa_bwd_workspace_size(1, 8, 2, 100, 64, 0, 0, ctypes.byref(out)) == ARG


def test_the_binding_takes_cuda_tensors_only():
    x = torch.zeros(1, 2, 5, 64, dtype=torch.bfloat16)
    t = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(9, 16)
    i = torch.zeros(5, 1, dtype=torch.int32)
    for call in (lambda: moba.swa_attn_fwd(x, x, x, 3, sink=1),
                 lambda: moba.swa_attn_bwd(x, x, x, x, torch.zeros(1, 2, 5), x, 3),
                 lambda: moba.qk_norm_rope_fwd(x, x, c, c),
                 lambda: moba.qk_norm_rope_bwd(x, x, x, x, c, c),
                 lambda: moba.kv_append(t, t, x, x, i, i[:, 0]),
                 lambda: moba.paged_decode_attn(t, x, x, i, i[:, 0])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="dimensions"):
        moba.swa_attn_fwd(x[0], x, x, 3)
    with pytest.raises(ValueError, match="dimensions"):
        moba.paged_decode_attn(x, x, x, i, i[:, 0])


class _Handle:
    """A stream of some other library: its handle alone."""
    cuda_stream = 0


def test_a_stream_of_another_device_is_refused():
    """(Tensors and streams of two GPUs, described.)"""
    class Tensor:
        is_cuda, device = True, torch.device("cuda", 0)

    class Elsewhere(_Handle):
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="the stream is on cuda:1, the tensors are on cuda:0"):
        moba._own_stream("paged_decode_attn", Elsewhere(), Tensor())
    assert moba._own_stream("paged_decode_attn", None, Tensor()) is None


def test_with_a_stream_the_tensors_are_still_named():
    t = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    x = torch.zeros(1, 2, 5, 64, dtype=torch.bfloat16)
    i = torch.zeros(5, 1, dtype=torch.int32)
    for call in (lambda: moba.paged_decode_attn(t, x, x, i, i[:, 0], stream=_Handle()),
                 lambda: moba.swa_attn_fwd(x, x, x, 3, stream=_Handle())):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
