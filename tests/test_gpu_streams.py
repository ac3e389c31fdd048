"""The calls around the prefill on a stream of the caller's choice: any object with a stream
handle, as the prefill takes it, and inputs that are dropped while the call still waits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _moba():
    import block_sparse_long_prefill_b200 as moba
    return moba


def _rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").bfloat16()


def _swa_fwd():
    x = dict(q=_rand(1, 4, 700, 80), k=_rand(1, 2, 700, 80, seed=1), v=_rand(1, 2, 700, 80, seed=2))
    return x, lambda x, **kw: _moba().swa_attn_fwd(x["q"], x["k"], x["v"], 100, sink=5, **kw)


def _swa_bwd():
    x, fwd = _swa_fwd()
    x["out"], x["lse"] = fwd(x)
    x["dout"] = _rand(1, 4, 700, 80, seed=3)
    names = ("q", "k", "v", "out", "lse", "dout")
    return x, lambda x, **kw: _moba().swa_attn_bwd(*(x[n] for n in names), 100, 5, **kw)


def _rope_inputs():
    a = torch.arange(300, device="cuda")[:, None] / 10.0 ** torch.arange(32, device="cuda")
    return dict(q=_rand(1, 8, 300, 128), k=_rand(1, 2, 300, 128, seed=1), cos=a.cos(), sin=a.sin(),
                pos=torch.arange(300, dtype=torch.int32, device="cuda")[None].contiguous(),
                wq=1 + 0.1 * _rand(128, seed=2).float(), wk=_rand(128, seed=3) + 1)


def _rope_fwd():
    names = ("q", "k", "cos", "sin", "pos", "wq", "wk")
    return _rope_inputs(), lambda x, **kw: _moba().qk_norm_rope_fwd(*(x[n] for n in names), **kw)


def _rope_bwd():
    x = _rope_inputs()
    x["dq"], x["dk"] = _rand(1, 8, 300, 128, seed=4), _rand(1, 2, 300, 128, seed=5)
    names = ("dq", "dk", "q", "k", "cos", "sin", "pos", "wq", "wk")
    return x, lambda x, **kw: _moba().qk_norm_rope_bwd(*(x[n] for n in names), **kw)


def _cache():
    return dict(kp=_rand(40, 2, 16, 64), vp=_rand(40, 2, 16, 64, seed=1),
                table=torch.randperm(40, generator=torch.Generator().manual_seed(2)).int().view(4, 10).cuda(),
                lens=torch.tensor([160, 3, 77, 100], dtype=torch.int32, device="cuda"))


def _append():
    x = _cache()
    r = _rope_inputs()
    x.update(k=_rand(9, 2, 64, seed=3), v=_rand(9, 2, 64, seed=4), q=_rand(9, 6, 64, seed=5),
             cu=torch.tensor([0, 4, 5, 5, 9], dtype=torch.int32, device="cuda"), cos=r["cos"], sin=r["sin"])

    def call(x, **kw):
        kp, vp = x["kp"].clone(), x["vp"].clone()    # (the caches are written)
        if "stream" in kw:
            torch.cuda.current_stream().synchronize()
        q = _moba().kv_append(x["k"], x["v"], kp, vp, x["table"], x["lens"], x["cu"], x["cos"], x["sin"], q=x["q"], **kw)
        return q, kp, vp
    return x, call


def _decode():
    x = dict(_cache(), q=_rand(4, 8, 64, seed=6))
    names = ("q", "kp", "vp", "table", "lens")
    return x, lambda x, **kw: _moba().paged_decode_attn(*(x[n] for n in names), 50, 4, **kw)


CALLS = dict(swa_fwd=_swa_fwd, swa_bwd=_swa_bwd, rope_fwd=_rope_fwd, rope_bwd=_rope_bwd, append=_append, decode=_decode)


@pytest.mark.parametrize("name", CALLS)
def test_any_object_with_a_stream_handle(name):
    x, call = CALLS[name]()
    want = call(x)
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    side.wait_stream(torch.cuda.current_stream())
    got = call(x, stream=Handle())
    side.synchronize()
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(want, got))
    assert _moba().device_status() == 0


@pytest.mark.parametrize("name", CALLS)
def test_inputs_stay_until_they_are_read(name):
    """The call's stream is busy; its inputs are dropped and the caller goes on allocating: the
    memory must not be handed out again before the call has read it."""
    x, call = CALLS[name]()
    want = call(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    copies = {n: t.clone() for n, t in x.items()}
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = call(copies, stream=side)
    copies.clear()
    junk = [torch.full_like(t, 1) for t in x.values() for _ in range(3)]
    torch.cuda.synchronize()
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(want, got))
    assert _moba().device_status() == 0 and junk


def test_given_results_stay_until_they_are_written():
    """An output of the caller's that is dropped before the call writes it: what is allocated
    meanwhile must not be written over."""
    moba = _moba()
    x = _swa_fwd()[0]
    side = torch.cuda.Stream()
    out = torch.empty_like(x["q"])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    moba.swa_attn_fwd(x["q"], x["k"], x["v"], 100, sink=5, out=out, stream=side)
    del out
    junk = [torch.full_like(x["q"], 9) for _ in range(3)]
    torch.cuda.synchronize()
    assert all((t == 9).all() for t in junk)


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_library_may_go_before_the_tensors(name):
    """Its handle is invalid by the time the inputs and results are freed: nothing of torch's may
    still refer to it."""
    import ctypes
    x, call = CALLS[name]()
    want = call(x)
    torch.cuda.synchronize()
    rt, handle = torch.cuda.cudart(), ctypes.c_void_p()
    assert int(rt.cudaStreamCreate(ctypes.addressof(handle))) == 0

    class Theirs:
        cuda_stream = handle.value

    copies = {n: t.clone() for n, t in x.items()}
    torch.cuda.synchronize()
    got = call(copies, stream=Theirs())
    torch.cuda.synchronize()
    assert int(rt.cudaStreamDestroy(handle.value)) == 0
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(want, got))
    copies.clear()
    del got
    torch.cuda.synchronize()
    again = [t.clone() for t in x.values()]
    assert _moba().device_status() == 0 and again


def test_the_default_stream_by_its_handle():
    """Handle 0, from within another stream."""
    x, call = CALLS["decode"]()
    want = call(x)

    class Default:
        cuda_stream = 0

    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(x, stream=Default())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("name", [n for n in CALLS if n != "append"])   # (its helper waits on the host)
def test_on_a_forked_stream_in_a_graph(name):
    """Captured on a stream of its own, with inputs made and dropped within the capture."""
    x, call = CALLS[name]()
    want = call(x)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        copies = {n: t.clone() for n, t in x.items()}
        side.wait_stream(torch.cuda.current_stream())
        got = call(copies, stream=side)
        copies.clear()
        junk = [torch.full_like(t, 1) for t in x.values() for _ in range(2)]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            if t is not None:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(want, got))
    del got, junk
    torch.cuda.synchronize()
    again = [t.clone() for t in x.values()]
    assert _moba().device_status() == 0 and again
