"""Host-side validation of the row movement's C entry points (no GPU: only
calls that return before any CUDA work)."""

import ctypes

import pytest

import sparse_top_mixture_b200 as stm


def _p(**kw):
    base = dict(T=64, H=256, E=8, k=2, I=128, dtype="bf16")
    base.update(kw)
    return ctypes.byref(stm.Problem(**base).c())


A = 16  # an aligned, never followed address


def test_permute_rows_validates():
    L = stm.lib()
    assert L.moe_permute_rows(None, A, A, A, A, None) == 1
    for args in ((None, A, A, A), (A, None, A, A), (A, A, None, A), (A, A, A, None), (8, A, A, A), (A, A, A, 24)):
        assert L.moe_permute_rows(_p(), *args, None) == 1
    assert L.moe_permute_rows(_p(k=9), A, A, A, A, None) == 1
    assert L.moe_permute_rows(_p(H=12), A, A, A, A, None) == 1
    assert L.moe_permute_rows(_p(T=0), None, None, None, None, None) == 0
    assert L.moe_permute_rows_backward(None, A, A, A, None) == 1
    assert L.moe_permute_rows_backward(_p(), A, A, 8, None) == 1
    assert L.moe_permute_rows_backward(_p(T=0), None, None, None, None) == 0


@pytest.mark.parametrize("dtype,y_dtype,ok", [("bf16", 0, True), ("bf16", 1, True), ("f32", 0, True),
                                              ("f32", 1, False), ("bf16", 2, False), ("bf16", -1, False)])
def test_row_types(dtype, y_dtype, ok):
    L = stm.lib()
    want = 0 if ok else 1
    assert L.moe_unpermute_rows(_p(T=0, dtype=dtype), y_dtype, None, None, None, None, None, None) == want
    assert L.moe_unpermute_rows_backward(_p(T=0, dtype=dtype), y_dtype, None, None, None, None, None, None, None,
                                         None) == want


def test_unpermute_rows_validates():
    L = stm.lib()
    for args in ((None, A, A, A, A), (A, None, A, A, A), (A, A, A, A, None), (A, A, 8, A, A), (A, A, A, 8, A)):
        assert L.moe_unpermute_rows(_p(), 1, *args, None) == 1


def test_unpermute_rows_backward_validates():
    L = stm.lib()
    # dout, y_perm, pair_pos, offsets, routing_weights, dy_perm, d_routing_weights
    bad = [(None, A, A, A, A, A, A), (A, A, None, A, A, A, A), (A, A, A, A, 8, A, A), (A, A, A, A, A, 8, A),
           (A, A, A, A, A, A, 8), (A, A, A, A, A, None, None),  # nothing asked for
           (A, None, A, A, A, A, A),   # the weights' gradient needs the rows
           (A, A, A, None, A, A, A)]   # the rows' gradient needs the offsets
    for args in bad:
        assert L.moe_unpermute_rows_backward(_p(), 1, *args, None) == 1


@pytest.mark.parametrize("current", [0, 1])
def test_a_launch_has_its_device_current_and_its_stream(monkeypatch, current):
    """For tensors on another device than the current one (no GPU: the calls that would ask for one are stood in for)."""
    import contextlib

    import torch

    state = {"device": current}

    @contextlib.contextmanager
    def device(d):
        before, state["device"] = state["device"], d.index
        yield
        state["device"] = before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    seen = []

    def call(a, b, stream):
        seen.append((a, b, stream, state["device"]))
        return 0

    stm._launch(call, torch.device("cuda", 1), 5, None)
    assert seen == [(5, None, 101, 1)] and state["device"] == current
    with pytest.raises(stm.MoeError):
        stm._launch(lambda *a: 1, torch.device("cuda", 0))


def test_a_stream_of_a_cpu_tensor_is_refused():
    """Calls that check nothing else of a workspace must not hand a host address to the library."""
    import torch

    ws = torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: stm._stream(ws.device), lambda: stm.read_device_error(ws),
                 lambda: stm.selftest_wait_timeout(ws), lambda: stm.new_workspace(stm.Problem(4, 32, 4, 2, 32), "cpu")):
        with pytest.raises(ValueError):
            call()


def test_a_problem_keeps_its_fields_only():
    """The C struct that the calls keep with a problem shows neither in vars() nor in copies."""
    import copy
    import dataclasses
    import json
    import pickle
    import weakref

    p = stm.Problem(T=64, H=256, E=8, k=2, I=128, shared="plain", I_shared=64)
    fields = dict(vars(p))
    assert bytes(p._struct()) == bytes(p.c()) and p._struct() is p._struct()
    assert vars(p) == fields and list(fields) == [f.name for f in dataclasses.fields(p)]
    assert stm.Problem(**vars(p)) == p and json.loads(json.dumps(vars(p))) == fields
    for q in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p)), dataclasses.replace(p)):
        assert q == p and hash(q) == hash(p) and vars(q) == fields and bytes(q._struct()) == bytes(p.c())
    q = dataclasses.replace(p, T=3)
    assert q._struct().T == 3 and p._struct().T == 64 and weakref.ref(p)() is p
