"""Host-side checks of the norm and clip entry points (no GPU work is
launched): workspace sizes, and every refusal before anything is enqueued.
Pointers are never dereferenced: each call fails validation first."""
import ctypes

import pytest

import bucketed_gradient_all_ddp_amd as ddp
from bucketed_gradient_all_ddp_amd.binding import load_library

FAKE = ctypes.c_void_p(0x100000000)
OUT = ctypes.c_void_p(0x200000000)
WS = ctypes.c_void_p(0x300000000)
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def _uploaded_empty(p=4, eb=4):
    """A plan of zero-size parameters: its empty descriptor table uploads
    without device memory."""
    plan = ddp.ddp_bucket_plan([0, 0, 0], eb, 64, 16)
    assert load_library().ddp_plan_upload_segments(plan.handle, p, None, 0, None) == 0
    return plan


def test_workspace_sizes():
    # fp32: tiles of 256 elements; groups of 16 tiles; a slot per group and
    # per parameter with elements, 8 bytes each
    sizes = [5000, 0, 7, 4096, 4097, 1, 33_333, 12, 0, 65_545]
    for eb, tile in ((4, 256), (2, 512)):
        plan = ddp.ddp_bucket_plan(sizes, eb, 96 * 1024, 8 * 1024)
        tiles = sum(-(-s // tile) for s in sizes)
        live = sum(1 for s in sizes if s)
        for p in (1, 3, 64):
            assert plan.grad_norm_workspace(p) == 8 * p * (-(-tiles // 16) + live)
        assert plan.grad_norm_workspace(0) == 0 and plan.grad_norm_workspace(65) == 0
        assert plan.sync_norm_workspace() == 8 * max(tiles, -(-tiles // 16) + live)
    # past 32768 tiles: a second level of sums per 256 tiles and parameter
    assert ddp.ddp_bucket_plan([32768 * 256, 0], 4).sync_norm_workspace() == 8 * 32768
    big = ddp.ddp_bucket_plan([32768 * 256, 0, 1], 4)
    assert big.sync_norm_workspace() == 8 * (32769 + 129 + 2)
    L = load_library()
    assert L.ddp_grad_norm_workspace(None, 4) == 0 and L.ddp_sync_norm_workspace(None) == 0
    empty = ddp.ddp_bucket_plan([], 4)
    assert empty.grad_norm_workspace(8) == 0 and empty.sync_norm_workspace() == 0


def test_grad_norm_argument_errors():
    L = load_library()
    f = L.ddp_grad_norm
    plan = ddp.ddp_bucket_plan([100, 200], 4, 1024, 256)
    assert f(None, 4, FAKE, 0, 0, OUT, None, WS, BIG, None) == 1
    assert f(plan.handle, 0, FAKE, 0, 0, OUT, None, WS, BIG, None) == 2
    assert f(plan.handle, 65, FAKE, 0, 0, OUT, None, WS, BIG, None) == 2
    assert f(plan.handle, 4, FAKE, 7, 0, OUT, None, WS, BIG, None) == 1
    assert f(plan.handle, 4, FAKE, 1, 0, OUT, None, WS, BIG, None) == 1   # bf16, fp32 plan
    assert b"2-byte" in L.ddp_last_error()
    assert f(plan.handle, 4, FAKE, 0, 0, OUT, None, WS, BIG, None) == 6   # not uploaded
    assert b"upload_segments" in L.ddp_last_error()
    ready = _uploaded_empty()
    assert f(ready.handle, 4, None, 0, 3, OUT, None, None, 0, None) == 1  # norm type
    assert f(ready.handle, 4, None, 0, -1, OUT, None, None, 0, None) == 1
    assert f(ready.handle, 4, None, 0, 0, None, None, None, 0, None) == 1  # no output
    odd = ctypes.c_void_p(OUT.value + 2)
    assert f(ready.handle, 4, None, 0, 0, odd, None, None, 0, None) == 3
    assert f(ready.handle, 4, None, 0, 0, OUT, odd, None, 0, None) == 3


def test_clip_argument_errors():
    L = load_library()
    f = L.ddp_clip_grads
    plan = ddp.ddp_bucket_plan([100, 200], 4, 1024, 256)
    assert f(None, 4, FAKE, 0, OUT, 1, 1.0, 1e-6, 0, None) == 1
    assert f(plan.handle, 65, FAKE, 0, OUT, 1, 1.0, 1e-6, 0, None) == 2
    assert f(plan.handle, 4, FAKE, 0, OUT, 1, 1.0, 1e-6, 0, None) == 6
    ready = _uploaded_empty()
    ok = (ready.handle, 4, FAKE, 0, OUT, 1, 1.0, 1e-6, 0, None)
    assert f(*ok) == 0  # nothing to clip: nothing launched
    for bad in (-1.0, NAN, -INF):
        assert f(ready.handle, 4, FAKE, 0, OUT, 1, bad, 1e-6, 0, None) == 1
        assert b"max_norm" in L.ddp_last_error()
    for bad in (-1e-9, NAN, INF):
        assert f(ready.handle, 4, FAKE, 0, OUT, 1, 1.0, bad, 0, None) == 1
        assert b"eps" in L.ddp_last_error()
    assert f(ready.handle, 4, FAKE, 0, OUT, 1, INF, 0.0, 0, None) == 0
    assert f(ready.handle, 4, FAKE, 0, None, 1, 1.0, 1e-6, 0, None) == 1
    assert f(ready.handle, 4, FAKE, 0, OUT, 4, 1.0, 1e-6, 0, None) == 0
    for n in (0, 2, 3, 5, -1):
        assert f(ready.handle, 4, FAKE, 0, OUT, n, 1.0, 1e-6, 0, None) == 1
    assert f(ready.handle, 4, FAKE, 0, OUT, 4, 1.0, 1e-6, 1, None) == 1  # replicated: one norm
    assert f(ready.handle, 4, FAKE, 0, OUT, 1, 1.0, 1e-6, 2, None) == 1


def test_sync_norm_argument_errors():
    L = load_library()
    plan = ddp.ddp_bucket_plan([100, 200], 4, 1024, 256)
    need = plan.sync_norm_workspace()
    f = L.ddp_allreduce_buckets_norm
    assert f(None, 0, 1, 4, FAKE, 0, 0, None, 0, WS, BIG, None, None) == 1
    assert f(plan.handle, 0, 1, 4, FAKE, 0, 0, None, 5, WS, BIG, None, None) == 1
    assert f(plan.handle, 0, 1, 4, FAKE, 0, 0, None, 0, None, 0, None, None) == 7
    assert f(plan.handle, 0, 1, 4, FAKE, 0, 0, None, 0, WS, need - 1, None, None) == 7
    odd = ctypes.c_void_p(WS.value + 8)
    assert f(plan.handle, 0, 1, 4, FAKE, 0, 0, None, 0, odd, BIG, None, None) == 3
    assert f(plan.handle, 0, 1, 4, FAKE, 0, 0, None, 0, WS, need, None, None) == 6
    assert f(plan.handle, 9, 1, 4, FAKE, 0, 0, None, 0, WS, need, None, None) == 2
    g = L.ddp_grad_norm_finish
    assert g(None, 0, OUT, None, WS, BIG, None) == 1
    assert g(plan.handle, 0, OUT, None, WS, BIG, None) == 6
    ready = _uploaded_empty()
    assert g(ready.handle, 3, OUT, None, None, 0, None) == 1
    assert g(ready.handle, 0, None, None, None, 0, None) == 1
    h = L.ddp_allreduce_clip
    assert h(None, 4, FAKE, 0, 0, None, 0, 1.0, 1e-6, OUT, None, WS, BIG, None, None) == 1
    assert h(plan.handle, 4, FAKE, 0, 0, None, 0, 1.0, 1e-6, OUT, None, WS, BIG, None, None) == 6
    # the fold needs the table for this p
    assert h(ready.handle, 3, FAKE, 0, 0, None, 0, 1.0, 1e-6, OUT, None, WS, BIG, None, None) == 6
    assert h(ready.handle, 4, FAKE, 0, 9, None, 0, 1.0, 1e-6, OUT, None, WS, BIG, None, None) == 1
    assert h(ready.handle, 4, FAKE, 0, 2, None, 0, 1.0, 1e-6, OUT, None, WS, BIG, None, None) == 1
    assert h(ready.handle, 4, FAKE, 0, 0, None, 9, 1.0, 1e-6, OUT, None, WS, BIG, None, None) == 1
    assert h(ready.handle, 4, FAKE, 0, 0, None, 0, -1.0, 1e-6, OUT, None, WS, BIG, None, None) == 1
    assert h(ready.handle, 4, FAKE, 0, 0, None, 0, 1.0, NAN, OUT, None, WS, BIG, None, None) == 1
    assert h(ready.handle, 4, FAKE, 0, 0, None, 0, 1.0, 1e-6, None, None, WS, BIG, None, None) == 1


def test_reducer_set_norm_errors():
    L = load_library()
    plan = _uploaded_empty()
    out = ctypes.c_void_p()
    assert L.ddp_reducer_create(plan.handle, 4, FAKE, 0, 1, None, None, ctypes.byref(out)) == 0
    try:
        assert L.ddp_reducer_set_norm(None, 0, WS, BIG) == 1
        assert L.ddp_reducer_set_norm(out, 4, WS, BIG) == 1
        assert L.ddp_reducer_set_norm(out, 0, None, 0) == 0
        assert L.ddp_reducer_set_norm(out, 2, WS, BIG) == 0
        assert L.ddp_reducer_prepare(out) == 0
        assert L.ddp_reducer_set_norm(out, 0, WS, BIG) == 1  # during a pass
        assert b"in progress" in L.ddp_last_error()
    finally:
        L.ddp_reducer_free(out)


def _table(p, numels, eb, dtypes=None):
    import torch

    t = torch.zeros(p * len(numels), dtype=torch.int64)
    t._ddp_ranks, t._ddp_numel, t._ddp_elem_bytes = p, tuple(numels), eb
    t._ddp_dtypes = frozenset(dtypes or [torch.float32 if eb == 4 else torch.bfloat16])
    return t


def test_binding_refusals():
    """What the binding refuses before the library sees the call."""
    import torch

    from bucketed_gradient_all_ddp_amd.binding import _check_norm_dtype, _floats, _workspace

    plan = ddp.ddp_bucket_plan([10, 20, 30], 4, 1024, 256)
    sizes = [10, 20, 30]
    with pytest.raises(ValueError, match="ranks"):
        ddp.ddp_grad_norm(plan, _table(2, sizes, 4), 3)
    with pytest.raises(TypeError, match="device"):
        ddp.ddp_grad_norm(plan, _table(2, sizes, 4), 2)
    with pytest.raises(ValueError, match="ranks"):
        ddp.ddp_clip_grads(plan, _table(2, sizes, 4), 3, torch.ones(1), 1.0)
    with pytest.raises(ValueError, match="ranks"):
        ddp.ddp_allreduce_clip(plan, _table(2, sizes, 4), 3, 1.0, torch.ones(1), torch.ones(4))
    # values are read: integers and half precision are refused, and mixtures
    for bad in ([torch.int32], [torch.float32, torch.int32]):
        with pytest.raises(TypeError, match="bfloat16"):
            _check_norm_dtype(_table(2, sizes, 4, bad), "t")
    for bad in ([torch.float16], [torch.bfloat16, torch.float16]):
        with pytest.raises(TypeError, match="bfloat16"):
            _check_norm_dtype(_table(2, sizes, 2, bad), "t")
    _check_norm_dtype(_table(2, sizes, 4), "t")
    _check_norm_dtype(_table(2, sizes, 2), "t")
    with pytest.raises(ValueError, match="float32"):
        _floats(torch.ones(2, dtype=torch.float64), 2, None, "t", "norms")
    with pytest.raises(ValueError, match="3 elements"):
        _floats(torch.ones(2), 3, None, "t", "norms")
    with pytest.raises(ValueError, match="contiguous"):
        _floats(torch.ones(4)[::2], 2, None, "t", "norms")
    with pytest.raises(TypeError, match="device"):
        _floats(torch.ones(2), 2, None, "t", "norms")
    with pytest.raises(TypeError, match="device"):
        _workspace(torch.ones(2), None, "t")
    with pytest.raises(ValueError, match="contiguous"):
        _workspace(torch.ones(4)[::2], None, "t")
