"""GPU: the gradient norm over many tensors, clipping by it, and both fused
into the bucket all-reduce, against plain numpy in 64 bits.

Norms: the kernels add in 64 bits and round to fp32 once. A sum of N terms in
64 bits is off by at most N 2^-53 of itself (here N < 2^24: 2^-29), its root
by half of that, and the rounding by 2^-24, so NORM_TOL = 2^-24 + 2^-29 bounds
the relative error. Clipped values are compared bit for bit: one fp32 division
for the coefficient, one fp32 product, one rounding to bf16."""
import numpy as np
import pytest
import torch

import bucketed_gradient_all_ddp_amd as ddp
from bucketed_gradient_all_ddp_amd import workloads as W
from helpers import assert_bits_equal, to_dev, to_host, tokens_for

pytestmark = pytest.mark.gpu

NORM_TOL = 2.0 ** -24 + 2.0 ** -29
# tiles are 256 (fp32) or 512 (bf16) elements, groups 16 tiles: parameters
# that end with a tile, with a group, one element around either, many in one
# group, none at all
SIZES = [5000, 0, 7, 4096, 4097, 1, 33_333, 12, 0, 65_536 + 9, 3, 100_000, 8192, 256, 255, 257,
         16 * 512, 3840, 4352] + [2, 5, 1, 0, 9] * 9 + [512, 12_288]
SHAPES = {
    "many": SIZES,
    "one": [1],
    "tiny": [3, 1, 2],
    "none": [0, 0],
    "holes": [0, 5, 0, 300, 0, 0, 1000],
    "group": [4096],
    "groups": [4096, 4096, 8192, 1],
    "small": [1] * 70 + [17] * 50,
}


class Set:
    """p ranks' gradients as views of one arena per rank, 7.0 between them."""

    def __init__(self, p, sizes, bf16, layout, oracle, seed=0, sigma=1.0):
        self.p, self.sizes, self.bf16 = p, sizes, bf16
        self.host = [[W.normal_np(n, sigma, seed, r, stream=i) for i, n in enumerate(sizes)]
                     for r in range(p)]
        if bf16:
            self.host = [[oracle.f32_to_bf16(g) for g in rank] for rank in self.host]
        dt = torch.bfloat16 if bf16 else torch.float32
        self.arenas, self.grads, self.gaps = [], [], []
        for r in range(p):
            arena = torch.full((sum(sizes) + 9 * len(sizes) + 16,), 7.0, dtype=dt, device="cuda")
            gap = np.ones(arena.numel(), dtype=bool)
            off = {"aligned": 0, "odd": 1, "mixed": r % 3 + 1}[layout]
            views = []
            for i, n in enumerate(sizes):
                if layout == "aligned":
                    off = (off + 7) // 8 * 8
                arena[off:off + n] = to_dev(self.host[r][i])
                gap[off:off + n] = False
                views.append(arena[off:off + n])
                off += n + (0 if layout == "aligned" else 1)
            self.arenas.append(arena)
            self.grads.append(views)
            self.gaps.append(gap)
        self.table = ddp.grad_pointer_table(self.grads)

    def values(self, r, i):
        """fp32 values of rank r's gradient i before any call."""
        return _wide(self.host[r][i])

    def check_gaps(self):
        for arena, gap in zip(self.arenas, self.gaps):
            assert (_wide(to_host(arena))[gap] == 7.0).all(), "a value between the gradients changed"


def _wide(a):
    """numpy fp32, or bf16 bits, as fp32 values."""
    if a.dtype == np.uint16:
        return (a.astype(np.uint32) << 16).view(np.float32)
    return a


def _narrow(a, bf16, oracle):
    return oracle.f32_to_bf16(a) if bf16 else a


def _plan(sizes, bf16, p, cap=96 * 1024, first=8 * 1024):
    return ddp.ddp_bucket_plan(sizes, 2 if bf16 else 4, cap, first).upload_segments(p)


def _norm64(parts, kind):
    """The norm of a list of fp32 arrays, in 64 bits."""
    x = np.concatenate([np.asarray(v, np.float64).reshape(-1) for v in parts] or [np.zeros(0)])
    if x.size == 0:
        return 0.0
    if kind == "inf":
        return float(np.abs(x).max())
    return float(np.sqrt((x * x).sum())) if kind == "l2" else float(np.abs(x).sum())


def _close(got, want, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    off = np.abs(got - want)
    assert (off <= NORM_TOL * want).all(), (what, got, want, off)


def _coefficient(norm, max_norm, eps):
    """min(1, max_norm / (norm + eps)) in fp32, as the header defines it."""
    norm, max_norm, eps = np.float32(norm), np.float32(max_norm), np.float32(eps)
    if norm == 0 or np.isinf(max_norm):
        return np.float32(1)
    with np.errstate(all="ignore"):
        c = max_norm / (norm + eps)
    return np.float32(1) if c >= 1 else c


def _workspace(nbytes):
    """A workspace of nbytes, all NaN, with a guard behind it."""
    t = torch.full((nbytes + 64,), 255, dtype=torch.uint8, device="cuda")
    return t[:nbytes], t[nbytes:]


def _averages(s, plan_sizes, oracle, avg, tokens, bf16, cap=96 * 1024, first=8 * 1024):
    """The fp32 averages (bf16 inputs widened, not rounded back) of every
    parameter, folded in ring order by the oracle."""
    oplan = oracle.bucket_plan(plan_sizes, 2 if bf16 else 4, cap, first)
    wide = [[s.values(r, i).copy() for i in range(len(plan_sizes))] for r in range(s.p)]
    for b in range(oplan.num_buckets):
        flats = [oracle.flatten(wide[r], oplan, b) for r in range(s.p)]
        red, _ = oracle.ring_allreduce(flats, avg=avg, tokens=tokens, want_log=False)
        oracle.unflatten(red[0], oplan, b, wide[0])
    return wide[0]


# ---------------------------------------------------------------------------
# The norm by itself
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["aligned", "odd", "mixed"])
@pytest.mark.parametrize("kind", ["l2", "l1", "inf"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_norm_of_each_rank_and_parameter(oracle, shape, bf16, kind, layout):
    p, sizes = 3, SHAPES[shape]
    s = Set(p, sizes, bf16, layout, oracle, seed=31)
    plan = _plan(sizes, bf16, p)
    ws, guard = _workspace(plan.grad_norm_workspace(p))
    each = torch.full((p, len(sizes)), -1.0, device="cuda")
    norms = ddp.ddp_grad_norm(plan, s.table, p, norm_type=kind, param_norms=each, workspace=ws)
    only = ddp.ddp_grad_norm(plan, s.table, p, norm_type=kind)
    torch.cuda.synchronize()
    assert (guard == 255).all()
    assert_bits_equal(to_host(only), to_host(norms))
    for r in range(p):
        vals = [s.values(r, i) for i in range(len(sizes))]
        _close(to_host(norms)[r], _norm64(vals, kind), f"rank {r}")
        _close(to_host(each)[r], [_norm64([v], kind) for v in vals], f"rank {r}")
        for i in range(len(sizes)):
            assert_bits_equal(to_host(s.grads[r][i]), s.host[r][i])
    # a rank by itself, with a table uploaded for another rank count
    one = ddp.ddp_grad_norm(plan, s.table, p, norm_type=kind, ranks=(2, 1))
    assert_bits_equal(to_host(one), to_host(norms)[2:])


@pytest.mark.parametrize("p", [1, 2, 13, 64])
def test_norm_rank_counts(oracle, p):
    sizes = [700, 33, 5000, 1]
    s = Set(p, sizes, False, "odd", oracle, seed=32)
    plan = _plan(sizes, False, p)
    got = to_host(ddp.ddp_grad_norm(plan, s.table, p))
    _close(got, [_norm64([s.values(r, i) for i in range(4)], "l2") for r in range(p)])


@pytest.mark.parametrize("kind", ["l2", "l1", "inf"])
@pytest.mark.parametrize("scale", [1e-30, 2.0 ** -149, 1e30, 3e38])
def test_norm_neither_overflows_nor_vanishes(kind, scale):
    """Squares of these leave fp32's range; the norm does not (but for the
    last scale, whose L2 and L1 norms are beyond fp32: infinite)."""
    n = 1000
    x = torch.full((n,), scale, device="cuda")
    x[::2] *= -1
    plan = _plan([n], False, 1)
    got = to_host(ddp.ddp_grad_norm(plan, ddp.grad_pointer_table([[x]]), 1, norm_type=kind))[0]
    want = _norm64([to_host(x)], kind)
    if want > float(np.finfo(np.float32).max):
        assert np.isinf(got)
    else:
        # below the smallest normal the rounding is to a multiple of 2^-149
        assert abs(float(got) - want) <= max(NORM_TOL * want, 2.0 ** -150)


@pytest.mark.parametrize("kind", ["l2", "l1", "inf"])
@pytest.mark.parametrize("at", [0, 1, 4999, 5000 + 17])
def test_norm_of_infinities_and_nan(oracle, kind, at):
    sizes = [5000, 18]
    for bad, check in ((np.inf, np.isinf), (-np.inf, np.isinf), (np.nan, np.isnan)):
        s = Set(2, sizes, False, "odd", oracle, seed=33)
        i, j = (0, at) if at < 5000 else (1, at - 5000)
        s.grads[1][i][j] = float(bad)
        plan = _plan(sizes, False, 2)
        each = torch.zeros(2, 2, device="cuda")
        got = to_host(ddp.ddp_grad_norm(plan, s.table, 2, norm_type=kind, param_norms=each))
        assert np.isfinite(got[0]) and check(got[1])
        e = to_host(each)
        assert check(e[1, i]) and np.isfinite(e[1, 1 - i]) and np.isfinite(e[0]).all()
        s.grads[1][1 - i][0] = float("inf")
        s.grads[1][i][j] = float("nan")
        assert np.isnan(to_host(ddp.ddp_grad_norm(plan, s.table, 2, norm_type=kind))[1])


def test_norm_is_the_same_bits_every_time(oracle):
    sizes = [300_000, 17, 40_001]
    s = Set(2, sizes, False, "odd", oracle, seed=34)
    plan = _plan(sizes, False, 2)
    runs = [to_host(ddp.ddp_grad_norm(plan, s.table, 2, norm_type="l1")) for _ in range(5)]
    for r in runs[1:]:
        assert_bits_equal(r, runs[0])


def test_offsets_past_32_bits(oracle):
    """One bf16 gradient of 2^31 + 2^20 + 3 elements, zero but for a few: the
    last one decides the norm and is clipped."""
    n = 2 ** 31 + 2 ** 20 + 3
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    spots = [0, 2 ** 31 - 1, 2 ** 31 + 5, n - 1]
    for k in spots:
        x[k] = 3.0
    plan = ddp.ddp_bucket_plan([n], 2).upload_segments(1)
    table = ddp.grad_pointer_table([[x]])
    norm = ddp.ddp_grad_norm(plan, table, 1)
    assert float(norm) == 6.0  # 4 squares of 9
    for replicated in (False, True):
        ddp.ddp_clip_grads(plan, table, 1, norm, 3.0, eps=0.0, replicated=replicated)
    assert [float(x[k]) for k in spots] == [0.75] * 4
    assert int((x != 0).sum()) == 4
    ws = torch.empty(plan.sync_norm_workspace(), dtype=torch.uint8, device="cuda")
    ddp.ddp_allreduce_clip(plan, table, 1, 0.75, norm, ws, eps=0.0)
    assert float(norm) == 1.5 and [float(x[k]) for k in spots] == [0.375] * 4


# ---------------------------------------------------------------------------
# Clipping
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["aligned", "odd", "mixed"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("p", [1, 3, 8])
@pytest.mark.parametrize("form", ["each", "shared", "replicated"])
def test_clip_bits(oracle, form, p, bf16, layout):
    s = Set(p, SIZES, bf16, layout, oracle, seed=41)
    plan = _plan(SIZES, bf16, p)
    if form == "replicated":  # the other ranks' contents are overwritten
        s.host = [s.host[0]] * p
    norms = np.array([2.5 + r if r != 1 else 0.5 for r in range(p)], np.float32)
    if form != "each":
        norms = norms[:1]
    ddp.ddp_clip_grads(plan, s.table, p, to_dev(norms), 1.75, replicated=form == "replicated")
    for r in range(p):
        c = _coefficient(norms[r if form == "each" else 0], 1.75, 1e-6)
        for i in range(len(SIZES)):
            want = s.values(r, i) * c
            assert_bits_equal(to_host(s.grads[r][i]), _narrow(want, bf16, oracle), f"{r} {i}")
    s.check_gaps()


@pytest.mark.parametrize("replicated", [False, True])
@pytest.mark.parametrize("norm,max_norm,eps", [
    (0.0, 1.0, 0.0), (0.0, 0.0, 0.0), (1.0, 1.0, 0.0), (1.0, 1.0, 1e-6), (3.0, 0.0, 1e-6),
    (np.inf, 1.0, 1e-6), (np.nan, 1.0, 1e-6), (np.inf, np.inf, 1e-6), (np.nan, np.inf, 1e-6),
    (2.0 ** -149, 1.0, 0.0), (3e38, 1e-3, 0.0)])
def test_clip_edges(oracle, norm, max_norm, eps, replicated):
    sizes = [1000, 3, 257]
    s = Set(2, sizes, False, "odd", oracle, seed=42)
    if replicated:
        for a, b in zip(s.grads[1], s.grads[0]):
            a.copy_(b)
        s.host = [s.host[0]] * 2
    plan = _plan(sizes, False, 2)
    ddp.ddp_clip_grads(plan, s.table, 2, torch.tensor([norm], device="cuda"), max_norm, eps,
                       replicated=replicated)
    c = _coefficient(norm, max_norm, eps)
    for r in range(2):
        for i in range(3):
            got, want = to_host(s.grads[r][i]), s.values(r, i) * c
            if np.isnan(c):
                assert np.isnan(got).all()
            else:
                assert_bits_equal(got, want)
    s.check_gaps()


def test_clip_of_infinite_gradients(oracle):
    """An infinite norm makes the coefficient 0: finite gradients become 0,
    the infinite one NaN, as the formula says."""
    s = Set(1, [600], False, "aligned", oracle, seed=43)
    s.grads[0][0][5] = float("inf")
    plan = _plan([600], False, 1)
    ddp.ddp_clip_grads(plan, s.table, 1, ddp.ddp_grad_norm(plan, s.table, 1), 1.0)
    got = to_host(s.grads[0][0])
    assert np.isnan(got[5]) and (np.delete(got, 5) == 0).all()


# ---------------------------------------------------------------------------
# Fused into the all-reduce
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["aligned", "odd", "mixed"])
@pytest.mark.parametrize("kind", ["l2", "l1", "inf"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("p,avg", [(1, "world"), (2, "none"), (3, "tokens"), (8, "world")])
def test_allreduce_with_norm(oracle, p, avg, bf16, kind, layout):
    s = Set(p, SIZES, bf16, layout, oracle, seed=51)
    plan = _plan(SIZES, bf16, p)
    tokens = tokens_for(p, 3) if avg == "tokens" else None
    ws, guard = _workspace(plan.sync_norm_workspace())
    st = ddp.ddp_allreduce_buckets_norm(plan, 0, plan.num_buckets, s.table, p, ws,
                                        norm_type=kind, avg=avg, tokens=tokens)
    assert st.hbm_bytes == 2 * p * sum(SIZES) * (2 if bf16 else 4)
    each = torch.full((len(SIZES),), -1.0, device="cuda")
    norm = ddp.ddp_grad_norm_finish(plan, ws, norm_type=kind, param_norms=each)
    torch.cuda.synchronize()
    assert (guard == 255).all()
    avgs = _averages(s, SIZES, oracle, avg, tokens, bf16)
    _close(to_host(norm)[0], _norm64(avgs, kind))
    _close(to_host(each), [_norm64([v], kind) for v in avgs])
    for r in range(p):
        for i in range(len(SIZES)):
            assert_bits_equal(to_host(s.grads[r][i]), _narrow(avgs[i], bf16, oracle), f"{r} {i}")
    s.check_gaps()


CLIP_CASES = [("many", 1, "tokens", 0.001), ("many", 1, "none", 0.5), ("many", 2, "world", 0.5),
              ("many", 3, "none", 1e9), ("many", 4, "world", 1.5), ("many", 5, "tokens", 1e-4),
              ("many", 8, "none", 2.0), ("many", 13, "world", 0.25), ("ranks", 64, "world", 0.25),
              ("ranks", 33, "none", 3.0)]
CLIP_CASES += [(shape, p, "world", 0.25) for shape in sorted(SHAPES) for p in (1, 2, 4, 7)
               if shape != "many"]


@pytest.mark.parametrize("layout", ["aligned", "odd", "mixed"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shape,p,avg,max_norm", CLIP_CASES)
def test_allreduce_clip(oracle, shape, p, avg, max_norm, bf16, layout):
    sizes = SHAPES.get(shape, [3000, 5, 0, 257])
    s = Set(p, sizes, bf16, layout, oracle, seed=52)
    plan = _plan(sizes, bf16, p)
    tokens = tokens_for(p, 3) if avg == "tokens" else None
    ws, guard = _workspace(plan.sync_norm_workspace())
    norm = torch.full((1,), -1.0, device="cuda")
    each = torch.full((len(sizes),), -1.0, device="cuda")
    st = ddp.ddp_allreduce_clip(plan, s.table, p, max_norm, norm, ws, avg=avg, tokens=tokens,
                                param_norms=each)
    torch.cuda.synchronize()
    assert (guard == 255).all()
    assert st.steps == 2 * (p - 1) * plan.num_buckets
    avgs = _averages(s, sizes, oracle, avg, tokens, bf16)
    _close(to_host(norm)[0], _norm64(avgs, "l2"))
    _close(to_host(each), [_norm64([v], "l2") for v in avgs])
    c = _coefficient(to_host(norm)[0], max_norm, 1e-6)
    for i in range(len(sizes)):
        want = _narrow(avgs[i] * c, bf16, oracle)
        for r in range(p):
            assert_bits_equal(to_host(s.grads[r][i]), want, f"{r} {i}")
    s.check_gaps()


@pytest.mark.parametrize("kind", ["l2", "l1", "inf"])
@pytest.mark.parametrize("sizes", [
    [9_000_000, 17, 0, 65_536, 65_536, 500_000, 1],   # ends on a group of 256 tiles, or off it
    [256 * 256] * 129,                                # every parameter ends with a group
    [300] * 17_000 + [70_000],                        # a hundred parameters in a group
])
def test_norm_of_many_tiles(oracle, sizes, kind):
    """Plans past 32768 tiles, whose tile sums are joined in two steps (and
    parameters with more sums than one wave joins)."""
    plan = ddp.ddp_bucket_plan(sizes, 4).upload_segments(1)
    ws, guard = _workspace(plan.sync_norm_workspace())
    s = Set(1, sizes, False, "odd", oracle, seed=55)
    each = torch.full((len(sizes),), -1.0, device="cuda")
    ddp.ddp_allreduce_buckets_norm(plan, 0, plan.num_buckets, s.table, 1, ws, norm_type=kind)
    norm = ddp.ddp_grad_norm_finish(plan, ws, norm_type=kind, param_norms=each)
    torch.cuda.synchronize()
    assert (guard == 255).all()
    vals = [s.values(0, i) for i in range(len(sizes))]
    _close(to_host(norm)[0], _norm64(vals, kind))
    _close(to_host(each), [_norm64([v], kind) for v in vals])
    ws, guard = _workspace(plan.grad_norm_workspace(1))
    each.fill_(-1.0)
    norm = ddp.ddp_grad_norm(plan, s.table, 1, norm_type=kind, param_norms=each, workspace=ws)
    torch.cuda.synchronize()
    assert (guard == 255).all()
    _close(to_host(norm)[0], _norm64(vals, kind))
    _close(to_host(each), [_norm64([v], kind) for v in vals])


@pytest.mark.parametrize("kind", ["l1", "inf"])
def test_allreduce_clip_other_norms(oracle, kind):
    p = 4
    s = Set(p, SIZES, False, "odd", oracle, seed=53)
    plan = _plan(SIZES, False, p)
    ws, _ = _workspace(plan.sync_norm_workspace())
    norm = torch.empty(1, device="cuda")
    ddp.ddp_allreduce_clip(plan, s.table, p, 0.5, norm, ws, norm_type=kind, avg="world")
    avgs = _averages(s, SIZES, oracle, "world", None, False)
    _close(to_host(norm)[0], _norm64(avgs, kind))
    c = _coefficient(to_host(norm)[0], 0.5, 1e-6)
    for i in range(len(SIZES)):
        assert_bits_equal(to_host(s.grads[p - 1][i]), avgs[i] * c)


@pytest.mark.parametrize("bf16", [False, True])
def test_one_call_equals_the_three(oracle, bf16):
    """ddp_allreduce_clip against ddp_allreduce_buckets_norm, finish and the
    replicated clip: the same norm, and in fp32 the same gradients."""
    p = 5
    a, b = (Set(p, SIZES, bf16, "odd", oracle, seed=54) for _ in range(2))
    plan = _plan(SIZES, bf16, p)
    ws, _ = _workspace(plan.sync_norm_workspace())
    one = torch.empty(1, device="cuda")
    ddp.ddp_allreduce_clip(plan, a.table, p, 0.75, one, ws, avg="world")
    ws2, _ = _workspace(plan.sync_norm_workspace())
    for k in range(plan.num_buckets):  # a run per bucket, in any order
        ddp.ddp_allreduce_buckets_norm(plan, plan.num_buckets - 1 - k, 1, b.table, p, ws2,
                                       avg="world")
    three = ddp.ddp_grad_norm_finish(plan, ws2)
    assert_bits_equal(to_host(three), to_host(one))
    if not bf16:
        ddp.ddp_clip_grads(plan, b.table, p, three, 0.75, replicated=True)
        for r in range(p):
            for i in range(len(SIZES)):
                assert_bits_equal(to_host(b.grads[r][i]), to_host(a.grads[r][i]))


@pytest.mark.parametrize("cap", [0, 5])
@pytest.mark.parametrize("bf16", [False, True])
def test_reducer_with_norm_then_clip(oracle, bf16, cap):
    """A step as it is run: gradients marked ready one by one, the buckets
    reduced on a second stream with their norm's sums, then the norm and the
    clip on the first; twice, with fresh gradients."""
    p = 4
    plan = _plan(SIZES, bf16, p)
    s = Set(p, SIZES, bf16, "aligned", oracle, seed=61)
    comm = torch.cuda.Stream()
    red = ddp.Reducer(plan, p, s.table, avg="world", comm_stream=comm)
    red.set_max_workgroups(cap)
    ws, guard = _workspace(plan.sync_norm_workspace())
    red.set_norm(ws, "l2")
    for step in range(2):
        fresh = Set(p, SIZES, bf16, "aligned", oracle, seed=62 + step)
        torch.cuda.synchronize()
        red.prepare()
        for i in reversed(range(len(SIZES))):
            for r in range(p):
                s.grads[r][i].copy_(fresh.grads[r][i])
            ev = torch.cuda.Event()
            ev.record()
            red.mark_ready(i, ev)
        red.finalize()
        norm = ddp.ddp_grad_norm_finish(plan, ws)
        ddp.ddp_clip_grads(plan, s.table, p, norm, 0.5, replicated=True)
        torch.cuda.synchronize()
        avgs = _averages(fresh, SIZES, oracle, "world", None, bf16)
        _close(to_host(norm)[0], _norm64(avgs, "l2"))
        c = _coefficient(to_host(norm)[0], 0.5, 1e-6)
        for i in range(len(SIZES)):
            held = _wide(_narrow(avgs[i], bf16, oracle))
            want = _narrow(held * c, bf16, oracle)
            for r in range(p):
                assert_bits_equal(to_host(s.grads[r][i]), want, f"step {step} {r} {i}")
    assert (guard == 255).all()
    # without the norm again: the plain all-reduce
    red.set_norm(None)
    red.prepare()
    ws.fill_(255)
    for i in range(len(SIZES)):
        red.mark_ready(i)
    red.finalize()
    torch.cuda.synchronize()
    assert (ws == 255).all()


@pytest.mark.parametrize("sizes", [
    [4096 * 1024, 1024 * 1024, 4096, 16_384 * 1024, 32],        # whole cache lines
    [4_000_003, 1_000_001, 77, 17_000_005, 1],                  # tiles inside lines
])
@pytest.mark.parametrize("bf16", [False, True])
def test_past_the_caches(sizes, bf16):
    """Sets beyond the Infinity Cache, where stores, residency and the tiles'
    order follow other rules. Small integers: averages of 8 and their squares
    add up exactly in any order, so every value has one right answer."""
    p, dt = 8, torch.bfloat16 if bf16 else torch.float32
    stride = sum(sizes) + 64
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    arena = torch.randint(-8, 9, (p, stride), generator=g, device="cuda").to(dt)
    assert arena.numel() * arena.element_size() > (256 << 20)
    grads = [list(arena[r][:sum(sizes)].split(sizes)) for r in range(p)]
    table = ddp.grad_pointer_table(grads)
    plan = ddp.ddp_bucket_plan(sizes, 2 if bf16 else 4).upload_segments(p)
    live = torch.zeros(stride, dtype=torch.bool, device="cuda")
    live[:sum(sizes)] = True

    def scales(norms, max_norm):
        # (in numpy: torch divides a number by a tensor as reciprocal and
        # product, two roundings)
        return to_dev(np.array([_coefficient(n, max_norm, 1e-6) for n in to_host(norms)]))

    # each rank clipped by its own norm
    norms = ddp.ddp_grad_norm(plan, table, p)
    exact = (arena.double() * live).square().sum(1).sqrt()
    _close(to_host(norms), exact.cpu().numpy())
    want = torch.where(live, arena.float() * scales(norms, 100.0)[:, None],
                       arena.float()).to(dt)
    keep = arena.clone()
    ddp.ddp_clip_grads(plan, table, p, norms, 100.0)
    assert torch.equal(arena, want)
    # the sum of all ranks, clipped
    arena.copy_(keep)
    total = keep.float().sum(0) / p
    ws, guard = _workspace(plan.sync_norm_workspace())
    norm = torch.empty(1, device="cuda")
    ddp.ddp_allreduce_clip(plan, table, p, 100.0, norm, ws, avg="world")
    _close(to_host(norm), (total.double() * live).square().sum().sqrt().reshape(1).cpu().numpy())
    got = (total * scales(norm, 100.0)).to(dt)
    want = torch.where(live, got.expand(p, -1), keep)
    assert torch.equal(arena, want)
    assert (guard == 255).all()
    # rank 0's spread to all, clipped again
    ddp.ddp_clip_grads(plan, table, p, norm, 50.0, replicated=True)
    got = (got.float() * scales(norm, 50.0)).to(dt)
    assert torch.equal(arena, torch.where(live, got.expand(p, -1), keep))
    # the averaging all-reduce with its norm
    arena.copy_(keep)
    ddp.ddp_allreduce_buckets_norm(plan, 0, plan.num_buckets, table, p, ws, avg="world")
    again = ddp.ddp_grad_norm_finish(plan, ws)
    _close(to_host(again), to_host(norm).astype(np.float64))
    assert torch.equal(arena, torch.where(live, total.to(dt).expand(p, -1), keep))


# ---------------------------------------------------------------------------
# Streams, graphs, timing
# ---------------------------------------------------------------------------

def test_captured_and_replayed(oracle):
    """Norm, clip and the fused call in one graph; every replay, on fresh
    gradients with eager work between, gives the eager bits."""
    p, sizes = 3, [3000, 17, 0, 40_000, 5, 12_345]
    plan = _plan(sizes, False, p)
    sets = [Set(p, sizes, False, "odd", oracle, seed=70) for _ in range(2)]
    ws = [_workspace(plan.sync_norm_workspace())[0] for _ in range(2)]
    ws.append(_workspace(plan.grad_norm_workspace(p))[0])
    norm, norms = torch.empty(1, device="cuda"), torch.empty(p, device="cuda")
    each = torch.empty(len(sizes), device="cuda")

    def fill(seed):
        for s in sets:
            for r in range(p):
                for i, n in enumerate(sizes):
                    s.grads[r][i].copy_(torch.from_numpy(W.normal_np(n, 1.0, seed, r, stream=i)))

    def work():
        ddp.ddp_grad_norm(plan, sets[0].table, p, norms, workspace=ws[2])
        ddp.ddp_clip_grads(plan, sets[0].table, p, norms, 1.0)
        ddp.ddp_allreduce_clip(plan, sets[1].table, p, 0.5, norm, ws[0], avg="world",
                               param_norms=each)
        ddp.ddp_allreduce_buckets_norm(plan, 0, plan.num_buckets, sets[0].table, p, ws[1])
        ddp.ddp_grad_norm_finish(plan, ws[1], norm_type="l2", param_norms=each)

    def state():
        torch.cuda.synchronize()
        return ([to_host(g) for s in sets for rank in s.grads for g in rank]
                + [to_host(norm), to_host(norms), to_host(each)])

    want = {}
    for seed in (1, 2, 3):
        fill(seed)
        work()
        want[seed] = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for seed in (1, 2, 3, 2):
        fill(seed)
        torch.cuda.synchronize()
        g.replay()
        for a, b in zip(state(), want[seed]):
            assert_bits_equal(a, b, f"seed {seed}")
        x = torch.randn(1 << 20, device="cuda")
        (x * 2).sum().item()


def test_on_another_stream(oracle):
    """`stream=` with outputs and workspaces of the call's own, several in a
    row, against the same on the current stream."""
    p, sizes = 2, [50_000, 3, 1000]
    a, b = (Set(p, sizes, True, "odd", oracle, seed=80) for _ in range(2))
    plan = _plan(sizes, True, p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        n = ddp.ddp_grad_norm(plan, a.table, p, stream=side)
        ddp.ddp_clip_grads(plan, a.table, p, n, 20.0, stream=side)
        got.append(n)
    side.synchronize()
    want = []
    for _ in range(3):
        n = ddp.ddp_grad_norm(plan, b.table, p)
        ddp.ddp_clip_grads(plan, b.table, p, n, 20.0)
        want.append(n)
    for x, y in zip(got, want):
        assert_bits_equal(to_host(x), to_host(y))
    for r in range(p):
        for i in range(len(sizes)):
            assert_bits_equal(to_host(a.grads[r][i]), to_host(b.grads[r][i]))


def test_events_bracket_the_calls(oracle):
    p, sizes = 2, [400_000, 3]
    s = Set(p, sizes, False, "aligned", oracle, seed=90)
    plan = _plan(sizes, False, p)
    ws, _ = _workspace(plan.sync_norm_workspace())
    norm = torch.empty(1, device="cuda")
    timer = ddp.CallTimer(pairs=4)
    calls = [lambda: ddp.ddp_grad_norm(plan, s.table, p),
             lambda: ddp.ddp_clip_grads(plan, s.table, p, norm, 1e-3),
             lambda: ddp.ddp_allreduce_clip(plan, s.table, p, 1e-3, norm, ws),
             lambda: ddp.ddp_grad_norm_finish(plan, ws, norm)]
    for call in calls:
        call()
        k = timer.arm()
        call()
        torch.cuda.synchronize()
        assert 0 < timer.elapsed_ms(k) < 50


def test_refusals_on_device(oracle):
    p, sizes = 2, [100, 20]
    s = Set(p, sizes, False, "aligned", oracle, seed=91)
    plan = ddp.ddp_bucket_plan(sizes, 4)
    with pytest.raises(ddp.DDPError, match="ENOTREADY"):
        ddp.ddp_grad_norm(plan, s.table, p)
    plan.upload_segments(p)
    small = torch.empty(8, dtype=torch.uint8, device="cuda")
    with pytest.raises(ddp.DDPError, match="EWORKSPACE"):
        ddp.ddp_grad_norm(plan, s.table, p, workspace=small)
    with pytest.raises(ddp.DDPError, match="EWORKSPACE"):
        ddp.ddp_allreduce_clip(plan, s.table, p, 1.0, torch.empty(1, device="cuda"), small)
    with pytest.raises(ddp.DDPError, match="EINVAL"):
        ddp.ddp_clip_grads(plan, s.table, p, torch.ones(1, device="cuda"), -1.0)
    with pytest.raises(ValueError, match="elements"):
        ddp.ddp_clip_grads(plan, s.table, p, torch.ones(3, device="cuda"), 1.0)
    with pytest.raises(ValueError, match="elements"):
        ddp.ddp_clip_grads(plan, s.table, p, torch.ones(2, device="cuda"), 1.0, replicated=True)
    with pytest.raises(ValueError, match="ranks"):
        ddp.ddp_grad_norm(plan, s.table, p, ranks=(1, 2))
    halves = [[torch.zeros(n, dtype=torch.float16, device="cuda") for n in sizes]
              for _ in range(p)]
    half_plan = ddp.ddp_bucket_plan(sizes, 2).upload_segments(p)
    with pytest.raises(TypeError, match="bfloat16"):
        ddp.ddp_grad_norm(half_plan, ddp.grad_pointer_table(halves), p)
    for r in range(p):
        for i in range(2):
            assert_bits_equal(to_host(s.grads[r][i]), s.host[r][i])
