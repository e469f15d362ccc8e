"""GPU: every launch form of the all-reduce with its norm and with clipping:
several tiles per wave (few ranks, many tiles), 32 and 8 rank loads in flight
(many ranks), tiles in runs per XCD and stores past the caches (large sets),
values that are not finite, and each call's outputs in a captured graph.

Norms: as in test_gpu_grad_norm.py, but the sets have up to 2^25.1 elements: a
sum of N terms in 64 bits is off by at most N 2^-53 of itself (2^-27 here),
the numpy sum by far less (pairwise), and the rounding to fp32 by 2^-24.
TOL = 2^-24 + 2^-27 + 2^-40 bounds the relative error of either norm. Sums of
small integers (the largest sets) are exact. Gradients are compared bit for
bit."""
import numpy as np
import pytest
import torch

import bucketed_gradient_all_ddp_amd as ddp
from bucketed_gradient_all_ddp_amd import workloads as W
from helpers import tokens_for
from test_gpu_grad_norm import _coefficient, _narrow, _norm64, _wide, _workspace

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -24 + 2.0 ** -27 + 2.0 ** -40


def _tiles(sizes, bf16):
    return sum(-(-n // (512 if bf16 else 256)) for n in sizes)


def _close(got, want, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert (np.abs(got - want) <= TOL * want).all(), (what, got, want)


def _same_bits(got, want, what):
    kind = np.uint16 if want.dtype == np.uint16 else np.uint32
    bad = np.nonzero(got.view(kind) != want.view(kind))[0]
    assert bad.size == 0, (what, bad.size, bad[:5].tolist(), got[bad[:3]], want[bad[:3]])


class Ranks:
    """p ranks' gradients in one host arena per rank, 7.0 between them:
    "aligned" at 32-byte places, "odd" one element apart from element 1 on
    (the same place on every rank), "mixed" shifted from rank to rank."""

    def __init__(self, p, sizes, bf16, layout, oracle, seed=0, scale=1.0):
        self.p, self.sizes, self.bf16, self.oracle = p, sizes, bf16, oracle
        self.places = []
        for r in range(p):
            at, offs = {"aligned": 0, "odd": 1, "mixed": r % 3 + 1}[layout], []
            for n in sizes:
                if layout == "aligned":
                    at = (at + 7) // 8 * 8
                offs.append(at)
                at += n + (0 if layout == "aligned" else 1)
            self.places.append(offs)
        self.length = (max(o[-1] for o in self.places) + sizes[-1] + 16 + 63) // 64 * 64
        total = sum(sizes)
        self.values = []  # fp32 values of each rank's gradients, end to end
        for r in range(p):
            v = np.resize(W.normal_np(min(total, 700_001 + 2 * r), scale, seed, r), total)
            self.values.append(_wide(oracle.f32_to_bf16(v)) if bf16 else v)
        self.cuts = np.concatenate([[0], np.cumsum(sizes)])

    def split(self, flat):
        return [flat[a:b] for a, b in zip(self.cuts[:-1], self.cuts[1:])]

    def arena(self, r, flat):
        """Rank r's arena with the fp32 values `flat` (rounded to the type)."""
        out = np.full(self.length, 7.0, np.float32)
        for o, v in zip(self.places[r], self.split(flat)):
            out[o:o + v.size] = v
        return _narrow(out, self.bf16, self.oracle)

    def upload(self):
        """Fresh copies of the inputs on the device."""
        rows = np.stack([self.arena(r, self.values[r]) for r in range(self.p)])
        if self.bf16:
            self.dev = torch.from_numpy(rows.view(np.int16)).cuda().view(torch.bfloat16)
        else:
            self.dev = torch.from_numpy(rows).cuda()
        grads = [[self.dev[r, o:o + n] for o, n in zip(self.places[r], self.sizes)]
                 for r in range(self.p)]
        self.grads = grads
        self.table = ddp.grad_pointer_table(grads)

    def averages(self, avg, tokens, cap, first):
        """The fp32 averages, folded in ring order by the oracle."""
        oplan = self.oracle.bucket_plan(self.sizes, 2 if self.bf16 else 4, cap, first)
        wide = [self.split(v.copy()) for v in self.values]
        for b in range(oplan.num_buckets):
            flats = [self.oracle.flatten(w, oplan, b) for w in wide]
            red, _ = self.oracle.ring_allreduce(flats, avg=avg, tokens=tokens, want_log=False)
            self.oracle.unflatten(red[0], oplan, b, wide[0])
        return np.concatenate(wide[0])

    def check(self, flat, what, nan=False):
        """Every rank holds `flat` (rounded to the type), and 7.0 between; with
        `nan` a NaN may be any NaN."""
        torch.cuda.synchronize()
        rows = self.dev.view(torch.int16) if self.bf16 else self.dev
        rows = rows.cpu().numpy()
        done = {}
        for r in range(self.p):
            key = tuple(self.places[r][:1])
            if key not in done:
                done[key] = self.arena(r, flat)
            got, want = rows[r].view(done[key].dtype), done[key]
            if nan:
                a, b = np.isnan(_wide(got)), np.isnan(_wide(want))
                assert np.array_equal(a, b), (what, r)
                got, want = np.where(b, 0, got).astype(got.dtype), np.where(b, 0, want).astype(
                    want.dtype)
            _same_bits(got, want, f"{what} rank {r}")


def _plan(s, cap, first):
    return ddp.ddp_bucket_plan(s.sizes, 2 if s.bf16 else 4, cap, first).upload_segments(s.p)


def _check_both(s, kind, avg, cap=96 * 1024, first=8 * 1024, param_norms=True):
    """ddp_allreduce_buckets_norm + finish, then ddp_allreduce_clip on fresh
    copies of the same gradients, against the oracle."""
    tokens = tokens_for(s.p, 3) if avg == "tokens" else None
    plan = _plan(s, cap, first)
    avgs = s.averages(avg, tokens, cap, first)
    norm64 = _norm64([avgs], kind)
    each64 = [_norm64([v], kind) for v in s.split(avgs)]
    ws, guard = _workspace(plan.sync_norm_workspace())

    s.upload()
    each = torch.full((len(s.sizes),), -1.0, device="cuda")
    ddp.ddp_allreduce_buckets_norm(plan, 0, plan.num_buckets, s.table, s.p, ws, norm_type=kind,
                                   avg=avg, tokens=tokens)
    norm = ddp.ddp_grad_norm_finish(plan, ws, norm_type=kind, param_norms=each)
    s.check(avgs, "norm")
    _close(norm.cpu().numpy()[0], norm64, "norm")
    _close(each.cpu().numpy(), each64, "parameter norms")

    s.upload()
    ws.fill_(255)
    norm.fill_(-1.0)
    each.fill_(-1.0)
    bound = 0.37 * norm64
    ddp.ddp_allreduce_clip(plan, s.table, s.p, bound, norm, ws, norm_type=kind, avg=avg,
                           tokens=tokens, param_norms=each if param_norms else None)
    c = _coefficient(norm.cpu().numpy()[0], bound, 1e-6)
    assert 0.3 < c < 0.4
    s.check(avgs * c, "clip")
    _close(norm.cpu().numpy()[0], norm64, "norm of the clip")
    if param_norms:
        _close(each.cpu().numpy(), each64, "parameter norms of the clip")
    assert (guard == 255).all()


# ---------------------------------------------------------------------------
# Few ranks: two and four tiles per wave
# ---------------------------------------------------------------------------

# parameters that end with a tile, inside one, one element around it, within a
# run of tiles; buckets of a few of them, so that the ring's chunk borders
# fall inside runs and inside vectors
MIXTURE = [300_001, 256 * 40, 1, 2, 3, 1023, 1024, 1025, 4096 + 5, 65_536, 7, 255, 257, 511, 513,
           33_333, 5, 0, 2048, 12]


def _many_tiles(tiles, bf16):
    """MIXTURE several times over and two large ones: at least `tiles` tiles."""
    sizes = MIXTURE * 3 + [1_234_567]
    per = 512 if bf16 else 256
    sizes += [(tiles - _tiles(sizes, bf16)) * per + 3, 9]
    return sizes


FEW = [(1, "tokens", "l2", 4), (2, "none", "l1", 4), (1, "tokens", "inf", 2), (2, "world", "l1", 2),
       (3, "world", "l2", 2), (4, "tokens", "inf", 2)]


@pytest.mark.parametrize("layout", ["aligned", "odd", "mixed"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("p,avg,kind,per_wave", FEW)
def test_several_tiles_per_wave(oracle, p, avg, kind, per_wave, bf16, layout):
    sizes = _many_tiles(16_384 * per_wave + 1, bf16)
    tiles = _tiles(sizes, bf16)
    # the sizes' rule: 16,384 waves, and not more parameters than waves
    assert 16_384 * per_wave <= tiles < 16_384 * 4 * (per_wave // 2)
    assert tiles >= per_wave * len(sizes)
    s = Ranks(p, sizes, bf16, layout, oracle, seed=110 + p)
    _check_both(s, kind, avg)


@pytest.mark.parametrize("bf16", [False, True])
def test_reducer_with_several_tiles_per_wave(oracle, bf16):
    """A capped reducer launch of one bucket that takes two tiles a wave, each
    workgroup several times."""
    p = 2
    sizes = _many_tiles(32_768 + 5, bf16)
    s = Ranks(p, sizes, bf16, "odd", oracle, seed=120)
    plan = _plan(s, 1 << 30, 1 << 30)
    assert plan.num_buckets == 1
    s.upload()
    red = ddp.Reducer(plan, p, s.table, avg="world", comm_stream=torch.cuda.Stream())
    red.set_max_workgroups(1000)
    ws, guard = _workspace(plan.sync_norm_workspace())
    red.set_norm(ws)
    torch.cuda.synchronize()
    red.prepare()
    for i in range(len(sizes)):
        red.mark_ready(i)
    red.finalize()
    norm = ddp.ddp_grad_norm_finish(plan, ws)
    avgs = s.averages("world", None, 1 << 30, 1 << 30)
    s.check(avgs, "reducer")
    _close(norm.cpu().numpy()[0], _norm64([avgs], "l2"))
    assert (guard == 255).all()


# ---------------------------------------------------------------------------
# Many ranks
# ---------------------------------------------------------------------------

MANY = [40_001, 256 * 40, 1, 2, 3, 1023, 1025, 4096 + 5, 255, 257, 20_000, 5, 0, 2048, 12, 9, 3]


@pytest.mark.parametrize("layout", ["aligned", "odd", "mixed"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("p,avg,kind,param_norms", [
    (9, "world", "l1", True), (17, "world", "l2", True), (32, "none", "l2", False),
    (33, "tokens", "inf", True), (64, "world", "l2", False), (64, "none", "l1", True)])
def test_many_ranks(oracle, p, avg, kind, param_norms, bf16, layout):
    """More tiles than one workgroup takes, few for the chip: 32 rank loads in
    flight, in one batch or two; joined by the second pass (no parameter
    norms) or by a launch."""
    assert 16 < _tiles(MANY, bf16) <= 1024
    s = Ranks(p, MANY, bf16, layout, oracle, seed=130 + p)
    _check_both(s, kind, avg, param_norms=param_norms)


@pytest.mark.parametrize("layout", ["aligned", "odd", "mixed"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("p,sizes", [
    (9, [700, 3, 0, 1300, 9, 256]), (16, [700, 3, 0, 1300, 9, 256]), (17, [700, 3, 0, 9]),
    (17, [700, 3, 0, 1300, 9, 256]), (33, [700, 3, 0, 9]), (64, [700, 3, 0, 1300, 9, 256]),
    (64, [700, 3, 0, 9])])
def test_few_tiles(oracle, p, sizes, bf16, layout):
    """Up to 16 tiles: by one workgroup or by several, with and without the
    parameters' norms."""
    assert _tiles(sizes, bf16) <= 16
    s = Ranks(p, sizes, bf16, layout, oracle, seed=135 + p)
    _check_both(s, "l2", "world", param_norms=False)
    _check_both(s, "l1", "tokens")


@pytest.mark.parametrize("layout", ["aligned", "odd", "mixed"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("p", [9, 33])
def test_many_ranks_many_tiles(oracle, p, bf16, layout):
    """Tiles for a full chip: 8 rank loads in flight, in p / 8 batches."""
    sizes = MANY + [(4100 * (512 if bf16 else 256)) + 1]
    assert _tiles(sizes, bf16) >= 4096
    s = Ranks(p, sizes, bf16, layout, oracle, seed=140 + p)
    _check_both(s, "l2", "world")


@pytest.mark.parametrize("layout", ["aligned", "odd", "mixed"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("p", [17, 33, 64])
def test_replicated_clip_many_ranks(oracle, p, bf16, layout):
    """Eight waves of a workgroup read one tile of rank 0 and write all ranks."""
    s = Ranks(p, MANY, bf16, layout, oracle, seed=150 + p)
    plan = _plan(s, 96 * 1024, 8 * 1024)
    s.upload()
    norm = torch.tensor([2.5], device="cuda")
    ddp.ddp_clip_grads(plan, s.table, p, norm, 1.75, replicated=True)
    s.check(s.values[0] * _coefficient(2.5, 1.75, 1e-6), "replicated")


# ---------------------------------------------------------------------------
# Values that are not finite, zeros with a sign, subnormal averages
# ---------------------------------------------------------------------------

SETS = {"one workgroup": [700, 3, 0, 300, 9], "two passes": [1400, 3, 30_001, 0, 9]}


@pytest.mark.parametrize("layout", ["aligned", "odd", "mixed"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["l2", "l1", "inf"])
@pytest.mark.parametrize("sizes", sorted(SETS))
@pytest.mark.parametrize("values", ["small", "inf", "nan"])
def test_special_values_through_the_fold(oracle, values, sizes, kind, bf16, layout):
    p, sizes = 4, SETS[sizes]
    s = Ranks(p, sizes, bf16, layout, oracle, seed=160)
    last = sum(sizes) - 1
    for r in range(p):
        v = s.values[r]
        v[:200] *= np.float32(2.0 ** -131)   # subnormal sums and averages
        if bf16:
            v[:200] = _wide(oracle.f32_to_bf16(v[:200]))
        v[5] = v[250] = v[last - 1] = -0.0   # on every rank: an average of -0
    if values != "small":
        s.values[1][300] = s.values[2][701] = np.inf
        s.values[0][last] = -np.inf
    if values == "nan":
        s.values[3][300] = -np.inf           # against rank 1's infinity
        s.values[2][702] = np.nan
    plan = _plan(s, 96 * 1024, 8 * 1024)
    with np.errstate(all="ignore"):
        avgs = s.averages("world", None, 96 * 1024, 8 * 1024)
        parts = s.split(avgs)
        norm64 = _norm64([avgs], kind)
        each64 = [_norm64([v], kind) for v in parts]
    assert (np.signbit(avgs) & (avgs == 0)).sum() >= 3
    tiny = np.abs(avgs[:200])
    assert ((tiny > 0) & (tiny < np.finfo(np.float32).tiny)).sum() > 100

    def norm_agrees(got, want, what):
        for g, w in zip(np.atleast_1d(got), np.atleast_1d(want)):
            if np.isfinite(w):
                _close(g, w, what)
            else:
                assert np.isnan(g) if np.isnan(w) else np.isposinf(g), (what, g, w)

    ws, guard = _workspace(plan.sync_norm_workspace())
    each = torch.full((len(sizes),), -1.0, device="cuda")
    s.upload()
    ddp.ddp_allreduce_buckets_norm(plan, 0, plan.num_buckets, s.table, p, ws, norm_type=kind,
                                   avg="world")
    norm = ddp.ddp_grad_norm_finish(plan, ws, norm_type=kind, param_norms=each)
    s.check(avgs, "norm", nan=True)
    norm_agrees(norm.cpu().numpy(), norm64, "norm")
    norm_agrees(each.cpu().numpy(), each64, "parameter norms")
    for bound in (0.25, np.inf):
        for wanted in (each, None):
            s.upload()
            norm.fill_(-1.0)
            each.fill_(-1.0)
            ddp.ddp_allreduce_clip(plan, s.table, p, bound, norm, ws, norm_type=kind, avg="world",
                                   param_norms=wanted)
            got = norm.cpu().numpy()
            norm_agrees(got, norm64, "norm of the clip")
            if wanted is not None:
                norm_agrees(each.cpu().numpy(), each64, "parameter norms of the clip")
            with np.errstate(all="ignore"):
                want = avgs * _coefficient(got[0], bound, 1e-6)
            s.check(want, f"clip {bound}", nan=True)
    assert (guard == 255).all()


# ---------------------------------------------------------------------------
# Large sets
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("form", ["whole lines", "inside lines"])
@pytest.mark.parametrize("p,avg", [(1, "tokens"), (2, "world"), (4, "none"), (8, "world")])
def test_past_the_caches_same_phase(p, avg, form, bf16):
    """Beyond the caches with every rank's row at the same place in a cache
    line: 16-byte accesses, with tiles on whole lines (stores past the caches)
    or inside lines (runs of neighbouring tiles per XCD, from 512 MiB on).
    Small integers divided by powers of two: one right answer."""
    dt, eb = (torch.bfloat16, 2) if bf16 else (torch.float32, 4)
    n = (560 << 20) // (p * eb)
    if form == "whole lines":
        n = n // 1024 * 1024
        sizes = [4096 * 1024, 1024 * 1024, 4096, 128]
        sizes = sizes + [n - sum(sizes)]
        assert all(k * eb % 128 == 0 for k in sizes)
    else:
        sizes = [4_000_003, 1_000_001, 77, 1]
        sizes = sizes + [n - sum(sizes)]
    total = sum(sizes)
    stride = (total + 64) // 64 * 64 + 64
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    keep = torch.randint(-8, 9, (p, stride), generator=g, device="cuda").to(dt)
    arena = keep.clone()
    assert arena.data_ptr() % 128 == 0 and stride * eb % 128 == 0 and p * total * eb > (512 << 20)
    grads = [list(arena[r][:total].split(sizes)) for r in range(p)]
    table = ddp.grad_pointer_table(grads)
    plan = ddp.ddp_bucket_plan(sizes, eb).upload_segments(p)
    tokens = [2] if avg == "tokens" else None
    ws, guard = _workspace(plan.sync_norm_workspace())

    folded = keep[:, :total].float().sum(0)
    if avg != "none":
        folded /= 2 if avg == "tokens" else p
    squares = folded.double().square()
    exact = float(squares.sum().sqrt())
    each64 = [float(v.sum().sqrt()) for v in squares.split(sizes)]
    del squares

    def whole(flat):
        out = keep.clone()
        out[:, :total] = flat.to(dt)
        return out

    each = torch.full((len(sizes),), -1.0, device="cuda")
    ddp.ddp_allreduce_buckets_norm(plan, 0, plan.num_buckets, table, p, ws, avg=avg, tokens=tokens)
    norm = ddp.ddp_grad_norm_finish(plan, ws, param_norms=each)
    assert torch.equal(arena, whole(folded))
    _close(norm.cpu().numpy()[0], exact)
    _close(each.cpu().numpy(), each64)

    arena.copy_(keep)
    norm.fill_(-1.0)
    each.fill_(-1.0)
    ddp.ddp_allreduce_clip(plan, table, p, 100.0, norm, ws, avg=avg, tokens=tokens,
                           param_norms=each)
    _close(norm.cpu().numpy()[0], exact)
    _close(each.cpu().numpy(), each64)
    c = torch.from_numpy(np.array([_coefficient(norm.cpu().numpy()[0], 100.0, 1e-6)])).cuda()
    assert torch.equal(arena, whole(folded * c))
    assert (guard == 255).all()

    # each rank by its own norm, then rank 0's to all
    arena.copy_(keep)
    norms = ddp.ddp_grad_norm(plan, table, p)
    _close(norms.cpu().numpy(),
           [float(keep[r, :total].double().square().sum().sqrt()) for r in range(p)])
    ddp.ddp_clip_grads(plan, table, p, norms, 100.0)
    host = norms.cpu().numpy()
    own = torch.from_numpy(np.array([_coefficient(v, 100.0, 1e-6) for v in host])).cuda()
    assert torch.equal(arena, whole(keep[:, :total].float() * own[:, None]))
    arena.copy_(keep)
    ddp.ddp_clip_grads(plan, table, p, norms[:1], 100.0, replicated=True)
    assert torch.equal(arena, whole(keep[0, :total].float() * own[:1]))


# ---------------------------------------------------------------------------
# Every output of every call in one captured graph
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bf16", [False, True])
def test_captured_outputs_apart(oracle, bf16):
    """Three forms of the clip (one workgroup; joined by the second pass; by a
    launch, with parameter norms) and the norm's own calls, each with outputs
    and a workspace of its own, replayed on fresh gradients."""
    p = 3
    shapes = {"small": [700, 3, 0, 300, 9], "inline": [30_000, 17, 0, 5],
              "joined": [30_000, 17, 0, 40_000, 5], "norm": [30_000, 17, 0, 5]}
    sets = {k: Ranks(p, v, bf16, "odd", oracle, seed=171) for k, v in shapes.items()}
    plans = {k: _plan(s, 96 * 1024, 8 * 1024) for k, s in sets.items()}
    ws = {k: _workspace(q.sync_norm_workspace())[0] for k, q in plans.items()}
    ws["own"] = _workspace(plans["norm"].grad_norm_workspace(p))[0]
    out = {k: torch.empty(1, device="cuda") for k in shapes}
    out["own"] = torch.empty(p, device="cuda")
    each = {k: torch.empty(len(v), device="cuda") for k, v in shapes.items() if k != "inline"}
    each["own"] = torch.empty(p, len(shapes["norm"]), device="cuda")
    for s in sets.values():
        s.upload()
    inputs = {}
    for seed in (1, 2, 3):
        for k, v in shapes.items():
            fresh = Ranks(p, v, bf16, "odd", oracle, seed=180 + seed)
            fresh.upload()
            inputs[seed, k] = fresh.dev

    def fill(seed):
        for k, s in sets.items():
            s.dev.copy_(inputs[seed, k])
        for t in list(out.values()) + list(each.values()):
            t.fill_(-1.0)

    def work():
        for k in ("small", "inline", "joined"):
            ddp.ddp_allreduce_clip(plans[k], sets[k].table, p, 0.5, out[k], ws[k], avg="world",
                                   param_norms=each.get(k))
        q, s = plans["norm"], sets["norm"]
        ddp.ddp_grad_norm(q, s.table, p, out["own"], param_norms=each["own"], workspace=ws["own"])
        ddp.ddp_allreduce_buckets_norm(q, 0, q.num_buckets, s.table, p, ws["norm"], avg="world")
        ddp.ddp_grad_norm_finish(q, ws["norm"], out["norm"], param_norms=each["norm"])

    def state():
        torch.cuda.synchronize()
        return {**{("grads", k): s.dev.clone() for k, s in sets.items()},
                **{("norm", k): t.clone() for k, t in out.items()},
                **{("each", k): t.clone() for k, t in each.items()}}

    want = {}
    for seed in (1, 2, 3):
        fill(seed)
        work()
        want[seed] = state()
        for k, s in sets.items():
            s.values = Ranks(p, shapes[k], bf16, "odd", oracle, seed=180 + seed).values
            avgs = s.averages("world", None, 96 * 1024, 8 * 1024)
            _close(out[k].cpu().numpy()[0], _norm64([avgs], "l2"), k)
            if k in each:
                _close(each[k].cpu().numpy(), [_norm64([v], "l2") for v in s.split(avgs)], k)
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
        for key, t in state().items():
            a, b = t, want[seed][key]
            kind = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
            assert torch.equal(a.view(kind), b.view(kind)), (seed, key)
        x = torch.randn(1 << 20, device="cuda")
        (x * 2).sum().item()


@pytest.mark.parametrize("handle", [False, True])
def test_abandoned_pass_keeps_the_workspace(oracle, handle):
    """A pass that is given up with launches still queued on the communication
    stream: the sums' memory is handed to nobody else before they have run."""
    p, sizes = 2, [30_000, 17, 0, 5]
    s = Ranks(p, sizes, False, "odd", oracle, seed=190)
    plan = _plan(s, 96 * 1024, 8 * 1024)
    s.upload()
    avgs = s.averages("world", None, 96 * 1024, 8 * 1024)
    comm = torch.cuda.Stream()
    red = ddp.Reducer(plan, p, s.table, avg="world",
                      comm_stream=comm.cuda_stream if handle else comm)
    big = torch.zeros(2, 1 << 28, device="cuda")
    torch.cuda.synchronize()
    ws = torch.empty(plan.sync_norm_workspace(), dtype=torch.uint8, device="cuda")
    address, nbytes = ws.data_ptr(), ws.numel()
    red.set_norm(ws)
    red.prepare()
    with torch.cuda.stream(comm):  # a few milliseconds of copies ahead of the launches
        for _ in range(60):
            big[1].copy_(big[0])
    for i in range(len(sizes)):
        red.mark_ready(i)
    del ws, red
    others = [torch.full((nbytes,), 9, dtype=torch.uint8, device="cuda") for _ in range(20)]
    assert all(t.data_ptr() != address for t in others)
    assert not comm.query()  # the launches had not run yet
    torch.cuda.synchronize()
    assert all(bool((t == 9).all()) for t in others)
    s.check(avgs, "all-reduce")
