"""The gradient-norm and clipping operators, case by case: what a training
step asks of the gradients of p ranks around their synchronisation.

  norm       the global norm (L2, L1 or largest magnitude) of each rank's
             gradients over many tensors, and each tensor's own norm
  clip       every gradient scaled by min(1, max_norm / (norm + 1e-6)), the
             norm taken from device memory: rank by rank, or one norm for
             gradients that are replicated (equal on every rank)
  sync_norm  the averaging all-reduce of all buckets, and the norm of the
             averaged gradient
  sync_clip  the averaging (or summing) all-reduce, its norm, and the clipped
             gradient on every rank

`own` False: plain torch operations on one arena of all gradients. `own`
True: the library's entry points on the per-parameter tensors, which are
views of that arena.
"""
import math
import random

import torch

own = False

EPS = 1e-6
MAX_NORM = 1.0  # the usual bound; inputs are scaled to norms of a few units


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _case(name, op, kind, p, dtype, **more):
    c = {"name": name, "op": op, "kind": kind, "p": p, "dtype": dtype, "norm": "l2",
         "packed": False, "param_norms": False}
    c.update(more)
    return c


def listed():
    return [
        # a probe or an adapter of a few tensors: the call's latency
        _case("norm-smallest", "norm", "spread", 1, "f32", count=4, elements=4099, spread=30.0,
              sizes=1),
        # GPT-2 small, one rank of a synchronised set, each tensor's norm for the log
        _case("norm-gpt2-f32", "norm", "gpt2", 1, "f32", layers=12, d=768, vocab=50257, ctx=1024,
              param_norms=True),
        # each rank's own norm before the sync (the gradient noise scale): one
        # Llama-7B layer, bf16, 8 ranks
        _case("norm-llama-bf16-8ranks", "norm", "llama", 8, "bf16", layers=1, d=4096, ffn=11008),
        # thousands of odd tensors back to back in a flat buffer, with their norms
        _case("norm-many-odd-l1", "norm", "spread", 4, "f32", count=2500, elements=23_750_003,
              spread=1000.0, sizes=2, norm="l1", packed=True, param_norms=True),
        # each rank clipped to its own norm (local clipping before the sync)
        _case("clip-ranks-odd-bf16", "clip", "spread", 5, "bf16", count=500, elements=7_654_321,
              spread=300.0, sizes=3, packed=True, replicated=False),
        # the synchronised GPT-2 small gradients on 8 ranks, one norm
        _case("clip-gpt2-replicated", "clip", "gpt2", 8, "f32", layers=12, d=768, vocab=50257,
              ctx=1024, replicated=True),
        # the ragged ring: 1,000,003 elements on 4 ranks, odd tensors, largest magnitude
        _case("sync-norm-ragged-inf", "sync_norm", "spread", 4, "f32", count=10,
              elements=1_000_003, spread=4096.0, sizes=4, norm="inf", packed=True, avg="world"),
        # GPT-2 small, 8 ranks: the step's sync with its norm for the log
        _case("sync-norm-gpt2", "sync_norm", "gpt2", 8, "f32", layers=12, d=768, vocab=50257,
              ctx=1024, avg="world"),
        # a small model on 2 ranks: latency
        _case("sync-clip-small-bf16", "sync_clip", "spread", 2, "bf16", count=12, elements=30_011,
              spread=100.0, sizes=5, avg="world"),
        # GPT-2 small, 8 ranks: the whole step between backward and optimizer
        _case("sync-clip-gpt2", "sync_clip", "gpt2", 8, "f32", layers=12, d=768, vocab=50257,
              ctx=1024, avg="world"),
        # two Llama-7B layers in bf16 on 8 ranks: the largest
        _case("sync-clip-llama-bf16", "sync_clip", "llama", 8, "bf16", layers=2, d=4096,
              ffn=11008, avg="world"),
        # many ranks: 300 tensors on 64 ranks, gradients summed
        _case("sync-clip-64ranks", "sync_clip", "spread", 64, "f32", count=300,
              elements=2_850_000, spread=1000.0, sizes=6, avg="none"),
    ]


def draw(rng):
    op = rng.choice(["norm", "clip", "sync_norm", "sync_clip"])
    p = max(1, min(64, int(round(2 ** rng.uniform(-0.4, 6.0)))))
    total = 2 ** rng.uniform(11.0, 29.5)  # elements over all ranks
    n = max(16, int(total / p))
    dtype = rng.choice(["f32", "bf16"])
    more = {"norm": rng.choice(["l2", "l2", "l2", "l1", "inf"]), "packed": rng.random() < 0.5,
            "param_norms": op != "clip" and rng.random() < 0.4}
    if op == "clip":
        more["replicated"] = rng.random() < 0.5
    elif op == "sync_norm":
        more["avg"] = "world"
    elif op == "sync_clip":
        more["avg"] = rng.choice(["world", "none"])
    if n > 4_000_000 and rng.random() < 0.4:
        # a GPT-2-shaped set of about n elements
        layers = rng.randint(1, 12)
        d = max(64, 8 * int(math.sqrt(n / (12 * layers + 30)) / 8))
        more.update(layers=layers, d=d, vocab=rng.randint(10, 40) * d, ctx=rng.choice([256, 512, 1024]))
        return {k: v for k, v in _case("", op, "gpt2", p, dtype, **more).items() if k != "name"}
    count = int(2 ** rng.uniform(0.0, min(11.0, math.log2(n / 8), math.log2(20000 / p))))
    more.update(count=max(1, count), elements=n, spread=round(10 ** rng.uniform(0.0, 3.5), 1),
                sizes=rng.randrange(1 << 20))
    return {k: v for k, v in _case("", op, "spread", p, dtype, **more).items() if k != "name"}


def _sizes(case):
    """Element count of every tensor, in registration order."""
    kind = case["kind"]
    if kind == "gpt2":
        d, out = case["d"], [case["vocab"] * case["d"], case["ctx"] * case["d"]]
        block = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, 4 * d * d, 4 * d, 4 * d * d, d]
        return out + block * case["layers"] + [d, d]
    if kind == "llama":
        d, f = case["d"], case["ffn"]
        return ([d * d] * 4 + [f * d] * 3 + [d, d]) * case["layers"] + [d]
    # sizes log-uniform over a factor of `spread`, adding up to `elements`
    r = random.Random(case["sizes"])
    w = [case["spread"] ** r.random() for _ in range(case["count"])]
    scale = case["elements"] / sum(w)
    out = [max(1, int(x * scale)) for x in w]
    out[-1] = max(1, out[-1] + case["elements"] - sum(out))
    return out


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _inputs(case, seed):
    """One [p, stride] arena: a row per rank, the tensors at 16-byte aligned
    places, or back to back (packed, as in a flat bucket); gaps are zero."""
    dev = "cuda"
    dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    sizes, p = _sizes(case), case["p"]
    vec = 16 // (4 if case["dtype"] == "f32" else 2)
    at, offsets = 0, []
    for n in sizes:
        offsets.append(at)
        at += n if case["packed"] else -(-n // vec) * vec
    stride = -(-at // vec) * vec
    n = sum(sizes)
    # gradients whose (averaged) norm is about four
    fold = {"world": 1 / math.sqrt(p), "none": math.sqrt(p)}.get(case.get("avg"), 1.0)
    unit = {"l2": math.sqrt(n), "l1": 0.8 * n, "inf": 4.5}[case["norm"]]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    arena = torch.empty(p, stride, dtype=dtype, device=dev)
    for r in range(p):
        arena[r] = torch.randn(stride, generator=g, device=dev).mul_(4.0 / (unit * fold))
    ends = offsets[1:] + [stride]
    for o, k, e in zip(offsets, sizes, ends):
        if o + k < e:
            arena[:, o + k:e] = 0
    norms = None
    if case["op"] == "clip":  # norms just over the bound
        norms = MAX_NORM * (1.001 + 0.009 * torch.rand(1 if case["replicated"] else p,
                                                       generator=g, device=dev))
        if case["replicated"]:
            arena[1:] = arena[:1]
    return arena, sizes, offsets, stride, norms


def prepare(case, seed):
    arena, sizes, offsets, stride, norms = _inputs(case, seed)
    p = case["p"]
    ends = offsets[1:] + [stride]
    lengths = [e - o for o, e in zip(offsets, ends)]
    sync = case["op"].startswith("sync")
    s = {"case": case, "arena": arena, "norms": norms,
         "grads": [list(arena[r].split(lengths)) for r in range(p)]}
    # for the plain form: each tensor's stretch (a gap after it holds zeros)
    # in pieces of at most 4096 elements, and the pieces of each tensor
    pieces = [min(4096, k - i) for k in lengths for i in range(0, k, 4096)]
    counts = [-(-k // 4096) for k in lengths]
    rows = 1 if sync else p
    s["pieces"] = torch.tensor(pieces, device="cuda").repeat(rows)
    s["counts"] = torch.tensor(counts, device="cuda").repeat(rows)
    s["grads"] = [[v[:n] for v, n in zip(rank, sizes)] for rank in s["grads"]]
    if own:
        import bucketed_gradient_all_ddp_amd as ddp

        s["ddp"] = ddp
        s["plan"] = ddp.ddp_bucket_plan(sizes, arena.element_size()).upload_segments(p)
        s["table"] = ddp.grad_pointer_table(s["grads"])
        s["out"] = torch.empty(rows, device="cuda")
        s["param_out"] = torch.empty(rows, len(sizes), device="cuda") if case["param_norms"] else None
        need = (s["plan"].sync_norm_workspace() if sync else s["plan"].grad_norm_workspace(p))
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _norms(rows, s):
    """The norm of each row of a float32 matrix and, where the case has them,
    of each of its tensors: segmented sums (or maxima) over the pieces of
    each tensor, the pieces' results joined in 64 bits. A few rows of little
    data are summed at once, which takes fewer launches."""
    kind, wanted = s["case"]["norm"], s["case"]["param_norms"]
    each, how = None, "max" if kind == "inf" else "sum"
    v = rows.square() if kind == "l2" else rows.abs()
    if wanted or v.numel() > 1 << 21:
        v = torch.segment_reduce(v.reshape(-1), how, lengths=s["pieces"]).double()
        each = torch.segment_reduce(v, how, lengths=s["counts"]) if wanted else None
        v = v.reshape(rows.shape[0], -1)
    v = v.amax(-1) if kind == "inf" else v.sum(-1, dtype=torch.float64)
    if wanted:
        each = (each.sqrt() if kind == "l2" else each).float().reshape(rows.shape[0], -1)
    return (v.sqrt() if kind == "l2" else v).float(), each


def _scale(norm):
    return (MAX_NORM / (norm + EPS)).clamp(max=1.0)


def _plain(s):
    case, arena = s["case"], s["arena"]
    op = case["op"]
    out = {}
    if op == "norm":
        out["norm"], each = _norms(arena.float(), s)
    elif op == "clip":
        if case["replicated"]:
            arena.copy_((arena[0].float() * _scale(s["norms"])).expand_as(arena))
        else:
            arena.copy_(arena.float() * _scale(s["norms"])[:, None])
        return {"grads": arena}
    else:
        rows = arena.sum(0, keepdim=True, dtype=torch.float32)
        if case["avg"] == "world":
            rows = rows / case["p"]
        out["norm"], each = _norms(rows, s)
        arena.copy_((rows * _scale(out["norm"]) if op == "sync_clip" else rows).expand_as(arena))
        out["grads"] = arena
    if case["param_norms"]:
        out["param_norms"] = each
    return out


def _own(s):
    case, ddp, plan, p = s["case"], s["ddp"], s["plan"], s["case"]["p"]
    op, kind = case["op"], case["norm"]
    out = {}
    if op == "norm":
        out["norm"] = ddp.ddp_grad_norm(plan, s["table"], p, s["out"], norm_type=kind,
                                        param_norms=s["param_out"], workspace=s["workspace"])
    elif op == "clip":
        ddp.ddp_clip_grads(plan, s["table"], p, s["norms"], MAX_NORM, eps=EPS,
                           replicated=case["replicated"])
        return {"grads": s["arena"]}
    elif op == "sync_norm":
        ddp.ddp_allreduce_buckets_norm(plan, 0, plan.num_buckets, s["table"], p, s["workspace"],
                                       norm_type=kind, avg=case["avg"])
        out["norm"] = ddp.ddp_grad_norm_finish(plan, s["workspace"], s["out"], norm_type=kind,
                                               param_norms=s["param_out"])
        out["grads"] = s["arena"]
    else:
        ddp.ddp_allreduce_clip(plan, s["table"], p, MAX_NORM, s["out"], s["workspace"], eps=EPS,
                               norm_type=kind, avg=case["avg"], param_norms=s["param_out"])
        out["norm"] = s["out"]
        out["grads"] = s["arena"]
    if case["param_norms"]:
        out["param_norms"] = s["param_out"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without, and its answer in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    n, p = sum(_sizes(case)), case["p"]
    eb = 4 if case["dtype"] == "f32" else 2
    rows = 1 if case["op"].startswith("sync") else p
    small = 4 * rows * (1 + (len(_sizes(case)) if case["param_norms"] else 0))
    if case["op"] == "norm":
        return {"bytes": p * n * eb + small, "flops": 2 * p * n}
    if case["op"] == "clip":
        return {"bytes": ((1 if case["replicated"] else p) + p) * n * eb + small,
                "flops": (1 if case["replicated"] else p) * n}
    return {"bytes": 2 * p * n * eb + small, "flops": (p + 4) * n}


def exact(case, seed):
    arena, sizes, offsets, stride, norms = _inputs(case, seed)
    op, kind, p = case["op"], case["norm"], case["p"]

    def of(x):
        if x.numel() == 0:
            return torch.zeros((), dtype=torch.float64, device=x.device)
        x = x.double().abs()
        if kind == "inf":
            return x.max()
        return x.sum() if kind == "l1" else torch.dot(x, x).sqrt()

    def scale(v):
        c = MAX_NORM / (v + EPS)
        return torch.where(c < 1, c, torch.ones_like(c))

    def each(row):
        return torch.stack([of(row[o:o + n]) for o, n in zip(offsets, sizes)])

    if op == "clip":
        c = scale(norms.double())
        return {"grads": torch.stack([arena[r].double() * (c[0] if case["replicated"] else c[r])
                                      for r in range(p)])}
    if op == "norm":
        out = {"norm": torch.stack([of(arena[r]) for r in range(p)])}
        if case["param_norms"]:
            out["param_norms"] = torch.stack([each(arena[r]) for r in range(p)])
        return out
    total = torch.zeros(stride, dtype=torch.float64, device=arena.device)
    for r in range(p):
        total += arena[r]
    if case["avg"] == "world":
        total /= p
    norm = of(total)
    out = {"norm": norm.reshape(1),
           "grads": (total * scale(norm) if op == "sync_clip" else total).expand(p, stride)}
    if case["param_norms"]:
        out["param_norms"] = each(total).reshape(1, -1)
    return out
