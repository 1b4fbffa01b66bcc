"""Cases that measure the operators of a block whose rows go to several experts.

Where an atom's species picks the weights of a grouped product, the species is
given.  In a sparse block it is learnt: the rows start from an embedding, a
router picks a few experts for each, the rows travel to the experts' grouped
products and back, and dropout sits on the way back to the residual stream.

``embed``    y[i] = scale * w[ids[i]]; a training pass sorts the ids and adds
             dw[v] = scale * sum of dy over the rows that hold v.
``route``    scores (softmax or sigmoid) of logits, the k experts with the
             largest score + bias among the best groups of experts, and their
             weights (renormalised or not, times scale); a training pass adds
             the gradient of the logits.
``experts``  the assignments (row i, choice j) sorted by expert, the rows
             copied into that order (xs), and the experts' results h summed
             back by weight; a training pass adds the gradients of h, of the
             weights and of the rows.
``dropout``  y = residual + h * keep / (1 - p), keep from 16 bits of a
             counter-based generator for each element (Philox 4x32, 10 rounds:
             Salmon, Moraes, Dror, Shaw 2011); a training pass adds dh.

``run`` has each operator in its plain form (elementary torch operations in
32 bits, or in 64 where a choice hangs on them and for long sums, rounded once
at the end), or where ``own`` is true as the calls of this package.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
PER_BLOCK = 8                                 # elements that share a counter of the generator
PHILOX_MUL = (0xD2511F53, 0xCD9E8D57)         # the generator's published multipliers and key increments
PHILOX_KEY = (0x9E3779B9, 0xBB67AE85)
PHILOX_ROUNDS = 10


def _zs():
    from equivariant_interatomic_potential_gb300 import zs
    return zs


def listed():
    """Real work over the range, from a single row to what fills the memory system for a third of a millisecond."""
    return [
        # one new row against a large table: what a single lookup costs
        dict(name="embed_one_bf16", op="embed", direction="forward", dtype="bf16", M=1, V=50021, C=4096, ids="zipf", pad=0.0),
        # the 4096 atoms of the benchmark graph, 89 species, 32 channels, a training step
        dict(name="embed_atoms_f32", op="embed", direction="train", dtype="f32", M=4096, V=89, C=32, ids="zipf", pad=0.0),
        # an embedding for each pair of species on the 647170 edges, 96 channels: few rows hold most of the edges
        dict(name="embed_edges_f32", op="embed", direction="train", dtype="f32", M=647170, V=7921, C=96, ids="zipf", pad=0.0),
        # a step's ids from a vocabulary far larger than the step, a ragged batch with padding
        dict(name="embed_tokens_bf16", op="embed", direction="train", dtype="bf16", M=16384, V=50021, C=1024, ids="zipf", pad=0.05),
        # one row's choice
        dict(name="route_one_bf16", op="route", direction="forward", dtype="bf16", M=1, E=64, k=6, score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renormalise=True, masked=0.0),
        # 32768 rows, 256 experts in 8 groups of which 4 are kept, a bias for balance, a training pass
        dict(name="route_groups_f32", op="route", direction="train", dtype="f32", M=32768, E=256, k=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renormalise=True, masked=0.0),
        # odd sizes, some experts closed to some rows
        dict(name="route_odd_f16", op="route", direction="train", dtype="f16", M=9973, E=61, k=3, score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renormalise=False, masked=0.2),
        # one row to its eight experts and back
        dict(name="experts_one_bf16", op="experts", direction="forward", dtype="bf16", M=1, E=256, k=8, C=4096, dropped=0.0),
        # 32768 rows of 1024 channels, eight of 256 experts each, a training pass
        dict(name="experts_wide_bf16", op="experts", direction="train", dtype="bf16", M=32768, E=256, k=8, C=1024, dropped=0.0),
        # odd sizes, assignments beyond an expert's capacity dropped
        dict(name="experts_odd_f16", op="experts", direction="train", dtype="f16", M=4097, E=37, k=3, C=301, dropped=0.05),
        # the residual stream of a wide block, a training pass
        dict(name="dropout_wide_bf16", op="dropout", direction="train", dtype="bf16", M=32768, C=2048, p=0.1, residual=True),
        # odd sizes, no residual
        dict(name="dropout_odd_f32", op="dropout", direction="train", dtype="f32", M=4097, C=1031, p=0.5, residual=False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case over the listed ranges: sizes spread over their logarithm, half of them made odd."""
    def size(lo, hi, multiple=8):
        n = _log_uniform(rng, lo, hi)
        return max(lo, n // multiple * multiple) if rng.random() < 0.5 else n | 1

    case = dict(op=rng.choice(("embed", "route", "experts", "dropout")), direction=rng.choice(("forward", "train", "train")),
                dtype=rng.choice(("f32", "bf16", "f16")))
    if case["op"] == "embed":
        while True:
            case |= dict(M=size(1, 650000), V=size(1, 60000), C=size(8, 4096))
            if max(case["M"], case["V"]) * case["C"] <= 2 ** 26:
                return case | dict(ids=rng.choice(("uniform", "zipf")), pad=rng.choice((0.0, 0.05)))
    if case["op"] == "route":
        E = size(2, 512)
        groups = rng.choice([g for g in (1, 1, 2, 4, 8, 16) if E % g == 0 and E // g >= 2])
        top_groups = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(16, top_groups * (E // groups)))
        return case | dict(M=size(1, 65536), E=E, k=k, score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5,
                           groups=groups, top_groups=top_groups, group_top=rng.choice((1, 2)),
                           renormalise=rng.random() < 0.6, masked=rng.choice((0.0, 0.2)))
    if case["op"] == "experts":
        while True:
            case |= dict(M=size(1, 65536), E=size(2, 512), k=rng.randint(1, 12), C=size(8, 8192))
            if case["k"] <= case["E"] and case["M"] * case["k"] * case["C"] * BYTES[case["dtype"]] <= 2 ** 29:
                return case | dict(dropped=rng.choice((0.0, 0.05)))
    while True:
        case |= dict(M=size(1, 650000), C=size(8, 8192))
        if case["M"] * case["C"] <= 2 ** 26:
            return case | dict(p=rng.choice((0.0, 0.02, 0.1, 0.5)), residual=rng.random() < 0.5)


def work(case):
    s, M, train = BYTES[case["dtype"]], case["M"], case["direction"] == "train"
    if case["op"] == "embed":
        C, V = case["C"], case["V"]
        bytes_ = 4 * M + s * C * (min(M, V) + M) + (s * C * (M + V) if train else 0)
        return {"bytes": bytes_, "flops": M * C * (2 if train else 1)}
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        bytes_ = s * M * E + 8 * M * k + (4 * E if case["bias"] else 0) + (4 * M * k + s * M * E if train else 0)
        return {"bytes": bytes_, "flops": M * E * (8 if train else 5)}
    if case["op"] == "experts":
        C, k, E = case["C"], case["k"], case["E"]
        bytes_ = s * M * C * (2 + 2 * k) + 12 * M * k + 4 * (E + 1)   # x, xs, h, y; ids, slots and weights
        if train:
            bytes_ += s * M * C * (2 + 2 * k) + 4 * M * k             # dy, dh, dxs, dx; the weights' gradients
        return {"bytes": bytes_, "flops": M * k * C * (7 if train else 2)}
    n = M * case["C"]
    return {"bytes": s * n * (2 + case["residual"] + (2 if train else 0)), "flops": n * (3 if train else 2)}


# ---------------------------------------------------------------- inputs

def _inputs(case, seed):
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    s = dict(case)
    train = case["direction"] == "train"
    M = case["M"]
    if case["op"] == "embed":
        V, C = case["V"], case["C"]
        if case["ids"] == "zipf":
            p = (np.arange(V) + 1.0) ** -1.1
            ids = rng.permutation(V)[rng.choice(V, size=M, p=p / p.sum())]
        else:
            ids = rng.integers(0, V, size=M)
        ids = np.where(rng.random(M) < case["pad"], -1, ids)
        s["ids"] = torch.from_numpy(ids.astype(np.int32)).cuda()
        s["w"], s["scale"] = normal(V, C), math.sqrt(C)
        s["dy"] = normal(M, C) if train else None
    elif case["op"] == "route":
        E, k = case["E"], case["k"]
        z = torch.randn(M, E, generator=gen, device="cuda")
        if case["masked"]:
            z = torch.where(torch.rand(M, E, generator=gen, device="cuda") < case["masked"], -math.inf, z)
        s["logits"], s["scale"] = z.to(dt), 2.5
        s["bias"] = normal(E, dtype=torch.float32, scale=0.1) if case["bias"] else None
        s["dweights"] = normal(M, k, dtype=torch.float32) if train else None
    elif case["op"] == "experts":
        E, k, C = case["E"], case["k"], case["C"]
        popular = torch.randn(E, generator=gen, device="cuda")   # some experts are asked for more often
        ids = (torch.randn(M, E, generator=gen, device="cuda") + 0.5 * popular).topk(k, 1).indices.int()
        s["ids"] = torch.where(torch.rand(M, k, generator=gen, device="cuda") < case["dropped"], -1, ids).contiguous()
        s["weights"] = torch.softmax(torch.randn(M, k, generator=gen, device="cuda"), 1)
        s["x"], s["h"] = normal(M, C), normal(M * k, C)
        s["dy"], s["dxs"] = (normal(M, C), normal(M * k, C)) if train else (None, None)
    else:
        C = case["C"]
        s["h"], s["r"] = normal(M, C), normal(M, C) if case["residual"] else None
        s["dy"] = normal(M, C) if train else None
        s["seed"], s["call"], s["step"] = int(rng.integers(0, 2 ** 63)), 3, int(rng.integers(0, 2 ** 20))
    return s


def prepare(case, seed):
    """The operands on the GPU; the seed and the counters of a step are numbers that the program has."""
    return _inputs(case, seed)


# ---------------------------------------------------------------- one pass

def run(s):
    if s["op"] == "embed":
        return _own_embed(s) if own else _plain_embed(s)
    if s["op"] == "route":
        return _own_route(s) if own else _plain_route(s)
    if s["op"] == "experts":
        return _own_experts(s) if own else _plain_experts(s)
    return _own_dropout(s) if own else _plain_dropout(s)


def _own_embed(s):
    zs = _zs()
    out = {"y": zs.zs_embedding(s["w"], s["ids"], s["scale"])}
    if s["dy"] is not None:
        row_ptr, perm, _ = zs.zs_build_csr(s["ids"], s["V"])
        out["dw"] = zs.zs_embedding_backward(s["dy"], row_ptr, perm, s["scale"])
    return out


def _own_route(s):
    zs = _zs()
    how = dict(score=s["score"], renormalise=s["renormalise"], scale=s["scale"])
    ids, weights = zs.zs_route(s["logits"], s["k"], s["bias"], groups=s["groups"], top_groups=s["top_groups"],
                               group_top=s["group_top"], **how)
    out = {"ids": ids, "weights": weights}
    if s["dweights"] is not None:
        out["dlogits"] = zs.zs_route_backward(s["dweights"], s["logits"], ids, **how)
    return out


def _own_experts(s):
    zs = _zs()
    row_ptr, perm, _ = zs.zs_build_csr(s["ids"].view(-1), s["E"])
    xs, slot = zs.zs_dispatch(s["x"], row_ptr, perm, s["k"])
    out = {"row_ptr": row_ptr, "xs": xs, "slot": slot, "y": zs.zs_combine(s["h"], slot, s["weights"])}
    if s["dy"] is not None:
        out["dh"], out["dweights"] = zs.zs_combine_backward(s["dy"], s["h"], slot, s["weights"], row_ptr)
        out["dx"] = zs.zs_combine(s["dxs"], slot)
    return out


def _own_dropout(s):
    zs = _zs()
    counters = (s["p"], s["seed"], s["call"], s["step"])
    out = {"y": zs.zs_dropout(s["h"], *counters, residual=s["r"])}
    if s["dy"] is not None:
        out["dh"] = zs.zs_dropout(s["dy"], *counters)
    return out


def _plain_embed(s):
    w, ids, dt = s["w"], s["ids"].long(), s["w"].dtype
    held = (ids >= 0) & (ids < s["V"])
    at = torch.where(held, ids, 0)
    out = {"y": torch.where(held[:, None], w[at].float() * s["scale"], 0.0).to(dt)}
    if s["dy"] is not None:
        dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda")   # few rows may hold most ids: long sums
        dw.index_add_(0, at, torch.where(held[:, None], s["dy"].double(), 0.0))
        out["dw"] = (dw * s["scale"]).to(dt)
    return out


def _scores(z, kind):
    """Scores of logits, zeros where they are -inf."""
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0)


def _plain_route(s):
    M, E, k = s["M"], s["E"], s["k"]
    z = s["logits"].double()
    # the choice in 64 bits: two scores may lie closer than 32 bits can tell
    choice = _scores(z, s["score"])
    if s["bias"] is not None:
        choice = choice + s["bias"].double()
    choice = torch.where(z == -math.inf, -math.inf, choice)
    if s["top_groups"] < s["groups"]:
        best = choice.view(M, s["groups"], -1).sort(dim=2, descending=True, stable=True)[0][:, :, :s["group_top"]]
        value = torch.where(best[:, :, 0] == -math.inf, -math.inf, torch.where(best == -math.inf, 0.0, best).sum(2))
        kept = value.sort(dim=1, descending=True, stable=True)[1][:, :s["top_groups"]]
        mask = torch.zeros(M, s["groups"], dtype=torch.bool, device="cuda")
        mask[torch.arange(M, device="cuda")[:, None], kept] = True
        choice = torch.where(mask.repeat_interleave(E // s["groups"], 1), choice, -math.inf)
    value, at = choice.sort(dim=1, descending=True, stable=True)
    at, none = at[:, :k], value[:, :k] == -math.inf
    p = _scores(z.float(), s["score"])
    chosen = torch.where(none, 0.0, torch.gather(p, 1, at))
    total = chosen.sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0) if s["renormalise"] else torch.ones_like(total)
    share = chosen / total
    out = {"ids": torch.where(none, -1, at).int(), "weights": share * s["scale"]}
    if s["dweights"] is not None:
        g = torch.where(none, 0.0, s["dweights"] * s["scale"])
        if s["renormalise"]:
            g = (g - (share * g).sum(1, keepdim=True)) / total
        d = torch.zeros(M, E, device="cuda")
        d.scatter_add_(1, at, torch.where(none, 0.0, g))
        if s["score"] == "sigmoid":
            d = d * p * (1.0 - p)
        else:
            d = p * (d - (p * d).sum(1, keepdim=True))
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _plain_experts(s):
    M, k, E, dt = s["M"], s["k"], s["E"], s["x"].dtype
    flat = s["ids"].view(-1).long()
    live = (flat >= 0) & (flat < E)
    key = torch.where(live, flat, E)
    perm = key.sort(stable=True)[1]
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda").index_add_(0, key, torch.ones_like(key))
    row_ptr = torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)])
    at = torch.arange(M * k, device="cuda")
    slot = torch.empty_like(at)
    slot[perm] = at
    used = (at < row_ptr[E])[:, None]
    xs = torch.where(used, s["x"][perm // k].float(), 0.0).to(dt)
    rows = s["h"].float()[slot]
    w = torch.where(live, s["weights"].view(-1), 0.0)[:, None]
    y = torch.where(live[:, None], rows * w, 0.0).view(M, k, -1).sum(1).to(dt)
    out = {"row_ptr": row_ptr.int(), "xs": xs, "slot": torch.where(live, slot, -1).view(M, k).int(), "y": y}
    if s["dy"] is not None:
        dy = s["dy"].float()
        out["dh"] = torch.where(used, dy[perm // k] * w[perm], 0.0).to(dt)
        dots = (dy.repeat_interleave(k, 0) * rows).sum(1)
        out["dweights"] = torch.where(live, dots, 0.0).view(M, k)
        back = torch.where(live[:, None], s["dxs"].float()[slot], 0.0)
        out["dx"] = back.view(M, k, -1).sum(1).to(dt)
    return out


def _low_high(a, m):
    """Low and high 32 bits of a * m, both of 32 bits and held in 64 (where the product wraps, its bits stay)."""
    product = a * m
    return product & 0xFFFFFFFF, (product >> 32) & 0xFFFFFFFF


def _plain_keep(shape, p, seed, call, step):
    """Which elements dropout keeps, and the factor of those."""
    n = math.prod(shape)
    c = [torch.arange(-(-n // PER_BLOCK), device="cuda")]
    c = [c[0] & 0xFFFFFFFF, c[0] >> 32, torch.full_like(c[0], call), torch.full_like(c[0], step & 0xFFFFFFFF)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(PHILOX_ROUNDS):
        (l0, h0), (l1, h1) = _low_high(c[0], PHILOX_MUL[0]), _low_high(c[2], PHILOX_MUL[1])
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(a + b) & 0xFFFFFFFF for a, b in zip(key, PHILOX_KEY)]
    bits = torch.stack([part for word in c for part in (word & 0xFFFF, word >> 16)], 1)
    limit = round(p * 65536)
    return (bits.view(-1)[:n] >= limit).view(shape), 65536.0 / (65536 - limit)


def _plain_dropout(s):
    dt = s["h"].dtype
    keep, factor = _plain_keep(s["h"].shape, s["p"], s["seed"], s["call"], s["step"])
    y = torch.where(keep, s["h"].float() * factor, 0.0)
    out = {"y": (y if s["r"] is None else y + s["r"].float()).to(dt)}
    if s["dy"] is not None:
        out["dh"] = torch.where(keep, s["dy"].float() * factor, 0.0).to(dt)
    return out


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    train, M = case["direction"] == "train", case["M"]
    if case["op"] == "embed":
        table = torch.cat([s["w"].double() * s["scale"], torch.zeros(1, case["C"], dtype=torch.float64, device="cuda")])
        at = torch.where(s["ids"] < 0, case["V"], s["ids"]).long()
        out = {"y": table[at]}
        if train:   # the rows in the order of their ids, each id's rows by differences of the running sum within it
            order = torch.argsort(at)
            counts = torch.bincount(at, minlength=case["V"] + 1)
            out["dw"] = torch.segment_reduce(s["dy"].double()[order], "sum", lengths=counts, axis=0, unsafe=True)[:-1] * s["scale"]
        return out
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        z = s["logits"].double().requires_grad_(train)
        open_ = s["logits"] != -math.inf
        p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(torch.where(open_.any(1, keepdim=True), z, 0.0), 1)
        left = torch.where(open_, p.detach() + (0.0 if s["bias"] is None else s["bias"].double()), -math.inf)

        def largest(a):   # the largest of each row, at its lowest index
            top = a.amax(1, keepdim=True)
            index = torch.arange(a.shape[1], device="cuda")
            return top[:, 0], torch.where(a == top, index, a.shape[1]).amin(1)

        rows = torch.arange(M, device="cuda")
        G, per = case["groups"], E // case["groups"]
        if case["top_groups"] < G:
            values = []
            for g in range(G):
                part = left[:, g * per:(g + 1) * per].clone()
                total, at = largest(part)
                if case["group_top"] == 2:
                    part[rows, at] = -math.inf
                    second = part.amax(1)
                    total = total + torch.where(second == -math.inf, 0.0, second)
                values.append(total)
            values = torch.stack(values, 1)
            closed = torch.ones(M, G, dtype=torch.bool, device="cuda")
            rank = torch.arange(G, device="cuda")
            for g in range(G):   # a group is kept where fewer than top_groups come before it
                ahead = (values > values[:, g:g + 1]) | ((values == values[:, g:g + 1]) & (rank < g))
                closed[:, g] = ahead.sum(1) >= case["top_groups"]
            for g in range(G):
                left[:, g * per:(g + 1) * per][closed[:, g]] = -math.inf
        ids = []
        for _ in range(k):
            top, at = largest(left)
            left[rows, at] = -math.inf
            ids.append(torch.where(top == -math.inf, -1, at))
        ids = torch.stack(ids, 1)
        chosen = torch.where(ids < 0, 0.0, torch.gather(p, 1, ids.clamp_min(0)))
        weights = chosen * s["scale"]
        if case["renormalise"]:
            weights = weights / chosen.sum(1, keepdim=True).clamp_min(1e-300)
        out = {"ids": ids.int(), "weights": weights.detach()}
        if train:
            grad, = torch.autograd.grad(weights, z, s["dweights"].double())
            out["dlogits"] = torch.where(open_, grad, 0.0)
        return out
    if case["op"] == "experts":
        E, k, C = case["E"], case["k"], case["C"]
        flat = s["ids"].view(-1).long()
        order = torch.cat([torch.nonzero(flat == e)[:, 0] for e in range(E)] + [torch.nonzero(flat < 0)[:, 0]])
        n = int((flat >= 0).sum())
        row_ptr = torch.tensor([0] + torch.bincount(flat[flat >= 0], minlength=E).cumsum(0).tolist(), device="cuda")
        xs = torch.zeros(M * k, C, dtype=torch.float64, device="cuda")
        xs[:n] = s["x"].double()[torch.div(order[:n], k, rounding_mode="floor")]
        slot = torch.full((M * k,), -1, dtype=torch.int64, device="cuda")
        slot[order[:n]] = torch.arange(n, device="cuda")
        slot = slot.view(M, k)
        y = torch.zeros(M, C, dtype=torch.float64, device="cuda")
        out = {"row_ptr": row_ptr.int(), "xs": xs, "slot": slot.int(), "y": y}
        if train:
            dy = s["dy"].double()
            dh, dw, dx = torch.zeros_like(xs), torch.zeros(M, k, dtype=torch.float64, device="cuda"), torch.zeros_like(y)
            out |= {"dh": dh, "dweights": dw, "dx": dx}
        for j in range(k):
            rows = torch.nonzero(slot[:, j] >= 0)[:, 0]
            at = slot[rows, j]
            h, w = s["h"][at].double(), s["weights"][rows, j].double()[:, None]
            y[rows] += w * h
            if train:
                dh[at] = w * dy[rows]
                dw[rows, j] = torch.linalg.vecdot(dy[rows], h)
                dx[rows] += s["dxs"][at].double()
        return out
    # the generator again, with products of 16-bit halves
    n, C = M * case["C"], case["C"]
    limit = round(case["p"] * 65536)

    def multiplied(a, m):
        a0, a1, m0, m1 = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
        low = a0 * m0
        mid = a1 * m0 + (low >> 16)
        rest = a0 * m1 + (mid & 0xFFFF)
        return ((rest & 0xFFFF) << 16) | (low & 0xFFFF), a1 * m1 + (mid >> 16) + (rest >> 16)

    block = torch.arange((n + 7) // 8, device="cuda")
    x0, x1, x2, x3 = block % 2 ** 32, block // 2 ** 32, torch.zeros_like(block) + s["call"], torch.zeros_like(block) + s["step"]
    for i in range(10):
        k0, k1 = (s["seed"] % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32, (s["seed"] // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32
        a_low, a_high = multiplied(x0, 0xD2511F53)
        b_low, b_high = multiplied(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = b_high ^ x1 ^ k0, b_low, a_high ^ x3 ^ k1, a_low
    element = torch.arange(n, device="cuda")
    word = torch.stack((x0, x1, x2, x3))[(element % 8) // 2, element // 8]
    u = torch.where(element % 2 == 1, word // 65536, word % 65536)
    gain = torch.where(u < limit, 0.0, 65536.0 / (65536.0 - limit)).double().view(M, C)
    out = {"y": s["h"].double() * gain + (0.0 if s["r"] is None else s["r"].double())}
    if train:
        out["dh"] = s["dy"].double() * gain
    return out
