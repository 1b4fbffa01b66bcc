"""Cases that measure the training operators of a species-resolved block.

Next to the zonal scatter, a potential's update block multiplies each row of
its features by the weights of the row's group (its chemical species, or its
species and degree), normalises the result, gates it and adds it to the
residual stream, and its weights are stepped by AdamW.  Three operators:

``grouped``  y[i] = w[g(i)] x[i] over rows grouped by a stable CSR, and
             for a training pass dx[i] = w[g(i)]^T dy[i] and
             dw[g] = sum over rows i of g of dy[i] x[i]^T.
``norm``     y = x + scale * gate * (norm(h) * w_post), u = norm(y) * w_pre,
             gate = sigmoid(z), norm the root-mean-square norm or the layer
             norm of a row without its affine part; a training pass adds the
             gradients of all operands.
``adamw``    one AdamW step over many tensors at once, with states in
             32 bits, or in 8-bit floats (e4m3) with a scale for each 256
             elements: the first moment, and the root of the second one.

``run`` has each operator in its plain form (elementary torch operations in
32 bits, rounded once at the end), or where ``own`` is true as the calls of
this package.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 256            # elements that share a scale of 8-bit states
E4M3_MAX = 448.0       # largest e4m3 value
E4M3_TINY = 2.0 ** -9  # smallest positive e4m3 value
SCALE_MIN = 1e-30      # a block whose largest magnitude is below this is held as zeros
BETA1, BETA2, ADAM_EPS, LR, DECAY = 0.9, 0.999, 1e-8, 1e-3, 0.01
NORM_EPS = 1e-6


def _zs():
    from equivariant_interatomic_potential_gb300 import zs
    return zs


def listed():
    """Real work over the range: node and edge features of the graphs this package is configured for, wider blocks."""
    return [
        # one small molecule's node features (64 atoms, 32 channels), four species: what a single evaluation costs
        dict(name="grouped_tiny_f32", op="grouped", direction="forward", dtype="f32", M=64, K=32, N=32, G=4,
             sizes="uniform", ordered=False),
        # self-interaction of the (4096, 16, 32) node block: a row for each node and component, weights by species
        # and degree (4 x 4 groups), a training pass
        dict(name="grouped_nodes_f32", op="grouped", direction="train", dtype="f32", M=65536, K=32, N=32, G=16,
             sizes="uniform", ordered=False),
        # 32768 atoms over most of the periodic table with skewed populations, 256 channels
        dict(name="grouped_species_bf16", op="grouped", direction="train", dtype="bf16", M=32768, K=256, N=256, G=89,
             sizes="zipf", ordered=False),
        # the wide products of a mixture of experts, rows already in order: the matrix units' limit
        dict(name="grouped_wide_bf16", op="grouped", direction="train", dtype="bf16", M=32768, K=1024, N=4096, G=8,
             sizes="uniform", ordered=True),
        # odd sizes in each direction
        dict(name="grouped_odd_f16", op="grouped", direction="train", dtype="f16", M=9973, K=187, N=301, G=37,
             sizes="zipf", ordered=False),
        # the same 64 atoms through the norms, gate and residual
        dict(name="norm_tiny_f32", op="norm", direction="forward", dtype="f32", M=64, C=32, gate="full", kind="rms"),
        # 32768 atoms, 512 channels, one gate for each atom, a training pass
        dict(name="norm_atoms_bf16", op="norm", direction="train", dtype="bf16", M=32768, C=512, gate="row", kind="rms"),
        # edge features of the 647170-edge graph, 128 channels, a training pass in 32 bits
        dict(name="norm_edges_f32", op="norm", direction="train", dtype="f32", M=647170, C=128, gate="full",
             kind="layer"),
        # odd channel count
        dict(name="norm_odd_f16", op="norm", direction="train", dtype="f16", M=4097, C=1031, gate="full", kind="rms"),
        # a small model's parameters: two dozen short tensors
        dict(name="adamw_small_f32", op="adamw", count=24, total=20011, dtype="f32", bits=32),
        # a large model's parameters, 8-bit states
        dict(name="adamw_many_8bit", op="adamw", count=400, total=30000007, dtype="f32", bits=8),
        # a very large model's parameters in bf16, 32-bit states
        dict(name="adamw_large_bf16", op="adamw", count=60, total=200000033, dtype="bf16", bits=32),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case over the listed ranges: sizes spread over their logarithm, half of them made odd."""
    def size(lo, hi, multiple=8):
        n = _log_uniform(rng, lo, hi)
        return max(lo, n // multiple * multiple) if rng.random() < 0.5 else n | 1

    op = rng.choice(("grouped", "norm", "adamw"))
    if op == "grouped":
        while True:
            case = dict(op=op, direction=rng.choice(("forward", "train", "train")), dtype=rng.choice(("f32", "bf16", "f16")),
                        M=size(1, 300000), K=size(16, 2048), N=size(16, 4096), G=_log_uniform(rng, 1, 128),
                        sizes=rng.choice(("uniform", "zipf")), ordered=rng.random() < 0.3)
            # no more than the largest listed product, and no more memory than the plain form's padding can take
            padded = min(case["M"] * (16 if case["sizes"] == "zipf" else 2), case["M"] * case["G"]) + case["G"]
            if (case["M"] * case["K"] * case["N"] <= 32768 * 1024 * 4096 and padded * (case["K"] + case["N"]) <= 2 ** 30
                    and padded * case["K"] * case["N"] <= 2 ** 38
                    and case["G"] * case["K"] * case["N"] <= 2 ** 27):
                return case
    if op == "norm":
        while True:
            case = dict(op=op, direction=rng.choice(("forward", "train", "train")), dtype=rng.choice(("f32", "bf16", "f16")),
                        M=size(1, 650000), C=size(8, 8192), gate=rng.choice(("full", "row", "none")),
                        kind=rng.choice(("rms", "layer")))
            if case["M"] * case["C"] <= 647170 * 128:
                return case
    total = _log_uniform(rng, 2000, 200000000)
    return dict(op=op, count=_log_uniform(rng, 1, min(600, total // 64)), total=total | 1, dtype=rng.choice(("f32", "bf16")),
                bits=rng.choice((8, 32)))


def work(case):
    s = BYTES[case["dtype"]]
    if case["op"] == "grouped":
        M, K, N, G = case["M"], case["K"], case["N"], case["G"]
        order = 4 * (G + 1) + (0 if case["ordered"] else 4 * M)
        forward = s * (M * K + M * N + min(G, M) * N * K)
        if case["direction"] == "forward":
            return {"bytes": forward + order, "flops": 2 * M * N * K}
        return {"bytes": forward + order + s * (M * N + M * K + G * N * K), "flops": 6 * M * N * K}
    if case["op"] == "norm":
        M, C = case["M"], case["C"]
        gate = {"full": M * C, "row": M, "none": 0}[case["gate"]]
        if case["direction"] == "forward":
            return {"bytes": s * (4 * M * C + gate) + 12 * C, "flops": 20 * M * C}
        return {"bytes": s * (8 * M * C + 2 * gate) + 24 * C, "flops": 60 * M * C}
    n = case["total"]
    state = 4 * 4 * n if case["bits"] == 32 else 4 * n + 16 * -(-n // BLOCK)
    return {"bytes": 3 * s * n + state, "flops": 16 * n}


# ---------------------------------------------------------------- inputs

def _tensor_sizes(case):
    """Sizes of the tensors of an adamw case: three decades of them, their sum near the total."""
    rng = np.random.default_rng(case["count"] * 1000003 + case["total"])
    w = np.exp(rng.uniform(0.0, math.log(1000.0), case["count"]))
    n = np.maximum(1, np.floor(case["total"] * (w / w.sum()))).astype(np.int64)
    n[-1] += max(0, case["total"] - int(n.sum()))
    return [int(v) for v in n]


def _inputs(case, seed):
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape, dtype=dt, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale + shift).to(dtype)

    s = dict(case)
    if case["op"] == "grouped":
        M, K, N, G = case["M"], case["K"], case["N"], case["G"]
        if case["sizes"] == "zipf":   # skewed populations, about one group in twenty empty
            live = G - G // 20
            p = (np.arange(live) + 1.0) ** -1.1
            group = rng.permutation(G)[rng.choice(live, size=M, p=p / p.sum())]
        else:
            group = rng.integers(0, G, size=M)
        if case["ordered"]:
            group = np.sort(group)
        counts = np.bincount(group, minlength=G)
        s["row_ptr"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        s["perm"] = None if case["ordered"] else torch.from_numpy(np.argsort(group, kind="stable").astype(np.int32)).cuda()
        s["largest"] = int(counts.max())   # rows of the largest group, which a program that grouped them knows
        s["x"] = normal(M, K)
        s["w"] = normal(G, N, K, scale=K ** -0.5)
        s["dy"] = normal(M, N) if case["direction"] == "train" else None
    elif case["op"] == "norm":
        M, C = case["M"], case["C"]
        s["h"], s["x"] = normal(M, C), normal(M, C, scale=2.0, shift=0.1)
        s["gate"] = None if case["gate"] == "none" else normal(M, 1 if case["gate"] == "row" else C)
        f32 = dict(dtype=torch.float32)
        s["w_post"], s["scale"], s["w_pre"] = (normal(C, scale=0.1, shift=1.0, **f32), normal(C, scale=0.3, **f32),
                                               normal(C, scale=0.1, shift=1.0, **f32))
        if case["direction"] == "train":
            s["dy"], s["du"] = normal(M, C), normal(M, C)
    else:
        # every tensor is a view of one buffer, each at a multiple of 256 elements
        sizes = _tensor_sizes(case)
        blocks = [-(-n // BLOCK) for n in sizes]
        total = sum(blocks) * BLOCK
        live = torch.zeros(total, dtype=torch.bool, device="cuda")
        _views(live, sizes, lambda v: v.fill_(True))
        s["sizes"], s["step"] = sizes, 100

        def buffer(scale, dtype, shift=0.0):
            return torch.where(live, torch.randn(total, generator=gen, device="cuda") * scale + shift, 0.0).to(dtype)

        s["p"], s["g"] = buffer(0.02, dt), buffer(0.01, dt)
        m, r = buffer(0.003, torch.float32), buffer(0.01, torch.float32).abs()
        if case["bits"] == 8:
            s["m"], s["m_scale"] = _to_e4m3(m, False)
            s["v"], s["v_scale"] = _to_e4m3(r, True)
        else:
            s["m"], s["v"] = m, r * r
        s["grad_scale"] = torch.full((1,), 0.5, device="cuda")
    return s


def _views(flat, sizes, then=lambda v: v):
    starts = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in sizes])])
    return [then(flat[int(a):int(a) + n]) for a, n in zip(starts, sizes)]


def prepare(case, seed):
    """The operands on the GPU, and for the kernels of adamw the plan that holds its tensors."""
    s = _inputs(case, seed)
    if case["op"] == "adamw" and own:
        views = [_views(s[k], s["sizes"]) for k in ("p", "g", "m", "v")]
        scales = (None, None)
        if case["bits"] == 8:
            per = [-(-n // BLOCK) for n in s["sizes"]]
            scales = tuple(list(torch.split(s[k], per)) for k in ("m_scale", "v_scale"))
        s["plan"] = _zs().AdamWPlan(*views, *scales)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if s["op"] == "grouped":
        return _own_grouped(s) if own else _plain_grouped(s)
    if s["op"] == "norm":
        return _own_norm(s) if own else _plain_norm(s)
    s["step"] += 1
    if own:
        _zs().zs_adamw_step(s["plan"], s["step"], lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY,
                            grad_scale=s["grad_scale"])
    else:
        _plain_adamw(s)
    return {k: s[k] for k in ("p", "m", "v", "m_scale", "v_scale") if k in s}


def _own_grouped(s):
    zs = _zs()
    out = {"y": zs.zs_grouped_matmul(s["x"], s["w"], s["row_ptr"], s["perm"])}
    if s["direction"] == "train":
        out["dx"], out["dw"] = zs.zs_grouped_matmul_backward(s["dy"], s["x"], s["w"], s["row_ptr"], s["perm"])
    return out


def _own_norm(s):
    zs = _zs()
    operands = (s["h"], s["x"], s["gate"], s["w_post"], s["scale"], s["w_pre"])
    y, u, stats = zs.zs_norm_gate_residual(*operands, eps=NORM_EPS, kind=s["kind"])
    out = {"y": y, "u": u}
    if s["direction"] == "train":
        grads = zs.zs_norm_gate_residual_backward(s["dy"], s["du"], *operands, stats, kind=s["kind"])
        out |= zip(("dh", "dx", "dgate", "dw_post", "dscale", "dw_pre"), grads)
    return out


def _plain_grouped(s):
    """The groups padded to the largest one, then batched products."""
    M, G, dt = s["M"], s["G"], s["x"].dtype
    at = torch.arange(M, dtype=torch.int32, device="cuda")
    group = torch.searchsorted(s["row_ptr"], at, right=True) - 1
    slot = at - s["row_ptr"][group]
    order = at if s["perm"] is None else s["perm"]
    wf = s["w"].float()

    def padded(rows):
        p = torch.zeros(G, s["largest"], rows.shape[1], device="cuda")
        p[group, slot] = rows.float()[order]
        return p

    def back(p):
        rows = torch.empty(M, p.shape[2], device="cuda")
        rows[order] = p[group, slot]
        return rows.to(dt)

    xp = padded(s["x"])
    out = {"y": back(torch.bmm(xp, wf.transpose(1, 2)))}
    if s["direction"] == "train":
        dyp = padded(s["dy"])
        out["dx"] = back(torch.bmm(dyp, wf))
        out["dw"] = torch.bmm(dyp.transpose(1, 2), xp).to(dt)
    return out


def _normalised(v, kind):
    """The rows of v without their mean (layer) over the root of their mean square, and one over that root."""
    c = v - v.mean(1, keepdim=True) if kind == "layer" else v
    r = torch.rsqrt((c * c).mean(1, keepdim=True) + NORM_EPS)
    return c * r, r


def _normalised_gradient(dn, n, r, kind):
    d = dn - n * (dn * n).mean(1, keepdim=True)
    return r * (d - dn.mean(1, keepdim=True) if kind == "layer" else d)


def _plain_norm(s):
    dt, kind = s["h"].dtype, s["kind"]
    h, x = s["h"].float(), s["x"].float()
    nh, rh = _normalised(h, kind)
    t = nh * s["w_post"]
    q = 1.0 if s["gate"] is None else 1.0 / (1.0 + torch.exp(-s["gate"].float()))
    y = x + s["scale"] * q * t
    ny, ry = _normalised(y, kind)
    out = {"y": y.to(dt), "u": (ny * s["w_pre"]).to(dt)}
    if s["direction"] == "train":
        du = s["du"].float()
        dx = s["dy"].float() + _normalised_gradient(du * s["w_pre"], ny, ry, kind)
        dt_ = dx * s["scale"] * q
        out["dh"] = _normalised_gradient(dt_ * s["w_post"], nh, rh, kind).to(dt)
        out["dx"] = dx.to(dt)
        if s["gate"] is not None:
            dz = dx * s["scale"] * t * (q * (1.0 - q))
            out["dgate"] = (dz.sum(1, keepdim=True) if s["gate"].shape[1] != dz.shape[1] else dz).to(dt)
        out["dw_post"] = (dt_ * nh).sum(0)
        out["dscale"] = (dx * q * t).sum(0)
        out["dw_pre"] = (du * ny).sum(0)
    return out


def _to_e4m3(values, root):
    """(codes, scales) of blocks of 256: a scale of the largest finite magnitude over 448; a root above zero is never held as zero."""
    b = values.view(-1, BLOCK)
    finite = torch.isfinite(b)
    top = torch.where(finite, b.abs(), 0.0).amax(1, keepdim=True)
    live = top >= SCALE_MIN
    scale = torch.where(live, top * (1.0 / E4M3_MAX), 0.0)
    q = b * torch.where(live, E4M3_MAX / top, 0.0)
    if root:
        q = torch.where((b > 0) & live, torch.clamp_min(q, E4M3_TINY), q)
    q = torch.where(finite, torch.clamp(q, -E4M3_MAX, E4M3_MAX), math.nan)
    return q.to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def _from_e4m3(codes, scales):
    return (codes.float().view(-1, BLOCK) * scales.view(-1, 1)).view(-1)


def _plain_adamw(s):
    t, eight = s["step"], "m_scale" in s
    g = s["g"].float() * s["grad_scale"]
    p = s["p"].float()
    if eight:
        m = _from_e4m3(s["m"], s["m_scale"])
        r = _from_e4m3(s["v"], s["v_scale"])
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * (g * g)
    r = torch.sqrt(v)
    denom = r * (1.0 / math.sqrt(1.0 - BETA2 ** t)) + ADAM_EPS
    p = p * (1.0 - LR * DECAY) - (LR / (1.0 - BETA1 ** t)) * (m / denom)
    s["p"].copy_(p)
    if eight:
        for key, value, root in (("m", m, False), ("v", r, True)):
            codes, scales = _to_e4m3(value, root)
            s[key].copy_(codes)
            s[key + "_scale"].copy_(scales)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "grouped":
        M, K, N = case["M"], case["K"], case["N"]
        if 6 * M * K * N > 4e12:
            return None   # 64-bit products take too long
        bounds = s["row_ptr"].tolist()
        order = torch.arange(M, device="cuda") if s["perm"] is None else s["perm"].long()
        wd, xd = s["w"].double(), s["x"].double()
        y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        train = case["direction"] == "train"
        if train:
            dyd = s["dy"].double()
            dx, dw = torch.zeros_like(xd), torch.zeros_like(wd)
        for g in range(case["G"]):
            rows = order[bounds[g]:bounds[g + 1]]
            y[rows] = xd[rows] @ wd[g].T
            if train:
                dx[rows] = dyd[rows] @ wd[g]
                dw[g] = dyd[rows].T @ xd[rows]
        return {"y": y, "dx": dx, "dw": dw} if train else {"y": y}
    if case["op"] == "norm":
        names = [k for k in ("h", "x", "gate", "w_post", "scale", "w_pre") if s[k] is not None]
        d = {k: s[k].double().requires_grad_(case["direction"] == "train") for k in names}

        def norm(v):
            if case["kind"] == "layer":
                return (v - v.mean(1, keepdim=True)) / torch.sqrt(v.var(1, unbiased=False, keepdim=True) + NORM_EPS)
            return v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + NORM_EPS)

        gate = torch.sigmoid(d["gate"]) if "gate" in d else 1.0
        y = d["x"] + d["scale"] * gate * (norm(d["h"]) * d["w_post"])
        u = norm(y) * d["w_pre"]
        out = {"y": y.detach(), "u": u.detach()}
        if case["direction"] == "train":
            grads = torch.autograd.grad((y, u), [d[k] for k in names], (s["dy"].double(), s["du"].double()))
            out |= {"d" + k: v for k, v in zip(names, grads)}
        return out
    # one step from the prepared states; what is held in 8 bits as the value it rounds
    def blocks(v):
        return v.double().view(-1, BLOCK)

    t = s["step"] + 1
    g = blocks(s["g"]) * s["grad_scale"].double()
    m, v = blocks(s["m"]), blocks(s["v"])
    if case["bits"] == 8:
        m = m * s["m_scale"].double()[:, None]
        v = (v * s["v_scale"].double()[:, None]) ** 2
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    update = (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS)
    p = (1 - LR * DECAY) * blocks(s["p"]) - LR * update
    out = {"p": p.view(-1)}
    if case["bits"] == 32:
        return out | {"m": m.view(-1), "v": v.view(-1)}
    for key, value in (("m", m), ("v", v.sqrt())):
        out[key + "_scale"] = value.abs().amax(1) / E4M3_MAX
        out[key] = (value / out[key + "_scale"][:, None].clamp_min(1e-300)).view(-1)
    return out
