"""Cases for the node-level operators of a training step: the type embedding and
its gradient, the norms around a layer with its gate and residual, and the
global gradient norm with clipping.

Each case is prepared on the GPU from a seed and run either in its plain form
(elementary torch operations in 32 bits, one rounding at the end) or through
the library's operators (``own``)."""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2, "int32": 4, "int64": 8}


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # one token at a time through a large table: what a single step of generation or of an MD query looks up
        dict(name="embed token", op="embed", N=1, V=32000, C=2048, table="bf16", out="bf16", ids="int64", scale=45.25),
        # the first features of a large graph: element types of 32768 nodes, 128 channels
        dict(name="embed nodes", op="embed", N=32768, V=118, C=128, table="fp32", out="fp32", ids="int32", scale=1.0),
        # gradient of a two-species table on the water box's 1503 atoms: every row is shared by hundreds of nodes
        dict(name="embed grad water box", op="embed_grad", N=1503, V=2, C=128, table="fp32", out="fp32", ids="int32",
             scale=1.0, skew=0.0, padding=-1),
        # gradient of an element table over a large batch of graphs (padded: type 0 is the filler)
        dict(name="embed grad nodes", op="embed_grad", N=500009, V=95, C=128, table="fp32", out="fp32", ids="int32",
             scale=1.0, skew=1.0, padding=0),
        # gradient of a large table, token frequencies falling like 1 / rank, 16-bit activations, fp32 weights
        dict(name="embed grad tokens", op="embed_grad", N=16384, V=65536, C=2048, table="fp32", out="bf16",
             ids="int64", scale=45.25, skew=1.0, padding=-1),
        # one row through a norm, its gate and residual: a single step of inference
        dict(name="norm row", op="norm", N=1, L=0, C=1024, dtype="bf16", gate="sigmoid", post=True, pre=True,
             train=False, scale=1.0),
        # one layer boundary of the water box at lmax 3, forward and backward
        dict(name="norm water box", op="norm", N=1503, L=3, C=128, dtype="fp32", gate="sigmoid", post=True, pre=True,
             train=True, scale=0.5),
        # one layer boundary of the lmax 2 workload (32768 nodes, 128 channels), forward and backward
        dict(name="norm lmax2", op="norm", N=32768, L=2, C=128, dtype="fp32", gate="silu", post=True, pre=True,
             train=True, scale=0.7),
        # wide invariant rows in 16 bits, an odd number of them, forward and backward
        dict(name="norm wide rows", op="norm", N=8191, L=0, C=4096, dtype="bf16", gate="tanh", post=True, pre=True,
             train=True, scale=1.0),
        # the weight gradients of a small lmax 3 model (radial MLPs, contraction weights, norms, table), clipped
        dict(name="clip model", op="clip", kind="model", n=2, dtype="fp32", clipped=True),
        # an ordinary step whose norm stays below the bound: odd-sized 32-bit gradients, in place
        dict(name="clip quiet step", op="clip", kind="ragged", n=20000003, dtype="fp32", clipped=False),
        # the largest: 512 MiB of 16-bit gradients with some 32-bit ones among them, clipped
        dict(name="clip large", op="clip", kind="mixed", n=268435456, dtype="bf16", clipped=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm", "clip"])
    if op == "embed":
        C = _log(rng, 4, 8192)
        table = rng.choice(["fp32", "bf16", "fp16"])
        return dict(op=op, N=_log(rng, 1, min(65536, 1 + 60_000_000 // C)), V=_log(rng, 1, min(131072, 130_000_000 // C)),
                    C=C, table=table, out=rng.choice([table, "bf16", "fp16"]) if table == "fp32" else table,
                    ids=rng.choice(["int32", "int64"]), scale=round(rng.uniform(0.1, 60.0), 3))
    if op == "embed_grad":
        C = _log(rng, 4, 4096)
        V = _log(rng, 1, min(131072, 130_000_000 // C))
        table = rng.choice(["fp32", "bf16", "fp16"])
        return dict(op=op, N=_log(rng, 1, min(500000, 1 + 60_000_000 // C)), V=V, C=C, table=table,
                    out=rng.choice([table, "bf16", "fp16"]) if table == "fp32" else table,
                    ids=rng.choice(["int32", "int64"]), scale=round(rng.uniform(0.1, 60.0), 3),
                    skew=rng.choice([0.0, 0.7, 1.0]), padding=rng.choice([-1, 0]) if V > 1 else -1)
    if op == "norm":
        L = rng.choice([0, 0, 1, 2, 3])
        C = _log(rng, 4, 8192 if L == 0 else 512)
        post = rng.random() < 0.85
        return dict(op=op, N=_log(rng, 1, min(40000, 1 + 26_000_000 // (C * (L + 1) ** 2))), L=L, C=C,
                    dtype=rng.choice(["fp32", "bf16", "fp16"]), gate=rng.choice(["none", "sigmoid", "silu", "tanh"]),
                    post=post, pre=not post or rng.random() < 0.8, train=rng.random() < 0.7,
                    scale=round(rng.uniform(0.1, 1.0), 3))
    kind = rng.choice(["model", "ragged", "mixed"])
    return dict(op="clip", kind=kind, n=rng.randrange(1, 4) if kind == "model" else _log(rng, 1000, 130_000_000),
                dtype="fp32" if kind == "model" else rng.choice(["fp32", "bf16", "fp16"]), clipped=rng.random() < 0.7)


# --------------------------------------------------------------- their inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ids(case, g):
    """Token ids: uniform, or with frequencies falling like rank^-skew over a shuffled table."""
    N, V, skew = case["N"], case["V"], case.get("skew", 0.0)
    if skew > 0:
        cum = torch.arange(1, V + 1, device="cuda", dtype=torch.float64).pow(-skew).cumsum(0)
        u = torch.rand(N, device="cuda", dtype=torch.float64, generator=g) * cum[-1]
        ids = torch.searchsorted(cum, u).clamp_(max=V - 1)
        ids = torch.randperm(V, device="cuda", generator=g)[ids]
    else:
        ids = torch.randint(0, V, (N,), device="cuda", generator=g)
    if case.get("padding", -1) >= 0 and N > 8:
        ids[-(N // 8):] = case["padding"]      # the filler behind the last sequence or graph
    return ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)


def _clip_sizes(case):
    if case["kind"] == "model":
        # per layer: radial MLP 8 -> 64 -> 64 -> 23 paths x 128, contraction weights of 4 species, norm weights
        layer = [(8, 64), (64, 64), (64, 23 * 128), (4, 4, 128), (4, 16, 128), (4, 128), (4, 128)]
        shapes = [(95, 128)] + layer * case["n"] + [(128,), (1,)]
        return [math.prod(s) for s in shapes]
    n, parts = case["n"], 23 if case["kind"] == "ragged" else 40
    w = [1 + (7 * i * i + 3 * i) % 61 for i in range(parts)]
    sizes = [max(1, n * k // sum(w)) for k in w]
    return [s | 1 for s in sizes] if case["kind"] == "ragged" else sizes


def _clip_types(case):
    sizes = _clip_sizes(case)
    if case["kind"] != "mixed":
        return [case["dtype"]] * len(sizes)
    return ["fp32" if i % 13 == 5 else case["dtype"] for i in range(len(sizes))]


def prepare(case, seed):
    g = _gen(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    if case["op"] in ("embed", "embed_grad"):
        T, O = TYPES[case["table"]], TYPES[case["out"]]
        st = dict(case=case, ids=_ids(case, g))
        if case["op"] == "embed":
            st["table"] = (randn(case["V"], case["C"]) * case["C"] ** -0.5).to(T)
        else:
            st["gy"] = (randn(case["N"], case["C"]) * 0.02).to(O)
        return st
    if case["op"] == "norm":
        N, L, C, T = case["N"], case["L"], case["C"], TYPES[case["dtype"]]
        D = (L + 1) ** 2
        # channels of unequal size, nodes of unequal size, as after a few layers
        size = torch.exp(0.5 * randn(N, 1, 1)) * torch.exp(0.5 * randn(C))
        make = lambda: (randn(N, D, C) * size).to(T)  # noqa: E731
        st = dict(case=case, deg=torch.tensor([math.isqrt(i) for i in range(D)], device="cuda"), x=make(),
                  b=make() if case["post"] else None,
                  gate=randn(N, L + 1, C).to(T) if case["post"] and case["gate"] != "none" else None,
                  w_post=1.0 + 0.2 * randn(L + 1, C) if case["post"] else None,
                  w_pre=1.0 + 0.2 * randn(L + 1, C) if case["pre"] else None, gx=None, gh=None)
        if case["train"]:
            st["gx"] = randn(N, D, C).to(T) if case["post"] else None
            st["gh"] = randn(N, D, C).to(T) if case["pre"] else None
        return st
    sizes, types = _clip_sizes(case), _clip_types(case)
    grads = [(torch.randn(n, device="cuda", generator=g) * (0.01 * (1 + i % 5))).to(TYPES[t])
             for i, (n, t) in enumerate(zip(sizes, types))]
    # the size that such gradients have is about 0.033 sqrt(n); a tenth of it clips, ten times it does not
    bound = 0.033 * math.sqrt(sum(sizes)) * (0.1 if case["clipped"] else 10.0)
    return dict(case=case, grads=grads, bound=bound, out=[torch.empty_like(v) for v in grads] if case["clipped"] else grads)


# ----------------------------------------------------------------- plain forms

def _act(kind, g):
    """The gate a(g) and a'(g)."""
    if kind == "sigmoid":
        a = 1.0 / (1.0 + torch.exp(-g))
        return a, a * (1.0 - a)
    if kind == "silu":
        a = 1.0 / (1.0 + torch.exp(-g))
        return g * a, a * (1.0 + g * (1.0 - a))
    a = torch.tanh(g)
    return a, 1.0 - a * a


def _per_degree(rows, deg, L):
    """Sums over a degree's rows: [N, D, ...] -> [N, L + 1, ...]."""
    if L == 0:
        return rows
    return torch.zeros((rows.shape[0], L + 1) + rows.shape[2:], device=rows.device).index_add_(1, deg, rows)


def _plain_norm(st):
    c, deg, L, eps = st["case"], st["deg"], st["case"]["L"], 1e-6
    T, count = st["x"].dtype, (2.0 * torch.arange(st["case"]["L"] + 1, device="cuda") + 1.0) * st["case"]["C"]
    mean = lambda v: _per_degree(v.sum(-1), deg, L) / count  # noqa: E731
    x, out = st["x"].float(), {}
    y = x
    if c["post"]:
        b = st["b"].float()
        sb = torch.rsqrt(mean(b * b) + eps)[:, deg, None]
        bn = b * sb
        u = bn * st["w_post"][deg]
        a, da = _act(c["gate"], st["gate"].float()) if st["gate"] is not None else (None, None)
        t = u * c["scale"] if a is None else u * c["scale"] * a[:, deg]
        y = x + t
        out["x"] = y.to(T)
    if c["pre"]:
        sy = torch.rsqrt(mean(y * y) + eps)[:, deg, None]
        yn = y * sy
        out["h"] = (yn * st["w_pre"][deg]).to(T)
    if not c["train"]:
        return out
    gy = st["gx"].float() if st["gx"] is not None else 0.0
    if c["pre"]:
        gh = st["gh"].float()
        out["dw_pre"] = _per_degree((gh * yn).sum(0, keepdim=True), deg, L)[0]
        p = gh * st["w_pre"][deg]
        gy = gy + sy * (p - yn * mean(p * yn)[:, deg, None])
    out["dx"] = gy.to(T)
    if c["post"]:
        if a is not None:
            out["dgate"] = (_per_degree(gy * u, deg, L) * da * c["scale"]).to(T)
        q = gy * c["scale"] if a is None else gy * c["scale"] * a[:, deg]
        out["dw_post"] = _per_degree((q * bn).sum(0, keepdim=True), deg, L)[0]
        q = q * st["w_post"][deg]
        out["db"] = (sb * (q - bn * mean(q * bn)[:, deg, None])).to(T)
    return out


def _plain(st):
    c = st["case"]
    if c["op"] == "embed":
        return (st["table"][st["ids"]].float() * c["scale"]).to(TYPES[c["out"]])
    if c["op"] == "embed_grad":
        wide = torch.float64 if c["N"] > 16384 else torch.float32     # sums of many thousand terms lose digits in 32 bits
        d = torch.zeros(c["V"], c["C"], device="cuda", dtype=wide).index_add_(0, st["ids"], st["gy"].to(wide))
        if c["padding"] >= 0:
            d[c["padding"]] = 0.0
        return (d * c["scale"]).to(TYPES[c["table"]])
    if c["op"] == "norm":
        return _plain_norm(st)
    norm = torch.stack([v.float().square().sum() for v in st["grads"]]).sum().sqrt()
    k = (st["bound"] / (norm + 1e-6)).clamp(max=1.0)
    return dict(norm=norm, grads=[o.copy_(v.float() * k) for o, v in zip(st["out"], st["grads"])])


# ------------------------------------------------------- the library's operators

_ops = {}


def _op(c):
    """The operator's handle, held for all batches, as a model holds its layers."""
    from equivariant_gnn_message_edge_b200 import layers
    key = tuple(sorted((k, v) for k, v in c.items() if k not in ("name", "N", "skew", "scale", "train", "ids")))
    if key not in _ops:
        if c["op"] == "norm":
            irreps = "+".join(["0e", "1o", "2e", "3o"][:c["L"] + 1])
            _ops[key] = layers.BlockNorm(irreps, c["C"], gate=c["gate"], eps=1e-6, dtype=TYPES[c["dtype"]])
        else:
            padding = c.get("padding", -1)
            _ops[key] = layers.Embedding(c["V"], c["C"], dtype=TYPES[c["table"]], out_dtype=TYPES[c["out"]],
                                         padding=padding if padding >= 0 else None)
    return _ops[key]


def _own(st):
    c = st["case"]
    if c["op"] != "clip" and "handle" not in st:
        st["handle"] = _op(c)          # found once: a program holds its layer and does not look it up at every call
    if c["op"] == "embed":
        return st["handle"].forward_raw(st["ids"], st["table"], c["scale"])
    if c["op"] == "embed_grad":
        return st["handle"].backward_raw(st["ids"], st["gy"], c["scale"])
    if c["op"] == "clip":
        from equivariant_gnn_message_edge_b200 import layers
        norm = layers.clip_gradients(st["grads"], st["bound"], out=st["out"])
        return dict(norm=norm, grads=st["out"])
    op = st["handle"]
    args = st["x"], st["b"], st["gate"], st["w_post"], st["w_pre"]
    x, h, stats = op.forward_raw(*args, scale=c["scale"], save=c["train"])
    out = dict(x=x) if c["post"] else {}
    if c["pre"]:
        out["h"] = h
    if c["train"]:
        dx, db, dgate, dw_post, dw_pre = op.backward_raw(*args, stats, st["gx"], st["gh"], scale=c["scale"])
        got = dict(dx=dx, db=db, dgate=dgate, dw_post=dw_post, dw_pre=dw_pre)
        out.update((k, v) for k, v in got.items() if v is not None)
    return out


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------ their work

def work(case):
    c = case
    if c["op"] == "embed":
        n = c["N"] * c["C"]
        rows = min(c["N"], c["V"]) * c["C"] * BYTES[c["table"]]
        return dict(bytes=n * BYTES[c["out"]] + rows + c["N"] * BYTES[c["ids"]], flops=n)
    if c["op"] == "embed_grad":
        n = c["N"] * c["C"]
        return dict(bytes=n * BYTES[c["out"]] + c["V"] * c["C"] * BYTES[c["table"]] + c["N"] * BYTES[c["ids"]], flops=2 * n)
    if c["op"] == "norm":
        n, g = c["N"] * (c["L"] + 1) ** 2 * c["C"], c["N"] * (c["L"] + 1) * c["C"]
        w = (c["L"] + 1) * c["C"] * 4
        gated = c["post"] and c["gate"] != "none"
        arrays = 1 + 2 * c["post"] + c["pre"] + c["train"] * (1 + 2 * c["post"] + c["pre"])
        small = gated * (1 + c["train"])
        weights = w * (c["post"] + c["pre"]) * (1 + c["train"])
        return dict(bytes=(arrays * n + small * g) * BYTES[c["dtype"]] + weights, flops=(12 + 30 * c["train"]) * n)
    each = [(n, BYTES[t]) for n, t in zip(_clip_sizes(c), _clip_types(c))]
    return dict(bytes=(2 if c["clipped"] else 1) * sum(n * b for n, b in each) + 4, flops=(3 if c["clipped"] else 2) * sum(n for n, _ in each))


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    st, c = prepare(case, seed), case
    f64 = lambda v: None if v is None else v.double()  # noqa: E731
    if c["op"] == "embed":
        return torch.nn.functional.embedding(st["ids"].long(), st["table"].double()) * c["scale"]
    if c["op"] == "embed_grad":
        ids, order = torch.sort(st["ids"].long(), stable=True)
        starts = torch.searchsorted(ids, torch.arange(c["V"] + 1, device="cuda"))
        d = torch.empty(c["V"], c["C"], device="cuda", dtype=torch.float64)
        for at in range(0, c["C"], 256):     # segment sums as differences of a running sum
            run_ = torch.zeros(c["N"] + 1, min(256, c["C"] - at), device="cuda", dtype=torch.float64)
            torch.cumsum(st["gy"][:, at:at + 256].double()[order], 0, out=run_[1:])
            d[:, at:at + 256] = run_[starts[1:]] - run_[starts[:-1]]
        if c["padding"] >= 0:
            d[c["padding"]] = 0.0
        return d * c["scale"]
    if c["op"] == "clip":
        if sum(_clip_sizes(c)) > 300_000_000:
            return None
        total = math.sqrt(math.fsum(float((v.double() ** 2).sum()) for v in st["grads"]))
        k = min(1.0, st["bound"] / (total + 1e-6))
        return dict(norm=total, grads=[v.double() * k for v in st["grads"]])
    # the definition degree by degree, its gradients by differentiating it
    N, L, C = c["N"], c["L"], c["C"]
    x, b, gate, wo, wi = (f64(st[k]) for k in ("x", "b", "gate", "w_post", "w_pre"))
    leaves = [v.requires_grad_(c["train"]) if v is not None else None for v in (x, b, gate, wo, wi)]
    act = {"none": None, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu, "tanh": torch.tanh}[c["gate"]]
    norm = lambda v: v / torch.sqrt((v ** 2).mean(dim=(1, 2), keepdim=True) + 1e-6)  # noqa: E731
    ys, hs = [], []
    for l in range(L + 1):
        block = slice(l * l, (l + 1) ** 2)
        y = x[:, block]
        if c["post"]:
            u = norm(b[:, block]) * wo[l]
            y = y + c["scale"] * (u if act is None else u * act(gate[:, l:l + 1]))
        ys.append(y)
        if c["pre"]:
            hs.append(norm(y) * wi[l])
    y, h = torch.cat(ys, 1), torch.cat(hs, 1) if hs else None
    out = dict(x=y.detach()) if c["post"] else {}
    if h is not None:
        out["h"] = h.detach()
    if c["train"]:
        total = 0.0
        if c["post"]:
            total = total + (y * f64(st["gx"])).sum()
        if c["pre"]:
            total = total + (h * f64(st["gh"])).sum()
        names = [n for n, v in zip(("dx", "db", "dgate", "dw_post", "dw_pre"), leaves) if v is not None]
        out.update(zip(names, torch.autograd.grad(total, [v for v in leaves if v is not None])))
    return out
