"""The node-level operators around a convolution on the GPU against the fp64
oracle (needs a B200): embedding and its gradient, block norm and its
gradients, gradient norm and clipping; and a run of them with the convolution.

Tolerances.  A value rounded once to type t is off by at most
finfo(t).eps / 2 relative to itself; HALF counts that.  What comes before it is
fp32 (or wider) arithmetic, whose error is bounded by its longest chain of
operations: a sum of n terms by warps and threads is off by less than
n 2^-24 sum |terms| (any order), and in practice by far less."""
import threading

import numpy as np
import pytest
import torch

from equivariant_gnn_message_edge_b200 import binding as B
from equivariant_gnn_message_edge_b200 import layers
from equivariant_gnn_message_edge_b200.workloads import natural_irreps
from oracle import layers as ol

pytestmark = pytest.mark.gpu

T = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24                                    # half a step of fp32


def half(dtype):
    return torch.finfo(dtype).eps / 2


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def randn(g, *shape, dtype=torch.float32, mul=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * mul).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def assert_within(name, got, want, tol):
    """|got - want| <= tol elementwise (tol: array or number)."""
    got = np64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(np.max(np.abs(got - want) - tol)))


# ------------------------------------------------------------------ embedding

EMBED = [  # N, V, C, table, out, ids
    (1, 1, 1, "fp32", "fp32", "int32"),
    (1, 50, 2048, "bf16", "bf16", "int64"),
    (7, 3, 5, "fp32", "bf16", "int32"),
    (333, 118, 128, "fp32", "fp32", "int32"),
    (1500, 2, 132, "fp32", "fp16", "int64"),
    (2050, 4000, 66, "fp16", "fp16", "int64"),
    (4097, 95, 36, "bf16", "bf16", "int32"),
    (70001, 9, 8, "fp32", "fp32", "int32"),
    (20000, 70000, 12, "fp32", "bf16", "int64"),
    (257, 33, 1030, "bf16", "bf16", "int64"),
    (30, 5, 20000, "fp32", "fp32", "int32"),
    (4096, 296, 32, "fp32", "fp32", "int64"),          # the largest of the one-launch gradient, and just over
    (4096, 297, 32, "fp16", "fp16", "int32"),
    (65536, 40, 4, "fp32", "fp32", "int64"),           # the largest one-cluster sort, and just over
    (65537, 600, 4, "bf16", "bf16", "int32"),
    (16384, 600, 8, "fp32", "bf16", "int64"),          # the same for two passes
    (16385, 70000, 8, "fp32", "fp32", "int32"),
    (30000, 3000, 36, "fp32", "fp32", "int64"),        # types of about a tile
    (9000, 40, 520, "fp16", "fp16", "int32"),          # types of many tiles, several slabs
]


def _embed_case(N, V, C, table, out, ids, seed=0, skew=False):
    g = gen(seed)
    z = torch.randint(0, V, (N,), device="cuda", generator=g)
    if skew:
        z = torch.minimum(z, torch.randint(0, V, (N,), device="cuda", generator=g) // 7)
    z = z.to(torch.int32 if ids == "int32" else torch.int64)
    return z, randn(g, V, C, dtype=T[table]), randn(g, N, C, dtype=T[out])


def _grad_tol(z, gy, V, scale, dtype, padding=None):
    """n 2^-24 sum |gy| over a type's nodes for the fp32 sum, one rounding more
    for the scale, and half a step of the output's type."""
    mag = ol.embedding_grad(np64(z), np.abs(np64(gy)), V, abs(scale), padding)
    n = np.bincount(np.clip(np64(z).astype(np.int64), 0, V - 1), minlength=V)[:, None] + 2
    want = ol.embedding_grad(np64(z), np64(gy), V, scale, padding)
    return want, n * U * mag + half(dtype) * np.abs(want) * (1 + 1e-3) + tiny(dtype)


def tiny(dtype):
    """Half the spacing of the type's subnormal numbers."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2 * (1 + 1e-6)


@pytest.mark.parametrize("case", EMBED, ids=str)
def test_embedding_forward(case):
    z, table, _ = _embed_case(*case)
    op = layers.Embedding(case[1], case[2], T[case[3]], T[case[4]])
    for scale in (1.0, 1.7):
        y = op.forward_raw(z, table, scale)
        assert y.dtype == T[case[4]]
        want = ol.embedding(np64(z), np64(table), np.float32(scale))
        # the product is rounded to fp32, then to the type
        assert_within("y", y, want, (U + half(y.dtype)) * np.abs(want) * (1 + 1e-3) + tiny(y.dtype))
    assert B.eqconv_get_device_error(op.plan) == B.EQCONV_OK


@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("case", EMBED, ids=str)
def test_embedding_gradient(case, skew):
    z, table, gy = _embed_case(*case, seed=3, skew=skew)
    V, C = case[1], case[2]
    op = layers.Embedding(V, C, T[case[3]], T[case[4]])
    d = op.backward_raw(z, gy, 0.5)
    want, tol = _grad_tol(z, gy, V, 0.5, d.dtype)
    assert_within("dtable", d, want, tol)
    assert torch.equal(d, op.backward_raw(z, gy, 0.5))                       # bitwise reproducible
    if V > 2:
        op = layers.Embedding(V, C, T[case[3]], T[case[4]], padding=1)
        d = op.backward_raw(z, gy, 0.5)
        want, tol = _grad_tol(z, gy, V, 0.5, d.dtype, padding=1)
        assert_within("dtable", d, want, tol)
        assert not d[1].any()


def test_embedding_one_type_owns_every_node():
    """One row of the table gets all nodes (exact sums: small whole numbers), others none."""
    N, V, C = 100003, 300, 8
    g = gen(5)
    gy = torch.randint(-3, 4, (N, C), device="cuda", generator=g).float()
    for v in (0, 137, 299):
        z = torch.full((N,), v, dtype=torch.int64, device="cuda")
        d = layers.Embedding(V, C).backward_raw(z, gy)
        want = torch.zeros(V, C, device="cuda")
        want[v] = gy.double().sum(0).float()
        assert torch.equal(d, want)


@pytest.mark.parametrize("N", [1, 31, 32, 33, 64, 1000, 2047, 2048, 2049, 8191, 8192, 8193, 40000])
def test_embedding_gradient_counts(N):
    """Every node counted once at sizes around the tiles' ends (exact: ones)."""
    V, C = 37, 4
    z = torch.randint(0, V, (N,), device="cuda", generator=gen(N))
    d = layers.Embedding(V, C).backward_raw(z, torch.ones(N, C, device="cuda"))
    assert torch.equal(d, torch.bincount(z, minlength=V).float()[:, None].expand(V, C))


@pytest.mark.parametrize("V", [1, 2, 255, 256, 257, 2047, 2048, 2049, 65535, 65536, 65537, 300000, 5000000])
def test_embedding_gradient_tables(V):
    """Every row written, the empty ones with zeros, at table sizes around the sort's digits."""
    N, C = 5000, 4
    g = gen(V)
    z = torch.randint(0, V, (N,), device="cuda", generator=g)
    z[:3] = torch.tensor([0, V - 1, V // 2], device="cuda")
    gy = torch.randint(-4, 5, (N, C), device="cuda", generator=g).float()
    out = torch.full((V, C), float("nan"), device="cuda")
    d = layers.Embedding(V, C).backward_raw(z, gy, out=out)
    assert torch.equal(d, torch.zeros(V, C, device="cuda").index_add_(0, z, gy))


@pytest.mark.parametrize("N", [16385, 40000])
@pytest.mark.parametrize("V", [262143, 262144, 300000, 5000000, 2 ** 27 + 3])
def test_embedding_gradient_of_many_passes(N, V):
    """Tables whose ids take two, three and four passes of the tiled sort, with
    padding and bad ids, in calls that follow one another in one workspace
    (exact: small whole numbers)."""
    C, pad = (4, 7) if V < 2 ** 27 else (1, 7)
    op = layers.Embedding(V, C, padding=pad)
    ws = torch.empty(B.eqconv_embedding_workspace_bytes(op.plan, N), dtype=torch.uint8, device="cuda")
    g = gen(V + N)
    calls = []
    for k in range(4):
        z = torch.randint(0, V, (N,), device="cuda", generator=g)
        z[1::2] = z[1::2] // (V // 300) * (V // 300) % V                    # half of them share 300 rows
        z[:5] = torch.tensor([0, V - 1, pad, -1, V], device="cuda")
        calls.append((z, torch.randint(-4, 5, (N, C), device="cuda", generator=g).float()))
    outs = [torch.full((V, C), float("nan"), device="cuda") for _ in calls]
    for (z, gy), out in zip(calls, outs):
        op.backward_raw(z, gy, out=out, workspace=ws)
    for (z, gy), out in zip(calls, outs):
        keep = (z >= 0) & (z < V) & (z != pad)
        assert torch.equal(out, torch.zeros(V, C, device="cuda").index_add_(0, z[keep], gy[keep]))
    assert B.eqconv_get_device_error(op.plan) == B.EQCONV_ERR_DEVICE_CHECK


def test_embedding_bad_ids():
    for dtype, bad in ((torch.int32, [-1, 7, 2 ** 31 - 1, -2 ** 31]), (torch.int64, [-1, 7, 2 ** 40, -2 ** 62, 2 ** 32])):
        z = torch.tensor([0, 6] + bad + [3], dtype=dtype, device="cuda")
        op = layers.Embedding(7, 12)
        table, gy = randn(gen(1), 7, 12), randn(gen(2), len(z), 12)
        y = op.forward_raw(z, table)
        assert B.eqconv_get_device_error(op.plan) == B.EQCONV_ERR_DEVICE_CHECK
        assert_within("y", y, ol.embedding(np64(z), np64(table)), 0.0)
        assert not y[2:-1].any()
        d = op.backward_raw(z, gy)
        assert B.eqconv_get_device_error(op.plan) == B.EQCONV_ERR_DEVICE_CHECK
        assert_within("dtable", d, ol.embedding_grad(np64(z).astype(np.int64), np64(gy), 7), 1e-6)
        assert B.eqconv_get_device_error(op.plan) == B.EQCONV_OK


def test_embedding_no_nodes_and_infinities():
    op = layers.Embedding(5, 6)
    z = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert op.forward_raw(z, randn(gen(1), 5, 6)).shape == (0, 6)
    assert torch.equal(op.backward_raw(z, torch.zeros(0, 6, device="cuda")), torch.zeros(5, 6, device="cuda"))
    z = torch.tensor([1, 1, 2], device="cuda")
    gy = torch.ones(3, 6, device="cuda")
    gy[0, 0], gy[2, 1] = float("inf"), float("nan")
    d = op.backward_raw(z, gy)
    assert d[1, 0] == float("inf") and d[2, 1].isnan() and int((~d.isfinite()).sum()) == 2
    # the padding row's gradient is not read into others
    op = layers.Embedding(5, 6, padding=2)
    d = op.backward_raw(z, gy)
    assert not d[2].any() and int((~d.isfinite()).sum()) == 1


def test_embedding_strided_rows():
    """The l = 0 rows of node features [N][D][C] as output and as gradient; a
    wider table; a gradient that repeats one row; unaligned starts."""
    N, D, C, V = 100, 9, 32, 11
    g = gen(9)
    z = torch.randint(0, V, (N,), device="cuda", generator=g, dtype=torch.int32)
    wide = randn(g, V, C + 8)
    op = layers.Embedding(V, C)
    x = torch.full((N, D, C), 7.0, device="cuda")
    op.forward_raw(z, wide[:, :C], out=x[:, 0, :])
    assert torch.equal(x[:, 0], wide[z.long(), :C]) and bool((x[:, 1:] == 7.0).all())
    op.forward_raw(z, wide[:, 3:3 + C], out=x[:, 2, :])
    assert torch.equal(x[:, 2], wide[z.long(), 3:3 + C])
    gx = torch.randint(-5, 6, (N, D, C), device="cuda", generator=g).float()
    assert torch.equal(op.backward_raw(z, gx[:, 0]), op.backward_raw(z, gx[:, 0].contiguous()))
    row = torch.randint(-5, 6, (1, C), device="cuda", generator=g).float()
    assert torch.equal(op.backward_raw(z, row.expand(N, C)), op.backward_raw(z, row.repeat(N, 1)))
    one = torch.ones((), device="cuda").expand(N, C)
    assert torch.equal(op.backward_raw(z, one), op.backward_raw(z, torch.ones(N, C, device="cuda")))
    ids2 = z.reshape(10, 10).t()
    assert torch.equal(op.forward_raw(ids2, wide[:, :C]), wide[ids2.long(), :C])


def test_embedding_autograd():
    op = layers.Embedding(6, 20, padding=0)
    z = torch.randint(0, 6, (4, 25), device="cuda", generator=gen(1))
    table = randn(gen(2), 6, 20).requires_grad_(True)
    w = randn(gen(3), 4, 25, 20)
    (op(z, table, 2.0) * w).sum().backward()
    want = torch.zeros(6, 20, device="cuda", dtype=torch.float64).index_add_(0, z.reshape(-1), w.double().reshape(-1, 20))
    want[0] = 0
    assert_within("table.grad", table.grad, 2 * np64(want), 100 * U * 40)
    with pytest.raises(RuntimeError):
        (d,) = torch.autograd.grad((op(z, table) ** 2).sum(), table, create_graph=True)
        d.sum().backward()


def test_embedding_tables_of_repeated_and_overlapping_rows():
    """Through autograd a table may be any view: one row for all types, rows that
    overlap, columns apart.  The raw form, which copies nothing, refuses them."""
    V, C = 6, 8
    op = layers.Embedding(V, C)
    z = torch.randint(0, V, (50,), device="cuda", generator=gen(1))
    w = torch.randint(-3, 4, (50, C), device="cuda", generator=gen(2)).float()
    views = {"repeated": (torch.randn(1, C, device="cuda"), lambda t: t.expand(V, C)),
             "overlapping": (torch.randn(2 * V + C, device="cuda"), lambda t: t.as_strided((V, C), (2, 1))),
             "columns apart": (torch.randn(V, 2 * C, device="cuda"), lambda t: t[:, ::2]),
             "transposed": (torch.randn(C, V, device="cuda"), lambda t: t.t())}
    for name, (leaf, view) in views.items():
        leaf.requires_grad_(True)
        y = op(z, view(leaf))
        assert torch.equal(y, view(leaf)[z]), name
        (got,) = torch.autograd.grad((y * w).sum(), leaf)
        (want,) = torch.autograd.grad((view(leaf)[z] * w).sum(), leaf)
        assert torch.equal(got, want), name                     # exact: whole numbers
        with pytest.raises(ValueError, match="rows"):
            op.forward_raw(z, view(leaf.detach()))
    with pytest.raises(ValueError, match="rows"):
        op.forward_raw(z, torch.zeros(V, C, device="cuda"), out=torch.zeros(1, C, device="cuda").expand(50, C))


# ----------------------------------------------------------------- block norm

NORM = [  # N, L, C, dtype, gate
    (1, 0, 1, "fp32", "sigmoid"),
    (1, 0, 1024, "bf16", "sigmoid"),
    (3, 3, 4, "fp32", "silu"),
    (50, 2, 128, "fp32", "silu"),
    (37, 1, 5, "bf16", "tanh"),
    (65, 3, 64, "bf16", "sigmoid"),
    (301, 2, 32, "fp16", "none"),
    (129, 3, 128, "fp32", "sigmoid"),
    (19, 0, 4096, "bf16", "tanh"),
    (7, 0, 8191, "fp32", "silu"),
    (5, 0, 8192, "fp16", "sigmoid"),
    (33, 1, 200, "fp32", "none"),
    (11, 2, 512, "bf16", "silu"),
    (9, 3, 510, "fp32", "tanh"),
    (6, 1, 1000, "fp32", "sigmoid"),
    (3, 3, 4096, "fp32", "sigmoid"),
    (2, 0, 16384, "bf16", "none"),
    (2000, 1, 16, "fp32", "sigmoid"),
    (4000, 0, 96, "bf16", "silu"),
    (6001, 2, 128, "fp32", "silu"),          # dozens of nodes for every warp of every SM
    (5003, 0, 2048, "bf16", "tanh"),
    (4001, 2, 37, "fp32", "tanh"),           # rows off the 16-byte boundaries
    (3001, 0, 2047, "fp16", "silu"),
    (2003, 1, 333, "bf16", "sigmoid"),
    (1501, 0, 3, "bf16", "none"),
    (301, 3, 210, "fp32", "silu"),
    (2, 0, 16384, "fp32", "sigmoid"),
    (40, 3, 502, "fp32", "tanh"),            # two nodes do not fit shared memory backward
    (40, 3, 700, "fp32", "silu"),
    (25, 1, 1500, "bf16", "sigmoid"),
    (25, 2, 900, "fp32", "none"),
    (30, 0, 6000, "fp32", "tanh"),
    (20, 0, 9000, "fp32", "silu"),           # too wide for registers too
    (20, 1, 1999, "fp16", "sigmoid"),
    (1400, 0, 264, "bf16", "silu"),          # many wide rows, from the narrowest
    (1190, 0, 1032, "fp32", "sigmoid"),
    (1184, 0, 4096, "fp16", "none"),
    (20011, 1, 8, "fp16", "sigmoid"),
]


def _norm_case(N, L, C, dtype, gate, seed=0):
    g = gen(seed)
    t = T[dtype]
    x, b, gx, gh = (randn(g, N, (L + 1) ** 2, C, dtype=t, mul=m) for m in (1.0, 3.0, 1.0, 1.0))
    q = randn(g, N, L + 1, C, dtype=t, mul=2.0) if gate != "none" else None
    wo, wi = (1 + 0.3 * randn(g, L + 1, C) for _ in range(2))
    return x, b, q, wo, wi, gx, gh


def _rms_err(L, C):
    """Relative error of 1 / rms in fp32: the sum of M positive squares (M 2^-24
    at the very worst; at most 64 in a row here in any kernel, then a tree of
    at most 15 levels) halved by the root, and a few roundings around it."""
    return (0.5 * min((2 * L + 1) * C, 64 + 15 + 8) + 6) * U


def _norm_tols(args, gx, gh, scale, eps, kind, dtype):
    """Tolerances of every output: relative errors of the factors counted along
    the formulas, times the sizes of the terms, plus half a step of the type."""
    x, b, gate, wo, wi = (np64(t) for t in args)
    L, C = int(round(x.shape[1] ** 0.5)) - 1, x.shape[2]
    r = _rms_err(L, C) + 12 * U                    # a product of up to a dozen rounded factors with 1/rms
    if kind == "tanh" and dtype != torch.float32:
        # (1 - q) / (1 + q) with q = exp(-2|g|): 1 - q >= 2|g| (1 - |g|) is off by about 2^-24, and 16-bit gates take
        # that form down to |g| = 2^-8, where it is 2^-24 / 2^-7 of the value; below, g itself is g^2 / 3 < 2^-17 off
        r += 2.0 ** -17
    ab = lambda v: None if v is None else np.abs(v)  # noqa: E731
    y, h = ol.block_norm(x, b, gate, wo, wi, scale, eps, kind)
    amp = y if y is not None else x
    # the size of x + t before cancellation
    ymag = np.abs(x) + (0 if b is None else np.abs(amp - x))
    hd = half(dtype)
    tol = {}
    if y is not None:
        tol["x"] = 2 * r * ymag + hd * np.abs(y) + tiny(dtype)
    rows = np.repeat(np.arange(L + 1), [2 * l + 1 for l in range(L + 1)])
    per = lambda v: np.stack([(v[:, rows == l]).mean(axis=(1, 2)) for l in range(L + 1)], 1)[:, rows][..., None]  # noqa: E731,E501
    sy = 1 / np.sqrt(per(amp ** 2) + eps)
    # sums of squares of y see y's own error, relative to |y| in the root mean square
    ry = r + 2 * r * np.sqrt(per(ymag ** 2)) * sy
    if h is not None:
        tol["h"] = (2 * r * ymag * sy + ry * np.abs(amp) * sy) * np.abs(wi)[rows] + hd * np.abs(h) + tiny(dtype)
    if gx is None and gh is None:
        return tol, (y, h), None
    grads = ol.block_norm_grad(x, b, gate, wo, wi, np64(gx), np64(gh), scale, eps, kind)
    t = np.zeros_like(x) if gx is None else ab(np64(gx))
    if gh is not None:
        p = ab(np64(gh)) * np.abs(wi)[rows]
        pm = per(p * ymag)
        tmag = t + sy * p + ymag * sy ** 3 * pm
        terr = 4 * ry * tmag + 64 * U * tmag
    else:
        tmag, terr = t, 2 * U * t
    tol["dx"] = terr + hd * np.abs(grads[0]) + tiny(dtype)
    n_sum = x.shape[0] + 40                        # nodes added one after the other, then warps and blocks
    if b is not None:
        sb = 1 / np.sqrt(per(b ** 2) + eps)
        a = ab(ol.gate_function(kind, gate))[:, rows] if gate is not None else 1.0
        # the gate's functions in fp32 with a few units in the last place
        rel = 2 * r + 16 * U
        wod = np.abs(wo)[rows]
        u, q = ab(b) * sb * wod, scale * a * tmag * wod
        qerr = scale * a * terr * wod + rel * q
        qm, qe = per(q * ab(b)), per(qerr * ab(b))
        db = sb * q + ab(b) * sb ** 3 * qm
        tol["db"] = 2 * rel * db + sb * qerr + ab(b) * sb ** 3 * qe + 64 * U * db + hd * np.abs(grads[1]) + tiny(dtype)
        sums = lambda v: np.stack([v[:, rows == l].sum(1) for l in range(L + 1)], 1)  # noqa: E731
        if gate is not None:
            # the derivative's own terms may cancel: bounded by 1.1 in size
            tol["dgate"] = scale * (sums(terr * u) * 1.1 + rel * 1.1 * sums(tmag * u)) + hd * np.abs(grads[2]) + tiny(dtype)
        w = sums(scale * a * (terr + rel * tmag) * ab(b) * sb)
        mag = sums(scale * a * tmag * ab(b) * sb)
        tol["dw_post"] = w.sum(0) + n_sum * U * mag.sum(0)
    if gh is not None:
        v = ab(np64(gh)) * ymag * sy
        sums = lambda v: np.stack([v[:, rows == l].sum(1) for l in range(L + 1)], 1)  # noqa: E731
        tol["dw_pre"] = sums(v * (ry + 4 * r)).sum(0) + n_sum * U * sums(v).sum(0)
    return tol, (y, h), grads


@pytest.mark.parametrize("form", ["both", "post", "pre"])
@pytest.mark.parametrize("case", NORM, ids=str)
def test_block_norm(case, form):
    N, L, C, dtype, kind = case
    x, b, gate, wo, wi, gx, gh = _norm_case(*case)
    if form == "pre":
        b = gate = wo = gx = None
    if form == "post":
        wi = gh = None
    op = layers.BlockNorm(natural_irreps(L), C, gate=kind if form != "pre" else "none", eps=1e-5, dtype=T[dtype])
    scale = 0.6
    args = (x, b, gate, wo, wi)
    xo, h, stats = op.forward_raw(*args, scale=scale, save=True)
    tol, (y64, h64), g64 = _norm_tols(args, gx, gh, np.float32(scale).astype(np.float64),
                                      np.float32(1e-5).astype(np.float64), op.gate, T[dtype])
    if form != "pre":
        assert_within("x_out", xo, y64, tol["x"])
    if form != "post":
        assert_within("h", h, h64, tol["h"])
    got = op.backward_raw(*args, stats, gx, gh, scale=scale)
    again = op.backward_raw(*args, stats, gx, gh, scale=scale)
    for name, g, a, w in zip(("dx", "db", "dgate", "dw_post", "dw_pre"), got, again, g64):
        assert (g is None) == (w is None), name
        if g is not None:
            assert_within(name, g, w, tol[name])
            assert torch.equal(g, a)                                        # bitwise reproducible
    # without statistics to keep, the same outputs
    xo2, h2, none = op.forward_raw(*args, scale=scale)
    assert none is None and (xo is None or torch.equal(xo, xo2)) and (h is None or torch.equal(h, h2))


@pytest.mark.parametrize("form", ["both", "post", "pre"])
@pytest.mark.parametrize("case", [
    (20000, 0, 33, "bf16", "silu"), (20000, 0, 32, "bf16", "tanh"), (200000, 0, 4, "bf16", "sigmoid"),
    (10000, 0, 65, "fp16", "none"), (5000, 0, 130, "bf16", "silu"), (5000, 0, 33, "fp32", "sigmoid"),
    (2000, 0, 96, "fp32", "none"), (9001, 0, 1, "bf16", "tanh"), (70, 0, 2, "fp16", "silu"), (3001, 0, 7, "fp32", "tanh"),
    (3000, 1, 1, "bf16", "sigmoid"), (777, 2, 3, "fp32", "silu")], ids=str)
def test_block_norm_narrow_rows(case, form):
    """Rows of few channels, whose ring of slots is small."""
    test_block_norm(case, form)


@pytest.mark.parametrize("form", ["both", "pre"])
@pytest.mark.parametrize("case", [(60, 3, 820, "bf16", "silu"), (33, 3, 1020, "fp16", "none"), (40, 3, 1018, "bf16", "tanh")],
                         ids=str)
def test_block_norm_wide_nodes_in_8_byte_rows(case, form):
    """16-bit nodes of which two do not fit shared memory backward, in rows of
    whole 8 bytes and of 4."""
    test_block_norm(case, form)


@pytest.mark.parametrize("missing", ["g_x", "g_h"])
def test_block_norm_one_gradient_only(missing):
    case = (40, 2, 64, "fp32", "sigmoid")
    x, b, gate, wo, wi, gx, gh = _norm_case(*case, seed=4)
    op = layers.BlockNorm(natural_irreps(2), 64, dtype=T["fp32"])
    _, _, stats = op.forward_raw(x, b, gate, wo, wi, save=True)
    zero = torch.zeros_like(x)
    a = op.backward_raw(x, b, gate, wo, wi, stats, None if missing == "g_x" else gx, None if missing == "g_h" else gh)
    c = op.backward_raw(x, b, gate, wo, wi, stats, zero if missing == "g_x" else gx, zero if missing == "g_h" else gh)
    for p, q in zip(a, c):
        assert torch.allclose(p, q, rtol=1e-5, atol=1e-5)


def test_block_norm_edges():
    """Rows of zeros stay finite (eps), a NaN or infinity stays in its node and
    degree, no nodes give empty outputs and zero weight gradients."""
    N, L, C = 6, 1, 32
    x, b, gate, wo, wi, gx, gh = _norm_case(N, L, C, "fp32", "sigmoid", seed=8)
    op = layers.BlockNorm(natural_irreps(L), C)
    x[0] = 0
    b[0] = 0
    b[1] = 0
    xo, h, stats = op.forward_raw(x, b, gate, wo, wi, save=True)
    assert not xo[0].any() and not h[0].any() and torch.equal(xo[1], x[1])
    assert all(bool(g.isfinite().all()) for g in op.backward_raw(x, b, gate, wo, wi, stats, gx, gh))
    b[2, 0, 3], x[3, 2, 5] = float("nan"), float("inf")
    xo, h, _ = op.forward_raw(x, b, gate, wo, wi)
    clean = [bool(v.isfinite().all()) for v in (xo[2, 1:], xo[3, :1], h[2, 1:], h[3, :1], xo[4:], h[4:])]
    assert all(clean) and bool(h[2, 0].isnan().all()) and bool(h[3, 2, 5].isnan())
    e = lambda t: t[:0]  # noqa: E731
    xo, h, stats = op.forward_raw(e(x), e(b), e(gate), wo, wi, save=True)
    assert xo.shape == h.shape == (0, 4, C)
    dw = op.backward_raw(e(x), e(b), e(gate), wo, wi, stats, e(gx), e(gh))[3:]
    assert all(torch.equal(d, torch.zeros_like(wo)) for d in dw)


def test_block_norm_extreme_gates():
    """Gates of large size saturate without NaN, in value and derivative."""
    for kind in ("sigmoid", "silu", "tanh"):
        x, b, gate, wo, wi, gx, gh = _norm_case(4, 0, 64, "fp32", kind, seed=2)
        gate = torch.linspace(-200, 200, 4 * 64, device="cuda").reshape(4, 1, 64)
        op = layers.BlockNorm("0e", 64, gate=kind)
        xo, h, stats = op.forward_raw(x, b, gate, wo, wi, save=True)
        got = op.backward_raw(x, b, gate, wo, wi, stats, gx, gh)
        want = ol.block_norm_grad(*(np64(t) for t in (x, b, gate, wo, wi, gx, gh)), 1.0, 1e-6, kind)
        for a, w in zip(got, want):
            assert bool(a.isfinite().all())
            assert np.abs(np64(a) - w).max() <= 1e-5 * np.abs(w).max() + 1e-6


@pytest.mark.parametrize("kind", ["sigmoid", "silu", "tanh"])
@pytest.mark.parametrize("dtype,L,C", [("fp32", 0, 64), ("fp32", 2, 41), ("fp32", 0, 1024), ("fp32", 0, 9000),
                                       ("fp32", 3, 700), ("bf16", 1, 64), ("bf16", 0, 4096), ("fp16", 0, 520)])
def test_block_norm_gradient_of_saturated_gates(kind, dtype, L, C):
    """The gate's gradient is right relative to itself where the gate is close to
    its limits, 0 and 1 (-1 and 1).

    dgate = scale a'(g) sum_m t u with t = g_x.  In units of 2^-24, a'(g) is off
    by 3 |g| (the argument of the power, 2 |g| log2 e, rounded, with a constant
    that is rounded too), 4 (2^x), 4 (1/x, twice) and 6 (sums and products); u by
    what 1 / rms and a dozen factors are."""
    N, t = 5, T[dtype]
    g = gen(C + L)
    x, b, gx = (randn(g, N, (L + 1) ** 2, C, dtype=t) for _ in range(3))
    gate = ((torch.rand(N, L + 1, C, device="cuda", generator=g) - 0.5) * 80).to(t)
    gate[0, 0, :8] = torch.tensor([0.0, -0.25, 0.25, 1e-3, 40.0, -40.0, 17.5, -17.5], device="cuda").to(t)
    wo = 1 + 0.3 * randn(g, L + 1, C)
    op = layers.BlockNorm(natural_irreps(L), C, gate=kind, dtype=t)
    _, _, stats = op.forward_raw(x, b, gate, wo, None, scale=0.6, save=True)
    dgate = op.backward_raw(x, b, gate, wo, None, stats, gx, None, scale=0.6)[2]
    q, b64, w64 = np64(gate), np64(b), np64(wo)
    s, r = 1 / (1 + np.exp(-q)), 1 / (1 + np.exp(q))
    da, mag = {"sigmoid": (s * r, s * r), "silu": (s * (1 + q * r), s * (1 + np.abs(q) * r)),
               "tanh": (1 / np.cosh(q) ** 2,) * 2}[kind]
    want, size = np.empty_like(q), np.empty_like(q)
    for l in range(L + 1):
        rows = slice(l * l, (l + 1) ** 2)
        v = b64[:, rows]
        u = v / np.sqrt((v ** 2).mean(axis=(1, 2), keepdims=True) + np.float64(np.float32(1e-6))) * w64[l]
        tu = np64(gx)[:, rows] * u * np.float64(np.float32(0.6))
        want[:, l], size[:, l] = da[:, l] * tu.sum(1), mag[:, l] * np.abs(tu).sum(1)
    rel = _rms_err(L, C) + (12 + 14 + 3 * np.abs(q) + 2 * L + 4) * U
    # (products of values below the normal range of fp32 may vanish on the way)
    assert_within("dgate", dgate, want, rel * size + half(t) * np.abs(want) * (1 + 1e-3) + tiny(t) + 2.0 ** -120)


@pytest.mark.parametrize("N,L,C", [(21, 1, 64), (100, 1, 7), (1, 0, 1), (40, 0, 3), (9, 0, 4001), (700, 2, 33)])
def test_block_norm_unaligned_views(N, L, C):
    """Tensors that start off the 16-byte boundary, each by its own step, give
    the aligned ones' results: the bytes before and behind them are NaN."""
    args = _norm_case(N, L, C, "bf16", "silu", seed=6)
    op = layers.BlockNorm(natural_irreps(L), C, gate="silu", dtype=torch.bfloat16)
    steps = iter(range(1, 100))

    def off(t):
        k = next(steps) % 7 + 1
        room = torch.full((t.numel() + 2 * k,), float("nan"), dtype=t.dtype, device="cuda")
        room[k:-k] = t.reshape(-1)
        return room[k:-k].view(t.shape)

    a = op.forward_raw(*args[:5], save=True)
    o = [off(t) for t in args]
    c = op.forward_raw(*o[:5], save=True)
    for p, q in zip(a, c):
        assert torch.allclose(p.float(), q.float(), rtol=2 ** -7, atol=1e-5)
    ga = op.backward_raw(*args[:5], a[2], *args[5:])
    gc = op.backward_raw(*o[:5], off(c[2]), *o[5:])
    for p, q in zip(ga, gc):
        assert torch.allclose(p.float(), q.float(), rtol=2 ** -6, atol=1e-2)


def test_block_norm_autograd_and_broadcast_gradients():
    N, L, C = 15, 1, 24
    x, b, gate, wo, wi, gx, gh = _norm_case(N, L, C, "fp32", "sigmoid", seed=11)
    op = layers.BlockNorm(natural_irreps(L), C)
    leaves = [t.clone().requires_grad_(True) for t in (x, b, gate, wo, wi)]
    xo, h = op(*leaves, scale=0.3)
    got = torch.autograd.grad((xo * gx).sum() + (h * gh).sum(), leaves)
    _, _, stats = op.forward_raw(x, b, gate, wo, wi, scale=0.3, save=True)
    for a, c in zip(got, op.backward_raw(x, b, gate, wo, wi, stats, gx, gh, scale=0.3)):
        assert torch.equal(a, c)
    # a gradient that is one number everywhere, through one output only
    xo, h = op(*leaves, scale=0.3)
    got = torch.autograd.grad(h.sum(), leaves)
    for a, c in zip(got, op.backward_raw(x, b, gate, wo, wi, stats, None, torch.ones_like(x), scale=0.3)):
        assert torch.equal(a, c)
    # a gate shared by all nodes: its gradient is summed over them
    g1 = gate[:1].clone().requires_grad_(True)
    xo, h = op(x, b, g1.expand(N, L + 1, C), wo, wi)
    (d,) = torch.autograd.grad((xo * gx).sum() + (h * gh).sum(), [g1])
    want = ol.block_norm_grad(np64(x), np64(b), np64(g1.expand(N, L + 1, C)), np64(wo), np64(wi), np64(gx), np64(gh),
                              1.0, 1e-6, "sigmoid")[2].sum(0, keepdims=True)
    assert np.abs(np64(d) - want).max() <= 1e-5 * np.abs(want).max()
    # pre only and post only through autograd
    xr = x.clone().requires_grad_(True)
    pre = layers.BlockNorm(natural_irreps(L), C, gate="none")
    same, h = pre(xr, w_pre=wi)
    assert same is xr
    h.sum().backward()
    assert xr.grad is not None
    xo, none = pre(xr, b=b, w_post=wo)
    assert none is None and torch.equal(xo, pre.forward_raw(x, b, None, wo, None)[0])
    with pytest.raises(RuntimeError):
        (d,) = torch.autograd.grad((pre(xr, w_pre=wi)[1] ** 2).sum(), xr, create_graph=True)
        d.sum().backward()


def test_block_norm_refusals():
    op = layers.BlockNorm("0e+1o", 8)
    x, b, gate, wo, wi, gx, gh = _norm_case(3, 1, 8, "fp32", "sigmoid")
    for bad in ((x, b, None, wo, wi), (x, None, gate, None, wi), (x, b, gate, None, wi), (x, None, None, None, None),
                (x[:, :1], b, gate, wo, wi), (x, b.half(), gate, wo, wi), (x, b, gate, wo.half(), wi),
                (x, b, gate, wo.cpu(), wi), (x.transpose(0, 2).contiguous().transpose(0, 2), b, gate, wo, wi)):
        with pytest.raises(ValueError):
            op.forward_raw(*bad)
    for out in ((x, torch.empty_like(x)), (torch.empty_like(x), b)):          # outputs on inputs
        with pytest.raises(B.EqconvError):
            op.forward_raw(x, b, gate, wo, wi, out=out)
    _, _, stats = op.forward_raw(x, b, gate, wo, wi, save=True)
    with pytest.raises(ValueError):
        op.backward_raw(x, b, gate, wo, None, stats, gx, gh)
    with pytest.raises(B.EqconvError):
        op.backward_raw(x, b, gate, wo, wi, stats, gx, gh, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    emb = layers.Embedding(4, 8)
    with pytest.raises(B.EqconvError):                                        # another operator's plan
        B.eqconv_block_norm(emb.plan, 3, x.data_ptr(), None, None, None, wi.data_ptr(), 1.0, None, gx.data_ptr(), None)
    with pytest.raises(B.EqconvError):
        B.eqconv_spherical_harmonics(0, 1, x, gx)


# ----------------------------------------------------------------------- clip

def _tensors(sizes, types, seed=0, mul=1.0):
    g = gen(seed)
    return [randn(g, *(s if isinstance(s, tuple) else (s,)), dtype=T[t], mul=mul) for s, t in zip(sizes, types)]


CLIP = [
    ([1], ["fp32"]),
    ([7, 0, 1, 4099], ["fp32", "fp32", "bf16", "fp16"]),
    ([(64, 100), (3, 5, 7), 16384, 16385, 8193], ["bf16", "fp32", "fp32", "bf16", "fp16"]),
    ([5] * 97, ["fp32"] * 97),
    ([33 + i for i in range(1500)], ["bf16" if i % 3 else "fp32" for i in range(1500)]),
    ([3_000_001, 20_000_003], ["fp32", "bf16"]),
]


@pytest.mark.parametrize("case", range(len(CLIP)))
@pytest.mark.parametrize("bound", [0.01, 1e9])
def test_clip(case, bound):
    ts = _tensors(*CLIP[case], seed=case)
    before = [t.clone() for t in ts]
    want_n, want = ol.clip([np64(t) for t in ts], np.float32(bound).astype(np.float64),
                           np.float32(1e-6).astype(np.float64))
    outs = [torch.empty_like(t) for t in ts]
    n = layers.clip_gradients(ts, bound, out=outs)
    assert n.dtype == torch.float32 and n.dim() == 0
    # fp64 sums (of 16-bit elements, of pairs of squares added in fp32: 2^-24 of the sum, half of it in the root), one
    # rounding to fp32 of the norm, of k and of the product, one to the type
    assert abs(n.item() - want_n) <= 2 * U * want_n
    assert torch.equal(n, layers.gradient_norm(ts))
    for t, b, o, w in zip(ts, before, outs, want):
        assert torch.equal(t, b)
        assert_within("out", o, w, (3 * U + half(o.dtype)) * np.abs(w) * (1 + 1e-3) + tiny(o.dtype))
    n2 = layers.clip_gradients(ts, bound)
    assert torch.equal(n, n2) and all(torch.equal(t, o) for t, o in zip(ts, outs))


@pytest.mark.parametrize("empties", ["none", "leading", "between", "trailing"])
@pytest.mark.parametrize("count", [40, 41, 96, 97, 1023, 1024, 1025, 2048])
def test_clip_lists_around_a_launch(count, empties):
    """Lists of as many tensors as a launch takes, and one more or fewer, with
    empty tensors at either end or between: all are clipped, in place and not."""
    ts = _tensors([1 + i % 5 for i in range(count)], ["bf16" if i % 7 == 3 else "fp32" for i in range(count)], seed=count)
    none = [torch.zeros(0, device="cuda") for _ in range(3)]
    if empties == "between":
        ts = [t for i, t in enumerate(ts) for t in ([none[0], t] if i % 100 == 50 else [t])]
    ts = none * (empties == "leading") + ts + none * (empties == "trailing")
    want_n, want = ol.clip([np64(t) for t in ts], 0.5, np.float32(1e-6).astype(np.float64))
    outs = [torch.full_like(t, float("nan")) for t in ts]
    n = layers.clip_gradients(ts, 0.5, out=outs)
    # roundings as in test_clip
    assert abs(n.item() - want_n) <= 2 * U * want_n
    for o, w in zip(outs, want):
        assert_within("out", o, w, (3 * U + half(o.dtype)) * np.abs(w) * (1 + 1e-3) + tiny(o.dtype))
    n2 = layers.clip_gradients(ts, 0.5)
    assert torch.equal(n, n2) and all(torch.equal(t, o) for t, o in zip(ts, outs))
    assert abs(layers.gradient_norm(ts).item() - 0.5) <= 0.5 * 2.0 ** -7


def test_clip_range_of_values():
    """Squares that fp32 cannot hold, large and small, still give the norm."""
    for v in (1e-30, 1e30, 3e38, 1e-44):
        t = torch.full((1000,), v, device="cuda")
        n = layers.gradient_norm([t]).item()
        want = float(t[0].double()) * np.sqrt(1000.0)
        if want > 3.4e38:
            assert n == float("inf")
        else:
            assert abs(n - want) <= max(2 * U * want, 1.5e-45)
    for v in (1e-30, 1e-19, 1e19, 3e38):
        t = torch.full((100000,), v, device="cuda", dtype=torch.bfloat16)
        t[::7] *= 0.5
        n, want = layers.gradient_norm([t]).item(), float(np.sqrt((np64(t) ** 2).sum()))
        assert n == float("inf") if want > 3.4e38 else abs(n - want) <= 2 * U * want
    big = torch.full((1000,), 1e30, device="cuda")
    layers.clip_gradients([big], 1.0)
    assert abs(layers.gradient_norm([big]).item() - 1.0) < 1e-6


def test_clip_non_finite():
    t, u = torch.ones(100, device="cuda"), torch.ones(50, device="cuda", dtype=torch.bfloat16)
    t[3] = float("inf")
    n = layers.clip_gradients([t, u], 1.0)
    assert n.item() == float("inf") and t[3].isnan() and not t[:3].any() and not u.any()
    t[3] = float("nan")
    n = layers.clip_gradients([t, u], 1.0)
    assert n.isnan() and bool(t.isnan().all()) and bool(u.isnan().all())


def test_clip_empty_and_zero():
    assert layers.clip_gradients([], 1.0).item() == 0.0
    assert layers.gradient_norm([torch.zeros(0, device="cuda")]).item() == 0.0
    z = torch.zeros(33, device="cuda")
    assert layers.clip_gradients([z, torch.zeros(0, device="cuda")], 0.0).item() == 0.0
    assert not z.any()
    t = torch.ones(5, device="cuda")
    layers.clip_gradients([t], 0.0)
    assert not t.any()


def test_clip_views():
    """Parts of one buffer at odd starts, transposed weights; nothing outside is touched."""
    buf = randn(gen(3), 5000)
    keep = buf.clone()
    parts = [buf[1:4], buf[7:1030], buf[1030:1031], buf[2000:4001]]
    want_n, want = ol.clip([np64(p) for p in parts], 0.5)
    layers.clip_gradients(parts, 0.5)
    for p, w in zip(parts, want):
        assert_within("part", p, w, 4 * U * np.abs(w))
    mask = torch.ones(5000, dtype=torch.bool, device="cuda")
    for a, b in ((1, 4), (7, 1031), (2000, 4001)):
        mask[a:b] = False
    assert torch.equal(buf[mask], keep[mask])
    w = randn(gen(4), 30, 40).t()
    want_n, (want,) = ol.clip([np64(w)], 0.5)
    layers.clip_gradients([w], 0.5)
    assert_within("transposed", w, want, 4 * U * np.abs(want))
    # an output off its input's alignment
    src, room = randn(gen(5), 4096), torch.zeros(4100, device="cuda")
    layers.clip_gradients([src], 0.5, out=[room[1:4097]])
    want_n, (want,) = ol.clip([np64(src)], 0.5)
    assert_within("shifted", room[1:4097], want, 4 * U * np.abs(want))
    assert not room[0].any() and not room[4097:].any()


def test_clip_refusals():
    t = torch.ones(8, device="cuda")
    for bad in ([t, t], [t, t[2:4]], [t[:5], t[4:]]):
        with pytest.raises(B.EqconvError):
            layers.clip_gradients(bad, 1.0)
    with pytest.raises(B.EqconvError):
        layers.clip_gradients([t[:4]], 1.0, out=[t[2:6]])
    for bad in ([t.double()], [torch.ones(4, 4, device="cuda")[:, :2]], [torch.ones(1, device="cuda").expand(4)]):
        with pytest.raises(ValueError):
            layers.clip_gradients(bad, 1.0)
    with pytest.raises(ValueError):
        layers.clip_gradients([t], 1.0, out=[t[:4]])
    with pytest.raises(ValueError):
        layers.clip_gradients([t], 1.0, out=[])
    assert bool((t == 1).all())


# --------------------------------------------------------- streams and graphs

@pytest.mark.parametrize("N,L,C,V", [(700, 1, 64, 50), (9000, 0, 33, 3000), (70000, 1, 8, 1000)])
def test_own_stream_and_graph_replay(N, L, C, V):
    """On a stream of their own, and captured: replays follow the inputs'
    current contents, and two graphs share no workspace."""
    s = torch.cuda.Stream()
    emb, norm = layers.Embedding(V, C), layers.BlockNorm(natural_irreps(L), C)
    z, table, gy = _embed_case(N, V, C, "fp32", "fp32", "int32")
    x, b, gate, wo, wi, gx, gh = _norm_case(N, L, C, "fp32", "sigmoid")
    ts = _tensors([1000, 33], ["fp32", "bf16"])
    outs = [torch.empty_like(t) for t in ts]

    def step(stream=None):
        y = emb.forward_raw(z, table, 1.3, stream=stream)
        d = emb.backward_raw(z, gy, 1.3, stream=stream)
        xo, h, st = norm.forward_raw(x, b, gate, wo, wi, save=True, stream=stream)
        g = norm.backward_raw(x, b, gate, wo, wi, st, gx, gh, stream=stream)
        n = layers.clip_gradients(ts, 0.1, out=outs, stream=stream)
        return [y, d, xo, h, *g, n]

    want = [t.clone() for t in step()]
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graphs, results = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(step())
        graphs.append(g)
    for t in (table, gy, x, b, gate, gx, gh, *ts):
        t.mul_(0.75)
    z.copy_((z + 1) % V)
    for g in graphs:
        g.replay()
    want = step()
    for r in results:
        assert all(torch.equal(a, c) for a, c in zip(r, want))


def test_captured_autograd_step():
    """Forward and backward through autograd in one captured graph: a replay
    gives the gradients of the inputs' current contents."""
    N, L, C, V = 500, 1, 48, 30
    emb, norm = layers.Embedding(V, C), layers.BlockNorm(natural_irreps(L), C)
    z, table, _ = _embed_case(N, V, C, "fp32", "fp32", "int32")
    x, b, gate, wo, wi, gx, gh = _norm_case(N, L, C, "fp32", "sigmoid")
    leaves = [t.requires_grad_(True) for t in (table, b, gate, wo, wi)]

    def step():
        x0 = torch.cat([emb(z, table, 1.5)[:, None], x[:, 1:]], 1)
        xo, h = norm(x0, b, gate, wo, wi, 0.7)
        return torch.autograd.grad((xo * gx).sum() + (h * gh).sum(), leaves)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    with torch.no_grad():
        for t in leaves:
            t.mul_(1.25)
    g.replay()
    torch.cuda.synchronize()
    for a, c in zip(got, step()):
        assert torch.equal(a, c)


def test_two_streams_at_once():
    """Calls of one operator that overlap on two streams do not disturb each other."""
    V, C, L = 5000, 64, 1
    emb, norm = layers.Embedding(V, C), layers.BlockNorm(natural_irreps(L), C)
    cases = [(_embed_case(30000, V, C, "fp32", "fp32", "int64", seed=k), _norm_case(3000, L, C, "fp32", "sigmoid", seed=k),
              _tensors([100000, 77], ["fp32", "bf16"], seed=k)) for k in range(2)]

    def run(k):
        (z, table, gy), (x, b, gate, wo, wi, gx, gh), ts = cases[k]
        outs = [torch.empty_like(t) for t in ts]
        _, _, st = norm.forward_raw(x, b, gate, wo, wi, save=True)
        return [emb.backward_raw(z, gy), *norm.backward_raw(x, b, gate, wo, wi, st, gx, gh),
                layers.clip_gradients(ts, 0.1, out=outs), *outs]

    want = [[t.clone() for t in run(k)] for k in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((k, run(k)))
    torch.cuda.synchronize()
    for k, r in got:
        assert all(torch.equal(a, c) for a, c in zip(r, want[k]))


def test_two_host_threads_at_once():
    """Rows of different widths through one kernel, from two host threads with a
    stream each: neither changes what the other's launches may take."""
    widths = (8196, 16384)                       # too wide for registers, 66 and 131 KB of shared memory backward
    cases = []
    for C in widths:
        x, b, gate, wo, wi, gx, gh = _norm_case(1, 0, C, "fp32", "sigmoid", seed=C)
        op = layers.BlockNorm("0e", C)
        stats = op.forward_raw(x, b, gate, wo, wi, save=True)[2]
        want = op.backward_raw(x, b, gate, wo, wi, stats, gx, gh)
        got = [torch.zeros_like(t) for t in want]
        ws = torch.empty(B.eqconv_block_norm_workspace_bytes(op.plan, 1), dtype=torch.uint8, device="cuda")
        p = [t.data_ptr() for t in (x, b, gate, wo, wi, stats, gx, gh, *got)]
        cases.append((op, p, ws, got, want, (x, b, gate, wo, wi, stats, gx, gh)))
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(2)

    def run(op, p, ws, got, want, inputs):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(3000):
                B.eqconv_block_norm_backward(op.plan, 1, *p[:5], 1.0, *p[5:], ws, ws.numel(), stream.cuda_stream)
            stream.synchronize()
            if not all(torch.equal(a, c) for a, c in zip(got, want)):
                wrong.append("results")
        except Exception as e:
            wrong.append(repr(e))

    threads = [threading.Thread(target=run, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_clip_counts_as_in_place():
    """Autograd notices that a tensor it saved was clipped in place."""
    w = randn(gen(1), 50).requires_grad_(True)
    y = w * 2
    z = (y * y).sum()
    layers.clip_gradients([y.detach()], 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()


def test_training_step_of_two_layers():
    """Embedding, norms, convolutions and clipping as one training step against
    the same step made of the oracle's pieces by differences: the loss falls
    along the clipped gradient by the amount that the gradient says."""
    from equivariant_gnn_message_edge_b200.conv import EqConv
    N, E, C, V = 40, 400, 32, 7
    g = gen(21)
    z = torch.randint(0, V, (N,), device="cuda", generator=g, dtype=torch.int32)
    s, r = (torch.randint(0, N, (E,), device="cuda", generator=g, dtype=torch.int32) for _ in range(2))
    vec = randn(g, E, 3)
    irreps = natural_irreps(1)
    conv = EqConv(irreps, 1, irreps, C)
    graph = conv.graph(s, r, N)
    emb, norm = layers.Embedding(V, C), layers.BlockNorm(irreps, C)
    weights = [randn(g, E, conv.P, C, mul=0.1) for _ in range(2)]
    params = [randn(g, V, C)] + [1 + 0.1 * randn(g, 2, C) for _ in range(5)] + [randn(g, N, 2, C) for _ in range(2)]
    target = randn(g, N, 4, C)

    def loss(p, leaves=None):
        x = torch.zeros(N, 4, C, device="cuda")
        x = torch.cat([emb(z, p[0], 2.0)[:, None], x[:, 1:]], 1)
        _, h = layers.BlockNorm(irreps, C, gate="none")(x, w_pre=p[1])
        x, h = norm(x, conv(graph, h, vec, weights[0]), p[6], p[2], p[3], 0.5)
        x, h = norm(x, conv(graph, h, vec, weights[1]), p[7], p[4], p[5], 0.5)
        return ((h - target) ** 2).double().sum() + (x.double() ** 2).sum()

    leaves = [t.clone().requires_grad_(True) for t in params]
    loss(leaves).backward()
    grads = [t.grad for t in leaves]
    free = torch.sqrt(sum((t.double() ** 2).sum() for t in grads)).item()
    n = layers.clip_gradients(grads, 1.0)
    assert abs(n.item() - free) <= 1e-6 * free
    # d/dt loss(p + t grad) at 0 = |clipped| |free| = free * free / (free + eps)
    step = 1e-2
    hi = loss([p + step * d for p, d in zip(params, grads)]).item()
    lo = loss([p - step * d for p, d in zip(params, grads)]).item()
    # the difference's own error: fp32 rounding of the outputs (about 1e-7 of the loss in all) over the step, and
    # the third derivative along a unit direction (at most about |loss| / 1) times step^2 / 6
    total = abs(loss(params).item())
    assert abs((hi - lo) / (2 * step) - free) <= 3e-5 * total + 1e-3 * free
