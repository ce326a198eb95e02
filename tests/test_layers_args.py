"""The node-level operators' checks of their arguments, without a GPU: every
refusal below comes before any device work."""
import copy
import ctypes
import os
import pickle

import numpy as np
import pytest
import torch

from equivariant_gnn_message_edge_b200 import binding as B
from equivariant_gnn_message_edge_b200 import layers


@pytest.mark.parametrize("args,status", [
    ((0, 8, 0, 0, -1), B.EQCONV_ERR_INVALID_ARG),           # no types
    ((8, 0, 0, 0, -1), B.EQCONV_ERR_INVALID_ARG),           # no channels
    ((8, 8, 3, 3, -1), B.EQCONV_ERR_INVALID_ARG),           # unknown element type
    ((8, 8, 0, 0, 8), B.EQCONV_ERR_INVALID_ARG),            # padding is no type
    ((8, 8, 0, 0, -2), B.EQCONV_ERR_INVALID_ARG),
    ((8, 8, 1, 0, -1), B.EQCONV_ERR_UNSUPPORTED),           # bf16 table, fp32 rows
    ((8, 8, 1, 2, -1), B.EQCONV_ERR_UNSUPPORTED),           # bf16 table, fp16 rows
    ((8, 65537, 0, 0, -1), B.EQCONV_ERR_UNSUPPORTED),       # too wide
    ((2 ** 31 - 1, 8, 0, 0, -1), B.EQCONV_ERR_UNSUPPORTED)])
def test_embedding_plans_validate(args, status):
    with pytest.raises(B.EqconvError) as e:
        B.eqconv_embedding_plan_create(*args)
    assert e.value.status == status


@pytest.mark.parametrize("args,status", [
    (("0e+1q", 8, 0, 1, 1e-6), B.EQCONV_ERR_INVALID_ARG),
    (("0e+2e", 8, 0, 1, 1e-6), B.EQCONV_ERR_UNSUPPORTED),
    (("0e", 0, 0, 1, 1e-6), B.EQCONV_ERR_INVALID_ARG),
    (("0e", 16385, 0, 1, 1e-6), B.EQCONV_ERR_UNSUPPORTED),
    (("0e", 8, 5, 1, 1e-6), B.EQCONV_ERR_INVALID_ARG),
    (("0e", 8, 0, 4, 1e-6), B.EQCONV_ERR_INVALID_ARG),
    (("0e", 8, 0, 1, 0.0), B.EQCONV_ERR_INVALID_ARG),
    (("0e", 8, 0, 1, float("nan")), B.EQCONV_ERR_INVALID_ARG),
    (("0e", 8, 0, 1, float("inf")), B.EQCONV_ERR_INVALID_ARG)])
def test_block_norm_plans_validate(args, status):
    with pytest.raises(B.EqconvError) as e:
        B.eqconv_block_norm_plan_create(*args)
    assert e.value.status == status


def test_null_and_foreign_plans_are_refused():
    assert B.eqconv_embedding_workspace_bytes(0, 10) == 0
    assert B.eqconv_block_norm_workspace_bytes(0, 10) == 0
    with pytest.raises(B.EqconvError) as e:
        B.eqconv_embedding(None, 1, 16, 32, 16, 8, 1.0, 16, 8, 0)
    assert e.value.status == B.EQCONV_ERR_INVALID_ARG
    with pytest.raises(B.EqconvError) as e:
        B.eqconv_block_norm(None, 1, 16, None, None, None, 16, 1.0, None, 16, None, 0)
    assert e.value.status == B.EQCONV_ERR_INVALID_ARG


def _list(*rows):
    return (B.eqconv_tensor_t * max(1, len(rows)))(*[B.eqconv_tensor_t(*r, 0) for r in rows]), len(rows)


# host addresses stand in for device memory: the refusals below never read them
BASE = 1 << 20


@pytest.mark.parametrize("rows", [
    [(BASE, BASE, -1, 0)],                                            # negative length
    [(BASE, BASE, 4, 3)],                                             # unknown type
    [(None, BASE, 4, 0)],                                             # no input
    [(BASE, None, 4, 0)],                                             # no output
    [(BASE + 2, BASE + 2, 4, 0)],                                     # half an element off
    [(BASE, BASE, 8, 0), (BASE, BASE, 8, 0)],                         # the same tensor twice
    [(BASE, BASE, 8, 0), (BASE + 16, BASE + 16, 8, 0)],               # neighbours that overlap
    [(BASE, BASE + 16, 8, 0)],                                        # an output inside its own input
    [(BASE, BASE + 4096, 8, 0), (BASE + 64, BASE + 4100, 8, 0)],      # two outputs overlap
    [(BASE, BASE + 64, 8, 0), (BASE + 64, BASE + 128, 8, 0)],         # an output is another's input
])
def test_clip_refuses(rows):
    arr, n = _list(*rows)
    with pytest.raises(B.EqconvError) as e:
        B.eqconv_clip_gradients(n, arr, 1.0, 1e-6, BASE * 4, BASE * 8, 1 << 30, 0)
    assert e.value.status == B.EQCONV_ERR_INVALID_ARG


@pytest.mark.parametrize("max_norm,eps", [(-1.0, 1e-6), (float("nan"), 1e-6), (1.0, 0.0), (1.0, -1.0),
                                          (1.0, float("inf")), (1.0, float("nan"))])
def test_clip_refuses_bounds(max_norm, eps):
    arr, n = _list((BASE, BASE, 8, 0))
    with pytest.raises(B.EqconvError) as e:
        B.eqconv_clip_gradients(n, arr, max_norm, eps, BASE * 4, BASE * 8, 1 << 30, 0)
    assert e.value.status == B.EQCONV_ERR_INVALID_ARG


def test_clip_workspace():
    arr, n = _list((BASE, BASE, 1 << 20, 0), (BASE * 64, BASE * 64, 5, 1))
    need = B.eqconv_clip_workspace_bytes(n, arr)
    assert need > 0
    for ws, size in ((None, need), (BASE * 8, need - 1), (BASE * 8 + 8, need)):
        with pytest.raises(B.EqconvError) as e:
            B.eqconv_clip_gradients(n, arr, 1.0, 1e-6, BASE * 4, ws, size, 0)
        assert e.value.status == B.EQCONV_ERR_WORKSPACE
        with pytest.raises(B.EqconvError) as e:
            B.eqconv_gradient_norm(n, arr, BASE * 4, ws, size, 0)
        assert e.value.status == B.EQCONV_ERR_WORKSPACE
    bad, m = _list((BASE, BASE, -1, 0))
    assert B.eqconv_clip_workspace_bytes(m, bad) == 0


@pytest.mark.parametrize("n,type_", [(2 ** 45 // 4, 0), (2 ** 45 // 4 - 3, 0), (2 ** 45 // 2, 1), (2 ** 62, 2)])
def test_clip_refuses_tensors_beyond_a_launch(n, type_):
    """A tensor that no launch could take is refused, not looked for without end."""
    arr, m = _list((BASE, BASE, n, type_))
    assert B.eqconv_clip_workspace_bytes(m, arr) == 0
    for call in (lambda: B.eqconv_gradient_norm(m, arr, BASE * 4, BASE * 8, 1 << 30, 0),
                 lambda: B.eqconv_clip_gradients(m, arr, 1.0, 1e-6, BASE * 4, BASE * 8, 1 << 30, 0)):
        with pytest.raises(B.EqconvError) as e:
            call()
        assert e.value.status == B.EQCONV_ERR_INVALID_ARG
    ok, m = _list((BASE + 4, BASE + 4, 2 ** 45 // 4 - 4, 0))            # the longest, off the 16-byte boundary
    assert B.eqconv_clip_workspace_bytes(m, ok) > 0


def test_python_refusals():
    with pytest.raises(TypeError):
        layers.clip_gradients(torch.zeros(3), 1.0)
    with pytest.raises(ValueError):
        layers.clip_gradients([torch.zeros(3)], 1.0)             # not on a GPU
    with pytest.raises(TypeError):
        layers.gradient_norm([np.zeros(3)])
    with pytest.raises(ValueError):
        layers.BlockNorm("0e", 8, gate="relu")
    with pytest.raises(ValueError):
        layers.BlockNorm("0e", 8, dtype=torch.float64)
    with pytest.raises(ValueError):
        layers.Embedding(4, 8, dtype=torch.float64)
    with pytest.raises(ValueError):
        layers.Embedding(4, 8, padding=4)


def test_copies_have_plans_of_their_own(monkeypatch):
    """Copied and pickled operators: no plan is destroyed twice or used after."""
    alive, made = set(), []

    def create(*args):
        made.append(args)
        alive.add(len(made))
        return len(made)

    monkeypatch.setattr(B, "eqconv_embedding_plan_create", create)
    monkeypatch.setattr(B, "eqconv_block_norm_plan_create", create)
    monkeypatch.setattr(B, "eqconv_plan_destroy", lambda plan: alive.remove(plan) if plan in alive else twice.append(plan))
    monkeypatch.setattr(B, "eqconv_plan_info", lambda plan: {"D_in": 9})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    twice = []
    for op in (layers.Embedding(7, 12, torch.float32, torch.bfloat16, padding=3),
               layers.BlockNorm("0e+1o+2e", 8, gate="silu", eps=1e-5, dtype=torch.float16)):
        keep = [op]
        for again in (copy.copy, copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o))):
            keep.append(again(op))
            state = lambda o: {k: v for k, v in vars(o).items() if k != "plan"}  # noqa: E731
            assert state(keep[-1]) == state(op) and made[-1] == made[op.plan - 1]
        assert len({o.plan for o in keep}) == 4
        del op, again
        while keep:
            assert all(o.plan in alive for o in keep)
            keep.pop()
    assert not alive and not twice and len(made) == 8


@pytest.mark.parametrize("tensors,gated,backward", [(1, 0, 0), (2, 0, 0), (2, 1, 0),              # forward
                                                    (1, 0, 1), (2, 0, 1), (3, 1, 1), (4, 1, 1)])    # backward
@pytest.mark.parametrize("es", [2, 4])
def test_narrow_nodes_are_staged(es, tensors, gated, backward):
    """Nodes of few channels take the block norm's staged kernels, aligned or
    not, however few tensors a call has: the others are for nodes too large."""
    probe = os.path.join(os.path.dirname(os.path.abspath(B.__file__)), "libeqc_bulk_wait_probe.so")
    assert os.path.exists(probe), "not built (python -m equivariant_gnn_message_edge_b200.build_lib)"
    staged = ctypes.CDLL(probe).eqc_probe_block_norm_staged
    for C in [*range(1, 40), 63, 64, 65, 96, 100, 127, 128, 129, 130, 200, 255, 256]:
        for N in (1, 100, 5000, 20000, 200000):
            for L in (0, 1, 2):
                if L and C > 64:
                    continue
                for aligned in (0, 1):
                    assert staged(N, L, C, es, tensors, gated, backward, aligned) >= 1, (N, L, C, aligned)


def test_tensor_record_layout():
    assert ctypes.sizeof(B.eqconv_tensor_t) == 32
    assert [getattr(B.eqconv_tensor_t, f).offset for f in ("in_", "out", "n", "type")] == [0, 8, 16, 24]
