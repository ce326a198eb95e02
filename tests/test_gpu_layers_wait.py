"""The block norm's bounded waits for its bulk copies give up, report and return
(needs a B200).

A test-only build of the kernels (csrc/testing/eqc_bulk_wait_probe.cu: every
phase expects 16 bytes more than its copies carry, and a wait ends after 2 ms)
can never see a copy complete.  Its launches must set status bit 4 and return
promptly, and the library's own block norm must give the same results
afterwards as before.  Nothing here faults or hangs the GPU: the copies are in
bounds and land, and every wait is bounded in time."""
import ctypes
import os
import time

import pytest
import torch

from equivariant_gnn_message_edge_b200 import binding as B
from equivariant_gnn_message_edge_b200 import layers
from equivariant_gnn_message_edge_b200.workloads import natural_irreps

pytestmark = pytest.mark.gpu

PROBE = os.path.join(os.path.dirname(os.path.abspath(B.__file__)), "libeqc_bulk_wait_probe.so")


@pytest.mark.parametrize("N,L,C", [
    (900, 2, 64),       # a warp a node
    (900, 2, 37),       # the same off the 16-byte boundaries
    (5000, 0, 64),      # several rows a slot
    (300, 1, 512),      # a CTA a node
    (300, 2, 301),      # the same off the boundaries
    (700, 0, 4096),     # wide rows
    (700, 0, 1031),
])
def test_waits_that_cannot_end(N, L, C):
    assert os.path.exists(PROBE), "libeqc_bulk_wait_probe.so not built (python -m equivariant_gnn_message_edge_b200.build_lib)"
    lib = ctypes.CDLL(PROBE)
    run = lib.eqc_probe_block_norm
    run.argtypes = [ctypes.c_int] * 4 + [ctypes.c_void_p] * 2
    assert all(lib.eqc_probe_block_norm_staged(N, L, C, 2, t, 1, back, 1) for t, back in ((2, 0), (4, 1)))
    g = torch.Generator(device="cuda").manual_seed(N + C)
    bf = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    x, b, gx, gh = (bf(N, (L + 1) ** 2, C) for _ in range(4))
    gate, wo, wi = bf(N, L + 1, C), torch.ones(L + 1, C, device="cuda"), torch.ones(L + 1, C, device="cuda")
    op = layers.BlockNorm(natural_irreps(L), C, dtype=torch.bfloat16)

    def own():
        xo, h, st = op.forward_raw(x, b, gate, wo, wi, save=True)
        return [xo, h, st, *op.backward_raw(x, b, gate, wo, wi, st, gx, gh)]

    before = own()
    outs = [torch.empty_like(t) for t in before]
    ws = torch.empty(B.eqconv_block_norm_workspace_bytes(op.plan, N), dtype=torch.uint8, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for backward in (0, 1):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        stats = before[2] if backward else outs[2]
        tensors = [x, b, gate, wo, wi, outs[0], outs[1], stats, gx, gh, *outs[3:], ws, status]
        p = (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])
        torch.cuda.synchronize()
        t0 = time.monotonic()
        rc = run(N, L, C, backward, p, stream)
        assert rc == 0, f"launch failed: {rc}"
        torch.cuda.synchronize()
        elapsed = time.monotonic() - t0
        assert int(status.item()) & 4, "the wait that timed out was not reported"
        assert elapsed < 5.0, f"the kernel took {elapsed:.1f} s to give up"
    assert all(torch.equal(a, c) for a, c in zip(before, own()))
    assert B.eqconv_get_device_error(op.plan) == B.EQCONV_OK
