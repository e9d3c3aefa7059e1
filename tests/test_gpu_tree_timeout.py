"""The bounded waits of the tensor-core tree decode, on the GPU, without a fault.

la_test_timeout_next_tree makes the next tensor-core tree decode wait for a copy
of the state that never counts as complete (16 bytes more are expected than
come). Its waits must give up after the kernels' limit (2 s), no row of the
output may be stored, and the per-device status word must read LA_ERR_TIMEOUT.
The context stays usable: the next call runs normally and matches the oracle.
"""

import time

import numpy as np
import pytest

import causal_linear_attention_la_gb300 as la
from causal_linear_attention_la_gb300 import synth
from helpers import TOL, build_lib, rel_err, to_dev, to_host
from oracle import spec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build_lib()
    la.lib()


# up to 16 nodes (the whole state in one copy), up to 32 and 48 (slabs in a ring
# of their own), up to 64 (the ring where the keys were); two slabs and more
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("T,d", [(9, 128), (24, 128), (24, 64), (40, 128), (64, 128), (64, 64)])
def test_tree_wait_gives_up_and_the_next_call_runs(T, d, delta):
    import torch
    q, k, v = synth.qkv(1, 1, T, d, d, seed=T + d, dtype="bf16")
    if delta:
        k = synth.round_to_bf16(k / np.linalg.norm(k, axis=-1, keepdims=True))
    rng = np.random.default_rng(T)
    S = rng.standard_normal((1, 1, d, d)).astype(np.float32)
    z = rng.random((1, 1, d)).astype(np.float32) + 1
    parent = (np.arange(T) - 1) // 2 * (np.arange(T) > 0) - (np.arange(T) == 0)
    assert la.la_tree_path(d, d, la.LA_BF16) == 1
    args = [to_dev(x, "bf16") for x in (q, k, v)] + [torch.from_numpy(parent[None].astype(np.int32)).cuda()]
    Sd, zd = torch.from_numpy(S).cuda(), torch.from_numpy(z).cuda()

    def call(out):
        return la.decode_tree_delta(Sd, *args, out=out) if delta else la.decode_tree(Sd, zd, *args, out=out)

    got = call(torch.zeros_like(args[2]))            # warm: attributes, tensor maps
    torch.cuda.synchronize()
    assert la.la_device_status(True) == la.LA_OK
    la.la_test_timeout_next_tree()
    out = torch.full_like(args[2], 7.0)
    t0 = time.perf_counter()
    call(out)
    torch.cuda.synchronize()
    waited = time.perf_counter() - t0
    assert la.la_device_status(True) == la.LA_ERR_TIMEOUT
    assert 1.5 < waited < 30.0, waited
    assert torch.all(out == 7.0), "nothing is stored without the state"
    # the switch was one-shot and the context is intact
    again = call(torch.zeros_like(args[2]))
    torch.cuda.synchronize()
    assert la.la_device_status(True) == la.LA_OK
    assert torch.equal(got, again)
    want = spec.decode_tree_delta(S, q, k, v, parent[None])[0] if delta else spec.decode_tree(S, z, q, k, v, parent[None])[0]
    assert rel_err(to_host(again), want, np.abs(want).max()) <= TOL["bf16"]
