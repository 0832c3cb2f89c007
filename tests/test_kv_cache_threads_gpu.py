"""The paged 8-bit cache's operators called from two host threads at once (what the header allows as long as no output is
shared): calls of one kernel that need different amounts of shared memory.  The threads call the C ABI, where hardly any
time passes in the interpreter, so that the calls themselves overlap."""
import threading

import numpy as np
import pytest
import torch

from gated_linear_attention_liger_b200 import ops
from tests import kv_reference as ref
from tests.test_kv_cache_gpu import BF16, E4M3, _attention_case, _close, _state, i32

pytestmark = pytest.mark.gpu


def _from_threads(calls):
    """The statuses of each list of calls (function, arguments), made by a host thread of its own; all start together."""
    start, statuses = threading.Barrier(len(calls)), [None] * len(calls)

    def loop(at):
        torch.cuda.set_device(0)
        start.wait()
        statuses[at] = [fn(*args) for fn, args in calls[at]]

    threads = [threading.Thread(target=loop, args=(at,)) for at in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return statuses


def test_attention_from_two_host_threads(cuda_device):
    rng = np.random.default_rng(26)
    dev, lib, times, calls, outs, wants, keep = cuda_device, ops.load(), 3000, [], [], [], []
    for B in (64, 256):
        lens = [int(x) for x in rng.integers(0, 40, B)]
        cache, scales, table, values, s64 = _attention_case(rng, lens, 1, 16, 128, E4M3, dev)
        q = torch.tensor(rng.normal(size=(B, 4, 128))).to(BF16)
        args = (q.to(dev), cache, scales, i32(table, dev), i32(lens, dev))
        wants.append(ops.cached_attention(*args))
        _close(wants[-1], ref.attention(q[:, None].double().numpy(), values, s64, table, lens), BF16, 128)
        out = torch.full((times, B, 4, 128), float("nan"), dtype=BF16, device=dev)
        ws, stream = torch.empty(ops.cached_attention_workspace_size(128), dtype=torch.uint8, device=dev), torch.cuda.Stream(dev)
        calls.append([(lib.liger_attn_cached, [t.data_ptr() for t in args] + [
            o.data_ptr(), B, 1, 4, 1, 128, table.shape[1], cache.shape[0], 16, 4 * 128, ops.LIGER_BF16, ops.LIGER_KV_E4M3,
            ws.data_ptr(), ws.numel(), stream.cuda_stream]) for o in out])
        outs.append(out)
        keep.append((args, ws, stream))
    torch.cuda.synchronize()
    for st in _from_threads(calls):
        assert set(st) == {ops.LIGER_OK}, st.count(ops.LIGER_OK)
    for out, want in zip(outs, wants):
        assert torch.equal(out, want.expand_as(out))


def test_assign_from_two_host_threads(cuda_device):
    rng = np.random.default_rng(27)
    dev, lib, times, calls, outs, wants, keep = cuda_device, ops.load(), 3000, [], [], [], []
    for B in (3000, 8192):
        lens = [int(x) for x in rng.integers(0, 40, B)]
        new = [int(x) for x in rng.choice([-1, 0, 1, 2], B)]
        table, ring, span = _state(rng, B, 4, 16, lens, B)
        t = [i32(x, dev) for x in (new, lens, table, ring, span)]
        N = 2 * B
        want = ref.assign(new, lens, [list(r) for r in table], list(ring), span, 16, N)[0]
        out = torch.full((times, N), -9, dtype=torch.int32, device=dev)
        other, stream = [torch.empty(B + 1, dtype=torch.int32, device=dev), torch.empty_like(t[1]), torch.empty_like(t[4])], torch.cuda.Stream(dev)
        calls.append([(lib.liger_kv_cache_assign, [x.data_ptr() for x in t + [o] + other] + [
            B, 4, len(ring), 16, N, stream.cuda_stream]) for o in out])
        outs.append(out)
        wants.append(i32(want, dev))
        keep.append((t, other, stream))
    torch.cuda.synchronize()
    for st in _from_threads(calls):
        assert set(st) == {ops.LIGER_OK}, st.count(ops.LIGER_OK)
    for out, want in zip(outs, wants):
        assert torch.equal(out, want.expand_as(out))
