"""Entry points called from host threads whose first CUDA call they are: such a thread has no current context yet, which
the tensor maps' encoder needs."""
import threading

import pytest
import torch

from gated_linear_attention_liger_b200 import ops
from tests.parity_util import assert_close, np64

pytestmark = pytest.mark.gpu


def _in_new_thread(call):
    got = []

    def body():
        try:
            got.append(call())
        except Exception as e:   # handed to the test's thread
            got.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    torch.cuda.synchronize()
    return got[0]


@pytest.mark.parametrize("entry", ["prefill", "backward", "full_causal", "cached"])
def test_first_cuda_call_of_a_host_thread(entry, cuda_device):
    """Through the C ABI, everything allocated and every stream made beforehand."""
    dev, lib, s = cuda_device, ops.load(), torch.cuda.Stream(cuda_device)
    g = torch.Generator(device=dev).manual_seed(30)
    q = torch.randn(1, 200, 4, 128, device=dev, generator=g).bfloat16()
    k, v = (torch.randn(1, 200, 2, 128, device=dev, generator=g).bfloat16() for _ in "kv")
    p = lambda t: t.data_ptr()  # noqa: E731
    if entry == "prefill":
        out, state = ops.prefill(q, k, v)
        ws = torch.empty(ops.prefill_workspace_size(1, 4, 2, 200, 128, 1), dtype=torch.uint8, device=dev)
        want, got = [out, state], [torch.empty_like(out), torch.empty_like(state)]
        call = lambda: lib.liger_attn_prefill(  # noqa: E731
            p(q), p(k), p(v), p(got[0]), p(got[1]), 1, 4, 2, 200, 128, 64, 0.5, ops.LIGER_BF16, None, None, 1, None, None,
            p(ws), ws.numel(), s.cuda_stream)
    elif entry == "backward":
        d_out = torch.randn(1, 200, 4, 128, device=dev, generator=g).bfloat16()
        want = list(ops.prefill_backward(q, k, v, d_out)[:3])
        got = [torch.empty_like(t) for t in want]
        ws = torch.empty(ops.prefill_backward_workspace_size(1, 4, 2, 200, 128, 1), dtype=torch.uint8, device=dev)
        call = lambda: lib.liger_attn_prefill_backward(  # noqa: E731
            p(q), p(k), p(v), p(d_out), None, None, 1, 4, 2, 200, 128, 64, 0.5, ops.LIGER_BF16, None, 1, p(got[0]), p(got[1]),
            p(got[2]), None, p(ws), ws.numel(), s.cuda_stream)
    elif entry == "full_causal":
        want = [ops.full_causal_attention(q, k, v)]
        got = [torch.empty_like(want[0])]
        call = lambda: lib.liger_attn_full_causal(  # noqa: E731
            p(q), p(k), p(v), p(got[0]), 1, 4, 2, 200, 128, ops.LIGER_BF16, None, 1, 0, s.cuda_stream)
    else:
        c = ops.kv_cache_new(13, 2, 128, 16, 1, 208, device=dev)
        lens, table = torch.full((1,), 200, dtype=torch.int32, device=dev), torch.arange(13, dtype=torch.int32, device=dev)[None]
        ops.kv_cache_append(k[0], v[0], torch.arange(200, dtype=torch.int32, device=dev), c["cache"], c["scales"])
        q1 = q[:, 0].contiguous()
        want = [ops.cached_attention(q1, c["cache"], c["scales"], table, lens)]
        got = [torch.empty_like(want[0])]
        ws = torch.empty(ops.cached_attention_workspace_size(128), dtype=torch.uint8, device=dev)
        call = lambda: lib.liger_attn_cached(  # noqa: E731
            p(q1), p(c["cache"]), p(c["scales"]), p(table), p(lens), p(got[0]), 1, 1, 4, 2, 128, 13, 13, 16, 512, ops.LIGER_BF16,
            ops.LIGER_KV_E4M3, p(ws), ws.numel(), s.cuda_stream)
    torch.cuda.synchronize()
    assert _in_new_thread(call) == ops.LIGER_OK
    for a, b in zip(got, want):
        if entry == "backward":   # (sums in shared memory whose order may differ)
            assert_close(np64(a), np64(b), torch.bfloat16, entry)
        else:
            assert torch.equal(a, b)
