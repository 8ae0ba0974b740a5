"""Streams given as handles to the calls around a step: 0 is the default stream, whose
earlier work the call follows."""
import pytest
import torch

from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("handle", [0, "current"])
def test_handle_of_the_default_stream(handle):
    """The inputs are written on the default stream, behind 50 ms of other work."""
    torch.cuda.synchronize()
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    if handle == "current":
        handle = torch.cuda.current_stream().cuda_stream
    S, nq, nkv, d = 3, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.randn(S, n, d, device="cuda", dtype=torch.bfloat16, generator=g)
            for n in (nq, nkv, nkv)]
    kc, vc = (torch.randn(8, 16, nkv, d, device="cuda", dtype=torch.bfloat16, generator=g)
              for _ in range(2))
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    lens, new, tables = _i32([16, 5, 30]), _i32([1] * S), _i32([[0, 1], [2, -1], [3, 4]])
    free, count, starts, slots = _i32([7, 6, 5] + [0] * 5), _i32([3]), _i32([0, 1, 2, 3]), \
        _i32([9, 40, 77])
    late = [x.clone() for x in (*rows, lens)]
    ws = ops.alloc_workspace(S, S, nq, nkv, d, 1, 32)

    def calls(stream):
        t, c = tables.clone(), count.clone()
        q, k, v, n = late
        return (ops.rotary_reshape_and_cache(q, k, v, n, f, k2, v2, slots, stream=stream),
                ops.paged_attention_window(q, kc, vc, tables, n, starts, 0.125, window=9,
                                           max_q_len=1, max_seq_len=32, workspace=ws,
                                           stream=stream),
                *ops.build_step(n, new, t, free, c, block_size=16, num_tokens=S, stream=stream))
    want = [x.clone() for x in calls(None)]
    for x in late:
        x.zero_()
    late[3].fill_(1)
    calls(handle)  # whatever the call allocates is there
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for x, y in zip(late, (*rows, lens)):
        x.copy_(y)
    got = calls(handle)
    torch.cuda.synchronize()
    ops.check_device_errors()
    for x, y in zip(got, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
