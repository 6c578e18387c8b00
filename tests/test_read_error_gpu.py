"""Reading a workspace's error bits waits for the calls that may still set them, whatever their stream."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import split_kv_async_gb300 as F
    from rows_harness import ints


def test_reading_errors_waits_for_every_stream():
    # a call with a slot out of range, behind some 50 ms of work on a stream that the legacy stream does not wait for
    d, T = 64, 4
    p = F.make_rope_params(num_tokens=T, num_q_heads=2, num_kv_heads=1, head_dim=d, rot_dim=d, dtype=F.FDPP_BF16, num_slots=8)
    q, k = torch.randn(T, 2, d).bfloat16().cuda(), torch.randn(T, 1, d).bfloat16().cuda()
    cache = torch.zeros(8, 1, d, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 1, 2, 8], dtype=torch.int64, device="cuda")
    rope, ws = torch.as_tensor(F.fdpp_rope_table(d, 1e4)).cuda(), F.alloc_rope_workspace()
    pos, q_out, v_cache = ints([0] * T), torch.empty_like(q), torch.zeros_like(cache)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = lambda: F.fdpp_rope_append(q, k, k, pos, slots, rope, p, q_out, cache, v_cache, ws, stream=s)  # noqa: E731
    call()                                  # (the kernel is loaded at its first launch, which may wait for the GPU)
    assert F.fdpp_read_error(ws) == F.FDPP_ERRBIT_SLOT
    F.fdpp_workspace_init(ws)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    call()
    assert F.fdpp_read_error(ws) == F.FDPP_ERRBIT_SLOT
    assert s.query()


def test_reading_a_linears_errors_waits_for_every_stream():
    M, N, K = 8, 256, 256
    x, w = torch.randn(M, K).bfloat16().cuda(), torch.randn(N, K).bfloat16().cuda()
    y, ws, s = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), F.alloc_flat_gemm_workspace(M, N, K), torch.cuda.Stream()
    torch.cuda.synchronize()
    F.fdpp_flat_gemm(x, w, y, ws, stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    F.fdpp_flat_gemm(x, w, y, ws, stream=s)
    assert F.fdpp_flat_gemm_read_error(ws) == 0
    assert s.query()                        # the call is over
