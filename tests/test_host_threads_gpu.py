"""Calls from host threads.

A thread's first CUDA call may be one of the library's: it passes, on the device's primary context.

Two threads call the same operator at once, each on its own stream with buffers of its own, at sizes
whose kernels need different amounts of shared memory: every call passes, and gives the bits of a call alone.
Each set of calls runs in a process of its own, so that nothing that the library keeps of the device (which
clusters fit) is there when the threads begin."""
import hashlib
import json
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
REPEATS = 3000
KINDS = ("scaled_gemm", "flat_gemm", "attention_sync", "attention_tcgen05")


def _call(kind, which):
    """A call of this kind as (function of a stream, output, function that gives its error bits)."""
    import split_kv_async_gb300 as F
    gen = torch.Generator("cuda").manual_seed(7 + which)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").bfloat16()

    if kind == "scaled_gemm":            # 33 to 48 and 49 to 64 rows share a kernel
        M, N, K = (40, 64, 150)[which], 512, 1024
        byte = lambda r: (100 * rnd(r, K).float()).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        x, w = byte(M), byte(N)
        x, w = (torch.where((t & 0x7F) == 0x7F, 0, t).contiguous() for t in (x, w))
        sx, sw = torch.rand(M, K // 128, generator=gen, device="cuda"), torch.rand(N // 128, K // 128, generator=gen, device="cuda")
        p = F.make_scaled_gemm_params(M=M, N=N, K=K)
        ws, y = F.alloc_scaled_gemm_workspace(p), torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        return lambda s: F.fdpp_scaled_gemm(x, sx, w, sw, p, ws, y, stream=s), y, lambda: F.fdpp_read_error(ws)
    if kind == "rows":
        T, L = 40, 300
        q, k, v = rnd(T, 8, 128), rnd(1, L, 2, 128), rnd(1, L, 2, 128)
        lens, out = torch.full((1,), L, dtype=torch.int32, device="cuda"), torch.zeros_like(q)
        p = F.make_rows_params(batch=1, num_q_heads=8, num_kv_heads=2, head_dim=128, dtype=F.FDPP_BF16, num_tokens=T, max_seq_len=L,
                               scale=128 ** -0.5, kernel=F.FDPP_KERNEL_TENSOR)
        ws = F.alloc_rows_workspace(p)
        return lambda s: F.fdpp_rows_attn(q, k, v, None, lens, None, p, ws, out, stream=s), out, lambda: F.fdpp_read_error(ws)
    if kind == "flat_gemm":
        M, N, K = (8, 128)[which], 512, 1024
        x, w, y = rnd(M, K), rnd(N, K), torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        ws = F.alloc_flat_gemm_workspace(M, N, K)
        return lambda s: F.fdpp_flat_gemm(x, w, y, ws, stream=s), y, lambda: F.fdpp_flat_gemm_read_error(ws)
    B, hq, hkv, d, L = (1, 64)[which], 16 if kind == "attention_tcgen05" else 8, 1, 128, 256
    q, k, v = rnd(B, hq, d), rnd(B, L, hkv, d), rnd(B, L, hkv, d)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    p = F.make_params(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=F.FDPP_BF16, max_seq_len=L, scale=d ** -0.5,
                      kernel=F.FDPP_KERNEL_TENSOR,
                      tc_mma=F.FDPP_TC_MMA_TCGEN05 if kind == "attention_tcgen05" else F.FDPP_TC_MMA_AUTO)
    ws, out = F.alloc_workspace(p), torch.zeros_like(q)
    return (lambda s: F.fdpp_decode_attn(q, k, v, None, lens, p, ws, out, stream=s), out,
            lambda: F.fdpp_read_diag(ws, p)[0]["error_bits"])


@pytest.mark.parametrize("kind,which", [("scaled_gemm", 0), ("scaled_gemm", 2), ("flat_gemm", 0), ("rows", 0), ("attention_sync", 0),
                                        ("attention_tcgen05", 1)])
def test_first_call_of_a_thread(kind, which):
    call, out, error_bits = _call(kind, which)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    call(stream)
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    raised = []

    def work():
        try:
            call(stream)
        except Exception as e:
            raised.append(str(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not raised and error_bits() == 0, raised
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def child(at_once):
    report = {}
    for kind in KINDS:
        calls = [_call(kind, which) for which in (0, 1)]
        streams = [torch.cuda.Stream() for _ in calls]
        torch.cuda.synchronize()
        failed = []
        start = threading.Barrier(2)

        def work(call, stream):
            if at_once:
                start.wait()
            for i in range(REPEATS if at_once else 1):
                try:
                    call(stream)
                except Exception as e:
                    failed.append(str(e))
                if i % 200 == 199:
                    stream.synchronize()

        threads = [threading.Thread(target=work, args=(c[0], s)) for c, s in zip(calls, streams)]
        for t in threads:
            t.start()
            if not at_once:
                t.join()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        failures = len(failed)
        for c, s in zip(calls, streams):         # and once more, alone
            c[0](s)
        torch.cuda.synchronize()
        bits = [hashlib.sha256(out.view(torch.int16).cpu().numpy().tobytes()).hexdigest() for _, out, _ in calls]
        report[kind] = dict(failures=failures, first=failed[:1], bits=bits, errors=[e() for _, _, e in calls])
    print("REPORT " + json.dumps(report))


def _run(at_once):
    code = f"import sys; sys.path[:0] = [{os.path.dirname(HERE)!r}, {HERE!r}]; import test_host_threads_gpu as t; t.child({at_once})"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    lines = [x for x in r.stdout.splitlines() if x.startswith("REPORT ")]
    assert r.returncode == 0 and lines, r.stdout[-2000:] + r.stderr[-2000:]
    return json.loads(lines[0][7:])


@pytest.fixture(scope="module")
def reports():
    return _run(False), _run(True)


@pytest.mark.parametrize("kind", KINDS)
def test_calls_of_two_threads_at_once(reports, kind):
    alone, together = (r[kind] for r in reports)
    assert alone["failures"] == 0, alone["first"]
    assert alone["errors"] == [0, 0]
    assert together["failures"] == 0, (together["failures"], together["first"])
    assert together["errors"] == [0, 0]
    assert together["bits"] == alone["bits"]
