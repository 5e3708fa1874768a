"""Calls of one entry point from two host threads, each on a stream of its own: what a call asks of
its kernel (the shared memory of a launch among it) must not depend on the other thread's calls."""
import threading

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import int4_quantized_b200 as m

    m.lib()
    return m


def together(calls, rounds):
    """Makes each call (of one stream's raw handle) `rounds` times in a thread and on a stream of its own; all
    must return 0."""
    import torch

    torch.cuda.synchronize()
    codes, start = [set() for _ in calls], threading.Barrier(len(calls))
    streams = [torch.cuda.Stream() for _ in calls]

    def run(i):
        raw = streams[i].cuda_stream
        start.wait()
        for _ in range(rounds):
            codes[i].add(calls[i](raw))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}] * len(calls), codes


@pytest.mark.parametrize("bits", [32, 64])
def test_sorts_of_different_sizes(q4, bits):
    # 32 warps' histograms: 143 KB for 1024 experts, 56 KB for 400; the C entry point itself, which
    # Python calls without its lock, so that the threads are inside it together
    import torch

    g = torch.Generator(device="cuda").manual_seed(bits)
    dtype = torch.int32 if bits == 32 else torch.int64
    T, k = 600, 2
    cases, calls = [], []
    for E in (1024, 400, 900, 500):
        ids = torch.randint(-1, E, (T, k), device="cuda", generator=g).to(dtype)
        want = q4.moe_sort(ids, E)
        got = [torch.full_like(t, -9) for t in want]
        args = (ids.data_ptr(), bits, T, k, E, *(t.data_ptr() for t in got))
        cases.append((want, got, ids))
        calls.append(lambda stream, args=args: q4.lib().q4_moe_sort(*args, stream))
    together(calls, 20000)
    for want, got, _ in cases:
        for u, v in zip(got, want):
            assert torch.equal(u, v)


def test_first_cuda_call_of_a_thread(q4):
    # every entry point that a new thread may call before any other CUDA call of its own
    import torch

    g = torch.Generator(device="cuda").manual_seed(1)
    N, K = 256, 1024
    w = torch.randn(N, K, device="cuda", generator=g)
    payload, scales = q4.qpack(w, 4, 128)
    x, xb = torch.randn(1, K, device="cuda", generator=g), torch.randn(64, K, device="cuda", generator=g).bfloat16()
    xq, wq = q4.fp8_pack(x), q4.fp8_pack_weights(w)
    big, ids = q4.fp8_pack(xb), torch.randint(0, 4, (16, 2), device="cuda", generator=g)
    offsets = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    calls = [lambda: q4.qgemm(x, payload, scales, N, K, 4, 128), lambda: q4.qgemm(xb, payload, scales, N, K, 4, 128),
             lambda: q4.qpack(w, 8, 128)[0], lambda: q4.qdequant(payload, scales, (N, K), 4, 128),
             lambda: q4.fp8_gemm(*xq, *wq), lambda: q4.fp8_gemm(*big, *wq),
             lambda: q4.fp8_gemm_grouped(*big, wq[0][None], wq[1][None], offsets),
             lambda: q4.fp8_pack(x)[1], lambda: q4.fp8_pack_weights(w)[1], lambda: q4.moe_sort(ids, 4)[1],
             lambda: q4.moe_gather(xb, offsets[:1]), lambda: q4.moe_combine(xb, ids.int())]
    want = [c() for c in calls]
    got = [None] * len(calls)
    torch.cuda.synchronize()

    def run(i):
        try:
            got[i] = calls[i]()
        except Exception as e:  # noqa: BLE001 (shown below, in the test's own thread)
            got[i] = e

    for i in range(len(calls)):
        t = threading.Thread(target=run, args=(i,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert isinstance(a, torch.Tensor) and torch.equal(a, b), (i, a)


@pytest.mark.parametrize("bits", [4, 8])
def test_gemvs_of_different_lengths(q4, bits):
    # one row of x: a CTA's share of K, and with it the shared memory of the launch, differs
    import torch

    g = torch.Generator(device="cuda").manual_seed(bits)
    N = 256
    cases, calls = [], []
    for K in (4096, 11008, 2048, 28672):
        payload, scales = q4.qpack(torch.randn(N, K, device="cuda", generator=g), bits, 128)
        x = torch.randn(1, K, device="cuda", generator=g)
        want = q4.qgemm(x, payload, scales, N, K, bits, 128)
        y = torch.zeros_like(want)
        ws = torch.empty(max(256, q4.qgemm_workspace_bytes(1, N, K, bits, 128)), dtype=torch.uint8, device="cuda")
        args = (x.data_ptr(), q4.Q4_X_F32, 1, payload.data_ptr(), scales.data_ptr(), N, K, bits, 128, y.data_ptr(), ws.data_ptr(),
                ws.numel(), 0, None)
        cases.append((want, y, x, payload, scales, ws))
        calls.append(lambda stream, args=args: q4.lib().qgemm_ex(*args, stream))
    together(calls, 20000)
    for want, y, *_ in cases:
        assert torch.equal(y, want)
