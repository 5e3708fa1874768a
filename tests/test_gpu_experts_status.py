"""Fp8Experts' status word: only rows that an expert takes can set it, at every size of the call."""
import pytest

pytestmark = pytest.mark.gpu

D, F, E, K = 1024, 16, 16, 8
# packed in sorted order, and (2^25 values and more) each row once
SIZES = [60, 4200]


@pytest.fixture(scope="module")
def q4():
    import int4_quantized_b200 as m

    m.lib()
    return m


def batch(T, seed):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, D, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, E, (T, K), device="cuda", generator=g)
    return x, ids, torch.rand(T, K, device="cuda", generator=g)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", SIZES)
def test_padding_rows_do_not_report(q4, T, bad):
    import torch

    g = torch.Generator(device="cuda").manual_seed(1)
    layer = q4.Fp8Experts.pack(torch.randn(E, 2 * F, D, device="cuda", generator=g) / 32, torch.randn(E, D, F, device="cuda", generator=g) / 4)
    x, ids, w = batch(T, T)
    ids[5] = -1
    ids[T - 1] = E  # both kinds of padding: nothing of these tokens has an expert
    ids[7, 1:] = -1  # one choice left: a row that counts
    want = layer(x, ids, w)
    x[5, 900], x[T - 1, 0] = bad, bad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = layer(x, ids, w, status=status)
    assert int(status.item()) == 0
    assert torch.equal(out, want) and bool((out[5] == 0).all()) and bool((out[T - 1] == 0).all())
    x[7, 3] = bad
    layer(x, ids, w, status=status)
    assert int(status.item()) == q4.STATUS_NONFINITE


@pytest.mark.parametrize("T", SIZES)
def test_sorted_rows_report_alike(q4, T):
    import torch

    x, ids, _ = batch(T, T + 1)
    ids[3] = -1
    x[3] = float("nan")
    tokens, pos, offsets = q4.moe_sort(ids, E)
    n = int(offsets[-1])
    want = q4.fp8_pack(x, rows=tokens)
    for p in (pos, None):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = q4.Fp8Experts.sorted_rows(x, tokens, status, p)
        assert int(status.item()) == 0
        assert torch.equal(got[0][:n].view(torch.uint8), want[0][:n].view(torch.uint8)) and torch.equal(got[1][:n], want[1][:n])


@pytest.mark.parametrize("T", SIZES)
def test_captured_with_a_status_word(q4, T):
    # the status word's way takes nothing from the host: it can be captured, and reads the routing of each replay
    import torch

    g = torch.Generator(device="cuda").manual_seed(2)
    layer = q4.Fp8Experts.pack(torch.randn(E, 2 * F, D, device="cuda", generator=g) / 32, torch.randn(E, D, F, device="cuda", generator=g) / 4)
    x, ids, w = batch(T, T + 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    layer(x, ids, w, status=status)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = layer(x, ids, w, status=status)
    want = layer(x, ids, w)
    x[9] = float("nan")
    kept = ids[9].clone()
    ids[9] = -1
    graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and bool((out[9] == 0).all())
    others = [t for t in range(T) if t != 9]
    assert torch.equal(out[others], want[others])
    ids[9] = kept
    graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == q4.STATUS_NONFINITE


def test_sorted_rows_of_odd_length(q4):
    import torch

    x = torch.randn(4200, 1001, device="cuda").bfloat16()
    ids = torch.randint(0, E, (4200, K), device="cuda")
    tokens, pos, _ = q4.moe_sort(ids, E)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, want = q4.Fp8Experts.sorted_rows(x, tokens, status, pos), q4.fp8_pack(x, rows=tokens)
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
