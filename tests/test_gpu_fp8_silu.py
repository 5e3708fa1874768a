"""fp8_pack(silu_mul=True) where gates are far below zero, against 64 bits.

Blocks of such gates alone: their values are small, but their own largest one sets the scale, so
that a value lost shows. The documented bound of a value is (10 + 1.2 |gate|) 2^-23 relative; a
scale is the largest value / 448, rounded once more (2^-24, or half of the smallest subnormal
number); a code is off by at most half a step, 2^-4 of the value or 2^-10 of the scale, and the
value's, the scale's and the quotient's own errors (below 2^-14 together) move that by less than 1 %.
"""
import numpy as np
import pytest

from oracle import fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import int4_quantized_b200 as m

    m.lib()
    return m


def check(q4, x):
    """x [M, 2K] on the GPU: scales and codes within their bounds."""
    import torch

    K = x.shape[1] // 2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = q4.fp8_pack(x, silu_mul=True, status=status)
    assert int(status.item()) == 0
    xn = x.double().cpu().numpy()
    h = fp8.silu_mul(xn)
    rel = (10 + 1.2 * np.abs(xn[:, :K])) * 2.0 ** -23
    cuts = range(128, K, 128)
    most = np.stack([np.abs(p).max(1) for p in np.split(h, cuts, axis=1)], 1) / 448
    slack = np.stack([(np.abs(p) * r).max(1) for p, r in zip(np.split(h, cuts, axis=1), np.split(rel, cuts, axis=1))], 1) / 448
    s = scales.cpu().numpy().astype(np.float64)
    assert most.min() > 2.0 ** -140  # every block has a scale of its own
    assert np.all(np.abs(s - most) <= slack * 1.01 + most * 2.0 ** -24 + 2.0 ** -150)
    got = fp8.dequant(codes.view(torch.uint8).cpu().numpy(), s)
    # 2^-150 of the scale's rounding counts 448 times at the most
    assert np.all(np.abs(got - h) <= (2.0 ** -4 * np.abs(h) + 2.0 ** -10 * fp8.spread(s, K, 1)) * 1.01 + 448 * 2.0 ** -150)


# (gate, magnitude of up): values from 1e-35 to 1e4
FAR = [(-86.5, 1.0), (-87.5, 1e4), (-88.5, 1e10), (-88.8, 1.0), (-95.0, 1e5), (-100.0, 1e38), (-120.0, 1e30), (-150.0, 1e35), (-172.0, 3e38)]


def far_rows(rng, M, K, cases):
    gate, up = np.empty((M, K)), np.empty((M, K))
    for m in range(M):
        for b in range(0, K, 128):
            g, u = cases[(m + b // 128) % len(cases)]
            n = min(128, K - b)
            gate[m, b:b + n] = g + rng.uniform(-0.5, 0.5, n)
            up[m, b:b + n] = u * rng.uniform(0.1, 1, n) * rng.choice([-1, 1], n)
    return np.concatenate([gate, up], 1).astype(np.float32)


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(9, 128), (4, 1000), (9, 1152), (2400, 1024), (2400, 1001)])
def test_far_gates_alone(q4, x_type, M, K):
    import torch

    cases = [c for c in FAR if x_type != "f16" or c in ((-86.5, 1.0), (-87.5, 1e4))]
    x = torch.from_numpy(far_rows(np.random.default_rng(M + K), M, K, cases))
    check(q4, x.to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[x_type]).cuda())


@pytest.mark.parametrize("at", [0, 15, 16, 127])
def test_one_far_gate_among_others(q4, at):
    # its large up makes the far value the block's largest, beside gates of every size
    import torch

    rng = np.random.default_rng(at)
    x = torch.from_numpy(rng.normal(0, 2, (3, 256)).astype(np.float32))
    x[:, 128:] *= 1e-6
    x[1, at], x[1, 128 + at] = -90.0, 1e38
    check(q4, x.cuda())


def test_row_list_with_far_gates(q4):
    # rows by index: the far gates are those of the row taken; rows that are left out stay as they were
    import torch

    x = torch.from_numpy(far_rows(np.random.default_rng(3), 9, 256, FAR)).cuda()
    rows = torch.tensor([8, -1, 3, 3, 0, 9], dtype=torch.int32, device="cuda")
    codes = torch.full((6, 256), 7.0, device="cuda").to(torch.float8_e4m3fn)
    scales = torch.full((6, 2), -1.0, device="cuda")
    q4.fp8_pack(x, rows=rows, silu_mul=True, codes=codes, scales=scales)
    want, ws = q4.fp8_pack(x, silu_mul=True)
    seven = torch.full((256,), 7.0, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    for i, r in enumerate(rows.tolist()):
        inside = 0 <= r < 9
        assert torch.equal(codes[i].view(torch.uint8), want[r].view(torch.uint8) if inside else seven)
        assert torch.equal(scales[i], ws[r] if inside else torch.full((2,), -1.0, device="cuda"))


@pytest.mark.parametrize("gate,up", [(float("-inf"), 1.0), (-100.0, float("inf")), (-300.0, float("-inf")), (float("nan"), 1.0)])
def test_nonfinite_far_gates_are_reported(q4, gate, up):
    import torch

    x = torch.ones(2, 512, device="cuda")
    x[1, 7], x[1, 256 + 7] = gate, up
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q4.fp8_pack(x, silu_mul=True, status=status)
    assert int(status.item()) == q4.STATUS_NONFINITE


def test_gates_too_far_for_any_up_give_zero(q4):
    # below -182 the largest up leaves less than 2^-126: 0, with the scale of an empty block
    import torch

    x = torch.full((1, 256), 3e38, device="cuda")
    x[0, :128] = torch.linspace(-3e38, -200, 128)
    codes, scales = q4.fp8_pack(x, silu_mul=True)
    assert bool((codes.float() == 0).all()) and bool((scales == 1).all())


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("M,K", [(9, 200), (9, 256), (2400, 1024)])
@pytest.mark.parametrize("at", [1, 3, 6])
def test_rows_at_any_byte(q4, x_type, silu, M, K, at):
    # "any alignment": rows that do not begin at a whole element, through the C entry point
    import torch

    dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[x_type]
    cases = [c for c in FAR if x_type != "f16" or c in ((-86.5, 1.0), (-87.5, 1e4))] + [(0.0, 1.0), (3.0, 1.0)]
    rows = far_rows(np.random.default_rng(at), M, K, cases)
    x = torch.from_numpy(rows if silu else rows[:, K:].copy()).to(dtype).cuda()
    want = q4.fp8_pack(x, silu_mul=silu)
    n = x.numel() * x.element_size()
    raw = torch.zeros(n + 16, dtype=torch.uint8, device="cuda")
    raw[at:at + n] = x.view(torch.uint8).view(-1)
    codes = torch.zeros(M * K + 16, dtype=torch.uint8, device="cuda")
    scales = torch.zeros_like(want[1])
    torch.cuda.synchronize()
    code = q4.lib().q4_fp8_pack(raw.data_ptr() + at, {"f32": 0, "bf16": 1, "f16": 2}[x_type], M, K, None, M, None, int(silu),
                                codes.data_ptr() + at, scales.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
    assert code == 0
    assert torch.equal(scales, want[1])
    assert torch.equal(codes[at:at + M * K].view(M, K), want[0].view(torch.uint8))
    assert int(codes[:at].sum()) == 0 and int(codes[at + M * K:].sum()) == 0
