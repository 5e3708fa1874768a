"""The tile shapes of fp8_gemm and the lane layouts of fp8_pack that large calls take.

Which sizes reach which tiles is wide_shape's choice in csrc/fp8_plan.h (148 SMs): a dense product of
333 rows and N of 9473 to 12544 is one round of 128 x 256 tiles and two of the others; pairs of CTAs
make products of three rounds and more. K from one block of 128 to more than any ring holds, and
ragged.

Products are compared, all of y, with float64 products of the same codes on the GPU. Within a block
of 128 the products are exact and each of at most 128 additions is off by at most 2^-23 of the
magnitudes' sum; so are, for every block, the product of the two scales and the fma; a split K
adds at most 8 more. Then half a step of y's type, and of fp16's subnormal numbers. The float64
side (sums of up to 5000 terms: 5000 x 2^-53) is nothing beside that.
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


def dt(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def codes(gen, rows_per_scale, *shape):
    """Random codes with scales that differ from block to block (whose sum no mix-up of blocks leaves alone)."""
    import torch

    c = (torch.randn(*shape, device="cuda", generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    kb = -(-shape[-1] // 128)
    rows = -(-shape[-2] // rows_per_scale)
    s = torch.exp(torch.randn(*shape[:-2], rows, kb, device="cuda", generator=gen)) / 1000
    return c, s


def product(x, xs, w, ws):
    """(y, sum of magnitudes) in float64 of [M, K] and [N, K] codes."""
    import torch

    b = torch.arange(x.shape[1], device="cuda") // 128
    a = x.double() * xs.double()[:, b]
    v = w.double() * ws.double()[torch.arange(w.shape[0], device="cuda") // 128][:, b]
    return a @ v.t(), a.abs() @ v.abs().t()


def check(y, ref, K, y_type):
    import torch

    y64, mag = ref
    half = torch.finfo(dt(y_type)).eps / 2
    lim = 2.0 ** -23 * (128 + 2 * -(-K // 128) + 8) * mag * (1 + half) + half * y64.abs() + (2.0 ** -25 if y_type == "f16" else 2.0 ** -134)
    bad = (y.double() - y64).abs() > lim
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"
    assert bool(y.isfinite().all())


@pytest.mark.parametrize("y_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [
    (333, 11008, 4096), (333, 10001, 1040), (300, 12000, 144), (257, 11008, 640), (300, 9473, 1040),  # 128 x 256
    (300, 9472, 2064), (300, 9471, 1040),
    (1500, 9472, 656), (1411, 9328, 4096), (1511, 9471, 400), (2045, 6152, 2064),  # pairs
    (512, 4096, 4096), (200, 4104, 1936), (700, 2305, 5008),                       # 128 x 128
])
def test_gemm_tiles(q4, M, N, K, y_type):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    x, xs = codes(gen, 1, M, K)
    w, ws = codes(gen, 128, N, K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((M + 2, N), 3.0, device="cuda", dtype=dt(y_type))
    q4.fp8_gemm(x, xs, w, ws, out=out[1:M + 1], status=status)
    assert int(status.item()) == 0
    check(out[1:M + 1], product(x, xs, w, ws), K, y_type)
    assert bool((out[0] == 3).all()) and bool((out[M + 1] == 3).all())
    again = q4.fp8_gemm(x, xs, w, ws, out_dtype=dt(y_type))
    assert torch.equal(again, out[1:M + 1])


@pytest.mark.parametrize("y_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("counts,N,K", [
    ([8, 0, 11, 13], 9472, 2064), ([1, 2, 30, 0], 9470, 272), ([4] * 8, 4736, 4096),  # few rows: 128 x 256
    ([700, 0, 513, 1300], 1408, 1936), ([2048, 600], 2304, 656), ([130, 60, 0, 257, 1], 1408, 2064),
    ([900, 1100], 9001, 400), ([2047, 2050], 2312, 2064), ([1500, 1500, 1200, 1], 2340, 1936),  # pairs
])
def test_grouped_tiles(q4, counts, N, K, y_type):
    import torch

    E, R = len(counts), sum(counts)
    gen = torch.Generator(device="cuda").manual_seed(R + N + K)
    x, xs = codes(gen, 1, R + 3, K)
    w, ws = codes(gen, 128, E, N, K)
    at = np.concatenate([[0], np.cumsum(counts)])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((R + 3, N), 3.0, device="cuda", dtype=dt(y_type))
    q4.fp8_gemm_grouped(x, xs, w, ws, torch.from_numpy(at.astype(np.int32)).cuda(), out=out, status=status)
    assert int(status.item()) == 0
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if b > a:
            check(out[a:b], product(x[a:b], xs[a:b], w[e], ws[e]), K, y_type)
    assert bool((out[R:] == 3).all())


@pytest.mark.parametrize("N,off", [(2304, 0), (2312, 0), (2312, 8), (2312, 3), (2305, 0), (2320, 5)])
def test_pairs_write_their_rows_only(q4, N, off):
    # full and partial groups of 32 rows, rows of whole and of partial 16-byte units, y at an offset, the
    # rows of no expert and all around y as they were; twice, the second over the first's answers
    import torch

    counts, head, tail, K = [2047, 0, 2050], 2, 5, 144
    at = np.concatenate([[head], head + np.cumsum(counts)])
    R = int(at[-1]) + tail
    gen = torch.Generator(device="cuda").manual_seed(N + off)
    x, xs = codes(gen, 1, R, K)
    w, ws = codes(gen, 128, 3, N, K)
    for y_type in ("bf16", "f16", "f32"):
        buf = torch.full((R * N + 64,), 5.0, device="cuda", dtype=dt(y_type))
        y = buf[off:off + R * N].view(R, N)
        for _ in range(2):
            q4.fp8_gemm_grouped(x, xs, w, ws, torch.from_numpy(at.astype(np.int32)).cuda(), out=y)
        for e, (a, b) in enumerate(zip(at, at[1:])):
            if b > a:
                check(y[a:b], product(x[a:b], xs[a:b], w[e], ws[e]), K, y_type)
        assert bool((y[:head] == 5).all()) and bool((y[R - tail:] == 5).all())
        assert bool((buf[:off] == 5).all()) and bool((buf[off + R * N:] == 5).all())


@pytest.mark.parametrize("M,N,K", [(333, 11008, 656), (300, 9472, 656), (1500, 9472, 656)])
def test_large_tiles_keep_bad_rows_apart(q4, M, N, K):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(M)
    x, xs = codes(gen, 1, M, K)
    w, ws = codes(gen, 128, N, K)
    ref = product(x, xs, w, ws)
    x.view(torch.uint8)[130, 600] = 0x7F
    xs[7, 4] = float("inf")
    y = q4.fp8_gemm(x, xs, w, ws)
    keep = [m for m in range(M) if m not in (7, 130)]
    assert bool(y[130].isnan().all()) and not bool(y[7].isfinite().any())
    check(y[keep], (ref[0][keep], ref[1][keep]), K, "bf16")


# ---- packing: two blocks a group of lanes, from 18944 blocks on -----------------------------------
def values(rng, M, K):
    x = rng.normal(0, 1, (M, K))
    x[:, ::97] *= 8
    x[rng.random((M, K)) < 0.02] = 0
    return x.astype(np.float32)


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(2400, 1024), (2400, 1001), (150, 16400), (19000, 65)])
def test_pack_many_rows(q4, x_type, M, K):
    import torch

    x = torch.from_numpy(values(np.random.default_rng(K), M, K)).to(dt(x_type))
    got, scales = q4.fp8_pack(x.cuda())
    rc, rs = fp8.pack(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(got.view(torch.uint8).cpu().numpy(), rc)


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(2400, 1024), (2400, 1001), (700, 4096)])
def test_pack_many_rows_silu(q4, x_type, M, K):
    # a value's relative error is below (10 + 1.2 x 16) 2^-23 < 2^-18 for gates within 16; a scale's,
    # with its own rounding, that and 2^-24; a code's half a step, which they move by less than 1 %
    import torch

    x = np.clip(np.random.default_rng(K).normal(0, 3, (M, 2 * K)), -16, 16).astype(np.float32)
    x = torch.from_numpy(x).to(dt(x_type))
    got, scales = q4.fp8_pack(x.cuda(), silu_mul=True)
    h = fp8.silu_mul(x.double().numpy())
    s = scales.cpu().numpy().astype(np.float64)
    want = np.stack([np.abs(p).max(1) for p in np.split(h, range(128, K, 128), axis=1)], 1) / 448
    assert np.all(np.abs(s - want) <= want * (2.0 ** -18 + 2.0 ** -24))
    err = np.abs(fp8.dequant(got.view(torch.uint8).cpu().numpy(), s) - h)
    assert np.all(err <= (2.0 ** -4 * np.abs(h) + 2.0 ** -10 * fp8.spread(s, K, 1)) * 1.01)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [1024, 1001])
def test_pack_many_rows_by_list(q4, K, silu):
    import torch

    rng = np.random.default_rng(K)
    x = torch.from_numpy(values(rng, 300, 2 * K if silu else K)).bfloat16().cuda()
    rows = rng.integers(0, 300, 3000).astype(np.int32)
    rows[rng.random(3000) < 0.1] = -1
    rows[[0, 2999]] = [300, -7]
    count = 2900
    got = torch.full((3000, K), 7.0, device="cuda").to(torch.float8_e4m3fn)
    scales = torch.full((3000, -(-K // 128)), -1.0, device="cuda")
    seven = got.view(torch.uint8)[0, 0].item()
    q4.fp8_pack(x, rows=torch.from_numpy(rows).cuda(), count=torch.tensor([count], dtype=torch.int32, device="cuda"), silu_mul=silu,
                codes=got, scales=scales)
    want, ws = q4.fp8_pack(x, silu_mul=silu)
    live = torch.from_numpy((rows >= 0) & (rows < 300) & (np.arange(3000) < count)).cuda()
    at = torch.from_numpy(rows).cuda().long()[live]
    assert torch.equal(got.view(torch.uint8)[live], want.view(torch.uint8)[at]) and torch.equal(scales[live], ws[at])
    assert bool((got.view(torch.uint8)[~live] == seven).all()) and bool((scales[~live] == -1).all())
