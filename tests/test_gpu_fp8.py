"""fp8_pack, fp8_pack_weights, fp8_gemm and fp8_gemm_grouped on the GPU against the oracle.

Packing is bit-exact. silu(gate) * up is computed in fp32 with __expf, whose error is at most
2 + 1.173 |gate| units in the last place, and four roundings of at most 2 units each: relative
2^-23 (10 + 1.173 |gate|), below 2^-18 for |gate| <= 16. A code is then off by at most half a
step: 2^-4 of the value, or 2^-10 of the scale below the normal range; the scale's own error
(2^-18 and one rounding) moves both by less than 1 %.

Products: within a block of 128 the products are exact and each of the at most 128 additions on
the tensor cores, and each of the promotions after it (one rounding of the product of the two
scales, one of the fma), is off by at most 2^-23 of the sum of the magnitudes; the partial sums
of a split K add at most 8 more. So |y - y64| <= 2^-23 (128 + 2 blocks + 8) sum |x w|, plus half a
step of y's type and, for fp16, half of its smallest subnormal.
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


def u8(t):
    import torch

    return t.view(torch.uint8).cpu().numpy()


def dt(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def values(rng, M, K, scale=1.0):
    x = rng.normal(0, 1, (M, K)) * scale
    x[:, ::13] *= 30
    x[rng.random((M, K)) < 0.05] = 0
    x[rng.random((M, K)) < 0.02] *= 1e-6
    return x.astype(np.float32)


# ---- packing ------------------------------------------------------------------------------
@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 127), (5, 128), (2, 129), (7, 136), (16, 4096), (33, 200), (1, 14336), (300, 4100),
                                 (301, 4104)])
def test_pack_rows(q4, x_type, M, K):
    import torch

    x = torch.from_numpy(values(np.random.default_rng(M * K), M, K)).to(dt(x_type))
    codes, scales = q4.fp8_pack(x.cuda())
    rc, rs = fp8.pack(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(u8(codes), rc)


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (127, 130), (300, 200), (256, 1024), (129, 4104)])
def test_pack_weights(q4, x_type, N, K):
    import torch

    x = torch.from_numpy(values(np.random.default_rng(N * K + 1), 2 * N, K, 0.02).reshape(2, N, K)).to(dt(x_type))
    codes, scales = q4.fp8_pack_weights(x.cuda())
    for e in range(2):
        rc, rs = fp8.pack(x[e].float().numpy(), 128)
        assert np.array_equal(scales[e].cpu().numpy(), rs)
        assert np.array_equal(u8(codes[e]), rc)


def test_pack_magnitudes(q4):
    # blocks whose scales run over the whole fp32 range, subnormal ones and zeros among them;
    # every quotient must be the IEEE one, also where scales are outside the fast division's range
    import torch

    rng = np.random.default_rng(5)
    x = rng.normal(0, 1, (278, 128)).astype(np.float64)
    x = np.ldexp(x, np.linspace(-148, 125, 278).astype(int)[:, None]).astype(np.float32)
    x[0] = 0
    x[1] = np.float32(1e-45)
    x[2, 0] = np.float32(3.4e38)
    for rows in (1, 128):
        codes, scales = (q4.fp8_pack if rows == 1 else q4.fp8_pack_weights)(torch.from_numpy(x).cuda())
        rc, rs = fp8.pack(x, rows)
        assert np.array_equal(scales.cpu().numpy(), rs)
        assert np.array_equal(u8(codes), rc)


def test_pack_ties(q4):
    # the block's largest value 448 makes the scale 1: every midpoint of the table is a tie
    import torch

    t = fp8.TABLE
    mid = ((t[1:] + t[:-1]) / 2).astype(np.float32)
    v = np.concatenate([mid, -mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9))])
    v = np.resize(v, (8, 127)).astype(np.float32)
    x = np.concatenate([np.full((8, 1), 448, np.float32), v], 1)
    codes, scales = q4.fp8_pack(torch.from_numpy(x).cuda())
    assert bool((scales == 1).all())
    assert np.array_equal(u8(codes), fp8.encode(x))


def test_pack_quotients_exactly(q4):
    # random significands against random scales: the reciprocal-and-residual quotient is IEEE's
    import torch

    rng = np.random.default_rng(9)
    bits = rng.integers(0, 1 << 23, (20000, 128), dtype=np.uint32) | (rng.integers(117, 137, (20000, 128), dtype=np.uint32) << 23)
    x = bits.view(np.float32)
    codes, scales = q4.fp8_pack(torch.from_numpy(x).cuda())
    rs = (x.max(1, keepdims=True) / np.float32(448)).astype(np.float32)
    assert np.array_equal(scales.cpu().numpy(), rs)
    q = (x / rs).astype(np.float32)
    assert torch.equal(codes.cpu().view(torch.uint8), torch.from_numpy(q).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(3, 128), (5, 100), (2, 1), (9, 1032), (40, 14336), (3, 333), (301, 4099)])
def test_pack_silu_mul(q4, x_type, M, K):
    import torch

    x = torch.from_numpy(np.clip(np.random.default_rng(K).normal(0, 3, (M, 2 * K)), -16, 16).astype(np.float32)).to(dt(x_type))
    codes, scales = q4.fp8_pack(x.cuda(), silu_mul=True)
    h = fp8.silu_mul(x.double().numpy())
    s = scales.cpu().numpy().astype(np.float64)
    want = np.stack([np.abs(p).max(1) for p in np.split(h, range(128, K, 128), axis=1)], 1) / 448
    assert np.all(np.abs(s - want) <= want * (2.0 ** -18 + 2.0 ** -24))
    err = np.abs(fp8.dequant(u8(codes), s) - h)
    assert np.all(err <= (2.0 ** -4 * np.abs(h) + 2.0 ** -10 * fp8.spread(s, K, 1)) * 1.01)


def test_pack_silu_far_gates(q4):
    import torch

    x = torch.zeros(1, 256)
    x[0, :128] = torch.linspace(-300, 300, 128)
    x[0, 128:] = 1
    codes, scales = q4.fp8_pack(x.cuda(), silu_mul=True)
    # below -88 the value is 0 instead of at most 88 exp(-88), nothing beside 300 / 448 x 2^-10
    h, s = fp8.silu_mul(x.double().numpy())[0], scales.cpu().numpy()
    assert np.all(np.abs(fp8.dequant(u8(codes), s)[0] - h) <= (2.0 ** -4 * np.abs(h) + 2.0 ** -10 * s[0, 0]) * 1.01)


@pytest.mark.parametrize("offset", [1, 2, 4])
def test_pack_unaligned(q4, offset):
    # x at an element offset, and codes at a byte offset: no 16-byte loads there
    import torch

    rng = np.random.default_rng(offset)
    for K in (256, 40):
        flat = torch.from_numpy(values(rng, 1, 6 * K + 8)[0]).to(torch.bfloat16).cuda()
        x = flat[offset:offset + 6 * K].view(6, K)
        cbuf = torch.zeros(6 * K + 8, dtype=torch.uint8, device="cuda")
        c = cbuf[offset:offset + 6 * K].view(6, K).view(torch.float8_e4m3fn)
        q4.fp8_pack(x, codes=c)
        rc, _ = fp8.pack(x.float().cpu().numpy())
        assert np.array_equal(u8(c), rc)
        assert int(cbuf[:offset].sum()) == 0 and int(cbuf[offset + 6 * K:].sum()) == 0
        q4.fp8_pack_weights(x, codes=c)
        rc, _ = fp8.pack(x.float().cpu().numpy(), 128)
        assert np.array_equal(u8(c), rc)
        assert int(cbuf[:offset].sum()) == 0 and int(cbuf[offset + 6 * K:].sum()) == 0


def test_pack_row_list_and_count(q4):
    import torch

    x = torch.from_numpy(values(np.random.default_rng(1), 10, 300)).cuda()
    rows = torch.tensor([9, 0, -1, 3, 3, 10, 2**31 - 1, 5], dtype=torch.int32, device="cuda")
    codes = torch.full((8, 300), 7.0, device="cuda").to(torch.float8_e4m3fn)
    before = u8(codes)[0, 0]
    scales = torch.full((8, 3), -1.0, device="cuda")
    q4.fp8_pack(x, rows=rows, codes=codes, scales=scales)
    rc, rs = fp8.pack(x.cpu().numpy())
    for i, r in enumerate(rows.tolist()):
        if 0 <= r < 10:
            assert np.array_equal(u8(codes[i]), rc[r]) and np.array_equal(scales[i].cpu().numpy(), rs[r])
        else:
            assert np.all(u8(codes[i]) == before) and bool((scales[i] == -1).all())
    for n in (0, 4, 8, 100, -1):
        count = torch.tensor([n], dtype=torch.int32, device="cuda")
        codes = torch.full((10, 300), 7.0, device="cuda").to(torch.float8_e4m3fn)
        q4.fp8_pack(x, count=count, codes=codes)
        live = min(max(n, 0), 10)
        assert np.array_equal(u8(codes)[:live], rc[:live]) and np.all(u8(codes)[live:] == before)


def test_pack_reports_nonfinite(q4):
    import torch

    for bad in (float("inf"), float("nan")):
        for f in (q4.fp8_pack, q4.fp8_pack_weights):
            x = torch.ones(4, 260, device="cuda")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            f(x, status=status)
            assert int(status.item()) == 0
            x[3, 259] = bad
            codes, _ = f(x, status=status)
            assert int(status.item()) == q4.STATUS_NONFINITE
            assert bool((codes[:, :256].float() == 448).all())  # the other blocks are whole


def test_pack_shapes(q4):
    import torch

    x = torch.randn(2, 3, 256, device="cuda")
    codes, scales = q4.fp8_pack(x)
    assert codes.shape == x.shape and scales.shape == (2, 3, 2)
    codes, scales = q4.fp8_pack(x[0, 0])
    assert codes.shape == (256,) and scales.shape == (2,)
    codes, scales = q4.fp8_pack(torch.empty(0, 256, device="cuda"))
    assert codes.shape == (0, 256) and scales.shape == (0, 2)


# ---- products -------------------------------------------------------------------------------
def problem(seed, M, N, K, E=None):
    """Codes and scales on the GPU of normal values, with a few far larger columns."""
    import torch

    rng = np.random.default_rng(seed)
    xc, xs = fp8.pack(values(rng, M, K))
    out = [xc, xs]
    if E is None:
        out += fp8.pack(values(rng, N, K, 0.02), 128)
    else:
        parts = [fp8.pack(values(rng, N, K, 0.02), 128) for _ in range(E)]
        out += [np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])]
    return out, [torch.from_numpy(a).cuda().view(torch.float8_e4m3fn) if a.dtype == np.uint8 else torch.from_numpy(a).cuda()
                 for a in out]


def limit(y64, mag, kb, y_type):
    import torch

    half = torch.finfo(dt(y_type)).eps / 2
    tiny = 2.0 ** -25 if y_type == "f16" else 2.0 ** -134
    return 2.0 ** -23 * (128 + 2 * kb + 8) * mag * (1 + half) + half * np.abs(y64) + tiny


def check(y, y64, mag, kb, y_type, what=""):
    err = np.abs(y.double().cpu().numpy() - y64)
    lim = limit(y64, mag, kb, y_type)
    assert np.all(err <= lim), f"{what}: worst {float((err / lim).max()):.3g} of the limit at {np.argwhere(~(err <= lim))[:4].tolist()}"


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 300])
@pytest.mark.parametrize("N,K,y_type", [(128, 128, "f32"), (1, 16, "f32"), (127, 112, "bf16"), (130, 144, "f16"), (300, 1040, "f32"),
                                        (384, 4096, "bf16")])
def test_gemm(q4, M, N, K, y_type):
    import torch

    (xc, xs, wc, ws), (x, xst, w, wst) = problem(M * N + K, M, N, K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = q4.fp8_gemm(x, xst, w, wst, out_dtype=dt(y_type), status=status)
    y64, mag = fp8.gemm(xc, xs, wc, ws)
    check(y, y64, mag, fp8.blocks(K), y_type, f"M{M} N{N} K{K}")
    assert int(status.item()) == 0


@pytest.mark.parametrize("M", [1, 40, 700])
def test_gemm_one_hot_is_exact(q4, M):
    # x = e_k with scale 1: y is the dequantized weight, one product: any mix-up of k or n shows
    import torch

    N, K = 260, 400
    (_, _, wc, ws), (_, _, w, wst) = problem(3, 1, N, K)
    ks = np.arange(M) * 7 % K
    xc = np.zeros((M, K), np.uint8)
    xc[np.arange(M), ks] = 0x38  # 1.0
    x = torch.from_numpy(xc).cuda().view(torch.float8_e4m3fn)
    y = q4.fp8_gemm(x, torch.ones(M, 4, device="cuda"), w, wst, out_dtype=torch.float32)
    want = (fp8.decode(wc).astype(np.float32) * fp8.spread(np.take(np.repeat(ws, 128, 0), np.arange(N), 0), K, 1))
    assert np.array_equal(y.cpu().numpy(), want[:, ks].T.astype(np.float32))


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 11008, 4096), (5, 4096, 11008), (333, 1000, 2048), (640, 2304, 1024)])
def test_gemm_sampled(q4, M, N, K):
    # larger products, sampled columns of y against 64 bits
    import torch

    g = torch.Generator(device="cuda").manual_seed(M + N)
    x, xs = q4.fp8_pack(torch.randn(M, K, device="cuda", generator=g))
    w, ws = q4.fp8_pack_weights(torch.randn(N, K, device="cuda", generator=g) * 0.02)
    y = q4.fp8_gemm(x, xs, w, ws, out_dtype=torch.float32)
    cols = np.unique(np.concatenate([np.arange(8), np.arange(N - 8, N), np.random.default_rng(M).integers(0, N, 120)]))
    a = fp8.dequant(u8(x), xs.cpu().numpy())
    wc, wsc = u8(w)[cols], ws.cpu().numpy()[cols // 128]
    b = fp8.decode(wc) * fp8.spread(wsc.astype(np.float64), K, 1)
    check(y[:, torch.from_numpy(cols).cuda()], a @ b.T, np.abs(a) @ np.abs(b).T, fp8.blocks(K), "f32")


@pytest.mark.parametrize("M", [1, 20, 200, 600])
def test_gemm_repeats_and_streams(q4, M):
    import torch

    _, (x, xs, w, ws) = problem(M, M, 500, 2048)
    y0 = q4.fp8_gemm(x, xs, w, ws)
    y1 = q4.fp8_gemm(x, xs, w, ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        y2 = q4.fp8_gemm(x, xs, w, ws)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(y0)
    with torch.cuda.graph(g):
        q4.fp8_gemm(x, xs, w, ws, out=out)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for y in (y1, y2, out):
        assert torch.equal(y0, y)


@pytest.mark.parametrize("M", [3, 90, 513])
def test_gemm_writes_its_rows_only(q4, M):
    import torch

    N, K = 201, 256
    (xc, xs, wc, ws), (x, xst, w, wst) = problem(8, M, N, K)
    buf = torch.full((M * N + 64,), 5.0, device="cuda", dtype=torch.bfloat16)
    y = buf[33:33 + M * N].view(M, N)  # an odd element offset
    q4.fp8_gemm(x, xst, w, wst, out=y)
    y64, mag = fp8.gemm(xc, xs, wc, ws)
    check(y, y64, mag, 2, "bf16")
    assert bool((buf[:33] == 5).all()) and bool((buf[33 + M * N:] == 5).all())


@pytest.mark.parametrize("M", [5, 100, 600])
def test_gemm_keeps_bad_rows_apart(q4, M):
    # a NaN code, and an infinite scale: their own rows of y and no other
    import torch

    (xc, xs, wc, ws), (x, xst, w, wst) = problem(4, M, 140, 256)
    x.view(torch.uint8)[2, 200] = 0x7F
    xst[4, 0] = float("inf")
    y = q4.fp8_gemm(x, xst, w, wst)
    assert bool(y[2].isnan().all()) and not bool(y[4].isfinite().any())
    keep = [m for m in range(M) if m not in (2, 4)]
    y64, mag = fp8.gemm(xc, xs, wc, ws)
    check(y[keep], y64[keep], mag[keep], 2, "bf16")


def test_gemm_shapes(q4):
    import torch

    _, (x, xs, w, ws) = problem(1, 6, 128, 256)
    y = q4.fp8_gemm(x.view(2, 3, 256), xs.view(2, 3, 2), w, ws)
    assert y.shape == (2, 3, 128)
    assert q4.fp8_gemm(x[:0], xs[:0], w, ws).shape == (0, 128)


def test_refusals(q4):
    import torch

    _, (x, xs, w, ws) = problem(1, 6, 128, 256)
    with pytest.raises(TypeError):
        q4.fp8_gemm(x.float(), xs, w, ws)
    with pytest.raises(TypeError):
        q4.fp8_gemm(x, xs, w, ws, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        q4.fp8_gemm(x, xs[:5], w, ws)
    with pytest.raises(ValueError):
        q4.fp8_gemm(x, xs, w, ws[:, :1].contiguous())
    with pytest.raises(ValueError):
        q4.fp8_gemm(x[:, :128], xs[:, :1].contiguous(), w[:, :128], ws)  # not contiguous
    with pytest.raises(ValueError):
        q4.fp8_gemm(x, xs, w, ws, out=torch.empty(6, 127, device="cuda"))
    with pytest.raises(TypeError):
        q4.fp8_gemm(x, xs.cpu(), w, ws)
    with pytest.raises(TypeError):
        q4.fp8_pack(torch.zeros(4, 128, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        q4.fp8_pack(torch.zeros(4, 129, device="cuda"), silu_mul=True)
    with pytest.raises(TypeError):
        q4.fp8_pack(torch.zeros(4, 128, device="cuda"), rows=torch.zeros(2, device="cuda", dtype=torch.int64))
    c, s = q4.fp8_pack(torch.ones(4, 24, device="cuda"))
    with pytest.raises(q4.Q4Error) as e:
        q4.fp8_gemm(c, s, c, s[:1].contiguous())
    assert e.value.code == q4.Q4_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        q4.fp8_gemm_grouped(x, xs, w[None], ws[None], torch.zeros(3, dtype=torch.int32, device="cuda"))


# ---- products by experts ------------------------------------------------------------------
def grouped_ref(p, offsets):
    xc, xs, wc, ws = p
    y, mag = np.full((len(xc), wc.shape[1]), np.nan), np.zeros((len(xc), wc.shape[1]))
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if b > a:
            y[a:b], mag[a:b] = fp8.gemm(xc[a:b], xs[a:b], wc[e], ws[e])
    return y, mag


@pytest.mark.parametrize("counts,head,tail", [
    ([1], 0, 0), ([0, 1, 0], 0, 0), ([3, 0, 5, 1], 0, 0), ([17, 16, 0, 15], 0, 0), ([0, 0, 0], 0, 4), ([2, 200, 1, 0, 64], 0, 0),
    ([40, 130, 0, 7], 3, 9), ([1] * 40, 0, 2), ([300, 257, 0, 513], 0, 5), ([0] * 30 + [600] + [0] * 3, 0, 0), ([128, 256, 384], 0, 0),
])
@pytest.mark.parametrize("N,K,y_type", [(130, 144, "f32"), (256, 1024, "bf16"), (72, 512, "f16")])
def test_grouped(q4, counts, head, tail, N, K, y_type):
    import torch

    offsets = np.concatenate([[head], head + np.cumsum(counts)]).astype(np.int32)
    R, E = int(offsets[-1]) + tail, len(counts)
    p, (x, xs, w, ws) = problem(R + N, R, N, K, E)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((R, N), 3.0, device="cuda", dtype=dt(y_type))
    y = q4.fp8_gemm_grouped(x, xs, w, ws, torch.from_numpy(offsets).cuda(), out=out, status=status)
    assert int(status.item()) == 0
    y64, mag = grouped_ref(p, offsets)
    live = ~np.isnan(y64[:, 0])
    t = torch.from_numpy(live).cuda()
    assert bool((y[~t] == 3).all())
    if live.any():
        check(y[t], y64[live], mag[live], fp8.blocks(K), y_type, f"{counts}")


def test_grouped_many_experts(q4):
    import torch

    rng = np.random.default_rng(2)
    E, N, K = 1024, 40, 32
    counts = rng.integers(0, 4, E)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    p, (x, xs, w, ws) = problem(7, int(offsets[-1]), N, K, E)
    y = q4.fp8_gemm_grouped(x, xs, w, ws, torch.from_numpy(offsets).cuda(), out_dtype=torch.float32)
    y64, mag = grouped_ref(p, offsets)
    check(y, y64, mag, 1, "f32")


@pytest.mark.parametrize("R", [6, 700])
def test_grouped_takes_any_offsets(q4, R):
    # descending, negative or too large offsets: a running maximum held inside 0 .. R, so every
    # access stays inside; the rows that the running maximum gives are the ones written
    import torch

    p, (x, xs, w, ws) = problem(11, R, 128, 128, 4)
    for bad in ([0, R, 2, R, R], [-5, 3, 1, R + 100, 2**31 - 1], [R, 0, 0, 0, 0], [2**31 - 1, -2**31, 0, 3, R]):
        held = np.maximum.accumulate(np.clip(bad, 0, R))
        y64, mag = grouped_ref(p, held)
        out = torch.full((R, 128), 3.0, device="cuda")
        q4.fp8_gemm_grouped(x, xs, w, ws, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out)
        live = ~np.isnan(y64[:, 0])
        t = torch.from_numpy(live).cuda()
        assert bool((out[~t] == 3).all())
        if live.any():
            check(out[t], y64[live], mag[live], 1, "f32")


def test_two_products_at_once(q4):
    # no workspace, nothing shared: calls on two streams and two captured graphs replayed together
    import torch

    p1 = problem(21, 9, 700, 2048)[1]
    p2 = problem(22, 260, 300, 2048)[1]
    want = [q4.fp8_gemm(*p1), q4.fp8_gemm(*p2)]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    graphs = []
    for p, o in zip((p1, p2), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q4.fp8_gemm(*p, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)


def test_offsets_beyond_32_bits(q4):
    # codes, and y, of more than 2^32 elements: the far rows are those of the near ones
    import torch

    x = torch.randn(7, 4096, device="cuda")
    R = 1 << 20 | 5
    rows = (torch.arange(R, device="cuda") % 7).int()
    codes, scales = q4.fp8_pack(x, rows=rows)
    near, near_s = q4.fp8_pack(x)
    assert codes.numel() > 1 << 32
    for i in (0, R // 2, R - 1):
        assert torch.equal(codes[i].view(torch.uint8), near[i % 7].view(torch.uint8)) and torch.equal(scales[i], near_s[i % 7])
    del codes, scales
    M, N, K = 70001, 65552, 16
    _, (xc, xs, w, ws) = problem(5, 64, 80, K)
    x = xc.view(torch.uint8).repeat(-(-M // 64), 1)[:M].contiguous().view(torch.float8_e4m3fn)
    w = w.view(torch.uint8).repeat(-(-N // 80), 1)[:N].contiguous().view(torch.float8_e4m3fn)
    xs = xs.repeat(-(-M // 64), 1)[:M].contiguous()
    ws = torch.ones(q4.fp8._blocks(N), 1, device="cuda")
    y = q4.fp8_gemm(x, xs, w, ws)
    assert y.numel() > 1 << 32
    near = q4.fp8_gemm(x[:64].contiguous(), xs[:64].contiguous(), w[:80].contiguous(), ws[:1].contiguous())
    for m in (0, 40000, M - 1):
        assert torch.equal(y[m, :80], near[m % 64]) and torch.equal(y[m, N - 32:], near[m % 64, (N - 32) % 80:][:32])


def test_static_weights_after_these_kernels(q4):
    # qpack, one of these kernels, then qgemm with its weights declared static: the promise (packed
    # before the kernel in between began) holds, because that kernel lets the next one come on only
    # when all before it is done
    import torch

    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn(8192, 8192, device="cuda", generator=g)
    small, x = torch.randn(4, 256, device="cuda", generator=g), torch.randn(1, 8192, device="cuda", generator=g)
    payload, scales = q4.qpack(w, 4, 128)
    want = q4.qgemm(x, payload, scales, 8192, 8192, 4, 128)
    c, s = q4.fp8_pack_weights(small)
    ids = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    between = [lambda: q4.fp8_pack(small), lambda: q4.fp8_pack_weights(small), lambda: q4.moe_sort(ids, 2),
               lambda: q4.moe_gather(small, ids[0]), lambda: q4.moe_combine(small, ids), lambda: q4.fp8_gemm(*q4.fp8_pack(small), c, s)]
    for f in between:
        for _ in range(3):
            payload.zero_()
            q4.qpack(w, 4, 128, payload=payload, scales=scales)
            f()
            y = q4.qgemm(x, payload, scales, 8192, 8192, 4, 128, weights_static=True)
            assert torch.equal(y, want)


@pytest.mark.parametrize("N,off", [(256, 0), (264, 0), (200, 0), (272, 8), (264, 3)])
@pytest.mark.parametrize("M", [1024, 1100])
def test_pairs_store_their_rows(q4, M, N, off):
    # experts of hundreds of rows (pairs of CTAs): full and partial groups of 32 rows, rows of whole
    # and of partial 16-byte units, y at an offset, and the rows around it as they were
    import torch

    K, E = 128, 2
    counts = [M - 513, 513]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    p, (x, xs, w, ws) = problem(M + N, M, N, K, E)
    for t in ("bf16", "f16", "f32"):
        buf = torch.full((M * N + 64,), 5.0, device="cuda", dtype=dt(t))
        y = buf[off:off + M * N].view(M, N)
        for _ in range(2):
            q4.fp8_gemm_grouped(x, xs, w, ws, torch.from_numpy(offsets).cuda(), out=y)
        y64, mag = grouped_ref(p, offsets)
        check(y, y64, mag, 1, t)
        assert bool((buf[:off] == 5).all()) and bool((buf[off + M * N:] == 5).all())
