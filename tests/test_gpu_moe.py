"""moe_sort, moe_gather, moe_combine, its backward and Fp8Experts on the GPU against the oracle.

Sums of k terms in fp32 fma steps are off by at most k 2^-24 of the sum of the magnitudes, and
their rounding by half a step of the type; a product rounded once by half a step; a dot product
of D terms, in any order, by at most D 2^-24 of the sum of the magnitudes.
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


def half_step(name):
    import torch

    return torch.finfo(dt(name)).eps / 2


def choices(rng, T, k, E, dropped=0.1):
    ids = rng.integers(0, E, (T, k))
    ids[rng.random((T, k)) < dropped] = -1
    return ids


# ---- sort -----------------------------------------------------------------------------------
@pytest.mark.parametrize("bits", [32, 64])
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (3, 2, 8), (32, 8, 64), (33, 3, 7), (1023, 2, 1000), (1025, 2, 1024),
                                   (1500, 8, 256), (4096, 8, 64), (0, 2, 5)])
def test_sort(q4, bits, T, k, E):
    import torch

    rng = np.random.default_rng(T * k + E)
    ids = choices(rng, T, k, E)
    if T > 2:
        ids[1, 0], ids[2, 0] = E, -5  # out of range on both sides
    t = torch.from_numpy(ids).to(torch.int32 if bits == 32 else torch.int64).cuda()
    tokens, pos, offsets = q4.moe_sort(t, E)
    for got, want in zip((tokens, pos, offsets), fp8.sort(ids, E)):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), want)


def test_sort_extremes(q4):
    import torch

    # all choices of one expert, none at all, and 64-bit ids that are in range in their low half only
    for ids in (np.full((3000, 2), 5), np.full((50, 2), -1), np.full((9, 1), (1 << 32) + 1)):
        got = q4.moe_sort(torch.from_numpy(ids).cuda(), 8)
        for g, want in zip(got, fp8.sort(ids, 8)):
            assert np.array_equal(g.cpu().numpy(), want)


def test_sort_large(q4):
    import torch

    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, 200, (70001, 6), device="cuda", generator=g)
    tokens, pos, offsets = q4.moe_sort(ids, 200)
    order = torch.sort(ids.reshape(-1), stable=True).indices
    assert torch.equal(tokens.long(), order // 6)
    assert torch.equal(pos.reshape(-1)[order].long(), torch.arange(order.numel(), device="cuda"))
    assert torch.equal(offsets[1:].long(), torch.bincount(ids.reshape(-1), minlength=200).cumsum(0))


# ---- gather and combine -----------------------------------------------------------------------
ROWS = [("bf16", 1001), ("f16", 2057), ("f32", 1), ("f32", 4), ("f32", 1023), ("bf16", 7), ("bf16", 64), ("bf16", 4096), ("f16", 258), ("f16", 2056)]


@pytest.mark.parametrize("x_type,D", ROWS)
def test_gather(q4, x_type, D):
    import torch

    rng = np.random.default_rng(D)
    x = torch.randn(11, D, device="cuda").to(dt(x_type))
    tokens = rng.integers(0, 11, 40).astype(np.int32)
    tokens[[3, 20, 39]] = [-1, 11, 2**31 - 1]
    out = torch.full((40, D), 2.0, device="cuda", dtype=dt(x_type))
    y = q4.moe_gather(x, torch.from_numpy(tokens).cuda(), out=out)
    for i, t in enumerate(tokens):
        assert torch.equal(y[i], x[t] if 0 <= t < 11 else torch.full_like(x[0], 2.0))


@pytest.mark.parametrize("x_type,D", ROWS)
@pytest.mark.parametrize("k", [1, 2, 4, 5, 8, 11])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(q4, x_type, D, k, weighted):
    import torch

    rng = np.random.default_rng(D + k)
    T, R = 13, 60
    ys = torch.randn(R, D, device="cuda").to(dt(x_type))
    ys[R - 1] = float("nan")  # a row that no token takes
    pos = rng.integers(0, R - 1, (T, k)).astype(np.int32)
    pos[rng.random((T, k)) < 0.1] = -1
    pos[5] = -1  # a token without experts
    pos[6, 0] = R  # out of range adds nothing
    w = rng.random((T, k)).astype(np.float32)
    out = q4.moe_combine(ys, torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda() if weighted else None)
    y64, mag = fp8.combine(ys.double().cpu().numpy(), pos, w if weighted else None)
    h = half_step(x_type)
    lim = k * 2.0 ** -24 * mag * (1 + h) + h * np.abs(y64) + (2.0 ** -25 if x_type == "f16" else 0)
    assert np.all(np.abs(out.double().cpu().numpy() - y64) <= lim)
    assert bool((out[5] == 0).all())


@pytest.mark.parametrize("x_type,D", ROWS)
@pytest.mark.parametrize("T,k", [(1, 1), (9, 2), (6, 8), (5, 11)])
def test_combine_backward(q4, x_type, D, T, k):
    import torch

    rng = np.random.default_rng(D * k)
    E = 16
    ids = choices(rng, T, k, E)
    _, pos, _ = fp8.sort(ids, E)
    R = T * k
    ys, dout = (torch.randn(n, D, device="cuda").to(dt(x_type)) for n in (R, T))
    w = rng.random((T, k)).astype(np.float32)
    dys = torch.full((R, D), 2.0, device="cuda", dtype=dt(x_type))
    got, dw = q4.moe_combine_backward(dout, ys, torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda(), dys=dys)
    assert got is dys
    want = np.full((R, D), 2.0)
    y64, d64 = ys.double().cpu().numpy(), dout.double().cpu().numpy()
    dw64, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                want[pos[t, j]] = w[t, j] * d64[t]
                dw64[t, j] = d64[t] @ y64[pos[t, j]]
                mag[t, j] = np.abs(d64[t]) @ np.abs(y64[pos[t, j]])
    tiny = 2.0 ** -25 if x_type == "f16" else 0
    # the product itself is rounded to fp32 before it is rounded to the type
    assert np.all(np.abs(dys.double().cpu().numpy() - want) <= (half_step(x_type) + 2.0 ** -24) * np.abs(want) * 1.001 + tiny)
    assert np.all(np.abs(dw.double().cpu().numpy() - dw64) <= D * 2.0 ** -24 * mag)


def test_gradients_against_differences(q4):
    # loss = <c, combine(gather(x), w)> in fp32 values that make every step exact enough for a
    # central difference in 64 bits of the oracle's formula
    import torch

    rng = np.random.default_rng(4)
    T, k, E, D = 5, 3, 4, 6
    ids = choices(rng, T, k, E)
    tokens, pos, _ = q4.moe_sort(torch.from_numpy(ids).cuda(), E)
    x, c, w = rng.normal(0, 1, (T, D)), rng.normal(0, 1, (T, D)), rng.random((T, k))
    g = [torch.from_numpy(a.astype(np.float32)).cuda() for a in (x, c, w)]
    xs = q4.moe_gather(g[0], tokens, out=torch.zeros(T * k, D, device="cuda"))
    dxs, dw = q4.moe_combine_backward(g[1], xs, pos, g[2], dys=torch.zeros(T * k, D, device="cuda"))
    dx = q4.moe_combine(dxs, pos)
    p, tk = pos.cpu().numpy(), tokens.cpu().numpy()
    x, c, w = (a.double().cpu().numpy() for a in g)

    def loss(x, w):
        rows = np.where((tk >= 0)[:, None], x[np.maximum(tk, 0)], 0)
        return (c * fp8.combine(rows, p, w)[0]).sum()

    h = 1e-4  # the loss is linear in each entry, so a central difference has no error but rounding: below 1e-10
    for a, grad, which in ((x, dx, 0), (w, dw, 1)):
        for i in np.ndindex(a.shape):
            d = np.zeros_like(a)
            d[i] = h
            num = (loss(x + d, w) - loss(x - d, w) if which == 0 else loss(x, w + d) - loss(x, w - d)) / (2 * h)
            # k rounded products of w and c, or D products of c and x, at most 4 in magnitude here
            assert abs(float(grad[i]) - num) <= 2.0 ** -24 * (2 * k if which == 0 else D) * 16 + 1e-9


def test_unaligned_rows(q4):
    import torch

    for t, D in (("bf16", 64), ("f32", 16)):
        n = 6 * D
        for off in (0, 1):
            buf = torch.randn(n + 8, device="cuda").to(dt(t))
            x = buf[off:off + n].view(6, D)
            tokens = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
            obuf = torch.zeros(3 * D + 8, device="cuda", dtype=dt(t))
            o = obuf[off:off + 3 * D].view(3, D)
            assert torch.equal(q4.moe_gather(x, tokens, out=o), x[tokens.long()])
            q4.moe_combine(x, tokens.view(3, 1), out=o)
            assert torch.equal(o, x[tokens.long()])
            assert bool((obuf[:off] == 0).all()) and bool((obuf[off + 3 * D:] == 0).all())


def test_refusals(q4):
    import torch

    x = torch.zeros(4, 8, device="cuda")
    pos = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for bad, err in ((lambda: q4.moe_sort(pos.float(), 4), TypeError), (lambda: q4.moe_sort(pos, 0), ValueError),
                     (lambda: q4.moe_sort(pos[0], 4), ValueError), (lambda: q4.moe_gather(x.double(), pos[:, 0].contiguous()), TypeError),
                     (lambda: q4.moe_gather(x, pos), ValueError), (lambda: q4.moe_gather(x, pos[:, 0]), ValueError),
                     (lambda: q4.moe_gather(x, pos[0].long()), TypeError), (lambda: q4.moe_combine(x, pos, w[:3]), ValueError),
                     (lambda: q4.moe_combine(x, pos, w.double()), TypeError), (lambda: q4.moe_combine(x, pos.long(), w), TypeError),
                     (lambda: q4.moe_combine_backward(x[:3], x, pos, w), ValueError),
                     (lambda: q4.moe_combine_backward(x, x, pos, None), TypeError),
                     (lambda: q4.moe_combine_backward(x.half(), x, pos, w), TypeError)):
        with pytest.raises(err):
            bad()
    with pytest.raises(q4.Q4Error) as e:
        q4.moe_sort(pos, 1025)
    assert e.value.code == q4.Q4_ERR_UNSUPPORTED


# ---- the layer ----------------------------------------------------------------------------
def experts_ref(q4, layer, x, ids, w):
    """The layer in 64 bits from the same codes, and how far each rounding on the way may move it.

    Rounded on the way: x to codes (the oracle's are the same, bit for bit), h to x's type (bf16
    where that is fp16), the
    activation to codes, the answers to x's type, and the sum. Returns (out, the sum over the
    experts of the weighted answers' bounds)."""
    import torch

    u8 = lambda t: t.view(torch.uint8).cpu().numpy()  # noqa: E731
    xn = x.float().cpu().numpy()
    xc, xs = fp8.pack(xn)
    a = fp8.dequant(xc, xs)
    h_step = torch.finfo(x.dtype).eps / 2
    between = torch.finfo(torch.bfloat16).eps / 2 if x.dtype == torch.float16 else h_step  # of gate and up
    gu, gus, dn, dns = u8(layer.gate_up), layer.gate_up_scales.cpu().numpy(), u8(layer.down), layer.down_scales.cpu().numpy()
    out, bound = np.zeros((len(xn), layer.D)), np.zeros((len(xn), layer.D))
    for t in range(len(xn)):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < layer.E:
                continue
            b, d = fp8.dequant(gu[e], gus[e], 128), fp8.dequant(dn[e], dns[e], 128)
            h, hm = b @ a[t], np.abs(b) @ np.abs(a[t])
            dh = between * np.abs(h) + 2.0 ** -15 * hm  # rounding of h, and the fp32 sums (2^-23 x (128 + 2 x blocks + 8) < 2^-15)
            F = layer.F
            act = fp8.silu_mul(h[None])[0]
            g, u = h[:F], h[F:]
            # |silu'| <= 1.1, |silu(g)| <= |g|
            dact = 1.1 * dh[:F] * (np.abs(u) + dh[F:]) + np.abs(g) * dh[F:]
            mx = np.repeat([np.abs(p).max() for p in np.split(act, range(128, F, 128))], 128)[:F]
            dmx = np.repeat([p.max() for p in np.split(dact, range(128, F, 128))], 128)[:F]
            # half a step of a code: 2^-4 of the value or 2^-10 of the scale
            dact = dact + (2.0 ** -4 * (np.abs(act) + dact) + 2.0 ** -10 * (mx + dmx) / 448) * 1.01
            y = d @ act
            dy = np.abs(d) @ dact + 2.0 ** -15 * (np.abs(d) @ (np.abs(act) + dact))
            dy += h_step * (np.abs(y) + dy)
            out[t] += w[t, j] * y
            bound[t] += np.abs(w[t, j]) * dy
    bound += (h_step + 2.0 ** -20) * (np.abs(out) + bound)
    return out, bound


@pytest.mark.parametrize("T,k,E,D,F,x_type", [(1, 2, 8, 256, 192, "bf16"), (7, 2, 4, 144, 128, "f32"), (40, 4, 16, 256, 112, "bf16"),
                                              (150, 2, 3, 128, 272, "f16")])
def test_experts(q4, T, k, E, D, F, x_type):
    import torch

    rng = np.random.default_rng(T)
    layer = q4.Fp8Experts.pack(torch.from_numpy(rng.normal(0, D ** -0.5, (E, 2 * F, D)).astype(np.float32)).cuda(),
                               torch.from_numpy(rng.normal(0, F ** -0.5, (E, D, F)).astype(np.float32)).cuda())
    x = torch.from_numpy(rng.normal(0, 1, (T, D)).astype(np.float32)).to(dt(x_type)).cuda()
    ids = choices(rng, T, k, E)
    w = rng.random((T, k)).astype(np.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
    out = layer(*args, status=status)
    y64, bound = experts_ref(q4, layer, x, ids, w)
    assert np.all(np.abs(out.double().cpu().numpy() - y64) <= bound)
    # the bound is wide where codes are rounded; as a whole the layer is far nearer: the codes'
    # errors are independent, so their relative size is below one step (2^-4) over the layer
    assert np.linalg.norm(out.double().cpu().numpy() - y64) <= 2.0 ** -4 * np.linalg.norm(y64)
    assert int(status.item()) == 0
    # captured with other tokens in the same buffers: the routing is read on the device
    cap = tuple(t.clone() for t in args)
    layer(*cap)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = layer(*cap)
    cap[1].copy_(args[1].flip(0))
    cap[0].copy_(args[0].flip(0))
    cap[2].copy_(args[2].flip(0))
    g.replay()
    torch.cuda.synchronize()
    y64f = y64[::-1]
    assert np.linalg.norm(again.double().cpu().numpy() - y64f) <= 2.0 ** -4 * np.linalg.norm(y64f)


def test_experts_wide_values_in_fp16(q4):
    # gate and up beyond fp16's range between the products, answers inside it
    import torch

    layer = q4.Fp8Experts.pack(torch.full((1, 64, 64), 40.0, device="cuda"), torch.full((1, 64, 32), 2.0 ** -24, device="cuda"))
    x = torch.full((2, 64), 50.0, device="cuda", dtype=torch.float16)  # gate = up = 128000
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = layer(x, torch.zeros(2, 1, dtype=torch.int64, device="cuda"), torch.ones(2, 1, device="cuda"), status=status)
    want = 128000.0 ** 2 * 32 * 2.0 ** -24
    assert int(status.item()) == 0
    # three bf16 or fp16 roundings (gate, up, the answer); the codes are the blocks' largest values, 448
    assert bool(((out.double() - want).abs() <= want * (2 * 2.0 ** -8 + 2.0 ** -11) * 1.01).all())


def test_experts_refusals(q4):
    import torch

    layer = q4.Fp8Experts.pack(torch.randn(2, 64, 32, device="cuda"), torch.randn(2, 32, 32, device="cuda"))
    x = torch.randn(3, 32, device="cuda")
    ids, w = torch.zeros(3, 2, dtype=torch.int64, device="cuda"), torch.ones(3, 2, device="cuda")
    assert layer(x, ids, w).shape == (3, 32)
    assert layer(x[:0], ids[:0], w[:0]).shape == (0, 32)
    for bad in (lambda: layer(x[:, :16].contiguous(), ids, w), lambda: layer(x[:2], ids, w), lambda: layer(x, ids, w[:, :1].contiguous()),
                lambda: q4.Fp8Experts.pack(torch.randn(2, 40, 32, device="cuda"), torch.randn(2, 32, 20, device="cuda")),
                lambda: q4.Fp8Experts(layer.gate_up, layer.gate_up_scales[:1], layer.down, layer.down_scales)):
        with pytest.raises(ValueError):
            bad()


def test_offsets_beyond_32_bits(q4):
    import torch

    T, D, R = 5, 4096, 1 << 20 | 3
    x = torch.randn(T, D, device="cuda").bfloat16()
    tokens = (torch.arange(R, device="cuda") % T).int()
    xs = q4.moe_gather(x, tokens)
    assert xs.numel() > 1 << 32
    for i in (0, R // 2, R - 1):
        assert torch.equal(xs[i], x[i % T])
    pos = torch.tensor([[0, R - 1], [R - 1, R - 2]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25], [1.0, 2.0]], device="cuda")
    out = q4.moe_combine(xs, pos, w)
    want = (xs[pos.long()].double() * w[..., None].double()).sum(1)
    assert bool(((out.double() - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -20 * 8).all())
    del out
    dout = torch.randn(2, D, device="cuda").bfloat16()
    pos = torch.tensor([[0, R - 1], [R // 2, R - 2]], dtype=torch.int32, device="cuda")
    dys, dw = q4.moe_combine_backward(dout, xs, pos, w)
    for t in range(2):
        for j in range(2):
            p = int(pos[t, j])
            assert torch.equal(dys[p], (dout[t].float() * w[t, j]).bfloat16())
            ref = (dout[t].double() * xs[p].double()).sum()
            assert abs(float(dw[t, j]) - float(ref)) <= D * 2.0 ** -24 * float((dout[t].double() * xs[p].double()).abs().sum())


def test_experts_on_two_streams_and_graphs(q4):
    # nothing is shared between calls: two captured layers replayed together give what one gives
    import torch

    layer = q4.Fp8Experts.pack(torch.randn(4, 128, 64, device="cuda") / 8, torch.randn(4, 64, 64, device="cuda") / 8)
    args = [(torch.randn(n, 64, device="cuda"), torch.randint(-1, 4, (n, 2), device="cuda"), torch.rand(n, 2, device="cuda")) for n in (3, 300)]
    want = [layer(*a) for a in args]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(*a))
        graphs.append(g)
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_captured_fork_and_join(q4):
    # kernels launched to overlap the one before, captured where what is before them is a copy, a
    # join of two streams, or nothing
    import torch

    layer = q4.Fp8Experts.pack(torch.randn(4, 128, 64, device="cuda") / 8, torch.randn(4, 64, 64, device="cuda") / 8)
    x, ids, w = torch.randn(30, 64, device="cuda"), torch.randint(0, 4, (30, 2), device="cuda"), torch.rand(30, 2, device="cuda")
    xb = torch.empty_like(x)
    want = layer(x, ids, w), layer(x * 2, ids, w)
    pos = torch.arange(60, dtype=torch.int32, device="cuda").view(30, 2)
    both = q4.moe_combine(torch.stack([want[0], want[1]], 1).view(60, 64), pos)
    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            b = layer(x * 2, ids, w)
        xb.copy_(x)
        a = layer(xb, ids, w)
        c = torch.empty(30, 2, 64, device="cuda")
        c[:, 0] = a
        main.wait_stream(side)
        c[:, 1] = b
        out = q4.moe_combine(c.view(60, 64), pos)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q = q4.fp8_pack(out)
        p = q4.fp8_pack(out)
        main.wait_stream(side)
        t = q4.moe_sort(ids, 4)  # after a join, with nothing in between
    for _ in range(5):
        xb.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(out, both)
    assert torch.equal(p[0].view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(t[1], q4.moe_sort(ids, 4)[1])


def test_sorted_rows_both_ways(q4):
    # many rows are packed once and gathered, few are packed in sorted order: the same codes
    import torch

    g = torch.Generator(device="cuda").manual_seed(5)
    for T, k, D in ((4200, 8, 1024), (60, 8, 1024)):
        x = torch.randn(T, D, device="cuda", generator=g).bfloat16()
        ids = torch.randint(-1, 16, (T, k), device="cuda", generator=g)
        tokens, _, offsets = q4.moe_sort(ids, 16)
        n = int(offsets[-1])
        got, want = q4.Fp8Experts.sorted_rows(x, tokens), q4.fp8_pack(x, rows=tokens)
        assert torch.equal(got[0][:n].view(torch.uint8), want[0][:n].view(torch.uint8))
        assert torch.equal(got[1][:n], want[1][:n])
