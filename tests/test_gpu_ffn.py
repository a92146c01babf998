"""The feed-forward operators on the GPU against plain float64 forms (ffn_ref), at the sizes,
layouts and values where they can go wrong."""
import pytest

import ffn_ref as ref

torch = pytest.importorskip("torch")
awq = pytest.importorskip("bit_weight_only_w4a16_amd.awq")
int8 = pytest.importorskip("bit_weight_only_w4a16_amd.int8")
moe = pytest.importorskip("bit_weight_only_w4a16_amd.moe")

pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])


def randn(*shape, seed, dtype=F16, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (gain * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# --------------------------------------------------------------------------------- rows

# each kernel's widths: full, one run less, one run more
WIDTHS = [8, 64, 504, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 32768]


@TYPES
@pytest.mark.parametrize("width", WIDTHS)
def test_rms_norm(dtype, width):
    tokens = 5
    x = randn(tokens, width, seed=width, dtype=dtype, gain=3.0)
    r = randn(tokens, width, seed=width + 1, dtype=dtype, gain=2.0)
    w = randn(width, seed=width + 2, dtype=dtype)
    for residual in (None, r):
        for weight in (None, w):
            h, v, off = ref.norm(x, weight, 1e-5, residual)
            got = int8.awq_rms_norm(x, weight, 1e-5, residual, i8=True)
            ref.check(got.y, v, off + ref.U[dtype] * v.abs() + ref.TINY[dtype], f"{width}")
            ref.check_rows8(got.q, got.scale, v, off, f"{width}")
            assert (got.h is None) if residual is None else same(got.h.cpu(), h)
            y = int8.awq_rms_norm(x, weight, 1e-5, residual)
            assert y.q is None and y.scale is None and same(y.y, got.y)
            q = int8.awq_rms_norm(x, weight, 1e-5, residual, y16=False, i8=True)
            assert q.y is None and same(q.q, got.q) and same(q.scale, got.scale)


@TYPES
@pytest.mark.parametrize("tokens", [0, 1, 2, 3, 255, 1025])
def test_rms_norm_rows_are_each_their_own(dtype, tokens):
    for width in (128, 2048, 4096):
        x = randn(tokens, width, seed=tokens, dtype=dtype)
        w = randn(width, seed=1, dtype=dtype)
        all_rows = int8.awq_rms_norm(x, w, i8=True)
        assert all_rows.y.shape == x.shape and all_rows.scale.shape == (tokens,)
        for t in {0, tokens // 2, tokens - 1} if tokens else ():
            one = int8.awq_rms_norm(x[t:t + 1], w, i8=True)
            assert same(one.y[0], all_rows.y[t]) and same(one.q[0], all_rows.q[t])
            assert same(one.scale, all_rows.scale[t:t + 1])


@TYPES
@pytest.mark.parametrize("width", [8, 520, 2056, 4104, 14336, 32768])
def test_quant(dtype, width):
    x = randn(6, width, seed=width, dtype=dtype, gain=4.0)
    f = randn(width, seed=3, dtype=dtype)
    for inv in (None, f):
        v = ref.cpu64(x) if inv is None else ref.cpu64(x) * ref.cpu64(inv)
        q, s = int8.awq_quant_i8(x, inv)
        ref.check_rows8(q, s, v, 2 * ref.E * v.abs(), f"{width}")


@TYPES
def test_quant_at_halves(dtype):
    """Values that lie halfway between two codes: the quotient by the scale decides, to even where the
    scale is exact."""
    for top in (127.0, 254.0, 63.5):   # scales 1, 2 and 1/2, as float32's product with 1 / 127 gives them
        x = torch.zeros(2, 256, dtype=dtype)
        x[:, 0] = top
        step = torch.tensor(top) * (torch.tensor(1.0) / 127.0)
        x[0, 1:128] = (torch.arange(127) + 0.5).to(dtype) * (top / 127)
        x[1, 1:128] = -x[0, 1:128]
        q, s = int8.awq_quant_i8(x.to(DEV))
        assert bool((s.cpu() == step).all())
        want = torch.round(x.float() / step).clamp(-127, 127)
        assert torch.equal(q.cpu().float(), want)


@TYPES
def test_quant_of_short_fractions(dtype):
    """Values of few bits: every code is the float32 quotient by the stored scale, rounded."""
    gen = torch.Generator().manual_seed(5)
    x = (torch.randint(-96, 97, (300, 520), generator=gen) * 2.0 ** torch.randint(-6, 3, (300, 1), generator=gen)).to(dtype)
    q, s = int8.awq_quant_i8(x.to(DEV))
    want = torch.round(x.float() / s.cpu()[:, None]).clamp(-127, 127)
    assert torch.equal(q.cpu().float(), want)


def test_rms_norm_refuses():
    x = randn(2, 64, seed=1)
    for bad, kind in ((dict(y16=False), ValueError), (dict(h=x), ValueError), (dict(weight=x[0].float()), TypeError),
                      (dict(weight=x), ValueError), (dict(residual=x[:1]), ValueError), (dict(eps=0.0), awq.AwqError),
                      (dict(q=torch.empty(2, 64, dtype=torch.uint8, device=DEV)), TypeError),
                      (dict(y=torch.empty(64, 2, dtype=F16, device=DEV).t()), ValueError)):
        with pytest.raises(kind):
            int8.awq_rms_norm(x, **bad)
    with pytest.raises(awq.AwqError):
        int8.awq_rms_norm(randn(2, 60, seed=1))


@TYPES
def test_rows_with_strides_and_in_place(dtype):
    width = 2064
    wide = randn(7, 3 * width + 24, seed=5, dtype=dtype)
    x, r = wide[:, 8:8 + width], wide[:, width + 16:2 * width + 16]
    w = randn(width, seed=6, dtype=dtype)
    want = int8.awq_rms_norm(x.contiguous(), w, residual=r.contiguous(), i8=True)
    got = int8.awq_rms_norm(x, w, residual=r, i8=True)
    assert all(same(a, b) for a, b in zip(got, want))
    # outputs in strided buffers; what lies between their rows stays
    buf = torch.full((7, width + 40), 7.0, dtype=dtype, device=DEV)
    qbuf = torch.full((7, width + 56), 99, dtype=torch.int8, device=DEV)
    int8.awq_rms_norm(x, w, residual=r, y=buf[:, 16:16 + width], q=qbuf[:, 32:32 + width])
    assert same(buf[:, 16:16 + width], want.y) and same(qbuf[:, 32:32 + width], want.q)
    assert bool((buf[:, :16] == 7).all()) and bool((buf[:, 16 + width:] == 7).all())
    assert bool((qbuf[:, :32] == 99).all()) and bool((qbuf[:, 32 + width:] == 99).all())
    # h in place of the residual, y in place of x; and the other way round
    a, b = x.contiguous(), r.contiguous()
    int8.awq_rms_norm(a, w, residual=b, h=b, y=a)
    assert same(a, want.y) and same(b, want.h)
    a, b = x.contiguous(), r.contiguous()
    int8.awq_rms_norm(a, w, residual=b, h=a, y=b)
    assert same(b, want.y) and same(a, want.h)


@TYPES
def test_rows_that_are_not_ordinary(dtype):
    """Zeros, one value, infinities, NaN, the type's largest and smallest values."""
    width, big, small = 512, torch.finfo(dtype).max, torch.finfo(dtype).tiny
    x = torch.zeros(8, width, dtype=dtype)
    x[1, 77] = -3.0
    x[2, 3], x[3, 3], x[4] = float("inf"), float("nan"), big
    x[5] = small
    x[6, ::2], x[6, 1] = -big, 1.0
    x[7] = torch.linspace(-1, 1, width)
    x = x.to(DEV)
    got = int8.awq_rms_norm(x, i8=True)
    y, s, q = got.y.cpu(), got.scale.cpu(), got.q.cpu()
    assert bool((y[0] == 0).all()) and s[0] == 0 and bool((q[0] == 0).all())
    assert torch.isnan(y[2, 3]) and bool((y[2, 4:] == 0).all()) and bool(torch.isnan(y[3]).all())
    assert bool(torch.isnan(s[2:4]).all()) and bool((q[2:4] == 0).all())
    at = [1, 4, 5, 6, 7]
    _, v, off = ref.norm(x[at], None, 1e-5)
    ref.check(got.y[at], v, off + ref.U[dtype] * v.abs() + ref.TINY[dtype])
    keep = [i for i, t in enumerate(at) if float(v[i].abs().max()) > 1e-29]
    ref.check_rows8(got.q[[at[i] for i in keep]], got.scale[[at[i] for i in keep]], v[keep], off[keep])
    # a residual that cancels, and one that overflows the type
    r = int8.awq_rms_norm(x[4:8], residual=-x[4:8], i8=True)
    assert bool((r.h == 0).all()) and bool((r.y == 0).all()) and bool((r.scale == 0).all())
    r = int8.awq_rms_norm(x[4:5], residual=x[4:5], i8=True)
    assert bool(torch.isinf(r.h).all()) and bool(torch.isnan(r.y).all()) and bool(torch.isnan(r.scale).all())
    # weights times values past float32 (bfloat16), and zeros
    w = torch.full((width,), big, dtype=dtype, device=DEV)
    v = ref.norm(x[7:8], w, 1e-5)
    got = int8.awq_rms_norm(x[7:8], w, i8=True)
    over = v[1].abs() >= big * (1 + ref.U[dtype])
    y = got.y.cpu()
    assert bool(torch.isinf(y[over]).all())
    if dtype == BF16:   # products of value and weight alone would pass float32
        x2 = randn(3, width, seed=4, dtype=dtype) * 2.0 ** torch.tensor([[40], [100], [-60]], device=DEV).to(dtype)
        w2 = randn(width, seed=5, dtype=dtype) * 2.0 ** 100
        _, v, off = ref.norm(x2, w2, 1e-5)
        got = int8.awq_rms_norm(x2, w2, i8=True)
        ref.check(got.y, v, off + ref.U[dtype] * v.abs() + ref.TINY[dtype])
        ref.check_rows8(got.q, got.scale, v, off)
    q, s = int8.awq_quant_i8(x)
    assert s.cpu()[0] == 0 and bool(torch.isnan(s.cpu()[2:4]).all()) and bool((q[[0, 2, 3]] == 0).all())
    v = ref.cpu64(x[[1, 4, 6, 7]])
    ref.check_rows8(q[[1, 4, 6, 7]], s[[1, 4, 6, 7]], v, 2 * ref.E * v.abs())


def test_rows_past_32_bit_offsets():
    width, stride = 1024, (1 << 31) - 8
    base = torch.empty(2 * stride + width, dtype=F16, device=DEV)
    x = base.as_strided((3, width), (stride, 1))
    rows = randn(3, width, seed=9)
    x.copy_(rows)
    assert same(int8.awq_rms_norm(x).y, int8.awq_rms_norm(rows).y)
    out = base.as_strided((3, width), (stride, 1))
    int8.awq_rms_norm(x, y=out)
    assert same(out, int8.awq_rms_norm(rows).y)


# ------------------------------------------------------------------------- 8-bit product

def layer8(n, k, seed, dtype=F16):
    w = randn(n, k, seed=seed, dtype=dtype, gain=0.05)
    packed = int8.awq_pack_i8(w)
    return packed, *ref.unpack_i8(packed, n, k)


@TYPES
@pytest.mark.parametrize("n,k", [(8, 16), (16, 64), (24, 80), (40, 1040), (264, 4096)])
def test_pack(dtype, n, k):
    w = randn(n, k, seed=n, dtype=dtype)
    w[1] = 0.0
    w[n - 1, 3] = float("nan")
    s_c = randn(k, seed=k, dtype=dtype).abs() + 0.5
    for fold in (None, s_c):
        packed = int8.awq_pack_i8(w, fold)
        assert packed.numel() == int8.awq_packed_i8_bytes(n, k)
        q, s = ref.unpack_i8(packed, n, k)
        v = ref.cpu64(w) if fold is None else ref.cpu64(w) * ref.cpu64(fold)
        assert s[1] == 0 and bool((q[1] == 0).all()) and bool(torch.isnan(s[n - 1])) and bool((q[n - 1] == 0).all())
        at = [i for i in range(n - 1) if i != 1]
        ref.check_rows8(q[at], s[at], v[at], 2 * ref.E * v[at].abs())
        # rows and channels of the padding are zeros
        units, tiles = -(-k // 64), -(-n // 16)
        codes = packed.cpu()[:tiles * units * 1024].view(torch.int8)
        assert int((codes != 0).sum()) == int((q != 0).sum())


# M, N, K: each kernel's sizes and their neighbours, ragged in every direction
PRODUCTS8 = [
    (1, 8, 16), (1, 4096, 4096), (2, 40, 80), (3, 264, 14336), (15, 136, 1024), (16, 4104, 640), (17, 520, 2064),
    (32, 72, 4096), (33, 1032, 512), (63, 2056, 1024), (64, 4096, 272), (65, 200, 4096), (100, 136, 11008),
    (127, 776, 2048), (128, 1024, 1024), (129, 1544, 528), (255, 264, 8192), (256, 4096, 256), (257, 520, 1040),
    (333, 4096, 2064), (511, 2056, 128), (700, 8, 64), (1000, 1000, 1008), (2049, 512, 400), (300, 14336, 144),
]


@TYPES
@pytest.mark.parametrize("m,n,k", PRODUCTS8)
@pytest.mark.parametrize("act,operands", [("none", ""), ("silu", "m"), ("gelu", "bmr"), ("relu", "b"), ("gelu_tanh", "r")])
def test_gemm_i8(dtype, m, n, k, act, operands):
    packed, w, s_w = layer8(n, k, seed=m + n, dtype=dtype)
    g = torch.Generator().manual_seed(k)
    q = torch.randint(-128, 128, (m, k), generator=g).to(torch.int8).to(DEV)
    scale = (0.5 + torch.rand(m, generator=g)).to(DEV) * 0.01
    bias = randn(n, seed=1, dtype=dtype) if "b" in operands else None
    mul = randn(m, n, seed=2, dtype=dtype) if "m" in operands else None
    residual = randn(m, n, seed=3, dtype=dtype) if "r" in operands else None
    y = int8.awq_gemm_i8(q, scale, packed, n, k, bias=bias, act=act, mul=mul, residual=residual, dtype=dtype)
    assert y.dtype == dtype and y.shape == (m, n)
    rows = torch.unique(torch.tensor([0, 1, m // 2, m - 2, m - 1]).clamp(0, m - 1))
    cols = torch.unique(torch.cat([torch.arange(0, min(n, 40)), torch.arange(n - 40, n)]).clamp_min(0))
    pick = lambda t: None if t is None else t[rows][:, cols]  # noqa: E731
    want, bound = ref.gemm_i8(q[rows], scale[rows], w[cols], s_w[cols], dtype, act, None if bias is None else bias[cols],
                              pick(mul), pick(residual))
    ref.check(y[rows][:, cols], want, bound, f"{m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (64, 520, 1040), (300, 1032, 4096), (700, 2048, 11008)])
def test_gemm_i8_every_output(m, n, k):
    """All outputs against the exact integers, computed on the device in float64."""
    packed, w, s_w = layer8(n, k, seed=k)
    q = torch.randint(-127, 128, (m, k), generator=torch.Generator().manual_seed(1)).to(torch.int8).to(DEV)
    one = torch.ones(m, device=DEV)
    y = int8.awq_gemm_i8(q, one, packed, n, k, dtype=BF16)
    want = (q.double() @ w.to(DEV).double().t().contiguous()) * s_w.to(DEV).double()
    assert bool(((y.double() - want).abs() <= (ref.U[BF16] + 4 * ref.E) * want.abs()).all())


def test_gemm_i8_largest_sums():
    """K at its limit with codes of -127 and -128: the sums come to 0.992 of 2^31."""
    k, n = 131056, 16
    packed = int8.awq_pack_i8(torch.full((n, k), -1.0, dtype=F16, device=DEV))
    _, s_w = ref.unpack_i8(packed, n, k)
    q = torch.full((20, k), -128, dtype=torch.int8, device=DEV)
    for rows in (1, 20):
        y = int8.awq_gemm_i8(q[:rows], torch.full((rows,), 1e-6, device=DEV), packed, n, k, dtype=BF16)
        want = (127.0 * 128 * k * 1e-6 * s_w.double()).expand(rows, n)
        assert bool(((y.cpu().double() - want).abs() <= (ref.U[BF16] + 4 * ref.E) * want).all())


@TYPES
@pytest.mark.parametrize("m", [1, 40, 300])
def test_gemm_i8_strides_in_place_and_neighbours(dtype, m):
    n, k = 520, 1040
    packed, _, _ = layer8(n, k, seed=m, dtype=dtype)
    wide = torch.randint(-127, 128, (m, k + 48), generator=torch.Generator().manual_seed(2)).to(torch.int8).to(DEV)
    q, scale = wide[:, 16:16 + k], torch.full((m,), 0.01, device=DEV)
    r = randn(m, n, seed=7, dtype=dtype)
    want = int8.awq_gemm_i8(q.contiguous(), scale, packed, n, k, residual=r, dtype=dtype)
    assert same(int8.awq_gemm_i8(q, scale, packed, n, k, residual=r, dtype=dtype), want)
    inside = r.clone()
    int8.awq_gemm_i8(q, scale, packed, n, k, residual=inside, y=inside, dtype=dtype)
    assert same(inside, want)
    gated = int8.awq_gemm_i8(q, scale, packed, n, k, act="silu", mul=r, dtype=dtype)
    inside = r.clone()
    int8.awq_gemm_i8(q, scale, packed, n, k, act="silu", mul=inside, y=inside, dtype=dtype)
    assert same(inside, gated)
    # nothing past the output's end is written
    buf = torch.full((m * n + 4096,), 7.0, dtype=dtype, device=DEV)
    int8.awq_gemm_i8(q, scale, packed, n, k, residual=r, y=buf[:m * n].view(m, n), dtype=dtype)
    assert same(buf[:m * n].view(m, n), want) and bool((buf[m * n:] == 7).all())


def test_gemm_i8_rows_whose_scale_is_nan_or_zero():
    m, n, k = 40, 264, 512
    packed, _, _ = layer8(n, k, seed=3)
    x = randn(m, k, seed=4)
    x[3, 5], x[7] = float("inf"), 0.0
    q, s = int8.awq_quant_i8(x)
    y = int8.awq_gemm_i8(q, s, packed, n, k)
    assert bool(torch.isnan(y[3]).all()) and bool((y[7] == 0).all())
    others = [i for i in range(m) if i not in (3, 7)]
    assert bool(torch.isfinite(y[others]).all())


def test_gemm_i8_past_32_bit_outputs():
    m, n, k = 70000, 32768, 16
    packed, w, s_w = layer8(n, k, seed=2)
    q = torch.randint(-127, 128, (m, k), generator=torch.Generator().manual_seed(5)).to(torch.int8).to(DEV)
    scale = torch.full((m,), 0.01, device=DEV)
    y = int8.awq_gemm_i8(q, scale, packed, n, k)
    rows, cols = torch.tensor([0, 65535, 65536, m - 1]), torch.arange(n - 64, n)
    want, bound = ref.gemm_i8(q[rows], scale[rows], w[cols], s_w[cols], F16)
    ref.check(y[rows][:, cols], want, bound)


def test_int8_linear():
    w, x = randn(264, 512, seed=1, gain=0.05), randn(9, 512, seed=2)
    cal = randn(32, 512, seed=3)
    s_c, inv = awq.awq_channel_scale(cal)
    layer = int8.Int8Linear.from_weight(w, s_c, inv)
    q, s = int8.awq_quant_i8(x, inv)
    r = randn(9, 264, seed=4)
    assert same(layer(x, residual=r), int8.awq_gemm_i8(q, s, layer.packed, 264, 512, residual=r))
    assert same(layer(q, s, residual=r), layer(x, residual=r))
    # 8 bits each: the product is near the plain one (a step is 1/127 of a row's largest value, off by
    # up to half; 512 products' errors add up like their root)
    want = x.float() @ w.float().t()
    step = (x.float() * inv.float()).abs().amax(1) / 127
    wstep = (w.float() * s_c.float()).abs().amax(1) / 127
    noise = (step[:, None] * (w.float() * s_c.float()).norm(dim=1) + wstep * (x.float() * inv.float()).norm(dim=1)[:, None])
    assert bool(((layer(x).float() - want).abs() <= 0.5 * 6 * noise + 2e-3 * want.abs() + 2e-3).all())


# ------------------------------------------------------------------------------- router

@TYPES
@pytest.mark.parametrize("tokens,hidden,experts,k", [
    (1, 8, 1, 1), (1, 4096, 8, 2), (2, 64, 3, 3), (7, 1000, 17, 4), (16, 2048, 64, 8), (17, 512, 65, 8), (33, 4104, 60, 6),
    (5, 328, 256, 8), (3, 256, 257, 32), (40, 136, 1024, 32), (517, 256, 128, 8), (4, 4096, 16, 8), (4, 1024, 64, 32),
    (3, 24, 5, 2), (4, 5000, 13, 3), (1, 65536, 1, 1), (2, 520, 33, 6),
])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(dtype, tokens, hidden, experts, k, score):
    x = randn(tokens, hidden, seed=tokens, dtype=dtype)
    w = randn(experts, hidden, seed=experts, dtype=dtype, gain=2.0 * hidden ** -0.5)
    bias = (0.1 * torch.randn(experts, generator=torch.Generator().manual_seed(1))).to(DEV)
    for b, renormalize, scale in ((None, True, 1.0), (bias, False, 2.5)):
        ids, weights = moe.awq_moe_route(x, w, k, b, score=score, renormalize=renormalize, scale=scale)
        want_ids, want = ref.route(x, w, k, b, score, renormalize, scale)
        assert ids.dtype == torch.int32 and torch.equal(ids.cpu(), want_ids)
        # float64 to about 1e-15 of the largest terms, rounded once
        ref.check(weights, want, 2 * ref.E * want.abs() + 2.0 ** -149)


def test_route_ties_nan_and_infinities():
    hidden, experts = 64, 20
    w = randn(experts, hidden, seed=1)
    w[5], w[11], w[3] = w[17], w[17], w[17]
    x = randn(6, hidden, seed=2)
    x[1], x[2, 0], x[3, 0] = 0.0, float("nan"), 1.0
    w[:, 0] = 0.0
    ids, weights = moe.awq_moe_route(x, w, 4)
    assert ids[1].tolist() == [0, 1, 2, 3] and bool((weights[1] == 0.25).all())   # all equal: the lowest
    assert ids[2].tolist() == [0, 1, 2, 3] and bool(torch.isnan(weights[2]).all())   # valid, if meaningless
    assert torch.equal(ids.cpu()[[0, 3, 4, 5]], ref.route(x[[0, 3, 4, 5]], w, 4)[0])
    # one expert's logit NaN: behind all others, also behind -infinity
    bias = torch.zeros(experts, device=DEV)
    bias[2], bias[4] = float("nan"), float("-inf")
    ids, weights = moe.awq_moe_route(x[:1], w, experts, bias, score="sigmoid", renormalize=False)
    assert ids[0, -2:].tolist() == [4, 2] and sorted(ids[0].tolist()) == list(range(experts))
    assert bool(torch.isfinite(weights).all())
    # sigmoids that are all 0: weights 0, not NaN
    x0, w0 = torch.full((1, hidden), -200.0, dtype=F16, device=DEV), torch.full((4, hidden), 200.0, dtype=F16, device=DEV)
    ids, weights = moe.awq_moe_route(x0, w0, 2, score="sigmoid")
    assert ids.tolist() == [[0, 1]] and weights.tolist() == [[0.0, 0.0]]


def test_route_borders():
    """Two experts whose logits differ in float64 alone are told apart; float32 sums would not."""
    hidden = 4096
    x = torch.full((2, hidden), 100.0, dtype=F16, device=DEV)
    w = torch.full((3, hidden), 1.0, dtype=F16, device=DEV)
    w[2, 7], w[1, 7] = 1.0 + 2.0 ** -10, 1.0
    x[:, 7] = 2.0 ** -14
    ids, _ = moe.awq_moe_route(x, w, 3)
    assert ids.tolist() == [[2, 0, 1]] * 2


def test_route_strided_tokens_and_empty():
    wide = randn(9, 304, seed=3)
    x, w = wide[:, 16:272], randn(12, 256, seed=4)
    a, b = moe.awq_moe_route(x, w, 3), moe.awq_moe_route(x.contiguous(), w, 3)
    assert same(a[0], b[0]) and same(a[1], b[1])
    ids, weights = moe.awq_moe_route(x[:0], w, 3)
    assert ids.shape == (0, 3) and weights.shape == (0, 3)


# ------------------------------------------------------------------------------ experts

def stack4(experts, n, k, group, fmt, seed):
    packed, dense = [], []
    for e in range(experts):
        w = randn(n, k, seed=seed + e, gain=1.5 * k ** -0.5)
        p = awq.awq_repack(*awq.awq_pack(w, None, group, fmt), n, k, group, fmt)
        packed.append(p)
        dense.append(awq.awq_dequant(p, None, None, awq.LAYOUT_GFX950, n, k, group, fmt))
    return torch.stack(packed), torch.stack(dense)


def experts4(experts, hidden, ffn, group, fmt, seed):
    (g, gd), (u, ud) = stack4(experts, ffn, hidden, group, fmt, seed), stack4(experts, ffn, hidden, group, fmt, seed + 100)
    d, dd = stack4(experts, hidden, ffn, group, fmt, seed + 200)
    return (g, u, d), (gd, ud, dd)


def choices(tokens, k, experts, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(max(experts, k), generator=g)[:k] for _ in range(tokens)]) if tokens else torch.zeros(0, k)
    return ids.to(torch.int32).to(DEV), torch.rand(tokens, k, generator=g).to(DEV)


@pytest.mark.parametrize("tokens,hidden,ffn,experts,k,group,fmt", [
    (1, 128, 128, 1, 1, 128, 0), (1, 1024, 384, 8, 2, 128, 0), (2, 256, 1408, 5, 3, 64, 1), (5, 384, 256, 40, 6, 32, 0),
    (16, 512, 512, 4, 2, 128, 1), (17, 256, 384, 3, 3, 128, 0), (33, 640, 128, 2, 2, 64, 0), (64, 256, 256, 70, 8, 128, 0),
    (64, 128, 256, 1, 1, 128, 1), (9, 256, 640, 16, 4, 128, 0), (12, 128, 1152, 16, 6, 128, 1), (20, 128, 640, 16, 4, 64, 0),
    (40, 4096, 128, 2, 1, 128, 0), (16, 4224, 128, 2, 2, 128, 1), (3, 2048, 256, 6, 2, 256, 0),
])
@pytest.mark.parametrize("act,extra", [("silu", False), ("gelu", True)])
def test_moe(tokens, hidden, ffn, experts, k, group, fmt, act, extra):
    packed, dense = experts4(experts, hidden, ffn, group, fmt, seed=tokens)
    x = randn(tokens, hidden, seed=1)
    ids, weights = choices(tokens, k, experts, seed=2)
    more = {}
    if extra:
        more = dict(inv_in=randn(experts, hidden, seed=3).abs() + 0.25, inv_down=randn(ffn, seed=4).abs() + 0.25,
                    residual=randn(tokens, hidden, seed=5))
    y = moe.awq_moe(x, ids, weights, *packed, ffn, group, fmt, act=act, **more)
    want, bound = ref.moe(x, ids, weights, *dense, act=act, **more)
    ref.check(y, want, bound)
    assert same(y, moe.awq_moe(x, ids, weights, *packed, ffn, group, fmt, act=act, **more))   # the same bits


def test_moe_ids_of_every_kind():
    """Ids outside the experts, tokens without any, one expert named twice, one for all tokens."""
    hidden, ffn, experts = 256, 384, 6
    packed, dense = experts4(experts, hidden, ffn, 128, 0, seed=7)
    x, r = randn(20, hidden, seed=8), randn(20, hidden, seed=9)
    ids, weights = choices(20, 4, experts, seed=10)
    ids[0], ids[1] = -1, torch.tensor([6, -5, 2 ** 31 - 1, -2 ** 31])
    ids[2], ids[3] = 3, torch.tensor([5, 1, 5, -1])
    ids[4, 1:] = 7
    for residual in (None, r):
        y = moe.awq_moe(x, ids, weights, *packed, ffn, residual=residual)
        want, bound = ref.moe(x, ids, weights, *dense, residual=residual)
        ref.check(y, want, bound)
        assert same(y[0], torch.zeros_like(y[0]) if residual is None else r[0]) and same(y[1], y[1] if residual is None else r[1])
    nobody = torch.full_like(ids, experts)
    assert same(moe.awq_moe(x, nobody, weights, *packed, ffn, residual=r), r)
    assert bool((moe.awq_moe(x, nobody, weights, *packed, ffn) == 0).all())
    everybody = torch.zeros_like(ids)
    want, bound = ref.moe(x, everybody, weights, *dense)
    ref.check(moe.awq_moe(x, everybody, weights, *packed, ffn), want, bound)
    assert moe.awq_moe(x[:0], ids[:0], weights[:0], *packed, ffn).shape == (0, hidden)


def test_moe_with_the_most_of_everything():
    """64 tokens of 32 experts each out of 1024: more experts named than a wavefront has lanes."""
    some, dense = experts4(8, 128, 128, 128, 0, seed=31)
    which = torch.arange(1024, device=DEV) % 8
    packed = [p[which].contiguous() for p in some]
    x, (ids, weights) = randn(64, 128, seed=32), choices(64, 32, 1024, seed=33)
    y = moe.awq_moe(x, ids, weights, *packed, 128)
    want, bound = ref.moe(x, ids % 8, weights, *dense)
    ref.check(y, want, bound)
    assert same(y, moe.awq_moe(x, ids, weights, *packed, 128))


def test_moe_strides_in_place_and_what_is_not_finite():
    hidden, ffn, experts = 256, 256, 4
    packed, _ = experts4(experts, hidden, ffn, 128, 0, seed=11)
    wide = randn(6, 2 * hidden + 40, seed=12)
    x, r = wide[:, 8:8 + hidden], wide[:, hidden + 16:2 * hidden + 16]
    ids, weights = choices(6, 2, experts, seed=13)
    want = moe.awq_moe(x.contiguous(), ids, weights, *packed, ffn, residual=r.contiguous())
    assert same(moe.awq_moe(x, ids, weights, *packed, ffn, residual=r), want)
    for alias in (0, 1):
        a, b = x.contiguous(), r.contiguous()
        moe.awq_moe(a, ids, weights, *packed, ffn, residual=b, y=(a, b)[alias])
        assert same((a, b)[alias], want)
    buf = torch.full((7, hidden + 16), 7.0, dtype=F16, device=DEV)
    moe.awq_moe(x, ids, weights, *packed, ffn, residual=r, y=buf[:6, 8:8 + hidden])
    assert same(buf[:6, 8:8 + hidden], want)
    assert bool((buf[6] == 7).all()) and bool((buf[:, :8] == 7).all()) and bool((buf[:, 8 + hidden:] == 7).all())
    # one token that is not finite stays alone
    bad = x.contiguous()
    bad[2, 5], bad[4, 0] = float("nan"), float("inf")
    y = moe.awq_moe(bad, ids, weights, *packed, ffn, residual=r)
    keep = [0, 1, 3, 5]
    assert same(y[keep], want[keep]) and bool(torch.isnan(y[2]).all()) and not bool(torch.isfinite(y[4]).all())
    # weights of 0, and one that is NaN
    none = torch.zeros_like(weights)
    assert bool((moe.awq_moe(x, ids, none, *packed, ffn) == 0).all())
    none[1, 0] = float("nan")
    y = moe.awq_moe(x, ids, none, *packed, ffn)
    assert bool(torch.isnan(y[1]).all()) and bool((y[[0, 2, 3, 4, 5]] == 0).all())


def test_moe_refuses_wrong_stacks():
    packed, _ = experts4(2, 256, 256, 128, 0, seed=1)
    x, (ids, weights) = randn(2, 256, seed=1), choices(2, 1, 2, seed=1)
    for bad in (dict(ffn=384), dict(group=100), dict(fmt=1), dict(ffn=250)):
        with pytest.raises(ValueError):
            moe.awq_moe(x, ids, weights, *packed, **{"ffn": 256, **bad})
    with pytest.raises(TypeError):
        moe.awq_moe(x.bfloat16(), ids, weights, *packed, 256)
    with pytest.raises(TypeError):
        moe.awq_moe(x, ids.long(), weights, *packed, 256)
    with pytest.raises(ValueError):
        moe.awq_moe(x, ids[:1], weights, *packed, 256)
    with pytest.raises(awq.AwqError):
        moe.awq_moe(randn(65, 256, seed=1), *choices(65, 1, 2, seed=1), *packed, 256)


def test_moe_layer():
    g = [randn(4, 256, 128, seed=s, gain=0.1) for s in (1, 2)]
    layer = moe.MoeLayer.from_weights(randn(4, 128, seed=3), *g, randn(4, 128, 256, seed=4, gain=0.1), 2)
    x, r = randn(130, 128, seed=5), randn(130, 128, seed=6)
    y = layer(x, r)
    ids, weights = moe.awq_moe_route(x, layer.router, 2)
    for at in (0, 64, 128):
        part = slice(at, at + 64)
        assert same(y[part], moe.awq_moe(x[part], ids[part], weights[part], layer.gate, layer.up, layer.down, 256,
                                         residual=r[part]))


# ----------------------------------------------------------------------- streams, graphs

def feed_forward(x, h, state):
    """Norm, router and experts, then the norm in 8 bits and its product."""
    n = int8.awq_rms_norm(x, state["w"], residual=h)
    ids, weights = moe.awq_moe_route(n.y, state["router"], 2)
    y = moe.awq_moe(n.y, ids, weights, *state["experts"], 256, residual=n.h)
    q = int8.awq_rms_norm(y, state["w"], residual=n.h, y16=False, i8=True)
    return int8.awq_gemm_i8(q.q, q.scale, state["packed"], 1032, 512, act="silu")


def ffn_state():
    return dict(w=randn(512, seed=1), router=randn(6, 512, seed=2), experts=experts4(6, 512, 256, 128, 0, seed=3)[0],
                packed=layer8(1032, 512, seed=4)[0])


@pytest.mark.parametrize("tokens", [1, 20, 64])
def test_together_on_another_stream_and_replayed(tokens):
    state = ffn_state()
    sets = [(randn(tokens, 512, seed=10 + i), randn(tokens, 512, seed=20 + i)) for i in range(3)]
    want = [feed_forward(x, h, state) for x, h in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [feed_forward(x, h, state) for x, h in sets]
    torch.cuda.current_stream().wait_stream(side)
    assert all(same(a, b) for a, b in zip(got, want))
    x, h = (t.clone() for t in sets[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = feed_forward(x, h, state)
    for i in (0, 1, 2, 0, 1):
        x.copy_(sets[i][0])
        h.copy_(sets[i][1])
        graph.replay()
        feed_forward(*sets[2], state)   # eager work between the replays
        torch.cuda.synchronize()
        assert same(out, want[i])


def test_two_graphs_side_by_side():
    state = ffn_state()
    sets = [(randn(20, 512, seed=30 + i), randn(20, 512, seed=40 + i)) for i in range(2)]
    want = [feed_forward(x, h, state) for x, h in sets]
    graphs, outs = [], []
    for x, h in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(feed_forward(x, h, state))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, want))
