"""The feed-forward operators on the GPU where tests of single kernels' sizes do not reach: loops of
many steps and units in every variant that the rules choose, runs of one expert, extremes."""
import pytest

import ffn_ref as ref

torch = pytest.importorskip("torch")
awq = pytest.importorskip("bit_weight_only_w4a16_amd.awq")
int8 = pytest.importorskip("bit_weight_only_w4a16_amd.int8")
moe = pytest.importorskip("bit_weight_only_w4a16_amd.moe")

from test_gpu_ffn import BF16, DEV, F16, TYPES, choices, experts4, randn, same  # noqa: E402

pytestmark = pytest.mark.gpu


def test_moe_runs_of_one_expert_give_the_same_bits():
    """Experts of more than 32 tokens, whose units are cut at different places for their first and their
    second 32: which token is among which is the ids' alone. Experts 0 and 1 are the same and
    their shares cancel, so that an output is what the sums' order leaves."""
    tokens, hidden, ffn, experts = 64, 512, 1408, 4
    packed, _ = experts4(experts, hidden, ffn, 128, 0, seed=41)
    for p in packed:
        p[1] = p[0]
    x = randn(tokens, hidden, seed=42, gain=4.0)
    ids = torch.tensor([0, 1, -1, 4], dtype=torch.int32).repeat(tokens, 1)
    ids[::5, 2] = 2   # a run between, of few tokens
    ids[1::3, 3] = 3
    weights = torch.tensor([1e3, -1e3, 0.0, 0.0]).repeat(tokens, 1)
    ids, weights = ids.to(DEV), weights.to(DEV)
    first = moe.awq_moe(x, ids, weights, *packed, ffn)
    assert bool((first != 0).any())   # the sums' roundings show
    for i in range(40):
        randn(64, 64, seed=i) @ randn(64, 64, seed=i)   # other work between
        assert same(first, moe.awq_moe(x, ids, weights, *packed, ffn)), i


@pytest.mark.parametrize("width", [8, 4096])
@pytest.mark.parametrize("eps", [1e30, 1e36, 3e38, 3.4e38])
def test_rms_norm_large_eps_beside_squares_past_float32(eps, width):
    """Rows whose squares' sum passes float32 are summed scaled down, and eps counts as much as it does
    in other rows; the mean and eps may each be in range and their sum not."""
    x = randn(4, width, seed=51, dtype=BF16) * torch.tensor([[59], [61], [62], [90]], device=DEV).exp2().to(BF16)
    w = randn(width, seed=52, dtype=BF16)
    _, v, off = ref.norm(x, w, eps)
    got = int8.awq_rms_norm(x, w, eps, i8=True)
    ref.check(got.y, v, off + ref.U[BF16] * v.abs() + ref.TINY[BF16])
    ref.check_rows8(got.q, got.scale, v, off)


@pytest.mark.parametrize("width", [512, 4104])
def test_rms_norm_small_values_beside_one_past_float32(width):
    """A value whose square passes float32 does not cost the small ones of its row their bits, which a
    large weight brings back."""
    x = randn(2, width, seed=53, dtype=BF16) * 2.0 ** -66
    x[0, 7], x[1, 11], x[1, 12] = 2.0 ** 64, -2.0 ** 66, 2.0 ** 63
    w = randn(width, seed=54, dtype=BF16) * 2.0 ** 20
    _, v, off = ref.norm(x, w, 1e-5)
    ref.check(int8.awq_rms_norm(x, w).y, v, off + ref.U[BF16] * v.abs() + ref.TINY[BF16])


def moe_weights(hidden=128, ffn=256, experts=4):
    return [randn(experts, *shape, seed=91 + i, gain=0.1)
            for i, shape in enumerate([(hidden,), (ffn, hidden), (ffn, hidden), (hidden, ffn)])]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize,scale", [(True, 1.0), (False, 1.0), (False, 2.5), (True, 0.5)])
def test_moe_layer_reaches_the_routers_forms(score, renormalize, scale):
    layer = moe.MoeLayer.from_weights(*moe_weights(), 2, score=score, renormalize=renormalize, scale=scale)
    x, r = randn(70, 128, seed=95), randn(70, 128, seed=96)
    ids, weights = moe.awq_moe_route(x, layer.router, 2, score=score, renormalize=renormalize, scale=scale)
    y = layer(x, r)
    for part in (slice(0, 64), slice(64, 70)):
        assert same(y[part], moe.awq_moe(x[part], ids[part], weights[part], layer.gate, layer.up, layer.down, 256,
                                         residual=r[part]))


@pytest.mark.parametrize("each", [False, True], ids=["one scale", "a scale for each expert"])
def test_moe_layer_folds_channel_scales(each):
    """The scales that x and the intermediate are divided by are in the weights: stacks packed by hand
    have the same bits, and the layer is the product of what they stand for."""
    router, gate, up, down = moe_weights(hidden=256)
    scale = lambda width, at: awq.awq_channel_scale(  # noqa: E731
        randn(32, width, seed=at) * (1.0 + 7.0 * (torch.arange(width, device=DEV) % 16 == 3)).half())
    pairs = [[scale(width, 10 * at + e) for e in range(4)] for at, width in enumerate((256, 256))]
    (s_in, inv_in), (s_down, inv_down) = (
        [torch.stack(t) for t in zip(*p)] if each else list(p[0]) for p in pairs)
    layer = moe.MoeLayer.from_weights(router, gate, up, down, 2, s_in=s_in, s_down=s_down, inv_in=inv_in,
                                      inv_down=inv_down)
    assert layer.inv_in is inv_in and layer.inv_down is inv_down
    for packed, w, s in ((layer.gate, gate, s_in), (layer.up, up, s_in), (layer.down, down, s_down)):
        for e in range(4):
            hand = awq.awq_repack(*awq.awq_pack(w[e], s[e] if each else s), *w.shape[1:])
            assert same(packed[e], hand)
    x = randn(9, 256, seed=97)
    ids, weights = moe.awq_moe_route(x, router, 2)
    dense = [torch.stack([awq.awq_dequant(p, None, None, awq.LAYOUT_GFX950, *w.shape[1:]) for p in packed])
             for packed, w in ((layer.gate, gate), (layer.up, up), (layer.down, down))]
    want, bound = ref.moe(x, ids, weights, *dense, inv_in=inv_in, inv_down=inv_down)
    ref.check(layer(x), want, bound)


# ------------------------------------------------------------ tiles of the 8-bit product

# a product for each kernel of tiles that the rule chooses, alone and with the channels split
# (test_ffn_choice.py holds that it is so): more steps than the loop has in a turn, not a multiple of
# them, ragged in every direction
TILES = {  # (tile, teams, split): M, N, K
    ("64x64", 1, False): (639, 3248, 1776), ("64x64", 1, True): (66, 2296, 2864),
    ("64x64", 2, False): (193, 1048, 3152), ("64x64", 2, True): (68, 1632, 12512),
    ("64x128", 1, False): (69, 8424, 1696), ("64x128", 1, True): (65, 2728, 7456),
    ("128x128", 1, False): (134, 11336, 1568), ("128x128", 1, True): (65, 8792, 4752),
    ("128x256", 1, False): (279, 13160, 1616), ("128x256", 1, True): (69, 11024, 11440),
}
EACH_TILE = pytest.mark.parametrize("kind", TILES, ids=lambda k: f"{k[0]}_{k[1]}_{'split' if k[2] else 'whole'}")


def codes(*shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)


def layer_of(w, s_w):
    """w int8 [N, K] and s_w [N] in the layout of awq_pack_i8."""
    n, k = w.shape
    rows, cols = -(-n // 16) * 16, -(-k // 64) * 64
    full = torch.zeros(rows, cols, dtype=torch.int8, device=DEV)
    full[:n, :k] = w
    units = full.view(rows // 16, 16, cols // 64, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1)
    scales = torch.zeros(rows, device=DEV)
    scales[:n] = s_w
    raw = torch.cat([units.view(torch.uint8), scales.view(torch.uint8)])
    return torch.nn.functional.pad(raw, (0, -raw.numel() % 256))


def product_of(kind, dtype):
    m, n, k = TILES[kind]
    assert (int8.awq_gemm_i8_workspace_bytes(m, n, k) > 0) == kind[2]
    g = torch.Generator().manual_seed(n)
    q, w = codes(m, k, seed=m), codes(n, k, seed=k)
    scale = ((0.5 + torch.rand(m, generator=g)) / 1024).to(DEV)
    s_w = ((0.5 + torch.rand(n, generator=g)) / (5.0 * k ** 0.5)).to(DEV)
    operands = dict(bias=randn(n, seed=1, dtype=dtype), mul=randn(m, n, seed=2, dtype=dtype),
                    residual=randn(m, n, seed=3, dtype=dtype))
    return (m, n, k), q, scale, w, s_w, layer_of(w, s_w), operands


@TYPES
@EACH_TILE
def test_gemm_i8_every_output_of_each_tile(kind, dtype):
    (m, n, k), q, scale, w, s_w, packed, operands = product_of(kind, dtype)
    sums = torch.mm(q.double(), w.double().t().contiguous())   # whole numbers, exact
    v = (sums * scale.double()[:, None] * s_w.double()).cpu()
    for act, names in (("none", ()), ("gelu", ("bias", "mul", "residual")), ("silu", ("mul",)), ("relu", ("bias",)),
                       ("gelu_tanh", ("residual",))):
        some = {name: operands[name] for name in names}
        y = int8.awq_gemm_i8(q, scale, packed, n, k, act=act, dtype=dtype, **some)
        want, bound = ref.tail(v, dtype, act, some.get("bias"), some.get("mul"), some.get("residual"), 4 * ref.E * v.abs())
        ref.check(y, want, bound, f"{m}x{n}x{k} {act}")


@TYPES
@EACH_TILE
def test_gemm_i8_strides_in_place_and_neighbours_of_each_tile(kind, dtype):
    (m, n, k), q, scale, _, _, packed, operands = product_of(kind, dtype)
    r = operands["mul"]
    wide = codes(m, k + 80, seed=9)
    wide[:, 32:32 + k] = q
    # nothing past the output's end is written, and what lies between the rows of codes is not used
    buf = torch.full((m * n + 8192,), 7.0, dtype=dtype, device=DEV)
    want = int8.awq_gemm_i8(q, scale, packed, n, k, bias=operands["bias"], residual=r, dtype=dtype,
                            y=buf[4096:4096 + m * n].view(m, n)).clone()
    assert bool((buf[:4096] == 7).all()) and bool((buf[4096 + m * n:] == 7).all())
    got = int8.awq_gemm_i8(wide[:, 32:32 + k], scale, packed, n, k, bias=operands["bias"], residual=r, dtype=dtype)
    assert same(got, want)
    inside = r.clone()
    int8.awq_gemm_i8(q, scale, packed, n, k, bias=operands["bias"], residual=inside, y=inside, dtype=dtype)
    assert same(inside, want)
    gated = int8.awq_gemm_i8(q, scale, packed, n, k, act="silu", mul=r, dtype=dtype)
    inside = r.clone()
    int8.awq_gemm_i8(q, scale, packed, n, k, act="silu", mul=inside, y=inside, dtype=dtype)
    assert same(inside, gated)


# ----------------------------------------------------------------- loops of the experts' launches

def moe_by_expert(x, ids, weights, gate, up, down, act, inv_in=None, inv_down=None, residual=None):
    """ffn_ref.moe, all tokens of an expert at a time."""
    u, tiny, big_e = ref.U[F16], ref.TINY[F16], ref.E
    (tokens, hidden), ffn = x.shape, down.shape[2]
    y = torch.zeros(tokens, hidden, dtype=torch.float64)
    err, big = torch.zeros_like(y), torch.zeros_like(y)
    share = ref.cpu64(weights)
    for e in range(gate.shape[0]):
        t, j = torch.nonzero(ids.cpu() == e, as_tuple=True)
        if not len(t):
            continue
        xs = ref.cpu64(x)[t]
        if inv_in is not None:
            xs = (xs * ref.cpu64(inv_in if inv_in.dim() == 1 else inv_in[e])).half().double()
        wg, wu, wd = (ref.cpu64(w[e]).t().contiguous() for w in (gate, up, down))
        g, v = xs @ wg, xs @ wu
        dg, dv = ((hidden + 64) * big_e * (xs.abs() @ w.abs()) for w in (wg, wu))
        a = ref.ACTS[act](g)
        da = 1.13 * dg + 2e-6 * g.abs()
        m, dm = a * v, da * v.abs() + (a.abs() + da) * dv
        if inv_down is not None:
            f = ref.cpu64(inv_down if inv_down.dim() == 1 else inv_down[e])
            m, dm = m * f, dm * f.abs()
        dm = dm + 4 * big_e * m.abs()
        r = m.half().double()
        dm = torch.where(dm > 0, dm + 2 * u * m.abs() + 2 * tiny, dm)
        wt = share[t, j][:, None]
        terms = r.abs() @ wd.abs()
        y.index_add_(0, t, wt * (r @ wd))
        err.index_add_(0, t, wt.abs() * (dm @ wd.abs() + (ffn + 64) * big_e * terms))
        big.index_add_(0, t, wt.abs() * terms)
    if residual is not None:
        y = y + ref.cpu64(residual)
    return y, err + 64 * big_e * big + (u + 2 * big_e) * y.abs() + tiny


# A wavefront of the first launch has a quarter of hidden / 128 units, and two tiles where ffn / 16
# times the experts that may be named is 512 or more; one of the second has a share of the runs' units
# (runs times ffn / 128), among 16 wavefronts for each of ceil(256 / (hidden / 32)) workgroups, at most
# 16. Here they have several, but for the last, and a run's units of one wavefront are several too.
@pytest.mark.parametrize("tokens,hidden,ffn,experts,k,group,fmt", [
    (5, 4096, 1408, 6, 2, 128, 0),    # two tiles, 8 units each; 32 wavefronts share 66 units of 6 runs
    (14, 1408, 1408, 8, 3, 64, 1),    # two tiles, 3 or 2 units; 96 wavefronts, 88 units
    (64, 1408, 2944, 6, 4, 128, 0),   # 32 rows at a time, experts of more than 32 tokens, two tiles
    (40, 8192, 640, 7, 2, 128, 1),    # one workgroup for 32 outputs: no sums are shared
    (3, 8320, 768, 5, 2, 32, 0),      # the same with up to 16 rows, hidden past 256 groups of outputs
    (20, 2048, 4224, 3, 2, 128, 0),   # 64 wavefronts, 99 units: runs cut anywhere
    (2, 128, 8448, 3, 2, 128, 0),     # one unit of hidden; 256 wavefronts, 198 units: some have none
])
def test_moe_loops(tokens, hidden, ffn, experts, k, group, fmt):
    packed, dense = experts4(experts, hidden, ffn, group, fmt, seed=tokens + 70)
    x, (ids, weights) = randn(tokens, hidden, seed=71), choices(tokens, k, experts, seed=72)
    ids[:, 0] = torch.where((ids == 0).any(1), ids[:, 0], 0)   # expert 0 has all tokens
    more = dict(inv_in=randn(hidden, seed=73).abs() + 0.25, inv_down=randn(experts, ffn, seed=74).abs() + 0.25,
                residual=randn(tokens, hidden, seed=75))
    for act, some in (("silu", {}), ("gelu", more)):
        y = moe.awq_moe(x, ids, weights, *packed, ffn, group, fmt, act=act, **some)
        want, bound = moe_by_expert(x, ids, weights, *dense, act=act, **some)
        ref.check(y, want, bound)
        assert same(y, moe.awq_moe(x, ids, weights, *packed, ffn, group, fmt, act=act, **some))


def test_moe_form_by_expert_is_the_other():
    packed, dense = experts4(5, 256, 384, 128, 0, seed=81)
    x, (ids, weights) = randn(9, 256, seed=82), choices(9, 3, 5, seed=83)
    a, b = ref.moe(x, ids, weights, *dense), moe_by_expert(x, ids, weights, *dense, act="silu")
    assert bool(((a[0] - b[0]).abs() <= 1e-9).all()) and bool(((a[1] - b[1]).abs() <= 1e-9).all())


def test_moe_token_whose_ids_are_all_outside():
    """It gets its residual, or zeros, whatever the ids and the weights are."""
    hidden, ffn, experts = 256, 384, 6
    packed, _ = experts4(experts, hidden, ffn, 128, 0, seed=61)
    x, r = randn(5, hidden, seed=62), randn(5, hidden, seed=63)
    ids, weights = choices(5, 4, experts, seed=64)
    ids[1] = torch.tensor([6, -5, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    ids[3] = -1
    weights[3] = float("nan")
    y = moe.awq_moe(x, ids, weights, *packed, ffn)
    for t in (1, 3):
        assert same(y[t], torch.zeros_like(y[t]))
    assert bool((y[[0, 2, 4]] != 0).any(1).all())
    y = moe.awq_moe(x, ids, weights, *packed, ffn, residual=r)
    for t in (1, 3):
        assert same(y[t], r[t])


# --------------------------------------------------------------- loops of the other kernels

# few rows, a workgroup's wavefronts with several turns of units each (one, two and four blocks of 16)
ROWS = [(5, 520, 7280), (14, 4232, 7280), (29, 4712, 4432), (34, 3240, 4304)]


@TYPES
@pytest.mark.parametrize("m,n,k", ROWS)
def test_gemm_i8_few_rows_of_many_channels(m, n, k, dtype):
    assert int8.awq_gemm_i8_workspace_bytes(m, n, k) == 0
    q, w, g = codes(m, k, seed=m), codes(n, k, seed=k), torch.Generator().manual_seed(n)
    scale, s_w = ((0.5 + torch.rand(s, generator=g)).to(DEV) / 1024 for s in (m, n))
    operands = dict(bias=randn(n, seed=1, dtype=dtype), mul=randn(m, n, seed=2, dtype=dtype),
                    residual=randn(m, n, seed=3, dtype=dtype))
    v = (torch.mm(q.double(), w.double().t().contiguous()) * scale.double()[:, None] * s_w.double()).cpu()
    y = int8.awq_gemm_i8(q, scale, layer_of(w, s_w), n, k, act="gelu", dtype=dtype, **operands)
    want, bound = ref.tail(v, dtype, "gelu", *operands.values(), 4 * ref.E * v.abs())
    ref.check(y, want, bound)


def test_gemm_i8_more_rows_than_a_launch_has():
    """65535 blocks of rows go in one launch of the kernel that takes so little work a row, the others in
    another."""
    m, n, k = 65535 * 64 + 134, 8, 16
    q, w = codes(m, k, seed=1), codes(n, k, seed=2)
    scale, s_w = torch.rand(m, device=DEV) / 64, torch.rand(n, device=DEV) / 64
    g = torch.Generator(device=DEV).manual_seed(3)
    mul, residual = (torch.randn(m, n, generator=g, device=DEV).half() for _ in range(2))
    y = int8.awq_gemm_i8(q, scale, layer_of(w, s_w), n, k, mul=mul, residual=residual)
    for part in (slice(0, 70), slice(65535 * 64 - 70, m)):
        want, bound = ref.gemm_i8(q[part], scale[part], w, s_w, F16, mul=mul[part], residual=residual[part])
        ref.check(y[part], want, bound)


@TYPES
@pytest.mark.parametrize("tokens,hidden,experts,k", [(70, 8200, 1024, 8), (16, 16392, 1000, 4), (517, 4104, 130, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_of_many_channels(dtype, tokens, hidden, experts, k, score):
    """Wavefronts that take several turns of the channels, with one tile of tokens and with two."""
    x = randn(tokens, hidden, seed=tokens, dtype=dtype)
    w = randn(experts, hidden, seed=experts, dtype=dtype, gain=2.0 * hidden ** -0.5)
    ids, weights = moe.awq_moe_route(x, w, k, score=score)
    want_ids, want = ref.route(x, w, k, score=score)
    assert torch.equal(ids.cpu(), want_ids)
    ref.check(weights, want, 2 * ref.E * want.abs() + 2.0 ** -149)


@pytest.mark.parametrize("width,first", [(8, 4 << 20), (1032, 1 << 20)])
def test_more_rows_than_a_launch_has(width, first):
    """Rows past the workgroups of a launch go in its workgroups' second turn."""
    tokens = first + 5
    g = torch.Generator(device=DEV).manual_seed(width)
    x = torch.randn(tokens, width, generator=g, device=DEV, dtype=F16)
    w = randn(width, seed=1)
    got = int8.awq_rms_norm(x, w, i8=True)
    q, s = int8.awq_quant_i8(x, w)
    for part in (slice(0, 9), slice(first - 3, tokens)):
        alone = int8.awq_rms_norm(x[part], w, i8=True)
        assert all(same(a[part], b) for a, b in zip(got[:3], alone[:3]))
        q1, s1 = int8.awq_quant_i8(x[part], w)
        assert same(q[part], q1) and same(s[part], s1)
        _, v, off = ref.norm(x[part], w, 1e-5)
        ref.check(alone.y, v, off + ref.U[F16] * v.abs() + ref.TINY[F16])


@pytest.mark.parametrize("m,n,k", [(3, 520, 1040), *TILES.values()], ids=lambda v: str(v))
def test_gemm_i8_of_rows_near_the_types_ends(m, n, k):
    """Rows whose scale times their sum passes float32 and whose result does not, next to small and to
    ordinary ones."""
    q, w = codes(m, k, seed=m), codes(n, k, seed=k)
    at = torch.arange(m, device=DEV) % 3
    scale = torch.tensor([2.0 ** 118, 2.0 ** -100, 2.0 ** -7], device=DEV)[at] * 1.25
    s_w = 2.0 ** -12 * (1.0 + torch.arange(n, device=DEV) % 5)
    y = int8.awq_gemm_i8(q, scale, layer_of(w, s_w), n, k, dtype=BF16)
    want = torch.mm(q.double(), w.double().t().contiguous()) * scale.double()[:, None] * s_w.double()
    most = torch.finfo(BF16).max
    over = want.abs() >= most * (1 - 2 * ref.U[BF16])
    assert float(over.double().mean()) < 0.5
    off = (ref.U[BF16] + 4 * ref.E) * want.abs() + ref.TINY[BF16]
    assert bool(((y.double() - want).abs() <= off)[~over].all())
